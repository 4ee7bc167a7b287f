// attention_prompt.cuh -- causal grouped-query attention of prompts (many new
// tokens per sequence) over the paged 8-bit cache, on the 5th-generation tensor
// cores: tcgen05.mma kind::f16 with fp32 accumulators in tensor memory.
//
// Same formulas as attention_tokens.cuh.  Bound by the tensor cores and the
// exponentials: 4 D flops and one exp2 per visible (query head, token) pair.  As
// built, a block of 128 tokens takes a CTA 5200 cycles (2.66 us, from the times of 512
// new tokens behind 16, 32 and 64 k cached ones; 2.6 us with D = 64), its four products
// 2048 of them: softmax and products of an MMA tile take turns, since weights lie over
// their scores, and the two tiles hide each other only in part (tensor pipe 36 % busy,
// exponentials 38 %, half of the issue slots used).
//
// Query rows of a (sequence, kv head) are its new tokens times the query heads
// of the group (row = token * group + head).  An MMA tile holds as many whole
// tokens as fit its 128 rows, a row tile is two of them, A and B, so that one's
// softmax runs while the other's products do.  Tokens are taken in blocks of 128.
// One CTA per SM.  Where no tile is dearer than a CTA's even share of the work, the
// CTAs claim whole tiles, dearest first (k_attention_plan sorts them), each when its
// last copies of the tile before are under way.  Else (few rows, long contexts) the
// list of all (sequence, kv head, row tile, block that the tile sees), with two more
// units per tile for loading its queries and storing its rows, is cut into equal
// contiguous shares, and tiles that two or more CTAs share are joined by
// k_attention_prompt_join through the workspace, in the order of the CTAs.  (Equal
// shares always: 144 us for a 4096-token prompt, the parts of 147 shared tiles
// written and read again; now 128 us, 0.67 PFLOP/s of visible products.)  Which CTA
// takes a tile does not change its result.
//
// One CTA, 24 warps:
//   warps 0-7, 8-15 softmax of tile A, B: two threads per row, 64 tokens of a block
//                   each (more warps in flight than a thread per row with 128 scores
//                   in registers, which was bound by latency).  Weights go back over
//                   their scores in tensor memory as the A operand of the second
//                   product; sums are rescaled and finally read there
//   warps 16-19     widen the int8 codes, rows of tokens in the 128-byte-swizzled
//                   layout that serves K (bf16) as a K-major and V (fp16) as an
//                   MN-major B operand (a row of V is contiguous in the head
//                   dimension, the N of that product)
//   warp 20         TMA of the codes (a box per page); steps
//   warp 21         MMA issuer, owner of tensor memory
//   warp 22         queries, as they are (bf16), by TMA
//   warp 23         walks the unit list and hands out the tiles
// Codes are exact in bf16 and in fp16.  Weights are fp16 and carry v_step: its
// power of two goes on the codes (exact in fp16 down to 2^-24), the rest, in
// [1, 2), into the weight's exponent as its logarithm; the sums are in units of a
// power of two near the current pages' steps.
#pragma once

#include "attention_tokens.cuh"

namespace bitnet {

constexpr int AP_ROWS = 256;      // query rows per tile (two MMA tiles), some of them dead
constexpr int AP_BLOCK = 128;     // tokens per block
constexpr int AP_THREADS = 768;
constexpr int AP_RAW = 3;         // ring of int8 tiles
constexpr int AP_CONV = 3;        // ring of 16-bit tiles
constexpr int AP_STEPS = 4;       // ring of blocks' steps (see the producer)
constexpr int AP_OVER = 2;        // units that a tile costs besides its blocks
constexpr int AP_MIN_UNITS = 4;   // units worth a CTA of their own
constexpr int AP_SEGS = 4;        // ring of tiles handed out
constexpr int AP_CONV_WARP0 = 16, AP_TMA_WARP = 20, AP_MMA_WARP = 21, AP_Q_WARP = 22, AP_SCHED_WARP = 23;
constexpr int AP_SEG_READERS = 23; // warps that read every tile's description
constexpr float AP_LAZY = 8.0f;   // the reference of a row's exponents lags its maximum by up to 2^8

constexpr int AP_HDR = 6144;      // barriers, steps, tiles, maxima on their way
constexpr __host__ __device__ int ap_smem(int d)
{
    return AP_HDR + 2 * 128 * d * 2 + AP_CONV * AP_BLOCK * d * 2 + AP_RAW * AP_BLOCK * d + 1024;
}

// Tokens of one MMA tile.
constexpr __host__ __device__ int ap_tokens(int group) { return 128 / group; }

// Blocks that row tile qt of a sequence sees (new token i sees tokens 0 .. len - n + i).
BITNET_DEVINL int ap_blocks(const AttnSeq &s, int group, int qt)
{
    const int last = min(s.n, (qt + 1) * 2 * ap_tokens(group)) - 1;
    const int lim = s.len - s.n + last;
    return lim < 0 ? 0 : lim / AP_BLOCK + 1;
}

BITNET_DEVINL int ap_tiles(const AttnSeq &s, int group)
{
    const int t = 2 * ap_tokens(group);
    return (s.n + t - 1) / t;
}

// Units of a tile: its blocks, behind AP_OVER for loading its queries and storing its rows.
BITNET_DEVINL int ap_units(int blocks) { return blocks > 0 ? blocks + AP_OVER : 0; }

BITNET_DEVINL int64_t ap_active(int64_t units, int ctas)
{
    const int64_t want = (units + AP_MIN_UNITS - 1) / AP_MIN_UNITS;
    return want < ctas ? want : ctas;
}

// Calls f(b, sequence, tile, blocks) for every row tile of one kv head, spread over the
// CTA's threads: a thread per sequence where there are many, else a warp.
template <typename F>
BITNET_DEVINL void ap_for_tiles(const AttnArgs &a, F f)
{
    const bool many = a.bt.n_seqs >= 256;
    const int first = many ? threadIdx.x : threadIdx.x >> 5, step = many ? 1024 : 32;
    for (int b = first; b < a.bt.n_seqs; b += step) {
        const AttnSeq s = attn_seq(a, b);
        const int nt = ap_tiles(s, a.group);
        for (int t = many ? 0 : threadIdx.x & 31; t < nt; t += many ? 1 : 32) f(b, s, t, ap_blocks(s, a.group, t));
    }
}

// One CTA: first unit of every sequence, the choice between whole tiles and shares, the
// tiles in order of their cost, rows that see nothing.
template <int D>
__global__ void __launch_bounds__(1024) k_attention_plan(const AttnArgs a, int ctas)
{
    __shared__ int64_t s_sum[32];
    __shared__ int64_t s_carry;
    __shared__ int s_most, s_tiles, s_bin[1024], s_wsum[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int n_seqs = a.bt.n_seqs, hk = a.kv.hk;
    if (tid == 0) {
        a.base[0] = 0;
        s_carry = 0;
        s_most = 0;
        s_tiles = 0;
    }
    s_bin[tid] = 0;
    for (int k = tid; k < ctas; k += 1024) a.shared[k].nrow = 0;
    int64_t claimed = 0; // rows of this thread's sequences
    for (int b = tid; b < n_seqs; b += 1024) {
        a.base[b + 1] = 0;
        claimed += attn_seq(a, b).n;
    }
    const int in_warp = __reduce_add_sync(0xffffffffu, (int)min(claimed, int64_t(1) << 25)); // T is at most 2^24
    if (lane == 0) s_wsum[warp] = in_warp;
    __syncthreads();
    claimed = 0;
    for (int w = 0; w < 32; ++w) claimed += s_wsum[w];
    if (claimed > a.bt.T) {
        // Sequences that claim the same rows: their tiles may outnumber those that the workspace holds and
        // 32 bits count, so none is taken.
        if (tid == 0) {
            record_batch_error();
            *a.claim = {1, 0, 0};
        }
        return;
    }
    int most = 0, tiles = 0;
    ap_for_tiles(a, [&](int b, const AttnSeq &s, int t, int blocks) {
        atomicAdd(reinterpret_cast<unsigned long long *>(&a.base[b + 1]), (unsigned long long)ap_units(blocks) * hk);
        most = max(most, blocks);
        tiles += blocks > 0;
        if (blocks == 0) // rows in front of their sequence's first token
            for (int i = 2 * t * ap_tokens(a.group); i < min(s.n, 2 * (t + 1) * ap_tokens(a.group)); ++i)
                for (int x = 0; x < hk * a.group * (D / 8); ++x)
                    reinterpret_cast<uint4 *>(a.out + (int64_t)(s.q0 + i) * a.out_stride)[x] = make_uint4(0, 0, 0, 0);
    });
    most = __reduce_max_sync(0xffffffffu, most);
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    if (lane == 0) {
        atomicMax(&s_most, most);
        atomicAdd(&s_tiles, tiles);
    }
    __syncthreads();
    for (int b0 = 0; b0 < n_seqs; b0 += 1024) {
        const int b = b0 + tid;
        int64_t v = b < n_seqs ? a.base[b + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += up;
        }
        if (lane == 31) s_sum[warp] = v;
        __syncthreads();
        int64_t before = s_carry;
        for (int w = 0; w < warp; ++w) before += s_sum[w];
        if (b < n_seqs) a.base[b + 1] = before + v;
        __syncthreads();
        if (tid == 1023) s_carry = before + v;
        __syncthreads();
    }
    const int64_t total = s_carry;
    most = s_most;
    const bool whole = (int64_t)ap_units(most) * ctas <= total;
    if (tid == 0) {
        a.claim->whole = whole;
        a.claim->next = 0;
        a.claim->tiles = s_tiles * hk;
    }
    if (!whole) return;
    // sorted by cost into 1024 bins, dearest first; the order within one is of no account
    const float scale = 1023.0f / (float)most;
    auto bin = [&](int blocks) { return 1023 - min(1023, (int)((float)blocks * scale)); };
    ap_for_tiles(a, [&](int b, const AttnSeq &s, int t, int blocks) {
        if (blocks > 0) atomicAdd(&s_bin[bin(blocks)], hk);
    });
    __syncthreads();
    int v = s_bin[tid];
    const int mine = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
    }
    if (lane == 31) s_wsum[warp] = v;
    __syncthreads();
    int before = v - mine;
    for (int w = 0; w < warp; ++w) before += s_wsum[w];
    s_bin[tid] = before;
    __syncthreads();
    ap_for_tiles(a, [&](int b, const AttnSeq &s, int t, int blocks) {
        if (blocks == 0) return;
        const int at = atomicAdd(&s_bin[bin(blocks)], hk);
        for (int h = 0; h < hk; ++h) a.tiles[at + h] = {b, t * hk + h};
    });
}

// Walks the unit list tile by tile.  A whole warp runs it.
struct ApIter {
    int b, h, qt, nt;
    int nkv;       // blocks that the tile sees
    int64_t first; // the tile's first unit
    AttnSeq s;

    // the tile that holds unit u
    BITNET_DEVINL void seek(const AttnArgs &a, int64_t u)
    {
        const int lane = threadIdx.x & 31;
        int lo = 0, hi = a.bt.n_seqs; // base[lo] <= u < base[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.base[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        s = attn_seq(a, b);
        nt = ap_tiles(s, a.group);
        const int64_t base = a.base[b], per_head = (a.base[b + 1] - base) / a.kv.hk;
        h = (int)((u - base) / per_head);
        first = base + h * per_head;
        qt = 0;
        nkv = 0;
        for (int t0 = 0; t0 < nt; t0 += 32) {
            const int blocks = t0 + lane < nt ? ap_blocks(s, a.group, t0 + lane) : 0;
            const int mine = ap_units(blocks);
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const int all = __shfl_sync(0xffffffffu, incl, 31);
            if (u < first + all) {
                const int at = __ffs(__ballot_sync(0xffffffffu, u < first + incl)) - 1;
                qt = t0 + at;
                nkv = __shfl_sync(0xffffffffu, blocks, at);
                first += __shfl_sync(0xffffffffu, incl - mine, at);
                break;
            }
            first += all;
        }
    }

    // the next tile that sees anything, if there is one
    BITNET_DEVINL void next(const AttnArgs &a)
    {
        first += ap_units(nkv);
        do {
            if (++qt >= nt) {
                qt = 0;
                if (++h >= a.kv.hk) {
                    h = 0;
                    do {
                        if (++b >= a.bt.n_seqs) return;
                        s = attn_seq(a, b);
                        nt = ap_tiles(s, a.group);
                    } while (nt == 0);
                }
            }
            nkv = ap_blocks(s, a.group, qt);
        } while (nkv == 0);
    }
};

// One lane of a converged warp, in the form that lets the compiler keep the
// operands of what it guards in uniform registers.
BITNET_DEVINL bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The same box into the L2 cache only.
BITNET_DEVINL void tma_prefetch_3d(const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// kind::f16 instruction descriptor: D fp32, M = 128; A and B bf16 or fp16.
constexpr __host__ __device__ uint32_t ap_idesc(int n, bool bf16, bool b_mn_major)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// MN-major operand, 128-byte swizzle: rows of 64 elements of the M/N dimension,
// consecutive k 128 bytes apart in groups of 8 (SBO 1024), the next 64 elements
// `lbo` bytes further.
BITNET_DEVINL uint64_t umma_desc_mn_sw128(uint32_t addr, uint32_t lbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

BITNET_DEVINL void umma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A from tensor memory: row m in lane m, two fp16 per column.
BITNET_DEVINL void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Warp-collective: 32 lanes x 16 consecutive 32-bit columns (the load waits for its data).
BITNET_DEVINL void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
BITNET_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

BITNET_DEVINL void tmem_ld16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}

// Exponent of a step (its power of two), -126 for zero and subnormal ones.
BITNET_DEVINL int step_exp(float x) { return max((int)((__float_as_uint(x) >> 23) & 0xff) - 127, -126); }
BITNET_DEVINL float exp2_int(int e) { return __uint_as_float((uint32_t)(max(-126, min(127, e)) + 127) << 23); }

constexpr int AP_NO_UNIT = -1000;
// The sums' unit stays above 2^-72 of the largest one before it: a token adds less than 2^21 units of its time (weight 2^8,
// the step's part in it 2, code 2^7, the step's part on it 2^5), 2^31 tokens less than 2^52, and those times 2^72 are finite.
constexpr int AP_UNIT_DEPTH = 72;

// What the other warps need of a block's pages, made by the producer.
struct ApSteps {
    float f[8];    // k_step * scale * log2(e), never 0: masked scores are -infinity.  2^-149 in place of 0: a sum of
                   // codes times queries below 2^128 then gives at most 2^-21
    float lg[8];   // log2 of the part of v_step that the weights carry
    float inv[8];  // its inverse
    float mul[8];  // the part that goes on V's codes: a power of two, or 0
    int unit;      // exponent of the sums' unit from this block on
    int pad[7];
};

// A CTA's part of a row tile.
struct ApSeg {
    int cnt;         // blocks of this CTA (0: no more tiles)
    int j0, nkv;     // the first of them; blocks that the tile sees
    int b, h, qt;
    int q0, n, len;  // AttnSeq of b
    int last;        // the CTA that holds the tile's last block
    int pad[2];
};

template <int N>
BITNET_DEVINL void regs_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
BITNET_DEVINL void regs_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
BITNET_DEVINL float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
BITNET_DEVINL float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

BITNET_DEVINL float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 3-D tiled tensor copy global -> shared (no multicast); c0 times the element size a multiple of 16 bytes.
BITNET_DEVINL void tma_load_3d(uint32_t dst_smem, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                               uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst_smem),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// Four codes -> two bf16 pairs (bytes 0, 1) and (2, 3): the low seven bits go
// under the exponent of 128 and 128, or 256 for a negative code, is subtracted.
BITNET_DEVINL void codes_to_bf16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    constexpr uint32_t k43 = 0x43434343u;
    const uint32_t low = w & 0x7f7f7f7fu, neg = w & 0x80808080u;
    const uint32_t a = __byte_perm(low, k43, 0x4140), b = __byte_perm(low, k43, 0x4342);
    const uint32_t c = __byte_perm(neg, k43, 0x4140), d = __byte_perm(neg, k43, 0x4342);
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&c));
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&b),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&d));
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// Four lanes l = 0..3 hold blocks [l][0..3] of four words; afterwards lane l holds [0..3][l].
BITNET_DEVINL void turn4x4(uint32_t (&o)[4][4], int lane)
{
#pragma unroll
    for (int step = 1; step <= 2; step *= 2) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & step) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) { // swap o[i ^ step] of the lower lane with o[i] of the upper one
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? o[i][e] : o[i ^ step][e], step);
                if (up)
                    o[i][e] = got;
                else
                    o[i ^ step][e] = got;
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(AP_THREADS, 1)
    k_attention_prompt(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_q, const AttnArgs a)
{
    constexpr uint32_t Q_TILE = 128 * D * 2;        // bytes of one MMA tile's queries
    constexpr uint32_t C_TILE = AP_BLOCK * D * 2;   // 16-bit tile of K or V
    constexpr uint32_t R_TILE = AP_BLOCK * D;       // int8 tile
    constexpr uint32_t SLAB = 128 * 128;            // 64 elements of 128 rows
    constexpr int GROUPS = AP_BLOCK / AT_GROUP;
    static_assert(sizeof(ApSteps) == 160 && 384 + AP_STEPS * sizeof(ApSteps) <= 1024 && 1024 + AP_SEGS * sizeof(ApSeg) + 4096 <= AP_HDR, "header");

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *raw_full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *raw_empty = raw_full + AP_RAW;
    uint64_t *cv_full = raw_empty + AP_RAW;
    uint64_t *cv_empty = cv_full + AP_CONV;
    uint64_t *seg_full = cv_empty + AP_CONV;
    uint64_t *seg_empty = seg_full + AP_SEGS;
    uint64_t *q_full = seg_empty + AP_SEGS;
    uint64_t *q_empty = q_full + 1;        // every product of the queries is complete
    uint64_t *s_full = q_empty + 1;        // [2] scores are in tensor memory
    uint64_t *p_full = s_full + 2;         // [2][2] weights of the block's halves are; the first one's also: all sums
                                           // are rescaled
    uint64_t *o_full = p_full + 4;         // [2] a tile's sums are complete
    uint64_t *pair = o_full + 2;           // [8] the two warps of 32 rows exchange a value per row
    uint64_t *seg_want = pair + 8;         // the producer asks for the next tile
    uint64_t *mma_done = seg_want + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    ApSteps *s_step = reinterpret_cast<ApSteps *>(smem + 384);              // [AP_STEPS]
    ApSeg *s_seg = reinterpret_cast<ApSeg *>(smem + 1024);                  // [AP_SEGS]
    float *s_mx = reinterpret_cast<float *>(smem + 1024 + AP_SEGS * sizeof(ApSeg)); // [2 turns][2 tiles][2 halves][128]
    unsigned char *s_q = smem + AP_HDR;
    unsigned char *s_conv = s_q + 2 * Q_TILE;
    unsigned char *s_raw = s_conv + AP_CONV * C_TILE;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < AP_RAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < AP_CONV; ++i) {
            mbar_init(&cv_full[i], 4);
            mbar_init(&cv_empty[i], 1);
        }
        for (int i = 0; i < AP_SEGS; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], AP_SEG_READERS);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[2 * x], 8);
            mbar_init(&p_full[2 * x + 1], 4);
            mbar_init(&o_full[x], 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&pair[i], 2);
        mbar_init(seg_want, 1);
        mbar_init(mma_done, 1);
        fence_mbarrier_init();
    }
    if (tid == AP_TMA_WARP * 32) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_q);
    }
    if (warp == AP_MMA_WARP) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    // Every wait below is by whole warps; `ok` is the same in all lanes.
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t par) {
        ok = __all_sync(0xffffffffu, ok && kv_wait(bar, par));
        return ok;
    };
    // the next tile's description (false: no more)
    uint32_t gslot = 0, gph = 0;
    ApSeg sg;
    auto next_seg = [&]() {
        if (!wait(&seg_full[gslot], gph)) return false;
        sg = s_seg[gslot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[gslot]);
        if (++gslot == AP_SEGS) {
            gslot = 0;
            gph ^= 1;
        }
        return sg.cnt > 0;
    };

    // registers: 16 warps x 88 + 4 x 64 + 4 x 64, the launch's 24 x 80
    if (warp >= AP_TMA_WARP) {
      regs_dec<64>();
      if (warp == AP_SCHED_WARP) {
        // ---------------- tiles ----------------
        const int64_t total = a.base[a.bt.n_seqs];
        const int64_t active = ap_active(total, gridDim.x);
        const bool whole = a.claim->whole != 0, idle = whole || blockIdx.x >= active;
        const int64_t u0 = idle ? 0 : total * blockIdx.x / active, u1 = idle ? 0 : total * (blockIdx.x + 1) / active;
        ApIter it;
        it.first = 0;
        it.b = it.h = it.qt = it.nkv = 0;
        it.s = {0, 0, 0};
        if (u0 < u1) it.seek(a, u0);
        uint32_t rph = 0;
        bool first = true;
        for (bool more = true; more;) {
            int j0 = 0, j1 = 0; // this CTA's blocks of the tile
            if (whole) {
                // claimed when the producer asks for the next tile, not before: tiles go to whoever is free
                if (!first) {
                    if (!wait(seg_want, rph)) break;
                    rph ^= 1;
                }
                first = false;
                int at = 0;
                if (lane == 0) at = atomicAdd(&a.claim->next, 1);
                at = __shfl_sync(0xffffffffu, at, 0);
                more = at < a.claim->tiles;
                if (more) {
                    const int2 tile = a.tiles[at];
                    it.b = tile.x;
                    it.qt = tile.y / a.kv.hk;
                    it.h = tile.y - it.qt * a.kv.hk;
                    it.s = attn_seq(a, it.b);
                    it.nkv = j1 = ap_blocks(it.s, a.group, it.qt);
                }
            } else {
                more = false;
                while (it.first < u1 && !more) {
                    j0 = (int)max((int64_t)0, u0 - it.first - AP_OVER);
                    j1 = (int)min((int64_t)it.nkv, u1 - it.first - AP_OVER);
                    more = j1 > j0;
                    if (!more) it.next(a);
                    if (it.b >= a.bt.n_seqs) break;
                }
            }
            if (!wait(&seg_empty[gslot], gph ^ 1)) break;
            if (lane == 0) {
                ApSeg &d = s_seg[gslot];
                d.cnt = more ? j1 - j0 : 0;
                d.j0 = j0;
                d.nkv = it.nkv;
                d.b = it.b;
                d.h = it.h;
                d.qt = it.qt;
                d.q0 = it.s.q0;
                d.n = it.s.n;
                d.len = it.s.len;
                d.last = !whole && more ? (int)(((it.first + AP_OVER + it.nkv) * active - 1) / total) : 0;
                mbar_arrive(&seg_full[gslot]);
                if (more) { // the queries are on their way to the L2 cache by the time they are asked for
                    const int tokens = ap_tokens(a.group);
                    for (int x = 0; x < 2; ++x)
                        for (int i = 0; i < D / 64; ++i)
                            tma_prefetch_3d(&tm_q, 64 * i, it.h * a.group, it.s.q0 + (2 * it.qt + x) * tokens);
                }
            }
            __syncwarp();
            if (++gslot == AP_SEGS) {
                gslot = 0;
                gph ^= 1;
            }
            if (!whole) {
                if (more) it.next(a);
                if (it.b >= a.bt.n_seqs) it.first = u1;
            }
        }
      } else if (warp == AP_TMA_WARP) {
        // ---------------- producer ----------------
        // Lanes 0-7: the 16-token groups of a block.  Page ids are fetched two blocks and
        // steps one block ahead.  A block's steps go to slot (block % 4): its first copy waits
        // for a raw tile that is free only after the products of the block three before it, so
        // nobody still reads the steps of the block four before.
        const int page_size = 1 << a.kv.page_shift;
        int j = 0; // of sg
        bool more = next_seg();
        auto fetch = [&](int &page, int &row, bool &valid, bool &head, bool &block) {
            page = -1;
            row = 0;
            valid = false;
            head = j == 0;
            block = more;
            if (!more) return;
            const int key0 = (sg.j0 + j) * AP_BLOCK + lane * AT_GROUP;
            valid = lane < GROUPS && key0 < sg.len;
            if (valid) {
                page = page_of(a.kv, a.bt, sg.b, key0 >> a.kv.page_shift);
                row = (sg.h << a.kv.page_shift) + (key0 & ((1 << a.kv.page_shift) - 1));
            }
            if (++j >= sg.cnt) {
                j = 0;
                if (lane == 0) mbar_arrive(seg_want);
                more = next_seg();
            }
        };
        auto steps = [&](int pg, int rw, float &k, float &v) {
            k = v = 0.0f;
            if (pg >= 0) {
                const int64_t at = (int64_t)pg * a.kv.hk + (rw >> a.kv.page_shift);
                k = a.kv.k_step[at];
                v = a.kv.v_step[at];
            }
        };
        int page, row, page1, row1, page2, row2;
        bool valid, valid1, valid2, head, head1, head2, block, block1, block2;
        float ks, vs, ks1, vs1;
        fetch(page, row, valid, head, block);
        fetch(page1, row1, valid1, head1, block1);
        steps(page, row, ks, vs);
        int stage = 0, slot = 0, unit = AP_NO_UNIT, top = AP_NO_UNIT;
        uint32_t phase = 0, issued = 0, last_par = 0;
        while (block && ok) {
            steps(page1, row1, ks1, vs1);
            fetch(page2, row2, valid2, head2, block2);
            // The sums' unit moves when the largest step of a block leaves [2^-4, 2^5) of it.  Limiting
            // each move instead of the whole descent would not do: what a page of step 1 left became
            // infinite two blocks behind it where steps are 1e-35.
            if (head) unit = top = AP_NO_UNIT;
            const float vmax = warp_max(vs);
            if (vmax > 0.0f) {
                const int e = step_exp(vmax);
                if (unit == AP_NO_UNIT || e - unit < -4 || e - unit > 4) unit = max(e, top - AP_UNIT_DEPTH);
                top = max(top, unit);
            }
            const int ce = max(-24, min(5, step_exp(vs) - unit)); // exponent that goes on the codes
            const float rest = vs > 0.0f ? vs * exp2_int(-(unit + ce)) : 1.0f;
            const bool copy = valid && page >= 0 && (lane * AT_GROUP & (page_size - 1)) == 0; // a page's first group
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copy)) * page_size * D;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (!wait(&raw_empty[stage], phase ^ 1)) break;
                if (kv == 0 && lane < GROUPS) {
                    ApSteps &st = s_step[slot];
                    st.f[lane] = fmaxf(a.scale_log2 * ks, 0x1p-149f);
                    st.lg[lane] = log2f(rest);
                    st.inv[lane] = 1.0f / rest;
                    st.mul[lane] = vs > 0.0f ? exp2_int(ce) : 0.0f;
                    if (lane == 0) st.unit = unit;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&raw_full[stage], bytes);
                __syncwarp();
                if (copy)
                    tma_load_3d(smem_u32(s_raw) + stage * R_TILE + lane * AT_GROUP * D, kv ? &tm_v : &tm_k, 0, row,
                                page, &raw_full[stage]);
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == AP_RAW) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            slot = (slot + 1) % AP_STEPS;
            page = page1;
            row = row1;
            valid = valid1;
            head = head1;
            block = block1;
            ks = ks1;
            vs = vs1;
            page1 = page2;
            row1 = row2;
            valid1 = valid2;
            head1 = head2;
            block1 = block2;
        }
        for (int s = 0; s < AP_RAW; ++s)
            if (issued & (1u << s)) mbar_wait_drain(&raw_full[s], (last_par >> s) & 1);
      } else if (warp == AP_MMA_WARP) {
        // ---------------- MMA issuer ----------------
        // Per block: weights of A times V, next scores of A, then the same for B: while one
        // tile's softmax runs the other's products do.
        constexpr uint32_t id_s = ap_idesc(AP_BLOCK, true, false), id_o = ap_idesc(D, false, true);
        uint32_t cslot = 0, cphase = 0;
        uint32_t qph = 0, pph[2] = {0, 0};
        auto scores = [&](int x, uint32_t kslot) {
            const uint64_t ad = umma_desc_k_sw128(s_q + x * Q_TILE), bd = umma_desc_k_sw128(s_conv + kslot * C_TILE);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = (uint64_t)((k >> 2) * (SLAB >> 4) + (k & 3) * 2);
                    umma_f16_ss(tmem + x * 128, ad + off, bd + off, id_s, k != 0);
                }
                umma_commit(&s_full[x]);
            }
            __syncwarp();
        };
        // a half's weights lie over the first half of its scores
        auto sums = [&](int x, uint32_t vslot, bool first) {
            const uint64_t bd = umma_desc_mn_sw128(smem_u32(s_conv + vslot * C_TILE), SLAB);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!wait(&p_full[2 * x + half], pph[x])) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + 64 * half + 8 * k,
                                    bd + (uint64_t)(4 * half + k) * (16 * 128 >> 4), id_o,
                                    !first || half != 0 || k != 0);
                }
                __syncwarp();
            }
            pph[x] ^= 1;
            return true;
        };
        auto commit = [&](uint64_t *bar) {
            if (elect_one()) umma_commit(bar);
            __syncwarp();
        };
        auto take = [&](uint32_t &s) { // the next 16-bit tile
            if (!wait(&cv_full[cslot], cphase)) return false;
            s = cslot;
            if (++cslot == AP_CONV) {
                cslot = 0;
                cphase ^= 1;
            }
            return true;
        };
        while (ok && next_seg()) {
            const bool two = sg.n > (2 * sg.qt + 1) * ap_tokens(a.group);
            uint32_t ks, vs;
            if (!take(ks) || !wait(q_full, qph)) break;
            qph ^= 1;
            tc_fence_after();
            scores(0, ks);
            if (two) scores(1, ks);
            commit(&cv_empty[ks]);
            if (sg.cnt == 1) commit(q_empty);
            for (int j = 0; j < sg.cnt && ok; ++j) {
                const bool more = j + 1 < sg.cnt;
                if (!take(vs) || !sums(0, vs, j == 0)) break;
                if (more) {
                    if (!take(ks)) break;
                    tc_fence_after();
                    scores(0, ks);
                } else {
                    commit(&o_full[0]);
                    if (!two) commit(&o_full[1]);
                }
                if (two) {
                    if (!sums(1, vs, j == 0)) break;
                    if (!more) commit(&o_full[1]);
                }
                commit(&cv_empty[vs]);
                if (more) {
                    if (two) scores(1, ks);
                    commit(&cv_empty[ks]);
                    if (j + 2 == sg.cnt) commit(q_empty);
                }
            }
        }
        if (elect_one()) {
            umma_commit(mma_done);
            mbar_wait_drain(mma_done, 0);
        }
        __syncwarp();
      } else {
        // ---------------- queries ----------------
        // rows behind the sequence's last token hold what follows it (or zeros), rows behind the
        // tile's last token what was there: a row's values go nowhere but its own scores
        const int tokens = ap_tokens(a.group);
        uint32_t qph = 0;
        while (ok && next_seg()) {
            if (!wait(q_empty, qph ^ 1)) break;
            qph ^= 1;
            if (lane == 0) {
                const int tiles = sg.n > (2 * sg.qt + 1) * tokens ? 2 : 1; // an MMA tile without rows is not used
                mbar_arrive_expect_tx(q_full, tiles * (D / 64) * tokens * a.group * 128);
                for (int x = 0; x < tiles; ++x)
                    for (int i = 0; i < D / 64; ++i)
                        tma_load_3d(smem_u32(s_q) + x * Q_TILE + i * SLAB, &tm_q, 64 * i, sg.h * a.group,
                                    sg.q0 + (2 * sg.qt + x) * tokens, q_full);
            }
            __syncwarp();
        }
        // let the last copies land before the CTA can exit
        if (qph) mbar_wait_drain(q_full, 0);
        else mbar_wait_drain(q_full, 1);
      }
    } else if (warp >= AP_CONV_WARP0) {
        regs_dec<64>();
        // ---------------- int8 -> bf16 (K), fp16 (V) ----------------
        const int r = tid - AP_CONV_WARP0 * 32; // row of the tile: a token
        int rs = 0, cs = 0, slot = 0;
        uint32_t rph = 0, cph = 0;
        while (ok && next_seg()) {
            for (int j = 0; j < sg.cnt && ok; ++j) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    if (!wait(&raw_full[rs], rph) || !wait(&cv_empty[cs], cph ^ 1)) break;
                    const uint32_t src = smem_u32(s_raw) + rs * R_TILE;
                    unsigned char *dst = s_conv + cs * C_TILE;
                    // V: code * 2^e = fma(1152 + code, 2^e, -1152 * 2^e), each a multiple of fp16's
                    // smallest 2^-24 with few bits, so exact for -24 <= e <= 5
                    const float mf = s_step[slot].mul[r / AT_GROUP];
                    const __half2 mul = __half2half2(__float2half_rn(mf));
                    const __half2 add = __half2half2(__float2half_rn(-1152.0f * mf));
                    uint4 raw[4]; // loads run four chunks ahead
#pragma unroll
                    for (int c = 0; c < 4; ++c) raw[c] = lds128(src + kv_swz<D>(r, c));
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 now = raw[c & 3];
                        if (c + 4 < D / 16) raw[c & 3] = lds128(src + kv_swz<D>(r, c + 4));
                        const uint32_t in[4] = {now.x, now.y, now.z, now.w};
                        uint32_t out[8];
                        if (kv == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) codes_to_bf16(in[i], out[2 * i], out[2 * i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t f = in[i] ^ 0x80808080u;
                                const uint32_t x = __byte_perm(f, kHalfMagic, 0x4140);
                                const uint32_t y = __byte_perm(f, kHalfMagic, 0x4342);
                                const __half2 hx = __hfma2(*reinterpret_cast<const __half2 *>(&x), mul, add);
                                const __half2 hy = __hfma2(*reinterpret_cast<const __half2 *>(&y), mul, add);
                                out[2 * i] = *reinterpret_cast<const uint32_t *>(&hx);
                                out[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&hy);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int cc = 2 * c + i; // 16-byte chunk of the row's 2 D bytes
                            *reinterpret_cast<uint4 *>(dst + (cc >> 3) * SLAB + r * 128 + (((cc & 7) ^ (r & 7)) << 4)) =
                                make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&cv_full[cs]);
                        mbar_arrive(&raw_empty[rs]);
                    }
                    if (++rs == AP_RAW) {
                        rs = 0;
                        rph ^= 1;
                    }
                    if (++cs == AP_CONV) {
                        cs = 0;
                        cph ^= 1;
                    }
                }
                slot = (slot + 1) % AP_STEPS;
            }
        }
    } else {
        regs_inc<88>();
        // ---------------- softmax ----------------
        const int x = warp >> 3, half = (warp >> 2) & 1; // MMA tile, half of a block's tokens
        const int r = (warp & 3) * 32 + lane;            // row of the tile = lane of tensor memory
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128 + half * 64; // this half's scores, then weights
        const uint32_t to = tmem + lanes + 256 + x * 128 + half * (D / 2);
        float *mx_mine = s_mx + (x * 2 + half) * 128 + r, *mx_other = s_mx + (x * 2 + (half ^ 1)) * 128 + r;
        const int tokens = ap_tokens(a.group), rtok = r / a.group, rhead = r - rtok * a.group;
        uint64_t *pair_bar = pair + x * 4 + (warp & 3);
        uint32_t sph = 0, oph = 0, turn = 0;
        int slot = 0;
        auto exchange = [&](float v) { // the same value of the row's other thread
            mx_mine[turn * 512] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(pair_bar);
            wait(pair_bar, turn);
            const float o = mx_other[turn * 512];
            turn ^= 1;
            return o;
        };
        while (ok && next_seg()) {
            const int tok = (2 * sg.qt + x) * tokens + rtok;
            const bool live = rtok < tokens && tok < sg.n;
            if ((2 * sg.qt + x) * tokens >= sg.n) { // a tile without rows keeps step with the issuer
                slot = (slot + sg.cnt) % AP_STEPS;
                wait(&o_full[x], oph);
                oph ^= 1;
                continue;
            }
            const int lim = live ? sg.len - sg.n + tok : -1; // last visible token
            // rows of this warp are consecutive: the first one sees least
            const int lim_min = __all_sync(0xffffffffu, live) ? __shfl_sync(0xffffffffu, lim, 0) : -1;
            float m = -INFINITY, l = 0.0f;
            int unit = AP_NO_UNIT;
            for (int j = 0; j < sg.cnt; ++j) {
                if (!wait(&s_full[x], sph)) break;
                sph ^= 1;
                tc_fence_after();
                const ApSteps &st = s_step[slot];
                const int key0 = (sg.j0 + j) * AP_BLOCK + half * 64;
                const int vis = lim - key0; // last visible column
                const bool masked = key0 + 63 > lim_min;
                // the largest score
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32];
                    tmem_ld32(ts + 32 * c, v);
                    tmem_wait_ld(v);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i > vis) v[i] = 0xff800000u; // -infinity
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float best = __uint_as_float(v[16 * h]);
#pragma unroll
                        for (int i = 1; i < 15; i += 2)
                            best = max3(best, __uint_as_float(v[16 * h + i]), __uint_as_float(v[16 * h + i + 1]));
                        best = fmaxf(best, __uint_as_float(v[16 * h + 15]));
                        mx = fmaxf(mx, best * st.f[4 * half + 2 * c + h]);
                    }
                }
                mx = fmaxf(mx, exchange(mx));
                // the row's reference follows its maximum when it lags too far
                float al = 1.0f;
                if (mx > m + AP_LAZY) {
                    al = m == -INFINITY ? 0.0f : fast_exp2(m - mx);
                    m = mx;
                    l *= al;
                }
                const int unit1 = st.unit;
                if (unit1 != unit && unit != AP_NO_UNIT) al *= exp2_int(unit - unit1);
                unit = unit1;
                if (j > 0 && __any_sync(0xffffffffu, al != 1.0f)) {
                    // scores of this block are complete, so are the sums of the one before
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t w[16];
                        tmem_ld16(to + 16 * c, w);
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * al);
                        tmem_st16(to + 16 * c, w);
                    }
                }
                // The first half's products add to every column of the sums, and this half holds the upper ones.
                if (half == 1) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * x]);
                }
                const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32], w[16];
                    tmem_ld32(ts + 32 * c, v);
                    tmem_wait_ld(v);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i > vis) v[i] = 0xff800000u;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 4 * half + 2 * c + h;
                        const float f = st.f[g], off = st.lg[g] - mu;
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 t = fma2(make_float2(__uint_as_float(v[16 * h + i]),
                                                              __uint_as_float(v[16 * h + i + 1])),
                                                  make_float2(f, f), make_float2(off, off));
                            const float2 p = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                            sum = add2(sum, p);
                            w[8 * h + i / 2] = pack_half2(p.x, p.y);
                        }
                        l = fmaf(sum.x + sum.y, st.inv[g], l);
                    }
                    tmem_st16(ts + 16 * c, w); // over scores that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
                slot = (slot + 1) % AP_STEPS;
            }
            if (!ok) break;
            l += exchange(l);
            // ---- the tile's sums ----
            if (!wait(&o_full[x], oph)) break;
            oph ^= 1;
            tc_fence_after();
            const bool whole = sg.cnt == sg.nkv;
            const float us = unit == AP_NO_UNIT ? 0.0f : exp2_int(unit);
            const float inv = m > -INFINITY ? 1.0f / l : 0.0f; // us / l may lie below the normal range
            const int64_t part = (2 * (int64_t)blockIdx.x + (sg.j0 == 0 ? 1 : 0)) * AP_ROWS;
            if (!whole && sg.j0 == 0 && warp == 0 && lane == 0)
                a.shared[blockIdx.x] = {sg.n, sg.last, sg.q0, sg.h, sg.qt};
            if (!whole && live && half == 0) a.part_ml[part + x * 128 + r] = make_float2(m, l);
            const int64_t row_at = live ? (int64_t)(sg.q0 + tok) * a.out_stride +
                                              ((int64_t)sg.h * a.group + rhead) * D + half * (D / 2)
                                        : -1;
            float4 *pdst = reinterpret_cast<float4 *>(a.part + part * D) + (half * (D / 8)) * AP_ROWS + x * 128 + r;
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                uint32_t v[32];
                tmem_ld32(to + 32 * c, v);
                tmem_wait_ld(v);
                if (whole) {
                    // 64 bytes of a row per lane; four lanes turn theirs so that each stores 16 bytes of
                    // four rows: a store then touches eight lines instead of 32
                    uint32_t o[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][e] = bf16_rn_bits(__uint_as_float(v[8 * i + 2 * e]) * inv * us) |
                                      (bf16_rn_bits(__uint_as_float(v[8 * i + 2 * e + 1]) * inv * us) << 16);
                    turn4x4(o, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) { // row (lane & ~3) + i, chunk lane & 3
                        const int64_t at = __shfl_sync(0xffffffffu, row_at, (lane & ~3) + i);
                        if (at >= 0)
                            *reinterpret_cast<uint4 *>(a.out + at + 32 * c + 8 * (lane & 3)) =
                                make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
                    }
                } else if (live) { // [D / 4][256 rows] groups of four
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        pdst[(8 * c + i) * AP_ROWS] =
                            make_float4(__uint_as_float(v[4 * i]) * us, __uint_as_float(v[4 * i + 1]) * us,
                                        __uint_as_float(v[4 * i + 2]) * us, __uint_as_float(v[4 * i + 3]) * us);
                }
                __syncwarp();
            }
            tc_fence_before(); // before the next tile's products, ordered by its p_full
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == AP_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the row tiles that more than one CTA shared: blocks (k, .) the one whose first
// part CTA k holds, a thread per row and 16 columns.
template <int D>
__global__ void __launch_bounds__(256) k_attention_prompt_join(const AttnArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, c0 = blockIdx.x;
    const AttnShared s = a.shared[c0]; // nrow: the sequence's new tokens, r0: the tile
    if (s.nrow == 0) return;
    const int tokens = ap_tokens(a.group);
    const int rtok = (tid & 127) / a.group, g = (tid & 127) - rtok * a.group;
    const int tok = (2 * s.r0 + (tid >> 7)) * tokens + rtok;
    if (rtok >= tokens || tok >= s.nrow) return;
    auto part = [&](int k) { return (2 * (int64_t)k + (k == c0 ? 1 : 0)) * AP_ROWS; };
    float m = -INFINITY, l = 0.0f;
    for (int k = c0; k <= s.last; ++k) m = fmaxf(m, a.part_ml[part(k) + tid].x);
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    const int col = blockIdx.y * 16;
    for (int k = c0; k <= s.last; ++k) {
        const float2 ml = a.part_ml[part(k) + tid];
        const float f = ml.x == -INFINITY ? 0.0f : fast_exp2(ml.x - m);
        l += ml.y * f;
        const float4 *src = reinterpret_cast<const float4 *>(a.part + part(k) * D) + (col / 4) * AP_ROWS + tid;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = src[i * AP_ROWS];
            acc[4 * i] += v.x * f;
            acc[4 * i + 1] += v.y * f;
            acc[4 * i + 2] += v.z * f;
            acc[4 * i + 3] += v.w * f;
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)(s.q0 + tok) * a.out_stride +
                                           ((int64_t)s.h * a.group + g) * D + col);
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = bf16_rn_bits(acc[2 * e] * inv) | (bf16_rn_bits(acc[2 * e + 1] * inv) << 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

} // namespace bitnet
