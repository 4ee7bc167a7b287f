// attention_tokens.cuh -- attention of few new tokens per sequence over the
// paged 8-bit cache (decoding, verification of drafts): at most 48 query rows
// (new tokens x query heads of the group) per sequence and kv head.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(c (q_r . k_j) - m_r),
//   c = scale * log2(e), k = code * k_step, v = code * v_step
//
// Bound by HBM: the codes of K and V are read once (2 D bytes per cached token
// and kv head; everything else is small).  The work is the list of all
// (sequence, kv head, tile of 8 or 16 rows, group of 16 tokens) in that order,
// cut into equal contiguous shares, one per CTA (one CTA per SM), and those into
// equal shares per warp, so ragged batches and single long sequences load every
// SM alike.  A warp works alone: it copies its groups' codes into its own
// buffers in shared memory, the next ones while it computes on one, keeps its own
// running maxima and sums, and waits for no other warp before the end.  Then the
// CTA adds up the pieces of (sequence, kv head, row tile) that its warps share, in
// the order of the warps; what it shares with other CTAs (at most two) goes to the
// workspace, and k_attention_join adds that up in the order of the CTAs: no
// atomics, the result does not depend on timing.
// (Before, a producer warp fed all warps through one ring by TMA, and the warps
// joined at the end of every row tile: 70 us for 64 sequences of up to 4096 tokens,
// 51 us of them without any computation; 16-token pages, a TMA each, took longer
// still.  Now, with the kernel's later steps: 45 us, 3.8 TB/s; one sequence of 131071
// tokens 41 us, 4.1 TB/s, join included.)
//
// The products run on mma.sync m16n8k16 in fp16 with fp32 sums and the tokens
// (K) and the head dimension (V transposed) on the side of 16, the rows on the
// side of 8: a row tile needs half the instructions and registers that it would
// with its rows on the side of 16, and instructions per byte of codes are what
// costs besides HBM.  Codes are exact in fp16 (the byte goes under the exponent of
// 1024 and 1152 is subtracted), queries are brought into fp16's range by a power of
// two per row.  K and V fragments are read from shared memory in the layout that
// the bytes already have: an order of the contraction index and of the output rows
// can be chosen freely, so a lane takes 16 consecutive bytes of a key (K) or of a
// value (V).
#pragma once

#include <cuda_fp16.h>

#include "kv_common.cuh"

namespace bitnet {

constexpr int AT_GROUP = 16;    // tokens a warp takes at a time (a page holds at least as many): a unit
// Query rows per (sequence, kv head) that this kernel is chosen for.  Its cost grows with every
// 16 rows, that of the kernel for prompts with every 256; measured (D = 128) with 48 and 64 rows: 64
// sequences of 2048 tokens 117 and 150 us here, 141 and 141 us there; with 64 rows 16 sequences
// of 8192 tokens (8 query heads a kv head) 117 us here, 107 us there, 64 sequences of 300 tokens
// 46 and 55 us.
constexpr int AT_MAX_ROWS = 48;
constexpr int AT_MAX_CTAS = 160;
constexpr int AT_MIN_UNITS = 16; // groups worth a CTA of their own
constexpr float AT_LAZY = 8.0f;  // a row's exponents refer to a maximum up to 2^8 behind

// A row tile whose first part is in CTA k's share and the rest in those of the CTAs up to `last`.
struct AttnShared {
    int nrow; // 0: CTA k has none
    int last;
    int q0, h, r0;
};

// Prompts: whether whole tiles are claimed, the next one and how many there are.
struct AttnClaim {
    int whole, next, tiles;
};

struct AttnArgs {
    KvView kv;
    BatchView bt;
    const uint16_t *q; // bf16
    int64_t q_stride;
    uint16_t *out;     // bf16
    int64_t out_stride;
    int group;         // query heads per kv head
    int max_new;
    float scale_log2;  // scale * log2(e)
    float *part;       // [2 * CTAs][rows][D] partial sums
    float2 *part_ml;   // [2 * CTAs][rows] their maxima and sums
    int64_t *base;     // [n_seqs + 1] first unit of each sequence (prompts)
    AttnShared *shared; // [CTAs] row tiles to join
    AttnClaim *claim;   // (prompts)
    int2 *tiles;        // (prompts) sequence, tile * kv heads + head, dearest first
};

// Warps for nq tiles of 8 rows: as many as leave each the registers it wants (168, 255).
// Tiles of 8 rows serve up to 8 rows (16 sequences of 8192 tokens, 8 rows: 40.5 us, against 47.1
// in a tile of 16), tiles of 16 more (16 rows: 49 us).
// With 16 and 12 warps of 128 and 168: 52 us instead of 47 (64 sequences), 64 instead of 48
// (16 sequences of four new tokens, 8 query heads a kv head).
constexpr __host__ __device__ int at_warps(int nq) { return nq == 1 ? 12 : 8; }
constexpr int AT_BUFS = 2; // a warp's buffers of a group's codes (three: no faster)

constexpr __host__ __device__ int at_smem(int d, int nq)
{
    return 4096 + at_warps(nq) * (AT_BUFS * 2 * AT_GROUP * d + 8 * nq * (d + 4) * 4 + 2 * 8 * nq * 8) + 1024;
}

BITNET_DEVINL void cp_async16_u32(uint32_t dst_smem, const void *src_gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src_gmem) : "memory");
}

BITNET_DEVINL uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
BITNET_DEVINL uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

BITNET_DEVINL uint32_t h2_sub(uint32_t a, uint32_t b)
{
    const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

constexpr uint32_t kHalfMagic = 0x64646464u; // high byte of fp16 1024 .. 2047 in steps of 1
constexpr uint32_t kHalfBias = 0x64806480u;  // fp16 1152 = 1024 + 128, twice

// Four codes with their sign bits flipped (code + 128) -> two fp16 pairs (bytes 0, 1) and (2, 3).
BITNET_DEVINL void codes_to_half(uint32_t flipped, uint32_t &lo, uint32_t &hi)
{
    lo = h2_sub(__byte_perm(flipped, kHalfMagic, 0x4140), kHalfBias);
    hi = h2_sub(__byte_perm(flipped, kHalfMagic, 0x4342), kHalfBias);
}

BITNET_DEVINL void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

BITNET_DEVINL uint32_t pack_half2(float a, float b)
{
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Transposes an 8 x 8 tile of fp16 held as row = lane / 4, columns 2 (lane % 4), + 1.
BITNET_DEVINL uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

BITNET_DEVINL float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest power of two not above x (x >= 0; the smallest normal one for less).
BITNET_DEVINL float pow2_floor(float x)
{
    const uint32_t e = __float_as_uint(x) & 0x7f800000u;
    return __uint_as_float(e == 0u ? 0x00800000u : e);
}

// Power of two that brings a row with largest magnitude amax into fp16's upper
// range [2^14, 2^15); its inverse is exact too.
BITNET_DEVINL float half_range_factor(float amax)
{
    const int e = (int)((__float_as_uint(amax) >> 23) & 0xff) - 127; // -127 for zero and subnormals
    return __uint_as_float((uint32_t)(min(14 - e, 126) + 127) << 23);
}

// New rows and cached tokens of sequence b as the attention sees them.
struct AttnSeq {
    int q0, n, len;
};

BITNET_DEVINL AttnSeq attn_seq(const AttnArgs &a, int b)
{
    AttnSeq s;
    s.q0 = a.bt.q_start[b];
    const int q1 = a.bt.q_start[b + 1];
    s.len = a.bt.lens[b];
    s.n = q1 - s.q0;
    if (s.q0 < 0 || q1 < s.q0 || q1 > a.bt.T || s.len < 0 || s.len > (a.bt.width << a.kv.page_shift) ||
        s.n > a.max_new) {
        record_batch_error();
        s.n = 0;
        s.len = 0;
    }
    return s;
}

BITNET_DEVINL int attn_groups(const AttnSeq &s) { return s.n > 0 ? (s.len + AT_GROUP - 1) / AT_GROUP : 0; }

// CTAs that share `units` groups.
BITNET_DEVINL int64_t attn_active(int64_t units, int ctas)
{
    const int64_t want = (units + AT_MIN_UNITS - 1) / AT_MIN_UNITS;
    return want < ctas ? want : ctas;
}

// a / b for a >= 0, b > 0; nearly always both are small.
BITNET_DEVINL int64_t div_fast(int64_t a, int b)
{
    return (a >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Row tiles of `rows` rows per kv head of a sequence, and its units.
BITNET_DEVINL int attn_row_tiles(const AttnArgs &a, const AttnSeq &s, int rows) { return (s.n * a.group + rows - 1) / rows; }
BITNET_DEVINL int64_t attn_units(const AttnArgs &a, const AttnSeq &s, int rows)
{
    return (int64_t)a.kv.hk * attn_row_tiles(a, s, rows) * attn_groups(s);
}

// Walks the unit list: sequence of unit u, given a sequence at or before it.
struct UnitIter {
    int b;
    int64_t base; // first unit of sequence b
    AttnSeq s;
    int nc, nt;   // groups, row tiles per kv head

    BITNET_DEVINL void load(const AttnArgs &a, int rows)
    {
        s = attn_seq(a, b);
        nc = attn_groups(s);
        nt = attn_row_tiles(a, s, rows);
    }
    BITNET_DEVINL void seek(const AttnArgs &a, int64_t u, int rows)
    {
        for (;;) {
            const int64_t n = (int64_t)a.kv.hk * nt * nc;
            if (u < base + n || b + 1 >= a.bt.n_seqs) return;
            base += n;
            ++b;
            load(a, rows);
        }
    }
};

// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows, as TMA's
// 128-byte (D = 128) and 64-byte (D = 64) swizzles place it.
template <int D>
BITNET_DEVINL uint32_t kv_swz(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// A warp's share of a row tile that it does not hold whole.
struct AtPiece {
    int64_t first, end; // units of the row tile; first = -1: no piece
    int q0, h, r0, nrow;
};

// NQ: tiles of 8 query rows.
template <int D, int NQ>
__global__ void __launch_bounds__(at_warps(NQ) * 32, 1) k_attention_tokens(const AttnArgs a)
{
    constexpr int WARPS = at_warps(NQ), THREADS = WARPS * 32;
    constexpr int DT = D / 16;              // output tiles of 16 elements
    constexpr int ROWS = 8 * NQ;
    constexpr uint32_t TILE = AT_GROUP * D; // bytes of K (or V) of a group
    constexpr int PROW = D + 4;             // floats of a row of a piece
    constexpr int CPR = D / 16;             // 16-byte chunks of a token
    constexpr int COPIES = AT_GROUP * CPR / 32;

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int64_t *s_scan = reinterpret_cast<int64_t *>(smem);            // [WARPS] sums
    AtPiece *s_piece = reinterpret_cast<AtPiece *>(smem + 256);     // [WARPS][2]
    float2 *s_step = reinterpret_cast<float2 *>(smem + 256 + 32 * 32 + 256); // [WARPS][buffers] k_step, v_step
    unsigned char *ring = smem + 4096;                              // [WARPS][buffers][K, V]
    float *s_first = reinterpret_cast<float *>(ring + WARPS * AT_BUFS * 2 * TILE); // [WARPS][ROWS][PROW]: first pieces
    float2 *s_ml = reinterpret_cast<float2 *>(s_first + WARPS * ROWS * PROW); // [WARPS][2][ROWS]
    static_assert(WARPS <= 16 && sizeof(AtPiece) == 32 && 256 + 1024 + 256 + 16 * AT_BUFS * 8 <= 4096, "layout");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();

    // ---- total units, this CTA's and this warp's share and the sequence that it starts in ----
    const int per = (a.bt.n_seqs + THREADS - 1) / THREADS;
    const int b_lo = min(a.bt.n_seqs, tid * per), b_hi = min(a.bt.n_seqs, b_lo + per);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += attn_units(a, attn_seq(a, b), ROWS);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (tid < WARPS * 2) s_piece[tid].first = -1;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int64_t active = attn_active(total, gridDim.x);
    const bool idle = blockIdx.x >= active;
    if (blockIdx.x == 0) { // rows of sequences without cached tokens see nothing
        for (int b = b_lo; b < b_hi; ++b) {
            const AttnSeq s = attn_seq(a, b);
            if (s.len > 0) continue;
            for (int t = 0; t < s.n; ++t)
                for (int x = 0; x < a.kv.hk * a.group * (D / 8); ++x)
                    reinterpret_cast<uint4 *>(a.out + (int64_t)(s.q0 + t) * a.out_stride)[x] = make_uint4(0, 0, 0, 0);
        }
    }
    if (tid == 0) a.shared[blockIdx.x].nrow = 0; // nothing to join yet
    if (idle) return;
    const int64_t c0 = div_fast(total * blockIdx.x, (int)active), c1 = div_fast(total * (blockIdx.x + 1), (int)active);
    // where the CTA starts; its warps walk on from there
    int *s_b = reinterpret_cast<int *>(s_step);
    int64_t *s_u = reinterpret_cast<int64_t *>(s_step) + 1;
    if (c0 >= before && c0 < before + mine) {
        int64_t at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            const int64_t un = attn_units(a, attn_seq(a, b), ROWS);
            if (c0 < at + un) {
                s_b[0] = b;
                s_u[0] = at;
                break;
            }
            at += un;
        }
    }
    __syncthreads();
    UnitIter it;
    it.b = s_b[0];
    it.base = s_u[0];
    it.load(a, ROWS);
    __syncthreads(); // s_step is the warps' own from here on

    const int64_t u0 = c0 + (c1 - c0) * warp / WARPS, u1 = c0 + (c1 - c0) * (warp + 1) / WARPS;
    const uint32_t ring_base = smem_u32(ring) + warp * AT_BUFS * 2 * TILE;
    float2 *steps = s_step + warp * AT_BUFS;

    // ---- copies ----
    // 32 groups at a time, a lane looks up a group's page and steps, one such batch ahead.
    UnitIter ahead = it;
    auto look_up = [&](int64_t u, int64_t &row, float &ks, float &vs) { // row of the codes' [page][head][slot], or -1
        row = -1;
        ks = vs = 0.0f;
        if (u >= u1) return;
        ahead.seek(a, u, ROWS);
        const int64_t rel = u - ahead.base;
        const int ht = (int)div_fast(rel, ahead.nc), key0 = (int)(rel - (int64_t)ht * ahead.nc) * AT_GROUP;
        const int page = page_of(a.kv, a.bt, ahead.b, key0 >> a.kv.page_shift);
        if (page < 0) return;
        const int64_t at = (int64_t)page * a.kv.hk + ht / ahead.nt;
        row = (at << a.kv.page_shift) + (key0 & ((1 << a.kv.page_shift) - 1));
        ks = a.kv.k_step[at];
        vs = a.kv.v_step[at];
    };
    int64_t row_a, row_b;
    float ks_a, vs_a, ks_b, vs_b;
    look_up(u0 + lane, row_a, ks_a, vs_a);
    look_up(u0 + 32 + lane, row_b, ks_b, vs_b);
    int issued = 0, buf = 0; // groups whose copies are under way or done, the next one's buffer
    auto copy = [&]() {
        const int from = issued & 31;
        const int64_t row = __shfl_sync(0xffffffffu, row_a, from);
        const float ks = __shfl_sync(0xffffffffu, ks_a, from), vs = __shfl_sync(0xffffffffu, vs_a, from);
        if (row >= 0) {
            const int8_t *k = a.kv.k + row * D + lane * 16, *v = a.kv.v + row * D + lane * 16;
            const uint32_t dst = ring_base + buf * 2 * TILE;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
                const int x = lane + 32 * i;
                const uint32_t at = dst + kv_swz<D>(x / CPR, x % CPR);
                cp_async16_u32(at, k + i * 512);
                cp_async16_u32(at + TILE, v + i * 512);
            }
        }
        if (lane == 0) steps[buf] = make_float2(ks, vs);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++buf == AT_BUFS) buf = 0;
        ++issued;
        if ((issued & 31) == 0) {
            row_a = row_b;
            ks_a = ks_b;
            vs_a = vs_b;
            look_up(u0 + issued + 32 + lane, row_b, ks_b, vs_b);
        }
    };
#pragma unroll 1
    for (int i = 0; i < AT_BUFS; ++i) copy();

    const int g = lane >> 2, c = lane & 3;
    const int key_g = (g & 1) ? ((g + 4) & 7) : g;      // token of score row g (g + 8: + 8): 0 5 2 7 4 1 6 3, see below
    const int key_e = 2 * c, key_o = (2 * c + 5) & 7;   // tokens of contraction indices 2c, 2c + 1 of the second product
    int use = 0; // buffer of the next group

    for (int64_t u = u0; u < u1;) {
        it.seek(a, u, ROWS);
        const int64_t rel = u - it.base;
        const int ht = (int)div_fast(rel, it.nc), t0 = (int)(rel - (int64_t)ht * it.nc);
        const int h = ht / it.nt, r0 = (ht - h * it.nt) * ROWS; // kv head, first row of the tile
        const int cnt = (int)min((int64_t)(it.nc - t0), u1 - u);
        const int nrow = min(ROWS, it.s.n * a.group - r0);
        const int len = it.s.len, first = len - it.s.n;

        // queries of this row tile, scaled into fp16's range row by row.  Rows of this lane: 8 t + g
        // (queries), 8 t + 2 c and + 1 (scores and weights).
        uint32_t qb[NQ][D / 64][8]; // contraction step 4 hh + w: qb[t][hh][2 w], [2 w + 1]
        float o[NQ][DT][4], m[NQ][2], l[NQ][2], fac[NQ][2];
        int lim[NQ][2];
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            const int r = 8 * t + g, tok = (r0 + r) / a.group;
            const bool live = r < nrow;
            const uint16_t *p = a.q + (int64_t)(it.s.q0 + (live ? tok : 0)) * a.q_stride +
                                ((int64_t)h * a.group + (live ? r0 + r - tok * a.group : 0)) * D + c * 16;
            uint4 w[D / 64][2];
            float mx = 0.0f;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[hh][e] = live ? *reinterpret_cast<const uint4 *>(p + 64 * hh + 8 * e) : make_uint4(0, 0, 0, 0);
                    const uint32_t v[4] = {w[hh][e].x, w[hh][e].y, w[hh][e].z, w[hh][e].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, fmaxf(fabsf(bf16_bits_lo(v[i])), fabsf(bf16_bits_hi(v[i]))));
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float f = half_range_factor(mx);
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t v[4] = {w[hh][e].x, w[hh][e].y, w[hh][e].z, w[hh][e].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qb[t][hh][4 * e + i] = pack_half2(bf16_bits_lo(v[i]) * f, bf16_bits_hi(v[i]) * f);
                }
            const float fr = a.scale_log2 / f;
            const int lr = live ? first + tok : -1; // last visible position
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                fac[t][e] = __shfl_sync(0xffffffffu, fr, 4 * (2 * c + e));
                lim[t][e] = __shfl_sync(0xffffffffu, lr, 4 * (2 * c + e));
                m[t][e] = -INFINITY;
                l[t][e] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < DT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.0f;
        }
        float unit = 0.0f, inv_unit = 0.0f; // o is in units of this power of two; 0: not chosen yet

        for (int i = 0; i < cnt; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(AT_BUFS - 1) : "memory"); // the oldest copies have landed
            __syncwarp();
            const int key0 = (t0 + i) * AT_GROUP;
            {
                const float2 step = steps[use];
                const float ks = step.x, vs = step.y;
                const uint32_t kb = ring_base + use * 2 * TILE, vb = kb + TILE;
                float s[NQ][4];
#pragma unroll
                for (int t = 0; t < NQ; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
                // scores: tokens x rows.  Contraction step 4 hh + w takes elements 16 (c + 4 hh) + 4 w
                // .. + 3 of lane column c.  Score row g is token key_g: the two tokens of a
                // shared-memory wavefront differ in bit 2, so their swizzled chunks differ.
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh) {
                    const uint4 k0 = lds128(kb + kv_swz<D>(key_g, c + 4 * hh));
                    const uint4 k1 = lds128(kb + kv_swz<D>(8 + key_g, c + 4 * hh));
                    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        codes_to_half(w0[w] ^ 0x80808080u, a0, a2);
                        codes_to_half(w1[w] ^ 0x80808080u, a1, a3);
#pragma unroll
                        for (int t = 0; t < NQ; ++t)
                            mma_f16(s[t], a0, a1, a2, a3, qb[t][hh][2 * w], qb[t][hh][2 * w + 1]);
                    }
                }
                // the values' codes are on their way during the softmax
                uint32_t vw[4][D / 32];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rw = (k & 1 ? key_o : key_e) + 8 * (k >> 1);
                    if constexpr (D == 128) {
                        const uint4 w = lds128(vb + kv_swz<D>(rw, g));
                        vw[k][0] = w.x;
                        vw[k][1] = w.y;
                        vw[k][2] = w.z;
                        vw[k][3] = w.w;
                    } else {
                        const uint2 w = lds64(vb + kv_swz<D>(rw, g >> 1) + 8 * (g & 1));
                        vw[k][0] = w.x;
                        vw[k][1] = w.y;
                    }
                }
                // softmax: s[t][2 k + e] is token key_g + 8 k, row 8 t + 2 c + e
                const bool masked = key0 + AT_GROUP - 1 > first;
                bool grown = false;
                float mx[NQ][2];
#pragma unroll
                for (int t = 0; t < NQ; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = fac[t][e] * ks;
                        float &x0 = s[t][e], &x1 = s[t][2 + e];
                        x0 *= f;
                        x1 *= f;
                        if (masked) {
                            if (key0 + key_g > lim[t][e]) x0 = -INFINITY;
                            if (key0 + 8 + key_g > lim[t][e]) x1 = -INFINITY;
                        }
                        float v = fmaxf(x0, x1);
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        mx[t][e] = v;
                        grown |= v > m[t][e] + AT_LAZY;
                    }
                // a row's reference follows its maximum when it lags too far, and o keeps units near the
                // current page's v_step: weights times v_step / unit stay in fp16's range, whatever the
                // steps of other pages.  A smaller unit makes larger numbers of what o holds already, so it
                // goes no lower than where those reach 2^120 (later products add less than 2^52); a page
                // that then lies far below the unit is lost against what the row tile holds.
                float r = vs * inv_unit;
                const bool move = vs > 0.0f && !(r >= 0x1p-4f && r <= 0x1p4f);
                if (__any_sync(0xffffffffu, grown) || move) {
#pragma unroll
                    for (int t = 0; t < NQ; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (!(mx[t][e] > m[t][e] + AT_LAZY)) continue;
                            const float al = fast_exp2(m[t][e] - mx[t][e]);
                            m[t][e] = mx[t][e];
                            l[t][e] *= al;
#pragma unroll
                            for (int n = 0; n < DT; ++n) {
                                o[t][n][e] *= al;
                                o[t][n][2 + e] *= al;
                            }
                        }
                    if (move) {
                        float om = 0.0f;
#pragma unroll
                        for (int t = 0; t < NQ; ++t)
#pragma unroll
                            for (int n = 0; n < DT; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) om = fmaxf(om, fabsf(o[t][n][e]));
                        om = warp_max(om);
                        const float want = pow2_floor(vs);
                        if (om > 0.0f) {
                            const float most = fminf(pow2_floor(0x1p120f / om), 0x1p120f);
                            float us = unit / want;
                            if (us <= most) {
                                unit = want;
                            } else {
                                us = most;
                                unit /= us;
                            }
#pragma unroll
                            for (int t = 0; t < NQ; ++t)
#pragma unroll
                                for (int n = 0; n < DT; ++n)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[t][n][e] *= us;
                        } else {
                            unit = want;
                        }
                        inv_unit = 1.0f / unit;
                        r = vs * inv_unit;
                    }
                }
                uint32_t pb[NQ][2];
#pragma unroll
                for (int t = 0; t < NQ; ++t) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mu = m[t][e] == -INFINITY ? 0.0f : m[t][e];
                        p[e] = fast_exp2(s[t][e] - mu);
                        p[2 + e] = fast_exp2(s[t][2 + e] - mu);
                        l[t][e] += p[e] + p[2 + e];
                    }
                    pb[t][0] = transpose8(pack_half2(p[0] * r, p[1] * r));
                    pb[t][1] = transpose8(pack_half2(p[2] * r, p[3] * r));
                }
                // o += v^T p: elements x rows.  Output rows g, g + 8 of tile n are elements
                // (D / 8) g + 2 n, + 1; contraction indices 2c, 2c + 1 (+ 8) are tokens key_e, key_o (+ 8).
                if (vs > 0.0f) {
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        uint32_t ab[2][4]; // [tokens 0-7, 8-15][element 4 w + x]
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = vw[2 * e][w] ^ 0x80808080u, y = vw[2 * e + 1][w] ^ 0x80808080u;
                            codes_to_half(__byte_perm(x, y, 0x5140), ab[e][0], ab[e][1]);
                            codes_to_half(__byte_perm(x, y, 0x7362), ab[e][2], ab[e][3]);
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int t = 0; t < NQ; ++t)
                                mma_f16(o[t][2 * w + x], ab[0][2 * x], ab[0][2 * x + 1], ab[1][2 * x], ab[1][2 * x + 1],
                                        pb[t][0], pb[t][1]);
                    }
                }
            }
            __syncwarp(); // the buffer has been read
            copy();
            if (++use == AT_BUFS) use = 0;
        }

        // ---- sums of the lanes; the piece or the result ----
#pragma unroll
        for (int t = 0; t < NQ; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], x);
        if (cnt == it.nc) {
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * t + 2 * c + e;
                    if (r >= nrow) continue;
                    const float inv = m[t][e] > -INFINITY ? 1.0f / l[t][e] : 0.0f;
                    const int tok = (r0 + r) / a.group;
                    uint16_t *p = a.out + (int64_t)(it.s.q0 + tok) * a.out_stride +
                                  ((int64_t)h * a.group + (r0 + r - tok * a.group)) * D + (D / 8) * g;
                    uint32_t w[DT];
#pragma unroll
                    for (int n = 0; n < DT; ++n)
                        w[n] = bf16_rn_bits(o[t][n][e] * inv * unit) | (bf16_rn_bits(o[t][n][2 + e] * inv * unit) << 16);
#pragma unroll
                    for (int n = 0; n < DT; n += 4)
                        *reinterpret_cast<uint4 *>(p + 2 * n) = make_uint4(w[n], w[n + 1], w[n + 2], w[n + 3]);
                }
        } else {
            // the first piece beside the buffers; a later one is the warp's last and takes their place
            const int k = u == u0 ? 0 : 1;
            if (k) asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            float *dst = k ? reinterpret_cast<float *>(ring + warp * AT_BUFS * 2 * TILE) : s_first + warp * ROWS * PROW;
            const int prow = k ? D : PROW;
#pragma unroll
            for (int t = 0; t < NQ; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * t + 2 * c + e;
#pragma unroll
                    for (int n = 0; n < DT; n += 2)
                        *reinterpret_cast<float4 *>(dst + r * prow + (D / 8) * g + 2 * n) =
                            make_float4(o[t][n][e] * unit, o[t][n][2 + e] * unit, o[t][n + 1][e] * unit,
                                        o[t][n + 1][2 + e] * unit);
                    if (g == 0) s_ml[(warp * 2 + k) * ROWS + r] = make_float2(m[t][e], l[t][e]);
                }
            if (lane == 0) {
                AtPiece &pc = s_piece[warp * 2 + k];
                pc.first = it.base + (int64_t)ht * it.nc;
                pc.end = pc.first + it.nc;
                pc.q0 = it.s.q0;
                pc.h = h;
                pc.r0 = r0;
                pc.nrow = nrow;
            }
        }
        u += cnt;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    // ---- pieces of the same row tile, in the order of the warps; a warp per row ----
    for (int p0 = 0; p0 < WARPS * 2;) {
        const AtPiece pc = s_piece[p0];
        if (pc.first < 0) {
            ++p0;
            continue;
        }
        int p1 = p0 + 1; // behind the last piece of this row tile (the next pieces that exist)
        while (p1 < WARPS * 2 && (s_piece[p1].first < 0 || s_piece[p1].first == pc.first)) ++p1;
        const bool whole = pc.first >= c0 && pc.end <= c1;
        const int slot = 2 * blockIdx.x + (pc.first >= c0 ? 1 : 0);
        for (int r = warp; r < pc.nrow; r += WARPS) {
            float mm = -INFINITY;
            for (int p = p0; p < p1; ++p)
                if (s_piece[p].first >= 0) mm = fmaxf(mm, s_ml[p * ROWS + r].x);
            float ll = 0.0f, acc[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
            if (mm > -INFINITY)
                for (int p = p0; p < p1; ++p) {
                    if (s_piece[p].first < 0) continue;
                    const float2 ml = s_ml[p * ROWS + r];
                    const float f = fast_exp2(ml.x - mm);
                    const float *src = (p & 1) ? reinterpret_cast<const float *>(ring + (p >> 1) * AT_BUFS * 2 * TILE) + r * D
                                               : s_first + (p >> 1) * ROWS * PROW + r * PROW;
                    ll += ml.y * f;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) acc[e] += src[lane * (D / 32) + e] * f;
                }
            if (whole) {
                const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
                const int tok = (pc.r0 + r) / a.group;
                uint32_t *p = reinterpret_cast<uint32_t *>(a.out + (int64_t)(pc.q0 + tok) * a.out_stride +
                                                           ((int64_t)pc.h * a.group + (pc.r0 + r - tok * a.group)) * D) +
                              lane * (D / 64);
#pragma unroll
                for (int e = 0; e < D / 64; ++e)
                    p[e] = bf16_rn_bits(acc[2 * e] * inv) | (bf16_rn_bits(acc[2 * e + 1] * inv) << 16);
            } else {
                float *p = a.part + ((int64_t)slot * ROWS + r) * D + lane * (D / 32);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) p[e] = acc[e];
                if (lane == 0) a.part_ml[(int64_t)slot * ROWS + r] = make_float2(mm, ll);
            }
        }
        if (tid == 0 && !whole && pc.first >= c0)
            a.shared[blockIdx.x] = {pc.nrow, (int)((pc.end * active - 1) / total), pc.q0, pc.h, pc.r0};
        p0 = p1;
    }
}

// Joins the row tiles that more than one CTA shared: block (k, r) row r of the one
// whose first part CTA k holds.  Four warps take the parts in turn (one warp after
// another part by part took 19 us for the 30 parts of one long sequence) and are
// added up in their order.
template <int D>
__global__ void __launch_bounds__(128) k_attention_join(const AttnArgs a, int rows)
{
    __shared__ float s_acc[4][D];
    __shared__ float s_l[4];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = blockIdx.x, r = blockIdx.y;
    const AttnShared s = a.shared[c0];
    if (r >= s.nrow) return;
    auto slot = [&](int k) { return (int64_t)(2 * k + (k == c0 ? 1 : 0)) * rows + r; };
    float m = -INFINITY;
    for (int k = c0 + lane; k <= s.last; k += 32) m = fmaxf(m, a.part_ml[slot(k)].x);
    m = warp_max(m);
    float acc[D / 32], l = 0.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
    if (m != -INFINITY) {
#pragma unroll 8
        for (int k = c0 + warp; k <= s.last; k += 4) {
            const float2 ml = a.part_ml[slot(k)];
            const float f = fast_exp2(ml.x - m);
            const float *src = a.part + slot(k) * D + lane * (D / 32);
            l += ml.y * f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] += src[e] * f;
        }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s_acc[warp][lane * (D / 32) + e] = acc[e];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int d = 2 * threadIdx.x + e;
        x[e] = ((s_acc[0][d] + s_acc[1][d]) + (s_acc[2][d] + s_acc[3][d])) * inv;
    }
    const int tok = (s.r0 + r) / a.group;
    reinterpret_cast<uint32_t *>(a.out + (int64_t)(s.q0 + tok) * a.out_stride +
                                 ((int64_t)s.h * a.group + (s.r0 + r - tok * a.group)) * D)[threadIdx.x] =
        bf16_rn_bits(x[0]) | (bf16_rn_bits(x[1]) << 16);
}

} // namespace bitnet
