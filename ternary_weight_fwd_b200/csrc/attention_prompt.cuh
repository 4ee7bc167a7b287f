// attention_prompt.cuh -- causal grouped-query attention of prompts (many new
// tokens per sequence) over the paged 8-bit cache, on the 5th-generation tensor
// cores: tcgen05.mma kind::f16 with fp32 accumulators in tensor memory.
//
// Same formulas as attention_tokens.cuh.  Bound by the tensor cores and the
// exponentials: 4 D flops and one exp2 per visible (query head, token) pair.
//
// Query rows of a (sequence, kv head) are its new tokens times the query heads
// of the group (row = token * group + head), cut into tiles of 256 rows: two MMA
// tiles A and B of 128, so that one's softmax runs while the other's products
// do.  Tokens are taken in blocks of 128.  The work is the list of all
// (sequence, kv head, row tile, block that the tile sees), cut into equal
// contiguous shares, one per CTA (one CTA per SM); tiles that two or more CTAs
// share are joined by k_attention_prompt_join through the workspace, in the
// order of the CTAs.
//
// One CTA, 16 warps:
//   warps 0-3, 4-7  softmax of tile A, B: a thread per row.  They load the
//                   queries (scaled by a power of two per row, fp16, into the
//                   K-major 128-byte-swizzled layout), read scores from tensor
//                   memory, write weights back over them as the next product's
//                   A operand, rescale and finally read the sums.
//   warps 8-11      int8 codes -> fp16, K and V tiles alike: rows of tokens, in
//                   the 128-byte-swizzled layout that serves K as a K-major and
//                   V as an MN-major B operand (a row of V is contiguous in the
//                   head dimension, the N of that product).
//   warp 12         TMA of the codes (16-token boxes, one page each)
//   warp 13         MMA issuer, owner of tensor memory
// Codes are exact in fp16.  A page's v_step is applied in two factors: a power of
// two on the code (exact in fp16 down to 2^-24) and the rest, in [1, 2), on the
// weight; the sums are in units of a power of two near the current pages' steps.
#pragma once

#include "attention_tokens.cuh"

namespace bitnet {

constexpr int AP_ROWS = 256;      // query rows per tile (two MMA tiles)
constexpr int AP_BLOCK = 128;     // tokens per block
constexpr int AP_THREADS = 512;
constexpr int AP_RAW = 3;         // ring of int8 tiles
constexpr int AP_CONV = 3;        // ring of fp16 tiles
constexpr int AP_STEPS = 4;       // ring of blocks' steps (see the producer)
constexpr int AP_MIN_UNITS = 2;   // blocks worth a CTA of their own
constexpr int AP_CONV_WARP0 = 8, AP_TMA_WARP = 12, AP_MMA_WARP = 13;
constexpr float AP_LAZY = 8.0f;   // the reference of a row's exponents lags its maximum by up to 2^8

constexpr __host__ __device__ int ap_smem(int d)
{
    return 1024 + 2 * 128 * d * 2 + AP_CONV * AP_BLOCK * d * 2 + AP_RAW * AP_BLOCK * d + 1024;
}

// Blocks that row tile qt of a sequence sees (rows see tokens 0 .. len - n + row / group).
BITNET_DEVINL int ap_blocks(const AttnSeq &s, int group, int qt)
{
    const int last = min(s.n - 1, (int)(((int64_t)(qt + 1) * AP_ROWS - 1) / group));
    const int lim = s.len - s.n + last;
    return lim < 0 ? 0 : lim / AP_BLOCK + 1;
}

BITNET_DEVINL int ap_tiles(const AttnSeq &s, int group)
{
    return (int)(((int64_t)s.n * group + AP_ROWS - 1) / AP_ROWS);
}

BITNET_DEVINL int64_t ap_active(int64_t units, int ctas)
{
    const int64_t want = (units + AP_MIN_UNITS - 1) / AP_MIN_UNITS;
    return want < ctas ? want : ctas;
}

// First unit of every sequence: a warp per sequence adds up its tiles' blocks, then one scan.
__global__ void __launch_bounds__(1024) k_attention_plan(const AttnArgs a)
{
    __shared__ int64_t s_sum[32];
    __shared__ int64_t s_carry;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int n_seqs = a.bt.n_seqs;
    for (int b = warp; b < n_seqs; b += 32) {
        const AttnSeq s = attn_seq(a, b);
        const int nt = ap_tiles(s, a.group);
        int64_t sum = 0;
        for (int t = lane; t < nt; t += 32) sum += ap_blocks(s, a.group, t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) a.base[b + 1] = sum * a.kv.hk;
    }
    if (tid == 0) {
        a.base[0] = 0;
        s_carry = 0;
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
}

// Position in the unit list, advanced tile by tile.  Whole warps run it.
struct ApIter {
    int b, h, qt, nt;
    int j0, cnt, nkv; // blocks [j0, j0 + cnt) of the tile's nkv
    AttnSeq s;

    // the tile that holds unit u
    BITNET_DEVINL void seek(const AttnArgs &a, int64_t u, int64_t u1)
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
        const int64_t first = a.base[b], per_head = (a.base[b + 1] - first) / a.kv.hk;
        h = (int)((u - first) / per_head);
        int64_t rel = (u - first) - h * per_head;
        qt = 0;
        nkv = 0;
        j0 = 0;
        for (int t0 = 0; t0 < nt; t0 += 32) {
            const int mine = t0 + lane < nt ? ap_blocks(s, a.group, t0 + lane) : 0;
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const int all = __shfl_sync(0xffffffffu, incl, 31);
            if (rel < all) {
                const int at = __ffs(__ballot_sync(0xffffffffu, rel < incl)) - 1;
                qt = t0 + at;
                nkv = __shfl_sync(0xffffffffu, mine, at);
                j0 = (int)rel - (__shfl_sync(0xffffffffu, incl, at) - nkv);
                break;
            }
            rel -= all;
        }
        cnt = (int)min((int64_t)(nkv - j0), u1 - u);
    }

    // the next tile that sees anything; u: its first unit (< u1)
    BITNET_DEVINL void next(const AttnArgs &a, int64_t u, int64_t u1)
    {
        do {
            if (++qt >= nt) {
                qt = 0;
                if (++h >= a.kv.hk) {
                    h = 0;
                    do {
                        ++b;
                        s = attn_seq(a, b);
                        nt = ap_tiles(s, a.group);
                    } while (nt == 0 && b + 1 < a.bt.n_seqs);
                }
            }
            nkv = nt > 0 ? ap_blocks(s, a.group, qt) : 0;
        } while (nkv == 0 && b + 1 < a.bt.n_seqs);
        j0 = 0;
        cnt = (int)min((int64_t)nkv, u1 - u);
    }
};

// kind::f16 instruction descriptor: D fp32, A and B fp16, M = 128.
constexpr __host__ __device__ uint32_t ap_idesc(int n, bool b_mn_major)
{
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
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

// Unit exponent of the sums from block to block: it moves when the largest step
// of a block leaves [2^-4, 2^5) of it, and not below 2^-60 of what it was (all
// roles follow the same rule on the same steps).
constexpr int AP_NO_UNIT = -1000;
BITNET_DEVINL int ap_unit(int unit, const float *vs)
{
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < AP_BLOCK / AT_GROUP; ++i) mx = fmaxf(mx, vs[i]);
    if (!(mx > 0.0f)) return unit;
    const int e = step_exp(mx);
    if (unit == AP_NO_UNIT) return e;
    return e - unit < -4 || e - unit > 4 ? max(e, unit - 60) : unit;
}
// Power of two that goes on the codes of a page with step v.
BITNET_DEVINL int ap_code_exp(float v, int unit) { return max(-24, min(5, step_exp(v) - unit)); }

template <int D>
__global__ void __launch_bounds__(AP_THREADS, 1)
    k_attention_prompt(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const AttnArgs a)
{
    constexpr uint32_t Q_TILE = 128 * D * 2;        // bytes of one MMA tile's queries
    constexpr uint32_t C_TILE = AP_BLOCK * D * 2;   // fp16 tile of K or V
    constexpr uint32_t R_TILE = AP_BLOCK * D;       // int8 tile
    constexpr uint32_t SLAB = 128 * 128;            // 64 elements of 128 rows
    constexpr int GROUPS = AP_BLOCK / AT_GROUP;

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *raw_full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *raw_empty = raw_full + AP_RAW;
    uint64_t *cv_full = raw_empty + AP_RAW;
    uint64_t *cv_empty = cv_full + AP_CONV;
    uint64_t *q_full = cv_empty + AP_CONV; // [2]
    uint64_t *s_full = q_full + 2;         // [2] scores are in tensor memory
    uint64_t *p_full = s_full + 2;         // [2] weights are
    uint64_t *o_full = p_full + 2;         // [2] a tile's sums are complete
    uint64_t *mma_done = o_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    float *s_step = reinterpret_cast<float *>(smem + 512); // [AP_STEPS][2][8]
    unsigned char *s_q = smem + 1024;
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
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 4);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_full[x], 1);
        }
        mbar_init(mma_done, 1);
        fence_mbarrier_init();
    }
    if (tid == AP_TMA_WARP * 32) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
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

    const int64_t total = a.base[a.bt.n_seqs];
    const int64_t active = ap_active(total, gridDim.x);
    const bool idle = blockIdx.x >= active;
    const int64_t u0 = idle ? 0 : total * blockIdx.x / active, u1 = idle ? 0 : total * (blockIdx.x + 1) / active;
    ApIter it;
    it.cnt = 0;
    if (u0 < u1) it.seek(a, u0, u1);

    if (warp == AP_TMA_WARP) {
        // ---------------- producer ----------------
        // Lanes 0-7: the 16-token groups of a block.  Page ids are fetched two blocks and
        // steps one block ahead.  A block's steps go to slot (block % 4): its first copy waits
        // for a raw tile that is free only after the products of the block three before it, so
        // nobody still reads the steps of the block four before.
        auto fetch = [&](const ApIter &w, int j, int64_t u, int &page, int &row, bool &valid) {
            page = -1;
            row = 0;
            const int key0 = j * AP_BLOCK + lane * AT_GROUP;
            valid = lane < GROUPS && u < u1 && key0 < w.s.len;
            if (valid) {
                page = page_of(a.kv, a.bt, w.b, key0 >> a.kv.page_shift);
                row = (w.h << a.kv.page_shift) + (key0 & ((1 << a.kv.page_shift) - 1));
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
        // `ahead` walks two blocks in front
        ApIter ahead = it;
        int64_t ua = u0;
        int ja = 0; // within ahead's blocks
        auto advance = [&]() {
            ++ua;
            if (++ja >= ahead.cnt && ua < u1) {
                ahead.next(a, ua, u1);
                ja = 0;
            }
        };
        int page, row, page1, row1, page2, row2;
        bool valid, valid1, valid2;
        float ks, vs, ks1, vs1;
        fetch(ahead, ahead.j0 + ja, ua, page, row, valid);
        advance();
        fetch(ahead, ahead.j0 + ja, ua, page1, row1, valid1);
        advance();
        steps(page, row, ks, vs);
        int stage = 0, slot = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok; ++u) {
            steps(page1, row1, ks1, vs1);
            fetch(ahead, ahead.j0 + ja, ua, page2, row2, valid2);
            advance();
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, valid && page >= 0)) * AT_GROUP * D;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                ok = __all_sync(0xffffffffu, mbar_wait(&raw_empty[stage], phase ^ 1));
                if (!ok) break;
                if (kv == 0 && lane < GROUPS) {
                    s_step[slot * 16 + lane] = ks;
                    s_step[slot * 16 + 8 + lane] = vs;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&raw_full[stage], bytes);
                __syncwarp();
                if (valid && page >= 0)
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
            ks = ks1;
            vs = vs1;
            page1 = page2;
            row1 = row2;
            valid1 = valid2;
        }
        for (int s = 0; s < AP_RAW; ++s)
            if (issued & (1u << s)) mbar_wait_drain(&raw_full[s], (last_par >> s) & 1);
    } else if (warp == AP_MMA_WARP) {
        // ---------------- MMA issuer ----------------
        // Per block: weights of A times V, next scores of A, then the same for B: while one
        // tile's softmax runs the other's products do.
        constexpr uint32_t id_s = ap_idesc(AP_BLOCK, false), id_o = ap_idesc(D, true);
        uint32_t cslot = 0, cphase = 0;
        uint32_t qph = 0, pph[2] = {0, 0};
        bool ok = true;
        auto scores = [&](int x, uint32_t kslot) {
            const uint64_t ad = umma_desc_k_sw128(s_q + x * Q_TILE), bd = umma_desc_k_sw128(s_conv + kslot * C_TILE);
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = (uint64_t)((k >> 2) * (SLAB >> 4) + (k & 3) * 2);
                    umma_f16_ss(tmem + x * 128, ad + off, bd + off, id_s, k != 0);
                }
                umma_commit(&s_full[x]);
            }
            __syncwarp();
        };
        auto sums = [&](int x, uint32_t vslot, bool first) {
            const uint64_t bd = umma_desc_mn_sw128(smem_u32(s_conv + vslot * C_TILE), SLAB);
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < AP_BLOCK / 16; ++k)
                    umma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + 8 * k, bd + (uint64_t)k * (16 * 128 >> 4), id_o,
                                !first || k != 0);
            }
            __syncwarp();
        };
        auto wait = [&](uint64_t *bar, uint32_t par) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, par));
            return ok;
        };
        auto release = [&](uint32_t s) {
            if (lane == 0) umma_commit(&cv_empty[s]);
            __syncwarp();
        };
        auto take = [&](uint32_t &s) { // the next fp16 tile
            if (!wait(&cv_full[cslot], cphase)) return false;
            s = cslot;
            if (++cslot == AP_CONV) {
                cslot = 0;
                cphase ^= 1;
            }
            return true;
        };
        for (int64_t u = u0; u < u1 && ok; u += it.cnt, (u < u1 ? it.next(a, u, u1) : (void)0)) {
            const int nrow = (int)min((int64_t)AP_ROWS, (int64_t)it.s.n * a.group - (int64_t)it.qt * AP_ROWS);
            const bool two = nrow > 128;
            uint32_t ks, vs;
            if (!take(ks)) break;
            tc_fence_after();
            if (!wait(&q_full[0], qph)) break;
            tc_fence_after();
            scores(0, ks);
            if (!wait(&q_full[1], qph)) break;
            tc_fence_after();
            if (two) scores(1, ks);
            release(ks);
            qph ^= 1;
            for (int j = 0; j < it.cnt && ok; ++j) {
                const bool more = j + 1 < it.cnt;
                if (!take(vs)) break;
                if (!wait(&p_full[0], pph[0])) break;
                pph[0] ^= 1;
                tc_fence_after();
                sums(0, vs, j == 0);
                if (!more) {
                    if (lane == 0) {
                        umma_commit(&o_full[0]);
                        if (!two) umma_commit(&o_full[1]);
                    }
                    __syncwarp();
                }
                if (more) {
                    if (!take(ks)) break;
                    tc_fence_after();
                    scores(0, ks);
                }
                if (two) {
                    if (!wait(&p_full[1], pph[1])) break;
                    pph[1] ^= 1;
                    tc_fence_after();
                    sums(1, vs, j == 0);
                    if (!more) {
                        if (lane == 0) umma_commit(&o_full[1]);
                        __syncwarp();
                    }
                }
                release(vs);
                if (more) {
                    if (two) scores(1, ks);
                    release(ks);
                }
            }
        }
        if (lane == 0) {
            umma_commit(mma_done);
            mbar_wait_drain(mma_done, 0);
        }
        __syncwarp();
    } else if (warp >= AP_CONV_WARP0 && warp < AP_CONV_WARP0 + 4) {
        // ---------------- int8 -> fp16 ----------------
        const int r = tid - AP_CONV_WARP0 * 32; // row of the tile: a token
        int rs = 0, cs = 0, slot = 0;
        uint32_t rph = 0, cph = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok; u += it.cnt, (u < u1 ? it.next(a, u, u1) : (void)0)) {
            int unit = AP_NO_UNIT;
            for (int j = 0; j < it.cnt && ok; ++j) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], rph) && mbar_wait(&cv_empty[cs], cph ^ 1));
                    if (!ok) break;
                    int e = 0;
                    if (kv) {
                        const float *vs = s_step + slot * 16 + 8;
                        unit = ap_unit(unit, vs);
                        e = ap_code_exp(vs[r / AT_GROUP], unit == AP_NO_UNIT ? 0 : unit);
                    }
                    // code * 2^e = fma(1152 + code, 2^e, -1152 * 2^e): each a multiple of fp16's
                    // smallest 2^-24 with few bits, so exact for -24 <= e <= 5
                    const __half2 mul = __half2half2(__float2half_rn(exp2_int(e)));
                    const __half2 add = __half2half2(__float2half_rn(-1152.0f * exp2_int(e)));
                    const uint32_t src = smem_u32(s_raw) + rs * R_TILE;
                    unsigned char *dst = s_conv + cs * C_TILE;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 w = lds128(src + kv_swz<D>(r, c));
                        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                        uint32_t out[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t f = in[i] ^ 0x80808080u;
                            const uint32_t x = __byte_perm(f, kHalfMagic, 0x4140), y = __byte_perm(f, kHalfMagic, 0x4342);
                            const __half2 hx = __hfma2(*reinterpret_cast<const __half2 *>(&x), mul, add);
                            const __half2 hy = __hfma2(*reinterpret_cast<const __half2 *>(&y), mul, add);
                            out[2 * i] = *reinterpret_cast<const uint32_t *>(&hx);
                            out[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&hy);
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
    } else if (warp < 8) {
        // ---------------- softmax ----------------
        const int x = warp >> 2;              // MMA tile
        const int r = tid & 127;              // row of it = lane of tensor memory
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128, to = tmem + lanes + 256 + x * 128;
        unsigned char *q_tile = s_q + x * Q_TILE;
        uint32_t sph = 0, oph = 0;
        int slot = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok; u += it.cnt, (u < u1 ? it.next(a, u, u1) : (void)0)) {
            const int64_t R = (int64_t)it.qt * AP_ROWS + x * 128 + r;
            const int64_t rows = (int64_t)it.s.n * a.group;
            const int tok = R < rows ? (int)(R / a.group) : 0;
            const int head = it.h * a.group + (int)(R - (int64_t)tok * a.group);
            const bool live = R < rows;
            const bool used = (int64_t)it.qt * AP_ROWS + x * 128 < rows; // this MMA tile has rows at all
            const int lim = live ? it.s.len - it.s.n + tok : -1;         // last visible token
            float fac = 0.0f;
            {   // queries; the products that read the last ones are complete (their scores were waited for)
                uint4 w[D / 8];
                float mx = 0.0f;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (int64_t)(it.s.q0 + tok) * a.q_stride + (int64_t)(live ? head : 0) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) w[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx = fmaxf(mx, fmaxf(fabsf(bf16_bits_lo(v[e])), fabsf(bf16_bits_hi(v[e]))));
                }
                const float f = half_range_factor(mx);
                fac = a.scale_log2 / f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = pack_half2(bf16_bits_lo(v[e]) * f, bf16_bits_hi(v[e]) * f);
                    *reinterpret_cast<uint4 *>(q_tile + (i >> 3) * SLAB + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[x]);
            }
            if (!used) { // keeps step with the issuer
                slot = (slot + it.cnt) % AP_STEPS;
                ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], oph));
                oph ^= 1;
                continue;
            }
            float m = -INFINITY, l = 0.0f;
            int unit = AP_NO_UNIT;
            // rows of this warp are consecutive: the first one sees least
            const int lim_min = __shfl_sync(0xffffffffu, lim, 0);
            const bool ragged = !__all_sync(0xffffffffu, live);
            for (int j = 0; j < it.cnt; ++j) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x], sph));
                if (!ok) break;
                sph ^= 1;
                tc_fence_after();
                const int key0 = (it.j0 + j) * AP_BLOCK;
                const float *ks = s_step + slot * 16, *vs = ks + 8;
                const bool masked = ragged || key0 + AP_BLOCK - 1 > lim_min;
                const int vis = lim - key0; // last visible column
                // the block's largest score
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < AP_BLOCK / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(ts + 32 * c, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float best = -INFINITY;
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (32 * c + 16 * g + i <= vis) best = fmaxf(best, __uint_as_float(v[16 * g + i]));
                            if (best != -INFINITY) mx = fmaxf(mx, best * (fac * ks[2 * c + g]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) best = fmaxf(best, __uint_as_float(v[16 * g + i]));
                            mx = fmaxf(mx, best * (fac * ks[2 * c + g]));
                        }
                    }
                }
                // the row's reference follows its maximum when it lags too far
                float al = 1.0f;
                if (mx > m + AP_LAZY || (m == -INFINITY && mx > m)) {
                    al = m == -INFINITY ? 0.0f : fast_exp2(m - mx);
                    m = mx;
                    l *= al;
                }
                const int unit1 = ap_unit(unit, vs);
                const bool move = unit1 != unit && unit != AP_NO_UNIT;
                if (move) al *= exp2_int(unit - unit1);
                unit = unit1;
                if (j > 0 && __any_sync(0xffffffffu, al != 1.0f)) {
                    // scores of this block are complete, so are the sums of the one before
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t v[16];
                        tmem_ld16(to + 16 * c, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * al);
                        tmem_st16(to + 16 * c, v);
                    }
                }
                const float mu = m == -INFINITY ? 0.0f : m;
                const int ub = unit == AP_NO_UNIT ? 0 : unit;
#pragma unroll
                for (int c = 0; c < AP_BLOCK / 32; ++c) {
                    uint32_t v[32], w[16];
                    tmem_ld32(ts + 32 * c, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float f = fac * ks[2 * c + g], vg = vs[2 * c + g];
                        const float rg = vg * exp2_int(-(ub + ap_code_exp(vg, ub)));
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float p0 = fast_exp2(fmaf(__uint_as_float(v[16 * g + i]), f, -mu));
                            float p1 = fast_exp2(fmaf(__uint_as_float(v[16 * g + i + 1]), f, -mu));
                            if (masked) {
                                if (32 * c + 16 * g + i > vis) p0 = 0.0f;
                                if (32 * c + 16 * g + i + 1 > vis) p1 = 0.0f;
                            }
                            l += p0 + p1;
                            w[8 * g + i / 2] = pack_half2(p0 * rg, p1 * rg);
                        }
                    }
                    tmem_st16(ts + 16 * c, w); // over scores that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
                slot = (slot + 1) % AP_STEPS;
            }
            if (!ok) break;
            // ---- the tile's sums ----
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], oph));
            if (!ok) break;
            oph ^= 1;
            tc_fence_after();
            const bool whole = it.cnt == it.nkv;
            const float us = unit == AP_NO_UNIT ? 0.0f : exp2_int(unit);
            const float inv = l > 0.0f ? us / l : 0.0f;
            const int64_t part = (2 * (int64_t)blockIdx.x + (it.j0 == 0 ? 1 : 0)) * AP_ROWS;
            if (!whole && live) a.part_ml[part + x * 128 + r] = make_float2(m, l);
            uint16_t *dst = a.out + (int64_t)(it.s.q0 + tok) * a.out_stride + (int64_t)head * D;
            float4 *pdst = reinterpret_cast<float4 *>(a.part + part * D) + x * 128 + r;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(to + 32 * c, v);
                tmem_wait_ld(v);
                if (live && whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = bf16_rn_bits(__uint_as_float(v[8 * i + 2 * e]) * inv) |
                                   (bf16_rn_bits(__uint_as_float(v[8 * i + 2 * e + 1]) * inv) << 16);
                        *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
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

// Joins the row tiles that more than one CTA shared and writes zeros for tiles
// that see nothing.  Tiles are numbered per kv head so that sequence b's start
// at q_start[b] * group / 256 + b (there is room for each one's tiles).  A thread per
// row and 16 columns.
template <int D>
__global__ void __launch_bounds__(256) k_attention_prompt_join(const AttnArgs a, int ctas)
{
    __shared__ int s_seq;
    __shared__ int64_t s_before[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) s_seq = -1;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int64_t item = blockIdx.x;
    for (int b = tid; b < a.bt.n_seqs; b += 256) {
        const int64_t lo = a.bt.q_start[b], hi = a.bt.q_start[b + 1];
        if (lo >= 0 && hi >= lo && hi <= a.bt.T && item >= lo * a.group / AP_ROWS + b &&
            item < hi * a.group / AP_ROWS + b + 1)
            s_seq = b;
    }
    __syncthreads();
    const int b = s_seq, h = blockIdx.y;
    if (b < 0) return;
    const AttnSeq s = attn_seq(a, b);
    const int64_t qt64 = item - ((int64_t)s.q0 * a.group / AP_ROWS + b);
    if (s.n == 0 || qt64 >= ap_tiles(s, a.group)) return;
    const int qt = (int)qt64;
    const int nkv = ap_blocks(s, a.group, qt);
    int64_t before = 0;
    for (int t = tid; t < qt; t += 256) before += ap_blocks(s, a.group, t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lane == 0) s_before[warp] = before;
    __syncthreads();
    before = 0;
    for (int w = 0; w < 8; ++w) before += s_before[w];
    const int64_t total = a.base[a.bt.n_seqs], first = a.base[b];
    const int64_t ub = first + (a.base[b + 1] - first) / a.kv.hk * h + before;
    int c0 = 0, c1 = -1;
    if (nkv > 0) {
        const int64_t active = ap_active(total, ctas);
        c0 = (int)(((ub + 1) * active - 1) / total);
        c1 = (int)(((ub + nkv) * active - 1) / total);
        if (c0 == c1) return;
    }
    const int64_t R = (int64_t)qt * AP_ROWS + tid;
    if (R >= (int64_t)s.n * a.group) return;
    const int tok = (int)(R / a.group), g = (int)(R - (int64_t)tok * a.group);
    float m = -INFINITY, l = 0.0f;
    for (int k = c0; k <= c1; ++k)
        m = fmaxf(m, a.part_ml[(2 * (int64_t)k + (k == c0 ? 1 : 0)) * AP_ROWS + tid].x);
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    const int col = blockIdx.z * 16;
    for (int k = c0; k <= c1; ++k) {
        const int64_t part = (2 * (int64_t)k + (k == c0 ? 1 : 0)) * AP_ROWS;
        const float2 ml = a.part_ml[part + tid];
        const float f = ml.x == -INFINITY ? 0.0f : fast_exp2(ml.x - m);
        l += ml.y * f;
        const float4 *src = reinterpret_cast<const float4 *>(a.part + part * D) + (col / 4) * AP_ROWS + tid;
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
                                           ((int64_t)h * a.group + g) * D + col);
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e] = bf16_rn_bits(acc[2 * e] * inv) | (bf16_rn_bits(acc[2 * e + 1] * inv) << 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

} // namespace bitnet
