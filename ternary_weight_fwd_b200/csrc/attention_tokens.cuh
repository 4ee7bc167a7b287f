// attention_tokens.cuh -- attention of few new tokens per sequence over the
// paged 8-bit cache (decoding, verification of drafts): at most 32 query rows
// (new tokens x query heads of the group) per sequence and kv head.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(c (q_r . k_j) - m_r),
//   c = scale * log2(e), k = code * k_step, v = code * v_step
//
// Bound by HBM: the codes of K and V are read once (2 D bytes per cached token
// and kv head; everything else is small).  The work is the list of all
// (sequence, kv head, chunk of 128 tokens) in that order, cut into equal
// contiguous shares, one per CTA (one CTA per SM), so ragged batches and single
// long sequences load every SM alike.  A share's partial softmax of a (sequence,
// kv head) that it does not hold whole goes to the workspace (at most two per
// CTA) and k_attention_join adds them up in the order of the CTAs: no atomics,
// the result does not depend on timing.
//
// Within a CTA a producer warp streams chunks through a ring in shared memory by
// TMA (16-token boxes: one page each, whatever the page size) and eight warps
// take 16 tokens each, with running maxima and sums of their own, joined once
// per (sequence, kv head).  The products run on mma.sync m16n8k16 in fp16 with
// fp32 sums: codes are exact in fp16 (integers up to 128; the byte goes under
// the exponent of 1024 and 1152 is subtracted), queries are brought into fp16's
// range by a power of two per row.  K and V fragments are read from the ring in
// the layout that the bytes already have: an order of the contraction index and
// of the output columns can be chosen freely, so a lane takes 16 consecutive
// bytes of a key (K) or of a value (V).
#pragma once

#include <cuda_fp16.h>

#include "kv_common.cuh"

namespace bitnet {

constexpr int AT_CHUNK = 128;   // tokens per ring stage
constexpr int AT_GROUP = 16;    // tokens per warp and stage, and per TMA box
constexpr int AT_WARPS = 8;     // consumer warps
constexpr int AT_THREADS = (AT_WARPS + 1) * 32;
constexpr int AT_STAGES = 5;
constexpr int AT_MAX_ROWS = 32; // query rows per (sequence, kv head)
constexpr int AT_MAX_CTAS = 160;
constexpr int AT_MIN_UNITS = 2; // chunks worth a CTA of their own

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
    int64_t *base;     // [n_seqs + 1] first unit of each sequence
};

constexpr __host__ __device__ int at_smem(int d, int mt)
{
    return 1024 + AT_STAGES * 2 * AT_CHUNK * d + 16 * mt * (2 * d + 16) + AT_WARPS * 16 * mt * (36 * 4 + 8) +
           16 * mt * 8 + 1024;
}

// 3-D tiled tensor copy global -> shared (no multicast); c0 is 0 here.
BITNET_DEVINL void tma_load_3d(uint32_t dst_smem, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2,
                               uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst_smem),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
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

BITNET_DEVINL int attn_chunks(const AttnSeq &s) { return s.n > 0 ? (s.len + AT_CHUNK - 1) / AT_CHUNK : 0; }

// CTAs that share `units` chunks.
BITNET_DEVINL int64_t attn_active(int64_t units, int ctas)
{
    const int64_t want = (units + AT_MIN_UNITS - 1) / AT_MIN_UNITS;
    return want < ctas ? want : ctas;
}

// Walks the unit list: sequence of unit u, given a sequence at or before it.
struct UnitIter {
    int b;
    int64_t base; // first unit of sequence b
    AttnSeq s;
    int nc;       // chunks per kv head

    BITNET_DEVINL void seek(const AttnArgs &a, int64_t u)
    {
        while (u >= base + (int64_t)nc * a.kv.hk && b + 1 < a.bt.n_seqs) {
            base += (int64_t)nc * a.kv.hk;
            ++b;
            s = attn_seq(a, b);
            nc = attn_chunks(s);
        }
    }
};

// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows as the TMA's
// swizzle leaves it (128-byte swizzle for D = 128, 64-byte for D = 64).
template <int D>
BITNET_DEVINL uint32_t kv_swz(int r, int c)
{
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, int MT>
__global__ void __launch_bounds__(AT_THREADS, 1)
    k_attention_tokens(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const AttnArgs a)
{
    constexpr int NT = D / 8;               // output column tiles
    constexpr int ROWS = 16 * MT;
    constexpr uint32_t TILE = AT_CHUNK * D; // bytes of K (or V) per stage
    constexpr int QROW = 2 * D + 16;        // bytes of a query row in shared memory
    constexpr int MROW = 36;                // floats of a row of the join buffer

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + AT_STAGES;
    int64_t *s_u = reinterpret_cast<int64_t *>(empty + AT_STAGES); // total units, first sequence's base
    int *s_b = reinterpret_cast<int *>(s_u + 2);
    float *s_step = reinterpret_cast<float *>(s_b + 4); // [stages][2][8]
    int64_t *s_scan = reinterpret_cast<int64_t *>(smem + 640); // [9] warp sums
    unsigned char *ring = smem + 1024;
    unsigned char *s_q = ring + AT_STAGES * 2 * TILE;
    float *s_join = reinterpret_cast<float *>(s_q + ROWS * QROW);       // [8 warps][ROWS][36]
    float2 *s_ml = reinterpret_cast<float2 *>(s_join + AT_WARPS * ROWS * MROW); // [8][ROWS]
    float *s_fac = reinterpret_cast<float *>(s_ml + AT_WARPS * ROWS);   // [ROWS] score factor
    int *s_lim = reinterpret_cast<int *>(s_fac + ROWS);                 // [ROWS] last visible position

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < AT_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], AT_WARPS);
        }
        fence_mbarrier_init();
    }
    if (tid == AT_WARPS * 32) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- total units, this CTA's share and the sequence it starts in ----
    const int per = (a.bt.n_seqs + AT_THREADS - 1) / AT_THREADS;
    const int b_lo = min(a.bt.n_seqs, tid * per), b_hi = min(a.bt.n_seqs, b_lo + per);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += (int64_t)attn_chunks(attn_seq(a, b)) * a.kv.hk;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w <= AT_WARPS; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int64_t active = attn_active(total, gridDim.x);
    const bool idle = blockIdx.x >= active;
    const int64_t u0 = idle ? 0 : total * blockIdx.x / active, u1 = idle ? 0 : total * (blockIdx.x + 1) / active;
    if (blockIdx.x == 0) { // the join kernel reads the units' bases
        int64_t at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            a.base[b] = at;
            at += (int64_t)attn_chunks(attn_seq(a, b)) * a.kv.hk;
        }
        if (tid == 0) a.base[a.bt.n_seqs] = total;
    }
    if (idle) return;
    if (u0 >= before && u0 < before + mine) {
        int64_t at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            const int64_t un = (int64_t)attn_chunks(attn_seq(a, b)) * a.kv.hk;
            if (u0 < at + un) {
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
    it.s = attn_seq(a, it.b);
    it.nc = attn_chunks(it.s);

    if (warp == AT_WARPS) {
        // ---------------- producer ----------------
        // A batch of four chunks: lane = chunk * 8 + 16-token group.  Page ids are
        // fetched two batches ahead and steps one batch ahead of their copies.
        const int sub = lane >> 3, grp = lane & 7;
        int page1 = -1, row1 = 0; // next batch
        bool valid1 = false;
        auto fetch = [&](int64_t u, int &page, int &row, bool &valid) {
            valid = false;
            page = -1;
            row = 0;
            if (u < u1) {
                it.seek(a, u);
                const int rel = (int)(u - it.base);
                const int h = rel / it.nc, key0 = (rel - h * it.nc) * AT_CHUNK + grp * AT_GROUP;
                if (key0 < it.s.len) {
                    valid = true;
                    page = page_of(a.kv, a.bt, it.b, key0 >> a.kv.page_shift);
                    row = (h << a.kv.page_shift) + (key0 & ((1 << a.kv.page_shift) - 1));
                }
            }
        };
        int page = -1, row = 0;
        bool valid = false;
        fetch(u0 + sub, page, row, valid);
        float ks = 0.0f, vs = 0.0f, ks1 = 0.0f, vs1 = 0.0f;
        auto steps = [&](int pg, int rw, float &k, float &v) {
            k = v = 0.0f;
            if (pg >= 0) {
                const int64_t at = (int64_t)pg * a.kv.hk + (rw >> a.kv.page_shift);
                k = a.kv.k_step[at];
                v = a.kv.v_step[at];
            }
        };
        steps(page, row, ks, vs);
        fetch(u0 + 4 + sub, page1, row1, valid1);
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok; u += 4) {
            steps(page1, row1, ks1, vs1);
            int page2, row2;
            bool valid2;
            fetch(u + 8 + sub, page2, row2, valid2);
#pragma unroll 1
            for (int s = 0; s < 4 && u + s < u1; ++s) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1));
                if (!ok) break;
                const bool here = sub == s && valid;
                if (here) {
                    s_step[stage * 16 + grp] = ks;
                    s_step[stage * 16 + 8 + grp] = vs;
                }
                const int copies = __popc(__ballot_sync(0xffffffffu, here && page >= 0));
                __syncwarp(); // the steps are written before the arrival that shows them
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], copies * 2 * AT_GROUP * D);
                __syncwarp();
                if (here && page >= 0) {
                    const uint32_t dst = smem_u32(ring) + stage * 2 * TILE + grp * AT_GROUP * D;
                    tma_load_3d(dst, &tm_k, 0, row, page, &full[stage]);
                    tma_load_3d(dst + TILE, &tm_v, 0, row, page, &full[stage]);
                }
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == AT_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            page = page1;
            row = row1;
            valid = valid1;
            ks = ks1;
            vs = vs1;
            page1 = page2;
            row1 = row2;
            valid1 = valid2;
        }
        // let every copy this CTA issued land before the CTA can exit
        for (int s = 0; s < AT_STAGES; ++s)
            if (issued & (1u << s)) mbar_wait_drain(&full[s], (last_par >> s) & 1);
        return;
    }

    // ---------------- consumers ----------------
    const int g = lane >> 2, c = lane & 3;
    const int perm_g = (g & 1) ? ((g + 4) & 7) : g; // token of MMA column g: 0 5 2 7 4 1 6 3 (see below)
    const int key_e = 2 * c, key_o = (2 * c + 5) & 7; // tokens of this lane's two score columns
    const uint32_t q_base = smem_u32(s_q), ring_base = smem_u32(ring);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;

    for (int64_t u = u0; u < u1;) {
        it.seek(a, u);
        const int rel = (int)(u - it.base);
        const int h = rel / it.nc, t0 = rel - h * it.nc;
        const int cnt = (int)min((int64_t)(it.nc - t0), u1 - u);
        const int nrow = it.s.n * a.group; // <= ROWS by the host's choice of MT and the check of n
        const int len = it.s.len, first = len - it.s.n;

        // queries of this (sequence, kv head), scaled into fp16's range row by row
        for (int r = warp; r < ROWS; r += AT_WARPS) {
            float x[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e) x[e] = 0.0f;
            const int tok = r / a.group;
            if (r < nrow) {
                const uint16_t *p = a.q + (int64_t)(it.s.q0 + tok) * a.q_stride +
                                    ((int64_t)h * a.group + (r - tok * a.group)) * D + lane * (D / 32);
                if constexpr (D == 128) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    x[0] = bf16_bits_lo(w.x);
                    x[1] = bf16_bits_hi(w.x);
                    x[2] = bf16_bits_lo(w.y);
                    x[3] = bf16_bits_hi(w.y);
                } else {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
                    x[0] = bf16_bits_lo(w);
                    x[1] = bf16_bits_hi(w);
                }
            }
            float mx = 0.0f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) mx = fmaxf(mx, fabsf(x[e]));
            mx = warp_max(mx);
            const float f = half_range_factor(mx);
            uint32_t *dst = reinterpret_cast<uint32_t *>(s_q + r * QROW + lane * (D / 16));
#pragma unroll
            for (int e = 0; e < D / 64; ++e) dst[e] = pack_half2(x[2 * e] * f, x[2 * e + 1] * f);
            if (lane == 0) {
                s_fac[r] = a.scale_log2 / f;
                s_lim[r] = r < nrow ? first + tok : -1;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(AT_WARPS * 32) : "memory");

        float o[MT][NT][4], m[MT][2], l[MT][2], fac[MT][2];
        int lim[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int n = 0; n < NT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[t][e] = -INFINITY;
                l[t][e] = 0.0f;
                fac[t][e] = s_fac[16 * t + 8 * e + g];
                lim[t][e] = s_lim[16 * t + 8 * e + g];
            }
        }
        float unit = 0.0f, inv_unit = 0.0f; // o is in units of this power of two; 0: not chosen yet

        for (int i = 0; i < cnt; ++i) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[stage], phase));
            const int key0 = (t0 + i) * AT_CHUNK + warp * AT_GROUP;
            if (ok && key0 < len) {
                const float ks = s_step[stage * 16 + warp], vs = s_step[stage * 16 + 8 + warp];
                const uint32_t kb = ring_base + stage * 2 * TILE + warp * AT_GROUP * D, vb = kb + TILE;
                float s[MT][2][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) s[t][j][0] = s[t][j][1] = s[t][j][2] = s[t][j][3] = 0.0f;
                // scores.  Contraction step 4 hh + w takes elements 16 (c + 4 hh) + 4 w .. + 3 of
                // lane column c.  Column g of MMA j is token 8 j + perm(g): the two tokens of a
                // shared-memory wavefront differ in bit 2, so their swizzled chunks differ.
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh) {
                    uint4 kw[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) kw[j] = lds128(kb + kv_swz<D>(8 * j + perm_g, c + 4 * hh));
                    uint4 qa[MT][4]; // rows g and g + 8, 16 elements each
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t qp = q_base + (16 * t + 8 * e + g) * QROW + (c + 4 * hh) * 32;
                            qa[t][2 * e] = lds128(qp);
                            qa[t][2 * e + 1] = lds128(qp + 16);
                        }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t b0[2], b1[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t word = w == 0 ? kw[j].x : w == 1 ? kw[j].y : w == 2 ? kw[j].z : kw[j].w;
                            codes_to_half(word ^ 0x80808080u, b0[j], b1[j]);
                        }
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 lo = qa[t][w >> 1], hi = qa[t][2 + (w >> 1)];
                            const uint32_t a0 = (w & 1) ? lo.z : lo.x, a2 = (w & 1) ? lo.w : lo.y;
                            const uint32_t a1 = (w & 1) ? hi.z : hi.x, a3 = (w & 1) ? hi.w : hi.y;
#pragma unroll
                            for (int j = 0; j < 2; ++j) mma_f16(s[t][j], a0, a1, a2, a3, b0[j], b1[j]);
                        }
                    }
                }
                // softmax: lane holds rows g, g + 8 x tokens key_e, key_o, 8 + key_e, 8 + key_o
                const bool masked = key0 + AT_GROUP - 1 > first;
                bool grown = false;
                float mx[MT][2];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = fac[t][e] * ks;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float &x0 = s[t][j][2 * e], &x1 = s[t][j][2 * e + 1];
                            x0 *= f;
                            x1 *= f;
                            if (masked) {
                                if (key0 + 8 * j + key_e > lim[t][e]) x0 = -INFINITY;
                                if (key0 + 8 * j + key_o > lim[t][e]) x1 = -INFINITY;
                            }
                        }
                        float v = fmaxf(fmaxf(s[t][0][2 * e], s[t][0][2 * e + 1]),
                                        fmaxf(s[t][1][2 * e], s[t][1][2 * e + 1]));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                        mx[t][e] = fmaxf(v, m[t][e]);
                        grown |= mx[t][e] > m[t][e];
                    }
                // o follows the running maximum, and keeps units near the current page's v_step
                // (weights times v_step / unit stay in fp16's range whatever the steps of other pages)
                float r = vs * inv_unit;
                const bool move = vs > 0.0f && !(r >= 0x1p-4f && r <= 0x1p8f);
                if (__any_sync(0xffffffffu, grown) || move) {
                    float us = 1.0f;
                    if (move) {
                        const float to = unit > 0.0f ? fmaxf(pow2_floor(vs), unit * 0x1p-60f) : pow2_floor(vs);
                        us = unit > 0.0f ? unit / to : 1.0f;
                        unit = to;
                        inv_unit = 1.0f / to;
                        r = vs * inv_unit;
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float al = mx[t][e] > m[t][e] ? fast_exp2(m[t][e] - mx[t][e]) : 1.0f;
                            m[t][e] = mx[t][e];
                            l[t][e] *= al;
                            const float ou = al * us;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[t][n][2 * e] *= ou;
                                o[t][n][2 * e + 1] *= ou;
                            }
                        }
                }
                uint32_t pa[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mu = m[t][e] == -INFINITY ? 0.0f : m[t][e];
                        float p[4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            p[2 * j] = fast_exp2(s[t][j][2 * e] - mu);
                            p[2 * j + 1] = fast_exp2(s[t][j][2 * e + 1] - mu);
                        }
                        l[t][e] += (p[0] + p[1]) + (p[2] + p[3]);
                        pa[t][e] = pack_half2(p[0] * r, p[1] * r);
                        pa[t][2 + e] = pack_half2(p[2] * r, p[3] * r);
                    }
                // o += p v.  Lane column g of output tile n is element (D / 8) g + n; contraction
                // indices 2c, 2c + 1 (+ 8) are tokens key_e, key_o (+ 8).
                if (vs > 0.0f) {
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
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        uint32_t bb[2][4]; // [b0, b1][tile 4 w + x]
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = vw[2 * e][w] ^ 0x80808080u, y = vw[2 * e + 1][w] ^ 0x80808080u;
                            codes_to_half(__byte_perm(x, y, 0x5140), bb[e][0], bb[e][1]);
                            codes_to_half(__byte_perm(x, y, 0x7362), bb[e][2], bb[e][3]);
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int t = 0; t < MT; ++t)
                                mma_f16(o[t][4 * w + x], pa[t][0], pa[t][1], pa[t][2], pa[t][3], bb[0][x], bb[1][x]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == AT_STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }

        // ---- join the eight warps ----
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 1);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 2);
                if (c == 0) s_ml[warp * ROWS + 16 * t + 8 * e + g] = make_float2(m[t][e], l[t][e]);
            }
        asm volatile("bar.sync 1, %0;" ::"n"(AT_WARPS * 32) : "memory");
        float wf[MT][2]; // this warp's weight of rows g, g + 8
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mm = -INFINITY;
                for (int w = 0; w < AT_WARPS; ++w) mm = fmaxf(mm, s_ml[w * ROWS + 16 * t + 8 * e + g].x);
                wf[t][e] = m[t][e] == -INFINITY ? 0.0f : fast_exp2(m[t][e] - mm) * unit;
            }
        const bool whole = cnt == it.nc;
        const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        // thread -> (row, column tile) of the result
        const int jr = tid >> 3, jn = tid & 7;
        float jm = -INFINITY, jl = 0.0f;
        if (jr < ROWS && jr < nrow) {
            for (int w = 0; w < AT_WARPS; ++w) jm = fmaxf(jm, s_ml[w * ROWS + jr].x);
            if (jm != -INFINITY)
                for (int w = 0; w < AT_WARPS; ++w) {
                    const float2 x = s_ml[w * ROWS + jr];
                    jl += x.y * fast_exp2(x.x - jm);
                }
            if (!whole && jn == 0) a.part_ml[(int64_t)slot * ROWS + jr] = make_float2(jm, jl);
        }
        const float inv = jl > 0.0f ? 1.0f / jl : 0.0f;
        const int jtok = jr / a.group;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            if (w) asm volatile("bar.sync 1, %0;" ::"n"(AT_WARPS * 32) : "memory");
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (16 * t + 8 * e + g >= nrow) continue;
                    float *dst = s_join + (warp * ROWS + 16 * t + 8 * e + g) * MROW;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<float4 *>(dst + (2 * c + k) * 4) =
                            make_float4(o[t][4 * w][2 * e + k] * wf[t][e], o[t][4 * w + 1][2 * e + k] * wf[t][e],
                                        o[t][4 * w + 2][2 * e + k] * wf[t][e], o[t][4 * w + 3][2 * e + k] * wf[t][e]);
                }
            asm volatile("bar.sync 1, %0;" ::"n"(AT_WARPS * 32) : "memory");
            if (jr < ROWS && jr < nrow) {
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < AT_WARPS; ++k) {
                    const float4 y = *reinterpret_cast<const float4 *>(s_join + (k * ROWS + jr) * MROW + jn * 4);
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                const int d = (D / 8) * jn + 4 * w;
                if (whole) {
                    uint16_t *p = a.out + (int64_t)(it.s.q0 + jtok) * a.out_stride +
                                  ((int64_t)h * a.group + (jr - jtok * a.group)) * D + d;
                    *reinterpret_cast<uint2 *>(p) =
                        make_uint2(bf16_rn_bits(x.x * inv) | (bf16_rn_bits(x.y * inv) << 16),
                                   bf16_rn_bits(x.z * inv) | (bf16_rn_bits(x.w * inv) << 16));
                } else {
                    *reinterpret_cast<float4 *>(a.part + ((int64_t)slot * ROWS + jr) * D + d) = x;
                }
            }
        }
        u += cnt;
        // the next pass writes s_q, s_fac, s_lim (not read any more) and only after its own
        // barrier anything that this one still reads
    }
}

// Joins the parts of every (sequence, kv head) that more than one CTA shared,
// and writes zeros for rows of sequences without cached tokens.  A warp per row;
// parts are added in the order of the CTAs.
template <int D>
__global__ void __launch_bounds__(128) k_attention_join(const AttnArgs a, int rows, int ctas)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.kv.hk, h = blockIdx.x - b * a.kv.hk;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5);
    const AttnSeq s = attn_seq(a, b);
    if (r >= s.n * a.group) return;
    const int64_t total = a.base[a.bt.n_seqs], base = a.base[b];
    const int nc = attn_chunks(s);
    const int tok = r / a.group;
    uint16_t *p = a.out + (int64_t)(s.q0 + tok) * a.out_stride + ((int64_t)h * a.group + (r - tok * a.group)) * D +
                  lane * (D / 32);
    float acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
    float inv = 0.0f;
    if (nc > 0) {
        const int64_t active = attn_active(total, ctas);
        const int64_t ub = base + (int64_t)h * nc, ue = ub + nc - 1;
        const int c0 = (int)(((ub + 1) * active - 1) / total), c1 = (int)(((ue + 1) * active - 1) / total);
        if (c0 == c1) return; // one CTA held it whole and wrote the result
        float m = -INFINITY;
        for (int k = c0 + lane; k <= c1; k += 32)
            m = fmaxf(m, a.part_ml[(int64_t)(2 * k + (k == c0 ? 1 : 0)) * rows + r].x);
        m = warp_max(m);
        if (m != -INFINITY) {
            float l = 0.0f;
            for (int k0 = c0; k0 <= c1; k0 += 32) {
                const int k = k0 + lane;
                float f = 0.0f;
                if (k <= c1) {
                    const float2 ml = a.part_ml[(int64_t)(2 * k + (k == c0 ? 1 : 0)) * rows + r];
                    f = fast_exp2(ml.x - m);
                    l += ml.y * f;
                }
                const int cnt = min(32, c1 - k0 + 1);
                for (int i = 0; i < cnt; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
                    const float *src =
                        a.part + ((int64_t)(2 * (k0 + i) + (k0 + i == c0 ? 1 : 0)) * rows + r) * D + lane * (D / 32);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) acc[e] += src[e] * fi;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            inv = 1.0f / l;
        }
    }
    uint32_t w[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
        w[e] = bf16_rn_bits(acc[2 * e] * inv) | (bf16_rn_bits(acc[2 * e + 1] * inv) << 16);
    if constexpr (D == 128)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = w[0];
}

} // namespace bitnet
