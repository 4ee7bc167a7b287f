// kv_append.cuh -- appending keys and values to the paged 8-bit cache, with the
// position rotation of queries and keys on the way.
//
// The step of a page is the largest |x| / 127 of all its tokens, so everything that
// decides it meets in one team of warps (one warp per 16 tokens of a page): the rows
// are read once, stay in registers across the maximum, and codes and step are
// written by the same threads.  No atomics and no second pass over q, k, v.  A CTA
// holds as many teams, for neighbouring kv heads, as fit (a CTA per
// 16-token page and head spent its time on being launched: 145 us for 17 k tokens
// of 16 heads, against 43 us for the bytes).  The team of a key also rotates the
// query heads of its group for the same tokens: they need the same row lookup, and
// the cosines and sines, twice a bf16 row's bytes, serve all of them from registers.
//
// Bound by HBM: q, k, v are read once, rotated queries and codes written once.
// Measured: 17 k ragged tokens of 16 heads of 64, fp32, 57 us (4.9 TB/s); a prompt of
// 4096 tokens, 20/5 heads of 128, bf16, 20 us (3.0 TB/s: 320 teams of four warps with
// queries, each a chain of load rounds).
#pragma once

#include "kv_common.cuh"

namespace bitnet {

// Warps per CTA for pages of 2^shift tokens: a page of 128 needs a team of eight, and
// small CTAs share the SMs more evenly.
constexpr __host__ __device__ int ka_warps(int page_shift) { return page_shift == 7 ? 8 : 4; }

struct AppendArgs {
    KvView kv;
    BatchView bt;
    const void *q, *k, *v;            // rows of dtype elements, strides in elements
    int64_t q_stride, k_stride, v_stride;
    const float *rope;                // [rope_len][D] or null
    int64_t rope_len;
    uint16_t *q_out;                  // bf16
    int64_t q_out_stride;
    int group;                        // query heads per kv head (0: no queries)
};

// Items (pages that get new tokens) are numbered so that sequence b's start at
// base(b) = min(q_start[b], q_start[b] / P + 2 b): n new tokens touch at most n
// and at most n / P + 2 pages, and base grows by at least as much from b to
// b + 1, so an item's sequence is found without a prefix sum over the batch.
__host__ BITNET_DEVINL int64_t ka_base(int64_t q0, int64_t b, int page_shift)
{
    const int64_t byp = (q0 >> page_shift) + 2 * b;
    return q0 < byp ? q0 : byp;
}

// Sixteen elements of a row as they lie in memory: eight at elem, eight at elem + D / 2.
template <bool F32, int D>
BITNET_DEVINL void ka_raw(const void *base, int64_t elem, uint4 (&w)[F32 ? 4 : 2])
{
    constexpr int size = F32 ? 4 : 2;
    const char *p = static_cast<const char *>(base) + elem * size;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < size / 2; ++i)
            w[h * (size / 2) + i] = reinterpret_cast<const uint4 *>(p + h * (D / 2) * size)[i];
}

template <bool F32>
BITNET_DEVINL void ka_values(const uint4 (&w)[F32 ? 4 : 2], float (&x)[16])
{
    constexpr int N = F32 ? 4 : 8; // elements of a 16-byte chunk
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (F32) {
                x[N * i + e] = __uint_as_float(v[e]);
            } else {
                x[N * i + 2 * e] = bf16_bits_lo(v[e]);
                x[N * i + 2 * e + 1] = bf16_bits_hi(v[e]);
            }
        }
    }
}

template <bool F32, int D>
BITNET_DEVINL void ka_load(const void *base, int64_t elem, float (&x)[16])
{
    uint4 w[F32 ? 4 : 2];
    ka_raw<F32, D>(base, elem, w);
    ka_values<F32>(w, x);
}

BITNET_DEVINL void ka_load8(const float *p, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
    }
}

BITNET_DEVINL void ka_rotate(const float (&c)[8], const float (&s)[8], float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(x[8 + i], s[i]));
        x[8 + i] = __fadd_rn(__fmul_rn(x[8 + i], c[i]), __fmul_rn(x[i], s[i]));
        x[i] = a;
    }
}

// rne(x / step) clamped to [-127, 127]; step > 0.
BITNET_DEVINL int ka_code(float x, float step)
{
    const int c = __float2int_rn(__fdiv_rn(x, step));
    return max(-127, min(127, c));
}

// Codes of sixteen elements, rne(fl(x / step)) each, four to a word.  x times the rounded
// inverse is within 127 * 3 * 2^-24 < 3e-5 of fl(x / step), so where it is not within 1e-4
// of the middle between two integers both round alike; else (one set of sixteen in 300), and
// for steps near the subnormal ones, the division itself decides.  (Dividing always: 81 us
// for 17 k tokens of 16 heads.)
BITNET_DEVINL void ka_codes(const float (&x)[16], float step, float inv, uint32_t (&w)[4])
{
    constexpr float magic = 12582912.0f; // 1.5 * 2^23: the sum's low byte is the nearest integer
    bool exact = step < 1e-30f;
    if (!exact) {
        float off = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t n[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = __fmul_rn(x[4 * i + e], inv), r = __fadd_rn(t, magic);
                off = fmaxf(off, fabsf(__fsub_rn(t, __fsub_rn(r, magic))));
                n[e] = __float_as_uint(r);
            }
            w[i] = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
        }
        exact = off > 0.4999f;
    }
    if (exact) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack4_s8(ka_code(x[4 * i], step), ka_code(x[4 * i + 1], step), ka_code(x[4 * i + 2], step),
                            ka_code(x[4 * i + 3], step));
    }
}

// D: head dimension; P: page size.
template <bool F32, int D, int P>
__global__ void __launch_bounds__(P == 128 ? 256 : 128, (D == 64 ? 6 : 4) / (P == 128 ? 2 : 1))
    k_kv_append(const AppendArgs a)
{
    constexpr int KA_WARPS = P == 128 ? 8 : 4, KA_THREADS = KA_WARPS * 32;
    constexpr int TEAM = P / 16;             // warps per (page, kv head)
    constexpr int LPR = D / 16;              // lanes per row, sixteen elements each
    constexpr int RPP = 32 / LPR;            // rows a warp holds side by side
    constexpr int NR = 16 / RPP;             // passes that hold the warp's 16 tokens
    constexpr int SHIFT = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    __shared__ int s_seq;
    __shared__ float s_max[KA_WARPS];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y * (KA_WARPS / TEAM) + warp / TEAM; // kv head of this team
    const bool is_k = blockIdx.z == 0, mine = h < a.kv.hk;
    if (tid == 0) s_seq = -1;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();

    // the sequence whose item range holds this CTA's item
    const int64_t item = blockIdx.x;
    for (int b = tid; b < a.bt.n_seqs; b += KA_THREADS) {
        const int64_t lo = a.bt.q_start[b], hi = a.bt.q_start[b + 1];
        if (lo < 0 || hi < lo || hi > a.bt.T) {
            record_batch_error();
            continue;
        }
        if (item >= ka_base(lo, b, SHIFT) && item < ka_base(hi, b + 1, SHIFT)) s_seq = b;
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const SeqInfo sq = seq_info(a.bt, SHIFT, b);
    const int first = sq.len - sq.n;
    const int64_t j64 = (first >> SHIFT) + (item - ka_base(sq.q0, b, SHIFT));
    if (!sq.ok || sq.n == 0 || j64 > ((sq.len - 1) >> SHIFT)) return;
    const int j = (int)j64;
    const int lo = max(first, j << SHIFT), hi = min(sq.len, (j + 1) << SHIFT); // positions of the new tokens here
    const int nn = hi - lo;
    if (a.rope && hi > a.rope_len) {
        if (tid == 0) record_batch_error();
        return;
    }
    const int64_t row0 = sq.q0 + (lo - first);
    const int page = page_of(a.kv, a.bt, b, j);
    const int col = (lane % LPR) * 8;
    const int r0 = (warp % TEAM) * 16 + lane / LPR; // this thread's rows: r0, r0 + RPP, ...

    // queries of the key's group: several heads' loads at a time, or each waits for the one before
    if (is_k && mine && a.group > 0) {
        constexpr int CH = F32 ? 2 : 4;
#pragma unroll 1
        for (int r = r0; r < min(nn, r0 + 16); r += RPP) {
            float c[8], s[8];
            if (a.rope) {
                const float *rope = a.rope + (int64_t)(lo + r) * D + col;
                ka_load8(rope, c);
                ka_load8(rope + D / 2, s);
            }
            const int64_t q = (row0 + r) * a.q_stride + (int64_t)h * a.group * D + col;
            uint16_t *out = a.q_out + (row0 + r) * a.q_out_stride + (int64_t)h * a.group * D + col;
#pragma unroll 1
            for (int g0 = 0; g0 < a.group; g0 += CH) {
                uint4 raw[CH][F32 ? 4 : 2];
#pragma unroll
                for (int g = 0; g < CH; ++g)
                    if (g0 + g < a.group) ka_raw<F32, D>(a.q, q + (g0 + g) * D, raw[g]);
#pragma unroll
                for (int g = 0; g < CH; ++g) {
                    if (g0 + g >= a.group) break;
                    float y[16];
                    ka_values<F32>(raw[g], y);
                    if (a.rope) ka_rotate(c, s, y);
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = bf16_rn_bits(y[2 * e]) | (bf16_rn_bits(y[2 * e + 1]) << 16);
                    *reinterpret_cast<uint4 *>(out + (g0 + g) * D) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(out + (g0 + g) * D + D / 2) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
    }

    // keys or values, rotated, kept until the page's maximum is known
    const void *src = is_k ? a.k : a.v;
    const int64_t stride = is_k ? a.k_stride : a.v_stride;
    float x[NR][16];
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * RPP;
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][e] = 0.0f;
        if (mine && r < nn) ka_load<F32, D>(src, (row0 + r) * stride + (int64_t)h * D + col, x[i]);
    }
    if (is_k && mine && a.rope) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i * RPP;
            if (r >= nn) continue;
            float c[8], s[8];
            const float *rope = a.rope + (int64_t)(lo + r) * D + col;
            ka_load8(rope, c);
            ka_load8(rope + D / 2, s);
            ka_rotate(c, s, x[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(x[i][e]));
    const int64_t head = (int64_t)page * a.kv.hk + h;
    const int off = lo & (P - 1); // slot of the first new token; tokens before it stay
    const bool write = mine && page >= 0;
    float *step_p = (is_k ? a.kv.k_step : a.kv.v_step) + head;
    const float old = write && off > 0 ? *step_p : 0.0f;
    mx = warp_max(mx);
    if constexpr (TEAM > 1) {
        if (lane == 0) s_max[warp] = mx;
        __syncthreads(); // also: the whole team has read the old step
#pragma unroll
        for (int w = 0; w < TEAM; ++w) mx = fmaxf(mx, s_max[warp / TEAM * TEAM + w]);
    }
    if (!write) return;
    int8_t *codes = (is_k ? a.kv.k : a.kv.v) + head * P * D;
    const float step = fmaxf(old, __fmul_rn(mx, 1.0f / 127.0f));
    const float inv = __frcp_rn(step);
    const int tl = tid % (TEAM * 32); // thread of the team
    if (step > old) {
        __syncwarp();
        if (tl == 0) *step_p = step;
        if (off > 0) { // the page's earlier codes in the new step
            const float ratio = __fdiv_rn(old, step);
            for (int w4 = tl; w4 < off * (D / 4); w4 += TEAM * 32) {
                uint32_t *p = reinterpret_cast<uint32_t *>(codes) + w4;
                const uint32_t w = *p;
                int q4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int v = (int)(int8_t)(w >> (8 * e));
                    q4[e] = __float2int_rn(__fmul_rn((float)v, ratio));
                }
                *p = pack4_s8(q4[0], q4[1], q4[2], q4[3]);
            }
        }
    } else if (tl == 0 && off == 0) {
        *step_p = step; // a fresh page of zeros
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * RPP;
        if (r >= nn) continue;
        uint32_t w[4] = {0, 0, 0, 0};
        if (step > 0.0f) ka_codes(x[i], step, inv, w);
        int8_t *dst = codes + (off + r) * D + col;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(dst + D / 2) = make_uint2(w[2], w[3]);
    }
}

// Rotation table: angles, cosines and sines in fp64 (a position of 2^20 times a
// frequency of 1 leaves fp32 no bits for the fraction of a turn).
__global__ void __launch_bounds__(256) k_rope_table(double theta, int64_t n, int d, float *table)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int half = d / 2;
    const int64_t p = i / half;
    const int j = (int)(i % half);
    const double w = pow(theta, -2.0 * j / d);
    double s, c;
    sincos((double)p * w, &s, &c);
    table[p * d + j] = (float)c;
    table[p * d + half + j] = (float)s;
}

} // namespace bitnet
