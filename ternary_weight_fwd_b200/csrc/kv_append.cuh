// kv_append.cuh -- appending keys and values to the paged 8-bit cache, with the
// position rotation of queries and keys on the way.
//
// One CTA per (page that gets new tokens, kv head, K or V): the step of a page
// is the largest |x| / 127 of all its tokens, so everything that decides it
// meets in one CTA, the rows are read once, stay in registers across the
// maximum, and codes and step are written by the same threads.  No atomics and
// no second pass over q, k, v.  The K CTA of a kv head also rotates the query
// heads of its group for the same tokens: they need the same row lookup and the
// same cosines.
//
// Bound by HBM: q, k, v are read once, rotated queries and codes written once.
#pragma once

#include "kv_common.cuh"

namespace bitnet {

constexpr int KA_THREADS = 256;
constexpr int KA_WARPS = KA_THREADS / 32;

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

// Four elements of one row: x[0..1] at j, x[2..3] at j + D / 2 (j = 2 * lane of the row).
template <bool F32, int D>
BITNET_DEVINL void ka_load(const void *base, int64_t elem, float (&x)[4])
{
    if constexpr (F32) {
        const float *p = static_cast<const float *>(base) + elem;
        const float2 a = *reinterpret_cast<const float2 *>(p);
        const float2 b = *reinterpret_cast<const float2 *>(p + D / 2);
        x[0] = a.x;
        x[1] = a.y;
        x[2] = b.x;
        x[3] = b.y;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + elem;
        const uint32_t a = *reinterpret_cast<const uint32_t *>(p);
        const uint32_t b = *reinterpret_cast<const uint32_t *>(p + D / 2);
        x[0] = bf16_bits_lo(a);
        x[1] = bf16_bits_hi(a);
        x[2] = bf16_bits_lo(b);
        x[3] = bf16_bits_hi(b);
    }
}

template <int D>
BITNET_DEVINL void ka_rotate(const float *rope_row, int j, float (&x)[4])
{
    const float2 c = *reinterpret_cast<const float2 *>(rope_row + j);
    const float2 s = *reinterpret_cast<const float2 *>(rope_row + D / 2 + j);
    const float a0 = __fsub_rn(__fmul_rn(x[0], c.x), __fmul_rn(x[2], s.x));
    const float a1 = __fsub_rn(__fmul_rn(x[1], c.y), __fmul_rn(x[3], s.y));
    const float b0 = __fadd_rn(__fmul_rn(x[2], c.x), __fmul_rn(x[0], s.x));
    const float b1 = __fadd_rn(__fmul_rn(x[3], c.y), __fmul_rn(x[1], s.y));
    x[0] = a0;
    x[1] = a1;
    x[2] = b0;
    x[3] = b1;
}

// rne(x / step) clamped to [-127, 127]; step > 0.
BITNET_DEVINL int ka_code(float x, float step)
{
    const int c = __float2int_rn(__fdiv_rn(x, step));
    return max(-127, min(127, c));
}

// D: head dimension; P: page size.
template <bool F32, int D, int P>
__global__ void __launch_bounds__(KA_THREADS) k_kv_append(const AppendArgs a)
{
    constexpr int LPR = D / 4;               // lanes per row, four elements each
    constexpr int RPW = 32 / LPR;            // rows a warp holds side by side
    constexpr int RSTEP = KA_WARPS * RPW;    // rows per pass of the CTA
    constexpr int NR = P / RSTEP;            // passes that hold a whole page
    constexpr int SHIFT = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    __shared__ int s_seq;
    __shared__ float s_max[KA_WARPS];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y;
    const bool is_k = blockIdx.z == 0;
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
    const int sub = lane / LPR, l = lane % LPR, col = 2 * l;
    const int r0 = warp * RPW + sub; // this thread's rows: r0, r0 + RSTEP, ...

    const int page = page_of(a.kv, a.bt, b, j);
    if (page >= 0) {
        const int64_t head = (int64_t)page * a.kv.hk + h;
        int8_t *codes = (is_k ? a.kv.k : a.kv.v) + head * P * D;
        float *step_p = (is_k ? a.kv.k_step : a.kv.v_step) + head;
        const int off = lo & (P - 1); // slot of the first new token; tokens before it stay
        const float old = off > 0 ? *step_p : 0.0f;

        const void *src = is_k ? a.k : a.v;
        const int64_t stride = is_k ? a.k_stride : a.v_stride;
        float x[NR][4];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i * RSTEP;
            x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
            if (r < nn) ka_load<F32, D>(src, (row0 + r) * stride + (int64_t)h * D + col, x[i]);
        }
        if (is_k && a.rope) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = r0 + i * RSTEP;
                if (r < nn) ka_rotate<D>(a.rope + (int64_t)(lo + r) * D, col, x[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[i][e]));
        mx = warp_max(mx);
        if (lane == 0) s_max[warp] = mx;
        __syncthreads(); // also: every thread has read the old step
        mx = s_max[0];
#pragma unroll
        for (int w = 1; w < KA_WARPS; ++w) mx = fmaxf(mx, s_max[w]);
        const float step = fmaxf(old, __fmul_rn(mx, 1.0f / 127.0f));

        if (step > old) {
            if (tid == 0) *step_p = step;
            if (off > 0) { // the page's earlier codes in the new step
                const float ratio = __fdiv_rn(old, step);
                for (int c = tid; c < off * (D / 4); c += KA_THREADS) {
                    uint32_t *p = reinterpret_cast<uint32_t *>(codes) + c;
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
        } else if (tid == 0 && off == 0) {
            *step_p = step; // a fresh page of zeros
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = r0 + i * RSTEP;
            uint32_t lo2 = 0, hi2 = 0; // two codes each of the row's halves
            if (step > 0.0f) {
                lo2 = pack4_s8(ka_code(x[i][0], step), ka_code(x[i][1], step), 0, 0);
                hi2 = pack4_s8(ka_code(x[i][2], step), ka_code(x[i][3], step), 0, 0);
            }
            // neighbours swap a pair, so that each stores four codes of one half
            const bool odd = l & 1;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo2 : hi2, 1);
            const uint32_t w = odd ? got | (hi2 << 16) : lo2 | (got << 16);
            if (r < nn) {
                const int at = odd ? D / 2 + col - 2 : col;
                *reinterpret_cast<uint32_t *>(codes + (off + r) * D + at) = w;
            }
        }
    }

    if (!is_k || a.group == 0) return;
    // rotated queries of this kv head's group, same tokens
    const int nq = nn * a.group;
    for (int i0 = KA_WARPS * RPW - 1 - r0; i0 < nq; i0 += 4 * RSTEP) {
        float y[4][4];
        int64_t tok[4];
        int hd[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * RSTEP;
            if (i < nq) {
                tok[u] = i / a.group;
                hd[u] = h * a.group + i % a.group;
                ka_load<F32, D>(a.q, (row0 + tok[u]) * a.q_stride + (int64_t)hd[u] * D + col, y[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i0 + u * RSTEP < nq) {
                if (a.rope) ka_rotate<D>(a.rope + (lo + tok[u]) * D, col, y[u]);
                uint16_t *o = a.q_out + (row0 + tok[u]) * a.q_out_stride + (int64_t)hd[u] * D + col;
                *reinterpret_cast<uint32_t *>(o) = bf16_rn_bits(y[u][0]) | (bf16_rn_bits(y[u][1]) << 16);
                *reinterpret_cast<uint32_t *>(o + D / 2) = bf16_rn_bits(y[u][2]) | (bf16_rn_bits(y[u][3]) << 16);
            }
        }
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
