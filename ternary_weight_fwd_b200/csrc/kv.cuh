// kv.cuh -- C ABI of the paged 8-bit key/value cache (bitnet_kv.h): argument
// validation before anything is launched, choice of kernels, launches.  Included
// behind bitnet.cu, whose host helpers it uses.
#pragma once

#include "bitnet_kv.h"
#include "attention_prompt.cuh"
#include "attention_tokens.cuh"
#include "kv_append.cuh"

namespace bitnet {
namespace {

constexpr int64_t kMaxSeqs = 65536;
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 32;
constexpr int kMaxKvHeads = 1024;
constexpr int kMaxGroup = 128;

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int page_shift_of(int page_size)
{
    switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
    }
}

bitnet_status_t check_cache(const bitnet_kv_cache_t *c, const bitnet_kv_batch_t *b, KvView &kv, BatchView &bt)
{
    if (!c || !b) return BITNET_ERR_INVALID_ARG;
    if (!c->k || !c->v || !c->k_step || !c->v_step || !b->page_table || !b->seq_lens || !b->q_start)
        return BITNET_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->n_kv_heads < 1 || b->n_seqs < 1 || b->T < 1 || b->table_width < 1)
        return BITNET_ERR_INVALID_ARG;
    const int shift = page_shift_of(c->page_size);
    if (shift < 0 || (c->head_dim != 64 && c->head_dim != 128) || c->n_kv_heads > kMaxKvHeads ||
        c->num_pages > INT32_MAX || b->n_seqs > kMaxSeqs || b->T > kMaxRows || b->table_width > (INT32_MAX >> shift))
        return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_step) || !aligned4(c->v_step) ||
        !aligned4(b->page_table) || !aligned4(b->seq_lens) || !aligned4(b->q_start))
        return BITNET_ERR_MISALIGNED;
    kv = {c->k, c->v, c->k_step, c->v_step, c->num_pages, c->n_kv_heads, shift};
    bt = {b->page_table, b->seq_lens, b->q_start, b->table_width, b->n_seqs, b->T};
    return BITNET_OK;
}

// Rows of `len` elements of `size` bytes, `stride` elements apart.
bitnet_status_t check_rows(const void *p, int64_t stride, int64_t len, int size)
{
    if (!p) return BITNET_ERR_INVALID_ARG;
    if (stride < len || stride > kMaxStride) return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(p) || (stride * size) % 16 != 0) return BITNET_ERR_MISALIGNED;
    return BITNET_OK;
}

// Whether two row sets of T rows share bytes (row bytes wa, wb; strides in bytes).
// Rows of equal strides may lie side by side; of other strides, overlapping
// ranges count as sharing.
bool rows_share(const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb, int64_t T)
{
    const ByteRange ra = range_of(a, (size_t)((T - 1) * sa + wa)), rb = range_of(b, (size_t)((T - 1) * sb + wb));
    if (!overlaps(ra, rb)) return false;
    if (sa != sb) return true;
    const int64_t d = (int64_t)(((int64_t)(rb.lo - ra.lo)) % sa + sa) % sa; // b's column offset seen from a
    return d < wa || d + wb > sa;
}

// The cache's codes and steps.
struct CacheRanges {
    ByteRange r[4];
    explicit CacheRanges(const bitnet_kv_cache_t &c)
    {
        const size_t steps = (size_t)c.num_pages * c.n_kv_heads;
        const size_t codes = steps * c.page_size * c.head_dim;
        r[0] = range_of(c.k, codes);
        r[1] = range_of(c.v, codes);
        r[2] = range_of(c.k_step, steps * 4);
        r[3] = range_of(c.v_step, steps * 4);
    }
    bool hit(ByteRange x) const
    {
        return overlaps(x, r[0]) || overlaps(x, r[1]) || overlaps(x, r[2]) || overlaps(x, r[3]);
    }
    bool apart() const // from one another
    {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < i; ++j)
                if (overlaps(r[i], r[j])) return false;
        return true;
    }
};

// Page table, lengths and row starts: the kernels read them at several places and take what they read for the same.
struct BatchRanges {
    ByteRange r[3];
    explicit BatchRanges(const BatchView &b)
    {
        r[0] = range_of(b.table, (size_t)b.n_seqs * b.width * 4);
        r[1] = range_of(b.lens, (size_t)b.n_seqs * 4);
        r[2] = range_of(b.q_start, ((size_t)b.n_seqs + 1) * 4);
    }
    bool hit(ByteRange x) const { return overlaps(x, r[0]) || overlaps(x, r[1]) || overlaps(x, r[2]); }
};

// From the first to the last byte of T rows of `len` elements of `size` bytes.
inline ByteRange rows_range(const void *p, int64_t stride, int64_t len, int size, int64_t T)
{
    return range_of(p, (size_t)(((T - 1) * stride + len) * size));
}

template <bool F32, int D>
cudaError_t launch_append(const AppendArgs &a, int page_shift, dim3 grid, cudaStream_t stream)
{
    const dim3 block(ka_warps(page_shift) * 32);
    switch (page_shift) {
    case 4: return launch_pdl(k_kv_append<F32, D, 16>, grid, block, 0, stream, a);
    case 5: return launch_pdl(k_kv_append<F32, D, 32>, grid, block, 0, stream, a);
    case 6: return launch_pdl(k_kv_append<F32, D, 64>, grid, block, 0, stream, a);
    default: return launch_pdl(k_kv_append<F32, D, 128>, grid, block, 0, stream, a);
    }
}

// 3-D map of the codes: [page][kv head * token][D], boxes of one page's tokens of one head.
bool encode_codes(CUtensorMap *map, const int8_t *codes, int64_t num_pages, int hk, int page_size, int d)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)hk * page_size, (cuuint64_t)num_pages};
    cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)hk * page_size * d};
    cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)page_size, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t *>(codes), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of the queries: [token][head][D], boxes of 64 elements of one kv head's group and an
// MMA tile's tokens.
bool encode_queries(CUtensorMap *map, const void *q, int64_t T, int64_t stride, int n_heads, int group, int d)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n_heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)ap_tokens(group)};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- attention: choice of kernel and workspace ----------------------------------
struct AttnPlan {
    bool ok;
    int nq; // tiles of 8 rows of the kernel for few tokens (1 or 2); 0: the kernel for prompts
    size_t shared_bytes, ml_bytes, part_bytes; // claim and shared row tiles; parts' maxima and sums; parts
    size_t base_bytes, tile_bytes;             // prompts: units' bases, tiles by cost
    size_t total() const { return shared_bytes + ml_bytes + part_bytes + base_bytes + tile_bytes; }
};

AttnPlan attn_plan(int64_t n_seqs, int64_t T, int64_t n_heads, int64_t hk, int d, int64_t max_new)
{
    AttnPlan p = {};
    if (n_seqs < 1 || n_seqs > kMaxSeqs || T < 1 || T > kMaxRows || hk < 1 || hk > kMaxKvHeads || n_heads < 1 ||
        n_heads % hk != 0 || n_heads / hk > kMaxGroup || (d != 64 && d != 128) || max_new < 1 || max_new > T)
        return p;
    const int64_t rows = n_heads / hk * max_new;
    p.nq = rows <= 8 ? 1 : rows <= AT_MAX_ROWS ? 2 : 0;
    const size_t part_rows = (size_t)2 * AT_MAX_CTAS * (p.nq ? 8 * p.nq : AP_ROWS);
    p.shared_bytes = 256 + align_up(AT_MAX_CTAS * sizeof(AttnShared), 256);
    if (p.nq == 0) {
        const int64_t tile = 2 * ap_tokens((int)(n_heads / hk));
        const int64_t tiles = (T / tile + n_seqs) * hk; // at least every sequence's
        if (tiles > INT32_MAX) return p;
        p.base_bytes = align_up((size_t)(n_seqs + 1) * 8, 256);
        p.tile_bytes = (size_t)tiles * sizeof(int2);
    }
    p.ml_bytes = align_up(part_rows * sizeof(float2), 256);
    p.part_bytes = part_rows * d * sizeof(float);
    p.ok = true;
    return p;
}

template <int D, int NQ>
cudaError_t launch_tokens(const AttnArgs &a, int ctas, int rows, cudaStream_t stream, int dev)
{
    static std::atomic<int> done[kMaxDevices];
    constexpr int smem = at_smem(D, NQ);
    cudaError_t e = ensure_smem(k_attention_tokens<D, NQ>, smem, done, dev);
    if (e == cudaSuccess)
        e = launch_pdl(k_attention_tokens<D, NQ>, dim3(ctas), dim3(at_warps(NQ) * 32), smem, stream, a);
    if (e == cudaSuccess)
        e = launch_pdl(k_attention_join<D>, dim3(ctas, (unsigned)std::min(rows, 8 * NQ)), dim3(128), 0,
                       stream, a, 8 * NQ);
    return e;
}

template <int D>
cudaError_t launch_prompt(const CUtensorMap &tk, const CUtensorMap &tv, const AttnArgs &a, int ctas,
                          cudaStream_t stream, int dev)
{
    static std::atomic<int> done[kMaxDevices];
    constexpr int smem = ap_smem(D);
    CUtensorMap tq;
    if (!encode_queries(&tq, a.q, a.bt.T, a.q_stride, a.kv.hk * a.group, a.group, D)) return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem(k_attention_prompt<D>, smem, done, dev);
    if (e == cudaSuccess) e = launch_pdl(k_attention_plan<D>, dim3(1), dim3(1024), 0, stream, a, ctas);
    if (e == cudaSuccess)
        e = launch_pdl(k_attention_prompt<D>, dim3(ctas), dim3(AP_THREADS), smem, stream, tk, tv, tq, a);
    if (e == cudaSuccess)
        e = launch_pdl(k_attention_prompt_join<D>, dim3(ctas, D / 16), dim3(256), 0, stream, a);
    return e;
}

} // namespace
} // namespace bitnet

using namespace bitnet;

extern "C" {

bitnet_status_t bitnet_rope_table(double theta, int64_t max_pos, int32_t head_dim, float *table, cudaStream_t stream)
{
    if (!table || !(theta > 0.0) || !std::isfinite(theta) || max_pos < 1) return BITNET_ERR_INVALID_ARG;
    if (max_pos > kMaxRows || (head_dim != 64 && head_dim != 128)) return BITNET_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(table)) return BITNET_ERR_MISALIGNED;
    const int64_t n = max_pos * (head_dim / 2);
    return cuda_status(launch_pdl(k_rope_table, dim3((unsigned)cdiv(n, 256)), dim3(256), 0, stream, theta, n,
                                  (int)head_dim, table));
}

bitnet_status_t bitnet_kv_append(const bitnet_kv_cache_t *cache, const bitnet_kv_batch_t *batch, const void *q,
                                 const void *k, const void *v, bitnet_dtype_t dtype, int32_t n_heads,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, const float *rope,
                                 int64_t rope_len, void *q_out, int64_t q_out_stride, cudaStream_t stream)
{
    AppendArgs a = {};
    bitnet_status_t st = check_cache(cache, batch, a.kv, a.bt);
    if (st != BITNET_OK) return st;
    if (dtype != BITNET_DTYPE_BF16 && dtype != BITNET_DTYPE_F32) return BITNET_ERR_INVALID_ARG;
    if (!q != !q_out || (rope && rope_len < 1)) return BITNET_ERR_INVALID_ARG;
    const int d = cache->head_dim, hk = cache->n_kv_heads;
    const int size = dtype == BITNET_DTYPE_F32 ? 4 : 2;
    const int64_t kw = (int64_t)hk * d, T = a.bt.T;
    if ((st = check_rows(k, k_stride, kw, size)) != BITNET_OK || (st = check_rows(v, v_stride, kw, size)) != BITNET_OK)
        return st;
    if (rope && !aligned16(rope)) return BITNET_ERR_MISALIGNED;
    // what is written (the cache, q_out) must not be what is read
    const CacheRanges written(*cache);
    const BatchRanges described(a.bt);
    const ByteRange rr = rope ? range_of(rope, (size_t)std::min<int64_t>(rope_len, INT32_MAX) * d * 4) : ByteRange{0, 0};
    if (!written.apart() || written.hit(rows_range(k, k_stride, kw, size, T)) ||
        written.hit(rows_range(v, v_stride, kw, size, T)) || written.hit(rr) || described.hit(written.r[0]) ||
        described.hit(written.r[1]) || described.hit(written.r[2]) || described.hit(written.r[3]))
        return BITNET_ERR_INVALID_ARG;
    if (q) {
        if (n_heads < 1) return BITNET_ERR_INVALID_ARG;
        if (n_heads % hk != 0 || n_heads / hk > kMaxGroup) return BITNET_ERR_UNSUPPORTED_SHAPE;
        const int64_t qw = (int64_t)n_heads * d;
        if ((st = check_rows(q, q_stride, qw, size)) != BITNET_OK ||
            (st = check_rows(q_out, q_out_stride, qw, 2)) != BITNET_OK)
            return st;
        const bool same = q == q_out && size == 2 && q_stride == q_out_stride;
        if ((!same && rows_share(q, q_stride * size, qw * size, q_out, q_out_stride * 2, qw * 2, T)) ||
            rows_share(k, k_stride * size, kw * size, q_out, q_out_stride * 2, qw * 2, T) ||
            rows_share(v, v_stride * size, kw * size, q_out, q_out_stride * 2, qw * 2, T) ||
            written.hit(rows_range(q, q_stride, qw, size, T)))
            return BITNET_ERR_INVALID_ARG;
        const ByteRange qo = rows_range(q_out, q_out_stride, qw, 2, T);
        if (written.hit(qo) || described.hit(qo) || overlaps(qo, rr)) return BITNET_ERR_INVALID_ARG;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.rope = rope;
    a.rope_len = rope ? rope_len : 0;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.q_out_stride = q_out_stride;
    a.group = q ? n_heads / hk : 0;
    const int heads = ka_warps(a.kv.page_shift) >> (a.kv.page_shift - 4); // kv heads per CTA
    const dim3 grid((unsigned)ka_base(a.bt.T, a.bt.n_seqs, a.kv.page_shift), (unsigned)cdiv(hk, heads), 2);
    const bool f32 = dtype == BITNET_DTYPE_F32;
    cudaError_t e;
    if (d == 128)
        e = f32 ? launch_append<true, 128>(a, a.kv.page_shift, grid, stream)
                : launch_append<false, 128>(a, a.kv.page_shift, grid, stream);
    else
        e = f32 ? launch_append<true, 64>(a, a.kv.page_shift, grid, stream)
                : launch_append<false, 64>(a, a.kv.page_shift, grid, stream);
    return cuda_status(e);
}

size_t bitnet_attention_workspace_size(int32_t n_seqs, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                       int32_t head_dim, int32_t max_new)
{
    const AttnPlan p = attn_plan(n_seqs, T, n_heads, n_kv_heads, head_dim, max_new);
    return p.ok ? p.total() : 0;
}

bitnet_status_t bitnet_attention(const bitnet_kv_cache_t *cache, const bitnet_kv_batch_t *batch, const void *q,
                                 int64_t q_stride, int32_t n_heads, int32_t max_new, float scale, void *out,
                                 int64_t out_stride, void *workspace, size_t ws_bytes, cudaStream_t stream)
{
    AttnArgs a = {};
    bitnet_status_t st = check_cache(cache, batch, a.kv, a.bt);
    if (st != BITNET_OK) return st;
    if (n_heads < 1 || max_new < 1 || max_new > a.bt.T || !(scale > 0.0f) || !std::isfinite(scale * 1.4427f))
        return BITNET_ERR_INVALID_ARG;
    const int d = cache->head_dim, hk = cache->n_kv_heads;
    const AttnPlan p = attn_plan(a.bt.n_seqs, a.bt.T, n_heads, hk, d, max_new);
    if (!p.ok) return BITNET_ERR_UNSUPPORTED_SHAPE;
    const int64_t qw = (int64_t)n_heads * d;
    if ((st = check_rows(q, q_stride, qw, 2)) != BITNET_OK || (st = check_rows(out, out_stride, qw, 2)) != BITNET_OK)
        return st;
    if (!(q == out && q_stride == out_stride) &&
        rows_share(q, q_stride * 2, qw * 2, out, out_stride * 2, qw * 2, a.bt.T))
        return BITNET_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < p.total()) return BITNET_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BITNET_ERR_MISALIGNED;
    const ByteRange wr = range_of(workspace, p.total()), written = rows_range(out, out_stride, qw, 2, a.bt.T);
    const CacheRanges cached(*cache);
    const BatchRanges described(a.bt);
    if (overlaps(wr, written) || overlaps(wr, rows_range(q, q_stride, qw, 2, a.bt.T)) || cached.hit(written) ||
        cached.hit(wr) || described.hit(written) || described.hit(wr))
        return BITNET_ERR_INVALID_ARG;
    const int dev = current_device();
    const int sms = num_sms_for(dev);
    if (sms <= 0) return BITNET_ERR_CUDA;
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.out = static_cast<uint16_t *>(out);
    a.out_stride = out_stride;
    a.group = n_heads / hk;
    a.max_new = max_new;
    a.scale_log2 = scale * 1.44269504088896341f;
    char *ws = static_cast<char *>(workspace);
    a.claim = reinterpret_cast<AttnClaim *>(ws);
    a.shared = reinterpret_cast<AttnShared *>(ws + 256);
    ws += p.shared_bytes;
    a.part_ml = reinterpret_cast<float2 *>(ws);
    ws += p.ml_bytes;
    a.part = reinterpret_cast<float *>(ws);
    ws += p.part_bytes;
    a.base = reinterpret_cast<int64_t *>(ws);
    a.tiles = reinterpret_cast<int2 *>(ws + p.base_bytes);
    const int ctas = std::min(sms, AT_MAX_CTAS);
    const int rows = a.group * max_new;
    cudaError_t e;
    if (p.nq == 0) {
        CUtensorMap tk, tv;
        if (!encode_codes(&tk, cache->k, cache->num_pages, hk, cache->page_size, d) ||
            !encode_codes(&tv, cache->v, cache->num_pages, hk, cache->page_size, d))
            return BITNET_ERR_CUDA;
        e = d == 128 ? launch_prompt<128>(tk, tv, a, ctas, stream, dev) : launch_prompt<64>(tk, tv, a, ctas, stream, dev);
    } else if (d == 128) {
        e = p.nq == 1 ? launch_tokens<128, 1>(a, ctas, rows, stream, dev) : launch_tokens<128, 2>(a, ctas, rows, stream, dev);
    } else {
        e = p.nq == 1 ? launch_tokens<64, 1>(a, ctas, rows, stream, dev) : launch_tokens<64, 2>(a, ctas, rows, stream, dev);
    }
    return cuda_status(e);
}

bitnet_status_t bitnet_batch_status(int clear, bitnet_status_t *status_out, cudaStream_t stream)
{
    if (!status_out) return BITNET_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return BITNET_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_batch_status, sizeof(int)) != cudaSuccess) return BITNET_ERR_CUDA;
    *status_out = static_cast<bitnet_status_t>(v);
    if (clear) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_batch_status, &zero, sizeof(int)) != cudaSuccess) return BITNET_ERR_CUDA;
    }
    return BITNET_OK;
}

} // extern "C"
