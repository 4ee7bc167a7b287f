// kv_common.cuh -- what the kernels of the paged 8-bit key/value cache share:
// device views of the cache and the batch, the batch status word, and the
// lookup of a sequence's extent with its checks.
#pragma once

#include "bitnet_kv.h"
#include "common.cuh"

namespace bitnet {

// Set once a kernel met a page id, length, offset or position out of range.
// Kept apart from the device status word: waits give up while that one is set,
// and a batch that a caller got wrong must not touch later calls.
__device__ int g_batch_status = 0;

BITNET_DEVINL void record_batch_error() { *(volatile int *)&g_batch_status = BITNET_ERR_INVALID_ARG; }

// Out-of-line part of kv_wait, asked every 256 tries: 0 to give up (as mbar_wait does),
// else the time of the first question (t0 = 0: this one).
__device__ __noinline__ unsigned long long kv_wait_on(unsigned long long t0)
{
    if (status_failed()) return 0;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) return now;
    if (now - t0 <= wait_limit_ns()) return t0;
    record_status(BITNET_ERR_TIMEOUT);
    return 0;
}

// mbar_wait in few instructions: the kernel for prompts waits at many places, and
// code beyond the instruction cache costs it more than the waits.
BITNET_DEVINL bool kv_wait(uint64_t *bar, uint32_t parity)
{
    const uint32_t a = smem_u32(bar);
    unsigned long long t0 = 0;
    for (uint32_t spin = 1;; ++spin) {
        if (mbar_try_wait(a, parity)) return true;
        if ((spin & 255u) == 0 && (t0 = kv_wait_on(t0)) == 0) return false;
    }
}

struct KvView {
    int8_t *k, *v;
    float *k_step, *v_step;
    int64_t num_pages;
    int hk;         // kv heads
    int page_shift; // page_size = 1 << page_shift
};

struct BatchView {
    const int32_t *table;
    const int32_t *lens;
    const int32_t *q_start;
    int64_t width;
    int n_seqs;
    int T;
};

// Sequence b: its new rows [q0, q0 + n), its cached tokens len; ok = false (and
// the error is recorded) if they contradict each other or the buffers.
struct SeqInfo {
    int q0, n, len;
    bool ok;
};

BITNET_DEVINL SeqInfo seq_info(const BatchView &bt, int page_shift, int b)
{
    SeqInfo s;
    s.q0 = bt.q_start[b];
    const int q1 = bt.q_start[b + 1];
    s.len = bt.lens[b];
    s.ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= bt.T && s.len >= 0 && s.len <= (bt.width << page_shift);
    s.n = s.ok ? q1 - s.q0 : 0;
    if (s.n > s.len) s.ok = false;
    if (!s.ok) {
        s.n = 0;
        s.len = 0;
        record_batch_error();
    }
    return s;
}

// Page of table row b, column j, or -1 (and the error is recorded).
BITNET_DEVINL int page_of(const KvView &kv, const BatchView &bt, int b, int j)
{
    const int p = bt.table[(int64_t)b * bt.width + j];
    if (p >= 0 && p < kv.num_pages) return p;
    record_batch_error();
    return -1;
}

} // namespace bitnet
