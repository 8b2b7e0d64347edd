// kv4.cuh -- the paged 4-bit cache as the kernels see it: block layout,
// a row's place, and the batch's tables with their device-side checks.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace lora {
namespace kv4 {

constexpr int kGroup = 64;          // dims that share a step and a lowest value
constexpr float kMaxAbs = 60000.f;  // stored values saturate here: code 15 stays inside fp16

struct Cache {
    uint8_t* pages;
    long long page_stride;
    int n_pages;
    int page_size;
    int page_shift;   // log2(page_size)
    int n_kv;
    int head_dim;
};

struct Batch {
    const int32_t* q_starts;
    const int32_t* ctx_lens;
    const int32_t* block_table;
    int ld_table;
    int n_seqs;
    int n_rows;
    int max_q_len;
    int max_ctx_len;
};

__host__ __device__ constexpr int block_bytes(int page_size, int head_dim)
{
    return page_size * (head_dim + 8 * (head_dim / kGroup));
}
// Byte offsets inside a block.
__host__ __device__ constexpr int v_codes_off(int page_size, int head_dim) { return page_size * head_dim / 2; }
__host__ __device__ constexpr int k_params_off(int page_size, int head_dim) { return page_size * head_dim; }
__host__ __device__ constexpr int v_params_off(int page_size, int head_dim)
{
    return page_size * (head_dim + 4 * (head_dim / kGroup));
}
// 32-bit word of K dims [8c, 8c + 8) inside a position's row of codes.
__host__ __device__ constexpr int k_word(int c, int head_dim) { return (c & 3) * (head_dim / 32) + (c >> 2); }

// Block of page `page`, kv head h.  64-bit: a cache passes 4 GB.
__device__ __forceinline__ uint8_t* block_of(const Cache& c, int page, int h)
{
    return c.pages + static_cast<long long>(page) * c.page_stride +
           static_cast<long long>(h) * block_bytes(c.page_size, c.head_dim);
}

// One sequence's entries, checked against the host's bounds.  False (and
// flagged): the sequence is skipped.
struct Seq {
    int row0, n, ctx;
};
__device__ __forceinline__ bool load_seq(const Batch& b, int s, Seq& q, int32_t* status)
{
    const int r0 = __ldg(b.q_starts + s), r1 = __ldg(b.q_starts + s + 1), ctx = __ldg(b.ctx_lens + s);
    q.row0 = r0;
    q.n = r1 - r0;
    q.ctx = ctx;
    if (r0 < 0 || r1 < r0 || r1 > b.n_rows || r1 - r0 > b.max_q_len || ctx < 0 || ctx > b.max_ctx_len) {
        flag(status, LORA_DEV_BAD_SEGMENT);
        q.n = 0;
        q.ctx = 0;
        return false;
    }
    return true;
}

// The sequence that owns a row: the last s with q_starts[s] <= row, found by
// the whole warp, 32 entries to a round.
__device__ __forceinline__ int find_seq_warp(const int32_t* q_starts, int n_seqs, int row)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n_seqs;   // the answer lies in [lo, lo + len)
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const int at = lane * step;
        const bool le = at < len && __ldg(q_starts + lo + at) <= row;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        len = min(step, len - k * step);
    }
    return lo;
}

// Page of a sequence's position p; -1 (flagged) where the table has none.
__device__ __forceinline__ int page_of(const Cache& c, const Batch& b, int s, int p, int32_t* status)
{
    const int page = __ldg(b.block_table + static_cast<long long>(s) * b.ld_table + (p >> c.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.n_pages)) {
        flag(status, LORA_DEV_BAD_PAGE);
        return -1;
    }
    return page;
}

}  // namespace kv4
}  // namespace lora
