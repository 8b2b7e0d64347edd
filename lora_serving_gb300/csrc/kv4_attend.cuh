// kv4_attend.cuh -- what the attention kernels share: finding a place in the
// batch's work, and the small steps from codes to fp16 operands.
#pragma once

#include "kv4.h"

namespace lora {
namespace kv4 {

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// m16n8k16, fp16 x fp16 -> fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from a start that differs by column only: c0 in even, c1 in odd ones.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1, float c0, float c1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held as an mma fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }

// Four pairs of codes of a word as fp16: pair i is (nibble i, nibble 4 + i).
// A nibble OR-ed into the mantissa of 1024 is 1024 + code (low nibble of a
// byte, even pairs) or 1024 + 16 code (high nibble, odd pairs).
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));   // (w & mask) | 1024
    return r;
}
__device__ __forceinline__ void codes_1024(uint32_t w, uint32_t (&c)[4])
{
    const uint32_t y = w >> 8;
    c[0] = pick(w, 0x000F000Fu);
    c[1] = pick(w, 0x00F000F0u);
    c[2] = pick(y, 0x000F000Fu);
    c[3] = pick(y, 0x00F000F0u);
}
// kWords adjacent words of shared memory.
template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[kWords])
{
    static_assert(kWords == 2 || kWords == 4, "words");
    if (kWords == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[kWords - 2] = v.z; w[kWords - 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    }
}
// code * step + low, one fp16 rounding.
__device__ __forceinline__ void values(uint32_t w, __half2 step, __half2 low, uint32_t (&v)[4])
{
    const __half2 k = __float2half2_rn(-1024.f), s = __float2half2_rn(1.f / 16), k16 = __float2half2_rn(-64.f);
    const uint32_t y = w >> 8;
    v[0] = as_u32(__hfma2(__hadd2(as_h2(pick(w, 0x000F000Fu)), k), step, low));
    v[1] = as_u32(__hfma2(__hfma2(as_h2(pick(w, 0x00F000F0u)), s, k16), step, low));
    v[2] = as_u32(__hfma2(__hadd2(as_h2(pick(y, 0x000F000Fu)), k), step, low));
    v[3] = as_u32(__hfma2(__hfma2(as_h2(pick(y, 0x00F000F0u)), s, k16), step, low));
}

// The first position that a row at p sees (with p before the first position, as it may be, 0: the row has nothing to
// see).  No window and no p take this out of 32 bits: p - window + 1 alone would leave them.
__device__ __forceinline__ int seen_from(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// Which halves of a (steps, lows) pair have codes whose value is no finite fp16 number: with step and low finite a value
// can still leave fp16, and code 15's does if any does (low itself is code 0's).  An append leaves none.
__device__ __forceinline__ uint32_t not_finite(uint32_t step, uint32_t low)
{
    const uint32_t end = as_u32(__hfma2(__float2half2_rn(15.f), as_h2(step), as_h2(low)));
    return ((end & 0x7C00u) == 0x7C00u ? 0xFFFFu : 0u) | ((end & 0x7C000000u) == 0x7C000000u ? 0xFFFF0000u : 0u);
}

// Running sum over the sequences of count(s), in shared memory (prefix: one
// entry more than sequences; sums: one per warp), by the whole CTA.
template <int kWarps, class F>
__device__ __forceinline__ void scan_seqs(int n_seqs, int* prefix, int* sums, F count)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    if (tid == 0) prefix[0] = 0;
    for (int s0 = 0; s0 < n_seqs; s0 += 32 * kWarps) {
        const int s = s0 + tid;
        int sum = s < n_seqs ? count(s) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        int before = base;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? sums[w] : 0;
            base += sums[w];
        }
        if (s < n_seqs) prefix[s + 1] = before + sum;
        __syncthreads();
    }
}
// A row (position x head) of a sequence to its position, without a division:
// exact for 2^26 rows, to which n times the magic number's error (group, at
// most 64) stays below 2^32; the kernel for few rows has far fewer.
__device__ __forceinline__ int by_group(const AttendArgs& a, int n)
{
    return a.group_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), a.group_magic)) : n;
}
// The last s with prefix[s] <= x.
__device__ __forceinline__ int seq_at(const int* prefix, int n_seqs, int x)
{
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Partial results.  Work is cut into equal ranges, one per CTA; what a range's
// end cuts leaves partial results: `rows` x D sums of weighted values, then the
// rows' maxima (log2) and sums of weights.  Slot 0 of a CTA: of what began
// before its range; slot 1: of what begins in it and goes on after it, which
// has a record.
struct Record {
    int rows, block_row0, seq_row0, h, last;   // rows 0: none; the pieces lie in CTAs [this, last]
};
struct Partials {
    Record* records;
    float* sums;
    int ctas, rows;   // ranges; rows of a slot
    __device__ __forceinline__ float* slot(int cta, int i, int D) const
    {
        return sums + (static_cast<long long>(cta) * 2 + i) * (static_cast<long long>(rows) * (D + 2));
    }
};
// Where they lie in a workspace, and its bytes (a multiple of 256).
inline Partials partials_at(void* ws, int ctas, int rows)
{
    return Partials{static_cast<Record*>(ws), reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + (ctas * sizeof(Record) + 255) / 256 * 256), ctas, rows};
}
inline size_t partials_bytes(int ctas, int rows, int D)
{
    return ((ctas * sizeof(Record) + 255) / 256 * 256 + static_cast<size_t>(ctas) * 2 * rows * (D + 2) * sizeof(float) + 255) / 256 * 256;
}

}  // namespace kv4

// Sequences with at most few_rows query rows to a kv head (rows x heads of
// the group), and the others; ws: the kernel's own workspace.  *left: the
// partial results to be joined (ctas 0: none).  after: the launch before it
// is the other kernel's of the same call, which it need not wait for.
cudaError_t launch_kv4_few(const AttendArgs& a, int few_rows, void* ws, bool after, kv4::Partials* left, cudaStream_t stream);
cudaError_t launch_kv4_many(const AttendArgs& a, int few_rows, void* ws, kv4::Partials* left, cudaStream_t stream);
size_t kv4_many_workspace(int head_dim);
size_t kv4_few_workspace(int head_dim);

}  // namespace lora
