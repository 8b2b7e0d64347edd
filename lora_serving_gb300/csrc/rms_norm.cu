// rms_norm.cu -- residual addition, root-mean-square norm, and the result in
// bf16 and in 8 bits with scales, in one pass.
//
// One CTA holds a row in registers (h is bf16, so four registers keep eight
// columns exactly), reduces sum h^2 and max |h w| together, and writes every
// output from them.  The row's largest |n| is max |h w| / rms up to fp32
// rounding, so a row scale needs no second reduction.  The bound is HBM: 2 + 2
// bytes in and 2 + 2 + 1 out per element (residual, both outputs).  Measured:
// 35402 rows of 4096 with all of these 187 us, 7.0 TB/s with what L2 keeps of
// the last writes (a copy: 6.7); one row 3.0 us, 64 rows 2.8, start to start.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

__device__ __forceinline__ float elem(const uint4& v, int i)
{
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
}

// max that keeps a NaN: non-negative floats order as their bits, and a NaN's
// bits lie above infinity's.
__device__ __forceinline__ float max_abs(float a, float b)
{
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b) & 0x7FFFFFFFu));
}

__device__ __forceinline__ uint2 to_e4m3x8(const float* n, float inv)
{
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(n[4 * i] * inv, n[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(n[4 * i + 2] * inv, n[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        r[i] = lo | (hi << 16);
    }
    return make_uint2(r[0], r[1]);
}

// Groups whose largest value is below kSmall (448 / g is finite down to 1.3e-36) are scaled up first.
constexpr float kSmall = 0x1p-64f, kUp = 0x1p64f;

// Chunk j of a thread: columns 8 * (j * blockDim.x + threadIdx.x).  Sixteen
// neighbouring lanes then hold the 128 columns of a scale.
template <int NCH>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormArgs a)
{
    __shared__ float red[2][32];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, threads = blockDim.x, nch = a.width >> 3;
    uint4 h[NCH];
    const bf16_t* x = a.x + row * a.ld_x;
    const bf16_t* res = a.res ? a.res + row * a.ld_res : nullptr;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = j * threads + tid;
        h[j] = c < nch ? *reinterpret_cast<const uint4*>(x + 8 * c) : make_uint4(0, 0, 0, 0);
    }
    if (res) {
        uint4 r[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = j * threads + tid;
            r[j] = c < nch ? *reinterpret_cast<const uint4*>(res + 8 * c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = j * threads + tid;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = elem(r[j], i);
            h[j] = add_round8(h[j], f);
            if (c < nch) *reinterpret_cast<uint4*>(a.res_out + row * a.ld_res_out + 8 * c) = h[j];
        }
    }
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = j * threads + tid;
        if (c >= nch) break;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.w + 8 * c));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = elem(h[j], i);
            sum = fmaf(v, v, sum);
            top = max_abs(top, v * elem(w, i));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        top = max_abs(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if ((tid & 31) == 0) {
        red[0][tid >> 5] = sum;
        red[1][tid >> 5] = top;
    }
    __syncthreads();
    const int warps = threads >> 5;
    sum = (tid & 31) < warps ? red[0][tid & 31] : 0.f;
    top = (tid & 31) < warps ? red[1][tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        top = max_abs(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    const float rs = 1.f / sqrtf(sum / static_cast<float>(a.width) + a.eps);
    const float row_top = max_abs(0.f, top * rs);
    if (a.y8 && a.group == 0 && tid == 0) a.scales[row * a.ld_scales] = row_top / 448.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = j * threads + tid;
        const bool live = c < nch;
        const uint4 w = live ? __ldg(reinterpret_cast<const uint4*>(a.w + 8 * c)) : make_uint4(0, 0, 0, 0);
        float n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = elem(h[j], i) * rs * elem(w, i);
        if (a.y && live) {
            uint4 o;
            o.x = pack_bf16x2(n[0], n[1]);
            o.y = pack_bf16x2(n[2], n[3]);
            o.z = pack_bf16x2(n[4], n[5]);
            o.w = pack_bf16x2(n[6], n[7]);
            *reinterpret_cast<uint4*>(a.y + row * a.ld_y + 8 * c) = o;
        }
        if (a.y8) {
            float g = row_top;
            if (a.group) {
                g = 0.f;
                if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) g = max_abs(g, n[i]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) g = max_abs(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
                if (live && (c & 15) == 0) a.scales[row * a.ld_scales + (c >> 4)] = g / 448.f;
            }
            if (g < kSmall) {   // 448 / g might be no fp32 number: both taken up by a power of two, unless the scale is 0
                g = g / 448.f == 0.f ? 0.f : g * kUp;
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] *= kUp;
            }
            // a NaN stays NaN through the product, so g == 0 is the only special case left
            const float inv = g == 0.f ? 0.f : 448.f / g;
            if (live) *reinterpret_cast<uint2*>(a.y8 + row * a.ld_y8 + 8 * c) = to_e4m3x8(n, inv);
        }
    }
}

template <int NCH>
cudaError_t run(const NormArgs& a, int threads, cudaStream_t stream)
{
    PdlLaunch l(dim3(static_cast<unsigned>(a.n_rows)), threads, 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, rms_norm_kernel<NCH>, a);
    note_launch();
    return e;
}

}  // namespace

int device_sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream)
{
    if (a.n_rows == 0) return cudaSuccess;
    // Chunks of eight columns to a thread.  A small call wants every thread there is (one chunk); a large one
    // more loads in flight per thread and fewer threads to meet at the row's sum.  Measured (us, residual and
    // both outputs, 1 / 2 / 4 chunks): 64 rows of 4096 2.4 / 2.6 / 3.2, 400 rows 4.4 / 3.6 / 4.0, 2500 rows
    // 15.1 / 12.8 / 11.7, 8000 rows 48.6 / 45.6 / 45.7; 8000 rows of 512 8.7 in each form.
    const int nch = a.width >> 3;
    const long long elems = static_cast<long long>(a.n_rows) * a.width;
    const int want = nch >= 256 && elems >= (8 << 20) ? 4 : elems >= (nch >= 256 ? 3 << 19 : 6 << 20) ? 2 : 1;
    const int per = std::max(want, nch <= 1024 ? 1 : nch <= 2048 ? 2 : nch <= 4096 ? 4 : 8);
    const int threads = std::max(32, ((nch + per - 1) / per + 31) / 32 * 32);
    switch (per) {
    case 1: return run<1>(a, threads, stream);
    case 2: return run<2>(a, threads, stream);
    case 4: return run<4>(a, threads, stream);
    default: return run<8>(a, threads, stream);
    }
}

}  // namespace lora
