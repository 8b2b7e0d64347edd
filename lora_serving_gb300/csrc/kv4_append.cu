// kv4_append.cu -- rotary embedding of q and k with up to three position
// axes, 4-bit quantisation of k and v into their pages, and the way back.
//
// A row is one CTA or, from kWarpRows rows on, one warp.  A team of head_dim / 16 lanes holds a head, sixteen dims
// a lane, as two chunks of eight; in the rotated part the chunks are the two
// halves of eight pairs, so a rotation needs no exchange.  The team's lanes
// hold the same pairs for every head they take, so a lane reads its (cos,
// sin) once per row.  A group's minimum and maximum cross the team by
// shuffles.  Bound: HBM (the row in, q and a quarter of k and v out), and with
// many rows instructions: products are rounded one by one, so that the cached
// bytes are the formula's whatever the compiler.  Measured, in a graph: 15,797
// rows of 32 + 2 * 8 heads 67 us (350 MB in and out, 5.2 TB/s, 0.77 of a copy's
// rate; an issue slot in two taken), their reading back 15 (cold and alone 72
// and 20); 256 rows 4.3 and 2.6, latency.
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

using kv4::Batch;
using kv4::Cache;
using kv4::Seq;

constexpr int kThreads = 128;
constexpr int kWarpRows = 2432;   // 16 warps on each of 152 SMs

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f)
{
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// rint(c) for c in [0, 2^22), as the low bits of c + 1.5 * 2^23 hold it.
constexpr float kMagic = 12582912.f;

__device__ __forceinline__ void prefetch_row(const bf16_t* p, int n, int i, int threads)
{
    for (; i * 64 < n; i += threads) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p + i * 64));
}

// Eight codes of a chunk, one per nibble.  Step and lowest value are rounded
// to fp16 first (fewer bits to read back per token; the codes are taken
// against the rounded ones, so that rounding only moves the grid).  Four
// codes at a time are put together in fp32, exactly: conversions to integers
// run at a quarter of the rate of the fp32 pipe.
__device__ __forceinline__ uint32_t codes8(const float* f, float inv, float low)
{
    uint32_t half[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = __fadd_rn(fminf(fmaxf(__fmul_rn(__fsub_rn(f[4 * k + i], low), inv), 0.f), 15.f), kMagic) - kMagic;
        half[k] = __float_as_uint(fmaf(fmaf(c[3], 16.f, c[2]), 256.f, fmaf(c[1], 16.f, c[0])) + kMagic) & 0xFFFFu;
    }
    return half[0] | (half[1] << 16);
}

__device__ __forceinline__ void rotate8(float* a, float* b, const float* cs, const float* sn)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float lo = a[i], hi = b[i];
        a[i] = __fsub_rn(__fmul_rn(lo, cs[i]), __fmul_rn(hi, sn[i]));
        b[i] = __fadd_rn(__fmul_rn(hi, cs[i]), __fmul_rn(lo, sn[i]));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 6) kv4_append_kernel(AppendArgs a, int per_row)
{
    constexpr int kLanes = D / 16, kGroups = D / kv4::kGroup;
    const int row = blockIdx.x * (kThreads / per_row) + threadIdx.x / per_row, of_row = threadIdx.x % per_row;
    const int lane = of_row % kLanes, team = of_row / kLanes, teams = per_row / kLanes;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (row >= a.batch.n_rows) return;
    // the row's lines are on their way while the tables are read
    prefetch_row(a.x + static_cast<long long>(row) * a.ld_x + a.q_off, a.n_heads * D, of_row, per_row);
    prefetch_row(a.x + static_cast<long long>(row) * a.ld_x + a.k_off, a.cache.n_kv * D, of_row, per_row);
    prefetch_row(a.x + static_cast<long long>(row) * a.ld_x + a.v_off, a.cache.n_kv * D, of_row, per_row);
    int at[LORA_MAX_ROPE_AXES] = {0, 0, 0};
    if (a.rot_dim && a.positions) {
#pragma unroll
        for (int x = 0; x < LORA_MAX_ROPE_AXES; ++x)
            if (x < a.n_axes) at[x] = __ldg(a.positions + static_cast<long long>(row) * a.ld_pos + x);
    }
    const int s = kv4::find_seq_warp(a.batch.q_starts, a.batch.n_seqs, row);
    Seq q;
    if (!kv4::load_seq(a.batch, s, q, of_row == 0 ? a.status : nullptr) || row < q.row0 || row >= q.row0 + q.n) return;
    const int p = q.ctx - q.n + (row - q.row0);
    if (p < 0) return;

    // this lane's chunks: dims [d0, d0 + 8) and [d1, d1 + 8)
    const int half = a.rot_dim >> 1, rot_lanes = half >> 3;
    const bool turns = lane < rot_lanes;
    const int d0 = turns ? 8 * lane : a.rot_dim + 16 * (lane - rot_lanes);
    const int d1 = turns ? half + d0 : d0 + 8;
    bool bad = false;
    if (a.rot_dim) {
#pragma unroll
        for (int x = 0; x < LORA_MAX_ROPE_AXES; ++x) {
            if (x >= a.n_axes) break;
            if (!a.positions) at[x] = p;
            bad |= static_cast<unsigned>(at[x]) >= static_cast<unsigned>(a.max_pos);
        }
    }
    if (bad) {
        if (of_row == 0) flag(a.status, LORA_DEV_BAD_POSITION);
        return;
    }
    float cs[8], sn[8];
    if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = d0 + i;
            const int pos = pair < a.axis_end[0] ? at[0] : pair < a.axis_end[1] ? at[1] : at[2];
            const float2 t = __ldg(reinterpret_cast<const float2*>(a.rope) + static_cast<long long>(pos) * half + pair);
            cs[i] = t.x;
            sn[i] = t.y;
        }
    }
    const int page = kv4::page_of(a.cache, a.batch, s, p, of_row == 0 ? a.status : nullptr);
    const int off = p & (a.cache.page_size - 1), ps = a.cache.page_size;

    const bf16_t* x = a.x + static_cast<long long>(row) * a.ld_x;
    const int n_kv = a.cache.n_kv;
    for (int h = team; h < a.n_heads; h += teams) {
        float f0[8], f1[8];
        unpack8(*reinterpret_cast<const uint4*>(x + a.q_off + h * D + d0), f0);
        unpack8(*reinterpret_cast<const uint4*>(x + a.q_off + h * D + d1), f1);
        if (turns) rotate8(f0, f1, cs, sn);
        bf16_t* o = a.q_out + static_cast<long long>(row) * a.ld_q + h * D;
        *reinterpret_cast<uint4*>(o + d0) = pack8(f0);
        *reinterpret_cast<uint4*>(o + d1) = pack8(f1);
    }
    if (page < 0) return;
    const float inf = __int_as_float(0x7F800000);
    const int g0 = d0 / kv4::kGroup, g1 = d1 / kv4::kGroup;
    // Every lane of a warp makes the same number of rounds (the shuffles
    // below need them all); a team past the last head does nothing with its.
    for (int first = 0; first < 2 * n_kv; first += teams) {
        const int head = first + team;
        const bool live = head < 2 * n_kv, is_k = head < n_kv;
        const int h = is_k ? head : head - n_kv;
        const bf16_t* src = x + (is_k ? a.k_off : a.v_off) + (live ? h : 0) * D;
        float f0[8], f1[8];
        unpack8(*reinterpret_cast<const uint4*>(src + d0), f0);
        unpack8(*reinterpret_cast<const uint4*>(src + d1), f1);
        if (is_k && turns) rotate8(f0, f1, cs, sn);
        // each chunk's ends, then its group's; a NaN stays
        float lo[2] = {inf, inf}, hi[2] = {-inf, -inf};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f0[i] = max_nan(min_nan(f0[i], kv4::kMaxAbs), -kv4::kMaxAbs);
            f1[i] = max_nan(min_nan(f1[i], kv4::kMaxAbs), -kv4::kMaxAbs);
            lo[0] = min_nan(lo[0], f0[i]);
            hi[0] = max_nan(hi[0], f0[i]);
            lo[1] = min_nan(lo[1], f1[i]);
            hi[1] = max_nan(hi[1], f1[i]);
        }
        if (kGroups == 1) {
            lo[0] = min_nan(lo[0], lo[1]);
            hi[0] = max_nan(hi[0], hi[1]);
        } else if (g0 == g1) {   // both chunks in one group: the other one's neutral
            const float l = min_nan(lo[0], lo[1]), m = max_nan(hi[0], hi[1]);
            lo[0] = g0 ? inf : l;
            lo[1] = g0 ? l : inf;
            hi[0] = g0 ? -inf : m;
            hi[1] = g0 ? m : -inf;
        }
        float low[kGroups], inv[kGroups];
        uint8_t* block = kv4::block_of(a.cache, page, live ? h : 0);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
                lo[g] = min_nan(lo[g], __shfl_xor_sync(0xFFFFFFFFu, lo[g], o));
                hi[g] = max_nan(hi[g], __shfl_xor_sync(0xFFFFFFFFu, hi[g], o));
            }
            const __half st = __float2half_rn(__fmul_rn(__fsub_rn(hi[g], lo[g]), 1.f / 15.f));
            const __half lw = __float2half_rn(lo[g]);
            const float stf = __half2float(st);
            low[g] = __half2float(lw);
            inv[g] = stf > 0.f ? __frcp_rn(stf) : 0.f;
            if (live && lane == 0) {
                if (is_k) {
                    reinterpret_cast<__half2*>(block + kv4::k_params_off(ps, D))[off * kGroups + g] = __halves2half2(st, lw);
                } else {
                    __half* d = reinterpret_cast<__half*>(block + kv4::v_params_off(ps, D)) +
                                ((off >> 1) * kGroups + g) * 4 + (off & 1);
                    d[0] = st;
                    d[2] = lw;
                }
            }
        }
        const uint32_t w0 = codes8(f0, g0 ? inv[kGroups - 1] : inv[0], g0 ? low[kGroups - 1] : low[0]);
        const uint32_t w1 = codes8(f1, g1 ? inv[kGroups - 1] : inv[0], g1 ? low[kGroups - 1] : low[0]);
        if (!live) continue;
        if (is_k) {
            uint32_t* d = reinterpret_cast<uint32_t*>(block) + off * (D / 8);
            d[kv4::k_word(d0 >> 3, D)] = w0;
            d[kv4::k_word(d1 >> 3, D)] = w1;
        } else {
            // halves of two neighbouring words, at this position's parity
            uint16_t* d = reinterpret_cast<uint16_t*>(block + kv4::v_codes_off(ps, D)) + (off >> 1) * (D / 2) + (off & 1);
            d[2 * (d0 >> 2)] = static_cast<uint16_t>(w0);
            d[2 * (d0 >> 2) + 2] = static_cast<uint16_t>(w0 >> 16);
            d[2 * (d1 >> 2)] = static_cast<uint16_t>(w1);
            d[2 * (d1 >> 2) + 2] = static_cast<uint16_t>(w1 >> 16);
        }
    }
}

// Eight dims a thread: k of every kv head, then v.
template <int D>
__global__ void __launch_bounds__(kThreads, 8) kv4_read_kernel(ReadArgs a, int per_row)
{
    constexpr int kChunks = D / 8, kGroups = D / kv4::kGroup;
    const int row = blockIdx.x * (kThreads / per_row) + threadIdx.x / per_row, of_row = threadIdx.x % per_row;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (row >= a.batch.n_rows) return;
    const int s = kv4::find_seq_warp(a.batch.q_starts, a.batch.n_seqs, row);
    Seq q;
    if (!kv4::load_seq(a.batch, s, q, of_row == 0 ? a.status : nullptr) || row < q.row0 || row >= q.row0 + q.n) return;
    const int p = q.ctx - q.n + (row - q.row0);
    if (p < 0) return;
    const int page = kv4::page_of(a.cache, a.batch, s, p, of_row == 0 ? a.status : nullptr);
    if (page < 0) return;
    const int ps = a.cache.page_size, off = p & (ps - 1), n_kv = a.cache.n_kv;
    // this thread's eight dims of every head it takes
    const int c = of_row % kChunks, g = c / 8, step_h = per_row / kChunks;
    const long long head_bytes = kv4::block_bytes(ps, D);
    const uint8_t* block = kv4::block_of(a.cache, page, of_row / kChunks);
    const uint8_t* kc = block + off * (D / 2) + 4 * kv4::k_word(c, D);
    const uint8_t* kp = block + kv4::k_params_off(ps, D) + 4 * (off * kGroups + g);
    const uint8_t* vc = block + kv4::v_codes_off(ps, D) + (off >> 1) * D + 2 * (off & 1) + 8 * c;
    const uint8_t* vp = block + kv4::v_params_off(ps, D) + ((off >> 1) * kGroups + g) * 8 + 2 * (off & 1);
    bf16_t* ko = a.k + static_cast<long long>(row) * a.ld_k + 8 * c;
    bf16_t* vo = a.v + static_cast<long long>(row) * a.ld_v + 8 * c;
    auto out8 = [](uint32_t w, float step, float low) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)   // 2^23 + code, less 2^23; code * step is exact
            f[j] = fmaf(__uint_as_float(((w >> (4 * j)) & 15u) | 0x4B000000u) - 8388608.f, step, low);
        return pack8(f);
    };
#pragma unroll 4
    for (int h = of_row / kChunks; h < n_kv; h += step_h) {
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(kc);
        const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(kp));
        const uint32_t vw = *reinterpret_cast<const uint16_t*>(vc) | (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vc + 4)) << 16);
        const float vs = __half2float(*reinterpret_cast<const __half*>(vp)), vl = __half2float(*reinterpret_cast<const __half*>(vp + 4));
        *reinterpret_cast<uint4*>(ko + h * D) = out8(kw, kf.x, kf.y);
        *reinterpret_cast<uint4*>(vo + h * D) = out8(vw, vs, vl);
        kc += step_h * head_bytes;
        kp += step_h * head_bytes;
        vc += step_h * head_bytes;
        vp += step_h * head_bytes;
    }
}

// Threads of a row: a CTA's four warps, or one where there are rows enough
// to fill the SMs' warps all the same (its tables are then read once for
// four times the work).
int threads_per_row(int n_rows) { return n_rows >= kWarpRows ? 32 : kThreads; }

template <class Args>
cudaError_t launch(void (*kernel)(Args, int), const Args& a, cudaStream_t stream)
{
    if (a.batch.n_rows == 0) return cudaSuccess;
    const int per_row = threads_per_row(a.batch.n_rows), rows = kThreads / per_row;
    PdlLaunch l(dim3(static_cast<unsigned>((a.batch.n_rows + rows - 1) / rows)), kThreads, 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, a, per_row);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_kv4_append(const AppendArgs& a, cudaStream_t stream)
{
    return a.cache.head_dim == 64 ? launch(kv4_append_kernel<64>, a, stream) : launch(kv4_append_kernel<128>, a, stream);
}

cudaError_t launch_kv4_read(const ReadArgs& a, cudaStream_t stream)
{
    return a.cache.head_dim == 64 ? launch(kv4_read_kernel<64>, a, stream) : launch(kv4_read_kernel<128>, a, stream);
}

}  // namespace lora
