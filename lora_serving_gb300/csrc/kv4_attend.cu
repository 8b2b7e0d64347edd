// kv4_attend.cu -- causal attention over the paged 4-bit cache.
//
// One warp per (row, q head), a position at a time: each lane holds
// head_dim / 32 dims of q and of the running sum, the score is a warp sum,
// and the softmax keeps its running maximum and sum in fp32.
#include "kv4_attend.cuh"
#include "tc_common.cuh"

namespace lora {

namespace {

using kv4::Seq;

template <int D>
__global__ void __launch_bounds__(128) kv4_attend_kernel(AttendArgs a)
{
    constexpr int kDims = D / 32, kGroups = D / kv4::kGroup;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int row = static_cast<int>(unit / a.n_heads), head = static_cast<int>(unit % a.n_heads);
    if (row >= a.batch.n_rows) return;
    const int s = kv4::find_seq_warp(a.batch.q_starts, a.batch.n_seqs, row);
    Seq q;
    if (!kv4::load_seq(a.batch, s, q, lane == 0 ? a.status : nullptr) || row < q.row0 || row >= q.row0 + q.n) return;
    const int p = q.ctx - q.n + (row - q.row0);
    const int h = head / (a.n_heads / a.cache.n_kv), ps = a.cache.page_size;
    const int d = lane * kDims, c = d >> 3, n0 = d & 7, g = d / kv4::kGroup;

    float qf[kDims], acc[kDims];
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        qf[i] = __uint_as_float(static_cast<uint32_t>(a.q[static_cast<long long>(row) * a.ld_q + head * D + d + i]) << 16) * a.scale;
        acc[i] = 0.f;
    }
    float m = -__int_as_float(0x7F800000), l = 0.f;
    const int j0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
    int page = -1;
    for (int j = j0; j <= p; ++j) {
        if (j == j0 || (j & (ps - 1)) == 0) page = kv4::page_of(a.cache, a.batch, s, j, lane == 0 ? a.status : nullptr);
        if (page < 0) continue;
        const int off = j & (ps - 1);
        const uint8_t* block = kv4::block_of(a.cache, page, h);
        const uint32_t kw = reinterpret_cast<const uint32_t*>(block)[off * (D / 8) + kv4::k_word(c, D)] >> (4 * n0);
        const __half2 kp = reinterpret_cast<const __half2*>(block + kv4::k_params_off(ps, D))[off * kGroups + g];
        const uint16_t* vd = reinterpret_cast<const uint16_t*>(block + kv4::v_codes_off(ps, D)) + (off >> 1) * (D / 2) + (off & 1);
        const uint32_t vw = vd[2 * (d >> 2)] >> (4 * (d & 3));
        const __half* vp = reinterpret_cast<const __half*>(block + kv4::v_params_off(ps, D)) + ((off >> 1) * kGroups + g) * 4 + (off & 1);
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kDims; ++i)
            part = fmaf(qf[i], fmaf(static_cast<float>((kw >> (4 * i)) & 15u), __low2float(kp), __high2float(kp)), part);
        const float score = warp_sum(part);
        const float top = fmaxf(m, score);
        const float keep = expf(m - top), w = expf(score - top);
        m = top;
        l = fmaf(l, keep, w);
        const float vs = __half2float(vp[0]), vl = __half2float(vp[2]);
#pragma unroll
        for (int i = 0; i < kDims; ++i) acc[i] = fmaf(acc[i], keep, w * fmaf(static_cast<float>((vw >> (4 * i)) & 15u), vs, vl));
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bf16_t* o = a.out + static_cast<long long>(row) * a.ld_out + head * D + d;
#pragma unroll
    for (int i = 0; i < kDims; i += 2) *reinterpret_cast<uint32_t*>(o + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
}

}  // namespace

size_t kv4_attend_workspace(int n_heads, int n_kv, int head_dim, int max_q_len) { return kv4_few_workspace(head_dim, 32); }

cudaError_t launch_kv4_attend(const AttendArgs& a, cudaStream_t stream)
{
    if (a.batch.n_rows == 0) return cudaSuccess;
    const int rows = a.batch.max_q_len * (a.n_heads / a.cache.n_kv);
    if (rows <= 32) return launch_kv4_few(a, rows, stream);
    const long long warps = static_cast<long long>(a.batch.n_rows) * a.n_heads;
    PdlLaunch l(dim3(static_cast<unsigned>((warps + 3) / 4)), 128, 0, stream);
    const cudaError_t e = a.cache.head_dim == 64 ? cudaLaunchKernelEx(&l.cfg, kv4_attend_kernel<64>, a)
                                                 : cudaLaunchKernelEx(&l.cfg, kv4_attend_kernel<128>, a);
    note_launch();
    return e;
}

}  // namespace lora
