// kv4_attend.cu -- which kernel takes which rows of lora_kv4_attend, and the
// joining of what their ranges' ends cut.
#include <algorithm>
#include <cmath>

#include "kv4_attend.cuh"
#include "tc_common.cuh"

namespace lora {

namespace {

// Query rows to a kv head (a sequence's rows x the heads of a group) up to
// which the kernel for few rows is the faster one whatever the lengths: it
// takes 8 rows at a time over 32 positions in 0.9 ns of the GPU's time, the
// tensor-memory kernel 256 rows over 128 positions in 11.5 ns.
constexpr int kFewRows = 24;

// The limit for a batch: all of its rows where the kernel for few rows takes
// the shorter time by that account and the launches' fixed times (9 and 22 us:
// so small batches of longer rows go to it too), otherwise kFewRows.
// Measured both ways (us, 8 kv heads of 128, few / many): one sequence of 1000
// positions with 256 rows 20 / 35, of 16000 with 40 rows 31 / 34 and with 64
// 40 / 35; 32 of 1000 with 40 rows 49 / 49, with 64 72 / 50, of 8000 287 / 196.
// The account takes the whole context, a window or not: 64 rows in 32000
// positions with a window of 1024 go to the kernel for many and take 25 us,
// where the same rows in 1088 positions take 14 in the other.
int few_limit(const AttendArgs& a)
{
    const int group = a.n_heads / a.cache.n_kv;
    const long long rows = static_cast<long long>(group) * a.batch.max_q_len;
    const double units = static_cast<double>(a.batch.n_seqs) * a.cache.n_kv, ctx = a.batch.max_ctx_len;
    const double few = 9e-6 + units * std::ceil(rows / 8.) * (ctx / 32 + 2) * 0.9e-9;
    const double many = 22e-6 + units * std::ceil(rows / 256.) * (ctx / 128 + 4) * 11.5e-9;
    if (rows <= kFewRows || few <= many) return static_cast<int>(std::min<long long>(rows, 1 << 30));
    return group <= kFewRows ? kFewRows : 0;
}

}  // namespace

long long kv4_attend_places(const AttendArgs& a)
{
    const long long group = a.n_heads / a.cache.n_kv, rows = group * a.batch.max_q_len;
    // positions that rows so many positions apart see
    auto span = [&](long long apart) { return a.window > 0 ? std::min(a.batch.max_ctx_len + 0LL, a.window + apart) : a.batch.max_ctx_len; };
    // units of 8 rows over tiles of 32 positions, items of 256 over 128: a tile cut at either end, and a start's cost
    const long long few = a.batch.n_seqs * ((std::min<long long>(few_limit(a), rows) + 7) / 8) * (span(a.batch.max_q_len) / 32 + 5);
    const long long many = (a.batch.n_rows * group / 256 + a.batch.n_seqs) * (span(256) / 128 + 6);
    return std::max(few, rows > few_limit(a) ? many : 0) * a.cache.n_kv;
}

namespace {

// Joins the pieces behind each record, in order: kQuads 16-byte pieces of a
// row's sums to a thread, as many CTAs to a record as its slot's rows need
// (most records are empty, and a CTA costs its launch: 24 requests in a window
// 65.1 us with one piece to a thread, 62.7 with 2, 63.1 with 4; 16 prompts
// 306, 308, 301).
constexpr int kJoinThreads = 256, kQuads = 4;
__host__ __device__ constexpr int join_ctas(int rows, int D) { return (rows * (D / 4) + kJoinThreads * kQuads - 1) / (kJoinThreads * kQuads); }

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(AttendArgs a, kv4::Partials p0, kv4::Partials p1)
{
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int n0 = p0.ctas * join_ctas(p0.rows, D);
    const bool second = static_cast<int>(blockIdx.x) >= n0;
    const kv4::Partials& p = second ? p1 : p0;
    const int per = join_ctas(p.rows, D), x = blockIdx.x - (second ? n0 : 0), b = x / per, group = a.group;
    const kv4::Record u = p.records[b];
    const float inf = __int_as_float(0x7F800000);
    for (int e = (x - b * per) * kJoinThreads + threadIdx.x; e < u.rows * (D / 4); e += per * kJoinThreads) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float m = -inf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = b; k <= u.last; ++k) m = fmaxf(m, p.slot(k, k == b, D)[p.rows * D + r]);
#pragma unroll 4
        for (int k = b; k <= u.last; ++k) {
            const float* s = p.slot(k, k == b, D);
            const float w = m == -inf ? 0.f : kv4::ex2(s[p.rows * D + r] - m);
            const float4 v = *reinterpret_cast<const float4*>(s + r * D + d);
            o.x = fmaf(v.x, w, o.x);
            o.y = fmaf(v.y, w, o.y);
            o.z = fmaf(v.z, w, o.z);
            o.w = fmaf(v.w, w, o.w);
            l = fmaf(s[p.rows * (D + 1) + r], w, l);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int row = u.block_row0 + r, tok = row / group;
        *reinterpret_cast<uint2*>(a.out + static_cast<long long>(u.seq_row0 + tok) * a.ld_out + (u.h * group + row - tok * group) * D + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
}

}  // namespace

// The kernels' workspaces lie one after the other (which of them a batch's
// longer rows go to depends on more than the arguments here).
size_t kv4_attend_workspace(int n_heads, int n_kv, int head_dim, int max_q_len)
{
    return kv4_few_workspace(head_dim) + (static_cast<long long>(n_heads / n_kv) * max_q_len > kFewRows ? kv4_many_workspace(head_dim) : 0);
}

cudaError_t launch_kv4_attend(const AttendArgs& a, cudaStream_t stream)
{
    if (a.batch.n_rows == 0 || a.batch.max_q_len == 0) return cudaSuccess;
    const int group = a.n_heads / a.cache.n_kv, D = a.cache.head_dim, few = few_limit(a);
    const bool many = static_cast<long long>(group) * a.batch.max_q_len > few;
    kv4::Partials p0{}, p1{};
    cudaError_t e = cudaSuccess;
    if (many) e = launch_kv4_many(a, few, static_cast<uint8_t*>(a.ws) + kv4_few_workspace(D), &p0, stream);
    if (e == cudaSuccess && few) e = launch_kv4_few(a, few, a.ws, many, &p1, stream);
    const int ctas = p0.ctas * join_ctas(p0.rows, D) + p1.ctas * join_ctas(p1.rows, D);
    if (e != cudaSuccess || ctas == 0) return e;
    PdlLaunch l(dim3(ctas), kJoinThreads, 0, stream);
    e = D == 64 ? cudaLaunchKernelEx(&l.cfg, kv4_join_kernel<64>, a, p0, p1) : cudaLaunchKernelEx(&l.cfg, kv4_join_kernel<128>, a, p0, p1);
    note_launch();
    return e;
}

}  // namespace lora
