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
// Drafted trees have an account of their own, from 70 batches of even lengths
// timed both ways (1 to 64 requests, up to 512 rows of a kv head, 100 to 8000
// positions): 1.2 % on the mean above the faster kernel, 3.5 % by the other
// account; 16 trees of 18 rows, 64 heads, over 164 positions 28 / 20, 13 of 9
// over 854 35 / 28, one of 26 over 6812 29 / 32.  It takes the window's positions.
int few_limit(const AttendArgs& a)
{
    const int group = a.n_heads / a.cache.n_kv;
    const long long rows = static_cast<long long>(group) * a.batch.max_q_len;
    const double units = static_cast<double>(a.batch.n_seqs) * a.cache.n_kv;
    const double ctx = a.tree && a.window > 0 ? std::min(a.batch.max_ctx_len + 0LL, a.window + 0LL + a.batch.max_q_len) : a.batch.max_ctx_len;
    const double slices = units * std::ceil(rows / 8.) * (ctx / 32 + 2), items = units * std::ceil(rows / 256.);
    const double few = a.tree ? 10e-6 + slices * (a.cache.head_dim == 64 ? 0.62e-9 : 0.9e-9) : 9e-6 + slices * 0.9e-9;
    const double many = 22e-6 + (a.tree ? items * (ctx / 128) * 12.5e-9 : items * (ctx / 128 + 4) * 11.5e-9);
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
    // (every row of a tree may see all of the tree's, whichever block of 256 it is in)
    const long long many = (a.batch.n_rows * group / 256 + a.batch.n_seqs) * (span(a.tree ? a.batch.max_q_len : 256) / 128 + 6);
    return std::max(few, rows > few_limit(a) ? many : 0) * a.cache.n_kv;
}

namespace {

// Joins the pieces behind each record, in order: kQuads 16-byte pieces of a
// row's sums to a thread, a row to neighbouring threads, as many CTAs to a
// record as its slot's rows need.  A chain of latencies: the first two pieces,
// most often all there are, come as one, and with short slots before the
// record says whether they count (with long ones what does not count costs more
// than it saves).  Measured (us, the call; 16 trees of 16 to 64 rows in a window
// of 4096 / 32 of 2 to 6): maxima, then sums, one row after another 49.0 / 16.2;
// together, with 1, 2, 4 and 8 pieces to a thread 45.7, 44.1, 44.2, 47.0 / 16.2;
// before the record 50.4 / 15.8.
constexpr int kJoinThreads = 256, kQuads = 4, kEarlyRows = 32;
__host__ __device__ constexpr int join_ctas(int rows, int D) { return (rows * (D / 4) + kJoinThreads * kQuads - 1) / (kJoinThreads * kQuads); }

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(AttendArgs a, kv4::Partials p0, kv4::Partials p1)
{
    tc::grid_dep_wait();
    // When the next launch may begin: at once, here, or at the end.  Measured (us, early / late).  Where the next launch is the same
    // call again, it decides which SMs that call's CTAs come to, and prompts gain by the late one: 16 prompts 302 / 291, trees of
    // 16 to 64 rows in a window 43.9 / 44.2.  Before a product of 4096 columns the early one gains a little: such trees 60.0 / 60.9,
    // tokens of 64 requests 31.1 / 31.4, a window 79.2 / 79.8, prompts 608 / 604 to 609.  Before a norm they differ by less than
    // runs do, but for small trees, 18.1 / 17.7.
    if (a.tree) tc::grid_dep_launch();
    const int n0 = p0.ctas * join_ctas(p0.rows, D);
    const bool second = static_cast<int>(blockIdx.x) >= n0;
    const kv4::Partials& p = second ? p1 : p0;
    const int per = join_ctas(p.rows, D), x = blockIdx.x - (second ? n0 : 0), b = x / per, group = a.group;
    const kv4::Record u = p.records[b];
    const float inf = __int_as_float(0x7F800000);
    constexpr int kPer = D / (4 * kQuads), kRows = kJoinThreads / kPer;   // threads of a row, rows of a CTA
    const int r = (x - b * per) * kRows + threadIdx.x / kPer, d = 4 * (threadIdx.x % kPer);
    const bool early = p.rows <= kEarlyRows;
    if (early ? r >= p.rows : r >= u.rows) return;
    // The first two pieces, most often all, are on their way together.
    float m = -inf, l = 0.f, top[2], sum[2];
    float4 o[kQuads], v[2][kQuads];
    auto load = [&](int k, float& at_top, float& at_sum, float4 (&to)[kQuads]) {
        const float* s = p.slot(k, k == b, D);
        at_top = s[p.rows * D + r];
        at_sum = s[p.rows * (D + 1) + r];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) to[i] = *reinterpret_cast<const float4*>(s + r * D + d + 4 * kPer * i);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (early ? b + k < p.ctas : b + k <= u.last) load(b + k, top[k], sum[k], v[k]);
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= u.rows) return;
    if (b >= u.last) top[1] = -inf;
    m = fmaxf(top[0], top[1]);
    for (int k = b + 2; k <= u.last; ++k) m = fmaxf(m, p.slot(k, false, D)[p.rows * D + r]);
    auto add = [&](float at_top, float at_sum, const float4 (&from)[kQuads]) {
        const float w = m == -inf ? 0.f : kv4::ex2(at_top - m);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            o[i].x = fmaf(from[i].x, w, o[i].x);
            o[i].y = fmaf(from[i].y, w, o[i].y);
            o[i].z = fmaf(from[i].z, w, o[i].z);
            o[i].w = fmaf(from[i].w, w, o[i].w);
        }
        l = fmaf(at_sum, w, l);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (b + k <= u.last) add(top[k], sum[k], v[k]);
    for (int k = b + 2; k <= u.last; ++k) {
        load(k, top[0], sum[0], v[0]);
        add(top[0], sum[0], v[0]);
    }
    if (!a.tree) tc::grid_dep_launch();
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = u.block_row0 + r, tok = row / group;
    bf16_t* const out = a.out + static_cast<long long>(u.seq_row0 + tok) * a.ld_out + (u.h * group + row - tok * group) * D + d;
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
        *reinterpret_cast<uint2*>(out + 4 * kPer * i) = make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
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
