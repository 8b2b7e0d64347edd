// kv4_plan.cu -- a step's tables from its requests' lengths: row starts,
// positions, pages from and to the stack of free ones, slots of the rows.
//
// Three running sums over the sequences (rows, pages asked for, pages given
// back) place everything: sequence s takes the stack's entries behind what the
// sequences before it asked for.  Every CTA of the one cluster computes them
// for itself, from all lengths, and writes a share of the results; the one
// barrier between them stands behind the pages given back, since the next are
// taken from the same stack, and behind the last read of counters that the
// results may go to in place.  A sequence that asks for more than there is
// gets nothing, and with it none after it gets any: the sums stay sums, no
// sequence waiting for another's answer.
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kMaxThreads = 1024, kOwn = kMaxSeqs / kMaxThreads;   // sequences of a thread
constexpr int kRun = 4;                                            // neighbouring rows of a thread
constexpr uint32_t kNoPlace = 0xFFFFFFFFu;

// Sums that stop at their limit: what passes it is refused whatever its size.
__device__ __forceinline__ uint32_t add_to(uint32_t a, uint32_t b, uint32_t limit) { return min(a + b, limit); }

__global__ void __launch_bounds__(kMaxThreads, 1) kv4_plan_kernel(PlanArgs a, int ranks)
{
    extern __shared__ uint32_t smem[];
    __shared__ uint32_t sums[3][32];
    __shared__ uint32_t taken;
    const int n = a.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int rank = static_cast<int>(blockIdx.x);
    uint32_t* const row_at = smem;               // [n + 1] a sequence's first row
    uint32_t* const need_at = smem + n + 1;      // [n] pages asked for before it; kNoPlace: it has none
    uint32_t* const held_s = need_at + n;        // [n]
    int32_t* const stack = a.pool.free_pages;
    const int per = (n + blockDim.x - 1) / blockDim.x;
    tc::grid_dep_wait();
    tc::grid_dep_launch();

    // ---- this thread's sequences
    const uint32_t limit[3] = {static_cast<uint32_t>(a.max_rows) + 1, static_cast<uint32_t>(a.pool.n_pages) + 1, static_cast<uint32_t>(a.pool.n_pages) + 1};
    uint32_t v[kOwn][3];   // rows, pages asked for, pages given back
    int ctx[kOwn], held[kOwn];
    int faults = 0;
    uint32_t sum[3] = {0, 0, 0};
    int n_free = __ldg(a.pool.n_free);
    if (n_free < 0 || n_free > a.pool.n_pages) {
        faults |= LORA_DEV_BAD_PAGE;
        n_free = 0;
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * per + i;
        v[i][0] = v[i][1] = v[i][2] = 0;
        ctx[i] = -1;
        held[i] = 0;
        if (i >= per || s >= n) continue;
        const int q = __ldg(a.q_lens + s), len = __ldg(a.lens + s), h = __ldg(a.pool.held + s);
        const bool counts = h >= 0 && h <= a.pool.ld_table;
        held[i] = h;
        if (!counts) faults |= LORA_DEV_BAD_SEGMENT;
        if (q < 0) {
            if (counts) v[i][2] = h;
            held[i] = 0;
            ctx[i] = 0;
        } else {
            v[i][0] = min(static_cast<uint32_t>(q), limit[0]);
            const bool fits = counts && q <= a.max_q_len && len >= 0 && len <= a.max_ctx_len && q <= a.max_ctx_len - len;
            if (fits) {
                ctx[i] = len + q;
                if (q > 0) v[i][1] = max(0, ((ctx[i] + a.pool.page_size - 1) >> a.page_shift) - h);
            } else {
                faults |= LORA_DEV_BAD_SEGMENT;
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k] = add_to(sum[k], v[i][k], limit[k]);
    }
    // ---- what lies before them
    uint32_t before[3], total[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t up = sum[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, up, o);
            if (lane >= o) up = add_to(up, x, limit[k]);
        }
        if (lane == 31) sums[k][warp] = up;
        before[k] = __shfl_up_sync(0xFFFFFFFFu, up, 1);
        if (lane == 0) before[k] = 0;
    }
    if (tid == 0) taken = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t x = lane < warps ? sums[k][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x = add_to(x, y, limit[k]);
        }
        total[k] = __shfl_sync(0xFFFFFFFFu, x, 31);
        const uint32_t w = __shfl_sync(0xFFFFFFFFu, x, max(warp - 1, 0));
        if (warp > 0) before[k] = add_to(w, before[k], limit[k]);
    }
    const uint32_t there = min(static_cast<uint32_t>(n_free) + total[2], static_cast<uint32_t>(a.pool.n_pages));
    if (static_cast<uint32_t>(n_free) + total[2] > there) faults |= LORA_DEV_BAD_PAGE;

    // ---- who gets what; pages given back, a warp to a sequence's
    uint32_t at[kOwn][3];
    bool got[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * per + i;
        const bool mine = i < per && s < n;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            at[i][k] = before[k];
            before[k] = add_to(before[k], v[i][k], limit[k]);
        }
        got[i] = ctx[i] >= 0;
        if (got[i] && v[i][0] > 0 && before[0] > static_cast<uint32_t>(a.max_rows)) {
            faults |= LORA_DEV_BAD_SEGMENT;
            got[i] = false;
        }
        if (got[i] && v[i][1] > 0 && before[1] > there) {
            faults |= LORA_DEV_NO_PAGES;
            got[i] = false;
        }
        if (!got[i]) v[i][1] = 0;
        if (v[i][1] > 0) atomicMax(&taken, before[1]);
        if (mine) {
            row_at[s] = at[i][0];
            need_at[s] = got[i] ? at[i][1] : kNoPlace;
            held_s[s] = held[i];
        }
        for (unsigned todo = __ballot_sync(0xFFFFFFFFu, v[i][2] > 0); todo; todo &= todo - 1) {
            const int who = __ffs(todo) - 1, from = __shfl_sync(0xFFFFFFFFu, s, who);
            const uint32_t count = __shfl_sync(0xFFFFFFFFu, v[i][2], who), to = n_free + __shfl_sync(0xFFFFFFFFu, at[i][2], who);
            const int32_t* row = a.pool.block_table + static_cast<long long>(from) * a.pool.ld_table;
            for (uint32_t j = lane + 32 * ((rank + from) % ranks); j < count; j += 32 * ranks)
                if (to + j < static_cast<uint32_t>(a.pool.n_pages)) stack[to + j] = row[j];
        }
    }
    if (tid == 0) row_at[n] = total[0];
    if (rank == 0 && faults) flag(a.status, faults);
    cluster_arrive();
    cluster_wait();

    // ---- lengths, and the new pages' table entries
    const uint32_t rows_cut = static_cast<uint32_t>(a.max_rows);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * per + i;
        if (i < per && s < n && s % ranks == rank) {
            a.q_starts[s] = static_cast<int32_t>(min(at[i][0], rows_cut));
            a.ctx_lens[s] = got[i] ? ctx[i] : 0;
            a.pool.held_out[s] = held[i] + static_cast<int>(v[i][1]);
        }
        for (unsigned todo = __ballot_sync(0xFFFFFFFFu, v[i][1] > 0); todo; todo &= todo - 1) {
            const int who = __ffs(todo) - 1, to = __shfl_sync(0xFFFFFFFFu, s, who), h = __shfl_sync(0xFFFFFFFFu, held[i], who);
            const uint32_t count = __shfl_sync(0xFFFFFFFFu, v[i][1], who), from = there - 1 - __shfl_sync(0xFFFFFFFFu, at[i][1], who);
            int32_t* row = a.pool.block_table + static_cast<long long>(to) * a.pool.ld_table + h;
            for (uint32_t j = lane + 32 * ((rank + to) % ranks); j < count; j += 32 * ranks) row[j] = __ldcg(stack + from - j);
        }
    }
    if (rank == 0 && tid == 0) {
        a.q_starts[n] = static_cast<int32_t>(min(total[0], rows_cut));
        *a.pool.n_free_out = static_cast<int32_t>(there - taken);
    }

    // ---- the rows, a run of neighbours to a thread: one search for their first
    if (!a.row_seq && !a.positions && !a.slots) return;
    for (int t0 = kRun * (rank * blockDim.x + tid); t0 < a.max_rows; t0 += kRun * ranks * blockDim.x) {
        int lo = 0, hi = n - 1;   // the last sequence that begins at t0 or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (row_at[mid] <= static_cast<uint32_t>(t0)) lo = mid; else hi = mid - 1;
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int t = t0 + k;
            if (t >= a.max_rows) break;
            int seq = -1, pos = -1;
            int64_t slot = -1;
            if (static_cast<uint32_t>(t) < total[0]) {
                while (row_at[lo + 1] <= static_cast<uint32_t>(t)) ++lo;
                if (need_at[lo] != kNoPlace) {
                    seq = lo;
                    const int len = __ldg(a.lens + lo), i = t - static_cast<int>(row_at[lo]), p = len + i;
                    const int depth = a.depths ? __ldg(a.depths + t) : i;
                    if (depth >= 0 && depth < a.max_ctx_len) pos = len + depth;
                    const int at_page = p >> a.page_shift, h = static_cast<int>(held_s[lo]);
                    const int page = at_page < h ? a.pool.block_table[static_cast<long long>(lo) * a.pool.ld_table + at_page]
                                                 : __ldcg(stack + (there - 1 - need_at[lo] - (at_page - h)));
                    if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pool.n_pages))
                        slot = (static_cast<int64_t>(page) << a.page_shift) + (p & (a.pool.page_size - 1));
                }
            }
            if (a.row_seq) a.row_seq[t] = seq;
            if (a.positions) a.positions[t] = pos;
            if (a.slots) a.slots[t] = slot;
        }
    }
}

}  // namespace

cudaError_t launch_kv4_plan(const PlanArgs& a, cudaStream_t stream)
{
    const int smem = 4 * (3 * a.n_seqs + 1);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_on_device(done, [] { return cudaFuncSetAttribute(kv4_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (3 * kMaxSeqs + 1)); });
    if (e != cudaSuccess) return e;
    const int threads = a.n_seqs <= 256 && a.max_rows <= 1024 ? 256 : kMaxThreads;
    const int ranks = a.max_rows > 4096 ? 8 : 1;
    PdlLaunch l(dim3(ranks), threads, smem, stream);
    cudaLaunchAttribute attr[2];
    attr[0] = l.attr[0];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    l.cfg.attrs = attr;
    l.cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&l.cfg, kv4_plan_kernel, a, ranks);
    note_launch();
    return e;
}

}  // namespace lora
