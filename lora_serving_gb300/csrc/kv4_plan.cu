// kv4_plan.cu -- a step's tables from its requests' lengths: row starts,
// positions, pages from and to the stack of free ones, slots of the rows.
//
// Three running sums over the sequences (rows, pages asked for, pages given
// back) place everything: sequence s takes the stack's entries behind what the
// sequences before it asked for.  Every CTA computes them for itself, from all
// lengths; rows, pages taken and pages given back are then jobs for any thread,
// which finds its sequence by a search in a running sum.  (A warp that went
// through its sequences one after another took 20 us for 4096 of them.)  No job
// waits for another: a page that was given back and is taken again in the same
// call is read where it came from.  Where the counters' results go to
// the place that other CTAs read them from, the CTAs are one cluster, whose one
// barrier, begun before the sums, stands before these results alone.  (What the
// kernel writes, counters, stack and table, it reads by ordinary loads: the
// read-only path is for what nobody writes while a kernel runs.)  A sequence
// that asks for more than there is gets nothing, and with it none after it gets
// any: the sums stay sums, no sequence waiting for another's answer.
// Bound: latency, of a chain of loads, sums over the CTA, a search, and loads;
// with thousands of sequences the sums' instructions, which every CTA repeats.
// Measured, start to start: 64 requests of a token 2.6 us (3.0 with the counters
// in place), 256 with 16 prompts among them (17 k rows) 3.6 (5.0), 4096 trees 6.3 (8.5).
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kMaxThreads = 1024, kFewThreads = 256, kMostOwn = 4;   // threads of a CTA; sequences of a thread
static_assert(kMaxThreads * kMostOwn >= kMaxSeqs, "every sequence has a thread");
constexpr int kRanks = 8;                                            // CTAs of a cluster, at most
constexpr uint32_t kNoPlace = 0xFFFFFFFFu;

// Sums that stop at their limit: what passes it is refused whatever its size.
__device__ __forceinline__ uint32_t add_to(uint32_t a, uint32_t b, uint32_t limit) { return __viaddmin_u32(a, b, limit); }

// kOwn: sequences of a thread; kRun: neighbouring rows of a job.
template <int kOwn, int kRun>
__global__ void __launch_bounds__(kMaxThreads, 1) kv4_plan_kernel(PlanArgs a, int ranks, int workers, int each, bool in_place)
{
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ uint32_t sums[3][32];
    __shared__ uint32_t taken;
    const int n = a.n_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int rank = static_cast<int>(blockIdx.x);
    const int n4 = (n + 3) & ~3;
    uint32_t* const need_at = smem;              // [n4] pages asked for before a sequence
    uint32_t* const back_at = need_at + n4;      // [n4] pages given back before it
    uint32_t* const held_s = back_at + n4;       // [n4] pages that it held; kNoPlace: it has no place
    uint32_t* const row_at = held_s + n4;        // [n4 + 1] its first row
    int32_t* const stack = a.pool.free_pages;
    tc::grid_dep_wait();
    tc::grid_dep_launch();

    // ---- this thread's sequences
    const uint32_t limit[3] = {static_cast<uint32_t>(a.max_rows) + 1, static_cast<uint32_t>(a.pool.n_pages) + 1, static_cast<uint32_t>(a.pool.n_pages) + 1};
    uint32_t v[kOwn][3];   // rows, pages asked for, pages given back
    int ctx[kOwn], held[kOwn];
    int faults = 0;
    uint32_t sum[3] = {0, 0, 0};
    int n_free = *a.pool.n_free;
    if (n_free < 0 || n_free > a.pool.n_pages) {
        faults |= LORA_DEV_BAD_PAGE;
        n_free = 0;
    }
    int q_of[kOwn], len_of[kOwn], held_of[kOwn];   // every load on its way before the first is looked at
    auto load = [&](const int32_t* from, int (&to)[kOwn]) {
        if (kOwn == 4 && a.wide_in && tid * 4 + 3 < n) {
            const int4 x = reinterpret_cast<const int4*>(from)[tid];
            to[0] = x.x; to[1 % kOwn] = x.y; to[2 % kOwn] = x.z; to[3 % kOwn] = x.w;
            return;
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) to[i] = tid * kOwn + i < n ? from[tid * kOwn + i] : 0;
    };
    load(a.q_lens, q_of);
    load(a.lens, len_of);
    load(a.pool.held, held_of);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * kOwn + i;
        v[i][0] = v[i][1] = v[i][2] = 0;
        ctx[i] = -1;
        held[i] = 0;
        if (s >= n) continue;
        const int q = q_of[i], len = len_of[i], h = held_of[i];
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
    if (in_place) cluster_arrive();   // (waited for at the end)
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

    // ---- who gets what
    uint32_t at[kOwn][3];
    bool got[kOwn];
    uint32_t mine_taken = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * kOwn + i;
        const bool mine = s < n;
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
        if (v[i][1] > 0) mine_taken = before[1];
        if (kOwn == 1 && mine) {
            row_at[s] = at[i][0];
            need_at[s] = at[i][1];
            back_at[s] = at[i][2];
            held_s[s] = got[i] ? held[i] : kNoPlace;
        }
    }
    if (kOwn == 4 && tid * 4 < n) {
        auto four = [&](uint32_t* to, uint32_t x, uint32_t y, uint32_t z, uint32_t w) { *reinterpret_cast<uint4*>(to + 4 * tid) = make_uint4(x, y, z, w); };
        four(row_at, at[0][0], at[1 % kOwn][0], at[2 % kOwn][0], at[3 % kOwn][0]);
        four(need_at, at[0][1], at[1 % kOwn][1], at[2 % kOwn][1], at[3 % kOwn][1]);
        four(back_at, at[0][2], at[1 % kOwn][2], at[2 % kOwn][2], at[3 % kOwn][2]);
        four(held_s, got[0] ? held[0] : kNoPlace, got[1 % kOwn] ? held[1 % kOwn] : kNoPlace, got[2 % kOwn] ? held[2 % kOwn] : kNoPlace, got[3 % kOwn] ? held[3 % kOwn] : kNoPlace);
    }
    mine_taken = __reduce_max_sync(0xFFFFFFFFu, mine_taken);
    if (lane == 0 && mine_taken) atomicMax(&taken, mine_taken);
    if (tid == 0) row_at[n] = total[0];
    if (rank == 0 && faults) flag(a.status, faults);
    __syncthreads();
    // the last sequence whose running sum is x or less: the one that x falls into, for x below the total
    auto seq_at = [&](const uint32_t* sum, uint32_t x) {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sum[mid] <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    // The f-th page taken: from the stack's top, which is what has been given back, where it still lies.
    auto page_taken = [&](uint32_t f) -> int {
        const uint32_t from = there - 1 - f;
        if (from < static_cast<uint32_t>(n_free)) return stack[from];
        const int s = seq_at(back_at, from - n_free);
        return a.pool.block_table[static_cast<long long>(s) * a.pool.ld_table + (from - n_free - back_at[s])];
    };
    const uint32_t n_back = there - n_free, n_taken = taken, runs = a.row_seq || a.positions || a.slots ? (a.max_rows + kRun - 1) / kRun : 0;
    for (uint32_t job = tid < workers ? rank * workers + tid : 0xFFFFFFFFu; job < runs + n_taken + n_back; job += ranks * workers) {
        if (job >= runs + n_taken) {   // a page given back: onto the stack
            const uint32_t f = job - runs - n_taken;
            const int s = seq_at(back_at, f);
            stack[n_free + f] = a.pool.block_table[static_cast<long long>(s) * a.pool.ld_table + (f - back_at[s])];
            continue;
        }
        if (job >= runs) {   // a page taken: into the table, behind those that the sequence holds
            const uint32_t f = job - runs;
            const int s = seq_at(need_at, f);
            a.pool.block_table[static_cast<long long>(s) * a.pool.ld_table + held_s[s] + (f - need_at[s])] = page_taken(f);
            continue;
        }
        // ---- a run of neighbouring rows: one search for their first
        const int t0 = kRun * static_cast<int>(job);
        int lo = seq_at(row_at, t0), seq[kRun], pos[kRun], len[kRun], depth[kRun], page[kRun];
        long long slot[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int t = t0 + k;
            const bool live = t < a.max_rows && static_cast<uint32_t>(t) < total[0];
            while (live && row_at[lo + 1] <= static_cast<uint32_t>(t)) ++lo;
            seq[k] = live && held_s[lo] != kNoPlace ? lo : -1;
            len[k] = seq[k] >= 0 ? __ldg(a.lens + lo) : 0;
            depth[k] = seq[k] >= 0 && a.depths ? __ldg(a.depths + t) : -1;
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            page[k] = -1;
            if (seq[k] < 0) continue;
            const uint32_t at_page = (len[k] + t0 + k - static_cast<int>(row_at[seq[k]])) >> a.page_shift, h = held_s[seq[k]];
            if (at_page < h) page[k] = a.pool.block_table[static_cast<long long>(seq[k]) * a.pool.ld_table + at_page];
            else page[k] = page_taken(need_at[seq[k]] + at_page - h);
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int i = t0 + k - (seq[k] >= 0 ? static_cast<int>(row_at[seq[k]]) : 0), d = a.depths ? depth[k] : i;
            pos[k] = seq[k] >= 0 && d >= 0 && d < a.max_ctx_len ? len[k] + d : -1;
            slot[k] = static_cast<uint32_t>(page[k]) < static_cast<uint32_t>(a.pool.n_pages)
                          ? (static_cast<long long>(page[k]) << a.page_shift) + ((len[k] + i) & (a.pool.page_size - 1)) : -1;
        }
        if (kRun == 4 && a.wide_out && t0 + kRun <= a.max_rows) {
            if (a.row_seq) *reinterpret_cast<int4*>(a.row_seq + t0) = make_int4(seq[0], seq[1 % kRun], seq[2 % kRun], seq[3 % kRun]);
            if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1 % kRun], pos[2 % kRun], pos[3 % kRun]);
            if (a.slots) {
                *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1 % kRun]);
                *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2 % kRun], slot[3 % kRun]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                if (t0 + k >= a.max_rows) break;
                if (a.row_seq) a.row_seq[t0 + k] = seq[k];
                if (a.positions) a.positions[t0 + k] = pos[k];
                if (a.slots) a.slots[t0 + k] = slot[k];
            }
        }
    }

    // ---- the sequences' own: one CTA writes a thread's (taken in turn, by a remainder for each, they cost 4096 trees 1.1 us)
    const bool writes = tid >= rank * each && tid < rank * each + each;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * kOwn + i;
        if (s < n && writes) {
            a.q_starts[s] = static_cast<int32_t>(min(at[i][0], static_cast<uint32_t>(a.max_rows)));
            a.ctx_lens[s] = got[i] ? ctx[i] : 0;
        }
    }
    if (in_place) cluster_wait();   // the other CTAs have read the counters, too, which these are in the place of
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int s = tid * kOwn + i;
        if (s < n && writes) a.pool.held_out[s] = held[i] + static_cast<int>(v[i][1]);
    }
    if (rank == 0 && tid == 0) {
        a.q_starts[n] = static_cast<int32_t>(min(total[0], static_cast<uint32_t>(a.max_rows)));
        *a.pool.n_free_out = static_cast<int32_t>(there - n_taken);
    }
}

template <int kOwn, int kRun>
cudaError_t run(const PlanArgs& a, int threads, bool in_place, cudaStream_t stream)
{
    const int smem = 4 * (4 * ((a.n_seqs + 3) & ~3) + 1);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_on_device(done, [] { return cudaFuncSetAttribute(kv4_plan_kernel<kOwn, kRun>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (4 * kMaxSeqs + 1)); });
    if (e != cudaSuccess) return e;
    const long long jobs = (a.max_rows + kRun - 1ll) / kRun + a.n_seqs;
    // Threads of a CTA that take jobs: 256 where the CTAs are enough for that, all where they are not (4096 requests, 262 k rows:
    // 13.0 us with 256, 7.2 with all; 31 k rows 5.9 and 5.9).
    const int workers = in_place || jobs > static_cast<long long>(device_sms()) * kFewThreads ? threads : kFewThreads;
    const int ranks = static_cast<int>(std::max(1ll, std::min((jobs + workers - 1) / workers, in_place ? kRanks + 0ll : device_sms() + 0ll)));
    PdlLaunch l(dim3(ranks), threads, smem, stream);
    cudaLaunchAttribute attr[2];
    attr[0] = l.attr[0];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    l.cfg.attrs = attr;
    l.cfg.numAttrs = in_place ? 2 : 1;
    e = cudaLaunchKernelEx(&l.cfg, kv4_plan_kernel<kOwn, kRun>, a, ranks, workers, (threads + ranks - 1) / ranks, in_place);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_kv4_plan(const PlanArgs& a, cudaStream_t stream)
{
    // Measured (us): a kernel that runs once is bound by the reading of its code, too: one sequence to a thread and one row to a
    // job where that does (64 requests 2.5, in code for four of each 5.1; 256 of 68 rows 3.2 and 4.8).  As many threads as that
    // needs (300 requests 3.3, with 1024 threads 3.8), 256 at least, as long as the CTAs hold the rows (256 requests, 128 k rows:
    // 5.8, with 1024 threads 4.2; in place, 15 k rows: 8.9 and 4.8, 4 k rows 3.7 both).  Runs of four rows only where a cluster's
    // threads would go through more than two rounds (in place, 4096 requests: 31 k rows 8.3 and, one by one, 9.7; 16 k rows
    // 8.4 and 7.2).
    const bool in_place = a.pool.n_free_out == a.pool.n_free || a.pool.held_out == a.pool.held;
    const int fewest = std::min(std::max((a.n_seqs + 255) / 256 * 256, kFewThreads), kMaxThreads);
    const int threads = a.max_rows <= fewest * (in_place ? 2 * kRanks : device_sms()) ? fewest : kMaxThreads;
    const bool runs = in_place && a.max_rows > 2 * kRanks * threads;
    if (a.n_seqs <= kMaxThreads) return runs ? run<1, 4>(a, threads, in_place, stream) : run<1, 1>(a, threads, in_place, stream);
    return runs ? run<kMostOwn, 4>(a, threads, in_place, stream) : run<kMostOwn, 1>(a, threads, in_place, stream);
}

}  // namespace lora
