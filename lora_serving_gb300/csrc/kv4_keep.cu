// kv4_keep.cu -- the accepted rows of drafted trees move up in the 4-bit
// caches: position base + path[i] becomes base + i, bytes as they are.
//
// A CTA takes a sequence in one layer's cache, a warp a kv head.  A lane holds
// the same columns of every position it moves (a word of K's codes, a half
// word of V's, a parameter), so a position that is both read and written is so
// by one thread in program order: kBatch moves are read before the first is
// written, and since path[i] >= i rises no later move reads what an earlier
// one wrote.
#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 8;

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_keep_kernel(const __grid_constant__ KeepArgs a)
{
    constexpr int kGroups = D / kv4::kGroup, kWords = D / 8;   // parameters, and words of codes, of a position of K
    const int s = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int32_t* const status = tid == 0 ? a.status : nullptr;
    kv4::Seq q;
    if (!kv4::load_seq(a.batch, s, q, status)) return;
    const int base = q.ctx - q.n;
    if (base < 0) return;   // a sequence without a place
    const int keep = __ldg(a.n_keep + s);
    if (keep < 0 || keep > q.n || keep > a.ld_path) {
        flag(status, LORA_DEV_BAD_SEGMENT);
        return;
    }
    const int32_t* path = a.path + static_cast<long long>(s) * a.ld_path;
    const int32_t* table = a.batch.block_table + static_cast<long long>(s) * a.batch.ld_table;
    const KeepArgs::Pages pages = a.layers[layer];
    const int ps = a.cache.page_size, shift = a.cache.page_shift;
    auto page_ok = [&](int p) { return static_cast<uint32_t>(__ldg(table + (p >> shift))) < static_cast<uint32_t>(pages.n_pages); };
    // ---- the whole path before anything moves (every warp for itself: they all see the same)
    bool rises = true, there = true, moves = false;
    for (int i0 = 0; i0 < keep; i0 += 32) {
        const int i = i0 + lane;
        if (i >= keep) break;
        const int at = __ldg(path + i), last = i > 0 ? __ldg(path + i - 1) : -1;
        const bool ok = at > last && at >= i && at < q.n;
        rises &= ok;
        if (ok && at != i) {
            moves = true;
            there &= page_ok(base + at) && page_ok(base + i);
        }
    }
    rises = __all_sync(0xFFFFFFFFu, rises);
    there = __all_sync(0xFFFFFFFFu, there);
    if (!rises) {
        flag(status, LORA_DEV_BAD_POSITION);
        return;
    }
    if (a.lens && layer == 0 && tid == 0) a.lens[s] = base + keep;
    if (!there) {
        flag(status, LORA_DEV_BAD_PAGE);
        return;
    }
    if (!__any_sync(0xFFFFFFFFu, moves)) return;
    // ---- a lane's columns: byte offsets in a block, and what a position adds to them
    const bool codes = lane < kWords, k_par = lane >= kWords && lane < kWords + kGroups, v_half = lane < D / 4, v_par = lane < 2 * kGroups;
    const int k_at = codes ? 4 * lane : kv4::k_params_off(ps, D) + 4 * (lane - kWords), k_step = codes ? D / 2 : 4 * kGroups;
    const int v_at = kv4::v_codes_off(ps, D) + 4 * lane;
    const int p_at = kv4::v_params_off(ps, D) + (lane >> 1) * 8 + (lane & 1) * 4;
    const long long head_bytes = kv4::block_bytes(ps, D);
    for (int i0 = 0; i0 < keep; i0 += 32) {
        // a lane to a move: where it comes from and goes to
        const int i = i0 + lane, from = i < keep ? __ldg(path + i) : i;
        long long src = 0, dst = 0;
        int so = 0, d_o = 0;
        const bool move = from != i;
        if (move) {
            src = __ldg(table + ((base + from) >> shift)) * pages.page_stride;
            dst = __ldg(table + ((base + i) >> shift)) * pages.page_stride;
            so = (base + from) & (ps - 1);
            d_o = (base + i) & (ps - 1);
        }
        const unsigned all = __ballot_sync(0xFFFFFFFFu, move);
        for (int h = warp; h < a.cache.n_kv; h += kWarps) {
            uint8_t* const block = pages.pages + h * head_bytes;
            for (unsigned todo = all; todo;) {
                uint32_t k[kBatch];
                uint16_t v[kBatch], p[kBatch];
                unsigned left = todo;
#pragma unroll
                for (int m = 0; m < kBatch; ++m) {
                    const int who = left ? __ffs(left) - 1 : 0;
                    const uint8_t* b = block + __shfl_sync(0xFFFFFFFFu, src, who);
                    const int o = __shfl_sync(0xFFFFFFFFu, so, who);
                    if (left) {
                        if (codes || k_par) k[m] = *reinterpret_cast<const uint32_t*>(b + k_at + o * k_step);
                        if (v_half) v[m] = *reinterpret_cast<const uint16_t*>(b + v_at + (o >> 1) * D + 2 * (o & 1));
                        if (v_par) p[m] = *reinterpret_cast<const uint16_t*>(b + p_at + (o >> 1) * (8 * kGroups) + 2 * (o & 1));
                    }
                    left &= left - 1;
                }
#pragma unroll
                for (int m = 0; m < kBatch; ++m) {
                    const int who = todo ? __ffs(todo) - 1 : 0;
                    uint8_t* b = block + __shfl_sync(0xFFFFFFFFu, dst, who);
                    const int o = __shfl_sync(0xFFFFFFFFu, d_o, who);
                    if (todo) {
                        if (codes || k_par) *reinterpret_cast<uint32_t*>(b + k_at + o * k_step) = k[m];
                        if (v_half) *reinterpret_cast<uint16_t*>(b + v_at + (o >> 1) * D + 2 * (o & 1)) = v[m];
                        if (v_par) *reinterpret_cast<uint16_t*>(b + p_at + (o >> 1) * (8 * kGroups) + 2 * (o & 1)) = p[m];
                    }
                    todo &= todo - 1;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv4_keep(const KeepArgs& a, int n_layers, cudaStream_t stream)
{
    PdlLaunch l(dim3(a.batch.n_seqs, n_layers), kThreads, 0, stream);
    const cudaError_t e = a.cache.head_dim == 64 ? cudaLaunchKernelEx(&l.cfg, kv4_keep_kernel<64>, a) : cudaLaunchKernelEx(&l.cfg, kv4_keep_kernel<128>, a);
    note_launch();
    return e;
}

}  // namespace lora
