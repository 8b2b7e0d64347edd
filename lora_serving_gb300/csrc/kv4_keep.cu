// kv4_keep.cu -- the accepted rows of drafted trees move up in the 4-bit
// caches: position base + path[i] becomes base + i, bytes as they are.
//
// A CTA takes a sequence in some layers' caches; a unit is one of their kv
// heads, always the same warp's.  Eight lanes hold a position (K's codes and
// V's words in eight parts each, its parameters in the first three lanes), so a
// warp has four moves of a unit on their way, and of kTogether units at once:
// where a lane reads and writes is worked out once for all units.  All of a
// batch is read before the first of it is written, and since the path rises,
// path[i] >= i, no later move reads what an earlier one wrote.  For the same
// reason the rows that move are the path's last ones, from the first with
// path[i] > i on.
// Bound: latency, of the tables (path, pages) and then of the positions
// themselves, 144 bytes in four places; beyond that the half words of V, which
// DRAM fetches and writes by sectors.  Measured, start to start: 64 requests in
// 32 layers (14 MB) 9.4 us, a quarter of a copy's rate; one request in 28 layers 2.5.
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMoves = 4;      // of a warp: eight lanes to each
// Units on their way, with the registers for four CTAs on an SM, and units of a CTA, fewer where the CTAs would not be three to
// an SM.  Measured (us, 16 / 64 / 256 requests, 32 layers of 8 heads): 3 and 24 4.7 / 9.2 / 32.6, 2 and 16 4.4 / 9.7 / 35.5, 4 and
// 32 5.4 / 11.2 / 33.2; 2 and 16 in five CTAs 5.1 / 9.8 / 33.4, in six 6.5 / 10.1 / 32.6.  32 requests 6.6, with CTAs for two to an SM 8.0.
constexpr int kTogether = 3, kUnits = 24;

// kBytes adjacent bytes, 4 to 16, in words.
template <int kBytes>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t (&w)[4])
{
    if (kBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if (kBytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) kv4_keep_kernel(const __grid_constant__ KeepArgs a, int n_layers, int layers_each)
{
    constexpr int kGroups = D / kv4::kGroup;
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int layer0 = blockIdx.y * layers_each, units = min(layers_each, n_layers - layer0) * a.cache.n_kv;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int32_t* const status = tid == 0 ? a.status : nullptr;
    // every table entry on its way before the first is looked at
    const int32_t* path = a.path + static_cast<long long>(s) * a.ld_path;
    const int32_t* table = a.batch.block_table + static_cast<long long>(s) * a.batch.ld_table;
    const int keep = __ldg(a.n_keep + s);
    const int held = a.held ? __ldg(a.held + s) : 0;
    const int early = lane < a.ld_path ? __ldg(path + lane) : 0;
    kv4::Seq q;
    if (!kv4::load_seq(a.batch, s, q, status)) return;
    const int base = q.ctx - q.n;
    if (base < 0 || (q.ctx == 0 && held != 0)) return;   // a sequence without a place; with rows or, holding pages, without
    if (keep < 0 || keep > q.n || keep > a.ld_path) {
        flag(status, LORA_DEV_BAD_SEGMENT);
        return;
    }
    const int ps = a.cache.page_size, shift = a.cache.page_shift;
    // ---- the whole path before anything moves (every warp for itself: they all see the same)
    auto from_of = [&](int i) { return i < 32 ? early : __ldg(path + i); };   // i: a lane's of its 32
    bool rises = true;
    uint32_t last_page = 0;   // the largest that a move touches (a negative id: larger than any)
    int first = keep;         // the first row that moves
    for (int i0 = 0; i0 < keep; i0 += 32) {
        const int i = i0 + lane;
        const int at = i < keep ? from_of(i) : 0, up = __shfl_up_sync(0xFFFFFFFFu, at, 1);
        const int before = lane > 0 ? up : i0 > 0 ? __ldg(path + i0 - 1) : -1;
        const bool ok = i >= keep || (at > before && at < q.n && at >= i);
        rises &= ok;
        const bool moves = i < keep && ok && at != i;
        if (moves) last_page = max(last_page, max(static_cast<uint32_t>(__ldg(table + ((base + at) >> shift))), static_cast<uint32_t>(__ldg(table + ((base + i) >> shift)))));
        const unsigned who = __ballot_sync(0xFFFFFFFFu, moves);
        if (who) first = min(first, i0 + __ffs(who) - 1);
    }
    if (!__all_sync(0xFFFFFFFFu, rises)) {
        flag(status, LORA_DEV_BAD_POSITION);
        return;
    }
    last_page = __reduce_max_sync(0xFFFFFFFFu, last_page);
    // (a sequence whose rows one of the caches cannot move has none of them from now on)
    if (a.lens && layer0 == 0 && tid == 0 && last_page < static_cast<uint32_t>(a.least_pages)) a.lens[s] = base + keep;
    if (first == keep) return;
    if (tid < min(layers_each, n_layers - layer0) && last_page >= static_cast<uint32_t>(a.layers[layer0 + tid].n_pages)) flag(a.status, LORA_DEV_BAD_PAGE);

    // ---- a lane's part of a position: kK bytes of K's codes, the halves of kV / 4 words of V; lane 0 K's parameters,
    // lanes 1..kGroups those of a group of V
    constexpr int kK = D / 16, kV = D / 8;
    const int part = lane & 7, n_kv = a.cache.n_kv;
    const long long head_bytes = kv4::block_bytes(ps, D);
    auto k_at = [&](int o) { return o * (D / 2) + part * kK; };
    auto v_at = [&](int o) { return kv4::v_codes_off(ps, D) + (o >> 1) * D + part * kV; };
    auto p_at = [&](int o) { return part == 0 ? kv4::k_params_off(ps, D) + o * 4 * kGroups : kv4::v_params_off(ps, D) + ((o >> 1) * kGroups + part - 1) * 8; };
    for (int m0 = first; m0 < keep; m0 += kMoves) {
        const int i = m0 + (lane >> 3);
        const bool mine = i < keep;
        const int from = base + (mine ? __ldg(path + i) : 0), to = base + i;
        const long long src_page = mine ? __ldg(table + (from >> shift)) : 0, dst_page = mine ? __ldg(table + (to >> shift)) : 0;
        const int so = from & (ps - 1), d_o = to & (ps - 1);
        const int sk = k_at(so), sv = v_at(so), sp = p_at(so), dk = k_at(d_o), dv = v_at(d_o) + 2 * (d_o & 1), dp = p_at(d_o) + (part ? 2 * (d_o & 1) : 0);
        const int half = 16 * (so & 1);
        for (int u0 = warp; u0 < units; u0 += kTogether * kWarps) {
            uint32_t k[kTogether][4], v[kTogether][4], p[kTogether][4];
            uint8_t* block[kTogether];
#pragma unroll
            for (int x = 0; x < kTogether; ++x) {
                const int u = u0 + x * kWarps, layer = layer0 + u / n_kv;
                block[x] = nullptr;
                if (u >= units || last_page >= static_cast<uint32_t>(a.layers[layer].n_pages)) continue;
                uint8_t* const b = a.layers[layer].pages + (u % n_kv) * head_bytes;
                if (!mine) continue;
                const uint8_t* from_b = b + src_page * a.layers[layer].page_stride;
                block[x] = b + dst_page * a.layers[layer].page_stride;
                load_bytes<kK>(from_b + sk, k[x]);
                load_bytes<kV>(from_b + sv, v[x]);
                if (part == 0) load_bytes<4 * kGroups>(from_b + sp, p[x]);
                else if (part <= kGroups) load_bytes<8>(from_b + sp, p[x]);
            }
            __syncwarp();   // other lanes write what these have read
#pragma unroll
            for (int x = 0; x < kTogether; ++x) {
                if (!block[x]) continue;
                uint8_t* const b = block[x];
                if (kK == 8) *reinterpret_cast<uint2*>(b + dk) = make_uint2(k[x][0], k[x][1]);
                else *reinterpret_cast<uint32_t*>(b + dk) = k[x][0];
#pragma unroll
                for (int w = 0; w < kV / 4; ++w) *reinterpret_cast<uint16_t*>(b + dv + 4 * w) = static_cast<uint16_t>(v[x][w] >> half);
                if (part == 0) {
                    if (kGroups == 2) *reinterpret_cast<uint2*>(b + dp) = make_uint2(p[x][0], p[x][1]);
                    else *reinterpret_cast<uint32_t*>(b + dp) = p[x][0];
                } else if (part <= kGroups) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) *reinterpret_cast<uint16_t*>(b + dp + 4 * w) = static_cast<uint16_t>(p[x][w] >> half);
                }
            }
            __syncwarp();   // and the next batch comes after
        }
    }
}

}  // namespace

cudaError_t launch_kv4_keep(const KeepArgs& a, int n_layers, cudaStream_t stream)
{
    int each = std::max(1, std::min(n_layers, kUnits / a.cache.n_kv));
    while (each > 1 && static_cast<long long>(a.batch.n_seqs) * ((n_layers + each - 1) / each) < 3 * device_sms()) --each;
    PdlLaunch l(dim3(a.batch.n_seqs, (n_layers + each - 1) / each), kThreads, 0, stream);
    const cudaError_t e = a.cache.head_dim == 64 ? cudaLaunchKernelEx(&l.cfg, kv4_keep_kernel<64>, a, n_layers, each) : cudaLaunchKernelEx(&l.cfg, kv4_keep_kernel<128>, a, n_layers, each);
    note_launch();
    return e;
}

}  // namespace lora
