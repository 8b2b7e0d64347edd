// kv4_many.cu -- attention of many query rows (prompts, chunks) over the
// paged 4-bit cache on the 5th-generation tensor cores.
//
// Work.  An item is (sequence, kv head, 256 query rows), rows being a
// sequence's positions x the heads of the group, so that the heads that
// share a kv head share its tiles.  Two tiles of 128 rows take turns on the
// tensor cores: while one's scores go through the softmax, the other's
// products run.
//
// Tile of 128 positions.  Four warps unpack the tile's codes to fp16 values
// in shared memory, K as [position][dim] and V transposed as
// [dim][position], both in the 128-byte-swizzled K-major form; one thread
// issues S = Q K^T (fp32 in tensor memory) and O += P V, P being read from
// tensor memory, where it takes the place of S.  Four warps per tile of rows do
// the softmax, one row to a thread: no row needs another thread's numbers.
// The running maximum moves only when a score passes it by 2^8, so O is
// seldom rescaled.  The dims of a K word come out of their nibbles in the
// order 0 4 1 5 2 6 3 7; Q is laid out in the same order instead of undoing
// it, a sum over dims not minding.
#include <algorithm>
#include <type_traits>

#include "kv4_attend.cuh"
#include "tc_common.cuh"

namespace lora {

namespace {

using namespace kv4;

constexpr int kRowsPerTile = 128, kRowsPerItem = 256;
constexpr int kTok = 128;                  // positions of a tile
constexpr int kSoftWarps = 8, kUnpackWarps = 4, kMmaWarp = kSoftWarps + kUnpackWarps;
constexpr int kWarps = 16, kThreads = 32 * kWarps;   // the MMA warp's three neighbours only scan
// Registers: 128 a thread at launch; the softmax warps, which hold a row's
// weights and the scores on their way, take what the others give up:
// 256 * 184 + 128 * 96 + 128 * 48 = 512 * 128.
constexpr int kSoftRegs = 184, kUnpackRegs = 96, kMmaRegs = 48;
static_assert(2 * kSoftRegs + kUnpackRegs + kMmaRegs <= 4 * 128, "registers");
constexpr float kSlack = 8.f, kLift = 7.f; // as in the kernel for few rows
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Shape {
    static constexpr int kGroups = D / kGroup;
    static constexpr int kWords = D / 32;                 // K words of one lane of the cache's layout
    static constexpr int kQTile = kRowsPerTile * D * 2;   // bytes
    static constexpr int kKTile = kTok * D * 2;
    static constexpr int kVTile = D * kTok * 2;
    static constexpr int kSmem = 2 * kQTile + 2 * kKTile + 2 * kVTile + 1024;   // and alignment
    // tensor memory columns
    static constexpr uint32_t kS = 0, kO = 256;           // S (and P) of tile x at 128 x, O at 256 + D x
};

// kind::f16, fp16 x fp16 -> fp32, both operands K-major.
__device__ constexpr uint32_t idesc_f16(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 columns of this warp's lanes, without waiting for them ...
__device__ __forceinline__ void tmem_ld16_start(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// ... and the wait for every load so far; the registers pass through it, so that no use moves ahead of it.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}

__device__ __forceinline__ void tmem_ld32_start(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// tc::mbar_wait in line: a call would cost the warps with a register budget
// of their own their registers.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity)
{
    if (tc::mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = tc::gtime();
    while (!tc::mbar_try_wait_suspend(bar, parity))
        if (tc::gtime() - t0 > tc::kTimeoutNs) return false;
    return true;
}

template <int kRegs>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;\n"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

struct Barriers {
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2];
};

// What the unpacking warps tell the softmax of a tile, a bit per position:
// positions on a page that the cache does not have, and, where not every row
// sees the whole tile, positions whose V is not finite in a group of dims.
// Four tiles deep: a tile's entry is written again four tiles later, whose
// stage is free only once both softmaxes are past the tile.
template <int kGroups>
struct Notes {
    uint4 hidden[4];
    uint32_t any_sick[4];
    uint32_t sick[4][kGroups][kTok / 32];
};

// Bits [lo, hi) of 32, whatever the bounds.
__device__ __forceinline__ uint32_t bits_in(int lo, int hi)
{
    const uint32_t below_hi = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t below_lo = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below_hi & ~below_lo;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_many_kernel(AttendArgs a, int few_rows)
{
    using S = Shape<D>;
    constexpr int kGroups = S::kGroups, kWords = S::kWords;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ Notes<kGroups> notes;
    __shared__ uint32_t tmem_base;
    __shared__ int sums[kWarps];
    __shared__ int failed;
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* q_s = smem;
    uint8_t* k_s = smem + 2 * S::kQTile;
    uint8_t* v_s = k_s + 2 * S::kKTile;
    int* prefix = reinterpret_cast<int*>(v_s + 2 * S::kVTile);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.k_full[i], kUnpackWarps);
            tc::mbar_init(&bar.v_full[i], kUnpackWarps);
            tc::mbar_init(&bar.k_free[i], 1);
            tc::mbar_init(&bar.v_free[i], 1);
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i], 4);
            tc::mbar_init(&bar.o_full[i], 1);
        }
        tc::mbar_init_fence();
        failed = 0;
    }
    if (tid < 4) notes.any_sick[tid] = 0;
    tc::grid_dep_wait();
    tc::grid_dep_launch();

    // ---- this CTA's item
    const int group = a.n_heads / a.cache.n_kv, ps = a.cache.page_size, n_kv = a.cache.n_kv;
    scan_seqs<kWarps>(a.batch.n_seqs, prefix, sums, [&](int s) {
        Seq q;
        const bool ok = load_seq(a.batch, s, q, blockIdx.x == 0 ? a.status : nullptr);
        return ok && q.n * group > few_rows ? (q.n * group + kRowsPerItem - 1) / kRowsPerItem * n_kv : 0;
    });
    tc::tc_fence_before();
    __syncthreads();   // barriers, the tensor memory's address, the running sum
    tc::tc_fence_after();
    const int item = blockIdx.x;
    const bool work = item < prefix[a.batch.n_seqs];
    const uint32_t tmem = tmem_base;
    if (work) {
        const int s = seq_at(prefix, a.batch.n_seqs, item);
        Seq q;
        load_seq(a.batch, s, q, nullptr);
        const int of = (prefix[s + 1] - prefix[s]) / n_kv, in = item - prefix[s];
        const int h = in % n_kv, block0 = (of - 1 - in / n_kv) * kRowsPerItem;   // the last rows see most: they come first
        const int rows = min(kRowsPerItem, q.n * group - block0);                // of this item
        const int tiles_q = rows > kRowsPerTile ? 2 : 1;
        // positions of the item's first and last row, and the positions that any of them sees
        const int p0 = q.ctx - q.n + block0 / group, p1 = q.ctx - q.n + (block0 + rows - 1) / group;
        const int j_begin = a.window > 0 ? max(0, p0 - a.window + 1) : 0, j_end = max(0, p1 + 1);
        const int tile0 = j_begin / kTok, n_tiles = max(1, (j_end + kTok - 1) / kTok - tile0);
        const int32_t* table = a.batch.block_table + static_cast<long long>(s) * a.batch.ld_table;
        auto inner = [&](int j, int lo, int hi) {   // rows at positions lo..hi see all of tile j
            const int c = (tile0 + j) * kTok;
            return c + kTok - 1 <= lo && (a.window == 0 || c > hi - a.window);
        };

        if (warp < kSoftWarps) {
            more_registers<kSoftRegs>();
            const int x = warp >> 2, r = x * kRowsPerTile + (tid & 127);   // row of the item
            // ---- Q: one row to a thread, taken to fp16 with a power of two, into the swizzled tile
            const int row = block0 + r;
            const bool live = r < rows;
            const int pos = q.ctx - q.n + row / group;
            float mult = 0.f;
            if (x < tiles_q) {
                const bf16_t* qp = a.q + static_cast<long long>(q.row0 + row / group) * a.ld_q + (h * group + row % group) * D;
                float top = 0.f;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = live ? *reinterpret_cast<const uint4*>(qp + 8 * c) : make_uint4(0, 0, 0, 0);
                    const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(p[e])), fabsf(bf16_hi(p[e]))));
                }
                const int fe = min(261 - static_cast<int>(__float_as_uint(top) >> 23), 253);
                float up = top > 0.f ? __uint_as_float(static_cast<uint32_t>(fe) << 23) : 1.f;
                const float down = top > 0.f ? __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) : 1.f;
                mult = fabsf(a.scale) * 1.4426950408889634f * down;   // scores in log2, never a negative factor
                if (a.scale < 0.f) up = -up;
                uint8_t* dst = q_s + x * S::kQTile;
                const int rt = tid & 127;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = live ? *reinterpret_cast<const uint4*>(qp + 8 * c) : make_uint4(0, 0, 0, 0);
                    const float f[8] = {bf16_lo(v.x) * up, bf16_hi(v.x) * up, bf16_lo(v.y) * up, bf16_hi(v.y) * up,
                                        bf16_lo(v.z) * up, bf16_hi(v.z) * up, bf16_lo(v.w) * up, bf16_hi(v.w) * up};
                    const uint4 o = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
                    *reinterpret_cast<uint4*>(dst + (c >> 3) * (kRowsPerTile * 128) + rt * 128 + (((c & 7) ^ (rt & 7)) << 4)) = o;
                }
            }
            tc::fence_async_smem();
            tc::named_barrier(1, 32 * (kSoftWarps + 1));   // Q is in place (the MMA warp waits too)

            // ---- softmax
            if (x < tiles_q) {
                const int x0 = block0 + x * kRowsPerTile, x1 = block0 + min(rows, (x + 1) * kRowsPerTile) - 1;
                const int lo = q.ctx - q.n + x0 / group, hi = q.ctx - q.n + x1 / group;
                const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 lanes of tensor memory, << 16
                const uint32_t ts = tmem + lanes + S::kS + 128 * x, to = tmem + lanes + S::kO + D * x;
                const float inf = __int_as_float(0x7F800000);
                float top = -inf, sum = 0.f;
                uint32_t sick = 0;   // groups of dims in which this row sees a value that is not finite
                bool ok = true;
                for (int j = 0; j < n_tiles; ++j) {
                    if (!wait_for(&bar.s_full[x], j & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                    const uint4 hid4 = notes.hidden[j & 3];
                    const uint32_t hid[4] = {hid4.x, hid4.y, hid4.z, hid4.w};
                    const bool all = inner(j, lo, hi) && (hid4.x | hid4.y | hid4.z | hid4.w) == 0;
                    const int c0 = (tile0 + j) * kTok;
                    // this row sees columns [c_lo, c_hi) of the tile
                    const int c_hi = pos + 1 - c0, c_lo = a.window > 0 ? pos + 1 - a.window - c0 : 0;
                    // Weights against the running maximum as it stands; where a score passes it by 2^8
                    // (always in the first tile) the maximum moves, O is rescaled and they are taken again.
                    uint32_t p[kTok / 2];
                    float2 part[2];
                    for (;;) {
                        const float off = top == -inf ? 0.f : kLift - top;
                        const float2 mult2 = make_float2(mult, mult), off2 = make_float2(off, off);
                        float m[4] = {-inf, -inf, -inf, -inf};
                        part[0] = part[1] = make_float2(0.f, 0.f);
                        auto weigh = [&](auto masked) {
                            constexpr bool kMasked = decltype(masked)::value;
                            uint32_t v[2][32];
                            tmem_ld32_start(ts, v[0]);
#pragma unroll
                            for (int c = 0; c < kTok / 32; ++c) {
                                uint32_t(&w)[32] = v[c & 1];
                                tmem_ld32_wait(w);
                                if (c + 1 < kTok / 32) tmem_ld32_start(ts + 32 * (c + 1), v[(c + 1) & 1]);
                                const uint32_t see = kMasked ? bits_in(c_lo - 32 * c, c_hi - 32 * c) & ~hid[c] : 0u;
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    float2 x2 = make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
                                    if (kMasked) {
                                        if (!((see >> e) & 1u)) x2.x = -inf;
                                        if (!((see >> e) & 2u)) x2.y = -inf;
                                    }
                                    m[(e >> 1) & 3] = fmaxf(m[(e >> 1) & 3], fmaxf(x2.x, x2.y));
                                    float2 y = fma2(x2, mult2, off2);
                                    y.x = ex2(y.x);
                                    y.y = ex2(y.y);
                                    if (kMasked) {   // 0 * -inf with a scale of 0
                                        if (!((see >> e) & 1u)) y.x = 0.f;
                                        if (!((see >> e) & 2u)) y.y = 0.f;
                                    }
                                    part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], y);
                                    p[16 * c + (e >> 1)] = pack_f16x2(y.x, y.y);
                                }
                            }
                        };
                        if (all) weigh(std::false_type{}); else weigh(std::true_type{});
                        float high = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * mult;
                        if (high != high) high = -inf;   // 0 * -inf: nothing seen
                        if (!__any_sync(0xFFFFFFFFu, high > top + kSlack)) break;
                        const float next = fmaxf(high, top);
                        const float keep = next == -inf ? 1.f : ex2(top - next);
                        top = next;
                        sum *= keep;
                        if (j > 0) {
#pragma unroll
                            for (int c = 0; c < D; c += 16) {
                                uint32_t w[16];
                                tmem_ld16_start(to + c, w);
                                tmem_ld16_wait(w);
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * keep);
                                tmem_st16(to + c, w);
                            }
                        }
                    }
                    sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
#pragma unroll
                    for (int c = 0; c < kTok / 2; c += 16) tmem_st16(ts + c, p + c);
                    if (notes.any_sick[j & 3] && !inner(j, p0, p1)) {
                        for (int g = 0; g < kGroups; ++g)
                            for (int c = 0; c < kTok; c += 32)
                                if (notes.sick[j & 3][g][c >> 5] & bits_in(c_lo - c, c_hi - c) & ~hid[c >> 5]) sick |= 1u << g;
                    }
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.p_full[x]);
                }
                // ---- the result
                if (ok) ok = wait_for(&bar.o_full[x], 0);
                tc::tc_fence_after();
                if (ok) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    bf16_t* o = a.out + static_cast<long long>(q.row0 + row / group) * a.ld_out + (h * group + row % group) * D;
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        tc::tmem_ld32(to + c, v);
                        const float k = (sick >> (c / kGroup)) & 1u ? __int_as_float(0x7FC00000) : inv;
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4*>(o + c + e) =
                                    make_uint4(pack_bf16x2(v[e] * k, v[e + 1] * k), pack_bf16x2(v[e + 2] * k, v[e + 3] * k),
                                               pack_bf16x2(v[e + 4] * k, v[e + 5] * k), pack_bf16x2(v[e + 6] * k, v[e + 7] * k));
                        }
                    }
                } else {
                    failed = 1;
                }
            }
        } else if (warp < kMmaWarp) {
            // ---- unpacking: K one position to a thread, V eight positions x 16 dims
            fewer_registers<kUnpackRegs>();
            const int u = tid - 32 * kSoftWarps;
            const int tok8 = u & 15, quad = u >> 4;            // quad: 16 dims of V
            const bool has_v = quad < D / 16;
            uint4 kr[D / 32];
            uint32_t kp[kGroups];
            uint4 vr[4];
            uint2 vp[4];
            // bytes of a place, or null where no row sees it or its page is bad
            auto place = [&](int p) -> const uint8_t* {
                if (p >= j_end) return nullptr;
                const int page = __ldg(table + (p >> a.cache.page_shift));
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.cache.n_pages)) {
                    flag(a.status, LORA_DEV_BAD_PAGE);
                    return nullptr;
                }
                return block_of(a.cache, page, h);
            };
            bool hidden = false;    // this position's page is bad
            uint32_t v_sick = 0;    // this position's groups with a V that is not finite
            auto load_k = [&](int j) {
                const int p = (tile0 + j) * kTok + u, off = p & (ps - 1);
                const uint8_t* b = place(p);
#pragma unroll
                for (int t = 0; t < D / 32; ++t) kr[t] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) kp[g] = 0;
                v_sick = 0;
                hidden = b == nullptr && p < j_end;
                if (b) {
#pragma unroll
                    for (int t = 0; t < D / 32; ++t) kr[t] = __ldg(reinterpret_cast<const uint4*>(b + off * (D / 2)) + t);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) kp[g] = __ldg(reinterpret_cast<const uint32_t*>(b + k_params_off(ps, D)) + off * kGroups + g);
                    if (!inner(j, p0, p1)) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            const uint16_t* w = reinterpret_cast<const uint16_t*>(b + v_params_off(ps, D)) + ((off >> 1) * kGroups + g) * 4 + (off & 1);
                            v_sick |= (not_finite(w[0]) || not_finite(w[2]) ? 1u : 0u) << g;
                        }
                    }
                }
            };
            auto load_v = [&](int j) {
                const int p = (tile0 + j) * kTok + 8 * tok8, off = p & (ps - 1);
                const uint8_t* b = has_v ? place(p) : nullptr;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    vr[i] = make_uint4(0, 0, 0, 0);
                    vp[i] = make_uint2(0, 0);
                }
                if (b) {
                    const uint8_t* c = b + v_codes_off(ps, D) + (off >> 1) * D + 16 * quad;
                    const uint8_t* w = b + v_params_off(ps, D) + ((off >> 1) * kGroups + quad * 16 / kGroup) * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        vr[i] = __ldg(reinterpret_cast<const uint4*>(c + i * D));
                        vp[i] = __ldg(reinterpret_cast<const uint2*>(w + i * 8 * kGroups));
                    }
                    if (!inner(j, p0, p1)) {
                        // positions past the last row's, and values that are not finite, count as zeros
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int at = p + 2 * i;
                            uint32_t keep = (at < j_end ? 0xFFFFu : 0u) | (at + 1 < j_end ? 0xFFFF0000u : 0u);
                            if (not_finite(vp[i].x & 0xFFFFu) || not_finite(vp[i].y & 0xFFFFu)) keep &= 0xFFFF0000u;
                            if (not_finite(vp[i].x & 0xFFFF0000u) || not_finite(vp[i].y & 0xFFFF0000u)) keep &= 0xFFFFu;
                            vp[i].x &= keep;
                            vp[i].y &= keep;
                        }
                    }
                }
            };
            load_k(0);
            load_v(0);
            bool ok = true;
            for (int j = 0; j < n_tiles && ok; ++j) {
                const int st = j & 1;
                if (j >= 2) ok = wait_for(&bar.k_free[st], ((j >> 1) & 1) ^ 1);
                uint8_t* kd = k_s + st * S::kKTile + u * 128;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    // 16 bytes of the row hold words (t, 0..kWords-1)
                    uint32_t w[4];
                    if (kWords == 4) {
                        w[0] = kr[t % (D / 32)].x; w[1] = kr[t % (D / 32)].y; w[2] = kr[t % (D / 32)].z; w[3] = kr[t % (D / 32)].w;
                    } else {
                        const uint4 v = kr[(t >> 1) % (D / 32)];
                        w[0] = t & 1 ? v.z : v.x; w[1] = t & 1 ? v.w : v.y;
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i) {
                        const __half2 pr = as_h2(kp[i / 2]);
                        uint32_t v[4];
                        values(w[i], __low2half2(pr), __high2half2(pr), v);
                        const int c = 4 * (i & 1) + t;
                        *reinterpret_cast<uint4*>(kd + (i >> 1) * (kTok * 128) + ((c ^ (u & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
                const uint32_t gone = __ballot_sync(0xFFFFFFFFu, hidden);
                if (lane == 0) reinterpret_cast<uint32_t*>(&notes.hidden[j & 3])[u >> 5] = gone;
                if (!inner(j, p0, p1)) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, (v_sick >> g) & 1u);
                        if (lane == 0) notes.sick[j & 3][g][u >> 5] = bits;
                    }
                    const bool any = __any_sync(0xFFFFFFFFu, v_sick != 0);
                    if (lane == 0 && any) notes.any_sick[j & 3] = 1;   // stays set: the bits say what is there
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.k_full[st]);
                if (j + 1 < n_tiles) load_k(j + 1);

                if (ok && j >= 2) ok = wait_for(&bar.v_free[st], ((j >> 1) & 1) ^ 1);
                if (has_v) {
                    uint8_t* vd = v_s + st * S::kVTile + (tok8 >> 3) * (D * 128);
                    const uint32_t* raw = reinterpret_cast<const uint32_t*>(vr);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t v[4][4];   // [pair of positions][dim]
#pragma unroll
                        for (int i = 0; i < 4; ++i) values(raw[4 * i + w], as_h2(vp[i].x), as_h2(vp[i].y), v[i]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = 16 * quad + 4 * w + e;
                            *reinterpret_cast<uint4*>(vd + d * 128 + (((tok8 & 7) ^ (d & 7)) << 4)) =
                                make_uint4(v[0][e], v[1][e], v[2][e], v[3][e]);
                        }
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.v_full[st]);
                if (j + 1 < n_tiles) load_v(j + 1);
            }
            if (!ok) failed = 1;
        } else {
            // ---- the products
            fewer_registers<kMmaRegs>();
            if (warp == kMmaWarp) tc::named_barrier(1, 32 * (kSoftWarps + 1));
            if (warp == kMmaWarp && lane == 0) {
                constexpr uint32_t id_s = idesc_f16(kRowsPerTile, kTok), id_o = idesc_f16(kRowsPerTile, D);
                const uint32_t qa = tc::smem_u32(q_s), ka = tc::smem_u32(k_s), va = tc::smem_u32(v_s);
                auto scores = [&](int x, int st) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = (k >> 2) * (128 * 128) + (k & 3) * 32;
                        tc::mma_bf16(tmem + S::kS + 128 * x, tc::sdesc_sw128(qa + x * S::kQTile + at),
                                     tc::sdesc_sw128(ka + st * S::kKTile + at), id_s, k > 0);
                    }
                    tc::mma_commit(&bar.s_full[x]);
                };
                bool ok = tc::mbar_wait_spin(&bar.k_full[0], 0);
                tc::tc_fence_after();
                for (int x = 0; ok && x < tiles_q; ++x) scores(x, 0);
                if (ok) tc::mma_commit(&bar.k_free[0]);
                for (int j = 0; ok && j < n_tiles; ++j) {
                    const int st = j & 1, nx = (j + 1) & 1;
                    ok = tc::mbar_wait_spin(&bar.v_full[st], (j >> 1) & 1);
                    for (int x = 0; ok && x < tiles_q; ++x) {
                        ok = tc::mbar_wait_spin(&bar.p_full[x], j & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
                            mma_ts(tmem + S::kO + D * x, tmem + S::kS + 128 * x + 8 * k,
                                   tc::sdesc_sw128(va + st * S::kVTile + (k >> 2) * (D * 128) + (k & 3) * 32), id_o, j > 0 || k > 0);
                        if (x == tiles_q - 1) tc::mma_commit(&bar.v_free[st]);
                        if (j + 1 < n_tiles) {
                            if (x == 0) {
                                ok = tc::mbar_wait_spin(&bar.k_full[nx], ((j + 1) >> 1) & 1);
                                if (!ok) break;
                                tc::tc_fence_after();
                            }
                            scores(x, nx);
                            if (x == tiles_q - 1) tc::mma_commit(&bar.k_free[nx]);
                        } else {
                            tc::mma_commit(&bar.o_full[x]);
                        }
                    }
                }
                if (!ok) failed = 1;
            }
            __syncwarp();
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && work && failed) flag(a.status, LORA_DEV_TIMEOUT);
}

template <int D>
cudaError_t run(const AttendArgs& a, int few_rows, cudaStream_t stream)
{
    using S = Shape<D>;
    constexpr int kMaxSmem = 226 * 1024;
    static_assert(S::kSmem + 4 * (kMaxSeqs + 1) <= kMaxSmem, "shared memory");
    static bool attr_set = false;
    if (!attr_set) {
        const cudaError_t e = cudaFuncSetAttribute(kv4_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    const int group = a.n_heads / a.cache.n_kv;
    // an upper bound on the items: a sequence's last block may be short
    const long long items = (static_cast<long long>(a.batch.n_rows) * group / kRowsPerItem + a.batch.n_seqs) * a.cache.n_kv;
    PdlLaunch l(dim3(static_cast<unsigned>(items)), kThreads, S::kSmem + 4 * (a.batch.n_seqs + 1), stream);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kv4_many_kernel<D>, a, few_rows);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_kv4_many(const AttendArgs& a, int few_rows, cudaStream_t stream)
{
    return a.cache.head_dim == 64 ? run<64>(a, few_rows, stream) : run<128>(a, few_rows, stream);
}

}  // namespace lora
