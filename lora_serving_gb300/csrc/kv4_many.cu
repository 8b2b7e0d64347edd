// kv4_many.cu -- attention of many query rows (prompts, chunks) over the
// paged 4-bit cache on the 5th-generation tensor cores.
//
// Work.  An item is (sequence, kv head, 256 query rows), rows being a
// sequence's positions x the heads of the group, so that the heads that
// share a kv head share its tiles.  Two tiles of 128 rows take turns on the
// tensor cores.  All items' tiles of positions laid end to end are cut into
// equal ranges, one per SM, an item counting kItemCost tiles more than it
// has, for its start and end; an item cut by a range's end leaves partial
// results, which a second kernel joins in a fixed order.
//
// Tile of 128 positions.  Four warps unpack K's codes to fp16 values in shared
// memory, as [position][dim], four warps V's, transposed as [dim][position],
// both in the 128-byte-swizzled K-major form; one thread per tile of rows
// issues S = Q K^T (fp32 in tensor memory) and O += P V, P being read from
// tensor memory, where it takes the place of S.  Four warps per tile of rows
// do the softmax, one row to a thread: no row needs another thread's numbers.
// The issuing threads take turns: the tensor cores serve two threads in
// alternation, which drew the tiles of rows into step, both waiting for their
// products at the same time and then both at the softmax.
// The running maximum moves only when a score passes it by 2^8, so O is
// seldom rescaled.  The dims of a K word come out of their nibbles in the
// order 0 4 1 5 2 6 3 7; Q is laid out in the same order instead of undoing
// it, a sum over dims not minding.
//
// From item to item.  The warps that unpack K copy the next item's Q as soon
// as the last scores of this one are there, and its first scores are computed
// while this one's result is written.
//
// What bounds it.  The two products take 2150 of an SM's clocks a tile, a
// tile of rows' own chain (softmax 1500, products 1075 and the ways between
// them) 3150 to 3300.  After that, an item's masked tile, Q and result, and the
// code's size: five roles share the SM's instruction cache, so what is seldom
// run (masked tiles, results, finding the pieces) is written small, as loops,
// and once: 115 KB instead of 80 took 16 prompts 357 us instead of 305.  A
// first tile that all rows see begins with its first columns' maximum: in the
// masked tiles' code it took the prompts 302 us, a chunk, where another test
// stands in every tile, 735.
//
// Measured: 1024 rows of 64 heads over 32768 positions 745 to 755 us (1.44
// PFLOP/s, 0.73 of the measured bf16 peak); 16 prompts of 149 to 2011 tokens,
// 32 heads, 290 us.
#include <algorithm>
#include <type_traits>

#include "kv4_attend.cuh"
#include "tc_common.cuh"

namespace lora {

namespace {

using namespace kv4;

constexpr int kRowsPerTile = 128, kRowsPerItem = 256;
constexpr int kTok = 128;                  // positions of a tile
constexpr int kStages = 2;                 // tiles of K, and of V, in shared memory
constexpr int kSoftWarps = 8, kVWarp = 12, kMmaWarp = 16;
constexpr int kWalkWarp = 18;              // beside the two MMA warps
constexpr int kWarps = 20, kThreads = 32 * kWarps;
constexpr int kPieces = 4;                 // pieces that the walking warp is ahead
constexpr int kNotes = 4;                  // tiles of which the softmax has notes (see Notes)
// Registers: 96 a thread at launch; the softmax warps, which hold a row's
// scores and weights, take what the others give up:
// 256 * 144 + 256 * 80 + 128 * 32 <= 640 * 96.
constexpr int kSoftRegs = 144, kUnpackRegs = 80, kMmaRegs = 32;
static_assert(2 * kSoftRegs + 2 * kUnpackRegs + kMmaRegs <= 5 * 96, "registers");
constexpr int kItemCost = 4;               // an item's start and end, in tiles
constexpr int kMinRange = 6;               // a CTA's range, at least
constexpr float kSlack = 8.f, kLift = 7.f; // as in the kernel for few rows
constexpr uint32_t kTmemCols = 512;
constexpr int kOutBytes = 32 * 64;         // a softmax warp's part of the result on its way out: 32 dims of 32 rows

template <int D>
struct Shape {
    static constexpr int kGroups = D / kGroup;
    static constexpr int kWords = D / 32;                 // K words of one lane of the cache's layout
    static constexpr int kQTile = kRowsPerTile * D * 2;   // bytes
    static constexpr int kKTile = kTok * D * 2;
    static constexpr int kVHalf = D * 64 * 2, kVTile = 2 * kVHalf;   // [64 positions each][dim][position]
    static constexpr int kSmem = 2 * kQTile + kStages * (kKTile + kVTile) + kSoftWarps * kOutBytes + 1024;   // and alignment
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
// Keeps uses of loaded registers behind the wait before it.
__device__ __forceinline__ void after_wait(uint32_t (&r)[32])
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Bounded waits, in line and timed by the SM's clock: a read of the global
// timer, before the first poll, took longer than most waits here.
constexpr long long kTimeoutClocks = 400000000;   // 0.2 s at 2 GHz
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity, long long limit = kTimeoutClocks)
{
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity))
        if (clock64() - t0 > limit) return false;
    return true;
}
// Polling, for the thread that feeds the tensor cores.
__device__ __forceinline__ bool wait_polling(uint64_t* bar, unsigned parity)
{
    if (tc::mbar_test_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_test_wait(bar, parity))
        if (clock64() - t0 > kTimeoutClocks) return false;
    return true;
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
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
    uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
    uint64_t q_raw[2], q_full[2], q_free[2];   // of a tile of rows: Q as copied, as the products want it, done with
    uint64_t s_full[2], p_full[2];
    uint64_t o_full[2];
    uint64_t turn[2];                // a tile of rows' products may be issued
    uint64_t piece_full[kPieces], piece_free[kPieces];
};

// What the unpacking warps tell the softmax of a tile, a bit per position:
// positions on a page that the cache does not have, and, where not every row
// sees the whole tile, positions whose V is not finite in a group of dims.
// A tile's entry is written again four tiles later: that tile's stage of K is
// free once both products of two tiles earlier are done, and these follow the
// softmax of the tile before.
template <int kGroups>
struct Notes {
    uint4 hidden[kNotes];
    uint32_t any_sick[kNotes];
    uint32_t sick[kNotes][kGroups][kTok / 32];
};

// Bits [lo, hi) of 32, whatever the bounds.
__device__ __forceinline__ uint32_t bits_in(int lo, int hi)
{
    const uint32_t below_hi = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t below_lo = lo >= 32 ? 0xFFFFFFFFu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below_hi & ~below_lo;
}

// 256 query rows of a sequence: its rows [row0, row0 + rows) of positions x
// heads, the positions of the first and the last, and the tiles they see.
struct Block {
    int row0, rows, p0, p1, tile0, tiles;
};
__device__ __forceinline__ Block block_at(const Seq& q, int i, int group, int window)
{
    Block b;
    b.row0 = i * kRowsPerItem;
    b.rows = min(kRowsPerItem, q.n * group - b.row0);
    b.p0 = q.ctx - q.n + b.row0 / group;
    b.p1 = q.ctx - q.n + (b.row0 + b.rows - 1) / group;
    b.tile0 = seen_from(b.p0, window) / kTok;
    b.tiles = max(1, (max(0, b.p1 + 1) + kTok - 1) / kTok - b.tile0);   // at least one: its rows get their zeros
    return b;
}

// A range's part of an item, in shared memory: one warp walks the range, the
// others wait for what it finds (a walk in each role's code doubled the
// kernel's instructions).
struct Piece {
    int s, h, row0;      // sequence, kv head, the batch row of the sequence's first
    int block, rows;     // the block's rows are [block, block + rows) of the sequence's
    int pos0, p0, p1;    // positions of the sequence's first row, of the block's first and last
    int tile0, tiles;    // the piece's tiles; 0: the range has ended
    int base;            // tiles of the range before it
    int starts, ends;    // whether the item begins, ends with it
    int last;            // the last CTA with a part of an item that begins but does not end here
};
struct Held : Piece {    // a softmax warp's copy
    int all0, all1;      // all of its tile of rows sees all of these tiles of the piece, [all0, all1)
};

__device__ __forceinline__ int range_count(int total, int ctas) { return min(ctas, max(1, total / kMinRange)); }
// total * b / n without leaving 32 bits (n is a number of CTAs)
__device__ __forceinline__ int range_at(int total, int n, int b)
{
    b = min(b, n);
    return total / n * b + total % n * b / n;
}

// A place on the line: block i of sequence s, which begins at `at`.
struct Place {
    int s, i, at;
    Seq q;
    Block b;
};

// Finds the pieces of a CTA's range.  The line goes by blocks of rows in the
// order of the sequences, the kv heads of a block one after another.
struct Walk : Place {
    const AttendArgs& a;
    const int* prefix;   // blocks before each sequence
    int group, share, x, end, base = 0;   // share: places of a range; x: place on the line

    __device__ __forceinline__ Walk(const AttendArgs& args, const int* pre, const Place& start, int share_, int begin, int end_)
        : Place(start), a(args), prefix(pre), group(args.n_heads / args.cache.n_kv), share(share_), x(begin), end(end_)
    {
    }
    __device__ __forceinline__ void next_block()
    {
        at += (b.tiles + kItemCost) * a.cache.n_kv;
        if (prefix[s] + ++i == prefix[s + 1]) {
            i = 0;
            do ++s; while (prefix[s] == prefix[s + 1]);
        }
        load_seq(a.batch, s, q, nullptr);
        b = block_at(q, i, group, a.window);
    }
    // The next piece; the place at which its item ends, 0 after the last.
    __device__ __forceinline__ int next(Piece& p)
    {
        while (x < end) {
            const int len = b.tiles + kItemCost;
            if (x >= at + len * a.cache.n_kv) {
                next_block();
                continue;
            }
            p.h = (x - at) / len;
            const int u0 = at + p.h * len;
            int t0 = max(0, x - u0 - kItemCost), t1 = max(0, min(len, end - u0) - kItemCost);
            if (8 * len <= share) {
                // An item that is short beside a range is not cut, since a cut costs partial results: it goes to
                // the range that its middle lies in.
                if (u0 + len / 2 < x || u0 + len / 2 >= end) t1 = t0; else { t0 = 0; t1 = b.tiles; }
            }
            x = min(end, u0 + len);
            if (t0 == t1) continue;   // nothing of it, or only its start, lies in the range
            p.s = s;
            p.row0 = q.row0;
            p.block = b.row0;
            p.rows = b.rows;
            p.pos0 = q.ctx - q.n;
            p.p0 = b.p0;
            p.p1 = b.p1;
            p.tile0 = b.tile0 + t0;
            p.tiles = t1 - t0;
            p.base = base;
            p.starts = t0 == 0;
            p.ends = t1 == b.tiles;
            base += p.tiles;
            return u0 + len;
        }
        p.tiles = 0;
        return 0;
    }
};
constexpr int kMaxCtas = 160;   // CTAs that the workspace has room for

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_many_kernel(AttendArgs a, int few_rows, Partials left)
{
    using S = Shape<D>;
    constexpr int kGroups = S::kGroups, kWords = S::kWords;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ Barriers bar;
    __shared__ Notes<kGroups> notes;
    __shared__ Place first;
    __shared__ Piece pieces[kPieces];
    __shared__ Held held[kSoftWarps][2];
    constexpr int kPieceWords = sizeof(Piece) / 4;
    static_assert(kPieceWords <= 32, "a lane to a word");
    __shared__ uint32_t tmem_base;
    __shared__ int sums[kWarps];
    __shared__ int failed;
    uint8_t* smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* q_s = smem;
    uint8_t* k_s = smem + 2 * S::kQTile;
    uint8_t* v_s = k_s + kStages * S::kKTile;
    uint8_t* out_s = v_s + kStages * S::kVTile;
    int* cost = reinterpret_cast<int*>(out_s);   // until the ranges' places are known
    static_assert(sizeof(int) * (kThreads + 1) <= kSoftWarps * kOutBytes, "shared memory");
    int* prefix = reinterpret_cast<int*>(out_s + kSoftWarps * kOutBytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;

    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&bar.k_full[i], 4);   // four warps
            tc::mbar_init(&bar.v_full[i], 4);
            tc::mbar_init(&bar.k_free[i], 2);   // both tiles' products
            tc::mbar_init(&bar.v_free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.q_raw[i], 128);   // the threads that unpack K
            tc::mbar_init(&bar.q_full[i], 4);
            tc::mbar_init(&bar.q_free[i], 1);
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i], 4);
            tc::mbar_init(&bar.o_full[i], 1);
            tc::mbar_init(&bar.turn[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            tc::mbar_init(&bar.piece_full[i], 1);
            tc::mbar_init(&bar.piece_free[i], kWalkWarp);   // the other roles' warps
        }
        tc::mbar_init_fence();
        failed = 0;
    }
    if (tid < kNotes) notes.any_sick[tid] = 0;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (tid == 0) left.records[blockIdx.x].rows = 0;

    // ---- this CTA's range: blocks before each sequence, then places before each thread's share of the blocks; the
    // thread in whose share the range begins finds its first block
    const int group = a.n_heads / a.cache.n_kv, ps = a.cache.page_size;
    Seq* const seqs = reinterpret_cast<Seq*>(k_s);   // until K is there
    static_assert(sizeof(Seq) * kMaxSeqs <= kStages * (S::kKTile + S::kVTile), "shared memory");
    bool falls = false;   // q_starts decreases: the sequences together may have more rows than the batch, and more tiles than are counted in 31 bits
    scan_seqs<kWarps>(a.batch.n_seqs, prefix, sums, [&](int s) {
        Seq q;
        const bool ok = load_seq(a.batch, s, q, blockIdx.x == 0 ? a.status : nullptr);
        seqs[s] = q;
        falls |= !ok && __ldg(a.batch.q_starts + s + 1) < __ldg(a.batch.q_starts + s);
        return ok && q.n * group > few_rows ? (q.n * group + kRowsPerItem - 1) / kRowsPerItem : 0;
    });
    const int blocks = __syncthreads_or(falls) ? 0 : prefix[a.batch.n_seqs], per = (blocks + kThreads - 1) / kThreads;
    Place mine;
    auto block = [&](int f) {
        mine.s = seq_at(prefix, a.batch.n_seqs, f);
        mine.i = f - prefix[mine.s];
        mine.q = seqs[mine.s];
        mine.b = block_at(mine.q, mine.i, group, a.window);
        return (mine.b.tiles + kItemCost) * a.cache.n_kv;
    };
    scan_seqs<kWarps>(kThreads, cost, sums, [&](int t) {
        int sum = 0;
#pragma unroll 1
        for (int f = t * per; f < min(blocks, (t + 1) * per); ++f) sum += block(f);
        return sum;
    });
    const int total = cost[kThreads], n_ranges = range_count(total, gridDim.x);
    const int begin = range_at(total, n_ranges, blockIdx.x), end = range_at(total, n_ranges, blockIdx.x + 1);
    if (begin < end && cost[tid] <= begin && begin < cost[tid + 1]) {
        mine.at = cost[tid];
        int len;
#pragma unroll 1
        for (int f = tid * per; begin >= mine.at + (len = block(f)); ++f) mine.at += len;
        first = mine;
    }
    tc::tc_fence_before();
    __syncthreads();   // barriers, the tensor memory's address, the running sums
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;
    {
        // The n-th piece of the range, null after the last (or with ok false); a warp gives it back when it is done with it.
        bool ok = true;
        auto piece = [&](int n) -> const Piece* {
            ok = ok && wait_for(&bar.piece_full[n % kPieces], (n / kPieces) & 1);
            return ok && pieces[n % kPieces].tiles ? &pieces[n % kPieces] : nullptr;
        };
        auto give_back = [&](int n) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.piece_free[n % kPieces]);
        };
        // rows at positions lo..hi see all of tile t
        auto inner = [&](int t, int lo, int hi) {
            const int c = t * kTok;
            return c + kTok - 1 <= lo && (a.window == 0 || c > hi - a.window);
        };

        if (warp < kSoftWarps) {
            more_registers<kSoftRegs>();
            const int x = warp >> 2;
            const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 lanes of tensor memory, << 16
            const uint32_t ts = tmem + lanes + S::kS + 128 * x, to = tmem + lanes + S::kO + D * x;
            const float inf = __int_as_float(0x7F800000);
            const int rt = x * kRowsPerTile + (tid & 127);   // this thread's row of an item
            uint8_t* const mine_s = out_s + warp * kOutBytes;
            int n = 0;   // pieces so far
            // The next piece with rows in this tile of rows, as the warp's own copy (it is still at the last one's result
            // when it looks for it, and there may be any number to pass by).
            auto next_piece = [&](int i) -> const Held* {
                const Piece* p;
                while ((p = piece(n))) {
                    const bool has = x * kRowsPerTile < p->rows;
                    Held& h = held[warp][i & 1];
                    if (has) {
                        if (lane < kPieceWords) reinterpret_cast<int*>(static_cast<Piece*>(&h))[lane] = reinterpret_cast<const int*>(p)[lane];
                        const int lo = p->pos0 + (p->block + x * kRowsPerTile) / group;
                        const int hi = p->pos0 + (p->block + min(p->rows, (x + 1) * kRowsPerTile) - 1) / group;
                        if (lane == 0) h.all0 = a.window > 0 && hi >= a.window ? (hi - a.window) / kTok + 1 - p->tile0 : 0;
                        if (lane == 0) h.all1 = (max(0, lo + 1)) / kTok - p->tile0;
                    }
                    give_back(n++);
                    if (has) return &h;
                }
                return nullptr;
            };
            // Q: one row to a thread, taken to fp16 with a power of two, in its place; the factor back to log2 scores
            auto take_q = [&](bool live, int items, float& mult) {
                if (!wait_for(&bar.q_raw[x], items & 1)) return false;
                const int r = tid & 127;
                uint8_t* dst = q_s + x * S::kQTile + r * 128;
                auto at = [&](int c) { return reinterpret_cast<uint4*>(dst + (c >> 3) * (kRowsPerTile * 128) + (((c & 7) ^ (r & 7)) << 4)); };
                __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = *at(c);
                    const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = p[e] & 0x7FFF7FFFu;
                        top2 = __hmax2(top2, *reinterpret_cast<const __nv_bfloat162*>(&u));
                    }
                }
                // (a row past the last holds what was there: its factor is 0, so that its scores are finite or NaN, and its own)
                const float top = live ? fmaxf(__low2float(top2), __high2float(top2)) : 0.f;
                const int fe = min(261 - static_cast<int>(__float_as_uint(top) >> 23), 253);
                float up = top > 0.f ? __uint_as_float(static_cast<uint32_t>(fe) << 23) : live ? 1.f : 0.f;
                const float down = top > 0.f ? __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) : 1.f;
                // scores in log2, never a negative factor; nor 0, which would make a masked score's -inf a NaN (1e-30 of
                // the largest product is below 2^-50)
                mult = fmaxf(fabsf(a.scale) * 1.4426950408889634f * down, 1e-30f);
                if (a.scale < 0.f) up = -up;
#pragma unroll 2
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = *at(c);
                    const float f[8] = {bf16_lo(v.x) * up, bf16_hi(v.x) * up, bf16_lo(v.y) * up, bf16_hi(v.y) * up,
                                        bf16_lo(v.z) * up, bf16_hi(v.z) * up, bf16_lo(v.w) * up, bf16_hi(v.w) * up};
                    *at(c) = make_uint4(pack_f16x2(f[0], f[4]), pack_f16x2(f[1], f[5]), pack_f16x2(f[2], f[6]), pack_f16x2(f[3], f[7]));
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.q_full[x]);
                return true;
            };
            int mine = 0, items = 0;   // tiles and items of this tile of rows so far
            float mult = 0.f;
            const Held* pc = next_piece(0);
            if (pc) ok = take_q(rt < pc->rows, 0, mult);
            while (pc && ok) {
                float top = -inf, sum = 0.f;
                uint32_t sick = 0;   // groups of dims in which this row sees a value that is not finite
                // Moves the running maximum where a score passes it by 2^8; `first`: there are no sums yet.  (The last
                // product with V is done: the scores at hand were issued after it.)
                auto raise = [&](float high, bool first) {
                    if (__builtin_expect(!__any_sync(0xFFFFFFFFu, high > top + kSlack), 1)) return false;
                    const float next = fmaxf(high, top);
                    const float keep = next == -inf ? 1.f : ex2(top - next);
                    top = next;
                    sum *= keep;
                    if (!first) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t w[16];
                            tmem_ld16_start(to + c, w);
                            tmem_ld16_wait(w);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * keep);
                            tmem_st16(to + c, w);
                        }
                    }
                    return true;
                };
                const int n_tiles = pc->tiles, ja = pc->all0, jb = pc->all1;
                for (int j = 0; j < n_tiles; ++j) {
                    const int note = (pc->base + j) & (kNotes - 1);
                    const bool in = j >= ja && j < jb;
                    if (!wait_for(&bar.s_full[x], (mine + j) & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                    uint32_t v[2][32];   // scores: one load ahead of the arithmetic
                    tmem_ld32_start(ts, v[0]);
                    const uint4 hid4 = notes.hidden[note];
                    const bool all = in && (hid4.x | hid4.y | hid4.z | hid4.w) == 0;
                    auto sees = [&](int c) {   // a bit for each of 32 columns that this row sees
                        const int c_hi = pc->pos0 + (pc->block + rt) / group + 1 - (pc->tile0 + j) * kTok - 32 * c;
                        return bits_in(a.window > 0 && c_hi > a.window ? c_hi - a.window : 0, c_hi) & ~reinterpret_cast<const uint32_t*>(&notes.hidden[note])[c];
                    };
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    if (__builtin_expect(all, 1)) {
                        // Weights against the running maximum as it stands, taken again where it has to move; in an
                        // item's first tile it begins as that of the first columns (and what O holds then does not matter).
                        if (__builtin_expect(j == 0, 0)) {
                            tmem_wait_ld();
                            after_wait(v[0]);
                            float m[2] = {-inf, -inf};
#pragma unroll
                            for (int e = 0; e < 32; ++e) m[e & 1] = fmaxf(m[e & 1], __uint_as_float(v[0][e]));
                            top = fmaxf(m[0], m[1]) * mult;
                        }
                        uint32_t p[kTok / 2];
                        for (;;) {
                            const float off = top == -inf ? 0.f : kLift - top;
                            const float2 mult2 = make_float2(mult, mult), off2 = make_float2(off, off);
                            float m[2] = {-inf, -inf};
                            part[0] = part[1] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int c = 0; c < kTok / 32; ++c) {
                                uint32_t(&w)[32] = v[c & 1];
                                tmem_wait_ld();
                                after_wait(w);
                                if (c + 1 < kTok / 32) tmem_ld32_start(ts + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 x2 = make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
                                    m[(e >> 1) & 1] = fmaxf(m[(e >> 1) & 1], fmaxf(x2.x, x2.y));
                                    float2 y = fma2(x2, mult2, off2);
                                    y.x = ex2(y.x);
                                    y.y = ex2(y.y);
                                    part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], y);
                                    p[16 * c + (e >> 1)] = pack_f16x2(y.x, y.y);
                                }
                            }
                            if (!raise(fmaxf(m[0], m[1]) * mult, false)) break;
                            tmem_ld32_start(ts, v[0]);
                        }
#pragma unroll
                        for (int c = 0; c < kTok / 2; c += 16) tmem_st16(ts + c, p + c);
                    } else {
                        // A tile that not every row sees all of: the maximum first, then the weights, 32 columns at a
                        // time (few instructions for what is seldom run: they are read from memory when it is).
                        float m[2] = {-inf, -inf};
                        tmem_wait_ld();
                        after_wait(v[0]);
#pragma unroll 1
                        for (int c = 0; c < kTok / 32; ++c) {
                            const uint32_t see = sees(c);
                            if (!__any_sync(0xFFFFFFFFu, see)) continue;
                            uint32_t w[32];
                            tmem_ld32_start(ts + 32 * c, w);
                            tmem_wait_ld();
                            after_wait(w);
#pragma unroll
                            for (int e = 0; e < 32; ++e) m[e & 1] = fmaxf(m[e & 1], (see >> e) & 1u ? __uint_as_float(w[e]) : -inf);
                        }
                        raise(fmaxf(m[0], m[1]) * mult, j == 0);
                        const float off = top == -inf ? 0.f : kLift - top;
                        const float2 mult2 = make_float2(mult, mult), off2 = make_float2(off, off);
#pragma unroll 1
                        for (int c = 0; c < kTok / 32; ++c) {
                            const uint32_t see = sees(c);
                            uint32_t p[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) p[e] = 0;
                            if (__any_sync(0xFFFFFFFFu, see)) {
                                uint32_t w[32];
                                tmem_ld32_start(ts + 32 * c, w);
                                tmem_wait_ld();
                                after_wait(w);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 x2 = make_float2((see >> e) & 1u ? __uint_as_float(w[e]) : -inf, (see >> e) & 2u ? __uint_as_float(w[e + 1]) : -inf);
                                    float2 y = fma2(x2, mult2, off2);
                                    y.x = ex2(y.x);
                                    y.y = ex2(y.y);
                                    part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], y);
                                    p[e >> 1] = pack_f16x2(y.x, y.y);
                                }
                            }
                            tmem_st16(ts + 16 * c, p);   // over scores that have been read
                        }
                    }
                    sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    if (__builtin_expect(notes.any_sick[note] && !inner(pc->tile0 + j, pc->p0, pc->p1), 0)) {
#pragma unroll 1
                        for (int c = 0; c < kTok / 32; ++c) {
                            const uint32_t see = all ? 0xFFFFFFFFu : sees(c);
                            for (int g = 0; g < kGroups; ++g)
                                if (notes.sick[note][g][c] & see) sick |= 1u << g;
                        }
                    }
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.p_full[x]);
                }
                // ---- the next item's Q, whose copy began when this one's last scores were there: its first scores are
                // computed while this result is written
                if (!ok) break;
                const Held* const old = pc;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                pc = next_piece(items + 1);
                if (pc) ok = take_q(rt < pc->rows, items + 1, mult);
                // ---- the result, or a partial one, 32 dims at a time
                if (ok) ok = wait_for(&bar.o_full[x], items & 1);
                if (!ok) break;
                tc::tc_fence_after();
                if (old->starts && old->ends) {   // through shared memory, 64 bytes of a row to four lanes
                    const int r0 = old->block + x * kRowsPerTile + (warp & 3) * 32 + (lane >> 2), r_end = old->block + old->rows;
                    bf16_t* o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = (r0 + 8 * i) / group;
                        o[i] = a.out + static_cast<long long>(old->row0 + t) * a.ld_out + (old->h * group + r0 + 8 * i - t * group) * D + 8 * (lane & 3);
                    }
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t w[32];
                        tmem_ld32_start(to + c, w);
                        tmem_wait_ld();
                        after_wait(w);
                        const float k = (sick >> (c / kGroup)) & 1u ? __int_as_float(0x7FC00000) : inv;
                        auto pair = [&](int e) { return pack_bf16x2(__uint_as_float(w[e]) * k, __uint_as_float(w[e + 1]) * k); };
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(mine_s + lane * 64 + (((e >> 3) ^ ((lane >> 1) & 3)) << 4)) = make_uint4(pair(e), pair(e + 2), pair(e + 4), pair(e + 6));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = (lane >> 2) + 8 * i;
                            const uint4 q = *reinterpret_cast<const uint4*>(mine_s + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                            if (r0 + 8 * i < r_end) *reinterpret_cast<uint4*>(o[i] + c) = q;
                        }
                        __syncwarp();
                    }
                } else {
                    float* part_o = left.slot(blockIdx.x, old->starts, D);
                    part_o[kRowsPerItem * D + rt] = top;
                    part_o[kRowsPerItem * (D + 1) + rt] = sum;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t w[32];
                        tmem_ld32_start(to + c, w);
                        tmem_wait_ld();
                        after_wait(w);
                        const float k = (sick >> (c / kGroup)) & 1u ? __int_as_float(0x7FC00000) : 1.f;
                        auto f = [&](int e) { return __uint_as_float(w[e]) * k; };
                        if (rt < old->rows) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(part_o + rt * D + c + e) = make_float4(f(e), f(e + 1), f(e + 2), f(e + 3));
                        }
                    }
                }
                // the loads above are done before the next item's first product with V: its weights come after
                tc::tc_fence_before();
                if (tid == 0 && old->starts && !old->ends) left.records[blockIdx.x] = Record{old->rows, old->block, old->row0, old->h, old->last};
                mine += old->tiles;
                ++items;
            }
            if (!ok) failed = 1;
        } else if (warp < kMmaWarp) {
            // ---- unpacking: four warps K, a position to a thread, four warps V, eight positions x 16 dims
            fewer_registers<kUnpackRegs>();
            const bool is_k = warp < kVWarp;
            const int u = tid & 127;                            // K: position in the tile
            const int half = (u >> 5) & 1, t8 = u & 7;          // V: eight positions of a half of 64,
            const int quad = ((u >> 6) << 2) | ((u >> 3) & 3);  // 16 dims; eight lanes of a dim write its 128 bytes
            const bool idle = !is_k && quad >= D / 16;
            const int my_tok = is_k ? u : 64 * half + 8 * t8;
            struct Raw {
                uint4 w[4];        // K: the row's words; V: four pairs' words
                uint32_t par[8];   // K: the groups' (step, low); V: four pairs' (steps, lows)
                uint32_t sick;     // K: groups in which the position's V is not finite
                bool hidden;       // K: the position's page is bad
                int page;          // of the tile to be loaded next
            };
            int p0 = 0, p1 = 0, j_begin = 0, j_end = 0, tile0 = 0, n_tiles = 0, head = 0;   // rows see [j_begin, j_end)
            const int reach = is_k ? 1 : 8;                     // positions of this thread
            const int32_t* table = nullptr;
            auto page_at = [&](int j) -> int {   // -1: no row sees the place; -2: its page is bad
                const int p = (tile0 + j) * kTok + my_tok;
                if (j >= n_tiles || p >= j_end || p + reach <= j_begin || idle) return -1;
                const int page = __ldg(table + (p >> a.cache.page_shift));
                return static_cast<unsigned>(page) < static_cast<unsigned>(a.cache.n_pages) ? page : -2;
            };
            // A tile begins where a page does, or in the middle of one of 256: where this thread's bytes lie in its block
            // is the same for every tile but for that half.
            const int off = my_tok & (ps - 1);
            const int codes_at = is_k ? off * (D / 2) : v_codes_off(ps, D) + (off >> 1) * D + 16 * quad;
            const int params_at = is_k ? k_params_off(ps, D) + off * kGroups * 4 : v_params_off(ps, D) + ((off >> 1) * kGroups + quad * 16 / kGroup) * 8;
            const long long head_bytes = block_bytes(ps, D);
            auto load = [&](Raw& r, int j) {
                const int page = r.page;
                r.page = page_at(j + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) r.w[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 8; ++i) r.par[i] = 0;
                r.sick = 0;
                r.hidden = page == -2;
                if (page == -2) flag(a.status, LORA_DEV_BAD_PAGE);
                if (page < 0) return;
                const int second = ps > kTok && (tile0 + j) & 1 ? kTok : 0;
                const uint8_t* b = a.cache.pages + page * a.cache.page_stride + head * head_bytes;
                const uint8_t* c = b + codes_at + second * (D / 2);
                const uint8_t* w = b + params_at + second * kGroups * 4;
                if (is_k) {
#pragma unroll
                    for (int t = 0; t < D / 32; ++t) r.w[t] = __ldg(reinterpret_cast<const uint4*>(c) + t);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) r.par[g] = __ldg(reinterpret_cast<const uint32_t*>(w) + g);
                    if (__builtin_expect(!inner(tile0 + j, p0, p1), 0)) {
                        const int at = off + second;
#pragma unroll 1
                        for (int g = 0; g < kGroups; ++g) {
                            const uint16_t* v = reinterpret_cast<const uint16_t*>(b + v_params_off(ps, D)) + ((at >> 1) * kGroups + g) * 4 + (at & 1);
                            r.sick |= (not_finite(v[0], v[2]) ? 1u : 0u) << g;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        r.w[i] = __ldg(reinterpret_cast<const uint4*>(c + i * D));
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(w + i * 8 * kGroups));
                        r.par[2 * i] = v.x;
                        r.par[2 * i + 1] = v.y;
                    }
                }
            };
            auto store_k = [&](const Raw& r, int j, int n) {   // n: the tile's place among all of the range
                uint8_t* kd = k_s + (n & (kStages - 1)) * S::kKTile + u * 128;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    // 16 bytes of the row hold words (t, 0..kWords-1)
                    uint32_t w[4];
                    if (kWords == 4) {
                        w[0] = r.w[t].x; w[1] = r.w[t].y; w[2] = r.w[t].z; w[3] = r.w[t].w;
                    } else {
                        w[0] = t & 1 ? r.w[t >> 1].z : r.w[t >> 1].x;
                        w[1] = t & 1 ? r.w[t >> 1].w : r.w[t >> 1].y;
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i) {
                        const __half2 pr = as_h2(r.par[i / 2]);
                        uint32_t v[4];
                        values(w[i], __low2half2(pr), __high2half2(pr), v);
                        const int c = 4 * (i & 1) + t;
                        *reinterpret_cast<uint4*>(kd + (i >> 1) * (kTok * 128) + ((c ^ (u & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
                n &= kNotes - 1;
                const uint32_t gone = __ballot_sync(0xFFFFFFFFu, r.hidden);
                if (lane == 0) reinterpret_cast<uint32_t*>(&notes.hidden[n])[u >> 5] = gone;
                if (!inner(tile0 + j, p0, p1)) {
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, (r.sick >> g) & 1u);
                        if (lane == 0) {
                            notes.sick[n][g][u >> 5] = bits;
                            if (bits) notes.any_sick[n] = 1;   // stays set: the bits say what is there
                        }
                    }
                }
            };
            auto store_v = [&](Raw& r, int j, int n) {
                if (idle) return;
                if (__builtin_expect(!inner(tile0 + j, p0, p1), 0)) {
                    // positions that no row sees, and values that are not finite, count as zeros
                    const int p = (tile0 + j) * kTok + my_tok;
                    auto seen = [&](int at) { return at >= j_begin && at < j_end; };
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = p + 2 * i;
                        uint32_t& step = r.par[2 * i];
                        uint32_t& low = r.par[2 * i + 1];
                        const uint32_t keep = ((seen(at) ? 0xFFFFu : 0u) | (seen(at + 1) ? 0xFFFF0000u : 0u)) & ~not_finite(step, low);
                        step &= keep;
                        low &= keep;
                    }
                }
                uint8_t* vd = v_s + (n & (kStages - 1)) * S::kVTile + half * S::kVHalf;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t v[4][4];   // [pair of positions][dim]
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t raw = w == 0 ? r.w[i].x : w == 1 ? r.w[i].y : w == 2 ? r.w[i].z : r.w[i].w;
                        values(raw, as_h2(r.par[2 * i]), as_h2(r.par[2 * i + 1]), v[i]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = 16 * quad + 4 * w + e;
                        *reinterpret_cast<uint4*>(vd + d * 128 + ((t8 ^ (d & 7)) << 4)) = make_uint4(v[0][e], v[1][e], v[2][e], v[3][e]);
                    }
                }
            };
            uint64_t* full = is_k ? bar.k_full : bar.v_full;
            uint64_t* free = is_k ? bar.k_free : bar.v_free;
            // Q's rows as they are into the swizzled tile, a row to D / 8 neighbouring lanes (16 bytes of 32 rows to an
            // instruction would cost as many lines as rows)
            uint32_t q_odd = 0, q_any = 0;   // a bit for each tile of rows: whether its items so far are odd, and any
            auto copy_q = [&](const Piece* pc, int x) {
                const int rows = min(kRowsPerTile, pc->rows - x * kRowsPerTile);
                if (rows <= 0) return true;
                if ((q_any >> x) & 1u && !wait_for(&bar.q_free[x], ((q_odd >> x) & 1u) ^ 1u)) return false;
                q_any |= 1u << x;
                q_odd ^= 1u << x;
                constexpr int kLanes = D / 8, kStep = 128 / kLanes;
                const int c = u % kLanes;
                int r = u / kLanes, hh = pc->block + x * kRowsPerTile + r, t = hh / group;
                hh -= t * group;
                const bf16_t* src = a.q + static_cast<long long>(pc->row0 + t) * a.ld_q + (head * group + hh) * D + 8 * c;
                const int dt = kStep / group, dh = kStep - dt * group;
                const uint32_t dst = tc::smem_u32(q_s) + x * S::kQTile + (c >> 3) * (kRowsPerTile * 128);
#pragma unroll 2
                for (; r < rows; r += kStep) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)), "l"(src) : "memory");
                    src += static_cast<long long>(dt) * a.ld_q + dh * D;
                    hh += dh;
                    if (hh >= group) {   // the next token's
                        hh -= group;
                        src += a.ld_q - group * D;
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];\n" ::"r"(tc::smem_u32(&bar.q_raw[x])) : "memory");
                return true;
            };
            // a tile on its way, and the page of the one after it
            int n = 0;   // tiles so far
            const Piece* pc;
            for (int i = 0; (pc = piece(i)) && ok; ++i) {
                p0 = pc->p0;
                p1 = pc->p1;
                tile0 = pc->tile0;
                n_tiles = pc->tiles;
                head = pc->h;
                j_begin = seen_from(p0, a.window);
                j_end = max(0, p1 + 1);
                table = a.batch.block_table + static_cast<long long>(pc->s) * a.batch.ld_table;
                if (is_k && i > 0) {   // these warps are ahead: Q's lines are on their way when its place is free
#pragma unroll 1
                    for (int i = u; i < pc->rows * (D / 64); i += 128) {
                        const int row = pc->block + i / (D / 64), t = row / group;
                        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(a.q + static_cast<long long>(pc->row0 + t) * a.ld_q +
                                                                       (head * group + row - t * group) * D + 64 * (i % (D / 64))));
                    }
                }
                Raw r;
                r.page = page_at(0);
                for (int j = -1; j < n_tiles; ++j) {
                    if (j >= 0) {
                        const int st = n & (kStages - 1);
                        if (n >= kStages && !wait_for(&free[st], ((n / kStages) & 1) ^ 1)) { ok = false; break; }
                        if (is_k) store_k(r, j, n); else store_v(r, j, n);
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&full[st]);
                        ++n;
                    }
                    if (j + 1 < n_tiles) load(r, j + 1);
                    // Q after the first tile: its place, and the next stage, are free when the last item's scores are done
                    if (is_k && j == (i > 0 ? 0 : -1)) {
#pragma unroll 1
                        for (int x = 0; x < 2; ++x) ok = ok && copy_q(pc, x);
                        if (!ok) break;
                    }
                }
                give_back(i);
            }
            if (!ok) failed = 1;
        } else {
            // ---- the products
            // The whole warp runs the loop and one elected lane issues: values that the compiler knows to be
            // the warp's own stay in uniform registers, where the instruction wants its operands.
            fewer_registers<kMmaRegs>();
            const int x = warp - kMmaWarp;   // the tile of rows whose products this warp issues
            if (x < 2) {
                constexpr uint32_t id_s = idesc_f16(kRowsPerTile, kTok), id_o = idesc_f16(kRowsPerTile, D);
                const uint32_t t0 = __shfl_sync(0xFFFFFFFFu, tmem, 0);
                const uint32_t s_t = t0 + S::kS + 128 * x, o_t = t0 + S::kO + D * x;
                const uint64_t q_d = tc::sdesc_sw128(tc::smem_u32(q_s) + x * S::kQTile);
                const uint64_t k_d = tc::sdesc_sw128(tc::smem_u32(k_s)), v_d = tc::sdesc_sw128(tc::smem_u32(v_s));
                const bool lead = elect_one();
                int n = 0, mine = 0, items = 0, turns = 0;   // tiles so far; of this tile of rows; its items and turns
                bool both = false;
                auto my_turn = [&]() { return !both || wait_polling(&bar.turn[x], turns++ & 1); };
                auto your_turn = [&]() { if (both) tc::mbar_arrive(&bar.turn[x ^ 1]); };
                auto scores = [&](int t, bool last) -> bool {   // t: the tile's place among all of the range; the item's last
                    const int st = t & (kStages - 1);
                    if (!wait_polling(&bar.k_full[st], (t / kStages) & 1)) return false;
                    tc::tc_fence_after();
                    if (lead) {
                        const uint64_t k_j = k_d + static_cast<uint64_t>(st * (S::kKTile >> 4));   // descriptors count 16 bytes
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const int at = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
                            tc::mma_bf16(s_t, q_d + at, k_j + at, id_s, k > 0);
                        }
                        tc::mma_commit(&bar.s_full[x]);
                        tc::mma_commit(&bar.k_free[st]);
                        if (last) tc::mma_commit(&bar.q_free[x]);
                        your_turn();
                    }
                    __syncwarp();
                    return true;
                };
                bool first = true;   // no turn has been taken
                const Piece* pc;
                for (int i = 0; (pc = piece(i)) && ok; give_back(i), ++i) {
                    const int n_tiles = pc->tiles;
                    both = pc->rows > kRowsPerTile;
                    if (x == 1 && !both) {
                        // the stages pass this tile of rows by, in step (a parity tells a phase only from its neighbours)
                        for (int j = 0; ok && j < n_tiles; ++j, ++n) {
                            const int st = n & (kStages - 1);
                            ok = wait_polling(&bar.k_full[st], (n / kStages) & 1);
                            if (lead) tc::mbar_arrive(&bar.k_free[st]);
                            ok = ok && wait_polling(&bar.v_full[st], (n / kStages) & 1);
                            if (lead) tc::mbar_arrive(&bar.v_free[st]);
                        }
                        continue;
                    }
                    ok = wait_polling(&bar.q_full[x], items++ & 1);
                    for (int j = 0; ok && j <= n_tiles; ++j) {
                        if (j == 0) {
                            // the first tile of rows goes first; later items wait for the turn that the last one left over
                            ok = (x == 0 && first) || my_turn();
                            if (both) first = false;
                        } else {
                            const int st = n & (kStages - 1);
                            ok = wait_polling(&bar.v_full[st], (n / kStages) & 1) && my_turn() && wait_polling(&bar.p_full[x], mine & 1);
                            if (!ok) break;
                            tc::tc_fence_after();
                            if (lead) {
                                const uint64_t v_j = v_d + static_cast<uint64_t>(st * (S::kVTile >> 4));
#pragma unroll
                                for (int k = 0; k < kTok / 16; ++k)
                                    mma_ts(o_t, s_t + 8 * k, v_j + (((k >> 2) * S::kVHalf + (k & 3) * 32) >> 4), id_o, j > 1 || k > 0);
                                tc::mma_commit(&bar.v_free[st]);
                                if (j == n_tiles) {
                                    tc::mma_commit(&bar.o_full[x]);
                                    your_turn();
                                }
                            }
                            __syncwarp();
                            ++n;
                            ++mine;
                        }
                        if (ok && j < n_tiles) ok = scores(n, j + 1 == n_tiles);
                    }
                }
                if (!ok) failed = 1;
            } else if (warp == kWalkWarp) {
                Walk walk(a, prefix, first, total / n_ranges, begin, end);
                int tiles[kPieces] = {};   // of the pieces not yet given back
                for (int i = 0;; ++i) {
                    Piece p;
                    const int u1 = walk.next(p);
                    p.last = blockIdx.x;
                    if (p.tiles && p.starts && !p.ends)
                        while (p.last + 1 < static_cast<int>(gridDim.x) && range_at(total, n_ranges, p.last + 1) < u1) ++p.last;
                    // a piece may take as long as it has tiles
                    long long limit = kTimeoutClocks;
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) limit += 20000ll * tiles[k];
                    if (i >= kPieces && !wait_for(&bar.piece_free[i % kPieces], (i / kPieces & 1) ^ 1, limit)) { ok = false; break; }
                    if (lane == 0) pieces[i % kPieces] = p;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.piece_full[i % kPieces]);
                    if (!p.tiles) break;
#pragma unroll
                    for (int k = kPieces - 1; k > 0; --k) tiles[k] = tiles[k - 1];
                    tiles[0] = p.tiles;
                }
                if (!ok) failed = 1;
            }
            __syncwarp();
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && failed) flag(a.status, LORA_DEV_TIMEOUT);
}

template <int D>
cudaError_t run(const AttendArgs& a, int few_rows, void* ws, Partials* left, cudaStream_t stream)
{
    using S = Shape<D>;
    constexpr int kMaxSmem = S::kSmem + 4 * (kMaxSeqs + 1);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_on_device(done, [&] { return cudaFuncSetAttribute(kv4_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem); });
    if (e != cudaSuccess) return e;
    const int ctas = std::min(kMaxCtas, device_sms());
    PdlLaunch l(dim3(ctas), kThreads, S::kSmem + 4 * (a.batch.n_seqs + 1), stream);
    *left = partials_at(ws, ctas, kRowsPerItem);
    e = cudaLaunchKernelEx(&l.cfg, kv4_many_kernel<D>, a, few_rows, *left);
    note_launch();
    return e;
}

}  // namespace

size_t kv4_many_workspace(int head_dim) { return partials_bytes(kMaxCtas, kRowsPerItem, head_dim); }

cudaError_t launch_kv4_many(const AttendArgs& a, int few_rows, void* ws, Partials* left, cudaStream_t stream)
{
    return a.cache.head_dim == 64 ? run<64>(a, few_rows, ws, left, stream) : run<128>(a, few_rows, ws, left, stream);
}

}  // namespace lora
