// kv4_few.cu -- attention of few query rows (single tokens, drafts) over the
// paged 4-bit cache: the cache's bytes are the cost, so every byte is read
// once and the codes are unpacked in registers.
//
// Work.  A unit is (sequence, kv head, slice of up to 8 query rows, rows
// being a sequence's rows x the heads of the group) over the sequence's tiles
// of 32 positions; the slices of a kv head lie next to each other, so that
// the second one's bytes come from L2.  All units laid end to end are cut
// into equal ranges, one per warp, whatever the lengths; a unit counts
// kUnitCost tiles more than it has, for its start.  A warp that has a whole
// unit writes its result; a unit cut by a range's end leaves partial results,
// which the CTA joins over shared memory where its warps have the whole unit,
// and a second kernel, in a fixed order, where other CTAs have a part.
//
// Tile.  A warp multiplies on mma.sync m16n8k16 with positions as M and query
// rows as N, so that groups of up to 8 heads waste nothing:
//   S[16 positions][8 rows] = codes(K) q^T, per group of 64 dims, then
//   score = sum_g step_g S_g + low_g sum(q_g)         (K is never rounded)
//   O[dims][8 rows] += V^T P, V = code * step + low in fp16, P in fp16.
// K's codes go in as 1024 + code, one instruction from the nibbles; the
// product's accumulator starts at -1024 sum(q), which takes the 1024 out.
// The K layout puts the 16 bytes that a lane feeds to its fragments side by
// side, the V layout pairs two positions in one 32-bit operand, and P goes
// from the first product's layout to the second's by a register transpose.
// The running maximum moves only when a score passes it by 2^8 (a vote per
// tile), so most tiles rescale nothing.
// A warp copies its own tiles ahead with cp.async into a ring of its own and
// meets no other warp until its range ends.
//
// Drafted trees (kTree) differ in tiles that reach past the sequence's first
// row: a row's 32 bits of such a tile come from its words at once.
//
// What bounds it.  HBM by its bytes, but the unpacking takes longer: 8 requests of
// 131072 positions, 64 heads in groups of 8, 231 us, 5.2 TB/s, 0.78 of a copy's
// rate, an issue slot in 0.63; without V's unpacking 197 us, without K's 220.
// Small batches are starts and ends: 64 requests of up to 8192 positions 25 us
// for 61 MB (start 4, about five tiles a warp 12, the second kernel 4), one of
// 1003 positions 6.2 in the form by clusters.
#include <algorithm>

#include "kv4_attend.cuh"
#include "tc_common.cuh"

namespace lora {

namespace {

using namespace kv4;

// Rows of a unit: one column block of the product.  Slices of 16 or 32 rows,
// which unpack once for more rows, were slower for their registers: one CTA on
// an SM (us, 32 requests of up to 1000 positions, rows of a kv head 16 / 32, by
// slices of 8, 16, 32: heads of 128 16 / 21, 16 / 22, 29 / 33; of 64 13 / 17, 12 / 15, 15 / 17).
// Those are starts and ends; wider slices were not timed on long contexts,
// where each slice unpacks its kv head's bytes again: 8 requests, 4 kv heads,
// 8 / 16 / 24 rows of each, 32000 positions 40 / 68 / 94 us, 131072 126 / 234 / 344.
constexpr int kRows = 8;
// Two CTAs of eight warps on an SM: 128 registers a thread.
constexpr int kCtas = 2, kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTile = 32;          // positions per tile: two halves of 16, the products' M
constexpr int kHalf = 16;
// A unit's start (tables, q, the first copies), in tiles: drafts 20.4 us, with 2
// 21.5; 64 requests 25.3 with 2 and with 3, 28.7 with 1, 25.9 with 4.
constexpr int kUnitCost = 3;
constexpr float kNone = -3e38f;    // the running maximum before any score (finite, so that no difference is NaN)
constexpr float kSlack = 8.f;      // log2 by which a score may pass the running maximum
constexpr float kLift = 7.f;       // weights carry 2^7: at most 2^15, and fp16 holds them down to 2^-31 of the largest

// Sizes for head dimension D.
template <int D>
struct Shape {
    static constexpr int kGroups = D / kGroup;
    static constexpr int kWords = D / 32;                 // words of a lane per position (K) and per pair (V)
    static constexpr int kCodeBytes = kHalf * D / 2;      // of K or V, of half a tile
    static constexpr int kParamBytes = kHalf * 4 * kGroups;
    // a stage: K codes, V codes, K params, V params, each of both halves
    static constexpr int kVAt = 2 * kCodeBytes, kKpAt = 4 * kCodeBytes, kVpAt = kKpAt + 2 * kParamBytes;
    static constexpr int kStage = kVpAt + 2 * kParamBytes;
    static constexpr int kPartial = kRows * (D + 2);      // floats of a partial result: sums, maxima, sums of weights
    // The ring is at least a partial result long: a warp's last one takes
    // the ring's place.
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kWarps * (kRing + 4 * kPartial) + 256;   // and the running sum of the sequences
    static_assert(kRing >= 4 * kPartial, "ring");
};

// Ranges are one per warp; range w of n begins here.
__device__ __forceinline__ int range_count(int total, int warps) { return min(warps, max(1, total)); }
__device__ __forceinline__ int range_at(int total, int n, int w)
{
    w = min(w, n);   // without leaving 32 bits: n is a number of warps
    return total / n * w + total % n * w / n;
}

// First tile, and tiles, that a sequence's rows see.
__device__ __forceinline__ int first_tile(const Seq& q, int window)
{
    return seen_from(q.ctx - q.n, window) / kTile;
}
__device__ __forceinline__ int tiles_of(const Seq& q, int window)
{
    return max(1, (q.ctx + kTile - 1) / kTile - first_tile(q, window));   // at least one: its rows get their zeros
}

// Slices of a sequence's rows, of kRows each.
__device__ __forceinline__ int slices_of(const Seq& q, int group) { return (q.n * group + kRows - 1) / kRows; }

// The unit that holds place x (< total) of the line: rows [row0, row0 + rows)
// of positions x heads.
struct Unit {
    int s, h, row0, rows, u0, len;   // u0: its first place; len: its places (kUnitCost, then its tiles)
    Seq q;
};
__device__ __forceinline__ Unit unit_at(const AttendArgs& a, const int* prefix, int x)
{
    const int lo = seq_at(prefix, a.batch.n_seqs, x);
    Unit u;
    u.s = lo;
    load_seq(a.batch, lo, u.q, nullptr);
    const int slices = slices_of(u.q, a.group);
    u.len = tiles_of(u.q, a.window) + kUnitCost;
    const int v = (x - prefix[lo]) / u.len;
    u.u0 = prefix[lo] + v * u.len;
    u.h = slices == 1 ? v : v / slices;
    u.row0 = (v - u.h * slices) * kRows;
    u.rows = min(kRows, u.q.n * a.group - u.row0);
    return u;
}

// A warp's partial result in shared memory.  Slot 0: of the unit that began
// before the warp's range; slot 1: of the last one, which goes on after it.
struct Piece {
    int u0;               // the unit's first place; -1: none
    int ends;             // whether the unit ends with this piece
    int h, seq_row0, row0, rows, u1;
};

constexpr int kMaxCtas = 2 * 160;   // CTAs that the workspace has room for

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// A warp's running result of a unit: fragments of the sums, and the maximum
// and the lane's part of the sum of weights of rows 2t, 2t + 1.
template <int D>
struct Sums {
    float acc[D / 16][4], top[2], sum[2];
};

// One warp: `n_mine` tiles from tile `tile` of sequence s, kv head h, for the
// rows [row0, row0 + rows).
template <int D, bool kTree>
__device__ __forceinline__ void attend_tiles(const AttendArgs& a, uint8_t* ring, int s, int h, const Seq& q, int row0, int rows, int tile, int n_mine,
                                             Sums<D>& out)
{
    using S = Shape<D>;
    constexpr int kGroups = S::kGroups, kWords = S::kWords, kStages = S::kStages;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int group = a.group, ps = a.cache.page_size;
    const int p0 = q.ctx - q.n;   // position of the first row
    const int32_t* table = a.batch.block_table + static_cast<long long>(s) * a.batch.ld_table;
    const float inf = __int_as_float(0x7F800000);

    // q's way begins before the tables'
    uint4 raw[kWords];
    {
        const int tok = by_group(a, row0 + g);
        const bf16_t* qp = a.q + static_cast<long long>(q.row0 + tok) * a.ld_q + (h * group + row0 + g - tok * group) * D + 8 * t;
#pragma unroll
        for (int w = 0; w < kWords; ++w) raw[w] = g < rows ? *reinterpret_cast<const uint4*>(qp + 32 * w) : make_uint4(0, 0, 0, 0);
    }

    // ---- the ring
    const int pos0 = tile * kTile;
    const uint8_t* head_pages = a.cache.pages + static_cast<long long>(h) * block_bytes(ps, D);
    unsigned has = 0;   // stages' halves that hold positions
    auto page_at = [&](int pos) -> int { return pos < q.ctx ? max(-1, __ldg(table + (pos >> a.cache.page_shift))) : -1; };
    // Bytes of a tile (or of half of one) in a block: codes at 16 lane, params at param_at.
    const uint32_t ring_at = tc::smem_u32(ring) + 16 * lane;
    const int codes_v = v_codes_off(ps, D);
    // the next page to be read; a page of half a tile, the first, may lie behind the window of every row
    constexpr int kUnseen = -2;
    int next = n_mine <= 0 ? -1 : ps < kTile && pos0 + kHalf <= seen_from(p0, a.window) ? kUnseen : page_at(pos0);
    const uint8_t *codes = nullptr, *params = nullptr;
    int left = 0;                                 // tiles left in the page
    auto issue = [&](int i) {
        const int pos = pos0 + i * kTile, st = i % kStages;
        const uint32_t dst = ring_at + st * S::kStage;
        has &= ~(3u << (2 * st));
        if (i < n_mine && ps >= kTile) {
            if (left == 0) {
                const int off = pos & (ps - 1);
                const bool ok = static_cast<unsigned>(next) < static_cast<unsigned>(a.cache.n_pages);
                if (!ok && pos < q.ctx && lane == 0) flag(a.status, LORA_DEV_BAD_PAGE);
                const uint8_t* block = head_pages + static_cast<long long>(next) * a.cache.page_stride;
                codes = ok ? block + off * (D / 2) + 16 * lane : nullptr;
                params = block + (lane & 16 ? v_params_off(ps, D) : k_params_off(ps, D)) + off * 4 * kGroups + 16 * (lane & 15);
                left = (ps - off) / kTile;
                next = page_at(pos + left * kTile);
            }
            if (codes) {
                has |= (pos + kHalf < q.ctx ? 3u : 1u) << (2 * st);
#pragma unroll
                for (int c = 0; c < 2 * S::kCodeBytes; c += 512) {
                    copy16(dst + c, codes + c);
                    copy16(dst + S::kVAt + c, codes + codes_v + c);
                }
                // sixteen lanes K's params, sixteen V's
                if ((lane & 15) < 2 * S::kParamBytes / 16)
                    copy16(dst + S::kKpAt + (lane >> 4) * (2 * S::kParamBytes - 256), params);
                codes += kTile * D / 2;
                params += kTile * 4 * kGroups;
            }
            --left;
        } else if (i < n_mine) {   // pages of half a tile
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int at = pos + kHalf * hf, page = next;
                next = page_at(at + kHalf);
                if (at >= q.ctx || page == kUnseen) continue;
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.cache.n_pages)) {
                    if (lane == 0) flag(a.status, LORA_DEV_BAD_PAGE);
                    continue;
                }
                has |= 1u << (2 * st + hf);
                const uint8_t* block = head_pages + static_cast<long long>(page) * a.cache.page_stride;
#pragma unroll
                for (int c = 0; c < S::kCodeBytes; c += 512) {
                    copy16(dst + hf * S::kCodeBytes + c, block + 16 * lane + c);
                    copy16(dst + S::kVAt + hf * S::kCodeBytes + c, block + codes_v + 16 * lane + c);
                }
                const int pl = lane & 15;
                if (pl < S::kParamBytes / 16)
                    copy16(dst + S::kKpAt + hf * S::kParamBytes + (lane >> 4) * (2 * S::kParamBytes - 256),
                           block + (lane & 16 ? v_params_off(ps, D) : k_params_off(ps, D)) + 16 * pl);
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- q as fragments: row g, dims 32 w + 8 t + (0..7)
    uint32_t qf[kWords][4];     // pairs (dims e, e + 4); odd pairs carry 1/16
    float mult[2], qsum[kGroups][2], qoff[kGroups][2];   // of rows 2t, 2t + 1
    {
        float top = 0.f;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const uint32_t part[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(part[e])), fabsf(bf16_hi(part[e]))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // a power of two that takes the row's largest into [2^7, 2^8)
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int fe = min(261 - e, 253);
        const float up = top > 0.f ? __uint_as_float(static_cast<uint32_t>(fe) << 23) : 1.f;
        const float down = top > 0.f ? __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) : 1.f;
        // sums of the fp16 values as the product takes them: of q, and of 1024 times the operand
        float sum[kGroups], ofs[kGroups];
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) sum[gr] = ofs[gr] = 0.f;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const float f[8] = {bf16_lo(raw[w].x) * up, bf16_hi(raw[w].x) * up, bf16_lo(raw[w].y) * up, bf16_hi(raw[w].y) * up,
                                bf16_lo(raw[w].z) * up, bf16_hi(raw[w].z) * up, bf16_lo(raw[w].w) * up, bf16_hi(raw[w].w) * up};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = (i & 1) ? 1.f / 16 : 1.f;
                qf[w][i] = pack_f16x2(f[i] * k, f[i + 4] * k);
                const float2 h = __half22float2(as_h2(qf[w][i]));
                sum[w / 2] = fmaf(h.x + h.y, (i & 1) ? 16.f : 1.f, sum[w / 2]);
                ofs[w / 2] = fmaf(h.x + h.y, -1024.f, ofs[w / 2]);
            }
        }
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
            sum[gr] += __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 1);
            sum[gr] += __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 2);
            ofs[gr] += __shfl_xor_sync(0xFFFFFFFFu, ofs[gr], 1);
            ofs[gr] += __shfl_xor_sync(0xFFFFFFFFu, ofs[gr], 2);
        }
        const float m = a.scale * 1.4426950408889634f * down;   // scores in log2
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            mult[c] = __shfl_sync(0xFFFFFFFFu, m, 8 * t + 4 * c);
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                qsum[gr][c] = __shfl_sync(0xFFFFFFFFu, sum[gr], 8 * t + 4 * c);
                qoff[gr][c] = __shfl_sync(0xFFFFFFFFu, ofs[gr], 8 * t + 4 * c);
            }
        }
    }
    int last[2];   // position of rows 2t, 2t + 1: the last one they see
#pragma unroll
    for (int c = 0; c < 2; ++c) last[c] = p0 + by_group(a, row0 + 2 * t + c);

    float (&acc)[D / 16][4] = out.acc;
    float (&top)[2] = out.top, (&sum)[2] = out.sum;
#pragma unroll
    for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = 0.f;
    top[0] = top[1] = kNone;
    sum[0] = sum[1] = 0.f;

    for (int i = 0; i < n_mine; ++i) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
        __syncwarp();
        const int st = i % kStages;
        const uint8_t* src = ring + st * S::kStage;
        const unsigned live = (has >> (2 * st)) & 3u;   // its halves
        issue(i + kStages - 1);
        if (!live) continue;
        const int j0 = pos0 + i * kTile;   // the tile's first position
        // every row sees every position?
        const bool inner = live == 3u && j0 + kTile - 1 <= p0 - (kTree ? 1 : 0) && (a.window == 0 || j0 > p0 + q.n - 1 - a.window);

        const int vg = g * (D / 8) / kGroup;
        bool poison = false;
        uint32_t see[2];   // of a tree's rows 2t, 2t + 1: the tile's positions that they see
        if (kTree && !inner) {
#pragma unroll
            for (int c = 0; c < 2; ++c) see[c] = 2 * t + c < rows ? tree_sees32(a, q, last[c] - p0, j0) : 0u;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            // ---- scores
            const bool there = (live >> hf) & 1u;
            float sc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[c] = 0.f;
            uint32_t kw[2][kWords];
#pragma unroll
            for (int r = 0; r < 2; ++r) load_words<kWords>(src + hf * S::kCodeBytes + (g + 8 * r) * (D / 2) + t * (4 * kWords), kw[r]);
            const __half2* kp = reinterpret_cast<const __half2*>(src + S::kKpAt + hf * S::kParamBytes);
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                float d[4];
#pragma unroll
                for (int w = 2 * gr; w < 2 * gr + 2; ++w) {
                    uint32_t lo[4], hi[4];
                    codes_1024(kw[0][w], lo);
                    codes_1024(kw[1][w], hi);
                    if (w == 2 * gr)
                        mma_f16_from(d, lo[0], hi[0], lo[1], hi[1], qf[w][0], qf[w][1], qoff[gr][0], qoff[gr][1]);
                    else
                        mma_f16(d, lo[0], hi[0], lo[1], hi[1], qf[w][0], qf[w][1]);
                    mma_f16(d, lo[2], hi[2], lo[3], hi[3], qf[w][2], qf[w][3]);
                }
                const float2 k0 = __half22float2(kp[g * kGroups + gr]), k1 = __half22float2(kp[(g + 8) * kGroups + gr]);
                sc[0] = fmaf(k0.x, d[0], fmaf(k0.y, qsum[gr][0], sc[0]));
                sc[1] = fmaf(k0.x, d[1], fmaf(k0.y, qsum[gr][1], sc[1]));
                sc[2] = fmaf(k1.x, d[2], fmaf(k1.y, qsum[gr][0], sc[2]));
                sc[3] = fmaf(k1.x, d[3], fmaf(k1.y, qsum[gr][1], sc[3]));
            }
            bool up = false;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sc[c] *= mult[c & 1];
                if (!inner) {
                    const int j = j0 + kHalf * hf + g + 8 * (c >> 1), p = last[c & 1];
                    if ((kTree ? !(see[c & 1] >> (j - j0) & 1u) : j > p || (a.window > 0 && j <= p - a.window)) || !there) sc[c] = -inf;
                }
                up |= sc[c] > top[c & 1] + kSlack;
            }
            if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float m = fmaxf(sc[c], sc[c + 2]);
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                    m = fmaxf(m, top[c]);
                    const float keep = ex2(top[c] - m);
                    top[c] = m;
                    sum[c] *= keep;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        acc[k][c] *= keep;
                        acc[k][c + 2] *= keep;
                    }
                }
            }
            uint32_t pf[2];
            float w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = ex2(sc[c] - (top[c & 1] - kLift));
                sum[c & 1] += w[c];
            }
            pf[0] = transpose8(pack_f16x2(w[0], w[1]));
            pf[1] = transpose8(pack_f16x2(w[2], w[3]));

            // ---- values: dims g * D/8 + 4 w + e of positions (2t, 2t+1) and (2t+8, 2t+9)
            uint32_t step[2], low[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint2 v = *reinterpret_cast<const uint2*>(src + S::kVpAt + hf * S::kParamBytes + ((t + 4 * r) * kGroups + vg) * 8);
                step[r] = v.x;
                low[r] = v.y;
            }
            if (!inner) {
                // positions that no row sees count as zeros whatever they hold, and a value that is
                // not finite is taken out here and put back below for the rows that see it
                const int j_end = there ? q.ctx : 0, j_begin = a.window > 0 ? p0 - a.window + 1 : 0;   // (seen_from's registers cost 1 % here)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int j = j0 + kHalf * hf + 2 * t + 8 * r;
                    const uint32_t keep = (j >= j_begin && j < j_end ? 0xFFFFu : 0u) | (j + 1 >= j_begin && j + 1 < j_end ? 0xFFFF0000u : 0u);
                    step[r] &= keep;
                    low[r] &= keep;
                    const uint32_t bad = not_finite(step[r], low[r]);
                    step[r] &= ~bad;
                    low[r] &= ~bad;
                    poison |= bad != 0;
                }
            }
            uint32_t vw[2][kWords];
#pragma unroll
            for (int r = 0; r < 2; ++r) load_words<kWords>(src + S::kVAt + hf * S::kCodeBytes + (t + 4 * r) * D + g * (4 * kWords), vw[r]);
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint32_t a0[4], a1[4];
                values(vw[0][w], as_h2(step[0]), as_h2(low[0]), a0);
                values(vw[1][w], as_h2(step[1]), as_h2(low[1]), a1);
                mma_f16(acc[2 * w], a0[0], a0[1], a1[0], a1[1], pf[0], pf[1]);
                mma_f16(acc[2 * w + 1], a0[2], a0[3], a1[2], a1[3], pf[0], pf[1]);
            }
        }
        if (!inner && __any_sync(0xFFFFFFFFu, poison)) {
            for (int k = 0; k < kTile; ++k) {
                if (!((live >> (k / kHalf)) & 1u)) continue;
                const int j = j0 + k;
                const __half* p = reinterpret_cast<const __half*>(src + S::kVpAt + (k / kHalf) * S::kParamBytes) +
                                  (((k % kHalf) >> 1) * kGroups + vg) * 4 + (k & 1);
                const float nan = __half2float(__hfma(__float2half_rn(15.f), p[0], p[2])) * 0.f;   // 0 where every value is finite
                if (nan == 0.f || j >= q.ctx) continue;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (kTree ? !(see[c] >> k & 1u) : j > last[c] || (a.window > 0 && j <= last[c] - a.window)) continue;
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        acc[m][c] += nan;
                        acc[m][c + 2] += nan;
                    }
                }
            }
        }
    }

    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncwarp();   // every lane is done with the ring
}

// The unit's rows (slot null), or a partial result.
template <int D>
__device__ __forceinline__ void put(const AttendArgs& a, int h, const Seq& q, int row0, int rows, const Sums<D>& o, float* slot)
{
    using S = Shape<D>;
    constexpr int kWords = S::kWords;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, group = a.group;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float l = o.sum[c];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        const int r = 2 * t + c;
        if (r >= rows) continue;
        if (!slot) {
            const float k = l == 0.f ? 0.f : 1.f / l;
            const int tok = by_group(a, row0 + r);
            bf16_t* d = a.out + static_cast<long long>(q.row0 + tok) * a.ld_out + (h * group + row0 + r - tok * group) * D + g * (D / 8);
#pragma unroll
            for (int w = 0; w < kWords; w += 2)
                *reinterpret_cast<uint4*>(d + 4 * w) =
                    make_uint4(pack_bf16x2(o.acc[2 * w][c] * k, o.acc[2 * w][c + 2] * k),
                               pack_bf16x2(o.acc[2 * w + 1][c] * k, o.acc[2 * w + 1][c + 2] * k),
                               pack_bf16x2(o.acc[2 * w + 2][c] * k, o.acc[2 * w + 2][c + 2] * k),
                               pack_bf16x2(o.acc[2 * w + 3][c] * k, o.acc[2 * w + 3][c + 2] * k));
        } else {
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                *reinterpret_cast<float4*>(slot + r * D + g * (D / 8) + 4 * w) =
                    make_float4(o.acc[2 * w][c], o.acc[2 * w][c + 2], o.acc[2 * w + 1][c], o.acc[2 * w + 1][c + 2]);
            if (g == 0) {
                slot[kRows * D + r] = o.top[c];
                slot[kRows * D + kRows + r] = l;
            }
        }
    }
}

template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads, kCtas) kv4_few_kernel(AttendArgs a, int few_rows, Partials left, bool after)
{
    using S = Shape<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Piece pieces[kWarps][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* ring = smem + warp * S::kRing;
    float* first_slot = reinterpret_cast<float*>(smem + kWarps * S::kRing);   // [warp] partial results of slot 0
    int* warp_sums = reinterpret_cast<int*>(smem + kWarps * (S::kRing + 4 * S::kPartial));
    int* prefix = warp_sums + 16;

    if (!after) tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int group = a.group;
    scan_seqs<kWarps>(a.batch.n_seqs, prefix, warp_sums, [&](int s) {
        Seq q;
        const bool ok = load_seq(a.batch, s, q, blockIdx.x == 0 ? a.status : nullptr);
        return ok && q.n > 0 && q.n * group <= few_rows ? (tiles_of(q, a.window) + kUnitCost) * a.cache.n_kv * slices_of(q, group) : 0;
    });
    const int total = prefix[a.batch.n_seqs];
    const int n_ranges = range_count(total, gridDim.x * kWarps), b = blockIdx.x;
    const int begin = range_at(total, n_ranges, b * kWarps + warp), end = range_at(total, n_ranges, b * kWarps + warp + 1);
    if (lane < 2) pieces[warp][lane].u0 = -1;
    const float inf = __int_as_float(0x7F800000);

    for (int x = begin; x < end;) {
        const Unit u = unit_at(a, prefix, x);
        const int t0 = max(0, x - u.u0 - kUnitCost), t1 = max(0, min(u.len, end - u.u0) - kUnitCost);
        x = min(end, u.u0 + u.len);
        if (t0 == t1) continue;   // only the unit's start lies in the range
        Sums<D> o;
        attend_tiles<D, kTree>(a, ring, u.s, u.h, u.q, u.row0, u.rows, first_tile(u.q, a.window) + t0, t1 - t0, o);
        const bool whole = t0 == 0 && t1 == u.len - kUnitCost;
        float* slot = t0 > 0 ? first_slot + warp * S::kPartial : reinterpret_cast<float*>(ring);
        if (!whole && lane == 0)
            pieces[warp][t0 > 0 ? 0 : 1] = Piece{u.u0, t1 == u.len - kUnitCost, u.h, u.q.row0, u.row0, u.rows, u.u0 + u.len};
        put<D>(a, u.h, u.q, u.row0, u.rows, o, whole ? nullptr : slot);
    }
    __syncthreads();

    // ---- join the CTA's partial results, unit by unit.  Units of heads of 64, which leave warps without work, begin
    // at the warp where the one before ended (drafts 19.7 -> 19.0 us; with heads of 128 the main loop lost more to
    // registers than that: 8 x 131072 positions 231 -> 234).
    int begin_warp = 0;
    auto slot_of = [&](int w, int k) {
        return k == 0 ? first_slot + w * S::kPartial : reinterpret_cast<const float*>(smem + w * S::kRing);
    };
    Record rec{0, 0, 0, 0, 0};
    // entry i: warp i / 2, slot i % 2; a unit's pieces follow each other
    const int entry_u0 = lane < 2 * kWarps ? pieces[lane >> 1][lane & 1].u0 : -1;
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, entry_u0 >= 0); todo;) {
        const int i0 = __ffs(todo) - 1;
        const unsigned set = __ballot_sync(0xFFFFFFFFu, entry_u0 == __shfl_sync(0xFFFFFFFFu, entry_u0, i0));
        todo &= ~set;
        const Piece first = pieces[i0 >> 1][i0 & 1];
        const int last = 31 - __clz(set), ends = pieces[last >> 1][last & 1].ends;
        const bool starts = i0 & 1;
        float* to = left.slot(b, starts, D);
        for (int e = D == 64 ? ((warp - begin_warp) & (kWarps - 1)) * 32 + lane : tid; e < first.rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            float m = -inf, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (unsigned k = set; k; k &= k - 1) m = fmaxf(m, slot_of((__ffs(k) - 1) >> 1, (__ffs(k) - 1) & 1)[kRows * D + r]);
            for (unsigned k = set; k; k &= k - 1) {
                const float* p = slot_of((__ffs(k) - 1) >> 1, (__ffs(k) - 1) & 1);
                const float w = m == -inf ? 0.f : ex2(p[kRows * D + r] - m);
                const float4 v = *reinterpret_cast<const float4*>(p + r * D + d);
                o.x = fmaf(v.x, w, o.x);
                o.y = fmaf(v.y, w, o.y);
                o.z = fmaf(v.z, w, o.z);
                o.w = fmaf(v.w, w, o.w);
                l = fmaf(p[kRows * D + kRows + r], w, l);
            }
            if (starts && ends) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int row = first.row0 + r;
                const int tok = by_group(a, row);
                *reinterpret_cast<uint2*>(a.out + static_cast<long long>(first.seq_row0 + tok) * a.ld_out + (first.h * group + row - tok * group) * D + d) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
            } else {
                *reinterpret_cast<float4*>(to + r * D + d) = o;
                if (d == 0) {
                    to[kRows * D + r] = m;
                    to[kRows * D + kRows + r] = l;
                }
            }
        }
        if (D == 64) begin_warp += (first.rows * (D / 4) + 31) / 32;
        if (starts && !ends) {
            rec = Record{first.rows, first.row0, first.seq_row0, first.h, b};
            while (rec.last + 1 < static_cast<int>(gridDim.x) && range_at(total, n_ranges, (rec.last + 1) * kWarps) < first.u1) ++rec.last;
        }
    }
    if (tid == 0) left.records[b] = rec;
    if (after) tc::grid_dep_wait();   // no kernel completes before the one before it
}

// The form for a few short units: a cluster of kCluster CTAs per unit, each
// warp an equal share of its tiles, joined over the CTAs' shared memory.  One
// launch, and no tables of the batch's work to build first.
constexpr int kCluster = 8;

template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads, kCtas) kv4_unit_kernel(AttendArgs a, int few_rows, bool after)
{
    using S = Shape<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, rank = static_cast<int>(cluster_rank());
    uint8_t* ring = smem + warp * S::kRing;
    float* mine = reinterpret_cast<float*>(smem + kWarps * S::kRing);   // the CTA's partial result: sums, then (maximum, sum of weights)
    const int group = a.group, slices = (few_rows + kRows - 1) / kRows, per_seq = a.cache.n_kv * slices;
    const int unit = blockIdx.x / kCluster, s = unit / per_seq, h = (unit - s * per_seq) / slices, row0 = (unit - s * per_seq - h * slices) * kRows;
    const float inf = __int_as_float(0x7F800000);

    if (!after) tc::grid_dep_wait();
    tc::grid_dep_launch();
    Seq q;
    const bool ok = load_seq(a.batch, s, q, rank == 0 && unit == s * per_seq && tid == 0 ? a.status : nullptr);
    if (after) tc::grid_dep_wait();   // no kernel completes before the one before it
    const int rows = min(kRows, q.n * group - row0);
    if (!ok || rows <= 0 || q.n * group > few_rows) return;   // the whole cluster leaves, or none of it
    const int tiles = tiles_of(q, a.window);
    auto share = [&](int w) { return static_cast<int>(static_cast<long long>(tiles) * w / (kCluster * kWarps)); };   // first tile of warp w of the cluster
    const int t0 = share(rank * kWarps + warp), t1 = share(rank * kWarps + warp + 1);
    if (t0 < t1) {
        Sums<D> o;
        attend_tiles<D, kTree>(a, ring, s, h, q, row0, rows, first_tile(q, a.window) + t0, t1 - t0, o);
        put<D>(a, h, q, row0, rows, o, reinterpret_cast<float*>(ring));
    }
    __syncthreads();
    const int work = rows * (D / 4);
    for (int e = tid; e < work; e += kThreads) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float m = -inf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kWarps; ++w)
            if (share(rank * kWarps + w) < share(rank * kWarps + w + 1)) m = fmaxf(m, reinterpret_cast<const float*>(smem + w * S::kRing)[kRows * D + r]);
        for (int w = 0; w < kWarps; ++w) {
            if (share(rank * kWarps + w) == share(rank * kWarps + w + 1)) continue;
            const float* p = reinterpret_cast<const float*>(smem + w * S::kRing);
            const float k = m == -inf ? 0.f : ex2(p[kRows * D + r] - m);
            const float4 v = *reinterpret_cast<const float4*>(p + r * D + d);
            o.x = fmaf(v.x, k, o.x);
            o.y = fmaf(v.y, k, o.y);
            o.z = fmaf(v.z, k, o.z);
            o.w = fmaf(v.w, k, o.w);
            l = fmaf(p[kRows * D + kRows + r], k, l);
        }
        *reinterpret_cast<float4*>(mine + r * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(mine + kRows * D + 2 * r) = make_float2(m, l);
    }
    cluster_arrive();
    cluster_wait();
    for (int e = rank * kThreads + tid; e < work; e += kCluster * kThreads) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float2 ml[kCluster];
        float4 v[kCluster];
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
            ml[k] = ld_dsmem_f2(map_rank(tc::smem_u32(mine + kRows * D + 2 * r), k));
            v[k] = ld_dsmem_f4(map_rank(tc::smem_u32(mine + r * D + d), k));
        }
        float m = -inf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kCluster; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {   // (a CTA without tiles left zeros)
            const float w = m == -inf ? 0.f : ex2(ml[k].x - m);
            o.x = fmaf(v[k].x, w, o.x);
            o.y = fmaf(v[k].y, w, o.y);
            o.z = fmaf(v[k].z, w, o.z);
            o.w = fmaf(v[k].w, w, o.w);
            l = fmaf(ml[k].y, w, l);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int row = row0 + r;
        const int tok = by_group(a, row);
        *reinterpret_cast<uint2*>(a.out + static_cast<long long>(q.row0 + tok) * a.ld_out + (h * group + row - tok * group) * D + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
    cluster_arrive();
    cluster_wait();   // no CTA leaves while another reads its result
}

constexpr int kUnitTiles = 16;
constexpr int kMaxSmem = 227 * 1024;
static_assert(Shape<128>::kSmem + 4 * kMaxSeqs <= kMaxSmem, "shared memory");

template <int D, bool kTree>
cudaError_t run(const AttendArgs& a, int few_rows, void* ws, bool after, Partials* left, cudaStream_t stream)
{
    using S = Shape<D>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> clusters[64];   // that each device has room for at once; 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>& room = clusters[dev & 63];
    e = once_on_device(done, [&] {
        const cudaError_t f = cudaFuncSetAttribute(kv4_few_kernel<D, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024);
        return f == cudaSuccess ? cudaFuncSetAttribute(kv4_unit_kernel<D, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) : f;
    });
    if (e != cudaSuccess) return e;
    const int ctas = std::min(kMaxCtas, device_sms() * kCtas);
    // Units that all have a cluster on the GPU at once, with at most kUnitTiles tiles to a warp: a cluster each.
    // Measured both ways (us, heads of 128 in groups of 4, cluster / ranges): one sequence of 1000, 8000, 32000
    // positions 6.3 / 9.9, 10.9 / 24.5, 28 / 32; four sequences 6.8 / 12.1, 14.6 / 20.9, 40 / 44; but two waves
    // of clusters (16 rows to a unit, two sequences of 1000) 16.3 / 15.6, and at more positions the ranges,
    // which every SM takes part in.
    const long long units = static_cast<long long>(a.batch.n_seqs) * a.cache.n_kv * ((few_rows + kRows - 1) / kRows);
    if (a.batch.max_ctx_len <= kTile * kUnitTiles * kCluster * kWarps) {
        PdlLaunch l(dim3(static_cast<unsigned>(units * kCluster)), kThreads, S::kSmem, stream);
        cudaLaunchAttribute attr[2];
        attr[0] = l.attr[0];
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kCluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        l.cfg.attrs = attr;
        l.cfg.numAttrs = 2;
        if (room == 0) {
            int n = 0;
            cudaLaunchConfig_t one = l.cfg;   // the query does without the other attribute
            one.gridDim = dim3(kCluster);
            one.attrs = attr + 1;
            one.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kv4_unit_kernel<D, kTree>, &one);
            if (e != cudaSuccess) return e;
            room = n;
        }
        if (units <= room) {
            left->ctas = 0;
            e = cudaLaunchKernelEx(&l.cfg, kv4_unit_kernel<D, kTree>, a, few_rows, after);
            note_launch();
            return e;
        }
    }
    PdlLaunch l(dim3(ctas), kThreads, S::kSmem + 4 * a.batch.n_seqs, stream);
    *left = partials_at(ws, ctas, kRows);
    e = cudaLaunchKernelEx(&l.cfg, kv4_few_kernel<D, kTree>, a, few_rows, *left, after);
    note_launch();
    return e;
}

}  // namespace

size_t kv4_few_workspace(int head_dim) { return partials_bytes(kMaxCtas, kRows, head_dim); }

cudaError_t launch_kv4_few(const AttendArgs& a, int few_rows, void* ws, bool after, Partials* left, cudaStream_t stream)
{
    if (a.tree) return a.cache.head_dim == 64 ? run<64, true>(a, few_rows, ws, after, left, stream) : run<128, true>(a, few_rows, ws, after, left, stream);
    return a.cache.head_dim == 64 ? run<64, false>(a, few_rows, ws, after, left, stream) : run<128, false>(a, few_rows, ws, after, left, stream);
}

}  // namespace lora
