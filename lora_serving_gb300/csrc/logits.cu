// logits.cu -- penalties for repeated tokens, biases and masks on logits.
//
// A CTA takes a chunk of the vocabulary for some neighbouring rows.  It counts
// the tokens of the row's request in shared memory, a 32-bit word to a token
// of the chunk (20 bits of count, a bit for the prompt, 11 bits for the last
// bias entry that names it), by integer atomics, whose order changes nothing,
// with a bit to each token that has a word.  The logits then stream past in
// vectors of eight, which look at their eight bits and at the words of those
// that are set; a row's vectors are on their way while the last row's are
// worked on.  Rows of one request that follow each other (a drafted tree)
// share the counts: only a row's own path is added before it and taken off
// after it, by each warp for its own tokens, so that no row waits for a barrier.
// A chunk is every n-th block of 256 tokens: a request's tokens lie close
// together in a vocabulary that is ordered by frequency, and a chunk of
// neighbours would have them all.
//
// What bounds it.  HBM by its bytes, then instructions (some 45 a vector of a
// warp without rules) and the start of a CTA's first row: tables, tokens,
// counts, 4 us, which few CTAs are there to hide.  Measured: 512 rows of 128256
// tokens in trees of 32, bf16, masks and penalties 57 us (263 MB, 0.69 of a
// copy's rate; with masks alone 44), 64 rows to fp32 14.4 (50 MB; 12.1), one row
// of 32000 tokens 1.9, start to start.
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kCount = (1u << 20) - 1, kPrompt = 1u << 20;
constexpr int kBiasShift = 21;
constexpr int kBlock = 256;  // neighbouring tokens of a chunk: a warp's vectors
constexpr int kAtOnce = 8;   // of a request's tokens, that a thread has on their way
constexpr int kRows = 4;     // of a CTA, at most
// CTAs with one vector to a thread, per SM, up to which a call is small: 4 rows of 128256 tokens 3.3 us (4.4 in larger
// chunks), 8 rows 4.8 (6.3), but 16 rows 9.2 (7.2).
constexpr int kSmall = 4;
// On an SM: 80 registers a thread, for the vectors on their way.  Measured (us, 64 / 256 rows of 128256 tokens, no drafts; CTAs
// and vectors): 3 and 5 15.2 / 45.3, 4 and 5 16.3 / 45.6, 4 and 4 16.2 / 48.0, 5 and 3 17.0 / 54.2.
constexpr int kCtas = 3;
constexpr int kVecs16 = 5;   // vectors of a thread and row; of fp32 logits, which are twice as long, 2

template <bool F32>
__device__ __forceinline__ float load1(const char* row, int c)
{
    return F32 ? reinterpret_cast<const float*>(row)[c] : bf16_lo(reinterpret_cast<const bf16_t*>(row)[c]);
}
template <bool F32>
__device__ __forceinline__ void store1(char* row, int c, float f)
{
    if (F32) reinterpret_cast<float*>(row)[c] = f;
    else reinterpret_cast<bf16_t*>(row)[c] = static_cast<bf16_t>(pack_bf16x2(f, 0.f));
}

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xFF800000); }

// Eight logits as they lie in memory.
template <bool F32>
struct Raw {
    uint4 u[F32 ? 2 : 1];
};
// (the row's address is the warp's own, the column's offset 32 bits: the one instruction adds both)
template <bool F32>
__device__ __forceinline__ void load8(const char* row, uint32_t c, Raw<F32>& r)
{
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) r.u[i] = *reinterpret_cast<const uint4*>(row + c * (F32 ? 4u : 2u) + 16 * i);
}
// Of two bf16 logits those that two bits keep, -infinity for the others.
__device__ __forceinline__ uint32_t keep2(uint32_t x, uint32_t bits)
{
    const uint32_t m = ((bits & 3u) * 0x8001u & 0x10001u) * 0xFFFFu;   // the halves that stay
    return (x & m) | (0xFF80FF80u & ~m);
}

struct Penalties {
    float repetition, frequency, presence;
    const float* bias;   // of the request
    __device__ __forceinline__ float operator()(float x, uint32_t w) const
    {
        if (w & (kCount | kPrompt)) x = x > 0.f ? __fdiv_rn(x, repetition) : x * repetition;
        if (w & kCount) x = x - frequency * static_cast<float>(w & kCount) - presence;
        if (w >> kBiasShift) x += __ldg(bias + (w >> kBiasShift) - 1);
        return x;
    }
};

// Eight logits to out's type and place: those with words (bits of `some`) under their rules, those whose bit is not set in
// keep as -infinity.
template <bool IN32, bool OUT32>
__device__ __forceinline__ void put8(char* to, const Raw<IN32>& r, uint32_t keep, uint32_t some, const uint32_t* words, const Penalties& rule)
{
    const uint4 v = r.u[0], w = r.u[IN32 ? 1 : 0];
    if (!IN32 && !OUT32) {
        uint32_t h[4] = {v.x, v.y, v.z, v.w};
        for (; some; some &= some - 1) {   // one after the other: few have any, and eight tests in a row cost every warp eight branches
            const int i = __ffs(some) - 1;
            const uint32_t pair = i & 4 ? (i & 2 ? h[3] : h[2]) : (i & 2 ? h[1] : h[0]);
            const float y = rule(i & 1 ? bf16_hi(pair) : bf16_lo(pair), words[i]);
            const uint32_t now = __byte_perm(pair, pack_bf16x2(y, y), i & 1 ? 0x5410 : 0x3254);
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = i >> 1 == k ? now : h[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = keep2(h[k], keep >> 2 * k);
        *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
        return;
    }
    float f[8];
    if (IN32) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        f[4] = __uint_as_float(w.x); f[5] = __uint_as_float(w.y); f[6] = __uint_as_float(w.z); f[7] = __uint_as_float(w.w);
    } else {
        f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
    }
    for (; some; some &= some - 1) {
        const int i = __ffs(some) - 1;
        float x = f[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) x = i == k ? f[k] : x;
        x = rule(x, words[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = i == k ? x : f[k];
    }
    if (keep != 0xFFu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = keep >> i & 1u ? f[i] : minus_inf();
    }
    if (OUT32) {
        reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
}

// A request's entries, checked.
struct Request {
    bool ok, counts, plain;   // counts: its tokens matter; plain: neither they nor biases do
    int len, prompt, biases;
    int first, end;           // with drafts: its rows
    Penalties rule;
};
__device__ __forceinline__ Request request_of(const LogitsArgs& a, int s)
{
    Request r{true, false, true, 0, 0, 0, 0, 0x7FFFFFFF, {1.f, 0.f, 0.f, nullptr}};
    r.ok = s >= -1;
    if (!a.rules.tokens) return r;
    r.ok = s >= 0 && s < a.rules.n_seqs;
    if (!r.ok) return r;
    r.len = __ldg(a.rules.token_lens + s);
    r.prompt = __ldg(a.rules.prompt_lens + s);
    if (a.rules.bias_ids) r.biases = __ldg(a.rules.n_bias + s);
    if (a.rules.repetition) r.rule.repetition = __ldg(a.rules.repetition + s);
    if (a.rules.frequency) r.rule.frequency = __ldg(a.rules.frequency + s);
    if (a.rules.presence) r.rule.presence = __ldg(a.rules.presence + s);
    r.rule.bias = a.rules.bias + static_cast<long long>(s) * a.rules.ld_bias;
    if (a.drafts) {
        r.first = __ldg(a.q_starts + s);
        r.end = __ldg(a.q_starts + s + 1);
    }
    r.ok = r.len >= 0 && r.len <= a.rules.ld_tokens && r.prompt >= 0 && r.prompt <= r.len && r.biases >= 0 && r.biases <= a.rules.ld_bias &&
           r.first >= 0 && r.first <= r.end && (!a.drafts || r.end <= a.n_rows);   // (in this order their difference stays in 32 bits)
    r.counts = r.rule.repetition != 1.f || r.rule.frequency != 0.f || r.rule.presence != 0.f;
    r.plain = !r.ok || (!r.counts && r.biases == 0);
    return r;
}

// What a row needs before its logits: read a row ahead.
struct Row {
    int seq, set;
    uint32_t bits[2];   // of its path, the first 64
};

// kVecs: vectors of a thread on their way; kTurns: so often, of a row.
template <int kVecs, int kTurns>
struct Shape {
    static constexpr int kChunk = 8 * kThreads * kVecs * kTurns;   // tokens of a CTA
    static constexpr int kSmem = kChunk * 4 + kChunk / 8;       // words, and a bit to each
};

// kDrafts: rows of drafted trees, which share a request's counts; without them a CTA has one row.
template <bool IN32, bool OUT32, int kVecs, int kTurns, bool kDrafts>
__global__ void __launch_bounds__(kThreads, kCtas) logits_adjust_kernel(LogitsArgs a, int rows_each, int chunks, uint32_t magic)
{
    using S = Shape<kVecs, kTurns>;
    constexpr int kIn = IN32 ? 4 : 2, kOut = OUT32 ? 4 : 2;
    extern __shared__ __align__(16) uint32_t words[];   // [kChunk]
    uint32_t* const some = words + S::kChunk;           // [kChunk / 32] the tokens that have a word (or had one on a path)
    const int tid = threadIdx.x, lane = tid & 31;
    const int group = blockIdx.x / chunks, x = blockIdx.x - group * chunks;
    const int place = ((tid >> 5) + x) % kWarps;        // the warp's blocks: the dense first ones go to another scheduler in every CTA
    const int t_begin = group * rows_each, t_end = kDrafts ? min(a.n_rows, t_begin + rows_each) : t_begin + 1;
    const bool rules = a.rules.tokens != nullptr;
    auto clear = [&] {
        for (int i = tid; i < S::kSmem / 16; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
    };
    if (rules) clear();
    bool clean = true;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int32_t* const status = x == 0 && tid == 0 ? a.status : nullptr;
    // the chunk: every chunks-th block of kBlock tokens, from the x-th on
    const uint32_t c0 = (place * chunks + x) * kBlock + 8 * lane, c_step = kWarps * chunks * kBlock;   // this thread's vectors
    const uint32_t full = a.vocab & ~7u;                // columns of whole vectors
    // the vocabulary's last columns, less than a vector: a thread's, and their place among its vectors
    const int tail = full < static_cast<uint32_t>(a.vocab) && full >= c0 && (full - c0) % c_step == 0 ? static_cast<int>((full - c0) / c_step) : -1;
    auto word_of = [&](int token) -> int {   // a token's place in the chunk, -1: it is not in it
        if (token < 0 || token >= a.vocab) return -1;
        const int b = token / kBlock, at = magic ? static_cast<int>(__umulhi(b, magic)) : b;   // exact: blocks times chunks stay below 2^32
        return b - at * chunks == x ? at * kBlock + token % kBlock : -1;
    };
    auto own_word = [&](int token) -> int {   // its word where it is in one of the warp's blocks, otherwise -1
        const int w = word_of(token);
        return w >= 0 && w / kBlock % kWarps == place ? w : -1;
    };
    auto note = [&](int w) { atomicOr(some + (w >> 5), 1u << (w & 31)); };
    // a row's vectors and what it needs, on their way before they are asked for
    Raw<IN32> raw[kVecs];
    uint32_t keep[kVecs];
    Row next{-1, -1, {0, 0}};
    auto mask_of = [&](int set) {
        return reinterpret_cast<const uint8_t*>(set >= 0 && set < a.n_allowed ? a.allowed + static_cast<long long>(set) * a.ld_allowed : nullptr);
    };
    auto in_row = [&](int t) { return static_cast<const char*>(a.logits) + static_cast<long long>(t) * a.ld * kIn; };
    auto fetch = [&](int k, int turn, const char* row, const uint8_t* mask) {
        const uint32_t c = c0 + (turn * kVecs + k) * c_step;
        if (c < full) {
            load8<IN32>(row, c, raw[k]);
            keep[k] = mask ? __ldg(mask + (c >> 3)) : 0xFFu;
        }
    };
    auto fetch_row = [&](int t) {
        next.seq = a.row_seq ? __ldg(a.row_seq + t) : t;
        next.set = !a.allowed ? -1 : a.allowed_rows ? __ldg(a.allowed_rows + t) : t;
#pragma unroll
        for (int i = 0; i < 2; ++i) next.bits[i] = kDrafts && i < a.ld_tree ? __ldg(a.tree + static_cast<long long>(t) * a.ld_tree + i) : 0;
    };
    fetch_row(t_begin);
    {
        const uint8_t* mask = mask_of(next.set);
#pragma unroll
        for (int k = 0; k < kVecs; ++k) fetch(k, 0, in_row(t_begin), mask);
    }
    int counted = -1;              // the request whose words these are
    Request r{};
    int mine[2] = {-1, -1};        // words of the lane's drafted tokens (of the first 64) that are in the warp's blocks
    bool paths = false;            // whether the warp has any: most have none (512 rows in trees of 32 57.4 us, 58.0 without the test)
    for (int t = t_begin; t < t_end; ++t) {
        const Row row = next;
        const int s = row.seq;
        if (t + 1 < t_end) fetch_row(t + 1);
        if (s != counted) {
            counted = s;
            // its first tokens and biases on their way with its lengths, which say later how many of them count
            const int32_t* const tokens = a.rules.tokens + static_cast<long long>(s) * a.rules.ld_tokens;
            const int32_t* const ids = a.rules.bias_ids + static_cast<long long>(s) * a.rules.ld_bias;
            // (registers that rows which follow need for their vectors: 512 rows in trees 60 us, 64 with this)
            const bool known = !kDrafts && rules && s >= 0 && s < a.rules.n_seqs;
            int early[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) early[k] = known && tid + k * kThreads < a.rules.ld_tokens ? __ldg(tokens + tid + k * kThreads) : -1;
            const int early_id = known && a.rules.bias_ids && tid < a.rules.ld_bias ? __ldg(ids + tid) : -1;
            r = request_of(a, s);
            mine[0] = mine[1] = -1;
            if (!r.plain) {
                if (kDrafts) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (lane + 32 * i < r.end - r.first) mine[i] = own_word(__ldg(a.drafts + r.first + lane + 32 * i));
                    paths = r.end - r.first > 64 || __any_sync(0xFFFFFFFFu, mine[0] >= 0 || mine[1] >= 0);
                }
                __syncthreads();   // the words are cleared, or the last request's have been read
                if (!clean) {
                    clear();
                    __syncthreads();
                }
                clean = false;
                if (r.biases) {
                    for (int i = tid; i < r.biases; i += kThreads) {
                        const int w = word_of(!kDrafts && i < kThreads ? early_id : __ldg(ids + i));
                        if (w >= 0 && atomicMax(words + w, static_cast<uint32_t>(i + 1) << kBiasShift) == 0) note(w);
                    }
                    __syncthreads();   // counts go on top of the largest
                }
                if (r.counts) {
                    for (int i0 = tid; i0 < r.len; i0 += kAtOnce * kThreads) {
                        int id[kAtOnce];
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k) id[k] = i0 + k * kThreads >= r.len ? -1 : !kDrafts && i0 < kAtOnce * kThreads ? early[k] : __ldg(tokens + i0 + k * kThreads);
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k) {
                            const int w = word_of(id[k]);
                            if (w >= 0 && (i0 + k * kThreads >= r.prompt ? atomicAdd(words + w, 1u) : atomicOr(words + w, kPrompt)) == 0) note(w);
                        }
                    }
                }
                __syncthreads();   // the counts are there
            }
        }
        // ---- whether the row is written
        bool live = s != -1;
        if (live && a.allowed && (row.set < -1 || row.set >= a.n_allowed)) {
            flag(status, LORA_DEV_SLOT_OUT_OF_RANGE);
            live = false;
        }
        if (live && (!r.ok || (kDrafts && (t < r.first || t >= r.end)))) {
            flag(status, LORA_DEV_BAD_SEGMENT);
            live = false;
        }
        // ---- the row's path, every warp those of its tokens that are in its blocks (no other looks at them)
        const int n_path = !kDrafts || !live || r.plain || !paths ? 0 : min(r.end - r.first, 32 * a.ld_tree);
        auto path = [&](auto each) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (mine[i] >= 0 && row.bits[i] >> lane & 1u && lane + 32 * i < n_path) each(mine[i]);
            for (int j = 64 + lane; j < n_path; j += 32)
                if (__ldg(a.tree + static_cast<long long>(t) * a.ld_tree + (j >> 5)) >> lane & 1u) {
                    const int w = own_word(__ldg(a.drafts + r.first + j));
                    if (w >= 0) each(w);
                }
        };
        if (n_path) {
            path([&](int w) { if (atomicAdd(words + w, 1u) == 0) note(w); });
            __syncwarp();
        }
        // ---- the logits
        const bool more = t + 1 < t_end;
        const char* const next_in = in_row(t + 1);   // (read where there is one)
        const uint8_t* const next_mask = mask_of(next.set);
        if (live) {
            char* const out = static_cast<char*>(a.out) + static_cast<long long>(t) * a.ld_out * kOut;
#pragma unroll 1
            for (int turn = 0; turn < kTurns; ++turn) {
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const uint32_t c = c0 + (turn * kVecs + k) * c_step;
                    const int at = ((turn * kVecs + k) * kWarps + place) * kBlock + 8 * lane;
                    if (c < full)
                        put8<IN32, OUT32>(out + c * kOut, raw[k], keep[k], r.plain ? 0 : reinterpret_cast<const uint8_t*>(some)[at >> 3], words + at, r.rule);
                    if (kTurns > 1 && turn + 1 < kTurns) fetch(k, turn + 1, in_row(t), mask_of(row.set));
                    else if (more) fetch(k, 0, next_in, next_mask);
                }
            }
            if (tail >= 0 && tail < kVecs * kTurns) {
                const char* const in = in_row(t);
                const uint8_t* const mask = mask_of(row.set);
                for (int c = full; c < a.vocab; ++c) {
                    const int at = (tail * kWarps + place) * kBlock + 8 * lane + c - static_cast<int>(full);
                    float f = load1<IN32>(in, c);
                    if (!r.plain && words[at]) f = r.rule(f, words[at]);
                    store1<OUT32>(out, c, !mask || (mask[c >> 3] >> (c & 7) & 1u) ? f : minus_inf());
                }
            }
        } else if (more) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) fetch(k, 0, next_in, next_mask);
        }
        if (n_path) {   // the path off again
            __syncwarp();
            path([&](int w) { atomicSub(words + w, 1u); });
        }
    }
}

template <bool IN32, bool OUT32, int kVecs, int kTurns, bool kDrafts>
cudaError_t run(const LogitsArgs& a, cudaStream_t stream)
{
    using S = Shape<kVecs, kTurns>;
    static std::atomic<uint64_t> done{0};
    if (S::kSmem > 48 * 1024) {
        const cudaError_t e = once_on_device(done, [] { return cudaFuncSetAttribute(logits_adjust_kernel<IN32, OUT32, kVecs, kTurns, kDrafts>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem); });
        if (e != cudaSuccess) return e;
    }
    const int chunks = (a.vocab + S::kChunk - 1) / S::kChunk;
    // Rows of a drafted tree to a CTA, that share its counts, as long as the CTAs fill the SMs.  Measured (us, 16 trees of
    // 32 rows, 128256 tokens; 3 waves of CTAs with 4 rows): 1 row 95, 4 rows 59.7, 8 rows 68.
    int rows_each = 1;
    while (kDrafts && rows_each < kRows && static_cast<long long>(chunks) * ((a.n_rows + 2 * rows_each - 1) / (2 * rows_each)) >= kCtas * device_sms()) rows_each *= 2;
    const long long ctas = static_cast<long long>(chunks) * ((a.n_rows + rows_each - 1) / rows_each);   // (the entry point bounds it)
    PdlLaunch l(dim3(static_cast<unsigned>(ctas)), kThreads, a.rules.tokens ? S::kSmem : 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, logits_adjust_kernel<IN32, OUT32, kVecs, kTurns, kDrafts>, a, rows_each, chunks, chunks > 1 ? static_cast<uint32_t>((1ull << 32) / chunks + 1) : 0);
    note_launch();
    return e;
}

template <bool IN32, bool OUT32>
cudaError_t pick(const LogitsArgs& a, cudaStream_t stream)
{
    // Small calls want their chunks on as many SMs as there are, and a vocabulary that fits in the short chunk has no use for the
    // long one's words (16384 rows of 2048 tokens 108 us, in long chunks 145; of 4096 tokens 196 and 162).
    const long long ctas = static_cast<long long>(a.n_rows) * ((a.vocab + 8 * kThreads - 1) / (8 * kThreads));
    constexpr int kVecs = IN32 ? kVecs16 / 2 : kVecs16;
    if (a.vocab <= 8 * kThreads || ctas < kSmall * device_sms()) return a.drafts ? run<IN32, OUT32, 1, 1, true>(a, stream) : run<IN32, OUT32, 1, 1, false>(a, stream);
    if (a.drafts) return run<IN32, OUT32, kVecs, 1, true>(a, stream);
    // Longer chunks, read in turns: fewer starts, but each takes longer.  Measured (us, rows of 128256 tokens): bf16 to fp32, where
    // they make one wave of two, 48 rows 12.7 in chunks of five vectors and 11.3 in three turns of three, 64 rows 14.1 and 12.7;
    // where they do not, 32 rows 8.8 and 10.1, 96 rows 23.1 and 23.3, 200 rows of 50257 18.8 and 21.8.  fp32, past two waves, in
    // chunks of two vectors and two turns of three 32 rows 10.4 and 9.9, 256 rows 69.5 and 51.1; before, 16 rows 6.4 and 7.9.
    const long long slots = kCtas * device_sms();
    auto takes = [&](int vecs) { return static_cast<long long>(a.n_rows) * ((a.vocab + 8 * kThreads * vecs - 1) / (8 * kThreads * vecs)); };
    if (IN32 ? takes(kVecs) > 2 * slots : takes(kVecs) > slots && takes(9) <= slots) return run<IN32, OUT32, 3, IN32 ? 2 : 3, false>(a, stream);
    return run<IN32, OUT32, kVecs, 1, false>(a, stream);
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsArgs& a, bool in_f32, bool out_f32, cudaStream_t stream)
{
    return in_f32 ? out_f32 ? pick<true, true>(a, stream) : pick<true, false>(a, stream)
                  : out_f32 ? pick<false, true>(a, stream) : pick<false, false>(a, stream);
}

}  // namespace lora
