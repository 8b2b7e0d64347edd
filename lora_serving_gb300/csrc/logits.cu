// logits.cu -- penalties for repeated tokens, biases and masks on logits.
//
// A CTA takes a chunk of the vocabulary for some neighbouring rows.  It counts
// the tokens of the row's request in shared memory, a 32-bit word to a token
// of the chunk (20 bits of count, a bit for the prompt, 11 bits for the last
// bias entry that names it), by integer atomics, whose order changes nothing;
// then the chunk's logits stream past the words.  Rows of one request that
// follow each other (a drafted tree) share the counts: only a row's own path
// is added before it and taken off after it.  Bound: HBM, the logits in and out.
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 8192;   // of a chunk
constexpr uint32_t kCount = (1u << 20) - 1, kPrompt = 1u << 20;
constexpr int kBiasShift = 21;

template <bool F32>
__device__ __forceinline__ void load8(const void* row, int c, float* f)
{
    if (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
        const float4 u = p[0], w = p[1];
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const bf16_t*>(row) + c);
        f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
        f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
    }
}
template <bool F32>
__device__ __forceinline__ void store8(void* row, int c, const float* f)
{
    if (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + c);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<bf16_t*>(row) + c) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
}

struct Penalties {
    float repetition, frequency, presence;
    const float* bias;   // of the request
    __device__ __forceinline__ float operator()(float x, uint32_t w) const
    {
        const float c = static_cast<float>(w & kCount);
        if (w & (kCount | kPrompt)) x = x > 0.f ? __fdiv_rn(x, repetition) : x * repetition;
        if (w & kCount) x = x - frequency * c - presence;
        if (w >> kBiasShift) x += __ldg(bias + (w >> kBiasShift) - 1);
        return x;
    }
};

template <bool IN32, bool OUT32>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(LogitsArgs a, int chunk, int rows_each)
{
    extern __shared__ __align__(16) uint32_t words[];   // [chunk]
    const int tid = threadIdx.x;
    const int v0 = blockIdx.x * chunk, v1 = min(a.vocab, v0 + chunk);
    const int t_end = min(a.n_rows, (static_cast<int>(blockIdx.y) + 1) * rows_each);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int32_t* const status = blockIdx.x == 0 && tid == 0 ? a.status : nullptr;
    const float inf = __int_as_float(0x7F800000);
    auto count = [&](int token, uint32_t what) {
        const uint32_t u = static_cast<uint32_t>(token) - static_cast<uint32_t>(v0);
        if (token >= 0 && u < static_cast<uint32_t>(v1 - v0)) atomicAdd(words + u, what);
    };
    int counted = -1;      // the request whose words these are
    bool plain = true;     // none of them matters
    Penalties rule{1.f, 0.f, 0.f, nullptr};
    for (int t = blockIdx.y * rows_each; t < t_end; ++t) {
        // ---- the row's request and mask
        const uint32_t* mask = nullptr;
        if (a.allowed) {
            const int m = a.allowed_rows ? __ldg(a.allowed_rows + t) : t;
            if (m < -1 || m >= a.n_allowed) {
                flag(status, LORA_DEV_SLOT_OUT_OF_RANGE);
                continue;
            }
            if (m >= 0) mask = a.allowed + static_cast<long long>(m) * a.ld_allowed;
        }
        const int s = a.row_seq ? __ldg(a.row_seq + t) : t;
        if (s == -1) continue;
        int first = 0, n_path = 0;
        if (a.rules.tokens) {
            bool ok = s >= 0 && s < a.rules.n_seqs;
            int len = 0, prompt = 0, biases = 0;
            if (ok) {
                len = __ldg(a.rules.token_lens + s);
                prompt = __ldg(a.rules.prompt_lens + s);
                biases = a.rules.bias_ids ? __ldg(a.rules.n_bias + s) : 0;
                ok = len >= 0 && len <= a.rules.ld_tokens && prompt >= 0 && prompt <= len && biases >= 0 && biases <= a.rules.ld_bias;
                if (a.drafts) {
                    first = __ldg(a.q_starts + s);
                    const int end = __ldg(a.q_starts + s + 1);
                    ok = ok && first >= 0 && t >= first && t < end && end <= a.n_rows;
                    n_path = min(end - first, 32 * a.ld_tree);
                }
            }
            if (!ok) {
                flag(status, LORA_DEV_BAD_SEGMENT);
                continue;
            }
            if (s != counted) {
                counted = s;
                rule.repetition = a.rules.repetition ? __ldg(a.rules.repetition + s) : 1.f;
                rule.frequency = a.rules.frequency ? __ldg(a.rules.frequency + s) : 0.f;
                rule.presence = a.rules.presence ? __ldg(a.rules.presence + s) : 0.f;
                rule.bias = a.rules.bias + static_cast<long long>(s) * a.rules.ld_bias;
                const bool even = rule.repetition == 1.f && rule.frequency == 0.f && rule.presence == 0.f;   // counts change nothing
                plain = even && biases == 0;
                if (!plain) {
                    __syncthreads();   // the last row's words have been read
                    for (int i = tid; i < chunk / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
                    __syncthreads();
                    const int32_t* ids = a.rules.bias_ids + static_cast<long long>(s) * a.rules.ld_bias;
                    for (int i = tid; i < biases; i += kThreads) {
                        const int token = __ldg(ids + i);
                        if (token >= v0 && token < v1) atomicMax(words + token - v0, static_cast<uint32_t>(i + 1) << kBiasShift);
                    }
                    if (biases) __syncthreads();
                    if (!even) {
                        const int32_t* tokens = a.rules.tokens + static_cast<long long>(s) * a.rules.ld_tokens;
#pragma unroll 4
                        for (int i = tid; i < len; i += kThreads) {
                            const int token = __ldg(tokens + i);
                            if (i >= prompt) count(token, 1);
                            else if (token >= v0 && token < v1) atomicOr(words + token - v0, kPrompt);
                        }
                    }
                }
            }
        }
        const uint32_t* bits = a.drafts ? a.tree + static_cast<long long>(t) * a.ld_tree : nullptr;
        auto path = [&](uint32_t what) {
            for (int j = tid; j < n_path; j += kThreads)
                if (__ldg(bits + (j >> 5)) >> (j & 31) & 1u) count(__ldg(a.drafts + first + j), what);
        };
        if (!plain) {
            if (n_path) path(1u);
            __syncthreads();
        }
        // ---- the logits
        const char* in = static_cast<const char*>(a.logits) + static_cast<long long>(t) * a.ld * (IN32 ? 4 : 2);
        char* out = static_cast<char*>(a.out) + static_cast<long long>(t) * a.ld_out * (OUT32 ? 4 : 2);
#pragma unroll 2
        for (int c = v0 + 8 * tid; c < v1; c += 8 * kThreads) {
            const uint32_t keep = mask ? __ldg(mask + (c >> 5)) >> (c & 31) & 0xFFu : 0xFFu;
            const int n = min(8, v1 - c);
            float f[8];
            if (n == 8) {
                load8<IN32>(in, c, f);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = i >= n ? 0.f : IN32 ? reinterpret_cast<const float*>(in)[c + i] : bf16_lo(reinterpret_cast<const bf16_t*>(in)[c + i]);
            }
            if (!plain) {
                const uint4 u = reinterpret_cast<const uint4*>(words)[(c - v0) / 4], w = reinterpret_cast<const uint4*>(words)[(c - v0) / 4 + 1];
                if (u.x | u.y | u.z | u.w | w.x | w.y | w.z | w.w) {
                    const uint32_t of[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (of[i]) f[i] = rule(f[i], of[i]);
                }
            }
            if (keep != 0xFFu) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!(keep >> i & 1u)) f[i] = -inf;
            }
            if (n == 8) {
                store8<OUT32>(out, c, f);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i >= n) break;
                    if (OUT32) reinterpret_cast<float*>(out)[c + i] = f[i];
                    else reinterpret_cast<bf16_t*>(out)[c + i] = static_cast<bf16_t>(pack_bf16x2(f[i], 0.f));
                }
            }
        }
        if (!plain && n_path) {   // off again, once everyone has read them
            __syncthreads();
            path(0u - 1u);
        }
    }
}

template <bool IN32, bool OUT32>
cudaError_t run(const LogitsArgs& a, int chunk, int rows_each, cudaStream_t stream)
{
    const unsigned chunks = (a.vocab + chunk - 1) / chunk, groups = (a.n_rows + rows_each - 1) / rows_each;
    PdlLaunch l(dim3(chunks, groups), kThreads, a.rules.tokens ? 4 * chunk : 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, logits_adjust_kernel<IN32, OUT32>, a, chunk, rows_each);
    note_launch();
    return e;
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsArgs& a, bool in_f32, bool out_f32, cudaStream_t stream)
{
    const int sms = device_sms();
    int chunk = kMostTokens;
    while (chunk > 8 * kThreads && static_cast<long long>(a.n_rows) * ((a.vocab + chunk - 1) / chunk) < 4 * sms) chunk /= 2;
    const long long ctas = static_cast<long long>(a.n_rows) * ((a.vocab + chunk - 1) / chunk);
    int rows_each = a.drafts ? static_cast<int>(std::min<long long>(16, std::max<long long>(1, ctas / (7 * sms)))) : 1;
    while ((a.n_rows + rows_each - 1) / rows_each > 65535) rows_each *= 2;   // a grid's second dimension
    return in_f32 ? out_f32 ? run<true, true>(a, chunk, rows_each, stream) : run<true, false>(a, chunk, rows_each, stream)
                  : out_f32 ? run<false, true>(a, chunk, rows_each, stream) : run<false, false>(a, chunk, rows_each, stream);
}

}  // namespace lora
