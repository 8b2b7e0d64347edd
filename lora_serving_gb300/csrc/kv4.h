// kv4.h -- internal launchers of the norm and the 4-bit cache's operators.
#pragma once

#include <atomic>
#include <cstdint>

#include "kv4.cuh"
#include "launch.h"

namespace lora {

// Multiprocessors of the current device (GB300: 152).
int device_sms();

// Runs `set` (a kernel's attributes) once on each device.
template <class F>
cudaError_t once_on_device(std::atomic<uint64_t>& done, F set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit)) return e;
    e = set();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launch configuration under programmatic dependent launch: every kernel
// here waits (griddepcontrol.wait) before its first read of memory, so only
// its own start overlaps the kernel before it (the second kernel of a call,
// whose first has waited, waits at its end).
struct PdlLaunch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    PdlLaunch(dim3 grid, int threads, size_t smem, cudaStream_t stream)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

struct NormArgs {
    bf16_t* y;
    int ld_y;
    uint8_t* y8;
    int ld_y8;
    float* scales;
    int ld_scales;
    int group;
    bf16_t* res_out;
    int ld_res_out;
    const bf16_t* x;
    int ld_x;
    const bf16_t* res;
    int ld_res;
    const bf16_t* w;
    int n_rows;
    int width;
    float eps;
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream);

struct AppendArgs {
    bf16_t* q_out;
    int ld_q;
    const bf16_t* x;
    int ld_x;
    int n_heads;
    int q_off, k_off, v_off;
    const float* rope;
    int rot_dim;
    int max_pos;
    const int32_t* positions;
    int ld_pos;
    int axis_end[LORA_MAX_ROPE_AXES];   // pairs below axis_end[a] and not below axis_end[a-1] turn with axis a
    int n_axes;
    kv4::Cache cache;
    kv4::Batch batch;
    int32_t* status;
};
cudaError_t launch_kv4_append(const AppendArgs& a, cudaStream_t stream);

struct ReadArgs {
    bf16_t* k;
    int ld_k;
    bf16_t* v;
    int ld_v;
    kv4::Cache cache;
    kv4::Batch batch;
    int32_t* status;
};
cudaError_t launch_kv4_read(const ReadArgs& a, cudaStream_t stream);

struct AttendArgs {
    bf16_t* out;
    int ld_out;
    const bf16_t* q;
    int ld_q;
    int n_heads;
    int group;              // heads to a kv head
    uint32_t group_magic;   // n / group is the upper half of n times this (0 where group is 1)
    float scale;
    int window;
    kv4::Cache cache;
    kv4::Batch batch;
    void* ws;
    size_t ws_bytes;
    int32_t* status;
    const uint32_t* tree;   // bits of drafted trees' rows, [n_rows][ld_tree]; NULL: rows see what lies before them
    int ld_tree;
};
constexpr int kMaxSeqs = 4096;   // sequences of one attention call (their running sum lies in shared memory)
// Positions of a sequence, and rows x heads of a kv head, of one attention
// call: the kernels count both in 32 bits, past the end of what they hold by
// a page, a tile or a block, and from a row before the first position back by
// a window (which the host cuts to the positions).
constexpr int kMaxPositions = 1 << 30;
// The longest line of tiles that a batch within these bounds lays out (the kernels count its places in 32 bits).
long long kv4_attend_places(const AttendArgs& a);
size_t kv4_attend_workspace(int n_heads, int n_kv, int head_dim, int max_q_len);
cudaError_t launch_kv4_attend(const AttendArgs& a, cudaStream_t stream);

struct PlanArgs {
    int32_t* q_starts;
    int32_t* ctx_lens;
    int32_t* row_seq;
    int32_t* positions;
    int64_t* slots;
    const int32_t* q_lens;
    const int32_t* lens;
    const int32_t* depths;
    int n_seqs;
    int max_rows;
    int max_q_len;
    int max_ctx_len;
    lora_kv4_pool_t pool;
    int page_shift;
    bool wide_in, wide_out;   // q_lens, lens and held on 16 bytes; row_seq, positions and slots
    int32_t* status;
};
cudaError_t launch_kv4_plan(const PlanArgs& a, cudaStream_t stream);

struct KeepArgs {
    struct Pages {
        uint8_t* pages;
        long long page_stride;
        int n_pages;
    };
    Pages layers[LORA_KEEP_LAYERS];
    kv4::Cache cache;   // what the layers have in common
    kv4::Batch batch;
    const int32_t* held;   // pages of each sequence, or NULL
    const int32_t* n_keep;
    const int32_t* path;
    int ld_path;
    int32_t* lens;      // NULL in all launches but a call's first
    int least_pages;    // pages of the smallest of the call's caches, whichever launch takes it
    int32_t* status;
};
cudaError_t launch_kv4_keep(const KeepArgs& a, int n_layers, cudaStream_t stream);

struct LogitsArgs {
    void* out;
    int ld_out;
    const void* logits;
    int ld;
    int n_rows;
    int vocab;
    lora_logits_rules_t rules;   // tokens NULL: none
    const int32_t* row_seq;
    const int32_t* drafts;
    const uint32_t* tree;
    int ld_tree;
    const int32_t* q_starts;
    const uint32_t* allowed;
    int ld_allowed;
    int n_allowed;
    const int32_t* allowed_rows;
    int32_t* status;
};
cudaError_t launch_logits_adjust(const LogitsArgs& a, bool in_f32, bool out_f32, cudaStream_t stream);

}  // namespace lora
