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

}  // namespace lora
