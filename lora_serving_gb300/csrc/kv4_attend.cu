// kv4_attend.cu -- which kernel takes which rows of lora_kv4_attend.
#include <algorithm>

#include "kv4_attend.cuh"

namespace lora {

namespace {

// Query rows to a kv head (a sequence's rows x the heads of a group) up to
// which a sequence goes to the kernel for few rows.  Where all of a batch's
// sequences are that short, all go there.  In a batch with longer ones the
// single tokens still do, in the narrowest form that holds them.
constexpr int kFewRows = 32;

int few_limit(int group, int max_q_len)
{
    const long long rows = static_cast<long long>(group) * max_q_len;
    if (rows <= kFewRows) return static_cast<int>(rows);
    return group <= 8 ? 8 : group <= 16 ? 16 : group <= kFewRows ? kFewRows : 0;
}

}  // namespace

// The kernels' workspaces lie one after the other.
size_t kv4_attend_workspace(int n_heads, int n_kv, int head_dim, int max_q_len)
{
    const int group = n_heads / n_kv, few = few_limit(group, max_q_len);
    return kv4_few_workspace(head_dim, few) + (static_cast<long long>(group) * max_q_len > few ? kv4_many_workspace(head_dim) : 0);
}

cudaError_t launch_kv4_attend(const AttendArgs& a, cudaStream_t stream)
{
    if (a.batch.n_rows == 0 || a.batch.max_q_len == 0) return cudaSuccess;
    const int group = a.n_heads / a.cache.n_kv, few = few_limit(group, a.batch.max_q_len);
    if (static_cast<long long>(group) * a.batch.max_q_len > few) {
        void* ws = static_cast<uint8_t*>(a.ws) + kv4_few_workspace(a.cache.head_dim, few);
        const cudaError_t e = launch_kv4_many(a, few, ws, stream);
        if (e != cudaSuccess) return e;
    }
    return few ? launch_kv4_few(a, few, a.ws, stream) : cudaSuccess;
}

}  // namespace lora
