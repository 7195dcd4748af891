// Internal launch interface of the AdamW lane's layers: the token embedding
// (embedding.cu), LayerNorm (layer_norm.cu) and the output head with its
// loss (head_loss.cu).  The C entry points are in lane_abi.cpp.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "muon_internal.h"

namespace muon {

// ---- shared with muon_abi.cpp ---------------------------------------------------

int abi_fail(int code, const char* msg);
// Status word, SM count and compute capability of the current device.  The
// first call on a device allocates, so it is refused under stream capture.
int abi_device(DeviceStatus** status, int* num_sms, int* cc_major);
void abi_count_launches(long long n);

// Bound of every device-side wait (MUON_WAIT_LIMIT_MS), in nanoseconds.
unsigned long long wait_limit_ns();

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// ---- token embedding --------------------------------------------------------------

struct EmbedFwd {
    const void* tokens;
    int tokens_i64;      // 1: int64 token ids, 0: int32
    long long count;     // tokens
    const void* table;   // vocab x dim, row-major
    int table_dt;
    long long vocab, dim;
    float scale;
    void* out;           // count x dim
    int out_dt;
    DeviceStatus* status;
};
cudaError_t launch_embedding(const EmbedFwd& L, cudaStream_t stream);

struct EmbedBwd {
    const void* tokens;
    int tokens_i64;
    long long count;
    const void* grad;    // count rows of dim elements, row stride ld
    int grad_dt;
    long long ld;
    long long vocab, dim;
    long long padding;   // token whose gradient row is zero, or -1
    float scale;
    void* out;           // vocab x dim
    int out_dt;
    void* workspace;
    DeviceStatus* status;
};
size_t embedding_backward_workspace(long long count, long long dim);
cudaError_t launch_embedding_backward(const EmbedBwd& L, int num_sms, cudaStream_t stream, int* launches);

// ---- LayerNorm --------------------------------------------------------------------

struct NormFwd {
    const void* x;       // rows of dim elements, row stride ldx
    int x_dt;
    long long ldx, rows, dim;
    const void* w;       // dim, or null
    const void* b;       // dim, or null
    int p_dt;            // dtype of w and b
    float eps;
    void* y;             // rows x dim, x_dt
    float* mean;
    float* rstd;
};
cudaError_t launch_layer_norm(const NormFwd& L, int num_sms, cudaStream_t stream);

struct NormBwd {
    const void* dy;      // row stride ldy
    const void* x;       // row stride ldx
    int x_dt;            // dtype of dy, x and dx
    long long ldy, ldx, rows, dim;
    const float* mean;
    const float* rstd;
    const void* w;       // or null
    int p_dt;            // dtype of w, dw and db
    void* dx;            // rows x dim
    void* dw;            // dim, or null
    void* db;            // dim, or null
    void* workspace;
};
size_t layer_norm_backward_workspace(long long rows, long long dim, int num_sms);
cudaError_t launch_layer_norm_backward(const NormBwd& L, int num_sms, cudaStream_t stream, int* launches);

// ---- output head and loss ---------------------------------------------------------

struct HeadLoss {
    const void* hidden;  // tokens rows of dim bf16, row stride ldh
    long long ldh;
    const void* weight;  // vocab x dim bf16
    const void* targets;
    int targets_i64;
    long long tokens, vocab, dim;
    long long ignore;    // targets of this value take no part
    float* loss;         // forward: tokens
    float* lse;          // forward: written; backward: read
    const float* dloss;  // backward: tokens
    void* dhidden;       // backward: tokens x dim bf16, or null
    void* dweight;       // backward: vocab x dim bf16, or null
    void* workspace;
    DeviceStatus* status;
    unsigned long long wait_ns;
};
size_t head_loss_workspace(long long tokens, long long vocab, long long dim, int backward);
// cudaErrorInvalidValue with *why set when a tensor map cannot be encoded
cudaError_t launch_head_loss(const HeadLoss& L, cudaStream_t stream, int* launches, const char** why);
cudaError_t launch_head_loss_backward(const HeadLoss& L, cudaStream_t stream, int* launches, const char** why);

}  // namespace muon
