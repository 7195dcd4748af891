// C entry points of the AdamW lane's layers (include/muon.h): argument checks
// and launches.  Every argument that the host can see is checked before
// anything is enqueued; token ids and targets are checked by the kernels.
// The calls keep no state of their own: their scratch is the caller's
// workspace, and tensor maps travel as kernel arguments, so a call can be
// captured and replayed, and calls with workspaces of their own may overlap.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdint>

#include "../../include/muon.h"
#include "lane.h"
#include "launch.h"

using namespace muon;

namespace {

constexpr long long kMaxCount = 0x7fffffff - 1024;  // tokens, rows and vocabulary are 32-bit in the kernels
constexpr long long kMaxDim = 1 << 20;
constexpr long long kMaxGrid = 0x7fffffff;

bool dtype_ok(int dt) { return dt == MUON_DTYPE_BF16 || dt == MUON_DTYPE_F32; }
bool index_ok(int dt) { return dt == MUON_INDEX_I32 || dt == MUON_INDEX_I64; }
int kernel_dtype(int dt) { return dt == MUON_DTYPE_F32 ? DT_F32 : DT_BF16; }
bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int invalid(const char* msg) { return abi_fail(MUON_ERR_INVALID_ARG, msg); }
int elem_size(int dt) { return dt == MUON_DTYPE_F32 ? 4 : 2; }
int index_size(int dt) { return dt == MUON_INDEX_I64 ? 8 : 4; }

// The launch's outcome as a status.
int launched(cudaError_t e, int launches, const char* why = nullptr) {
    abi_count_launches(launches);
    if (e == cudaSuccess) return MUON_OK;
    cudaGetLastError();
    return abi_fail(MUON_ERR_CUDA, why ? why : cudaGetErrorString(e));
}

struct Device {
    DeviceStatus* status = nullptr;
    int num_sms = 0, cc_major = 0;
};

int tokens_check(const void* tokens, int token_dtype, long long count, long long vocab, long long dim) {
    if (count < 0 || count > kMaxCount) return invalid("count must be 0 .. 2^31 - 1025");
    if (vocab < 1 || vocab > kMaxCount) return invalid("vocab must be 1 .. 2^31 - 1025");
    if (dim < 1 || dim > kMaxDim) return invalid("dim must be 1 .. 2^20");
    if (!index_ok(token_dtype))
        return abi_fail(MUON_ERR_UNSUPPORTED, "tokens must be MUON_INDEX_I32 or MUON_INDEX_I64");
    if (count > 0 && !tokens) return invalid("tokens must not be NULL");
    if (count > 0 && !aligned(tokens, index_size(token_dtype))) return invalid("tokens must be aligned to their type");
    return MUON_OK;
}

int head_check(const void* hidden, long long ld_hidden, const void* weight, const void* targets, int target_dtype,
               long long tokens, long long vocab, long long dim) {
    const int st = tokens_check(targets, target_dtype, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    if (dim % 8 != 0) return abi_fail(MUON_ERR_UNSUPPORTED, "dim must be a multiple of 8");
    if (!weight || !aligned(weight, 16)) return invalid("weight must be 16-byte aligned and not NULL");
    if (tokens > 0 && (!hidden || !aligned(hidden, 16))) return invalid("hidden must be 16-byte aligned and not NULL");
    if (ld_hidden < dim || ld_hidden % 8 != 0) return invalid("ld_hidden must be >= dim and a multiple of 8");
    if ((tokens + 255) / 256 * ((vocab + 255) / 256) > kMaxGrid) return invalid("tokens x vocab too large for one call");
    return MUON_OK;
}

HeadLoss head_args(const void* hidden, long long ld_hidden, const void* weight, const void* targets, int target_dtype,
                   long long tokens, long long vocab, long long dim, long long ignore_index, void* workspace,
                   const Device& dev) {
    HeadLoss L{};
    L.hidden = hidden;
    L.ldh = ld_hidden;
    L.weight = weight;
    L.targets = targets;
    L.targets_i64 = target_dtype == MUON_INDEX_I64;
    L.tokens = tokens;
    L.vocab = vocab;
    L.dim = dim;
    L.ignore = ignore_index;
    L.workspace = workspace;
    L.status = dev.status;
    L.wait_ns = wait_limit_ns();
    return L;
}

int workspace_check(const void* workspace, long long have, size_t need) {
    if (need == 0) return MUON_OK;
    if (!workspace || !aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned and not NULL");
    if (have < 0 || static_cast<size_t>(have) < need) return invalid("workspace too small");
    return MUON_OK;
}

// NVTX range of one call
struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

extern "C" {

int muon_embedding(const void* tokens, int token_dtype, long long count, const void* table, int table_dtype,
                   long long vocab, long long dim, float scale, void* out, int out_dtype) {
    int st = tokens_check(tokens, token_dtype, count, vocab, dim);
    if (st != MUON_OK) return st;
    if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype))
        return abi_fail(MUON_ERR_UNSUPPORTED, "table and out must be MUON_DTYPE_BF16 or MUON_DTYPE_F32");
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    if (count == 0) return MUON_OK;
    if (!table || !out) return invalid("table and out must not be NULL");
    if (!aligned(table, elem_size(table_dtype)) || !aligned(out, elem_size(out_dtype)))
        return invalid("table and out must be aligned to their type");
    if ((count + 3) / 4 * ((dim + 1023) / 1024) >= kMaxGrid) return invalid("count x dim too large for one call");
    Device dev;
    st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    EmbedFwd L{};
    L.tokens = tokens;
    L.tokens_i64 = token_dtype == MUON_INDEX_I64;
    L.count = count;
    L.table = table;
    L.table_dt = kernel_dtype(table_dtype);
    L.vocab = vocab;
    L.dim = dim;
    L.scale = scale;
    L.out = out;
    L.out_dt = kernel_dtype(out_dtype);
    L.status = dev.status;
    Range r("muon embedding");
    return launched(launch_embedding(L, bound_stream()), 1);
}

long long muon_embedding_backward_workspace(long long count, long long vocab, long long dim) {
    if (count < 0 || count > kMaxCount || vocab < 1 || vocab > kMaxCount || dim < 1 || dim > kMaxDim)
        return invalid("count, vocab or dim out of range");
    return static_cast<long long>(embedding_backward_workspace(count, dim));
}

int muon_embedding_backward(const void* tokens, int token_dtype, long long count, const void* grad_out, int grad_dtype,
                            long long ld_grad, long long vocab, long long dim, float scale, long long padding_token,
                            void* dtable, int dtable_dtype, void* workspace, long long workspace_bytes) {
    int st = tokens_check(tokens, token_dtype, count, vocab, dim);
    if (st != MUON_OK) return st;
    if (!dtype_ok(grad_dtype) || !dtype_ok(dtable_dtype))
        return abi_fail(MUON_ERR_UNSUPPORTED, "grad_out and dtable must be MUON_DTYPE_BF16 or MUON_DTYPE_F32");
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    if (padding_token < -1 || padding_token >= vocab) return invalid("padding_token must be -1 (none) or a token");
    if (!dtable || !aligned(dtable, elem_size(dtable_dtype)))
        return invalid("dtable must be aligned to its type and not NULL");
    if (count > 0 && (!grad_out || !aligned(grad_out, elem_size(grad_dtype))))
        return invalid("grad_out must be aligned to its type and not NULL");
    if (ld_grad < dim) return invalid("ld_grad must be >= dim");
    if ((count + 63) / 64 * ((dim + 255) / 256) >= kMaxGrid) return invalid("count x dim too large for one call");
    st = workspace_check(workspace, workspace_bytes, embedding_backward_workspace(count, dim));
    if (st != MUON_OK) return st;
    Device dev;
    st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    EmbedBwd L{};
    L.tokens = tokens;
    L.tokens_i64 = token_dtype == MUON_INDEX_I64;
    L.count = count;
    L.grad = grad_out;
    L.grad_dt = kernel_dtype(grad_dtype);
    L.ld = ld_grad;
    L.vocab = vocab;
    L.dim = dim;
    L.padding = padding_token;
    L.scale = scale;
    L.out = dtable;
    L.out_dt = kernel_dtype(dtable_dtype);
    L.workspace = workspace;
    L.status = dev.status;
    Range r("muon embedding backward");
    int n = 0;
    const cudaError_t e = launch_embedding_backward(L, dev.num_sms, bound_stream(), &n);
    return launched(e, n);
}

int muon_layer_norm(const void* x, int x_dtype, long long ld_x, long long rows, long long dim, const void* weight,
                    const void* bias, int param_dtype, float eps, void* y, float* mean, float* rstd) {
    if (rows < 0 || rows > kMaxCount) return invalid("rows must be 0 .. 2^31 - 1025");
    if (dim < 1 || dim > kMaxDim) return invalid("dim must be 1 .. 2^20");
    if (!dtype_ok(x_dtype) || !dtype_ok(param_dtype))
        return abi_fail(MUON_ERR_UNSUPPORTED, "x and the parameters must be MUON_DTYPE_BF16 or MUON_DTYPE_F32");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return invalid("eps must be finite and >= 0");
    if (ld_x < dim) return invalid("ld_x must be >= dim");
    if (rows == 0) return MUON_OK;
    if (!x || !y || !mean || !rstd) return invalid("x, y, mean and rstd must not be NULL");
    if (!aligned(x, elem_size(x_dtype)) || !aligned(y, elem_size(x_dtype)) || !aligned(weight, elem_size(param_dtype)) ||
        !aligned(bias, elem_size(param_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
        return invalid("every tensor must be aligned to its type");
    Device dev;
    const int st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    NormFwd L{};
    L.x = x;
    L.x_dt = kernel_dtype(x_dtype);
    L.ldx = ld_x;
    L.rows = rows;
    L.dim = dim;
    L.w = weight;
    L.b = bias;
    L.p_dt = kernel_dtype(param_dtype);
    L.eps = eps;
    L.y = y;
    L.mean = mean;
    L.rstd = rstd;
    Range r("muon layer norm");
    return launched(launch_layer_norm(L, dev.num_sms, bound_stream()), 1);
}

long long muon_layer_norm_backward_workspace(long long rows, long long dim) {
    if (rows < 0 || rows > kMaxCount || dim < 1 || dim > kMaxDim) return invalid("rows or dim out of range");
    // the partial rows of the largest device the library knows: the count
    // follows the SM count, so a caller without a device can ask
    return static_cast<long long>(layer_norm_backward_workspace(rows, dim, 148));
}

int muon_layer_norm_backward(const void* grad_out, long long ld_grad, const void* x, int x_dtype, long long ld_x,
                             long long rows, long long dim, const float* mean, const float* rstd, const void* weight,
                             int param_dtype, void* dx, void* dweight, void* dbias, void* workspace,
                             long long workspace_bytes) {
    if (rows < 0 || rows > kMaxCount) return invalid("rows must be 0 .. 2^31 - 1025");
    if (dim < 1 || dim > kMaxDim) return invalid("dim must be 1 .. 2^20");
    if (!dtype_ok(x_dtype) || !dtype_ok(param_dtype))
        return abi_fail(MUON_ERR_UNSUPPORTED, "x and the parameters must be MUON_DTYPE_BF16 or MUON_DTYPE_F32");
    if (ld_x < dim || ld_grad < dim) return invalid("ld_x and ld_grad must be >= dim");
    if (rows > 0 && (!grad_out || !x || !mean || !rstd || !dx))
        return invalid("grad_out, x, mean, rstd and dx must not be NULL");
    if (!aligned(x, elem_size(x_dtype)) || !aligned(grad_out, elem_size(x_dtype)) || !aligned(dx, elem_size(x_dtype)) ||
        !aligned(weight, elem_size(param_dtype)) || !aligned(dweight, elem_size(param_dtype)) ||
        !aligned(dbias, elem_size(param_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4))
        return invalid("every tensor must be aligned to its type");
    int st = workspace_check(workspace, workspace_bytes, layer_norm_backward_workspace(rows, dim, 148));
    if (st != MUON_OK) return st;
    Device dev;
    st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    NormBwd L{};
    L.dy = grad_out;
    L.x = x;
    L.x_dt = kernel_dtype(x_dtype);
    L.ldy = ld_grad;
    L.ldx = ld_x;
    L.rows = rows;
    L.dim = dim;
    L.mean = mean;
    L.rstd = rstd;
    L.w = weight;
    L.p_dt = kernel_dtype(param_dtype);
    L.dx = dx;
    L.dw = dweight;
    L.db = dbias;
    L.workspace = workspace;
    Range r("muon layer norm backward");
    int n = 0;
    const cudaError_t e = launch_layer_norm_backward(L, dev.num_sms < 148 ? dev.num_sms : 148, bound_stream(), &n);
    return launched(e, n);
}

long long muon_head_loss_workspace(long long tokens, long long vocab, long long dim, int backward) {
    if (tokens < 0 || tokens > kMaxCount || vocab < 1 || vocab > kMaxCount || dim < 1 || dim > kMaxDim)
        return invalid("tokens, vocab or dim out of range");
    return tokens == 0 ? 0 : static_cast<long long>(head_loss_workspace(tokens, vocab, dim, backward));
}

int muon_head_loss(const void* hidden, long long ld_hidden, const void* weight, const void* targets, int target_dtype,
                   long long tokens, long long vocab, long long dim, long long ignore_index, float* loss, float* lse,
                   void* workspace, long long workspace_bytes) {
    int st = head_check(hidden, ld_hidden, weight, targets, target_dtype, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    if (tokens == 0) return MUON_OK;
    if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)) return invalid("loss and lse must not be NULL");
    st = workspace_check(workspace, workspace_bytes, head_loss_workspace(tokens, vocab, dim, 0));
    if (st != MUON_OK) return st;
    Device dev;
    st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    if (dev.cc_major != 10) return abi_fail(MUON_ERR_UNSUPPORTED, "the tensor-core path needs an sm_100 GPU (B200)");
    HeadLoss L = head_args(hidden, ld_hidden, weight, targets, target_dtype, tokens, vocab, dim, ignore_index, workspace,
                           dev);
    L.loss = loss;
    L.lse = lse;
    Range r("muon head loss");
    int n = 0;
    const char* why = nullptr;
    const cudaError_t e = launch_head_loss(L, bound_stream(), &n, &why);
    return launched(e, n, why);
}

int muon_head_loss_backward(const void* hidden, long long ld_hidden, const void* weight, const void* targets,
                            int target_dtype, long long tokens, long long vocab, long long dim, long long ignore_index,
                            const float* lse, const float* dloss, void* dhidden, void* dweight, void* workspace,
                            long long workspace_bytes) {
    int st = head_check(hidden, ld_hidden, weight, targets, target_dtype, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    if (!dhidden && !dweight) return invalid("dhidden and dweight must not both be NULL");
    if (!aligned(dhidden, 16) || !aligned(dweight, 16)) return invalid("dhidden and dweight must be 16-byte aligned");
    if (tokens > 0 && (!lse || !dloss || !aligned(lse, 4) || !aligned(dloss, 4)))
        return invalid("lse and dloss must not be NULL");
    st = workspace_check(workspace, workspace_bytes, tokens ? head_loss_workspace(tokens, vocab, dim, 1) : 0);
    if (st != MUON_OK) return st;
    Device dev;
    st = abi_device(&dev.status, &dev.num_sms, &dev.cc_major);
    if (st != MUON_OK) return st;
    if (dev.cc_major != 10) return abi_fail(MUON_ERR_UNSUPPORTED, "the tensor-core path needs an sm_100 GPU (B200)");
    Range r("muon head loss backward");
    if (tokens == 0 && !dweight) return MUON_OK;
    if (tokens == 0)  // no token, no gradient
        return launched(cudaMemsetAsync(dweight, 0, static_cast<size_t>(vocab) * dim * 2, bound_stream()), 0);
    HeadLoss L = head_args(hidden, ld_hidden, weight, targets, target_dtype, tokens, vocab, dim, ignore_index, workspace,
                           dev);
    L.lse = const_cast<float*>(lse);
    L.dloss = dloss;
    L.dhidden = dhidden;
    L.dweight = dweight;
    int n = 0;
    const char* why = nullptr;
    const cudaError_t e = launch_head_loss_backward(L, bound_stream(), &n, &why);
    return launched(e, n, why);
}

}  // extern "C"
