// Python binding of the AdamW lane's layers: checks torch tensors, allocates
// outputs and workspaces on the current stream, and calls the C entry points
// of include/muon.h.  Compiled code instead of ctypes, because the calls on a
// few tokens take a few microseconds on the GPU: a 16-row LayerNorm is issued
// in a third of the time that the same checks take in Python.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <tuple>

#include "../../../include/muon.h"

namespace {

using at::ScalarType;
using at::Tensor;
using std::optional;

// muon_error(code, message) of the package, for a status that the library returns
[[noreturn]] void raise_status(int rc) {
    py::object make = py::module_::import("matrix_orthogonalizing_optimizer_step_b200").attr("MuonError");
    py::object e = make(rc, py::str(muon_last_error()));
    PyErr_SetObject(make.ptr(), e.ptr());
    throw py::error_already_set();
}
void check(int rc) {
    if (rc != MUON_OK) raise_status(rc);
}

int dtype_code(ScalarType t, const char* name) {
    TORCH_CHECK_VALUE(t == at::kBFloat16 || t == at::kFloat, name, " must be bfloat16 or float32");
    return t == at::kFloat ? MUON_DTYPE_F32 : MUON_DTYPE_BF16;
}

int index_code(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kLong || t.scalar_type() == at::kInt, name, " must be int32 or int64");
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    return t.scalar_type() == at::kLong ? MUON_INDEX_I64 : MUON_INDEX_I32;
}

void check_device(const Tensor& first, const Tensor& other) {
    TORCH_CHECK_VALUE(other.device() == first.device(), "tensors must be on one device");
}
void check_cuda(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda(), "tensors must be CUDA tensors"); }

// t as rows of its last dimension
struct Rows {
    Tensor t;
    int64_t rows, dim, ld;
};
Rows rows_of(const Tensor& x, const char* name) {
    TORCH_CHECK_VALUE(x.dim() > 0, name, " must have at least one dimension");
    const int64_t dim = x.size(-1);
    TORCH_CHECK_VALUE(dim > 0, name, " must not have an empty last dimension");
    if (x.is_contiguous()) return {x, x.numel() / dim, dim, dim};
    Tensor t = x;
    if (x.dim() != 2) {
        try {
            t = x.view({-1, dim});
        } catch (const c10::Error&) {
            TORCH_CHECK_VALUE(false, name, " must be viewable as rows of one stride");
        }
    }
    const int64_t rows = t.size(0);
    TORCH_CHECK_VALUE((dim == 1 || t.stride(1) == 1) && (rows <= 1 || t.stride(0) >= dim), name,
                      " must have contiguous rows that do not overlap");
    return {t, rows, dim, rows > 1 ? t.stride(0) : dim};
}

void check_matrix(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.dim() == 2 && t.is_contiguous(), name, " must be a contiguous 2-D tensor");
    TORCH_CHECK_VALUE(t.numel() > 0, name, " must not be empty");
}

void check_vector(const Tensor& t, const char* name, int64_t n) {
    TORCH_CHECK_VALUE(t.numel() == n && t.is_contiguous(), name, " must be contiguous with ", n, " elements");
}
void check_fp32(const Tensor& t, const char* name, int64_t n) {
    check_vector(t, name, n);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat, name, " must be float32");
}

Tensor empty(at::IntArrayRef size, ScalarType t, const Tensor& like) {
    return at::detail::empty_cuda(size, t, like.device(), std::nullopt);
}

Tensor workspace(long long bytes, const Tensor& like) {
    if (bytes < 0) raise_status(static_cast<int>(bytes));
    return empty({bytes}, at::kByte, like);
}

const void* ptr(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
const void* ptr(const optional<Tensor>& t) { return t ? ptr(*t) : nullptr; }
void* out_ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The tensors' device current and its current stream bound, for one call.  A
// binding belongs to its thread: backward passes run on autograd's threads,
// beside whatever the program's own thread has enqueued or is enqueueing.
struct Call {
    c10::cuda::CUDAGuard guard;
    explicit Call(const Tensor& t) : guard(t.device()) {
        muon_set_stream(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
    }
};

std::vector<int64_t> with_last(at::IntArrayRef s, int64_t dim) {
    std::vector<int64_t> v(s.begin(), s.end());
    v.push_back(dim);
    return v;
}

Tensor embedding(const Tensor& tokens, const Tensor& table, double scale, optional<ScalarType> out_dtype) {
    check_matrix(table, "table");
    const int it = index_code(tokens, "tokens");
    const int td = dtype_code(table.scalar_type(), "table");
    const ScalarType ot = out_dtype.value_or(table.scalar_type());
    const int od = dtype_code(ot, "out_dtype");
    check_cuda(table);
    check_device(table, tokens);
    const int64_t n = tokens.numel(), dim = table.size(1);
    Tensor out = empty(with_last(tokens.sizes(), dim), ot, table);
    if (n == 0) return out;
    Call call(table);
    check(muon_embedding(ptr(tokens), it, n, ptr(table), td, table.size(0), dim, static_cast<float>(scale),
                         out.data_ptr(), od));
    return out;
}

Tensor embedding_backward(const Tensor& tokens, const Tensor& grad_out, int64_t num_embeddings, double scale,
                          optional<int64_t> padding_idx, optional<ScalarType> grad_dtype, optional<Tensor> out) {
    const int it = index_code(tokens, "tokens");
    const int gd = dtype_code(grad_out.scalar_type(), "grad_out");
    const Rows g = rows_of(grad_out, "grad_out");
    const int64_t n = tokens.numel();
    TORCH_CHECK_VALUE(g.rows == n, "grad_out must have one row per token");
    TORCH_CHECK_VALUE(num_embeddings >= 1, "num_embeddings must be >= 1");
    TORCH_CHECK_VALUE(!padding_idx || (*padding_idx >= 0 && *padding_idx < num_embeddings),
                      "padding_idx must be a token");
    const ScalarType ot = grad_dtype.value_or(out ? out->scalar_type() : grad_out.scalar_type());
    const int od = dtype_code(ot, "grad_dtype");
    if (out) {
        check_matrix(*out, "out");
        TORCH_CHECK_VALUE(out->size(0) == num_embeddings && out->size(1) == g.dim && out->scalar_type() == ot,
                          "out must have shape (num_embeddings, dim) and grad_dtype");
    }
    check_cuda(grad_out);
    check_device(grad_out, tokens);
    if (out) check_device(grad_out, *out);
    Tensor r = out ? *out : empty({num_embeddings, g.dim}, ot, grad_out);
    const Tensor ws = workspace(muon_embedding_backward_workspace(n, num_embeddings, g.dim), grad_out);
    Call call(grad_out);
    check(muon_embedding_backward(ptr(tokens), it, n, ptr(g.t), gd, g.ld, num_embeddings, g.dim,
                                  static_cast<float>(scale), padding_idx.value_or(-1), r.data_ptr(), od, ws.data_ptr(),
                                  ws.numel()));
    return r;
}

// type code of weight and bias
int norm_params(const Tensor& x, int64_t dim, const optional<Tensor>& weight, const optional<Tensor>& bias) {
    if (weight) {
        check_vector(*weight, "weight", dim);
        check_device(x, *weight);
    }
    if (bias) {
        check_vector(*bias, "bias", dim);
        check_device(x, *bias);
        TORCH_CHECK_VALUE(!weight || weight->scalar_type() == bias->scalar_type(),
                          "weight and bias must have one dtype");
    }
    return weight ? dtype_code(weight->scalar_type(), "weight and bias")
                  : (bias ? dtype_code(bias->scalar_type(), "weight and bias") : MUON_DTYPE_F32);
}

std::tuple<Tensor, Tensor, Tensor> layer_norm(const Tensor& x, const optional<Tensor>& weight,
                                              const optional<Tensor>& bias, double eps) {
    const int xd = dtype_code(x.scalar_type(), "x");
    const Rows r = rows_of(x, "x");
    const int pd = norm_params(x, r.dim, weight, bias);
    check_cuda(x);
    Tensor y = empty(x.sizes(), x.scalar_type(), x);
    const at::IntArrayRef outer = x.sizes().slice(0, x.dim() - 1);
    Tensor mean = empty(outer, at::kFloat, x), rstd = empty(outer, at::kFloat, x);
    if (r.rows > 0) {
        Call call(x);
        check(muon_layer_norm(ptr(r.t), xd, r.ld, r.rows, r.dim, ptr(weight), ptr(bias), pd, static_cast<float>(eps),
                              y.data_ptr(), mean.data_ptr<float>(), rstd.data_ptr<float>()));
    }
    return {y, mean, rstd};
}

std::tuple<Tensor, optional<Tensor>, optional<Tensor>> layer_norm_backward(
    const Tensor& grad_out, const Tensor& x, const Tensor& mean, const Tensor& rstd, const optional<Tensor>& weight,
    bool bias, optional<ScalarType> param_dtype, bool weight_grad) {
    const int xd = dtype_code(x.scalar_type(), "x");
    TORCH_CHECK_VALUE(grad_out.sizes() == x.sizes() && grad_out.scalar_type() == x.scalar_type(),
                      "grad_out must have x's shape and dtype");
    const Rows r = rows_of(x, "x"), g = rows_of(grad_out, "grad_out");
    check_fp32(mean, "mean", r.rows);
    check_fp32(rstd, "rstd", r.rows);
    int pd = norm_params(x, r.dim, weight, std::nullopt);
    check_cuda(x);
    check_device(x, grad_out);
    check_device(x, mean);
    check_device(x, rstd);
    ScalarType pt = param_dtype.value_or(weight ? weight->scalar_type() : at::kFloat);
    TORCH_CHECK_VALUE(!weight || pt == weight->scalar_type(), "param_dtype must be the weight's dtype");
    pd = dtype_code(pt, "param_dtype");
    Tensor dx = empty(x.sizes(), x.scalar_type(), x);
    optional<Tensor> dw, db;
    if (weight && weight_grad) dw = empty(weight->sizes(), pt, x);
    if (bias) db = empty({r.dim}, pt, x);
    const Tensor ws = workspace(muon_layer_norm_backward_workspace(r.rows, r.dim), x);
    Call call(x);
    check(muon_layer_norm_backward(ptr(g.t), g.ld, ptr(r.t), xd, r.ld, r.rows, r.dim, mean.const_data_ptr<float>(),
                                   rstd.const_data_ptr<float>(), ptr(weight), pd, dx.data_ptr(),
                                   dw ? dw->data_ptr() : nullptr, db ? db->data_ptr() : nullptr, out_ptr(ws),
                                   ws.numel()));
    return {dx, dw, db};
}

struct Head {
    Rows h;
    int targets;
};
Head head_args(const Tensor& hidden, const Tensor& weight, const Tensor& targets) {
    check_matrix(weight, "weight");
    TORCH_CHECK_VALUE(hidden.scalar_type() == at::kBFloat16 && weight.scalar_type() == at::kBFloat16,
                      "hidden and weight must be bfloat16");
    const int it = index_code(targets, "targets");
    Rows h = rows_of(hidden, "hidden");
    TORCH_CHECK_VALUE(h.dim == weight.size(1), "hidden and weight must have one width");
    TORCH_CHECK_VALUE(h.dim % 8 == 0 && h.ld % 8 == 0,
                      "the width and hidden's row stride must be multiples of 8");
    TORCH_CHECK_VALUE(targets.numel() == h.rows, "targets must have one entry per row of hidden");
    check_cuda(weight);
    check_device(weight, hidden);
    check_device(weight, targets);
    TORCH_CHECK_VALUE(reinterpret_cast<uintptr_t>(ptr(h.t)) % 16 == 0 && reinterpret_cast<uintptr_t>(ptr(weight)) % 16 == 0,
                      "hidden and weight must be 16-byte aligned");
    return {h, it};
}

std::tuple<Tensor, Tensor> head_loss(const Tensor& hidden, const Tensor& weight, const Tensor& targets,
                                     int64_t ignore_index) {
    const Head a = head_args(hidden, weight, targets);
    Tensor loss = empty(targets.sizes(), at::kFloat, weight), lse = empty(targets.sizes(), at::kFloat, weight);
    if (a.h.rows == 0) return {loss, lse};
    const Tensor ws = workspace(muon_head_loss_workspace(a.h.rows, weight.size(0), a.h.dim, 0), weight);
    Call call(weight);
    check(muon_head_loss(ptr(a.h.t), a.h.ld, ptr(weight), ptr(targets), a.targets, a.h.rows, weight.size(0), a.h.dim,
                         ignore_index, loss.data_ptr<float>(), lse.data_ptr<float>(), ws.data_ptr(), ws.numel()));
    return {loss, lse};
}

std::tuple<optional<Tensor>, optional<Tensor>> head_loss_backward(const Tensor& hidden, const Tensor& weight,
                                                                  const Tensor& targets, const Tensor& lse,
                                                                  const Tensor& grad_loss, int64_t ignore_index,
                                                                  bool hidden_grad, bool weight_grad) {
    const Head a = head_args(hidden, weight, targets);
    check_fp32(lse, "lse", a.h.rows);
    check_fp32(grad_loss, "grad_loss", a.h.rows);
    check_device(weight, lse);
    check_device(weight, grad_loss);
    TORCH_CHECK_VALUE(hidden_grad || weight_grad, "one gradient at least");
    optional<Tensor> dh, dw;
    if (hidden_grad) dh = empty(hidden.sizes(), at::kBFloat16, weight);
    if (weight_grad) dw = empty(weight.sizes(), at::kBFloat16, weight);
    if (a.h.rows == 0 && !weight_grad) return {dh, dw};
    const Tensor ws = workspace(muon_head_loss_workspace(a.h.rows, weight.size(0), a.h.dim, 1), weight);
    Call call(weight);
    check(muon_head_loss_backward(ptr(a.h.t), a.h.ld, ptr(weight), ptr(targets), a.targets, a.h.rows, weight.size(0),
                                  a.h.dim, ignore_index, lse.const_data_ptr<float>(),
                                  grad_loss.const_data_ptr<float>(), dh ? dh->data_ptr() : nullptr,
                                  dw ? dw->data_ptr() : nullptr, out_ptr(ws), ws.numel()));
    return {dh, dw};
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    using namespace py::literals;
    m.doc() =
        "The AdamW lane's layers: token embedding, LayerNorm and output head with its loss, and the gradients that "
        "the lane's step reads.  Outputs and workspaces are torch allocations on the current stream, so the calls can "
        "be captured into a CUDA graph (each graph then has workspaces of its own) and several streams may use them "
        "at once.  All tensors of a call must be on one device, which need not be the current one; tensors made on "
        "another stream need that stream's work ordered before the call, as for any torch operator.";
    m.def("muon_embedding", &embedding, "tokens"_a, "table"_a, "scale"_a = 1.0, "out_dtype"_a = py::none(),
          "scale * table[tokens]: tokens int32 or int64 of any shape, table (vocab, dim) bf16 or fp32; the result has "
          "tokens' shape with dim appended, in out_dtype (default: the table's).  Rows of tokens outside the "
          "vocabulary are NaN (muon_device_status reports them).");
    m.def("muon_embedding_backward", &embedding_backward, "tokens"_a, "grad_out"_a, "num_embeddings"_a,
          "scale"_a = 1.0, "padding_idx"_a = py::none(), "grad_dtype"_a = py::none(), "out"_a = py::none(),
          "Gradient of the table of muon_embedding: (num_embeddings, dim) in grad_dtype (default: grad_out's), dense, "
          "rows of unused tokens and of padding_idx zero.  grad_out: tokens.numel() rows.  out: the contiguous tensor "
          "to write instead of a new one.");
    m.def("muon_layer_norm", &layer_norm, "x"_a, "weight"_a = py::none(), "bias"_a = py::none(), "eps"_a = 1e-5,
          "LayerNorm over x's last dimension: (y, mean, rstd).  x bf16 or fp32 with contiguous rows; weight and bias "
          "bf16 or fp32.  y is contiguous in x's dtype; mean and rstd are fp32, one per row, for the backward pass.");
    m.def("muon_layer_norm_backward", &layer_norm_backward, "grad_out"_a, "x"_a, "mean"_a, "rstd"_a,
          "weight"_a = py::none(), "bias"_a = true, "param_dtype"_a = py::none(), "weight_grad"_a = true,
          "Gradients of muon_layer_norm: (dx, dweight, dbias) in x's dtype and in the weight's (without a weight: "
          "param_dtype, default fp32).  dweight is None without a weight or with weight_grad=False, dbias None with "
          "bias=False.");
    m.def("muon_head_loss", &head_loss, "hidden"_a, "weight"_a, "targets"_a, "ignore_index"_a = -100,
          "(loss, lse) per token of the softmax cross entropy of hidden . weight^T: hidden (..., dim) and weight "
          "(vocab, dim) bf16 with dim a multiple of 8, targets int32 or int64.  Both results are fp32 in targets' "
          "shape, 0 for tokens whose target is ignore_index; the logits are not kept.");
    m.def("muon_head_loss_backward", &head_loss_backward, "hidden"_a, "weight"_a, "targets"_a, "lse"_a, "grad_loss"_a,
          "ignore_index"_a = -100, "hidden_grad"_a = true, "weight_grad"_a = true,
          "(dhidden, dweight), bf16, from the lse of muon_head_loss and the fp32 gradient of its per-token loss.  "
          "Either can be left out (None).");
}
