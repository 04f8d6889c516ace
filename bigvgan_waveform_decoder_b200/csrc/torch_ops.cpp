// torch_ops.cpp -- the operators over channels-last frames for torch tensors: argument checks and
// allocation around the C ABI of include/mh3a.h, nothing else.  It is compiled code because the
// smallest calls take 3 to 4 us on the GPU: the same marshalling in Python took 19 us a call.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/extension.h>

#include <algorithm>

#include "mh3a.h"

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

// Becomes the package's MH3AError(status, what, detail).
struct Error {
    int status;
    const char* what;
    std::string detail;
};

void require(bool ok, const char* what, const char* detail, int status = MH3A_ERR_INVALID_ARG) {
    if (!ok) throw Error{status, what, detail};
}

template <typename... A>
[[noreturn]] void refuse(const char* what, int status, A&&... detail) {
    throw Error{status, what, c10::str(std::forward<A>(detail)...)};
}

void check(mh3a_status st, const char* what) {
    if (st != MH3A_OK) throw Error{st, what, st == MH3A_ERR_CUDA ? mh3a_last_error() : ""};
}

// The device and stream of a call: torch allocates on that stream while it lives.  Tensors that cross
// between it and the caller's stream are recorded, so that the allocator keeps them until both are done.
class Launch {
  public:
    Launch(const c10::Device& device, const std::optional<int64_t>& stream)
        : device_(device), current_(c10::cuda::getCurrentCUDAStream(device.index())), stream_(current_) {
        if (stream && reinterpret_cast<cudaStream_t>(*stream) != current_.stream()) {
            stream_ = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*stream), device.index());
            guard_.emplace(stream_);
            side_ = true;
        }
    }
    void* stream() const { return stream_.stream(); }
    void inputs(std::initializer_list<const Tensor*> ts) const {
        if (side_)
            for (const Tensor* t : ts)
                if (t) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), stream_);
    }
    void outputs(std::initializer_list<const Tensor*> ts) const {
        if (side_)
            for (const Tensor* t : ts)
                if (t->defined()) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), current_);
    }

  private:
    c10::cuda::CUDAGuard device_;
    c10::cuda::CUDAStream current_, stream_;
    std::optional<c10::cuda::CUDAStreamGuard> guard_;
    bool side_ = false;
};

const Tensor* opt(const Opt& t) { return t ? &*t : nullptr; }

// The calls record no gradient.  Where autograd is recording and an input requires one, the results lead
// back to a node that raises, so that none is lost without a word; as for torch's own operators, `out` is
// refused then.
class NoGradient {
  public:
    NoGradient(const char* what, const char* instead, const Tensor* out, std::initializer_list<const Tensor*> inputs) {
        if (!at::GradMode::is_enabled()) return;
        torch::autograd::edge_list edges;
        for (const Tensor* t : inputs)
            if (t && t->requires_grad()) edges.push_back(torch::autograd::impl::gradient_edge(*t));
        if (edges.empty() && !(out && out->requires_grad())) return;
        if (out) refuse(what, MH3A_ERR_INVALID_ARG, "out cannot be given where an input or out requires a gradient");
        node_ = std::shared_ptr<torch::autograd::Node>(
            new torch::autograd::Error(c10::str(what, " records no gradient: ", instead, ", or detach its inputs"), std::move(edges)),
            torch::autograd::deleteNode);
    }
    void from(std::initializer_list<const Tensor*> results) const {
        if (node_)
            for (const Tensor* t : results) torch::autograd::set_history(*t, node_);
    }

  private:
    std::shared_ptr<torch::autograd::Node> node_;
};

int dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return MH3A_DTYPE_F32;
        case at::kHalf: return MH3A_DTYPE_F16;
        case at::kBFloat16: return MH3A_DTYPE_BF16;
        default: return -1;
    }
}

Tensor empty(at::IntArrayRef size, at::ScalarType type, const c10::Device& device) {
    return Tensor(at::detail::empty_cuda(size, type, device, std::nullopt));
}

// A contiguous tensor of a type and shape on the call's device.
void check_plain(const char* what, const char* name, const Tensor& t, const c10::Device& device, at::ScalarType type,
                 at::IntArrayRef shape) {
    if (t.device() != device || t.scalar_type() != type || !t.is_contiguous())
        refuse(what, MH3A_ERR_INVALID_ARG, name, " is not a contiguous ", type, " tensor on ", device);
    if (t.sizes() != shape) refuse(what, MH3A_ERR_SHAPE, name, " is ", t.sizes(), ": ", shape, " is wanted");
}

// The stride of a dimension of one element says nothing.
int64_t stride_of(const Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

// Whether a tensor starts on a 16-byte boundary with strides of whole 16 bytes (but the last).
bool aligned16(const Tensor& t) {
    if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16) return false;
    const int64_t per = 16 / t.element_size();
    for (int64_t i = 0; i + 1 < t.dim(); ++i)
        if (stride_of(t, i) % per) return false;
    return true;
}
bool aligned16(const Opt& t) { return !t || aligned16(*t); }

template <typename T>
T* data(const Opt& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// The bytes of a tensor whose last dimension is adjacent: `items` x `rows` runs of `run` bytes from `at` on.
struct Bytes {
    int64_t at, run, row, rows, item, items;

    explicit Bytes(const Tensor& t) {
        const int64_t e = t.element_size(), d = t.dim();
        at = reinterpret_cast<intptr_t>(t.data_ptr());
        run = t.size(d - 1) * e;
        rows = d > 1 ? t.size(d - 2) : 1;
        row = d > 1 ? stride_of(t, d - 2) * e : 0;
        items = d > 2 ? t.size(d - 3) : 1;
        item = d > 2 ? stride_of(t, d - 3) * e : 0;
        if (rows == 1) {  // the items are the rows
            rows = items;
            row = item;
            items = 1;
            item = 0;
        } else if (items > 1 && item == rows * row) {  // one follows the other as the rows do
            rows *= items;
            items = 1;
            item = 0;
        }
        if (rows > 1 && row == run) {
            run *= rows;
            rows = 1;
            row = 0;
        }
    }
    int64_t end() const { return at + (items - 1) * item + (rows - 1) * row + run; }
};

// Whether some run of `n` of them, `step` apart (>= 0) from `at` on, meets [from, to).
bool runs_meet(int64_t at, int64_t run, int64_t step, int64_t n, int64_t from, int64_t to) {
    if (step == 0) return at < to && at + run > from;
    const int64_t first = from - run - at < 0 ? 0 : (from - run - at) / step + 1;  // ends behind `from`
    return first < n && at + first * step < to;
}

bool meet(const Bytes& a, const Bytes& b) {
    if (a.at >= b.end() || b.at >= a.end()) return false;
    if (a.items == 1 && b.items == 1 && a.row == b.row && a.row >= std::max(a.run, b.run)) {
        // rows as far apart, as columns of one buffer have them: row i of a begins `r` bytes into the place of row i + q of b
        const int64_t d = a.at - b.at, q = d >= 0 ? d / a.row : -((-d + a.row - 1) / a.row), r = d - q * a.row;
        auto row_there = [&](int64_t k) { return k < b.rows && k + a.rows > 0; };  // some i with 0 <= i + k < b.rows
        return (r < b.run && row_there(q)) || (r + a.run > a.row && row_there(q + 1));
    }
    const Bytes &few = a.rows * a.items <= b.rows * b.items ? a : b, &many = &few == &a ? b : a;
    for (int64_t i = 0; i < few.items; ++i)
        for (int64_t r = 0; r < few.rows; ++r) {
            const int64_t from = few.at + i * few.item + r * few.row;
            for (int64_t k = 0; k < many.items; ++k)
                if (runs_meet(many.at + k * many.item, many.run, many.row, many.rows, from, from + few.run)) return true;
        }
    return false;
}

// An output that a caller brings must not lie over an input: blocks would read what others have written.
void check_apart(const char* what, const Opt& out, std::initializer_list<std::pair<const char*, const Tensor*>> inputs) {
    if (!out) return;
    const Bytes to(*out);
    for (const auto& [name, in] : inputs)
        if (in && meet(to, Bytes(*in))) refuse(what, MH3A_ERR_INVALID_ARG, "out overlaps ", name);
}

void check_frames(const char* what, const char* name, const Tensor& x) {
    if (!x.is_cuda()) refuse(what, MH3A_ERR_INVALID_ARG, name, " is not a CUDA tensor");
    if (x.dim() != 3) refuse(what, MH3A_ERR_SHAPE, name, " is not [B, T, C]");
    if (dtype_of(x.scalar_type()) < 0) refuse(what, MH3A_ERR_INVALID_ARG, name, " has type ", x.scalar_type());
    for (int i = 0; i < 3; ++i)
        if (x.size(i) < 1 || x.size(i) > INT_MAX) refuse(what, MH3A_ERR_SHAPE, name, " is empty, or a size passes 2^31");
    if (x.size(2) > 1 && x.stride(2) != 1) refuse(what, MH3A_ERR_INVALID_ARG, "the channels of ", name, " are not adjacent");
}

mh3a_norm norm_args(const char* what, const Tensor& x, int64_t groups, const Opt& weight, const Opt& bias, std::string_view act,
                    const Opt& alpha, const Opt& beta, double eps, const Opt& lengths) {
    check_frames(what, "x", x);
    mh3a_norm p{};
    p.dtype = dtype_of(x.scalar_type());
    p.B = (int)x.size(0);
    p.T = (int)x.size(1);
    p.C = (int)x.size(2);
    if (act == "snake_beta") p.act = MH3A_ACT_SNAKE_BETA;
    else if (act == "silu") p.act = MH3A_ACT_SILU;
    else if (act == "none") p.act = MH3A_ACT_NONE;
    else refuse(what, MH3A_ERR_INVALID_ARG, "unknown activation ", act);
    const bool snake = p.act == MH3A_ACT_SNAKE_BETA;
    require(alpha.has_value() == snake && beta.has_value() == snake, what, "alpha and beta belong to snake_beta, and it needs both");
    const c10::Device device = x.device();
    const int64_t per_channel[1] = {p.C}, per_item[1] = {p.B};
    if (weight) check_plain(what, "weight", *weight, device, at::kFloat, per_channel);
    if (bias) check_plain(what, "bias", *bias, device, at::kFloat, per_channel);
    if (alpha) check_plain(what, "alpha", *alpha, device, at::kFloat, per_channel);
    if (beta) check_plain(what, "beta", *beta, device, at::kFloat, per_channel);
    if (lengths) check_plain(what, "lengths", *lengths, device, at::kInt, per_item);
    if (groups < 1 || p.C % groups) refuse(what, MH3A_ERR_SHAPE, groups, " groups do not divide ", p.C, " channels");
    p.groups = (int)groups;
    p.eps = (float)eps;
    p.weight = data<float>(weight);
    p.bias = data<float>(bias);
    p.alpha = data<float>(alpha);
    p.beta = data<float>(beta);
    p.lengths = data<int>(lengths);
    return p;
}

std::tuple<Tensor, Tensor, Tensor> group_norm_act(const Tensor& x, int64_t groups, const Opt& weight, const Opt& bias,
                                                  std::string_view act, const Opt& alpha, const Opt& beta, double eps,
                                                  const Opt& lengths, const Opt& out, const std::optional<int64_t>& stream) {
    constexpr const char* what = "mh3a_group_norm_act";
    const mh3a_norm p = norm_args(what, x, groups, weight, bias, act, alpha, beta, eps, lengths);
    const c10::Device device = x.device();
    if (out) check_plain(what, "out", *out, device, x.scalar_type(), x.sizes());
    check_apart(what, out, {{"x", &x}, {"weight", opt(weight)}, {"bias", opt(bias)}, {"alpha", opt(alpha)}, {"beta", opt(beta)},
                            {"lengths", opt(lengths)}});
    const NoGradient none(what, "call group_norm_act_backward", opt(out), {&x, opt(weight), opt(bias), opt(alpha), opt(beta)});
    const Launch on(device, stream);
    Tensor y = out ? *out : empty(x.sizes(), x.scalar_type(), device);
    Tensor mean = empty({p.B, groups}, at::kFloat, device), rstd = empty({p.B, groups}, at::kFloat, device);
    const size_t n = mh3a_group_norm_act_workspace(
        &p, 0, aligned16(x) && aligned16(y) && aligned16(weight) && aligned16(bias) && aligned16(alpha) && aligned16(beta));
    Tensor ws;
    if (n) ws = empty({(int64_t)n}, at::kByte, device);
    check(mh3a_group_norm_act(&p, x.data_ptr(), stride_of(x, 0), stride_of(x, 1), y.data_ptr(), mean.data_ptr<float>(),
                              rstd.data_ptr<float>(), n ? ws.data_ptr() : nullptr, n, on.stream()),
          what);
    on.inputs({&x, opt(weight), opt(bias), opt(alpha), opt(beta), opt(lengths), opt(out)});
    on.outputs({&y, &mean, &rstd});
    none.from({&y, &mean, &rstd});
    return {y, mean, rstd};
}

std::tuple<Tensor, Opt, Opt, Opt, Opt> group_norm_act_backward(const Tensor& dy, const Tensor& x, const Tensor& mean,
                                                               const Tensor& rstd, int64_t groups, const Opt& weight,
                                                               const Opt& bias, std::string_view act, const Opt& alpha,
                                                               const Opt& beta, const Opt& lengths,
                                                               const std::optional<int64_t>& stream) {
    constexpr const char* what = "mh3a_group_norm_act_backward";
    const mh3a_norm p = norm_args(what, x, groups, weight, bias, act, alpha, beta, 0.0, lengths);
    const c10::Device device = x.device();
    check_frames(what, "dy", dy);
    require(dy.device() == device && dy.scalar_type() == x.scalar_type(), what, "dy is not of x's type and device");
    require(dy.sizes() == x.sizes(), what, "dy is not of x's shape", MH3A_ERR_SHAPE);
    const int64_t stats[2] = {p.B, groups};
    check_plain(what, "mean", mean, device, at::kFloat, stats);
    check_plain(what, "rstd", rstd, device, at::kFloat, stats);
    const NoGradient none(what, "it is a gradient itself", nullptr,
                          {&dy, &x, &mean, &rstd, opt(weight), opt(bias), opt(alpha), opt(beta)});
    const Launch on(device, stream);
    const Tensor dx = empty(x.sizes(), x.scalar_type(), device);
    const Opt* params[4] = {&weight, &bias, &alpha, &beta};
    Opt grads[4];
    for (int i = 0; i < 4; ++i)
        if (*params[i]) grads[i] = empty({p.C}, at::kFloat, device);
    const size_t n = mh3a_group_norm_act_workspace(
        &p, 1, aligned16(x) && aligned16(dy) && aligned16(dx) && aligned16(weight) && aligned16(bias) && aligned16(alpha) && aligned16(beta));
    Tensor ws;
    if (n) ws = empty({(int64_t)n}, at::kByte, device);
    check(mh3a_group_norm_act_backward(&p, x.data_ptr(), stride_of(x, 0), stride_of(x, 1), dy.data_ptr(), stride_of(dy, 0), stride_of(dy, 1),
                                       mean.data_ptr<float>(), rstd.data_ptr<float>(), dx.data_ptr(), data<float>(grads[0]),
                                       data<float>(grads[1]), data<float>(grads[2]), data<float>(grads[3]), n ? ws.data_ptr() : nullptr, n,
                                       on.stream()),
          what);
    on.inputs({&dy, &x, &mean, &rstd, opt(weight), opt(bias), opt(alpha), opt(beta), opt(lengths)});
    on.outputs({&dx});
    none.from({&dx});
    for (const Opt& g : grads)
        if (g) {
            on.outputs({&*g});
            none.from({&*g});
        }
    return {dx, grads[0], grads[1], grads[2], grads[3]};
}

// ------------------------------------------------------------------------------------------- fp8
constexpr int64_t kBlock = 128;

int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

void check_matrix(const char* what, const char* name, const Tensor& x) {
    if (!x.is_cuda()) refuse(what, MH3A_ERR_INVALID_ARG, name, " is not a CUDA tensor");
    if (x.dim() != 2) refuse(what, MH3A_ERR_SHAPE, name, " is not a matrix");
    for (int i = 0; i < 2; ++i)
        if (x.size(i) < 1 || x.size(i) > INT_MAX) refuse(what, MH3A_ERR_SHAPE, name, " is empty, or a size passes 2^31");
    if (x.size(1) > 1 && x.stride(1) != 1) refuse(what, MH3A_ERR_INVALID_ARG, "the columns of ", name, " are not adjacent");
}

void check_values(const char* what, const char* name, const Tensor& x) {
    check_matrix(what, name, x);
    if (dtype_of(x.scalar_type()) < 0) refuse(what, MH3A_ERR_INVALID_ARG, name, " has type ", x.scalar_type());
}

// A stored fp8 matrix and its scales.
struct Stored {
    int64_t rows, cols, stride;
    int block_rows;
};

Stored check_stored(const char* what, const char* name, const Tensor& q, const Tensor& scale) {
    check_matrix(what, name, q);
    if (q.scalar_type() != at::kFloat8_e4m3fn) refuse(what, MH3A_ERR_INVALID_ARG, name, " has type ", q.scalar_type());
    Stored s{q.size(0), q.size(1), q.stride(0), 1};
    if (s.rows == 1) s.stride = (s.cols + 15) / 16 * 16;
    if (s.stride < s.cols || s.stride % 16 || reinterpret_cast<uintptr_t>(q.data_ptr()) % 16)
        refuse(what, MH3A_ERR_INVALID_ARG, "the rows of ", name, " do not start on 16-byte boundaries");
    if (scale.scalar_type() != at::kFloat || scale.device() != q.device() || !scale.is_contiguous())
        refuse(what, MH3A_ERR_INVALID_ARG, "the scales of ", name, " are not a contiguous float32 tensor on ", q.device());
    const int64_t kb = blocks(s.cols);
    if (scale.dim() == 2 && scale.size(0) == kb) {
        if (scale.size(1) == s.rows) return s;
        s.block_rows = (int)kBlock;
        if (scale.size(1) == blocks(s.rows)) return s;
    }
    refuse(what, MH3A_ERR_SHAPE, "the scales of ", name, " are ", scale.sizes(), ": [", kb, ", ", s.rows, "] or [", kb, ", ",
           blocks(s.rows), "] are wanted");
}

void check_bias_out(const char* what, const Opt& bias, const Opt& out, const c10::Device& device, int64_t M, int64_t N,
                    at::ScalarType type) {
    const int64_t cols[1] = {N};
    if (bias) check_plain(what, "bias", *bias, device, at::kFloat, cols);
    if (out) {
        if (out->device() != device || out->scalar_type() != type)
            refuse(what, MH3A_ERR_INVALID_ARG, "out is not a ", type, " tensor on ", device);
        if (out->dim() != 2 || out->size(0) != M || out->size(1) != N)
            refuse(what, MH3A_ERR_SHAPE, "out is ", out->sizes(), ": [", M, ", ", N, "] is wanted");
        require((N == 1 || out->stride(1) == 1) && (M == 1 || out->stride(0) >= N), what,
                "the columns of out are not adjacent, or its rows overlap");
    }
}

int64_t row_stride(const Tensor& t, int64_t cols) { return t.size(0) > 1 ? t.stride(0) : cols; }

std::tuple<Tensor, Tensor> fp8_quantize(const Tensor& x, int64_t block_rows, bool transpose, const std::optional<int64_t>& stream) {
    constexpr const char* what = "mh3a_fp8_quantize";
    check_values(what, "x", x);
    if (block_rows != 1 && block_rows != kBlock) refuse(what, MH3A_ERR_INVALID_ARG, "block_rows is ", block_rows, ": 1 or 128 is wanted");
    const int64_t rows = x.size(0), cols = x.size(1), outer = transpose ? cols : rows, inner = transpose ? rows : cols;
    const NoGradient none(what, "differentiate what it is used for", nullptr, {&x});
    const Launch on(x.device(), stream);
    const int64_t ld = (inner + 15) / 16 * 16;
    Tensor q = empty({outer, ld}, at::kFloat8_e4m3fn, x.device());
    const Tensor scale = empty({blocks(inner), block_rows == 1 ? outer : blocks(outer)}, at::kFloat, x.device());
    check(mh3a_fp8_quantize(x.data_ptr(), dtype_of(x.scalar_type()), (int)rows, (int)cols, row_stride(x, cols), (int)block_rows,
                            transpose, q.data_ptr(), ld, scale.data_ptr<float>(), on.stream()),
          what);
    on.inputs({&x});
    on.outputs({&q, &scale});
    none.from({&q, &scale});
    if (ld != inner) q = q.narrow(1, 0, inner);
    return {q, scale};
}

Tensor fp8_matmul(const Tensor& a, const Tensor& a_scale, const Tensor& b, const Tensor& b_scale, at::ScalarType out_dtype,
                  const Opt& bias, const Opt& out, const std::optional<int64_t>& stream) {
    constexpr const char* what = "mh3a_fp8_matmul";
    const Stored sa = check_stored(what, "a", a, a_scale), sb = check_stored(what, "b", b, b_scale);
    require(sa.block_rows == 1, what, "a has blocks of 128 rows: block_rows 1 is wanted");
    if (sa.cols != sb.cols) refuse(what, MH3A_ERR_SHAPE, "a has ", sa.cols, " columns and b ", sb.cols);
    require(a.device() == b.device(), what, "a and b are on different devices");
    if (dtype_of(out_dtype) < 0) refuse(what, MH3A_ERR_INVALID_ARG, "out_dtype is ", out_dtype);
    check_bias_out(what, bias, out, a.device(), sa.rows, sb.rows, out_dtype);
    check_apart(what, out, {{"a", &a}, {"b", &b}, {"a_scale", &a_scale}, {"b_scale", &b_scale}, {"bias", opt(bias)}});
    const NoGradient none(what, "form the products of the gradients", opt(out), {&a, &a_scale, &b, &b_scale, opt(bias)});
    const Launch on(a.device(), stream);
    const Tensor y = out ? *out : empty({sa.rows, sb.rows}, out_dtype, a.device());
    check(mh3a_fp8_matmul(a.data_ptr(), sa.stride, a_scale.data_ptr<float>(), b.data_ptr(), sb.stride, b_scale.data_ptr<float>(),
                          sb.block_rows, (int)sa.rows, (int)sb.rows, (int)sa.cols, data<float>(bias), dtype_of(out_dtype),
                          y.data_ptr(), row_stride(y, sb.rows), on.stream()),
          what);
    on.inputs({&a, &a_scale, &b, &b_scale, opt(bias), opt(out)});
    on.outputs({&y});
    none.from({&y});
    return y;
}

Tensor fp8_linear(const Tensor& x, const Tensor& w, const Tensor& w_scale, const Opt& bias, const Opt& out,
                  const std::optional<int64_t>& stream) {
    constexpr const char* what = "mh3a_fp8_linear";
    check_values(what, "x", x);
    const Stored sw = check_stored(what, "w", w, w_scale);
    const int64_t M = x.size(0), K = x.size(1), N = sw.rows;
    if (K != sw.cols) refuse(what, MH3A_ERR_SHAPE, "x has ", K, " columns and w ", sw.cols);
    require(x.device() == w.device(), what, "x and w are on different devices");
    check_bias_out(what, bias, out, x.device(), M, N, x.scalar_type());
    check_apart(what, out, {{"x", &x}, {"w", &w}, {"w_scale", &w_scale}, {"bias", opt(bias)}});
    const NoGradient none(what, "call fp8_linear and fp8_matmul on the transposed operands", opt(out), {&x, &w, &w_scale, opt(bias)});
    const Launch on(x.device(), stream);
    const Tensor y = out ? *out : empty({M, N}, x.scalar_type(), x.device());
    const size_t n = mh3a_fp8_linear_workspace((int)M, (int)N, (int)K);
    Tensor ws;
    if (n) ws = empty({(int64_t)n}, at::kByte, x.device());
    check(mh3a_fp8_linear(x.data_ptr(), dtype_of(x.scalar_type()), row_stride(x, K), w.data_ptr(), sw.stride,
                          w_scale.data_ptr<float>(), sw.block_rows, (int)M, (int)N, (int)K, data<float>(bias), y.data_ptr(),
                          row_stride(y, N), n ? ws.data_ptr() : nullptr, n, on.stream()),
          what);
    on.inputs({&x, &w, &w_scale, opt(bias), opt(out)});
    on.outputs({&y});
    none.from({&y});
    return y;
}

}  // namespace

PYBIND11_MODULE(_ops, m) {
    const py::object type = py::module_::import("bigvgan_waveform_decoder_b200.binding").attr("MH3AError");
    static PyObject* error = type.inc_ref().ptr();
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const Error& e) {
            PyErr_SetObject(error, py::make_tuple(e.status, e.what, e.detail).ptr());
        }
    });
    m.def("group_norm_act", &group_norm_act);
    m.def("group_norm_act_backward", &group_norm_act_backward);
    m.def("fp8_quantize", &fp8_quantize);
    m.def("fp8_matmul", &fp8_matmul);
    m.def("fp8_linear", &fp8_linear);
}
