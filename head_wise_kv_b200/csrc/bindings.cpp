// Compiled half of the Python binding: the calls that a program makes once
// per layer and step, with their checks of shapes, types and devices, and the
// autograd function of the windowed attention.  A decode step's kernels run
// for a few microseconds; the same checks and conversions in Python and
// ctypes cost more than that (8 to 15 us a call, 200 us for a small
// attention's forward and backward).  Nothing is computed here: every step of
// the path runs in the library's kernels (duo_kv.h).
#include <ATen/TracerMode.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/extension.h>

#include <algorithm>
#include <limits>
#include <mutex>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <tuple>
#include <unordered_set>
#include <vector>

#include "duo_kv.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

// An error code of the library; Python sees _lib.DuoError.
struct DuoFailure : std::runtime_error {
    int code;
    std::string what_call;
    DuoFailure(int c, const char* call)
        : std::runtime_error(std::string(call) + ": " + duo_strerror(c)), code(c), what_call(call) {}
};

void check(int code, const char* call) {
    if (code != DUO_OK) throw DuoFailure(code, call);
}

std::string shape_of(at::IntArrayRef s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << ')';
    return o.str();
}

// A contiguous tensor of one type, shape and device.
void need(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& dev) {
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, ": dtype ", t.scalar_type(), ", expected ", type);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, ": shape ", shape_of(t.sizes()), ", expected ", shape_of(shape));
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", expected ", dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}

const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
const int32_t* ints(const OptTensor& t) { return t ? ints(*t) : nullptr; }

// What reads a tensor's memory alone loses what rides along with it: a forward-mode tangent, or the
// operations that a trace records.  Refused instead of left out without a word.
void check_plain(const Tensor& t, const char* name) {
    TORCH_CHECK_NOT_IMPLEMENTED(!t._fw_grad(0).defined(), name,
                                ": forward-mode derivatives are not implemented, the tangent would be lost");
}

// A tensor that a call has written, as in-place operations mark theirs: a backward pass that saved what was there
// before then says so.
void mark_written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void check_not_traced(const char* call) {
    TORCH_CHECK_NOT_IMPLEMENTED(!at::tracer::impl::is_dispatch_enabled(), call,
                                " cannot be traced: the trace would hold an empty result");
}

// A backward pass captured into a graph must not meet a leaf whose gradient
// node lives on the default stream (an eager graph of the same leaf keeps it):
// the engine would make the capture wait for that stream, which cannot join
// it, on a thread of its own, where the error ends the process.  Refused here
// instead: at the forward call where a leaf is its input, in the backward pass
// where leaves lie further up (parts of a projection, its weights).  Another
// stream joins the capture, as that of the warm-up before it does.
bool capturing_on(const at::Device& dev) {
    const c10::cuda::OptionalCUDAGuard guard(dev);
    return c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None;
}

void check_leaf(torch::autograd::Node& node, const at::Device& dev, const char* name) {
    const auto stream = node.stream();
    TORCH_CHECK_VALUE(!stream || *stream != c10::cuda::getDefaultCUDAStream(dev.index()).unwrap(), name,
                      " is a leaf of an eager graph that is still alive: drop that graph, or give the capture a leaf of its "
                      "own, before its backward pass is captured");
}

void check_capture(const Tensor& t, const char* name) {
    if (!t.requires_grad() || !t.is_leaf() || !at::GradMode::is_enabled() || !t.is_cuda()) return;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
    if (node && capturing_on(t.device())) check_leaf(*node, t.device(), name);
}

// In a backward pass on `dev`: the leaves that it will reach from here.
void check_captured_backward(const at::Device& dev) {
    if (!capturing_on(dev)) return;
    const auto start = torch::autograd::get_current_node();
    const auto* plan = torch::autograd::get_current_graph_task_exec_info();     // empty: every node runs
    std::vector<torch::autograd::Node*> stack;
    std::unordered_set<torch::autograd::Node*> seen;
    const auto follow = [&](const torch::autograd::Node& node) {
        for (const auto& edge : node.next_edges()) {
            if (!edge.function || !seen.insert(edge.function.get()).second) continue;
            if (plan && !plan->empty()) {
                const auto it = plan->find(edge.function.get());
                if (it == plan->end() || !it->second.should_execute()) continue;
            }
            stack.push_back(edge.function.get());
        }
    };
    if (start) follow(*start);
    while (!stack.empty()) {
        torch::autograd::Node* node = stack.back();
        stack.pop_back();
        if (dynamic_cast<torch::autograd::AccumulateGrad*>(node)) check_leaf(*node, dev, "what this backward pass reaches");
        follow(*node);
    }
}

cudaStream_t stream_of(const at::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// ------------------------------------------------------------------ overlap
// A tensor's memory: blocks of `block` bytes at base + the sum of c_k step_k, 0 <= c_k < count_k.
struct Blocks {
    int64_t base = 0, block = 0, end = 0;       // end: behind the last byte
    struct Dim {
        int64_t step, count;
    };
    c10::SmallVector<Dim, 4> dims;              // of more than one entry

    explicit Blocks(const Tensor& t) {
        if (t.numel() == 0) return;
        base = int64_t(reinterpret_cast<uintptr_t>(t.data_ptr()));
        block = t.element_size();
        end = base + block;
        for (int64_t i = t.dim() - 1; i >= 0; --i) {
            if (t.size(i) == 1) continue;
            const int64_t step = t.stride(i) * t.element_size();
            end += (t.size(i) - 1) * step;
            if (step == block && dims.empty())
                block *= t.size(i);             // the inner dimensions that lie end to end
            else
                dims.push_back({step, t.size(i)});
        }
    }
};

// at + the sum of c_k step_k for some lo_k <= c_k <= hi_k lies in [first, last].  Steps are given in falling order, so
// that few c_k of each come into question where the dimensions nest; a search that grows long says yes.
struct Term {
    int64_t step, lo, hi;
};

bool reaches(const Term* t, size_t n, int64_t at, int64_t first, int64_t last, int& budget) {
    if (n == 0) return at >= first && at <= last;
    if (--budget < 0) return true;
    int64_t lo = 0, hi = 0;                     // of the later ones together
    for (size_t k = 1; k < n; ++k) {
        lo += t[k].step * t[k].lo;
        hi += t[k].step * t[k].hi;
    }
    const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t c0 = std::max(t[0].lo, -floor_div(-(first - at - hi), t[0].step));
    const int64_t c1 = std::min(t[0].hi, floor_div(last - at - lo, t[0].step));
    for (int64_t c = c0; c <= c1; ++c)
        if (reaches(t + 1, n - 1, at + c * t[0].step, first, last, budget)) return true;
    return false;
}

constexpr int kSearch = 4096;

void in_order(c10::SmallVector<Term, 8>& t) {
    std::sort(t.begin(), t.end(), [](const Term& a, const Term& b) { return a.step > b.step; });
}

// Whether two tensors share a byte.
bool overlap(const Tensor& x, const Tensor& y) {
    const Blocks a(x), b(y);
    if (a.block == 0 || b.block == 0 || a.end <= b.base || b.end <= a.base) return false;
    c10::SmallVector<Term, 8> terms;
    const auto add = [&](int64_t step, int64_t lo, int64_t hi) {
        if (step == 0) return;
        for (Term& t : terms)
            if (t.step == step) {
                t.lo += lo;
                t.hi += hi;
                return;
            }
        terms.push_back({step, lo, hi});
    };
    for (const auto& d : a.dims) add(d.step, -(d.count - 1), 0);
    for (const auto& d : b.dims) add(d.step, 0, d.count - 1);
    in_order(terms);
    int budget = kSearch;
    return reaches(terms.data(), terms.size(), b.base - a.base, -(b.block - 1), a.block - 1, budget);
}

// Whether two elements of a tensor share a byte.
bool overlaps_itself(const Tensor& x) {
    const Blocks a(x);
    c10::SmallVector<Term, 8> terms;
    for (const auto& d : a.dims) {
        if (d.step == 0) return true;
        terms.push_back({d.step, -(d.count - 1), d.count - 1});
    }
    in_order(terms);
    int budget = kSearch;
    for (size_t k = 0; k < terms.size(); ++k) {     // the first index in which the two differ
        Term save = terms[k];
        terms[k].lo = 1;
        if (reaches(terms.data() + k, terms.size() - k, 0, -(a.block - 1), a.block - 1, budget)) return true;
        terms[k] = save;
    }
    return false;
}

// The same elements at the same places.
bool same_view(const Tensor& x, const Tensor& y) {
    if (x.data_ptr() != y.data_ptr() || x.sizes() != y.sizes() || x.scalar_type() != y.scalar_type()) return false;
    for (int64_t i = 0; i < x.dim(); ++i)
        if (x.size(i) > 1 && x.stride(i) != y.stride(i)) return false;
    return true;
}

// ------------------------------------------------------------------ rotary positions
int rope_dtype(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return DUO_BF16;
        case at::kHalf: return DUO_FP16;
        case at::kFloat: return DUO_FP32;
        default: return -1;
    }
}

// A tensor of a launch and where it goes: null where that is made by the call.
struct RopeTask {
    const Tensor* x;
    const Tensor* out;
    bool rotate;
};

// In place each thread writes what it has read; any other overlap would be a race.
void check_apart(const RopeTask* tasks, size_t count) {
    for (size_t i = 0; i < count; ++i) {
        const Tensor& out = *tasks[i].out;
        TORCH_CHECK_VALUE(!overlaps_itself(out), "out must not overlap itself");
        for (size_t k = 0; k < count; ++k) {
            TORCH_CHECK_VALUE((k == i && same_view(out, *tasks[i].x)) || !overlap(out, *tasks[k].x),
                              "out must be x or lie apart from it");
            TORCH_CHECK_VALUE(k >= i || !overlap(out, *tasks[k].out), "results must lie apart");
        }
    }
}

// One launch over up to three tensors of a batch: their checks, then duo_rope_apply.  Returns the first result.
Tensor rope_launch(uintptr_t plan, int64_t d, const RopeTask* tasks, size_t tensors, const Tensor& positions,
                   const OptTensor& n_new, bool transpose) {
    check_not_traced("Rope.apply");
    TORCH_CHECK_VALUE(tensors >= 1 && tensors <= 3, "one to three tensors in a launch");
    for (size_t i = 0; i < tensors; ++i) {
        check_plain(*tasks[i].x, "x");
        if (tasks[i].out) check_plain(*tasks[i].out, "out");
    }
    const Tensor& x0 = *tasks[0].x;
    const int dtype = rope_dtype(x0.scalar_type());
    TORCH_CHECK_TYPE(dtype >= 0, "dtype ", x0.scalar_type(), ", expected bfloat16, float16 or float32");
    const at::Device dev = x0.device();
    TORCH_CHECK_VALUE(dev.is_cuda(), "the tensors must be on a CUDA device");
    for (size_t i = 0; i < tensors; ++i)
        TORCH_CHECK_VALUE(tasks[i].x->dim() == 4 && tasks[i].x->size(3) == d, "shape ", shape_of(tasks[i].x->sizes()),
                          ", expected [batch][heads][tokens][", d, "]");
    const int64_t B = x0.size(0), n = x0.size(2), top = std::numeric_limits<int32_t>::max();
    const bool per_token = positions.dim() == 2;
    TORCH_CHECK_VALUE(positions.scalar_type() == at::kInt && positions.device() == dev && positions.is_contiguous(),
                      "positions must be contiguous int32 on the tensors' device");
    TORCH_CHECK_VALUE(per_token ? positions.sizes() == at::IntArrayRef({B, n}) : positions.sizes() == at::IntArrayRef({B}),
                      "positions: shape ", shape_of(positions.sizes()), ", expected (", B, ",) or (", B, ", ", n, ")");
    if (n_new)
        TORCH_CHECK_VALUE(n_new->scalar_type() == at::kInt && n_new->device() == dev && n_new->is_contiguous() &&
                              n_new->sizes() == at::IntArrayRef({B}),
                          "n_new must be contiguous int32 [", B, "] on the tensors' device");
    const c10::cuda::CUDAGuard guard(dev);
    duo_rope_tensor list[3] = {};
    Tensor made;
    for (size_t i = 0; i < tensors; ++i) {
        const Tensor& x = *tasks[i].x;
        TORCH_CHECK_VALUE(x.scalar_type() == x0.scalar_type() && x.device() == dev && x.size(0) == B && x.size(2) == n,
                          "tensors of one launch share dtype, device, batch and tokens");
        TORCH_CHECK_VALUE(B <= top && x.size(1) <= top && n <= top, "too large a tensor");
        TORCH_CHECK_VALUE(x.stride(3) == 1, "the elements of a head must be contiguous");
        TORCH_CHECK_VALUE(x.size(1) >= 1 || B * n == 0, "a tensor has at least one head");
        if (!tasks[i].out) made = n_new ? at::zeros(x.sizes(), x.options()) : at::empty(x.sizes(), x.options());
        const Tensor& out = tasks[i].out ? *tasks[i].out : made;
        if (tasks[i].out) {
            TORCH_CHECK_VALUE(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() && out.device() == dev,
                              "out must have the input's shape, dtype and device");
            TORCH_CHECK_VALUE(out.stride(3) == 1, "the elements of a head must be contiguous");
        }
        duo_rope_tensor& t = list[i];
        t.in = x.data_ptr();
        t.out = out.data_ptr();
        t.heads = int32_t(x.size(1));
        t.rotate = tasks[i].rotate;
        for (int k = 0; k < 3; ++k) {     // a dimension of one entry has no stride that matters
            t.in_stride[k] = x.size(k) > 1 ? x.stride(k) : 0;
            t.out_stride[k] = x.size(k) > 1 ? out.stride(k) : 0;
        }
    }
    if (tasks[0].out) check_apart(tasks, tensors);
    const Tensor& first = tasks[0].out ? *tasks[0].out : made;
    if (x0.numel() == 0) return first;
    check(duo_rope_apply(reinterpret_cast<const duo_rope*>(plan), dtype, transpose, int32_t(B), int32_t(n), list,
                         int32_t(tensors), ints(positions), per_token, ints(n_new), stream_of(dev)),
          "duo_rope_apply");
    for (size_t i = 0; i < tensors; ++i)
        if (tasks[i].out) mark_written(*tasks[i].out);
    return first;
}

Tensor rope_apply(uintptr_t plan, int64_t d, const Tensor& x, const Tensor& positions, const OptTensor& n_new,
                  bool transpose, const OptTensor& given) {
    const RopeTask task{&x, given ? &*given : nullptr, true};
    return rope_launch(plan, d, &task, 1, positions, n_new, transpose);
}

// ------------------------------------------------------------------ the cache's calls
// A projection's rows [lead...][heads][d], bf16, token-major.
duo_rows rows_of(const Tensor& t, const char* name, int64_t heads, int64_t d, at::IntArrayRef lead, const at::Device& dev) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, name, ": dtype ", t.scalar_type(), ", expected ", at::kBFloat16);
    const size_t n = lead.size();
    bool same = size_t(t.dim()) == n + 2 && t.size(n) == heads && t.size(n + 1) == d;
    for (size_t i = 0; same && i < n; ++i) same = t.size(i) == lead[i];
    TORCH_CHECK_VALUE(same, name, ": shape ", shape_of(t.sizes()), ", expected ", shape_of(lead), " x (", heads, ", ", d, ")");
    TORCH_CHECK_VALUE(t.device() == dev, name, ": on ", t.device(), ", expected ", dev);
    TORCH_CHECK_VALUE(t.stride(n + 1) == 1, name, ": the elements of a head must be contiguous");
    TORCH_CHECK_VALUE(n == 1 || lead[0] <= 1 || lead[1] <= 1 || t.stride(0) == lead[1] * t.stride(1), name,
                      ": sequences must follow one another at the token stride");
    const int64_t token = n == 1 || lead[1] == 1 ? t.stride(0) : t.stride(1);
    // a dimension of one row has no stride that matters
    return duo_rows{static_cast<const uint16_t*>(t.data_ptr()), t.numel() > heads * d ? token : 0,
                    heads > 1 ? t.stride(n) : 0};
}

void check_rows(const char* call, const OptTensor& q, const Tensor& k, const Tensor& v) {
    check_not_traced(call);
    if (q) check_plain(*q, "q");
    check_plain(k, "k");
    check_plain(v, "v");
}

struct Cache {
    duo_kv* kv;
    at::Device dev;
    int64_t B, hq, n_kv, d;

    Cache(uintptr_t handle, int64_t device, int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim)
        : kv(reinterpret_cast<duo_kv*>(handle)),
          dev(at::kCUDA, at::DeviceIndex(device)),
          B(batch),
          hq(q_heads),
          n_kv(kv_heads),
          d(head_dim) {}

    OptTensor append_rope(int64_t layer, uintptr_t rope, int64_t rope_d, const OptTensor& q, const Tensor& k, const Tensor& v,
                          const Tensor& len_before, const py::object& tokens, const OptTensor& n_new,
                          const OptTensor& given) const {
        TORCH_CHECK_VALUE(rope_d == d, "rope of head_dim ", rope_d, ", expected ", d);
        check_rows("append_rope", q, k, v);
        duo_token_map map{};
        const bool ragged = !tokens.is_none();
        std::vector<int64_t> lead;
        Tensor seq, pos, slot, after;
        if (ragged) {
            TORCH_CHECK_VALUE(!n_new, "n_new belongs to a padded batch: the token map says how many tokens there are");
            const int64_t T = tokens.attr("max_tokens").cast<int64_t>();
            TORCH_CHECK_VALUE(tokens.attr("batch").cast<int64_t>() == B, "the token map is of another batch or device");
            lead = {T};
            seq = tokens.attr("seq").cast<Tensor>();
            pos = tokens.attr("pos").cast<Tensor>();
            slot = tokens.attr("slot").cast<Tensor>();
            after = tokens.attr("len_after").cast<Tensor>();
            TORCH_CHECK_VALUE(seq.device() == dev, "the token map is of another batch or device");
            need(seq, "seq", at::kInt, {T}, dev);
            need(pos, "pos", at::kInt, {T}, dev);
            if (slot.numel() != 0) need(slot, "slot", at::kLong, {T}, dev);   // none: read through the page table
            need(after, "len_after", at::kInt, {B}, dev);
            map.seq = ints(seq);
            map.pos = ints(pos);
            map.slot = slot.numel() ? static_cast<const int64_t*>(slot.data_ptr()) : nullptr;
            map.len_after = ints(after);
        } else {
            TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == B, "a padded batch is [", B, "][tokens][heads][", d, "]");
            lead = {k.size(0), k.size(1)};
            if (n_new) need(*n_new, "n_new", at::kInt, {B}, dev);
        }
        need(len_before, "len_before", at::kInt, {B}, dev);
        const duo_rows kr = rows_of(k, "k", n_kv, d, lead, dev), vr = rows_of(v, "v", n_kv, d, lead, dev);
        const c10::cuda::CUDAGuard guard(dev);
        duo_rows qr{};
        OptTensor out;
        if (q) {
            qr = rows_of(*q, "q", hq, d, lead, dev);
            std::vector<int64_t> shape = lead;
            shape.push_back(hq);
            shape.push_back(d);
            if (given) {
                need(*given, "out", at::kBFloat16, shape, dev);
                TORCH_CHECK_VALUE(!overlap(*given, *q) && !overlap(*given, k) && !overlap(*given, v),
                                  "out must lie apart from q, k and v");
                out = given;
            } else {        // rows without a token are zero where out is new
                out = ragged || n_new ? at::zeros(shape, k.options()) : at::empty(shape, k.options());
            }
        } else {
            TORCH_CHECK_VALUE(!given, "out without q");
        }
        TORCH_CHECK_VALUE(lead.back() <= std::numeric_limits<int32_t>::max(), "too many tokens");
        check(duo_kv_append_rope(kv, int32_t(layer), reinterpret_cast<const duo_rope*>(rope), q ? &qr : nullptr, &kr, &vr,
                                 ints(len_before), ragged ? &map : nullptr, ints(n_new), int32_t(lead.back()),
                                 out ? static_cast<uint16_t*>(out->data_ptr()) : nullptr, stream_of(dev)),
              "duo_kv_append_rope");
        if (given) mark_written(*given);
        return out;
    }

    py::object reserve(const Tensor& len_before, const OptTensor& n_new, const py::object& tokens) const {
        need(len_before, "len_before", at::kInt, {B}, dev);
        if (n_new) need(*n_new, "n_new", at::kInt, {B}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        if (tokens.is_none()) {
            Tensor after = at::empty({B}, len_before.options());
            check(duo_kv_reserve(kv, ints(len_before), ints(n_new), 0, static_cast<int32_t*>(after.data_ptr()), nullptr,
                                 nullptr, nullptr, nullptr, stream_of(dev)),
                  "duo_kv_reserve");
            return py::cast(after);
        }
        const int64_t T = tokens.attr("max_tokens").cast<int64_t>();
        TORCH_CHECK_VALUE(tokens.attr("batch").cast<int64_t>() == B, "the token map is of another batch or device");
        const Tensor seq = tokens.attr("seq").cast<Tensor>(), pos = tokens.attr("pos").cast<Tensor>(),
                     slot = tokens.attr("slot").cast<Tensor>(), after = tokens.attr("len_after").cast<Tensor>(),
                     cu = tokens.attr("cu").cast<Tensor>();
        TORCH_CHECK_VALUE(seq.device() == dev, "the token map is of another batch or device");
        need(seq, "seq", at::kInt, {T}, dev);
        need(pos, "pos", at::kInt, {T}, dev);
        need(slot, "slot", at::kLong, {T}, dev);
        need(after, "len_after", at::kInt, {B}, dev);
        need(cu, "cu", at::kInt, {B + 1}, dev);
        TORCH_CHECK_VALUE(T <= std::numeric_limits<int32_t>::max(), "too many tokens");
        // a map without entries still has its counts: the arrays are not looked at
        void* const none = cu.data_ptr();
        check(duo_kv_reserve(kv, ints(len_before), ints(n_new), int32_t(T), static_cast<int32_t*>(after.data_ptr()),
                             static_cast<int32_t*>(cu.data_ptr()), static_cast<int32_t*>(T ? seq.data_ptr() : none),
                             static_cast<int32_t*>(T ? pos.data_ptr() : none),
                             static_cast<int64_t*>(T ? slot.data_ptr() : none), stream_of(dev)),
              "duo_kv_reserve");
        for (const Tensor* t : {&seq, &pos, &slot, &after, &cu}) mark_written(*t);
        return tokens;
    }

    // out, lse and q_rot come checked or new
    py::object step_rope(int64_t layer, uintptr_t rope, int64_t rope_d, const Tensor& q, const Tensor& k, const Tensor& v,
                         const Tensor& len_before, const Tensor& lengths, double scale, const OptTensor& given_out,
                         const OptTensor& given_lse, bool want_lse, const OptTensor& given_rot, const Tensor& ws) const {
        TORCH_CHECK_VALUE(rope_d == d, "rope of head_dim ", rope_d, ", expected ", d);
        check_rows("step_rope", q, k, v);
        const duo_rows qr = rows_of(q, "q", hq, d, {B}, dev), kr = rows_of(k, "k", n_kv, d, {B}, dev),
                       vr = rows_of(v, "v", n_kv, d, {B}, dev);
        need(len_before, "len_before", at::kInt, {B}, dev);
        need(lengths, "lengths", at::kInt, {B}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        if (given_rot) need(*given_rot, "q_rot", at::kBFloat16, {B, hq, d}, dev);
        if (given_out) need(*given_out, "out", at::kFloat, {B, hq, d}, dev);
        if (given_lse) need(*given_lse, "lse", at::kFloat, {B, hq}, dev);
        // rotated in place each thread writes what it has read; the decode starts while the append runs
        const OptTensor* const given[3] = {&given_rot, &given_out, &given_lse};
        for (int i = 0; i < 3; ++i) {
            if (!*given[i]) continue;
            const Tensor& t = **given[i];
            TORCH_CHECK_VALUE(((i == 0 && same_view(t, q)) || !overlap(t, q)) && !overlap(t, k) && !overlap(t, v),
                              "out, lse and q_rot must lie apart from q, k and v (but q_rot may be q)");
            for (int j = 0; j < i; ++j)
                TORCH_CHECK_VALUE(!*given[j] || !overlap(t, **given[j]), "out, lse and q_rot must lie apart");
        }
        const auto fp32 = q.options().dtype(at::kFloat);
        const Tensor rot = given_rot ? *given_rot : at::empty({B, hq, d}, q.options());
        const Tensor out = given_out ? *given_out : at::empty({B, hq, d}, fp32);
        OptTensor lse = given_lse;
        if (want_lse && !lse) lse = at::empty({B, hq}, fp32);
        check(duo_decode_step_rope(kv, int32_t(layer), reinterpret_cast<const duo_rope*>(rope), &qr, &kr, &vr,
                                   ints(len_before), ints(lengths), float(scale), static_cast<uint16_t*>(rot.data_ptr()),
                                   static_cast<float*>(out.data_ptr()),
                                   lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws.data_ptr(), ws.numel(),
                                   stream_of(dev)),
              "duo_decode_step_rope");
        for (const OptTensor* t : given)
            if (*t) mark_written(**t);
        if (lse) return py::make_tuple(out, *lse);
        return py::cast(out);
    }
};

// ------------------------------------------------------------------ windowed attention
// One status word per device, never freed: kernels may still hold it when the process ends.  It is
// memory of its own, cleared before the call goes on: made by the allocator in a captured call, its
// clearing would belong to the graph, and each replay would take back the bits of other calls.
Tensor status_word(const at::Device& dev) {
    static std::mutex lock;
    static auto* words = new std::vector<Tensor>();
    const std::lock_guard<std::mutex> hold(lock);
    const size_t i = size_t(dev.index());
    if (words->size() <= i) words->resize(i + 1);
    if (!(*words)[i].defined()) {
        const c10::cuda::CUDAGuard guard(dev);
        const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);
        void* word = nullptr;
        cudaStream_t own = nullptr;
        C10_CUDA_CHECK(cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking));
        cudaError_t e = cudaMalloc(&word, sizeof(int32_t));
        if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(int32_t), own);
        if (e == cudaSuccess) e = cudaStreamSynchronize(own);
        (void)cudaStreamDestroy(own);
        if (e != cudaSuccess && word) (void)cudaFree(word);
        C10_CUDA_CHECK(e);
        const c10::InferenceMode off(false);      // it outlives the mode of its first call, and is cleared outside it
        (*words)[i] = at::from_blob(word, {1}, at::TensorOptions().dtype(at::kInt).device(dev));
    }
    return (*words)[i];
}

// x, or a copy that the kernels can read: contiguous heads, strides in 16-byte steps and none of them 0.
Tensor usable(const Tensor& x) {
    bool ok = x.stride(3) == 1 && reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0;
    for (int i = 0; ok && i < 3; ++i)
        if (x.size(i) > 1) ok = x.stride(i) % 8 == 0 && x.stride(i) >= x.size(3);
    return ok ? x : x.clone(at::MemoryFormat::Contiguous);
}

// A new dense tensor with x's shape and order of dimensions.
Tensor like(const Tensor& x) {
    int order[3] = {0, 1, 2};
    if (x.numel() > 0)
        std::stable_sort(order, order + 3, [&](int a, int b) { return x.stride(a) > x.stride(b); });
    int64_t strides[4] = {0, 0, 0, 1}, step = x.size(3);
    for (int i = 2; i >= 0; --i) {
        strides[order[i]] = step;
        step *= std::max<int64_t>(x.size(order[i]), 1);
    }
    return at::empty_strided(x.sizes(), strides, x.options());
}

duo_heads heads_of(const Tensor& x) { return duo_heads{x.data_ptr(), x.stride(0), x.stride(1), x.stride(2)}; }

struct Shape {
    int64_t sink, window;
    double scale;
};

duo_window_attn_desc desc_of(const Tensor& q, const Tensor& k, const Shape& s, const Tensor& lengths) {
    duo_window_attn_desc d{};
    d.dtype = rope_dtype(q.scalar_type());
    d.batch = int32_t(q.size(0));
    d.num_q_heads = int32_t(q.size(1));
    d.num_kv_heads = int32_t(k.size(1));
    d.head_dim = int32_t(q.size(3));
    d.tokens = int32_t(q.size(2));
    d.sink = int32_t(s.sink);
    d.window = int32_t(s.window);
    d.scale = float(s.scale);
    d.lengths = lengths.defined() ? ints(lengths) : nullptr;
    return d;
}

struct WindowAttention : torch::autograd::Function<WindowAttention> {
    static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& q0, const Tensor& k0, const Tensor& v0,
                          const OptTensor& given, int64_t sink, int64_t window, double scale) {
        const Tensor lengths = given ? *given : Tensor();
        const c10::cuda::CUDAGuard guard(q0.device());
        const Tensor q = usable(q0), k = usable(k0), v = usable(v0);
        const duo_window_attn_desc d = desc_of(q, k, {sink, window, scale}, lengths);
        size_t bytes = 0;
        check(duo_window_attn_stats_bytes(&d, &bytes), "duo_window_attn");
        const Tensor out = like(q);
        const Tensor stats = at::empty({int64_t(bytes)}, q.options().dtype(at::kByte));
        const duo_heads hq = heads_of(q), hk = heads_of(k), hv = heads_of(v), ho = heads_of(out);
        check(duo_window_attn(&d, &hq, &hk, &hv, &ho, static_cast<float*>(stats.data_ptr()),
                              static_cast<int32_t*>(status_word(q.device()).data_ptr()), stream_of(q.device())),
              "duo_window_attn");
        ctx->save_for_backward({q, k, v, out, stats, lengths});
        ctx->saved_data["sink"] = sink;
        ctx->saved_data["window"] = window;
        ctx->saved_data["scale"] = scale;
        return out;
    }

    static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                   torch::autograd::variable_list grads) {
        const auto saved = ctx->get_saved_variables();
        const Tensor &q = saved[0], &k = saved[1], &v = saved[2], &out = saved[3], &stats = saved[4], &lengths = saved[5];
        const c10::cuda::CUDAGuard guard(q.device());
        check_captured_backward(q.device());
        torch::autograd::variable_list res(7);
        {
            const at::AutoGradMode off(false);
            const Tensor g = usable(grads[0]);
            const Shape s{ctx->saved_data["sink"].toInt(), ctx->saved_data["window"].toInt(),
                          ctx->saved_data["scale"].toDouble()};
            const duo_window_attn_desc d = desc_of(q, k, s, lengths);
            size_t bytes = 0;
            check(duo_window_attn_workspace_bytes(&d, &bytes), "duo_window_attn_grad");
            const Tensor dq = like(q), dk = like(k), dv = like(v);
            const Tensor ws = at::empty({int64_t(std::max<size_t>(bytes, 256))}, q.options().dtype(at::kByte));
            const duo_heads h[8] = {heads_of(q), heads_of(k),  heads_of(v),  heads_of(out),
                                    heads_of(g), heads_of(dq), heads_of(dk), heads_of(dv)};
            check(duo_window_attn_grad(&d, &h[0], &h[1], &h[2], &h[3], &h[4], static_cast<const float*>(stats.data_ptr()),
                                       &h[5], &h[6], &h[7], ws.data_ptr(), ws.numel(),
                                       static_cast<int32_t*>(status_word(q.device()).data_ptr()), stream_of(q.device())),
                  "duo_window_attn_grad");
            const Tensor* got[3] = {&dq, &dk, &dv};
            for (int i = 0; i < 3; ++i)
                if (ctx->needs_input_grad(i)) res[i] = *got[i];
        }
        if (at::GradMode::is_enabled()) {       // create_graph: the gradients exist, theirs do not
            torch::autograd::variable_list some;
            for (int i = 0; i < 3; ++i)
                if (res[i].defined()) some.push_back(res[i].set_requires_grad(true));
            const auto err = std::make_shared<torch::autograd::DelayedError>(
                "window_attention is differentiable once: its gradients have none", int64_t(some.size()));
            const auto marked = (*err)(std::move(some));
            for (int i = 0, j = 0; i < 3; ++i)
                if (res[i].defined()) res[i] = marked[j++];
        }
        return res;
    }
};

Tensor window_attention(const Tensor& q, const Tensor& k, const Tensor& v, int64_t sink, std::optional<int64_t> window,
                        const OptTensor& lengths, std::optional<double> given_scale) {
    const Tensor* in[3] = {&q, &k, &v};
    const char* names[3] = {"q", "k", "v"};
    check_not_traced("window_attention");
    for (int i = 0; i < 3; ++i) check_plain(*in[i], names[i]);
    for (int i = 0; i < 3; ++i) {
        const Tensor& t = *in[i];
        TORCH_CHECK_TYPE((t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf) &&
                             t.scalar_type() == q.scalar_type(),
                         names[i], ": dtype ", t.scalar_type(), ", expected bfloat16 or float16, the same for q, k and v");
        TORCH_CHECK_VALUE(t.is_cuda() && t.device() == q.device(), names[i], ": on ", t.device(),
                          ", expected one CUDA device for q, k and v");
        check_capture(t, names[i]);
        TORCH_CHECK_VALUE(t.dim() == 4, names[i], ": shape ", shape_of(t.sizes()), ", expected [batch][heads][tokens][128]");
    }
    const int64_t B = q.size(0), hq = q.size(1), T = q.size(2), d = q.size(3), n_kv = k.size(1);
    TORCH_CHECK_VALUE(k.sizes() == v.sizes() && k.size(0) == B && k.size(2) == T && k.size(3) == d, "k, v: shapes ",
                      shape_of(k.sizes()), ", ", shape_of(v.sizes()), ", expected (", B, ", key heads, ", T, ", ", d, ")");
    TORCH_CHECK_VALUE(d == 128, "heads of ", d, " elements, expected 128");
    TORCH_CHECK_VALUE(n_kv >= 1 && hq >= 1 && hq % n_kv == 0, hq, " query heads over ", n_kv, " key heads");
    TORCH_CHECK_VALUE(sink >= 0 && (!window || *window >= 1), "sink must be at least 0 and window at least 1 (or None)");
    if (lengths)
        TORCH_CHECK_VALUE(lengths->scalar_type() == at::kInt && lengths->device() == q.device() &&
                              lengths->sizes() == at::IntArrayRef({B}) && lengths->is_contiguous(),
                          "lengths must be contiguous int32 [", B, "] on the tensors' device");
    const double scale = given_scale ? *given_scale : 0.08838834764831845;      // 128 ** -0.5
    TORCH_CHECK_VALUE(scale > 0 && scale < 1e30, "scale must be above 0");
    const int64_t top = std::numeric_limits<int32_t>::max();
    TORCH_CHECK_VALUE(B <= top && T <= top && hq <= top, "too large a tensor");
    return WindowAttention::apply(q, k, v, lengths, std::min(sink, top),
                                  window ? std::min(*window, top) : int64_t(0), scale);
}

int64_t window_attention_status(int64_t device, bool clear) {
    const at::Device dev(at::kCUDA, at::DeviceIndex(device));
    const c10::cuda::CUDAGuard guard(dev);
    Tensor word = status_word(dev);
    const int64_t bits = word.item<int32_t>();
    if (clear) word.zero_();
    return bits;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    py::register_exception_translator([](std::exception_ptr e) {
        try {
            if (e) std::rethrow_exception(e);
        } catch (const DuoFailure& f) {
            const py::object type = py::module_::import("head_wise_kv_b200._lib").attr("DuoError");
            PyErr_SetObject(type.ptr(), type(f.code, f.what_call).ptr());
        }
    });
    m.def("rope_apply", &rope_apply);
    m.def("rope_launch", [](uintptr_t plan, int64_t d, const std::vector<std::tuple<Tensor, Tensor, bool>>& tensors,
                            const Tensor& positions, const OptTensor& n_new, bool transpose) {
        std::vector<RopeTask> tasks;
        for (const auto& [x, out, rotate] : tensors) tasks.push_back({&x, &out, rotate});
        rope_launch(plan, d, tasks.data(), tasks.size(), positions, n_new, transpose);
    });
    m.def("overlap", &overlap);
    m.def("overlaps_itself", &overlaps_itself);
    m.def("check_captured_backward", [](const Tensor& t) { check_captured_backward(t.device()); });
    m.def("check_recorded", [](const Tensor& t) {       // what an autograd function of Python's checks first
        check_not_traced("Rope.apply");
        check_plain(t, "x");
        check_capture(t, "x");
    });
    py::class_<Cache>(m, "Cache")
        .def(py::init<uintptr_t, int64_t, int64_t, int64_t, int64_t, int64_t>())
        .def("append_rope", &Cache::append_rope)
        .def("reserve", &Cache::reserve)
        .def("step_rope", &Cache::step_rope);
    m.def("window_attention", &window_attention);
    m.def("window_attention_status", &window_attention_status);
    m.def("status_word", [](int64_t device) { return status_word(at::Device(at::kCUDA, at::DeviceIndex(device))); });
}
