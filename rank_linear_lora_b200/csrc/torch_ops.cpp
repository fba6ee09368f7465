// torch_ops.cpp -- the operators around the LoRA layer for PyTorch: argument checks, outputs,
// workspaces and autograd nodes over the C entry points of include/lora_linear.h.  Host code
// only; every value is computed by the library's kernels.
//
// One token's projection is 18 us on the device and a training step of the head norms at 8192
// tokens 32 + 55 us; marshalled in Python they took the host 23 us and 182 us (an autograd function
// in Python that computes nothing takes 59 us by itself), so these operators are marshalled here:
// 12 us and 90 us.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <array>
#include <list>
#include <memory>
#include <mutex>
#include <optional>
#include <string>
#include <tuple>
#include <vector>

#include "lora_linear.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;

// A status of the library other than LORA_OK (LoraError in Python).
struct StatusError : std::runtime_error {
    int status;
    std::string where;
    StatusError(int s, const char *w)
        : std::runtime_error(std::string(w) + ": " + lora_status_string(static_cast<lora_status_t>(s))), status(s), where(w) {}
};

void check(lora_status_t s, const char *where) {
    if (s != LORA_OK) throw StatusError(s, where);
}

// ------------------------------------------------------------------ arguments
bool has(const OptTensor &t) { return t.has_value() && t->defined(); }
void *addr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
template <class T>
T *addr(const Tensor &t) { return static_cast<T *>(addr(t)); }
const uint16_t *bf16(const Tensor &t) { return addr<const uint16_t>(t); }
const uint16_t *bf16(const OptTensor &t) { return has(t) ? bf16(*t) : nullptr; }

std::string expected(at::ScalarType type, at::IntArrayRef shape, int dev, const Tensor &t) {
    std::ostringstream s;
    s << "expected a contiguous " << type << " tensor of shape " << shape << " on cuda:" << dev << ", the current device, got "
      << t.scalar_type() << " " << t.sizes() << " on " << t.device();
    return s.str();
}

// t contiguous, of this type and shape, on the current device.
void need(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == shape && t.is_contiguous(),
                      name, ": ", expected(type, shape, dev, t));
}
void need(const OptTensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    if (has(t)) need(*t, name, type, shape, dev);
}

// The frozen weight: bf16 [d_out, d_in], or codes with scales (and a codebook).
struct Weight {
    int format = 0;
    Tensor data, scale;
    std::array<float, 16> codebook{};
    int64_t d_out = 0, d_in = 0;

    int op(bool bwd) const { return 2 * format + bwd; }  // lora_op_t

    lora_weight_t c() const {
        lora_weight_t w;
        w.format = format;
        w.data = addr(data);
        w.scale = addr<uint16_t>(scale);
        w.codebook = format == LORA_W_NF4 ? codebook.data() : nullptr;
        return w;
    }
};
static_assert(LORA_OP_FWD_Q4 == 2 * LORA_W_Q4 && LORA_OP_FWD_FP8 == 2 * LORA_W_FP8 && LORA_OP_BWD_NF4 == 2 * LORA_W_NF4 + 1, "");

Weight make_weight(int64_t format, const Tensor &data, const OptTensor &scale, const std::vector<float> &codebook, int dev) {
    TORCH_CHECK_VALUE(data.dim() == 2, "W: expected a tensor [d_out, d_in], got shape ", data.sizes());
    Weight w;
    w.format = static_cast<int>(format);
    w.data = data;
    const bool packed = format == LORA_W_Q4 || format == LORA_W_NF4;
    w.d_out = data.size(0);
    w.d_in = data.size(1) * (packed ? 2 : 1);
    if (format == LORA_W_BF16) {
        need(data, "W", at::kBFloat16, {w.d_out, w.d_in}, dev);
        return w;
    }
    need(data, "W's codes", at::kByte, data.sizes(), dev);
    TORCH_CHECK_VALUE(has(scale), "W: codes need scales");
    w.scale = *scale;
    if (packed) need(w.scale, "W's scales", at::kBFloat16, {w.d_out, w.d_in / 64}, dev);
    else need(w.scale, "W's scales", at::kBFloat16, {w.d_out}, dev);
    if (format == LORA_W_NF4) {
        TORCH_CHECK_VALUE(codebook.size() == 16, "codebook: expected 16 values");
        std::copy(codebook.begin(), codebook.end(), w.codebook.begin());
    }
    return w;
}

// The library reads 16 bytes at a time: a tensor that starts elsewhere is copied (contiguous tensors
// keep their layout).  Frozen weights and the rotation's tables are not: a copy a call would hide
// what it costs, so the library refuses them.
Tensor on_16_bytes(const Tensor &t) {
    return t.defined() && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 ? t.clone() : t;
}
OptTensor on_16_bytes(const OptTensor &t) { return has(t) ? OptTensor(on_16_bytes(*t)) : t; }

Tensor new_bf16(const Tensor &like, at::IntArrayRef shape) { return at::empty(shape, like.options().dtype(at::kBFloat16)); }

// fp32 gradients of bf16 parameters next to each other, and all of them rounded to bf16 by one
// launch.  (Every size is a multiple of 8: A [r, d_in], B [d_out, r] and the bias [d_out].)
struct Grads {
    Tensor flat;
    std::vector<Tensor> like;

    explicit Grads(std::vector<Tensor> params) : like(std::move(params)) {
        int64_t n = 0;
        for (const Tensor &t : like) n += t.defined() ? t.numel() : 0;
        flat = at::empty({n}, like[0].options().dtype(at::kFloat));
    }
    float *operator[](size_t i) const {
        if (!like[i].defined()) return nullptr;
        int64_t at = 0;
        for (size_t j = 0; j < i; ++j) at += like[j].defined() ? like[j].numel() : 0;
        return flat.data_ptr<float>() + at;
    }
    variable_list rounded() const {
        const Tensor all = flat.to(at::kBFloat16);
        variable_list out;
        int64_t at = 0;
        for (const Tensor &t : like) {
            out.push_back(t.defined() ? all.narrow(0, at, t.numel()).view(t.sizes()) : Tensor());
            at += t.defined() ? t.numel() : 0;
        }
        return out;
    }
};

// ------------------------------------------------------------------ workspaces
// Kept per device, stream, shape and plan, so that calls on two streams never share one; under
// capture a new one from the graph's pool, so that two graphs can replay at the same time.  Two
// threads may call on one stream: a call holds its workspace's lock until all its kernels are
// enqueued, so that none of another call's, which would use the same workspace, come between them.
// No lock is held over an allocation or a release, which may want the interpreter's lock (a recorded
// stack) or wait for another thread, and the list's lock not over a launch, which may wait for the
// device.
struct Workspaces {
    using Key = std::tuple<int, void *, bool, int, int64_t, int64_t, int64_t, int, uint64_t>;
    struct Entry {
        Key key;
        Tensor ws;
        std::mutex mu;
        Entry(const Key &k, Tensor t) : key(k), ws(std::move(t)) {}
    };
    using List = std::list<std::shared_ptr<Entry>>;
    static constexpr size_t KEPT = 64;  // the least recently used goes first

    std::mutex mu;
    List kept;

    std::shared_ptr<Entry> find(const Key &key) {  // the list's lock is held
        for (auto it = kept.begin(); it != kept.end(); ++it)
            if ((*it)->key == key) {
                kept.splice(kept.begin(), kept, it);
                return kept.front();
            }
        return nullptr;
    }

    static Workspaces &all() {
        static Workspaces *const w = new Workspaces;  // never destroyed: tensors must not outlive the device at exit
        return *w;
    }
};

struct Lease {
    Tensor ws;
    std::shared_ptr<Workspaces::Entry> entry;  // null: a captured call's own
    std::unique_lock<std::mutex> lock;

    explicit Lease(Tensor own) : ws(std::move(own)) {}
    explicit Lease(std::shared_ptr<Workspaces::Entry> e) : ws(e->ws), entry(std::move(e)), lock(entry->mu) {}
    void *data() const { return ws.data_ptr(); }
    size_t bytes() const { return ws.nbytes(); }
};

// `layer`: the layer's own workspace (lora_linear_workspace_size), else lora_linear_act_workspace_size's.
Lease workspace(bool layer, int op, int64_t M, int64_t d_in, int64_t d_out, int r, const c10::cuda::CUDAStream &st) {
    Workspaces &w = Workspaces::all();
    auto make = [&] {
        const size_t n = layer ? lora_linear_workspace_size(op, M, d_in, d_out, r)
                               : lora_linear_act_workspace_size(op, M, d_in, d_out, r);
        TORCH_CHECK_VALUE(n > 0, "invalid sizes: ", M, " tokens, ", d_in, " -> ", d_out, ", rank ", r);
        const c10::InferenceMode off(false);  // kept beyond the mode of this call, and zeroed again outside it
        return at::zeros({static_cast<int64_t>(n)}, at::TensorOptions().dtype(at::kByte).device(st.device()));
    };
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return Lease(make());
    const Workspaces::Key key(st.device_index(), st.stream(), layer, op, M, d_in, d_out, r, lora_linear_plan_epoch());
    std::shared_ptr<Workspaces::Entry> known;
    {
        const std::lock_guard<std::mutex> lk(w.mu);
        known = w.find(key);
    }
    if (known) return Lease(std::move(known));
    auto fresh = std::make_shared<Workspaces::Entry>(key, make());
    // a workspace that goes returns to its stream's pool of the caching allocator, in stream order
    // behind the kernels that still use it
    Workspaces::List gone;
    {
        const std::lock_guard<std::mutex> lk(w.mu);
        if (auto e = w.find(key)) fresh.swap(e), gone.push_back(std::move(e));  // another thread was first
        else w.kept.push_front(fresh);
        while (w.kept.size() > Workspaces::KEPT) gone.splice(gone.end(), w.kept, std::prev(w.kept.end()));
    }
    gone.clear();  // before the lease's lock
    return Lease(std::move(fresh));
}

// The workspaces kept on the current device.
std::vector<std::shared_ptr<Workspaces::Entry>> kept_here() {
    const int dev = c10::cuda::current_device();
    Workspaces &w = Workspaces::all();
    std::vector<std::shared_ptr<Workspaces::Entry>> out;
    const std::lock_guard<std::mutex> lk(w.mu);
    for (const auto &e : w.kept)
        if (std::get<0>(e->key) == dev) out.push_back(e);
    return out;
}

// Waits for the device's work on every kept workspace and reads its error word.  One whose bounded
// wait ran out is zeroed whole, as lora_linear.h asks: a hand-over flag that came late must not meet
// the next call.
void check_workspaces() {
    lora_status_t worst = LORA_OK;
    for (const auto &e : kept_here()) {
        const std::lock_guard<std::mutex> lk(e->mu);  // no call enqueues on it meanwhile
        c10::cuda::device_synchronize();
        const lora_status_t s = lora_linear_check(e->ws.data_ptr(), c10::cuda::getCurrentCUDAStream().stream());
        if (s == LORA_OK) continue;
        worst = s;
        if (s != LORA_ERR_TIMEOUT) break;
        e->ws.zero_();
        c10::cuda::device_synchronize();
    }
    check(worst, "block.check_workspaces");
}

std::vector<Tensor> kept_workspaces() {
    std::vector<Tensor> out;
    for (const auto &e : kept_here()) out.push_back(e->ws);
    return out;
}

// ------------------------------------------------------------------ autograd
bool trained(const Tensor &t) { return t.requires_grad(); }
bool trained(const OptTensor &t) { return has(t) && t->requires_grad(); }
template <class... Ts>
bool wants_grad(const Ts &...ts) { return at::GradMode::is_enabled() && (trained(ts) || ...); }

// The operators have no forward-mode derivative, and forward mode is on under no_grad too: a result
// without its tangent would be a wrong one.
bool has_tangent(const Tensor &t) { return t.defined() && t._fw_grad(/*level=*/0).defined(); }
bool has_tangent(const OptTensor &t) { return has(t) && has_tangent(*t); }
template <class... Ts>
void no_tangents(const char *name, const Ts &...ts) {
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode())
        TORCH_CHECK_NOT_IMPLEMENTED(!(has_tangent(ts) || ...), name, ": derivatives in forward mode are not implemented");
}

// A tensor that a node keeps but does not save: a constant of the call (the frozen weight, the
// rotation's tables), which no hook on saved tensors should move to the host and back each step.  Like
// a saved one it must not change before the backward.
struct Constant {
    Tensor t;
    int64_t version = 0;

    Constant() = default;
    Constant(const Tensor &v) : t(v), version(now()) {}
    Constant(const OptTensor &v) : Constant(has(v) ? *v : Tensor()) {}
    int64_t now() const { return t.defined() && !t.is_inference() ? static_cast<int64_t>(t._version()) : 0; }
    const Tensor &unchanged(const char *name) const {
        TORCH_CHECK(now() == version, "one of the variables needed for gradient computation has been modified by an inplace "
                    "operation: ", name, " is at version ", now(), "; expected version ", version);
        return t;
    }
};

// What a node keeps besides its saved tensors.
struct Kept : torch::CustomClassHolder {
    Weight w;
    Constant data, scale, cos, sin;
    double alpha = 0, eps = 0;
    int act = 0;
    bool interleaved = false, norm = true, bias = false, residual = false;
    int64_t hq = 0, hk = 0, D = 0;
};
void keep(AutogradContext *ctx, c10::intrusive_ptr<Kept> k) { ctx->saved_data["kept"] = c10::IValue::make_capsule(std::move(k)); }
const Kept &kept(AutogradContext *ctx, c10::intrusive_ptr<torch::CustomClassHolder> &hold) {
    hold = ctx->saved_data["kept"].toCapsule();
    return static_cast<const Kept &>(*hold);
}

// The kernels' gradients have no graph of their own: where one is asked for (create_graph),
// differentiating through them is an error, not a term that is silently missing.  They depend on the
// saved tensors too, so an upstream gradient that is a constant changes nothing.
variable_list once(variable_list grads) {
    if (!at::GradMode::is_enabled()) return grads;
    for (Tensor &t : grads)
        if (t.defined()) t = t.detach().requires_grad_(true);
    auto err = std::make_shared<torch::autograd::DelayedError>(
        "trying to differentiate twice a function that can be differentiated once", static_cast<int64_t>(grads.size()));
    return (*err)(std::move(grads));
}

// ------------------------------------------------------------------ gated projections
struct GluOut {
    Tensor p, gu, xa;
};
GluOut glu_forward(const Tensor &x, const Tensor &A, const Tensor &B, double alpha, const Weight &w, int act, bool save) {
    const int dev = c10::cuda::current_device();
    const int64_t M = x.size(0), r = A.size(0), n = w.d_out;
    TORCH_CHECK_VALUE(n % 2 == 0, "W: the gate's and the up projection's rows, got ", n);
    need(x, "x", at::kBFloat16, {M, w.d_in}, dev);
    need(A, "A", at::kBFloat16, {r, w.d_in}, dev);
    need(B, "B", at::kBFloat16, {n, r}, dev);
    GluOut o;
    o.p = new_bf16(x, {M, n / 2});
    if (save) {
        o.gu = new_bf16(x, {M, n});
        o.xa = new_bf16(x, {M, r});
    }
    if (M > 0) {
        const auto st = c10::cuda::getCurrentCUDAStream(dev);
        const Lease ws = workspace(false, w.op(false), M, w.d_in, n, static_cast<int>(r), st);
        const lora_weight_t cw = w.c();
        check(lora_glu_fwd(bf16(x), &cw, bf16(A), bf16(B), addr<uint16_t>(o.p), addr<uint16_t>(o.gu), addr<uint16_t>(o.xa), M,
                           w.d_in, n / 2, static_cast<int>(r), static_cast<float>(alpha), act, ws.data(), ws.bytes(),
                           st.stream()),
              "lora_glu_fwd");
    }
    return o;
}

// p = act(g) * u, [g | u] = x.w^T + (alpha / r).(x.A^T).B^T
struct Glu : torch::autograd::Function<Glu> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Tensor &A, const Tensor &B, double alpha,
                          const Weight &w, int64_t act) {
        GluOut o = glu_forward(x, A, B, alpha, w, static_cast<int>(act), true);
        ctx->save_for_backward({x, A, B, o.xa, o.gu});
        auto k = c10::make_intrusive<Kept>();
        k->w = w;
        k->data = w.data;
        k->scale = w.scale;
        k->alpha = alpha;
        k->act = static_cast<int>(act);
        keep(ctx, std::move(k));
        return o.p;
    }

    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list s = ctx->get_saved_variables();
        c10::intrusive_ptr<torch::CustomClassHolder> hold;
        const Kept &k = kept(ctx, hold);
        k.data.unchanged("the frozen weight");
        k.scale.unchanged("the frozen weight's scales");
        const Tensor &x = s[0], &A = s[1], &B = s[2], &xa = s[3], &gu = s[4];
        const int dev = c10::cuda::current_device();
        const int64_t M = x.size(0), r = A.size(0), n = k.w.d_out;
        Tensor dX = ctx->needs_input_grad(0) ? at::empty_like(x) : Tensor();
        if (M == 0) return once({dX, at::zeros_like(A), at::zeros_like(B), Tensor(), Tensor(), Tensor()});
        const Tensor dP = on_16_bytes(up[0].contiguous());
        need(dP, "the gradient of p", at::kBFloat16, {M, n / 2}, dev);
        const Grads d({A, B});
        const Tensor dGU = at::empty_like(gu);
        const auto st = c10::cuda::getCurrentCUDAStream(dev);
        const lora_weight_t cw = k.w.c();
        {
            const Lease ws = workspace(true, k.w.op(true), M, k.w.d_in, n, static_cast<int>(r), st);
            check(lora_glu_bwd(bf16(dP), bf16(gu), bf16(x), &cw, bf16(A), bf16(B), bf16(xa), addr<uint16_t>(dGU),
                               addr<uint16_t>(dX), d[0], d[1], M, k.w.d_in, n / 2, static_cast<int>(r),
                               static_cast<float>(k.alpha), k.act, ws.data(), ws.bytes(), st.stream()),
                  "lora_glu_bwd");
        }
        const variable_list g = d.rounded();
        return once({dX, g[0], g[1], Tensor(), Tensor(), Tensor()});
    }
};

Tensor glu(const Tensor &x_in, const Tensor &A_in, const Tensor &B_in, double alpha, int64_t act, int64_t format,
           const Tensor &data, const OptTensor &scale, const std::vector<float> &codebook) {
    no_tangents("lora_glu", x_in, A_in, B_in, data, scale);
    const Tensor x = on_16_bytes(x_in), A = on_16_bytes(A_in), B = on_16_bytes(B_in);
    const Weight w = make_weight(format, data, scale, codebook, c10::cuda::current_device());
    if (wants_grad(x, A, B))
        return Glu::apply(x, A, B, alpha, w, act);
    return glu_forward(x, A, B, alpha, w, static_cast<int>(act), false).p;
}

// ------------------------------------------------------------------ projection with an epilogue
struct ActOut {
    Tensor out, pre, xa;
};
ActOut act_forward(const Tensor &x, const Tensor &A, const Tensor &B, const OptTensor &bias, const OptTensor &residual,
                   double alpha, const Weight &w, int act, bool save) {
    const int dev = c10::cuda::current_device();
    const int64_t M = x.size(0), r = A.size(0), n = w.d_out;
    need(x, "x", at::kBFloat16, {M, w.d_in}, dev);
    need(A, "A", at::kBFloat16, {r, w.d_in}, dev);
    need(B, "B", at::kBFloat16, {n, r}, dev);
    need(bias, "bias", at::kBFloat16, {n}, dev);
    need(residual, "residual", at::kBFloat16, {M, n}, dev);
    ActOut o;
    o.out = new_bf16(x, {M, n});
    if (save) {
        if (act != LORA_ACT_NONE) o.pre = new_bf16(x, {M, n});
        o.xa = new_bf16(x, {M, r});
    }
    if (M > 0) {
        const auto st = c10::cuda::getCurrentCUDAStream(dev);
        const Lease ws = workspace(false, w.op(false), M, w.d_in, n, static_cast<int>(r), st);
        const lora_weight_t cw = w.c();
        check(lora_linear_act_fwd(bf16(x), &cw, bf16(A), bf16(B), bf16(bias), bf16(residual), addr<uint16_t>(o.out),
                                  addr<uint16_t>(o.pre), addr<uint16_t>(o.xa), M, w.d_in, n, static_cast<int>(r),
                                  static_cast<float>(alpha), act, ws.data(), ws.bytes(), st.stream()),
              "lora_linear_act_fwd");
    }
    return o;
}

// out = act(x.w^T + (alpha / r).(x.A^T).B^T + bias) + residual
struct LinearAct : torch::autograd::Function<LinearAct> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Tensor &A, const Tensor &B, const OptTensor &bias,
                          const OptTensor &residual, double alpha, const Weight &w, int64_t act) {
        ActOut o = act_forward(x, A, B, bias, residual, alpha, w, static_cast<int>(act), true);
        ctx->save_for_backward({x, A, B, o.xa, o.pre, has(bias) ? *bias : Tensor()});
        auto k = c10::make_intrusive<Kept>();
        k->w = w;
        k->data = w.data;
        k->scale = w.scale;
        k->alpha = alpha;
        k->act = static_cast<int>(act);
        k->bias = has(bias);
        k->residual = has(residual);
        keep(ctx, std::move(k));
        return o.out;
    }

    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list s = ctx->get_saved_variables();
        c10::intrusive_ptr<torch::CustomClassHolder> hold;
        const Kept &k = kept(ctx, hold);
        k.data.unchanged("the frozen weight");
        k.scale.unchanged("the frozen weight's scales");
        const Tensor &x = s[0], &A = s[1], &B = s[2], &xa = s[3], &pre = s[4], &bias = s[5];
        const int dev = c10::cuda::current_device();
        const int64_t M = x.size(0), r = A.size(0), n = k.w.d_out;
        // needs_input_grad counts the tensors that were given
        const bool want_bias = k.bias && ctx->needs_input_grad(3);
        const bool want_res = k.residual && ctx->needs_input_grad(3 + k.bias);
        Tensor dX = ctx->needs_input_grad(0) ? at::empty_like(x) : Tensor(), dRes = want_res ? up[0] : Tensor();
        if (M == 0)
            return once({dX, at::zeros_like(A), at::zeros_like(B), want_bias ? at::zeros_like(bias) : Tensor(), dRes, Tensor(),
                         Tensor(), Tensor()});
        const Tensor dOut = on_16_bytes(up[0].contiguous());
        need(dOut, "the gradient of out", at::kBFloat16, {M, n}, dev);
        const Grads d({A, B, want_bias ? bias : Tensor()});
        const Tensor dPre = k.act != LORA_ACT_NONE ? at::empty_like(dOut) : Tensor();
        const auto st = c10::cuda::getCurrentCUDAStream(dev);
        const lora_weight_t cw = k.w.c();
        {
            const Lease ws = workspace(false, k.w.op(true), M, k.w.d_in, n, static_cast<int>(r), st);
            check(lora_linear_act_bwd(bf16(dOut), bf16(pre), bf16(x), &cw, bf16(A), bf16(B), bf16(xa), addr<uint16_t>(dPre),
                                      addr<uint16_t>(dX), d[0], d[1], d[2], M, k.w.d_in, n, static_cast<int>(r),
                                      static_cast<float>(k.alpha), k.act, ws.data(), ws.bytes(), st.stream()),
                  "lora_linear_act_bwd");
        }
        const variable_list g = d.rounded();
        return once({dX, g[0], g[1], g[2], dRes, Tensor(), Tensor(), Tensor()});
    }
};

Tensor linear_act(const Tensor &x_in, const Tensor &A_in, const Tensor &B_in, const OptTensor &bias_in,
                  const OptTensor &residual_in, double alpha, int64_t act, int64_t format, const Tensor &data,
                  const OptTensor &scale, const std::vector<float> &codebook) {
    no_tangents("lora_linear_act", x_in, A_in, B_in, bias_in, residual_in, data, scale);
    const Tensor x = on_16_bytes(x_in), A = on_16_bytes(A_in), B = on_16_bytes(B_in);
    const OptTensor bias = on_16_bytes(bias_in), residual = on_16_bytes(residual_in);
    const Weight w = make_weight(format, data, scale, codebook, c10::cuda::current_device());
    if (wants_grad(x, A, B, bias, residual))
        return LinearAct::apply(x, A, B, bias, residual, alpha, w, act);
    return act_forward(x, A, B, bias, residual, alpha, w, static_cast<int>(act), false).out;
}

// ------------------------------------------------------------------ norms of q and k with the rotation
int head_type(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return LORA_T_BF16;
        case at::kHalf: return LORA_T_FP16;
        case at::kFloat: return LORA_T_FP32;
        default: TORCH_CHECK_VALUE(false, "q, k: bfloat16, float16 or float32, got ", t.scalar_type());
    }
}

// t [M, heads, D] itself if the library's strides can name it, else a contiguous copy: strides of
// whole 16-byte units, tokens outside heads or heads outside tokens (what names an element twice, or
// might, can still be read as an input).
Tensor addressable(const Tensor &t) {
    if (t.dim() != 3) return t;
    const int64_t M = t.size(0), H = t.size(1), D = t.size(2), unit = 16 / t.element_size();
    const int64_t ts = M > 1 ? t.stride(0) : 0, hs = H > 1 ? t.stride(1) : 0;
    auto named = [&](int64_t n, int64_t stride) { return n <= 1 || (stride >= D && stride % unit == 0); };
    const bool apart = M <= 1 || H <= 1 || ts >= (H - 1) * hs + D || hs >= (M - 1) * ts + D;
    if (t.stride(2) == 1 && named(M, ts) && named(H, hs) && apart && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0)
        return t;
    return on_16_bytes(t.contiguous());
}

lora_heads_t heads(const Tensor &t, const char *name, const Tensor &like, int dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == like.scalar_type() && t.sizes() == like.sizes() && t.stride(2) == 1 && t.is_cuda() &&
                          t.get_device() == dev,
                      name, ": expected a ", like.scalar_type(), " tensor ", like.sizes(), " on cuda:", dev,
                      ", the current device, its last dimension contiguous, got ", t.scalar_type(), " ", t.sizes(),
                      " with strides ", t.strides(), " on ", t.device());
    lora_heads_t h;
    h.data = addr(t);
    h.token_stride = t.stride(0);
    h.head_stride = t.stride(1);
    h.heads = static_cast<int32_t>(t.size(1));
    return h;
}

struct Rope {
    const float *cos = nullptr, *sin = nullptr;
    const int64_t *positions = nullptr;
    int64_t n_pos = 0;
    int rot = 0;
};
Rope rope(const OptTensor &cos, const OptTensor &sin, const OptTensor &positions, int64_t M, int dev) {
    Rope t;
    if (!has(cos)) return t;
    TORCH_CHECK_VALUE(has(sin) && has(positions) && cos->dim() == 2, "cos, sin [n_pos, rot / 2] and positions go together");
    need(*cos, "cos", at::kFloat, cos->sizes(), dev);
    need(*sin, "sin", at::kFloat, cos->sizes(), dev);
    need(*positions, "positions", at::kLong, {M}, dev);
    t.cos = addr<float>(*cos);
    t.sin = addr<float>(*sin);
    t.positions = addr<int64_t>(*positions);
    t.n_pos = cos->size(0);
    t.rot = static_cast<int>(2 * cos->size(1));
    return t;
}

std::pair<Tensor, Tensor> heads_forward(const Tensor &q, const Tensor &k, const OptTensor &wq, const OptTensor &wk,
                                        const OptTensor &cos, const OptTensor &sin, const OptTensor &positions, double eps,
                                        bool interleaved, bool norm) {
    const int dev = c10::cuda::current_device();
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3 && k.size(0) == q.size(0) && k.size(2) == q.size(2),
                      "q, k: expected [tokens, heads, D] of the same tokens and D, got ", q.sizes(), " and ", k.sizes());
    const int64_t M = q.size(0), D = q.size(2);
    TORCH_CHECK_VALUE(k.scalar_type() == q.scalar_type(), "k: ", k.scalar_type(), ", q: ", q.scalar_type());
    const int type = head_type(q);
    need(wq, "q_weight", q.scalar_type(), {D}, dev);
    need(wk, "k_weight", q.scalar_type(), {D}, dev);
    const Rope t = rope(cos, sin, positions, M, dev);
    const lora_heads_t qi = heads(q, "q", q, dev), ki = heads(k, "k", k, dev);
    Tensor q_out = at::empty(q.sizes(), q.options()), k_out = at::empty(k.sizes(), k.options());
    if (M > 0) {
        const lora_heads_t qo = heads(q_out, "q_out", q, dev), ko = heads(k_out, "k_out", k, dev);
        check(lora_qk_norm_rope_fwd(type, &qi, &ki, has(wq) ? addr(*wq) : nullptr, has(wk) ? addr(*wk) : nullptr, t.cos, t.sin,
                                    t.positions, t.n_pos, &qo, &ko, M, static_cast<int>(D), t.rot, interleaved, norm,
                                    static_cast<float>(eps), c10::cuda::getCurrentCUDAStream(dev).stream()),
              "lora_qk_norm_rope_fwd");
    }
    return {q_out, k_out};
}

// dq, dk and the weights' gradients from up[0], up[1]; the saved tensors from s[at] on are the
// weights and positions.  `edge`: the first weight's place among the tensors that were
// given, which needs_input_grad counts.
std::pair<Tensor, Tensor> heads_backward(AutogradContext *ctx, const Kept &kp, const variable_list &up, const Tensor &q,
                                         const Tensor &k, const variable_list &s, size_t at, int edge, const Tensor &dq,
                                         const Tensor &dk) {
    const Tensor &wq = s[at], &wk = s[at + 1];
    const int dev = c10::cuda::current_device();
    const int64_t M = q.size(0), D = q.size(2);
    Tensor dwq, dwk;
    if (wq.defined() && ctx->needs_input_grad(edge++)) dwq = M ? at::empty_like(wq) : at::zeros_like(wq);
    if (wk.defined() && ctx->needs_input_grad(edge++)) dwk = M ? at::empty_like(wk) : at::zeros_like(wk);
    if (M > 0) {
        const Tensor dqo = addressable(up[0]), dko = addressable(up[1]);
        const Rope t = rope(kp.cos.unchanged("cos"), kp.sin.unchanged("sin"), s[at + 2], M, dev);
        const lora_heads_t qi = heads(q, "q", q, dev), ki = heads(k, "k", k, dev), gq = heads(dqo, "the gradient of q", q, dev),
                           gk = heads(dko, "the gradient of k", k, dev), qo = heads(dq, "dq", q, dev),
                           ko = heads(dk, "dk", k, dev);
        Tensor ws;
        if (dwq.defined() || dwk.defined())
            ws = at::empty({static_cast<int64_t>(lora_qk_norm_rope_workspace_size(M, static_cast<int>(q.size(1) + k.size(1)),
                                                                                  static_cast<int>(D)))},
                           q.options().dtype(at::kByte));
        check(lora_qk_norm_rope_bwd(head_type(q) | LORA_T_WEIGHT_GRADS, &gq, &gk, &qi, &ki, addr(wq), addr(wk), t.cos, t.sin,
                                    t.positions, t.n_pos, &qo, &ko, addr(dwq), addr(dwk), M, static_cast<int>(D), t.rot,
                                    kp.interleaved, kp.norm, static_cast<float>(kp.eps), addr(ws), ws.defined() ? ws.nbytes() : 0,
                                    c10::cuda::getCurrentCUDAStream(dev).stream()),
              "lora_qk_norm_rope_bwd");
    }
    return {dwq, dwk};
}

struct QkNormRope : torch::autograd::Function<QkNormRope> {
    static variable_list forward(AutogradContext *ctx, const Tensor &q, const Tensor &k, const OptTensor &wq,
                                 const OptTensor &wk, const OptTensor &cos, const OptTensor &sin, const OptTensor &positions,
                                 double eps, bool interleaved, bool norm) {
        auto o = heads_forward(q, k, wq, wk, cos, sin, positions, eps, interleaved, norm);
        auto t = [](const OptTensor &v) { return has(v) ? *v : Tensor(); };
        ctx->save_for_backward({q, k, t(wq), t(wk), t(positions)});
        auto kp = c10::make_intrusive<Kept>();
        kp->cos = cos;
        kp->sin = sin;
        kp->eps = eps;
        kp->interleaved = interleaved;
        kp->norm = norm;
        keep(ctx, std::move(kp));
        return {o.first, o.second};
    }

    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list s = ctx->get_saved_variables();
        c10::intrusive_ptr<torch::CustomClassHolder> hold;
        const Kept &kp = kept(ctx, hold);
        const Tensor &q = s[0], &k = s[1];
        const Tensor dq = at::empty(q.sizes(), q.options()), dk = at::empty(k.sizes(), k.options());
        const auto dw = heads_backward(ctx, kp, up, q, k, s, 2, 2, dq, dk);
        return once({dq, dk, dw.first, dw.second, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()});
    }
};

// The same on the stacked projection h [M, (hq + 2 hk) D] = [q | k | v]: v is a view of h, and the
// backward writes dq and dk straight into their columns of one dh.
std::array<Tensor, 3> split_heads(const Tensor &h, int64_t hq, int64_t hk, int64_t D) {
    const int64_t M = h.size(0), row = h.stride(0);
    auto part = [&](int64_t col, int64_t n) { return h.narrow(1, col, n * D).as_strided({M, n, D}, {row, D, 1}); };
    return {part(0, hq), part(hq * D, hk), part((hq + hk) * D, hk)};
}

struct QkvHeads : torch::autograd::Function<QkvHeads> {
    static variable_list forward(AutogradContext *ctx, const Tensor &h, const OptTensor &wq, const OptTensor &wk,
                                 const OptTensor &cos, const OptTensor &sin, const OptTensor &positions, int64_t hq,
                                 int64_t hk, int64_t D, double eps, bool interleaved, bool norm) {
        auto qkv = split_heads(h, hq, hk, D);
        auto o = heads_forward(qkv[0], qkv[1], wq, wk, cos, sin, positions, eps, interleaved, norm);
        auto t = [](const OptTensor &v) { return has(v) ? *v : Tensor(); };
        ctx->save_for_backward({h, t(wq), t(wk), t(positions)});
        auto kp = c10::make_intrusive<Kept>();
        kp->cos = cos;
        kp->sin = sin;
        kp->eps = eps;
        kp->interleaved = interleaved;
        kp->norm = norm;
        kp->hq = hq;
        kp->hk = hk;
        kp->D = D;
        keep(ctx, std::move(kp));
        return {o.first, o.second, qkv[2]};
    }

    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list s = ctx->get_saved_variables();
        c10::intrusive_ptr<torch::CustomClassHolder> hold;
        const Kept &kp = kept(ctx, hold);
        const auto in = split_heads(s[0], kp.hq, kp.hk, kp.D);
        const Tensor dh = at::empty_like(s[0]);
        const auto d = split_heads(dh, kp.hq, kp.hk, kp.D);
        d[2].copy_(up[2]);
        const auto dw = heads_backward(ctx, kp, up, in[0], in[1], s, 1, 1, d[0], d[1]);
        variable_list out(12);
        out[0] = dh;
        out[1] = dw.first;
        out[2] = dw.second;
        return once(std::move(out));
    }
};

std::pair<Tensor, Tensor> qk_norm_rope(const Tensor &q_in, const Tensor &k_in, const OptTensor &wq_in, const OptTensor &wk_in,
                                       const OptTensor &cos, const OptTensor &sin, const OptTensor &positions, double eps,
                                       bool interleaved, bool norm) {
    no_tangents("qk_norm_rope", q_in, k_in, wq_in, wk_in, cos, sin);
    const Tensor q = addressable(q_in), k = addressable(k_in);
    const OptTensor wq = on_16_bytes(wq_in), wk = on_16_bytes(wk_in);
    if (wants_grad(q, k, wq, wk)) {
        const variable_list o = QkNormRope::apply(q, k, wq, wk, cos, sin, positions, eps, interleaved, norm);
        return {o[0], o[1]};
    }
    return heads_forward(q, k, wq, wk, cos, sin, positions, eps, interleaved, norm);
}

std::tuple<Tensor, Tensor, Tensor> qkv_heads(const Tensor &h_in, const OptTensor &wq_in, const OptTensor &wk_in,
                                             const OptTensor &cos, const OptTensor &sin, const OptTensor &positions,
                                             int64_t hq, int64_t hk, int64_t D, double eps, bool interleaved, bool norm) {
    no_tangents("qkv_heads", h_in, wq_in, wk_in, cos, sin);
    const Tensor h = on_16_bytes(h_in);
    const OptTensor wq = on_16_bytes(wq_in), wk = on_16_bytes(wk_in);
    TORCH_CHECK_VALUE(h.dim() == 2 && hq > 0 && hk > 0 && D > 0 && h.size(1) == (hq + 2 * hk) * D, "h: expected ",
                      (hq + 2 * hk) * D, " columns, got ", h.sizes());
    if (wants_grad(h, wq, wk)) {
        const variable_list o = QkvHeads::apply(h, wq, wk, cos, sin, positions, hq, hk, D, eps, interleaved, norm);
        return {o[0], o[1], o[2]};
    }
    const auto qkv = split_heads(h, hq, hk, D);
    const auto o = heads_forward(qkv[0], qkv[1], wq, wk, cos, sin, positions, eps, interleaved, norm);
    return {o.first, o.second, qkv[2]};
}

}  // namespace

PYBIND11_MODULE(_ops, m) {
    m.doc() = "The operators around the LoRA layer over liblora_linear.so, with autograd.";
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError &e) {
            const py::object type = py::module_::import("rank_linear_lora_b200.lora_linear").attr("LoraError");
            const py::object value = type(e.status, e.where);
            PyErr_SetObject(type.ptr(), value.ptr());
        }
    });
    m.def("check_workspaces", &check_workspaces, py::call_guard<py::gil_scoped_release>());
    m.def("kept_workspaces", &kept_workspaces, py::call_guard<py::gil_scoped_release>());
    m.def("glu", &glu, py::call_guard<py::gil_scoped_release>());
    m.def("linear_act", &linear_act, py::call_guard<py::gil_scoped_release>());
    m.def("qk_norm_rope", &qk_norm_rope, py::call_guard<py::gil_scoped_release>());
    m.def("qkv_heads", &qkv_heads, py::call_guard<py::gil_scoped_release>());
}
