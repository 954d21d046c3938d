// Part of wtconv_tok_torch.cpp: layer norm, the gated recurrence, and experts'
// rows and products.
#pragma once

namespace {

// ================================================================== kernels
// t [n, C] whose rows start at multiples of 16 bytes no further apart than the products take; a copy where they do not.
Tensor aligned_rows(const Tensor& t) {
    const int64_t unit = 16 / t.element_size();
    if (dense(t) && t.stride(0) % unit == 0 && t.stride(0) <= WTC_EXPERT_MAX_STRIDE &&
        reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0)
        return t;
    return t.clone(at::MemoryFormat::Contiguous);
}
Tensor aligned(const Tensor& t) {
    return reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0 ? t : t.clone(at::MemoryFormat::Contiguous);
}
Tensor dense_rows(const Tensor& t) { return dense(t) ? t : t.contiguous(); }
float* floats(const Tensor& t) { return static_cast<float*>(out(t)); }
int* ints(const Tensor& t) { return static_cast<int*>(out(t)); }
OptTensor some(const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; }

namespace op {

// ------------------------------------------------------------------ layer norm
struct Layer {
    Tensor y, h, stats;
};
Layer layer_forward(const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual, double eps,
                    bool keep) {
    TORCH_CHECK_VALUE(x.dim() >= 1, "x has no axis");
    check_residual(x, residual);
    const int dtype = activation(x, "x", -1);
    const int C = narrow(x.size(-1), "channels of x");
    check(weight, "weight", at::kFloat, x, {C});
    if (bias) check(*bias, "bias", at::kFloat, x, {C});
    const Tensor xr = rows(x), rr = residual ? rows(*residual) : Tensor();
    const int64_t n = xr.size(0);
    Layer o;
    o.y = empty(x.sizes(), x);
    if (residual) o.h = empty(x.sizes(), x);
    if (keep) o.stats = empty({n, 2}, x, at::kFloat);
    const wtc_layer_desc d = {n, xr.stride(0), residual ? rr.stride(0) : 0, 0, C, dtype, (float)eps};
    const On on(x);
    raise_on(wtconv_layer_norm_forward(&d, in(xr), in(rr), in_as<float>(weight), bias ? in_as<float>(*bias) : nullptr, out(o.y),
                                       out(o.h), floats(o.stats), on.stream),
             "wtconv_layer_norm_forward");
    return o;
}
// [y], or [y, h] with a residual
Tensors layer_norm(const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual, double eps) {
    const Layer o = layer_forward(x, weight, bias, residual, eps, false);
    return residual ? Tensors{o.y, o.h} : Tensors{o.y};
}
// [stats, y], or [stats, y, h]
Tensors _layer_norm_forward(const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual,
                            double eps) {
    const Layer o = layer_forward(x, weight, bias, residual, eps, true);
    return residual ? Tensors{o.stats, o.y, o.h} : Tensors{o.stats, o.y};
}
// [dx, dw], or [dx, dw, db]; h: what was normed (x without a residual)
Tensors _layer_norm_backward(const Tensor& dy0, const OptTensor& dh0, const Tensor& h0, const Tensor& weight,
                             const Tensor& stats, bool bias) {
    TORCH_CHECK_VALUE(h0.dim() >= 1, "h has no axis");
    const int dtype = activation(h0, "h", -1);
    const int C = narrow(h0.size(-1), "channels of h");
    check(weight, "weight", at::kFloat, h0, {C});
    check_like(dy0, "dy", h0);
    if (dh0) check_like(*dh0, "dh", h0);
    const Tensor h = rows(h0), dy = rows(dy0), dh = dh0 ? rows(*dh0).contiguous() : Tensor();
    const int64_t n = h.size(0);
    check(stats, "stats", at::kFloat, h0, {n, 2});
    const wtc_layer_desc d = {n, h.stride(0), 0, dy.stride(0), C, dtype, 0.f};
    const size_t bytes = wtconv_layer_norm_backward_workspace(&d);
    const Tensor dx = empty(h0.sizes(), h), dw = empty({C}, h, at::kFloat), db = bias ? empty({C}, h, at::kFloat) : Tensor(),
                 ws = workspace(bytes, h);
    const On on(h);
    raise_on(wtconv_layer_norm_backward(&d, in(dy), in(dh), in(h), in_as<float>(weight), in_as<float>(stats), out(dx), floats(dw),
                                        floats(db), out(ws), bytes, on.stream),
             "wtconv_layer_norm_backward");
    return bias ? Tensors{dx, dw, db} : Tensors{dx, dw};
}

// ------------------------------------------------------------------ gated recurrence
wtc_scan_desc scan_desc(const Tensor& x, const Tensor& gate, const Tensor& cu, bool reverse) {
    const int dtype = activation(x, "x", 2);
    check_like(gate, "gate", x);
    cu_check(cu, x);
    return {x.size(0), x.stride(0), gate.stride(0), 0, sequences(cu), narrow(x.size(1), "channels of x"), dtype, reverse};
}
// a state [n, C], or its gradient, as the kernels read it; undefined if there is none
Tensor state_of(const OptTensor& t, const char* name, const Tensor& x, const Tensor& cu) {
    if (!t) return Tensor();
    check(*t, name, at::kFloat, x, {cu.size(0) - 1, x.size(1)}, false);
    return t->contiguous();
}
Tensors scan_forward(const Tensor& x0, const Tensor& gate0, const Tensor& cu, const OptTensor& state0, bool reverse, bool keep) {
    scan_desc(x0, gate0, cu, reverse);
    const Tensor x = dense_rows(x0), gate = dense_rows(gate0), state = state_of(state0, "state", x0, cu);
    const wtc_scan_desc d = scan_desc(x, gate, cu, reverse);
    const size_t bytes = wtconv_gated_scan_workspace(&d), kept = keep ? wtconv_gated_scan_kept(&d) : 0;
    const Tensor y = empty(x.sizes(), x), last = empty({d.n_seq, d.C}, x, at::kFloat),
                 k = keep ? empty({(int64_t)(kept / sizeof(float))}, x, at::kFloat) : Tensor(), ws = workspace(bytes, x);
    const On on(x);
    raise_on(wtconv_gated_scan_forward(&d, in(x), in(gate), in_as<int>(cu), in_as<float>(state), out(y),
                                       floats(last), floats(k), out(ws), bytes, on.stream),
             "wtconv_gated_scan_forward");
    return keep ? Tensors{y, last, k} : Tensors{y, last};
}
// [y, last]
Tensors gated_scan(const Tensor& x, const Tensor& gate, const Tensor& cu, const OptTensor& state, bool reverse) {
    return scan_forward(x, gate, cu, state, reverse, false);
}
// [y, last, kept]
Tensors _gated_scan_forward(const Tensor& x, const Tensor& gate, const Tensor& cu, const OptTensor& state, bool reverse) {
    return scan_forward(x, gate, cu, state, reverse, true);
}
// [dx, dgate], or [dx, dgate, dstate] with a state
Tensors _gated_scan_backward(const Tensor& dy0, const OptTensor& dlast0, const Tensor& x0, const Tensor& gate0, const Tensor& cu,
                             const OptTensor& state0, const Tensor& kept, bool reverse) {
    scan_desc(x0, gate0, cu, reverse);
    check_like(dy0, "dy", x0);
    const Tensor state = state_of(state0, "state", x0, cu), dlast = state_of(dlast0, "dlast", x0, cu);
    const Tensor x = dense_rows(x0), gate = dense_rows(gate0), dy = dense_rows(dy0);
    wtc_scan_desc d = scan_desc(x, gate, cu, reverse);
    d.g_stride = dy.stride(0);
    check(kept, "kept", at::kFloat, x, {(int64_t)(wtconv_gated_scan_kept(&d) / sizeof(float))});
    const size_t bytes = wtconv_gated_scan_workspace(&d);
    const Tensor dx = empty(x.sizes(), x), dgate = empty(x.sizes(), x), ws = workspace(bytes, x),
                 dstate = state0 ? empty({d.n_seq, d.C}, x, at::kFloat) : Tensor();
    const On on(x);
    raise_on(wtconv_gated_scan_backward(&d, in(x), in(gate), in_as<int>(cu), in_as<float>(state), in_as<float>(kept), in(dy),
                                        in_as<float>(dlast), out(dx), out(dgate),
                                        floats(dstate), out(ws), bytes, on.stream),
             "wtconv_gated_scan_backward");
    return state0 ? Tensors{dx, dgate, dstate} : Tensors{dx, dgate};
}
// `to`, contiguous, may be t itself, but no part of one of t's rows.  PyTorch does not say so of rows that are apart.
void check_apart(const Tensor& to, const Tensor& t) {
    at::assert_no_partial_overlap(to, t);
    if (t.numel() == 0 || !dense(t) || (t.is_contiguous() && t.const_data_ptr() == to.const_data_ptr())) return;
    // rows number `from` up to `end` have a byte in to's
    const int64_t step = t.stride(0) * t.element_size(), length = t.size(1) * t.element_size(), bytes = to.numel() * to.element_size(),
                  at = reinterpret_cast<intptr_t>(to.const_data_ptr()) - reinterpret_cast<intptr_t>(t.const_data_ptr());
    const int64_t rows = step > 0 ? t.size(0) : 1, from = at < length ? 0 : step > 0 ? (at - length) / step + 1 : 1,
                  end = at + bytes <= 0 ? 0 : step > 0 ? std::min(rows, (at + bytes - 1) / step + 1) : 1;
    TORCH_CHECK(from >= end, "out and an input share a part of their memory");
}
// y; the new state goes to `to`, which may be state
Tensor gated_scan_step(const Tensor& x0, const Tensor& gate0, const Tensor& state, Tensor to) {
    const int dtype = activation(x0, "x", 2);
    check_like(gate0, "gate", x0);
    check(state, "state", at::kFloat, x0, x0.sizes());
    check(to, "out", at::kFloat, x0, x0.sizes());
    for (const Tensor& t : {state, x0, gate0}) check_apart(to, t);
    const Tensor x = dense_rows(x0), gate = dense_rows(gate0), y = empty(x.sizes(), x);
    const wtc_scan_desc d = {x.size(0), x.stride(0), gate.stride(0), 0, 0, narrow(x.size(1), "channels of x"), dtype, 0};
    const On on(x);
    raise_on(wtconv_gated_scan_step(&d, in(x), in(gate), in_as<float>(state), out(y), floats(to), on.stream),
             "wtconv_gated_scan_step");
    return y;
}

// ------------------------------------------------------------------ experts' rows
// [slot, pair, cu_experts]
Tensors expert_order(const Tensor& experts, int64_t n_experts) {
    TORCH_CHECK_VALUE(experts.is_cuda(), "experts must be a CUDA tensor");
    TORCH_CHECK_VALUE(experts.dim() == 2 && experts.size(1) >= 1, "experts has shape ", experts.sizes(), ", expected [T, k]");
    TORCH_CHECK_VALUE(experts.scalar_type() == at::kInt, "experts has dtype ", experts.scalar_type(), ", expected ", at::kInt);
    const int E = narrow(n_experts, "experts");
    const Tensor e = experts.contiguous();
    const size_t bytes = wtconv_expert_order_workspace(e.numel(), E);
    const Tensor slot = empty(e.sizes(), e), pair = empty({e.numel()}, e), ws = workspace(bytes, e);
    const Tensor cu = empty({(int64_t)(E > 0 ? E : 0) + 1}, e);
    const On on(e);
    raise_on(wtconv_expert_order(e.numel(), E, in_as<int>(e), ints(slot), ints(pair), ints(cu), out(ws), bytes, on.stream),
             "wtconv_expert_order");
    return {slot, pair, cu};
}
int experts_of(const Tensor& cu, const Tensor& like) {
    TORCH_CHECK_VALUE(cu.dim() == 1 && cu.size(0) >= 2, "cu_experts must be [E + 1]");
    check(cu, "cu_experts", at::kInt, like, cu.sizes());
    return narrow(cu.size(0) - 1, "experts");
}
wtc_rows_desc rows_desc(const Tensor& like, const Tensor& slot, int E, const char* name) {
    const int dtype = activation(like, name, 2);
    TORCH_CHECK_VALUE(slot.dim() == 2 && slot.size(1) >= 1, "slot has shape ", slot.sizes(), ", expected [T, k]");
    check(slot, "slot", at::kInt, like, slot.sizes());
    return {slot.size(0), 0, 0, narrow(slot.size(1), "choices"), E, narrow(like.size(1), "channels"), dtype};
}
Tensor expert_gather(const Tensor& x0, const Tensor& slot, const Tensor& cu) {
    wtc_rows_desc d = rows_desc(x0, slot, experts_of(cu, x0), "x");
    TORCH_CHECK_VALUE(x0.size(0) == slot.size(0), "x has ", x0.size(0), " rows, slot ", slot.size(0));
    const Tensor x = dense_rows(x0), r = empty({slot.numel(), x.size(1)}, x);
    d.x_stride = x.stride(0);
    const On on(x);
    raise_on(wtconv_expert_gather(&d, in(x), in_as<int>(slot), in_as<int>(cu), out(r), on.stream), "wtconv_expert_gather");
    return r;
}
// by token, the sum of its rows, with weights if given
Tensor _expert_sum(const Tensor& rows0, const OptTensor& weights, const Tensor& slot) {
    wtc_rows_desc d = rows_desc(rows0, slot, 1, "rows");
    TORCH_CHECK_VALUE(rows0.size(0) == slot.numel(), "rows has ", rows0.size(0), " rows, slot ", slot.numel(), " places");
    if (weights) check(*weights, "weights", at::kFloat, rows0, slot.sizes(), false);
    const Tensor r = dense_rows(rows0), w = weights ? weights->contiguous() : Tensor(), y = empty({slot.size(0), r.size(1)}, r);
    d.r_stride = r.stride(0);
    const On on(r);
    raise_on(wtconv_expert_combine(&d, in(r), in_as<float>(w), in_as<int>(slot), out(y), on.stream),
             "wtconv_expert_combine");
    return y;
}
Tensor expert_combine(const Tensor& rows, const Tensor& weights, const Tensor& slot, const Tensor& cu) {
    experts_of(cu, rows);
    return _expert_sum(rows, weights, slot);
}
std::tuple<Tensor, Tensor> _expert_combine_backward(const Tensor& dy0, const Tensor& rows0, const Tensor& weights0,
                                                    const Tensor& slot, const Tensor& cu) {
    wtc_rows_desc d = rows_desc(rows0, slot, experts_of(cu, rows0), "rows");
    TORCH_CHECK_VALUE(rows0.size(0) == slot.numel(), "rows has ", rows0.size(0), " rows, slot ", slot.numel(), " places");
    check(weights0, "weights", at::kFloat, rows0, slot.sizes(), false);
    check(dy0, "dy", rows0.scalar_type(), rows0, {slot.size(0), rows0.size(1)}, false);
    const Tensor r = dense_rows(rows0), dy = dense_rows(dy0), weights = weights0.contiguous(), dr = empty(r.sizes(), r), dw = empty(slot.sizes(), r, at::kFloat);
    d.r_stride = r.stride(0);
    d.x_stride = dy.stride(0);
    const On on(r);
    raise_on(wtconv_expert_combine_backward(&d, in(dy), in(r), in_as<float>(weights), in_as<int>(slot), in_as<int>(cu), out(dr),
                                            floats(dw), on.stream),
             "wtconv_expert_combine_backward");
    return {dr, dw};
}

// ------------------------------------------------------------------ experts' products
wtc_expert_desc expert_desc(int64_t R, int64_t K, int64_t N, const Tensor& like, const Tensor& cu) {
    return {R, 0, 0, experts_of(cu, like), narrow(K, "channels"), narrow(N, "channels"), dtype_of(like)};
}
void weight_check(const Tensor& weight, const Tensor& like, const Tensor& cu) {
    experts_of(cu, like);
    TORCH_CHECK_VALUE(weight.dim() == 3 && weight.size(0) == cu.size(0) - 1, "weight has shape ", weight.sizes(), ", expected [",
                      cu.size(0) - 1, ", N, K]");
    check(weight, "weight", like.scalar_type(), like, weight.sizes());
}
Tensor expert_linear(const Tensor& x0, const Tensor& weight, const OptTensor& bias, const Tensor& cu) {
    activation(x0, "x", 2);
    weight_check(weight, x0, cu);
    const int64_t K = x0.size(1), N = weight.size(1);
    TORCH_CHECK_VALUE(weight.size(2) == K, "weight has shape ", weight.sizes(), " for ", K, " channels of x");
    if (bias) check(*bias, "bias", x0.scalar_type(), x0, {weight.size(0), N});
    const Tensor x = aligned_rows(x0), w = aligned(weight), b = bias ? aligned(*bias) : Tensor(), y = empty({x.size(0), N}, x);
    wtc_expert_desc d = expert_desc(x.size(0), K, N, x, cu);
    d.x_stride = x.stride(0);
    const On on(x);
    raise_on(wtconv_expert_linear_forward(&d, in(x), in(w), in(b), in_as<int>(cu), out(y), on.stream),
             "wtconv_expert_linear_forward");
    return y;
}
Tensor _expert_linear_input_grad(const Tensor& dy0, const Tensor& weight, const Tensor& cu) {
    activation(dy0, "dy", 2);
    weight_check(weight, dy0, cu);
    TORCH_CHECK_VALUE(weight.size(1) == dy0.size(1), "weight has shape ", weight.sizes(), " for ", dy0.size(1), " channels of dy");
    const Tensor dy = aligned_rows(dy0), w = aligned(weight), dx = empty({dy.size(0), w.size(2)}, dy);
    wtc_expert_desc d = expert_desc(dy.size(0), w.size(2), w.size(1), dy, cu);
    d.g_stride = dy.stride(0);
    const On on(dy);
    raise_on(wtconv_expert_linear_input_grad(&d, in(dy), in(w), in_as<int>(cu), out(dx), on.stream),
             "wtconv_expert_linear_input_grad");
    return dx;
}
// [dweight], or [dweight, dbias]
Tensors _expert_linear_weight_grad(const Tensor& dy0, const Tensor& x0, const Tensor& cu, bool bias) {
    activation(x0, "x", 2);
    check(dy0, "dy", x0.scalar_type(), x0, {x0.size(0), dy0.dim() == 2 ? dy0.size(1) : 0}, false);
    const int E = experts_of(cu, x0);
    const Tensor dy = aligned_rows(dy0), x = aligned_rows(x0);
    wtc_expert_desc d = expert_desc(x.size(0), x.size(1), dy.size(1), x, cu);
    d.x_stride = x.stride(0);
    d.g_stride = dy.stride(0);
    const size_t bytes = wtconv_expert_linear_weight_grad_workspace(&d);
    const Tensor dw = empty({E, d.N, d.K}, x), db = bias ? empty({E, d.N}, x) : Tensor(), ws = workspace(bytes, x);
    const On on(x);
    raise_on(wtconv_expert_linear_weight_grad(&d, in(dy), in(x), in_as<int>(cu), out(dw), out(db), out(ws), bytes, on.stream),
             "wtconv_expert_linear_weight_grad");
    return bias ? Tensors{dw, db} : Tensors{dw};
}

}  // namespace op

// ================================================================== gradients
// Whether the backward pass from `node` on, as far as it is wanted, runs through a node of the default stream: a node
// belongs to the stream of the forward pass that made it, and a leaf's gradient to that on which the leaf was first used,
// for as long as a pass that used it lives.
bool meets_default_stream(torch::autograd::Node* node) {
    std::vector<torch::autograd::Node*> open = {node};
    std::unordered_set<torch::autograd::Node*> seen;
    while (!open.empty()) {
        torch::autograd::Node* at = open.back();
        open.pop_back();
        for (size_t i = 0; i < at->num_outputs(); ++i) {
            torch::autograd::Node* to = at->next_edge(i).function.get();
            if (!to || !at->task_should_compute_output(i) || !seen.insert(to).second) continue;
            const auto stream = to->stream();
            if (stream && stream->id() == 0) return true;
            open.push_back(to);
        }
    }
    return false;
}
// PyTorch would make the default stream wait for the capture, which ends the process.  Refused; what the pass meets before
// its first node of these operators is not seen.
void check_capture() {
    const auto node = torch::autograd::get_current_node();
    if (!node) return;
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(c10::hip::getCurrentHIPStream().stream(), &status) != hipSuccess || status == hipStreamCaptureStatusNone)
        return;
    TORCH_CHECK(!meets_default_stream(node.get()), "a backward pass cannot be captured while an eager pass of the same leaves lives; "
                "delete its outputs, or detach the leaves anew");
}

struct LayerNorm : torch::autograd::Function<LayerNorm> {
    // Saves the norm's input (h, or x without a residual) and two floats per row.
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const OptTensor& bias,
                                 const OptTensor& residual, double eps) {
        const NoGraph guard;
        Tensors o = OP(_layer_norm_forward).call(x, weight, bias, residual, eps);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({residual ? o[2] : x, weight, o[0]});
        ctx->saved_data["bias"] = bias.has_value();
        o.erase(o.begin());
        return o;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        check_capture();
        const variable_list s = ctx->get_saved_variables();
        const Tensor dh = g.size() > 1 ? g[1] : Tensor();
        if (!g[0].defined()) return {dh, Tensor(), Tensor(), dh, Tensor()};
        const bool bias = ctx->saved_data["bias"].toBool();
        const NoGraph guard;
        const Tensors d = OP(_layer_norm_backward).call(g[0], some(dh), s[0], s[1], s[2], bias);
        return {d[0], d[1], bias ? d[2] : Tensor(), g.size() > 1 ? d[0] : Tensor(), Tensor()};
    }
};

struct GatedScan : torch::autograd::Function<GatedScan> {
    // Saves its inputs and the state before every 8th token.
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& gate, const Tensor& cu,
                                 const OptTensor& state, bool reverse) {
        const NoGraph guard;
        Tensors o = OP(_gated_scan_forward).call(x, gate, cu, state, reverse);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({x, gate, cu, state ? *state : Tensor(), o[2]});
        ctx->saved_data["reverse"] = reverse;
        o.pop_back();
        return o;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        check_capture();
        if (!g[0].defined() && !g[1].defined()) return variable_list(5);
        const variable_list s = ctx->get_saved_variables();
        const NoGraph guard;
        const Tensors d = OP(_gated_scan_backward).call(g[0].defined() ? g[0] : at::zeros_like(s[0]), some(g[1]), s[0], s[1], s[2],
                                                        some(s[3]), s[4], ctx->saved_data["reverse"].toBool());
        return {d[0], d[1], Tensor(), d.size() > 2 ? d[2] : Tensor(), Tensor()};
    }
};

struct ExpertGather : torch::autograd::Function<ExpertGather> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& slot, const Tensor& cu) {
        const NoGraph guard;
        ctx->save_for_backward({slot});
        return OP(expert_gather).call(x, slot, cu);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, true);
        check_capture();
        const Tensor slot = ctx->get_saved_variables()[0];
        const NoGraph guard;
        return {OP(_expert_sum).call(g[0], std::nullopt, slot), Tensor(), Tensor()};
    }
};

struct ExpertCombine : torch::autograd::Function<ExpertCombine> {
    static Tensor forward(AutogradContext* ctx, const Tensor& rows, const Tensor& weights, const Tensor& slot, const Tensor& cu) {
        const NoGraph guard;
        ctx->save_for_backward({rows, weights, slot, cu});
        return OP(expert_combine).call(rows, weights, slot, cu);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        check_capture();
        const variable_list s = ctx->get_saved_variables();
        const NoGraph guard;
        const auto [dr, dw] = OP(_expert_combine_backward).call(g[0], s[0], s[1], s[2], s[3]);
        return {dr, dw, Tensor(), Tensor()};
    }
};

struct ExpertLinear : torch::autograd::Function<ExpertLinear> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const OptTensor& bias, const Tensor& cu) {
        const NoGraph guard;
        ctx->save_for_backward({x, weight, cu});
        ctx->saved_data["bias"] = bias.has_value();
        return OP(expert_linear).call(x, weight, bias, cu);
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& g) {
        once(g, false);
        check_capture();
        const variable_list s = ctx->get_saved_variables();
        const bool has_bias = ctx->saved_data["bias"].toBool(), bias = has_bias && ctx->needs_input_grad(2);
        variable_list r(4);
        const NoGraph guard;
        if (ctx->needs_input_grad(0)) r[0] = OP(_expert_linear_input_grad).call(g[0], s[1], s[2]);
        if (ctx->needs_input_grad(1) || bias) {
            const Tensors d = OP(_expert_linear_weight_grad).call(g[0], s[0], s[2], bias);
            r[1] = d[0];
            if (bias) r[2] = d[1];
        }
        return r;
    }
};

namespace graph {

Tensors layer_norm(const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual, double eps) {
    refuse_tangents(x, weight, bias, residual);
    if (wants_grad(x, weight) || wants_grad_opt(bias) || wants_grad_opt(residual))
        return LayerNorm::apply(x, weight, bias, residual, eps);
    const NoGraph guard;
    return OP(layer_norm).call(x, weight, bias, residual, eps);
}
Tensors gated_scan(const Tensor& x, const Tensor& gate, const Tensor& cu, const OptTensor& state, bool reverse) {
    refuse_tangents(x, gate, state);
    if (wants_grad(x, gate) || wants_grad_opt(state)) return GatedScan::apply(x, gate, cu, state, reverse);
    const NoGraph guard;
    return OP(gated_scan).call(x, gate, cu, state, reverse);
}
Tensor gated_scan_step(const Tensor& x, const Tensor& gate, const Tensor& state, Tensor to) {
    refuse_tangents(x, gate, state, to);
    TORCH_CHECK_VALUE(!wants_grad(x, gate, state, to), "gated_scan_step has no gradient; call it under torch.no_grad()");
    Tensor y;
    {
        const NoGraph guard;
        y = OP(gated_scan_step).call(x, gate, state, to);
    }
    torch::autograd::increment_version(to);
    return y;
}
Tensor expert_gather(const Tensor& x, const Tensor& slot, const Tensor& cu) {
    refuse_tangents(x);
    if (wants_grad(x)) return ExpertGather::apply(x, slot, cu);
    const NoGraph guard;
    return OP(expert_gather).call(x, slot, cu);
}
Tensor expert_combine(const Tensor& rows, const Tensor& weights, const Tensor& slot, const Tensor& cu) {
    refuse_tangents(rows, weights);
    if (wants_grad(rows, weights)) return ExpertCombine::apply(rows, weights, slot, cu);
    const NoGraph guard;
    return OP(expert_combine).call(rows, weights, slot, cu);
}
Tensor expert_linear(const Tensor& x, const Tensor& weight, const OptTensor& bias, const Tensor& cu) {
    refuse_tangents(x, weight, bias);
    if (wants_grad(x, weight) || wants_grad_opt(bias)) return ExpertLinear::apply(x, weight, bias, cu);
    const NoGraph guard;
    return OP(expert_linear).call(x, weight, bias, cu);
}

}  // namespace graph

void mixer_kernels(torch::Library& m) {
    m.impl("layer_norm", &op::layer_norm);
    m.impl("gated_scan", &op::gated_scan);
    m.impl("gated_scan_step", &op::gated_scan_step);
    m.impl("expert_order", &op::expert_order);
    m.impl("expert_gather", &op::expert_gather);
    m.impl("expert_combine", &op::expert_combine);
    m.impl("expert_linear", &op::expert_linear);
    m.impl("_layer_norm_forward", &op::_layer_norm_forward);
    m.impl("_layer_norm_backward", &op::_layer_norm_backward);
    m.impl("_gated_scan_forward", &op::_gated_scan_forward);
    m.impl("_gated_scan_backward", &op::_gated_scan_backward);
    m.impl("_expert_sum", &op::_expert_sum);
    m.impl("_expert_combine_backward", &op::_expert_combine_backward);
    m.impl("_expert_linear_input_grad", &op::_expert_linear_input_grad);
    m.impl("_expert_linear_weight_grad", &op::_expert_linear_weight_grad);
}

}  // namespace

TORCH_LIBRARY_FRAGMENT(wtconv_tokens, m) {
    m.def("layer_norm(Tensor x, Tensor weight, Tensor? bias, Tensor? residual, float eps) -> Tensor[]");
    m.def("gated_scan(Tensor x, Tensor gate, Tensor cu_seqlens, Tensor? state, bool reverse) -> Tensor[]");
    m.def("gated_scan_step(Tensor x, Tensor gate, Tensor state, Tensor(a!) out) -> Tensor");
    m.def("expert_order(Tensor experts, int n_experts) -> Tensor[]");
    m.def("expert_gather(Tensor x, Tensor slot, Tensor cu_experts) -> Tensor");
    m.def("expert_combine(Tensor rows, Tensor weights, Tensor slot, Tensor cu_experts) -> Tensor");
    m.def("expert_linear(Tensor x, Tensor weight, Tensor? bias, Tensor cu_experts) -> Tensor");
    m.def("_layer_norm_forward(Tensor x, Tensor weight, Tensor? bias, Tensor? residual, float eps) -> Tensor[]");
    m.def("_layer_norm_backward(Tensor dy, Tensor? dh, Tensor h, Tensor weight, Tensor stats, bool bias) -> Tensor[]");
    m.def("_gated_scan_forward(Tensor x, Tensor gate, Tensor cu_seqlens, Tensor? state, bool reverse) -> Tensor[]");
    m.def("_gated_scan_backward(Tensor dy, Tensor? dlast, Tensor x, Tensor gate, Tensor cu_seqlens, Tensor? state, Tensor kept, "
          "bool reverse) -> Tensor[]");
    m.def("_expert_sum(Tensor rows, Tensor? weights, Tensor slot) -> Tensor");
    m.def("_expert_combine_backward(Tensor dy, Tensor rows, Tensor weights, Tensor slot, Tensor cu_experts) -> (Tensor, Tensor)");
    m.def("_expert_linear_input_grad(Tensor dy, Tensor weight, Tensor cu_experts) -> Tensor");
    m.def("_expert_linear_weight_grad(Tensor dy, Tensor x, Tensor cu_experts, bool bias) -> Tensor[]");
}
TORCH_LIBRARY_IMPL(wtconv_tokens, CUDA, m) { mixer_kernels(m); }
TORCH_LIBRARY_IMPL(wtconv_tokens, CPU, m) { mixer_kernels(m); }
TORCH_LIBRARY_IMPL(wtconv_tokens, Autograd, m) {
    m.impl("layer_norm", &graph::layer_norm);
    m.impl("gated_scan", &graph::gated_scan);
    m.impl("gated_scan_step", &graph::gated_scan_step);
    m.impl("expert_gather", &graph::expert_gather);
    m.impl("expert_combine", &graph::expert_combine);
    m.impl("expert_linear", &graph::expert_linear);
    for (const char* part : {"_layer_norm_forward", "_layer_norm_backward", "_gated_scan_forward", "_gated_scan_backward",
                             "_expert_sum", "_expert_combine_backward", "_expert_linear_input_grad", "_expert_linear_weight_grad"})
        m.impl(part, torch::autograd::autogradNotImplementedFallback());
}

namespace {

void mixer_python(py::module_& m) {
    using nogil = py::call_guard<py::gil_scoped_release>;
    // of the pass behind a tensor; what a captured backward pass is refused by
    m.def("_meets_default_stream", [](const Tensor& t) { return t.grad_fn() && meets_default_stream(t.grad_fn().get()); });
    m.def("layer_norm", [](const Tensor& x, const Tensor& weight, const OptTensor& bias, const OptTensor& residual, double eps) {
        return OP(layer_norm).call(x, weight, bias, residual, eps);
    }, nogil());
    m.def("gated_scan", [](const Tensor& x, const Tensor& gate, const Tensor& cu, const OptTensor& state, bool reverse) {
        return OP(gated_scan).call(x, gate, cu, state, reverse);
    }, nogil());
    m.def("gated_scan_step", [](const Tensor& x, const Tensor& gate, const Tensor& state, const OptTensor& out) {
        Tensor to = out ? *out : at::empty_like(state, state.options(), at::MemoryFormat::Contiguous);
        Tensor y = OP(gated_scan_step).call(x, gate, state, to);
        return std::make_tuple(std::move(y), std::move(to));
    }, nogil());
    m.def("expert_order", [](const Tensor& experts, int64_t n_experts) { return OP(expert_order).call(experts, n_experts); },
          nogil());
    m.def("expert_gather", [](const Tensor& x, const Tensor& slot, const Tensor& cu) {
        return OP(expert_gather).call(x, slot, cu);
    }, nogil());
    m.def("expert_combine", [](const Tensor& rows, const Tensor& weights, const Tensor& slot, const Tensor& cu) {
        return OP(expert_combine).call(rows, weights, slot, cu);
    }, nogil());
    m.def("expert_linear", [](const Tensor& x, const Tensor& weight, const OptTensor& bias, const Tensor& cu) {
        return OP(expert_linear).call(x, weight, bias, cu);
    }, nogil());
}

}  // namespace
