// block_binding.cpp -- the Python entry points of nonlinear_rnn_solve_amd.block over the C ABI of include/pararnn_block.h.
#include "binding_common.h"
#include <torch/csrc/autograd/python_variable.h>

#include "pararnn_block.h"

namespace {

// offsets of sequences along T: their number and address; states have one more dimension with them
struct Offsets {
  const int32_t* p = nullptr;
  int64_t n = 1;
  Offsets(const Maybe& cu, c10::Device device) {
    if (!cu) return;
    if (cu->dim() != 1 || cu->numel() < 2) refuse("cu_seqlens must be a 1-D tensor of n_seqs + 1 offsets");
    n = cu->numel() - 1;
    p = dense<int32_t>(cu, "cu_seqlens", at::kInt, {n + 1}, device);
  }
};
// sizes of a state array, [B, rest] or, with offsets, [B, n, rest]; of `given` where that is [B, 1, rest]
std::vector<int64_t> state_shape(int64_t B, const Offsets& cu, std::vector<int64_t> rest, const Maybe& given, const char* name) {
  std::vector<int64_t> shape{B};
  if (cu.p) shape.push_back(cu.n);
  shape.insert(shape.end(), rest.begin(), rest.end());
  if (given) {
    std::vector<int64_t> one{B, 1};
    one.insert(one.end(), rest.begin(), rest.end());
    const auto s = given->sizes();
    if (s != at::IntArrayRef(shape) && !(!cu.p && s == at::IntArrayRef(one)))
      refuse(std::string(name) + " must be " + text(shape) + ", got " + text(s));
    shape.assign(s.begin(), s.end());
  }
  return shape;
}
void copy_strides(int64_t* to, const Tensor& t, int n) {
  for (int k = 0; k < n; ++k) to[k] = t.stride(k);
}
float* floats_of(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }
Maybe given_at(const std::optional<std::vector<Maybe>>& out, size_t k) { return out ? (*out)[k] : Maybe(); }
const Tensor* maybe(const Maybe& t) { return t ? &*t : nullptr; }
// Whether two tensors are seen to share memory: they begin at the same place, or both fill theirs without gaps and the two overlap (slices
// of one tensor interleave, so of tensors with gaps only the same beginning tells).
bool meet(const Tensor& a, const Tensor& b) {
  if (!a.numel() || !b.numel()) return false;
  const char *pa = static_cast<const char*>(a.data_ptr()), *pb = static_cast<const char*>(b.data_ptr());
  if (pa == pb) return true;
  return pa < pb + b.nbytes() && pb < pa + a.nbytes() && a.is_non_overlapping_and_dense() && b.is_non_overlapping_and_dense();
}
using Named = std::pair<const Tensor*, const char*>;
// a caller's output takes no input's place, nor another output's
void apart(const Maybe& out, const char* name, std::initializer_list<Named> others) {
  if (!out) return;
  for (const auto& [t, what] : others)
    if (t && meet(*out, *t)) refuse(std::string(name) + " must not share memory with " + what);
}
// a state that leaves may be the one that entered, but no part of it
void apart_or_same(const Maybe& last, const char* name, const Maybe& state, const char* what) {
  if (last && state && last->data_ptr() != state->data_ptr()) apart(last, name, {{&*state, what}});
}

// ---------------------------------------------------------------- causal convolution
struct Conv {
  pararnn_block_conv p{};
  std::vector<int64_t> shape;
  Conv(const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& state, const Maybe& cu_, bool silu) {
    p.dtype = storage(x, "x");
    if (x.dim() != 3) refuse("x must be [B, T, D], got " + text(x.sizes()));
    plane(x, "x", x);
    const auto dev = x.device();
    const Offsets cu(cu_, dev);
    p.silu = silu;
    p.B = x.size(0), p.T = x.size(1), p.D = x.size(2);
    if (weight.dim() != 2 || weight.size(0) != p.D || weight.size(1) < 1 || weight.size(1) > PARARNN_BLOCK_MAX_TAPS)
      refuse("weight must be [" + std::to_string(p.D) + ", taps] with 1 to " + std::to_string(PARARNN_BLOCK_MAX_TAPS) +
             " taps, got " + text(weight.sizes()));
    p.K = weight.size(1);
    p.x = x.data_ptr();
    copy_strides(p.sx, x, 2);
    p.weight = floats(weight, "weight", weight.sizes(), dev);
    p.bias = floats(bias, "bias", {p.D}, dev);
    shape = state_shape(p.B, cu, {p.K - 1, p.D}, state, "state");
    p.state = floats(state, "state", shape, dev);
    p.cu_seqlens = cu.p, p.n_seqs = cu.n;
  }
};

std::tuple<Tensor, Tensor> causal_conv(const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& state, const Maybe& cu,
                                       bool silu, const Maybe& out, const Maybe& last) {
  const Conv c(x, weight, bias, state, cu, silu);
  const Call call(x.device());
  const Tensor y = output(out, "out", x);
  apart(out, "out", {{&x, "x"}, {&weight, "weight"}, {maybe(bias), "bias"}, {maybe(state), "state"}, {maybe(cu), "cu_seqlens"}});
  apart(last, "last", {{maybe(out), "out"}, {&x, "x"}, {&weight, "weight"}, {maybe(bias), "bias"}, {maybe(cu), "cu_seqlens"}});
  apart_or_same(last, "last", state, "a part of state");
  const Tensor left = last ? *last : new_floats(c.shape, x);
  float* pl = floats(left, "last", c.shape, x.device());
  const int64_t sy[2] = {y.stride(0), y.stride(1)};
  check(pararnn_block_causal_conv(&c.p, y.data_ptr(), sy, pl, call.stream), "pararnn_block_causal_conv");
  written(out);
  written(last);
  return {y, left};
}

py::dict causal_conv_vjp(const Tensor& x, const Tensor& weight, const Tensor& dy, const Maybe& bias, const Maybe& state,
                         const Maybe& d_last, const Maybe& cu, bool silu, const Maybe& out, bool want_params, bool want_state) {
  const Conv c(x, weight, bias, state, cu, silu);
  const Call call(x.device());
  plane(dy, "dy", x);
  const Tensor dx = output(out, "out", x);
  apart(out, "out", {{&x, "x"}, {&dy, "dy"}, {&weight, "weight"}, {maybe(bias), "bias"}, {maybe(state), "state"}, {maybe(d_last), "d_last"},
                     {maybe(cu), "cu_seqlens"}});
  pararnn_block_conv_grad g{};
  g.dy = dy.data_ptr();
  g.d_last = floats(d_last, "d_last", c.shape, x.device());
  g.d_x = dx.data_ptr();
  copy_strides(g.sdy, dy, 2);
  copy_strides(g.sdx, dx, 2);
  py::dict res;
  res["d_x"] = dx;
  if (want_params) {
    const Tensor dw = new_floats({c.p.D, c.p.K}, x), db = new_floats({c.p.D}, x);
    g.d_weight = floats_of(dw), g.d_bias = floats_of(db);
    res["d_weight"] = dw, res["d_bias"] = db;
  }
  if (want_state) {
    const Tensor ds = new_floats(c.shape, x);
    g.d_state = floats_of(ds);
    res["d_state"] = ds;
  }
  const Tensor ws = call.workspace(pararnn_block_conv_workspace_bytes(c.p.B, c.p.T, c.p.D, c.p.K));
  check(pararnn_block_causal_conv_vjp(&c.p, &g, ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_block_causal_conv_vjp");
  written(out);
  return res;
}

// ---------------------------------------------------------------- selective scan
// b or c: [B, T, N] or [B, T, G, N] as strides over b, t and g
void shared_plane(const Tensor& t, const char* name, const Tensor& x, const Tensor& like) {
  on_device(t, name, x.scalar_type(), x.device());
  if (t.sizes() != like.sizes()) refuse(std::string(name) + " must be " + text(like.sizes()) + ", got " + text(t.sizes()));
  if (t.size(-1) > 1 && t.stride(-1) != 1) refuse(std::string(name) + " must be dense in its last dimension");
}
void shared_strides(int64_t* to, const Tensor& t) {
  to[0] = t.stride(0), to[1] = t.stride(1), to[2] = t.dim() == 4 ? t.stride(2) : 0;
}

struct Ssm {
  pararnn_block_ssm p{};
  std::vector<int64_t> shape;
  Ssm(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& b, const Tensor& c, const Maybe& skip, const Maybe& z,
      const Maybe& dt_bias, const Maybe& h0, const Maybe& cu_) {
    p.dtype = storage(x, "x");
    if (x.dim() != 3) refuse("x must be [B, T, D], got " + text(x.sizes()));
    plane(x, "x", x);
    plane(dt, "dt", x);
    if (z) plane(*z, "z", x);
    const auto dev = x.device();
    const Offsets cu(cu_, dev);
    p.B = x.size(0), p.T = x.size(1), p.D = x.size(2);
    if (A.dim() != 2 || A.size(0) != p.D || A.size(1) < 1 || A.size(1) > PARARNN_BLOCK_MAX_STATES)
      refuse("A must be [" + std::to_string(p.D) + ", states] with 1 to " + std::to_string(PARARNN_BLOCK_MAX_STATES) +
             " states, got " + text(A.sizes()));
    p.N = A.size(1);
    if ((b.dim() != 3 && b.dim() != 4) || b.size(0) != p.B || b.size(1) != p.T || b.size(-1) != p.N)
      refuse("b must be [B, T, states] or [B, T, groups, states] with x's B and T and A's states, got " + text(b.sizes()));
    p.G = b.dim() == 4 ? b.size(2) : 1;
    if (p.G < 1 || p.D % p.G) refuse("b's groups must divide x's channels, got " + std::to_string(p.G) + " of " + std::to_string(p.D));
    shared_plane(b, "b", x, b);
    shared_plane(c, "c", x, b);
    p.x = x.data_ptr(), p.delta = dt.data_ptr(), p.z = z ? z->data_ptr() : nullptr, p.b = b.data_ptr(), p.c = c.data_ptr();
    copy_strides(p.sx, x, 2);
    copy_strides(p.sdelta, dt, 2);
    if (z) copy_strides(p.sz, *z, 2);
    shared_strides(p.sb, b);
    shared_strides(p.sc, c);
    p.A = floats(A, "A", A.sizes(), dev);
    p.skip = floats(skip, "skip", {p.D}, dev);
    p.dt_bias = floats(dt_bias, "dt_bias", {p.D}, dev);
    shape = state_shape(p.B, cu, {p.D, p.N}, h0, "h0");
    p.h0 = floats(h0, "h0", shape, dev);
    p.cu_seqlens = cu.p, p.n_seqs = cu.n;
  }
  std::vector<int64_t> carry_shape() const { return {p.B, pararnn_block_ssm_chunks(p.T), p.N, p.D}; }
  size_t workspace(bool gradient) const { return pararnn_block_ssm_workspace_bytes(p.B, p.T, p.D, p.N, p.G, gradient); }
};

std::tuple<Tensor, Tensor, Maybe> selective_scan(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& b, const Tensor& c,
                                                 const Maybe& skip, const Maybe& z, const Maybe& dt_bias, const Maybe& h0,
                                                 const Maybe& cu, bool want_carry, const Maybe& out, const Maybe& h_last) {
  const Ssm s(x, dt, A, b, c, skip, z, dt_bias, h0, cu);
  const Call call(x.device());
  const Tensor y = output(out, "out", x);
  for (const auto& [t, name] : {std::pair<const Maybe&, const char*>{out, "out"}, {h_last, "h_last"}})
    apart(t, name, {{&x, "x"}, {&dt, "dt"}, {maybe(z), "z"}, {&b, "b"}, {&c, "c"}, {&A, "A"}, {maybe(skip), "skip"},
                    {maybe(dt_bias), "dt_bias"}, {maybe(cu), "cu_seqlens"}});
  apart(out, "out", {{maybe(h0), "h0"}, {maybe(h_last), "h_last"}});
  apart_or_same(h_last, "h_last", h0, "a part of h0");
  const Tensor last = h_last ? *h_last : new_floats(s.shape, x);
  float* pl = floats(last, "h_last", s.shape, x.device());
  Maybe carry;
  if (want_carry) carry = new_floats(s.carry_shape(), x);
  const int64_t sy[2] = {y.stride(0), y.stride(1)};
  const Tensor ws = call.workspace(s.workspace(false));
  check(pararnn_block_selective_scan(&s.p, y.data_ptr(), sy, pl, carry ? floats_of(*carry) : nullptr, ws.data_ptr(),
                                     static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_block_selective_scan");
  written(out);
  written(h_last);
  return {y, last, carry};
}

// a tensor for the gradient of b or c
Tensor shared_output(const Maybe& given, const char* name, const Tensor& x, const Tensor& like) {
  if (!given) return at::empty(like.sizes(), like.options());
  shared_plane(*given, name, x, like);
  for (int64_t k = 0; k < given->dim(); ++k)
    if (given->size(k) > 1 && given->stride(k) == 0) refuse(std::string(name) + " must not be a broadcast view: it is written");
  return *given;
}

py::dict selective_scan_vjp(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& b, const Tensor& c, const Maybe& carry,
                            const Tensor& dy, const Maybe& skip, const Maybe& z, const Maybe& dt_bias, const Maybe& h0,
                            const Maybe& d_last, const Maybe& cu, const std::optional<std::vector<Maybe>>& out, bool want_params,
                            bool want_h0) {
  const Ssm s(x, dt, A, b, c, skip, z, dt_bias, h0, cu);
  const Call call(x.device());
  plane(dy, "dy", x);
  if (!carry) refuse("carry is missing: call selective_scan with want_carry=True");
  if (out && out->size() != 5) refuse("out must be five tensors or None (d_x, d_dt, d_z, d_b, d_c)");
  if (!z && given_at(out, 2)) refuse("out holds a d_z, but there is no z");
  const Tensor dx = output(given_at(out, 0), "out", x), dd = output(given_at(out, 1), "out", x);
  const Tensor db = shared_output(given_at(out, 3), "out", x, b), dc = shared_output(given_at(out, 4), "out", x, b);
  for (size_t k = 0; out && k < 5; ++k) {
    apart((*out)[k], "out", {{&x, "x"}, {&dt, "dt"}, {maybe(z), "z"}, {&b, "b"}, {&c, "c"}, {&dy, "dy"}, {&A, "A"}, {maybe(skip), "skip"},
                             {maybe(dt_bias), "dt_bias"}, {maybe(h0), "h0"}, {maybe(d_last), "d_last"}, {maybe(carry), "carry"},
                             {maybe(cu), "cu_seqlens"}});
    for (size_t j = 0; j < k; ++j) apart((*out)[k], "out", {{maybe((*out)[j]), "another of out"}});
  }
  pararnn_block_ssm_grad g{};
  g.carry = floats(carry, "carry", s.carry_shape(), x.device());
  g.dy = dy.data_ptr();
  const std::vector<int64_t> states = !h0 && d_last ? state_shape(s.p.B, Offsets(cu, x.device()), {s.p.D, s.p.N}, d_last, "d_last") : s.shape;
  g.d_last = floats(d_last, "d_last", states, x.device());
  g.d_x = dx.data_ptr(), g.d_delta = dd.data_ptr(), g.d_b = db.data_ptr(), g.d_c = dc.data_ptr();
  copy_strides(g.sdy, dy, 2);
  copy_strides(g.sdx, dx, 2);
  copy_strides(g.sddelta, dd, 2);
  shared_strides(g.sdb, db);
  shared_strides(g.sdc, dc);
  py::dict res;
  res["d_x"] = dx, res["d_dt"] = dd, res["d_b"] = db, res["d_c"] = dc;
  if (z) {
    const Tensor dz = output(given_at(out, 2), "out", x);
    g.d_z = dz.data_ptr();
    copy_strides(g.sdz, dz, 2);
    res["d_z"] = dz;
  }
  if (want_params) {
    const Tensor dA = new_floats({s.p.D, s.p.N}, x), ds = new_floats({s.p.D}, x), dbias = new_floats({s.p.D}, x);
    g.d_A = floats_of(dA), g.d_skip = floats_of(ds), g.d_dt_bias = floats_of(dbias);
    res["d_A"] = dA, res["d_skip"] = ds, res["d_dt_bias"] = dbias;
  }
  if (want_h0) {
    const Tensor dh = new_floats(states, x);
    g.d_h0 = floats_of(dh);
    res["d_h0"] = dh;
  }
  const Tensor ws = call.workspace(s.workspace(true));
  check(pararnn_block_selective_scan_vjp(&s.p, &g, ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_block_selective_scan_vjp");
  if (out)
    for (const Maybe& t : *out) written(t);
  return res;
}

// ---------------------------------------------------------------- gated feed-forward product
struct Linear {
  int dtype, act;
  int64_t R, D, F, sx;
  std::vector<int64_t> lead;     // x's leading dimensions
  Linear(const Tensor& x, const Tensor& w_gate, const Tensor& w_up, const std::string& activation) {
    dtype = storage(x, "x");
    plane(x, "x", x);
    if (activation == "silu") act = PARARNN_BLOCK_SILU;
    else if (activation == "gelu") act = PARARNN_BLOCK_GELU;
    else refuse("activation must be \"silu\" or \"gelu\", got \"" + activation + "\"");
    if (w_gate.dim() != 2 || w_gate.size(1) != x.size(-1))
      refuse("w_gate must be [F, " + std::to_string(x.size(-1)) + "], got " + text(w_gate.sizes()));
    weight(w_gate, "w_gate", x, w_gate);
    weight(w_up, "w_up", x, w_gate);
    D = x.size(-1), F = w_gate.size(0);
    std::tie(R, sx) = rows(x, "x");
    lead.assign(x.sizes().begin(), x.sizes().end() - 1);
  }
  static void weight(const Tensor& t, const char* name, const Tensor& x, const Tensor& like) {
    on_device(t, name, x.scalar_type(), x.device());
    if (t.sizes() != like.sizes()) refuse(std::string(name) + " must be " + text(like.sizes()) + ", got " + text(t.sizes()));
    if (t.size(-1) > 1 && t.stride(-1) != 1) refuse(std::string(name) + " must be dense in its last dimension");
  }
  std::vector<int64_t> with(int64_t n) const {
    std::vector<int64_t> s = lead;
    s.push_back(n);
    return s;
  }
};

std::tuple<Tensor, Maybe> gated_linear(const Tensor& x, const Tensor& w_gate, const Tensor& w_up, const std::string& activation,
                                       bool want_pre, const Maybe& out) {
  const Linear l(x, w_gate, w_up, activation);
  const Call call(x.device());
  Tensor h;
  if (out) {
    on_device(*out, "out", x.scalar_type(), x.device());
    if (out->sizes() != at::IntArrayRef(l.with(l.F))) refuse("out must be " + text(l.with(l.F)) + ", got " + text(out->sizes()));
    h = output(out, "out", *out);
    apart(out, "out", {{&x, "x"}, {&w_gate, "w_gate"}, {&w_up, "w_up"}});
  } else {
    h = at::empty(l.with(l.F), x.options());
  }
  Maybe pre;
  if (want_pre) pre = new_floats({l.R, 2 * l.F}, x);
  const Tensor ws = call.workspace(pararnn_block_gated_linear_workspace_bytes(l.dtype, l.R, l.D, l.F, 0));
  check(pararnn_block_gated_linear(l.dtype, l.act, l.R, l.D, l.F, x.data_ptr(), l.sx, w_gate.data_ptr(), w_gate.stride(0),
                                   w_up.data_ptr(), w_up.stride(0), h.data_ptr(), rows(h, "out").second,
                                   pre ? floats_of(*pre) : nullptr, ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_block_gated_linear");
  written(out);
  return {h, pre};
}

py::dict gated_linear_vjp(const Tensor& x, const Tensor& w_gate, const Tensor& w_up, const Maybe& pre, const Tensor& dh,
                          const std::string& activation, bool want_x, bool want_params, const Maybe& out,
                          const std::optional<std::vector<Maybe>>& w_out) {
  const Linear l(x, w_gate, w_up, activation);
  const Call call(x.device());
  if (!pre) refuse("pre is missing: call gated_linear with want_pre=True");
  on_device(dh, "dh", x.scalar_type(), x.device());
  if (dh.sizes() != at::IntArrayRef(l.with(l.F))) refuse("dh must be " + text(l.with(l.F)) + ", got " + text(dh.sizes()));
  plane(dh, "dh", dh);
  if (!want_x && out) refuse("out needs want_x");
  if (w_out && (!want_params || w_out->size() != 2)) refuse("w_out must be two tensors or None (d_w_gate, d_w_up), with want_params");
  py::dict res;
  Tensor dx, dg, du;
  if (want_x) res["d_x"] = dx = output(out, "out", x);
  if (want_params) {
    res["d_w_gate"] = dg = output(given_at(w_out, 0), "w_out", w_gate);
    res["d_w_up"] = du = output(given_at(w_out, 1), "w_out", w_up);
  }
  for (const Maybe& t : {out, given_at(w_out, 0), given_at(w_out, 1)})
    apart(t, "an output", {{&x, "x"}, {&w_gate, "w_gate"}, {&w_up, "w_up"}, {&dh, "dh"}, {maybe(pre), "pre"}});
  apart(given_at(w_out, 1), "w_out", {{maybe(given_at(w_out, 0)), "another of w_out"}, {maybe(out), "out"}});
  apart(given_at(w_out, 0), "w_out", {{maybe(out), "out"}});
  const Tensor ws = call.workspace(pararnn_block_gated_linear_workspace_bytes(l.dtype, l.R, l.D, l.F, 1));
  check(pararnn_block_gated_linear_vjp(l.dtype, l.act, l.R, l.D, l.F, x.data_ptr(), l.sx, w_gate.data_ptr(), w_gate.stride(0),
                                       w_up.data_ptr(), w_up.stride(0),
                                       floats(pre, "pre", {l.R, 2 * l.F}, x.device()), dh.data_ptr(),
                                       rows(dh, "dh").second, want_x ? dx.data_ptr() : nullptr,
                                       want_x ? rows(dx, "out").second : 0, want_params ? dg.data_ptr() : nullptr,
                                       want_params ? dg.stride(0) : 0, want_params ? du.data_ptr() : nullptr,
                                       want_params ? du.stride(0) : 0, ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_block_gated_linear_vjp");
  written(out);
  if (w_out)
    for (const Maybe& t : *w_out) written(t);
  return res;
}

// ---------------------------------------------------------------- AdamW
// a number or a tensor of one element on the device
template <typename P>
const P* number(const py::object& v, const char* name, at::ScalarType type, c10::Device device, double& value) {
  if (THPVariable_Check(v.ptr())) return dense<P>(v.cast<Tensor>(), name, type, {1}, device);
  value = v.cast<double>();
  return nullptr;
}
int64_t blocks_of(int64_t n) { return (n + PARARNN_BLOCK_ADAMW_BLOCK - 1) / PARARNN_BLOCK_ADAMW_BLOCK; }

int64_t adamw_state_size(const std::vector<Tensor>& params) {
  int64_t n = 0;
  for (const Tensor& t : params) n += blocks_of(t.numel());
  return n * PARARNN_BLOCK_ADAMW_BLOCK;
}

// the scales of 8-bit moments
float* scales(const Maybe& t, const char* name, int64_t n, c10::Device device) {
  if (!t) refuse(std::string(name) + " is missing: moments in 8 bits have scales");
  return floats(t, name, {n / PARARNN_BLOCK_ADAMW_BLOCK}, device);
}

void adamw_step(const std::vector<Tensor>& params, const std::vector<Tensor>& grads, const Tensor& m, const Tensor& v,
                const py::object& step, const py::object& lr, std::pair<double, double> betas, double eps, double weight_decay,
                const py::object& grad_scale, const Maybe& m_scale, const Maybe& v_scale, uint64_t seed) {
  if (params.size() != grads.size())
    refuse("as many gradients as parameters, got " + std::to_string(grads.size()) + " and " + std::to_string(params.size()));
  if (!m.is_cuda()) refuse("m must be a GPU tensor (no CPU path exists)");
  const auto dev = m.device();
  const bool eight = m.scalar_type() == at::kByte;
  if (!eight && m.scalar_type() != at::kFloat)
    refuse(std::string("m must be float32 or uint8, got ") + c10::toString(m.scalar_type()));
  const Call call(dev);
  std::vector<pararnn_block_adamw_tensor> list;
  list.reserve(params.size());
  std::vector<std::pair<const char*, const char*>> places;
  int64_t size = 0;
  for (size_t k = 0; k < params.size(); ++k) {
    const Tensor &p = params[k], &g = grads[k];
    const std::string at = "[" + std::to_string(k) + "]", pn = "params" + at, gn = "grads" + at;
    pararnn_block_adamw_tensor t{};
    for (const auto& [a, name, type] : {std::tuple<const Tensor&, const std::string&, int32_t&>{p, pn, t.param_dtype},
                                        std::tuple<const Tensor&, const std::string&, int32_t&>{g, gn, t.grad_dtype}}) {
      if (!a.is_cuda()) refuse(name + " must be a GPU tensor (no CPU path exists)");
      if (a.scalar_type() != at::kFloat && a.scalar_type() != at::kBFloat16)
        refuse(name + " must be float32 or bfloat16, got " + c10::toString(a.scalar_type()));
      on_device(a, name.c_str(), a.scalar_type(), dev);
      if (!a.is_contiguous()) refuse(name + " must be contiguous");
      type = a.scalar_type() == at::kBFloat16 ? PARARNN_BF16 : PARARNN_F32;
    }
    if (g.sizes() != p.sizes()) refuse(gn + " must be " + text(p.sizes()) + ", got " + text(g.sizes()));
    t.param = p.data_ptr(), t.grad = g.data_ptr(), t.numel = p.numel(), t.offset = size;
    size += blocks_of(t.numel) * PARARNN_BLOCK_ADAMW_BLOCK;
    if (t.numel) {
      const char* a = static_cast<const char*>(t.param);
      places.emplace_back(a, a + p.nbytes());
    }
    list.push_back(t);
  }
  for (const Tensor* t : {&m, &v, maybe(m_scale), maybe(v_scale)})
    if (t && t->is_cuda() && t->numel()) {
      const char* a = static_cast<const char*>(t->data_ptr());
      places.emplace_back(a, a + t->nbytes());
    }
  std::sort(places.begin(), places.end());
  for (size_t k = 1; k < places.size(); ++k)
    if (places[k].first < places[k - 1].second)
      refuse("params must not overlap, nor the moments and their scales (a tensor is given twice, or two share memory)");
  pararnn_block_adamw_args a{};
  a.bits = eight ? 8 : 32;
  a.beta1 = betas.first, a.beta2 = betas.second, a.eps = eps, a.weight_decay = weight_decay;
  a.m = dense<void>(m, "m", m.scalar_type(), {size}, dev);
  a.v = dense<void>(v, "v", m.scalar_type(), {size}, dev);
  if (eight) a.m_scale = scales(m_scale, "m_scale", size, dev), a.v_scale = scales(v_scale, "v_scale", size, dev);
  else if (m_scale || v_scale) refuse("m_scale and v_scale are for moments in 8 bits");
  a.lr_ptr = number<float>(lr, "lr", at::kFloat, dev, a.lr);
  a.grad_scale_ptr = number<float>(grad_scale, "grad_scale", at::kFloat, dev, a.grad_scale);
  if (THPVariable_Check(step.ptr())) a.step_ptr = dense<int64_t>(step.cast<Tensor>(), "step", at::kLong, {1}, dev);
  else a.step = step.cast<int64_t>();
  a.seed = seed;
  check(pararnn_block_adamw(&a, list.data(), static_cast<int64_t>(list.size()), call.stream), "pararnn_block_adamw");
  for (const Tensor& t : params) written(t);
  for (const Maybe& t : {Maybe(m), Maybe(v), m_scale, v_scale}) written(t);
}

std::tuple<Tensor, Tensor> adamw_moments(const Tensor& m, const Tensor& v, const Maybe& m_scale, const Maybe& v_scale) {
  if (!m.is_cuda()) refuse("m must be a GPU tensor (no CPU path exists)");
  const auto dev = m.device();
  const Call call(dev);
  const int64_t n = m.numel();
  if (n % PARARNN_BLOCK_ADAMW_BLOCK) refuse("m must be a state of adamw_step: whole blocks of " + std::to_string(PARARNN_BLOCK_ADAMW_BLOCK));
  const void* pm = dense<void>(m, "m", at::kByte, {n}, dev);
  const void* pv = dense<void>(v, "v", at::kByte, {n}, dev);
  const Tensor a = at::empty({n}, m.options().dtype(at::kBFloat16)), b = at::empty({n}, m.options().dtype(at::kBFloat16));
  check(pararnn_block_adamw_moments(n, pm, pv, scales(m_scale, "m_scale", n, dev), scales(v_scale, "v_scale", n, dev), a.data_ptr(),
                                    b.data_ptr(), call.stream),
        "pararnn_block_adamw_moments");
  return {a, b};
}

}  // namespace

PYBIND11_MODULE(_block_binding, m) {
  m.attr("ABI_VERSION") = PARARNN_BLOCK_ABI_VERSION;
  m.attr("MAX_TAPS") = PARARNN_BLOCK_MAX_TAPS;
  m.attr("MAX_STATES") = PARARNN_BLOCK_MAX_STATES;
  m.attr("SSM_CHUNK") = PARARNN_BLOCK_SSM_CHUNK;
  m.attr("ADAMW_BLOCK") = PARARNN_BLOCK_ADAMW_BLOCK;
  m.def("abi_version", &pararnn_block_abi_version);
  m.def("causal_conv", &causal_conv);
  m.def("causal_conv_vjp", &causal_conv_vjp);
  m.def("selective_scan", &selective_scan);
  m.def("selective_scan_vjp", &selective_scan_vjp);
  m.def("gated_linear", &gated_linear);
  m.def("gated_linear_vjp", &gated_linear_vjp);
  m.def("adamw_state_size", &adamw_state_size);
  m.def("adamw_step", &adamw_step);
  m.def("adamw_moments", &adamw_moments);
}
