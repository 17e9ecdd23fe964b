// lm_binding.cpp -- the Python entry points of nonlinear_rnn_solve_amd.lm over the C ABI of include/pararnn_lm.h:
// argument checks, output allocation, the current stream and a workspace for each stream.  In C++ because a single-token
// call is bound by the host: through ctypes such calls took 13 us, two thirds of it in the interpreter.
#include "binding_common.h"
#include "pararnn_lm.h"

namespace {

// ---------------------------------------------------------------- gated linear recurrence
struct Scan {
  pararnn_lm_scan p{};
  int64_t n = 1;                  // sequences of a row
  std::vector<int64_t> shape;     // of a state array
  Scan(const Tensor& x, const Tensor& r, const Tensor& i, const Tensor& lam, const Maybe& h0, double c, const Maybe& cu) {
    p.dtype = storage(x, "x");
    if (x.dim() != 3) refuse("x must be [B, T, D], got " + text(x.sizes()));
    plane(x, "x", x);
    plane(r, "r", x);
    plane(i, "i", x);
    const auto dev = x.device();
    p.B = x.size(0), p.T = x.size(1), p.D = x.size(2);
    if (cu) {
      if (cu->dim() != 1 || cu->numel() < 2) refuse("cu_seqlens must be a 1-D tensor of n_seqs + 1 offsets");
      n = cu->numel() - 1;
      p.cu_seqlens = dense<int32_t>(cu, "cu_seqlens", at::kInt, {n + 1}, dev);
      p.n_seqs = n;
      shape = {p.B, n, p.D};
    } else {
      shape = {p.B, p.D};
    }
    if (h0) {
      const auto s = h0->sizes();
      if (s != at::IntArrayRef(shape) && !(!cu && s == at::IntArrayRef({p.B, 1, p.D})))
        refuse("h0 must be " + text(shape) + ", got " + text(s));
      shape.assign(s.begin(), s.end());
    }
    p.x = x.data_ptr(), p.r = r.data_ptr(), p.i = i.data_ptr();
    for (int k = 0; k < 2; ++k) p.sx[k] = x.stride(k), p.sr[k] = r.stride(k), p.si[k] = i.stride(k);
    p.lam = floats(lam, "lam", {p.D}, dev);
    p.h0 = floats(h0, "h0", shape, dev);
    p.c = static_cast<float>(c);
  }
};

std::tuple<Tensor, Tensor, Maybe> gated_scan(const Tensor& x, const Tensor& r, const Tensor& i, const Tensor& lam,
                                             const Maybe& h0, double c, const Maybe& cu, bool want_carry, const Maybe& out,
                                             const Maybe& h_last) {
  const Scan s(x, r, i, lam, h0, c, cu);
  const Call call(x.device());
  const Tensor h = output(out, "out", x);
  const Tensor last = h_last ? *h_last : new_floats(s.shape, x);
  float* pl = floats(last, "h_last", s.shape, x.device());
  Maybe carry;
  if (want_carry) carry = new_floats({s.p.B, pararnn_lm_scan_chunks(s.p.T), s.p.D}, x);
  const int64_t sh[2] = {h.stride(0), h.stride(1)};
  const Tensor ws = call.workspace(pararnn_lm_scan_workspace_bytes(s.p.B, s.p.T, s.p.D));
  check(pararnn_lm_gated_scan(&s.p, h.data_ptr(), sh, pl, carry ? static_cast<float*>(carry->data_ptr()) : nullptr,
                              ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_lm_gated_scan");
  written(out);
  written(h_last);
  return {h, last, carry};
}

py::dict gated_scan_vjp(const Tensor& x, const Tensor& r, const Tensor& i, const Tensor& lam, const Maybe& carry,
                        const Tensor& dh, const Maybe& h0, const Maybe& d_last, double c, const Maybe& cu,
                        const std::optional<std::vector<Tensor>>& out, bool want_lam, bool want_h0) {
  const Scan s(x, r, i, lam, h0, c, cu);
  const Call call(x.device());
  plane(dh, "dh", x);
  if (!carry) refuse("carry is missing: call gated_scan with want_carry=True");
  if (out && out->size() != 3) refuse("out must be three tensors (d_x, d_r, d_i)");
  Tensor d[3];
  for (int k = 0; k < 3; ++k) d[k] = output(out ? Maybe((*out)[k]) : Maybe(), "out", x);
  pararnn_lm_scan_grad g{};
  g.carry = floats(carry, "carry", {s.p.B, pararnn_lm_scan_chunks(s.p.T), s.p.D}, x.device());
  g.dh = dh.data_ptr();
  g.d_last = floats(d_last, "d_last", s.shape, x.device());
  g.d_x = d[0].data_ptr(), g.d_r = d[1].data_ptr(), g.d_i = d[2].data_ptr();
  for (int k = 0; k < 2; ++k)
    g.sdh[k] = dh.stride(k), g.sdx[k] = d[0].stride(k), g.sdr[k] = d[1].stride(k), g.sdi[k] = d[2].stride(k);
  py::dict res;
  res["d_x"] = d[0], res["d_r"] = d[1], res["d_i"] = d[2];
  if (want_lam) {
    const Tensor d_lam = new_floats({s.p.D}, x);
    g.d_lam = static_cast<float*>(d_lam.data_ptr());
    res["d_lam"] = d_lam;
  }
  if (want_h0) {
    const Tensor d_h0 = new_floats(!h0 && d_last ? d_last->sizes() : at::IntArrayRef(s.shape), x);
    g.d_h0 = static_cast<float*>(d_h0.data_ptr());
    res["d_h0"] = d_h0;
  }
  const Tensor ws = call.workspace(pararnn_lm_scan_workspace_bytes(s.p.B, s.p.T, s.p.D));
  check(pararnn_lm_gated_scan_vjp(&s.p, &g, ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_lm_gated_scan_vjp");
  if (out)
    for (const Tensor& t : *out) written(t);
  return res;
}

// ---------------------------------------------------------------- layer normalisation
std::tuple<Tensor, Tensor, Maybe> layer_norm(const Tensor& x, const Tensor& weight, const Maybe& bias, const Maybe& residual,
                                             double eps, bool want_stats, const Maybe& out, const Maybe& sum_out) {
  const int dt = storage(x, "x");
  plane(x, "x", x);
  const auto dev = x.device();
  const Call call(dev);
  const int64_t D = x.size(-1);
  const auto [N, xs] = rows(x, "x");
  Tensor s = x;
  int64_t rs = 0, ss = 0;
  if (residual) {
    plane(*residual, "residual", x);
    rs = rows(*residual, "residual").second;
    s = output(sum_out, "sum_out", x);
    ss = rows(s, "sum_out").second;
  } else if (sum_out) {
    refuse("sum_out needs a residual");
  }
  const Tensor y = output(out, "out", x);
  Maybe stats;
  if (want_stats) stats = new_floats({N, 2}, x);
  check(pararnn_lm_layer_norm(dt, N, D, x.data_ptr(), xs, residual ? residual->data_ptr() : nullptr, rs,
                              floats(weight, "weight", {D}, dev), floats(bias, "bias", {D}, dev), static_cast<float>(eps),
                              y.data_ptr(), rows(y, "out").second, residual ? s.data_ptr() : nullptr, ss,
                              stats ? static_cast<float*>(stats->data_ptr()) : nullptr, call.stream),
        "pararnn_lm_layer_norm");
  written(out);
  written(sum_out);
  return {y, s, stats};
}

py::dict layer_norm_vjp(const Tensor& dy, const Tensor& s, const Tensor& weight, const Maybe& stats, const Maybe& d_sum,
                        const Maybe& out, bool want_params) {
  const int dt = storage(s, "s");
  plane(s, "s", s);
  plane(dy, "dy", s);
  const auto dev = s.device();
  const Call call(dev);
  const int64_t D = s.size(-1);
  const auto [N, ss] = rows(s, "s");
  if (!stats) refuse("stats are missing: call layer_norm with want_stats=True");
  std::vector<int64_t> pairs{N, 2};   // or with s's leading dimensions
  if (stats->dim() > 2) pairs.assign(s.sizes().begin(), s.sizes().end()), pairs.back() = 2;
  int64_t ps = 0;
  if (d_sum) {
    plane(*d_sum, "d_sum", s);
    ps = rows(*d_sum, "d_sum").second;
  }
  const Tensor dx = output(out, "out", s);
  py::dict res;
  res["d_x"] = dx;
  float *pw = nullptr, *pb = nullptr;
  if (want_params) {
    const Tensor dw = new_floats({D}, s), db = new_floats({D}, s);
    pw = static_cast<float*>(dw.data_ptr()), pb = static_cast<float*>(db.data_ptr());
    res["d_weight"] = dw, res["d_bias"] = db;
  }
  const Tensor ws = call.workspace(pararnn_lm_layer_norm_vjp_workspace_bytes(N, D));
  check(pararnn_lm_layer_norm_vjp(dt, N, D, dy.data_ptr(), rows(dy, "dy").second, s.data_ptr(), ss,
                                  floats(weight, "weight", {D}, dev), floats(stats, "stats", pairs, dev),
                                  d_sum ? d_sum->data_ptr() : nullptr, ps, dx.data_ptr(), rows(dx, "out").second, pw, pb,
                                  ws.data_ptr(), static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_lm_layer_norm_vjp");
  written(out);
  return res;
}

// ---------------------------------------------------------------- log probabilities of tokens
// address and bytes of a target; (null, 0) without targets
std::pair<const void*, int> targets_of(const Maybe& t, const Tensor& logits) {
  if (!t) return {nullptr, 0};
  if (t->scalar_type() != at::kLong && t->scalar_type() != at::kInt)
    refuse(std::string("targets must be int64 or int32, got ") + c10::toString(t->scalar_type()));
  if (t->sizes() != logits.sizes().slice(0, logits.dim() - 1))
    refuse("targets must be " + text(logits.sizes().slice(0, logits.dim() - 1)) + ", got " + text(t->sizes()));
  return {dense<void>(t, "targets", t->scalar_type(), t->sizes(), logits.device()), t->scalar_type() == at::kLong ? 8 : 4};
}

std::tuple<Maybe, Tensor, Tensor, Maybe, Maybe> token_logprobs(const Tensor& logits, const Maybe& targets, int64_t top) {
  const int dt = storage(logits, "logits");
  plane(logits, "logits", logits);
  const Call call(logits.device());
  const int64_t V = logits.size(-1), most = std::min<int64_t>(V, PARARNN_LM_MAX_TOP);
  const auto [N, stride] = rows(logits, "logits");
  const auto [tp, tb] = targets_of(targets, logits);
  if (top < 0 || top > most)
    refuse("top must be in 0 .. min(V, " + std::to_string(PARARNN_LM_MAX_TOP) + ") = " + std::to_string(most) + ", got " +
           std::to_string(top));
  std::vector<int64_t> lead(logits.sizes().begin(), logits.sizes().end() - 1);
  const Tensor lse = new_floats(lead, logits), entropy = new_floats(lead, logits);
  Maybe logp, top_logp, top_ids;
  if (tb) logp = new_floats(lead, logits);
  if (top) {
    lead.push_back(top);
    top_logp = new_floats(lead, logits);
    top_ids = at::empty(lead, logits.options().dtype(at::kLong));
  }
  const Tensor ws = call.workspace(pararnn_lm_token_logprobs_workspace_bytes(N, V, static_cast<int>(top)));
  check(pararnn_lm_token_logprobs(dt, N, V, logits.data_ptr(), stride, tp, tb, static_cast<float*>(lse.data_ptr()),
                                  logp ? static_cast<float*>(logp->data_ptr()) : nullptr,
                                  static_cast<float*>(entropy.data_ptr()), static_cast<int>(top),
                                  top ? static_cast<float*>(top_logp->data_ptr()) : nullptr,
                                  top ? static_cast<int64_t*>(top_ids->data_ptr()) : nullptr, ws.data_ptr(),
                                  static_cast<size_t>(ws.numel()), call.stream),
        "pararnn_lm_token_logprobs");
  return {logp, entropy, lse, top_logp, top_ids};
}

Tensor token_logprobs_vjp(const Tensor& logits, const Maybe& targets, const Tensor& lse, const Maybe& entropy,
                          const Maybe& g_logp, const Maybe& g_entropy, const Maybe& out) {
  const int dt = storage(logits, "logits");
  plane(logits, "logits", logits);
  const auto dev = logits.device();
  const Call call(dev);
  const int64_t V = logits.size(-1);
  const auto [N, stride] = rows(logits, "logits");
  const auto lead = logits.sizes().slice(0, logits.dim() - 1);
  const auto [tp, tb] = targets_of(targets, logits);
  if (tb && !g_logp) refuse("g_logp is missing");
  if (g_entropy && !entropy) refuse("entropy is missing");
  const Tensor dz = output(out, "out", logits);
  check(pararnn_lm_token_logprobs_vjp(dt, N, V, logits.data_ptr(), stride, tp, tb, floats(lse, "lse", lead, dev),
                                      floats(entropy, "entropy", lead, dev), tb ? floats(g_logp, "g_logp", lead, dev) : nullptr,
                                      floats(g_entropy, "g_entropy", lead, dev), dz.data_ptr(), rows(dz, "out").second,
                                      call.stream),
        "pararnn_lm_token_logprobs_vjp");
  written(out);
  return dz;
}

}  // namespace

PYBIND11_MODULE(_lm_binding, m) {
  m.attr("ABI_VERSION") = PARARNN_LM_ABI_VERSION;
  m.attr("SCAN_CHUNK") = PARARNN_LM_SCAN_CHUNK;
  m.attr("NORM_MAX_D") = PARARNN_LM_NORM_MAX_D;
  m.attr("MAX_TOP") = PARARNN_LM_MAX_TOP;
  m.def("abi_version", &pararnn_lm_abi_version);
  m.def("gated_scan", &gated_scan);
  m.def("gated_scan_vjp", &gated_scan_vjp);
  m.def("layer_norm", &layer_norm);
  m.def("layer_norm_vjp", &layer_norm_vjp);
  m.def("token_logprobs", &token_logprobs);
  m.def("token_logprobs_vjp", &token_logprobs_vjp);
}
