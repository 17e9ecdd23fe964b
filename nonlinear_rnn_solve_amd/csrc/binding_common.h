// binding_common.h -- what the Python bindings share: argument checks, output allocation, the current stream and a workspace
// for each stream.  In an unnamed namespace: each binding is a module of its own.
#ifndef PARARNN_BINDING_COMMON_H
#define PARARNN_BINDING_COMMON_H

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <map>
#include <optional>
#include <string>
#include <tuple>
#include <utility>
#include <vector>

#include "pararnn.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t k = 0; k < s.size(); ++k) r += (k ? ", " : "") + std::to_string(s[k]);
  return r + "]";
}

// the storage type of the big planes
int storage(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a GPU tensor (no CPU path exists)");
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
    refuse(std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
  if (t.dim() < 1) refuse(std::string(name) + " must have at least one dimension");
  return t.scalar_type() == at::kBFloat16 ? PARARNN_BF16 : PARARNN_F32;
}

void on_device(const Tensor& t, const char* name, at::ScalarType type, c10::Device device) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a GPU tensor (no CPU path exists)");
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.device() != device) refuse("all tensors must be on " + device.str() + " (got " + t.device().str() + ")");
}

// a big plane in the type, shape and device of `like`: its last dimension dense, the others strided as they are
void plane(const Tensor& t, const char* name, const Tensor& like) {
  on_device(t, name, like.scalar_type(), like.device());
  if (t.sizes() != like.sizes()) refuse(std::string(name) + " must be " + text(like.sizes()) + ", got " + text(t.sizes()));
  if (t.size(-1) > 1 && t.stride(-1) != 1) refuse(std::string(name) + " must be dense in its last dimension");
}

// Whether a contiguous tensor of sizes `got` holds the values of one of sizes `want` in the same order: dimensions of one entry
// aside the sizes are equal, or it is flat.  (As many values are not enough: a transposed array would be read as another's rows.)
bool same_order(at::IntArrayRef got, at::IntArrayRef want) {
  if (got.size() == 1) return got[0] == c10::multiply_integers(want);
  size_t a = 0, b = 0;
  while (true) {
    while (a < got.size() && got[a] == 1) ++a;
    while (b < want.size() && want[b] == 1) ++b;
    if (a == got.size() || b == want.size()) return a == got.size() && b == want.size();
    if (got[a++] != want[b++]) return false;
  }
}

// the address of an optional contiguous tensor of `sizes`
template <typename P>
P* dense(const Maybe& t, const char* name, at::ScalarType type, at::IntArrayRef sizes, c10::Device device) {
  if (!t) return nullptr;
  on_device(*t, name, type, device);
  if (!t->is_contiguous() || !same_order(t->sizes(), sizes))
    refuse(std::string(name) + " must be " + text(sizes) + " and contiguous, got " + text(t->sizes()));
  return static_cast<P*>(t->data_ptr());
}
float* floats(const Maybe& t, const char* name, at::IntArrayRef sizes, c10::Device device) {
  return dense<float>(t, name, at::kFloat, sizes, device);
}

// [..., D] as rows of D: their number and stride, without a copy
std::pair<int64_t, int64_t> rows(const Tensor& t, const char* name) {
  const int64_t D = t.size(-1);
  int64_t n = 1, stride = D;
  bool first = true;   // of the dimensions longer than one, from the innermost
  for (int64_t k = t.dim() - 2; k >= 0; --k) {
    if (t.size(k) == 1) continue;
    if (first) stride = t.stride(k);
    else if (t.numel() && t.stride(k) != stride * n)
      refuse(std::string(name) + ": its leading dimensions must merge into rows of one stride");
    first = false;
    n *= t.size(k);
  }
  return {n, stride};
}

// A caller's tensor has been written: autograd refuses to use what it has saved of it (tensors made in inference mode are
// not counted).
void written(const Maybe& t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

Tensor output(const Maybe& given, const char* name, const Tensor& like) {
  if (!given) return at::empty(like.sizes(), like.options());
  plane(*given, name, like);
  for (int64_t k = 0; k < given->dim(); ++k)
    if (given->size(k) > 1 && given->stride(k) == 0) refuse(std::string(name) + " must not be a broadcast view: it is written");
  return *given;
}
Tensor new_floats(at::IntArrayRef sizes, const Tensor& like) { return at::empty(sizes, like.options().dtype(at::kFloat)); }

// One call of the C ABI: its device is current, its stream that of the device, its workspace that of the stream (calls on
// different streams may overlap, calls on one stream follow each other), grown on demand.  A call that is being captured
// into a graph takes a workspace of its own, which the graph's memory pool keeps: the stream's may be outgrown and
// given back while the graph is still replayed, and two graphs captured on one stream may replay on two.
struct Call {
  c10::DeviceGuard guard;
  c10::DeviceIndex index;
  hipStream_t hip;
  void* stream;
  explicit Call(c10::Device device)
      : guard(device), index(device.index()), hip(c10::hip::getCurrentHIPStream(device.index()).stream()), stream(hip) {}
  Tensor workspace(size_t bytes) const {
    const auto fresh = [&](size_t n) {
      return at::empty({static_cast<int64_t>(n)},
                       at::TensorOptions().dtype(at::kByte).device(c10::Device(c10::DeviceType::CUDA, index)));
    };
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (hip && hipStreamIsCapturing(hip, &capture) == hipSuccess && capture == hipStreamCaptureStatusActive)
      return fresh(bytes);
    // never destroyed: at exit the GPU runtime may be gone before a static's turn
    static auto* cache = new std::map<std::pair<int, void*>, Tensor>;
    Tensor& ws = (*cache)[{index, stream}];
    if (!ws.defined() || static_cast<size_t>(ws.numel()) < bytes) ws = fresh(std::max<size_t>(bytes, 1 << 16));
    return ws;
  }
};

void check(pararnn_status status, const char* entry) {
  if (status == PARARNN_OK) return;
  const py::object error = py::module_::import("nonlinear_rnn_solve_amd.api").attr("PararnnError");
  PyErr_SetObject(error.ptr(), error(static_cast<int>(status), entry).ptr());
  throw py::error_already_set();
}

}  // namespace
#endif
