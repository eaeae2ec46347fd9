// fp8q_torch.cpp -- argument marshalling of the routing, dispatch, combine and
// checkpoint calls: torch tensors in, the C ABI of fp8q.h out.
//
// A decode step's calls take 3 to 6 us on the device each; marshalled through
// ctypes, with the checks and allocations in Python, they took 11 to 24 us to
// issue.  Here the same checks (types, ranks, layouts, agreement of the shapes,
// element counts of every buffer that the caller passes, one CUDA device for
// all), the outputs' allocation and the call run in C++.  The module computes
// nothing and launches nothing by itself.
#include <torch/extension.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "fp8q.h"

namespace {

using at::Tensor;
using Opt = std::optional<Tensor>;
using Types = std::initializer_list<at::ScalarType>;

constexpr int64_t kTile = 128;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxGroups = 32;
constexpr int64_t kWgradTokenGroup = 4 * kTile;

const Types kFp8 = {at::kFloat8_e4m3fn, at::kByte};
const Types kBf16 = {at::kBFloat16};
const Types kF32 = {at::kFloat};
const Types kI32 = {at::kInt};
const Types kLogits = {at::kFloat, at::kBFloat16};

std::string word(const char* s) { return s; }
std::string word(const std::string& s) { return s; }
std::string word(int64_t v) { return std::to_string(v); }
std::string word(at::ScalarType t) { return c10::toString(t); }
std::string word(const at::Device& d) { return d.str(); }
template <typename... A>
std::string text(const A&... a) {
  return (word(a) + ...);
}
template <typename... A>
[[noreturn]] void bad_value(const A&... a) {
  throw py::value_error(text(a...));
}
template <typename... A>
[[noreturn]] void bad_type(const A&... a) {
  throw py::type_error(text(a...));
}

// Type, rank and layout of one argument (the device comes last, for all).
void spec(const Tensor& t, const char* name, Types types, int64_t lo = 0, int64_t hi = 64) {
  bool ok = false;
  for (at::ScalarType s : types) ok = ok || t.scalar_type() == s;
  if (!ok) bad_type(name, ": dtype ", t.scalar_type(), " is not supported here");
  if (t.dim() < lo || t.dim() > hi)
    bad_value(name, ": expected ", lo, lo == hi ? "" : text(" to ", hi), " dims, got ", t.dim());
  if (!t.is_contiguous()) bad_value(name, " must be contiguous");
}
void holds(const Tensor& t, const char* name, int64_t n) {
  if (t.numel() != n) bad_value(name, " holds ", t.numel(), " elements, the call needs ", n);
}
// A buffer that may be left out.
void buffer(const Opt& t, const char* name, Types types, int64_t n) {
  if (!t) return;
  spec(*t, name, types);
  holds(*t, name, n);
}
void multiple(int64_t v, const char* name) {
  if (v % kTile) bad_value(name, " = ", v, " is not a multiple of ", kTile);
}

// An output may not share memory with an input whose elements other threads still read.
void apart(const Opt& out, const char* name, const Tensor& in, const char* other, const char* why) {
  if (!out || out->numel() == 0 || in.numel() == 0) return;
  const auto a = reinterpret_cast<uintptr_t>(out->data_ptr()), b = reinterpret_cast<uintptr_t>(in.data_ptr());
  if (a < b + in.nbytes() && b < a + out->nbytes())
    bad_value(name, " may not be ", other, ", or overlap it: ", why);
}

// All tensors are CUDA tensors on one device (there is no CPU path).
struct Place {
  std::optional<at::Device> dev;
  void add(const Tensor& t, const char* name) {
    if (!t.is_cuda()) bad_value(name, " must be a CUDA tensor");
    if (!dev)
      dev = t.device();
    else if (t.device() != *dev)
      bad_value(name, " is on ", t.device(), ", the other arguments on ", *dev);
  }
  void add(const Opt& t, const char* name) {
    if (t) add(*t, name);
  }
};

template <typename T = void>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
template <typename T = void>
T* ptr(const Opt& t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The call's device, made current, and its stream: None (the device's current
// stream), a torch.cuda.Stream, or a handle.
c10::cuda::CUDAStream call_stream(const py::object& s, const c10::cuda::CUDAStream& current) {
  if (s.is_none()) return current;
  const auto handle = (py::hasattr(s, "cuda_stream") ? s.attr("cuda_stream") : s).cast<uintptr_t>();
  if (handle == reinterpret_cast<uintptr_t>(current.stream())) return current;
  // cudaStreamLegacy is the default stream; as a handle of its own the allocator would take it for a pool's number
  const auto named = handle == reinterpret_cast<uintptr_t>(cudaStreamLegacy) ? 0 : handle;
  return c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(named), current.device_index());
}

// Memory that a call allocates comes from the pool of the stream it runs on: a
// block of the current stream's pool may have work of that stream queued on it,
// which another stream would not wait for.
struct On {
  c10::cuda::CUDAGuard guard;
  c10::cuda::CUDAStream caller;  // the device's current stream
  c10::cuda::CUDAStream own;     // the call's
  cudaStream_t stream;
  On(const Place& p, const py::object& s)
      : guard(*p.dev),
        caller(c10::cuda::getCurrentCUDAStream(p.dev->index())),
        own(call_stream(s, caller)),
        stream(own.stream()) {}
  Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    if (own == caller) return at::Tensor(at::detail::empty_cuda(shape, type, guard.current_device(), std::nullopt));
    const c10::cuda::CUDAStreamGuard on_own(own);
    return at::Tensor(at::detail::empty_cuda(shape, type, guard.current_device(), std::nullopt));
  }
  // n int32 of scratch for this call's work (an undefined tensor for none).  Dropped when the call returns, its
  // memory goes to later work of the same stream.
  Tensor scratch(int64_t n) const { return n == 0 ? Tensor() : make({n}, at::kInt); }
  // An output the caller did not pass.  Work that the current stream has queued on it when it is dropped ends before
  // its memory is handed out again.
  Tensor fresh(const Opt& given, at::IntArrayRef shape, at::ScalarType type) const {
    if (given) return *given;
    Tensor t = make(shape, type);
    if (own != caller) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller);
    return t;
  }
};

void check(int rc, const char* what) {
  if (rc == FP8Q_OK) return;
  const py::object err = py::module_::import("fp8_fine_grained_quant_b200").attr("Fp8qError");
  PyErr_SetObject(err.ptr(), err(rc, what).ptr());
  throw py::error_already_set();
}

int is_sigmoid(const std::string& score) {
  if (score != "softmax" && score != "sigmoid") bad_value("score must be 'softmax' or 'sigmoid', got '", score, "'");
  return score == "sigmoid";
}
void router(const Tensor& logits, int64_t top_k) {
  spec(logits, "logits", kLogits, 2, 2);
  const int64_t E = logits.size(1), most = E < kMaxTopK ? E : kMaxTopK;
  if (E < 1 || E > kMaxExperts) bad_value("logits have ", E, " experts, 1 to ", kMaxExperts, " are supported");
  if (top_k < 1 || top_k > most) bad_value("top_k = ", top_k, " is not in 1..", most);
}

py::tuple route(const Tensor& logits, int64_t top_k, const Opt& bias, const std::string& score, int64_t n_group,
                int64_t topk_group, int64_t group_top, bool renorm, double scale, const Opt& ids, const Opt& weights,
                const py::object& stream) {
  router(logits, top_k);
  const int64_t T = logits.size(0), E = logits.size(1);
  const int sigmoid = is_sigmoid(score);
  if (n_group < 1 || n_group > kMaxGroups || E % n_group)
    bad_value("n_group = ", n_group, " does not divide ", E, " experts, or is not in 1..", kMaxGroups);
  if (topk_group < 1 || topk_group > n_group) bad_value("topk_group = ", topk_group, " is not in 1..", n_group);
  if (group_top < 1 || group_top > 2) bad_value("group_top = ", group_top, " is not 1 or 2");
  if (top_k > topk_group * (E / n_group))
    bad_value("top_k = ", top_k, " exceeds the ", topk_group * (E / n_group), " experts of ", topk_group, " groups");
  buffer(bias, "bias", kF32, E);
  buffer(ids, "ids", kI32, T * top_k);
  buffer(weights, "weights", kF32, T * top_k);
  Place p;
  p.add(logits, "logits");
  p.add(bias, "bias");
  p.add(ids, "ids");
  p.add(weights, "weights");
  const On on(p, stream);
  const Tensor i = on.fresh(ids, {T, top_k}, at::kInt), w = on.fresh(weights, {T, top_k}, at::kFloat);
  check(fp8_moe_route(ptr(logits), logits.scalar_type() == at::kBFloat16, T, E, ptr<float>(bias), sigmoid, top_k,
                      n_group, topk_group, group_top, renorm, static_cast<float>(scale), ptr<int32_t>(i),
                      ptr<float>(w), on.stream),
        "fp8_moe_route");
  return py::make_tuple(i, w);
}

Tensor route_bwd(const Tensor& logits, const Tensor& ids, const Tensor& dweights, const std::string& score,
                 bool renorm, double scale, const Opt& dlogits, const py::object& stream) {
  spec(ids, "ids", kI32, 2, 2);
  const int64_t top_k = ids.size(1);
  router(logits, top_k);
  const int64_t T = logits.size(0), E = logits.size(1);
  const int sigmoid = is_sigmoid(score);
  holds(ids, "ids", T * top_k);
  spec(dweights, "dweights", kF32);
  holds(dweights, "dweights", T * top_k);
  buffer(dlogits, "dlogits", {logits.scalar_type()}, T * E);
  Place p;
  p.add(logits, "logits");
  p.add(ids, "ids");
  p.add(dweights, "dweights");
  p.add(dlogits, "dlogits");
  const On on(p, stream);
  const Tensor d = on.fresh(dlogits, {T, E}, logits.scalar_type());
  check(fp8_moe_route_bwd(ptr(logits), logits.scalar_type() == at::kBFloat16, T, E, ptr<int32_t>(ids),
                          ptr<float>(dweights), sigmoid, top_k, renorm, static_cast<float>(scale), ptr(d), on.stream),
        "fp8_moe_route_bwd");
  return d;
}

void layout_ids(const Tensor& ids, int64_t E) {
  spec(ids, "ids", kI32, 2, 2);
  if (E < 1 || E > kMaxExperts) bad_value("E = ", E, " is not in 1..", kMaxExperts);
  if (ids.size(1) < 1 || ids.size(1) > kMaxTopK)
    bad_value("ids have ", ids.size(1), " columns, 1 to ", kMaxTopK, " are supported");
}

py::tuple layout_contiguous(const Tensor& ids, int64_t E, const Opt& slots, const Opt& m_indices, const Opt& counts,
                            const py::object& stream) {
  layout_ids(ids, E);
  const int64_t T = ids.size(0), top_k = ids.size(1), n = T * top_k, B = (n + 127 * (n < E ? n : E)) / 128;
  buffer(slots, "slots", kI32, n);
  buffer(m_indices, "m_indices", kI32, B);
  buffer(counts, "counts", kI32, E);
  Place p;
  p.add(ids, "ids");
  p.add(slots, "slots");
  p.add(m_indices, "m_indices");
  p.add(counts, "counts");
  const On on(p, stream);
  const Tensor s = on.fresh(slots, {T, top_k}, at::kInt), m = on.fresh(m_indices, {B}, at::kInt),
               c = on.fresh(counts, {E}, at::kInt);
  const Tensor w = on.scratch(fp8_moe_layout_workspace(T, top_k, E));
  check(fp8_moe_layout_contiguous(ptr<int32_t>(ids), T, top_k, E, ptr<int32_t>(s), ptr<int32_t>(m), ptr<int32_t>(c),
                                  ptr<int32_t>(w), on.stream),
        "fp8_moe_layout_contiguous");
  return py::make_tuple(s, m, c);
}

py::tuple layout_masked(const Tensor& ids, int64_t E, int64_t cap, const Opt& slots, const Opt& masked_m,
                        const py::object& stream) {
  layout_ids(ids, E);
  if (cap < kTile) bad_value("cap = ", cap, " is below ", kTile);
  multiple(cap, "cap");
  const int64_t T = ids.size(0), top_k = ids.size(1);
  buffer(slots, "slots", kI32, T * top_k);
  buffer(masked_m, "masked_m", kI32, E);
  Place p;
  p.add(ids, "ids");
  p.add(slots, "slots");
  p.add(masked_m, "masked_m");
  const On on(p, stream);
  const Tensor s = on.fresh(slots, {T, top_k}, at::kInt), m = on.fresh(masked_m, {E}, at::kInt);
  const Tensor w = on.scratch(fp8_moe_layout_workspace(T, top_k, E));
  check(fp8_moe_layout_masked(ptr<int32_t>(ids), T, top_k, E, cap, ptr<int32_t>(s), ptr<int32_t>(m), ptr<int32_t>(w),
                              on.stream),
        "fp8_moe_layout_masked");
  return py::make_tuple(s, m);
}

int64_t slot_columns(const Tensor& slots, int64_t T) {
  spec(slots, "slots", kI32, 2, 2);
  if (slots.size(0) != T) bad_value("slots are for ", slots.size(0), " tokens, the call has ", T);
  if (slots.size(1) < 1 || slots.size(1) > kMaxTopK)
    bad_value("slots have ", slots.size(1), " columns, 1 to ", kMaxTopK, " are supported");
  return slots.size(1);
}

// The contiguous layout's arrays (both or neither); returns the expert count.
int64_t pad_layout(const Opt& m_indices, const Opt& counts, int64_t rows) {
  if (m_indices.has_value() != counts.has_value()) bad_value("m_indices and counts go together");
  if (!m_indices) return 0;
  multiple(rows, "rows");
  buffer(m_indices, "m_indices", kI32, rows / kTile);
  spec(*counts, "counts", kI32);
  const int64_t E = counts->numel();
  if (E < 1 || E > kMaxExperts) bad_value("counts hold ", E, " experts, 1 to ", kMaxExperts, " are supported");
  return E;
}

py::tuple dispatch_1x128(const Tensor& x, const Tensor& slots, int64_t rows, const Opt& m_indices, const Opt& counts,
                         const Opt& q, const Opt& s, const py::object& stream) {
  spec(x, "x", kBf16, 2, 2);
  const int64_t T = x.size(0), D = x.size(1);
  multiple(D, "D");
  if (rows < 0) bad_value("rows = ", rows, " is negative");
  const int64_t top_k = slot_columns(slots, T), E = pad_layout(m_indices, counts, rows);
  buffer(q, "q", kFp8, rows * D);
  buffer(s, "s", kF32, rows * (D / kTile));
  Place p;
  p.add(x, "x");
  p.add(slots, "slots");
  p.add(m_indices, "m_indices");
  p.add(counts, "counts");
  p.add(q, "q");
  p.add(s, "s");
  const On on(p, stream);
  const Tensor oq = on.fresh(q, {rows, D}, at::kFloat8_e4m3fn), os = on.fresh(s, {rows, D / kTile}, at::kFloat);
  check(fp8_moe_dispatch_1x128(ptr(x), T, D, ptr<int32_t>(slots), top_k, rows, ptr<int32_t>(m_indices),
                               ptr<int32_t>(counts), E, ptr<uint8_t>(oq), ptr<float>(os), on.stream),
        "fp8_moe_dispatch_1x128");
  return py::make_tuple(oq, os);
}

// Expert outputs [rows, D] or [E, cap, D]: their width.
int64_t expert_rows(const Tensor& y, int64_t& rows) {
  spec(y, "y", kBf16, 2, 3);
  const int64_t D = y.size(-1);
  multiple(D, "D");
  rows = y.dim() == 2 ? y.size(0) : y.size(0) * y.size(1);
  return D;
}

Tensor combine(const Tensor& y, const Tensor& slots, const Opt& weights, const Opt& out, const py::object& stream) {
  int64_t rows = 0;
  const int64_t D = expert_rows(y, rows);
  spec(slots, "slots", kI32, 2, 2);
  const int64_t T = slots.size(0), top_k = slot_columns(slots, T);
  buffer(weights, "weights", kF32, T * top_k);
  buffer(out, "out", kBf16, T * D);
  Place p;
  p.add(y, "y");
  p.add(slots, "slots");
  p.add(weights, "weights");
  p.add(out, "out");
  apart(out, "out", y, "y", "its rows are read while out is written");
  const On on(p, stream);
  const Tensor o = on.fresh(out, {T, D}, at::kBFloat16);
  check(fp8_moe_combine(ptr(y), rows, D, ptr<int32_t>(slots), ptr<float>(weights), T, top_k, ptr(o), on.stream),
        "fp8_moe_combine");
  return o;
}

py::tuple combine_bwd(const Tensor& dout, const Tensor& y, const Tensor& slots, const Opt& weights,
                      const Opt& m_indices, const Opt& counts, const Opt& dy, const Opt& dweights,
                      const py::object& stream) {
  int64_t rows = 0;
  const int64_t D = expert_rows(y, rows);
  spec(dout, "dout", kBf16, 2, 2);
  const int64_t T = dout.size(0);
  if (dout.size(1) != D) bad_value("dout and y differ in D (", dout.size(1), ", ", D, ")");
  const int64_t top_k = slot_columns(slots, T);
  if (!weights) bad_type("weights must be a torch.Tensor");
  buffer(weights, "weights", kF32, T * top_k);
  const int64_t E = pad_layout(m_indices, counts, rows);
  buffer(dy, "dy", kBf16, rows * D);
  buffer(dweights, "dweights", kF32, T * top_k);
  Place p;
  p.add(dout, "dout");
  p.add(y, "y");
  p.add(slots, "slots");
  p.add(weights, "weights");
  p.add(m_indices, "m_indices");
  p.add(counts, "counts");
  p.add(dy, "dy");
  p.add(dweights, "dweights");
  apart(dy, "dy", y, "y", "its rows are read while dy is written");
  apart(dy, "dy", dout, "dout", "its rows are read while dy is written");
  const On on(p, stream);
  const Tensor od = on.fresh(dy, y.sizes(), at::kBFloat16), ow = on.fresh(dweights, {T, top_k}, at::kFloat);
  check(fp8_moe_combine_bwd(ptr(dout), ptr(y), rows, D, ptr<int32_t>(slots), ptr<float>(weights), T, top_k,
                            ptr<int32_t>(m_indices), ptr<int32_t>(counts), E, ptr(od), ptr<float>(ow), on.stream),
        "fp8_moe_combine_bwd");
  return py::make_tuple(od, ow);
}

py::tuple swiglu_ckpt(const Tensor& c1, const Opt& qh, const Opt& sh, const Opt& qc, const Opt& sc,
                      const py::object& stream) {
  spec(c1, "c1", kBf16, 2, 2);
  if (c1.size(1) % (2 * kTile)) bad_value("c1's last dim ", c1.size(1), " is not 2 x a multiple of ", kTile);
  const int64_t rows = c1.size(0), inter = c1.size(1) / 2, nt = inter / kTile;
  buffer(qh, "qh", kFp8, rows * inter);
  buffer(sh, "sh", kF32, rows * nt);
  buffer(qc, "qc", kFp8, rows * 2 * inter);
  buffer(sc, "sc", kF32, rows * 2 * nt);
  Place p;
  p.add(c1, "c1");
  p.add(qh, "qh");
  p.add(sh, "sh");
  p.add(qc, "qc");
  p.add(sc, "sc");
  const On on(p, stream);
  const Tensor a = on.fresh(qh, {rows, inter}, at::kFloat8_e4m3fn), b = on.fresh(sh, {rows, nt}, at::kFloat),
               c = on.fresh(qc, {rows, 2 * inter}, at::kFloat8_e4m3fn), d = on.fresh(sc, {rows, 2 * nt}, at::kFloat);
  check(fp8_swiglu_ckpt_1x128(ptr(c1), rows, inter, ptr<uint8_t>(a), ptr<float>(b), ptr<uint8_t>(c), ptr<float>(d),
                              on.stream),
        "fp8_swiglu_ckpt_1x128");
  return py::make_tuple(py::make_tuple(a, b), py::make_tuple(c, d));
}

py::tuple swiglu_bwd(const Tensor& dh, const Tensor& qc, const Tensor& sc, const Opt& dc, const Opt& q, const Opt& s,
                     const py::object& stream) {
  spec(dh, "dh", kBf16, 2, 2);
  spec(qc, "qc", kFp8, 2, 2);
  spec(sc, "sc", kF32);
  const int64_t rows = dh.size(0), inter = dh.size(1), nt = inter / kTile;
  multiple(inter, "inter");
  if (qc.size(0) != rows || qc.size(1) != 2 * inter)
    bad_value("qc is [", qc.size(0), ", ", qc.size(1), "], dh [", rows, ", ", inter, "] needs [", rows, ", ",
              2 * inter, "]");
  holds(sc, "sc", rows * 2 * nt);
  buffer(dc, "dc", kBf16, rows * 2 * inter);
  buffer(q, "q", kFp8, rows * 2 * inter);
  buffer(s, "s", kF32, rows * 2 * nt);
  Place p;
  p.add(dh, "dh");
  p.add(qc, "qc");
  p.add(sc, "sc");
  p.add(dc, "dc");
  p.add(q, "q");
  p.add(s, "s");
  apart(q, "q", qc, "qc", "the checkpoint is read while q is written");
  apart(s, "s", sc, "sc", "the checkpoint is read while s is written");
  apart(dc, "dc", dh, "dh", "it is read while dc is written");
  const On on(p, stream);
  const Tensor a = on.fresh(dc, {rows, 2 * inter}, at::kBFloat16),
               b = on.fresh(q, {rows, 2 * inter}, at::kFloat8_e4m3fn), c = on.fresh(s, {rows, 2 * nt}, at::kFloat);
  check(fp8_swiglu_bwd_1x128(ptr(dh), ptr<uint8_t>(qc), ptr<float>(sc), rows, inter, ptr(a), ptr<uint8_t>(b),
                             ptr<float>(c), on.stream),
        "fp8_swiglu_bwd_1x128");
  return py::make_tuple(a, py::make_tuple(b, c));
}

py::tuple ckpt_128x1_t(const Tensor& q, const Tensor& s, std::optional<int64_t> padded, const Opt& qt,
                       const Opt& st, const py::object& stream) {
  spec(q, "q", kFp8, 2, 2);
  spec(s, "s", kF32);
  const int64_t M = q.size(0), K = q.size(1);
  multiple(K, "K");
  holds(s, "s", M * (K / kTile));
  const int64_t Mp = padded ? *padded : (M + kWgradTokenGroup - 1) / kWgradTokenGroup * kWgradTokenGroup;
  multiple(Mp, "Mp");
  if (Mp < M) bad_value("Mp = ", Mp, " is below the token count ", M);
  buffer(qt, "qt", kFp8, K * Mp);
  buffer(st, "st", kF32, Mp / kTile * K);
  Place p;
  p.add(q, "q");
  p.add(s, "s");
  p.add(qt, "qt");
  p.add(st, "st");
  const On on(p, stream);
  const Tensor a = on.fresh(qt, {K, Mp}, at::kFloat8_e4m3fn), b = on.fresh(st, {Mp / kTile, K}, at::kFloat);
  check(fp8_ckpt_128x1_t(ptr<uint8_t>(q), ptr<float>(s), M, K, Mp, ptr<uint8_t>(a), ptr<float>(b), on.stream),
        "fp8_ckpt_128x1_t");
  return py::make_tuple(a, b);
}

}  // namespace

PYBIND11_MODULE(_calls, m) {
  m.def("route", &route);
  m.def("route_bwd", &route_bwd);
  m.def("layout_contiguous", &layout_contiguous);
  m.def("layout_masked", &layout_masked);
  m.def("dispatch_1x128", &dispatch_1x128);
  m.def("combine", &combine);
  m.def("combine_bwd", &combine_bwd);
  m.def("swiglu_ckpt", &swiglu_ckpt);
  m.def("swiglu_bwd", &swiglu_bwd);
  m.def("ckpt_128x1_t", &ckpt_128x1_t);
}
