// mala_torch.cpp -- the torch side of the operators beside attention: checks of
// the tensors, allocation of outputs and workspaces, and the call into the C ABI.
//
// A decoding step's rotation takes 3 us on the GPU; the same checks and
// marshalling written in Python around ctypes took 20 us of host time, this
// takes 2. The package's functions of the same names call these.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <sstream>

#include "../../include/mala.h"
#include "mala_evict_check.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

template <typename... A>
[[noreturn]] void refuse(const char* where, const A&... parts) {
  std::ostringstream s;
  s << where << ": ";
  (s << ... << parts);
  throw py::value_error(s.str());
}

// The package's MalaError, set when the package loads this module (under whatever name it has
// itself); never released, as the interpreter may be gone by then.
PyObject* error_class = nullptr;

void check(int rc, const char* where) {
  if (rc == MALA_OK) return;
  const auto cls = py::reinterpret_borrow<py::object>(error_class ? error_class : PyExc_RuntimeError);
  const py::object error = cls(rc, where);
  PyErr_SetObject(cls.ptr(), error.ptr());
  throw py::error_already_set();
}

// The call's device (the current one), its stream, and allocation in that
// stream's order (torch reuses a freed block by the stream it was allocated on).
struct Place {
  const char* where;
  c10::DeviceIndex dev;
  c10::cuda::CUDAStream stream;
  bool current;  // torch's current stream

  Place(const char* where_, const Tensor& x, const py::object& s)
      : where(where_), dev(device(where_, x)), stream(pick(dev, s)), current(stream == c10::cuda::getCurrentCUDAStream(dev)) {}

  static c10::DeviceIndex device(const char* where, const Tensor& x) {
    if (!x.is_cuda() || x.get_device() != c10::cuda::current_device())
      refuse(where, "tensors must be on the current CUDA device, got ", x.device());
    return static_cast<c10::DeviceIndex>(x.get_device());
  }
  static c10::cuda::CUDAStream pick(c10::DeviceIndex dev, const py::object& s) {
    if (s.is_none()) return c10::cuda::getCurrentCUDAStream(dev);
    const py::object h = py::isinstance<py::int_>(s) ? s : py::object(s.attr("cuda_stream"));
    return c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(h.cast<uintptr_t>()), dev);
  }
  void* handle() const { return stream.stream(); }

  void need(const Tensor& x, at::ScalarType type, bool contiguous = true) const {
    if (x.scalar_type() != type || x.get_device() != dev || (contiguous && !x.is_contiguous()))
      refuse(where, "expected a ", contiguous ? "contiguous " : "", c10::toString(type), " tensor on device ",
             static_cast<int>(dev), ", got ", x.dtype(), " ", x.sizes(), " with strides ", x.strides(), " on ", x.device());
  }
  void need(const OptTensor& x, at::ScalarType type, bool contiguous = true) const {
    if (x) need(*x, type, contiguous);
  }
  void shape(const Tensor& x, const char* name, at::IntArrayRef want) const {
    if (x.sizes() != want) refuse(where, name, " must have shape ", want, ", got ", x.sizes());
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (!current) guard.reset_stream(stream);
    return at::empty(size, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, dev)));
  }
  // (pointer, bytes) of the workspace: the caller's, or a new one, kept in `hold`
  std::pair<void*, size_t> scratch(const OptTensor& given, size_t bytes, Tensor& hold) const {
    if (given) {
      if (given->get_device() != dev || !given->is_contiguous())
        refuse(where, "the workspace must be contiguous and on device ", static_cast<int>(dev));
      return {given->data_ptr(), given->nbytes()};
    }
    if (bytes == 0) return {nullptr, 0};
    hold = empty({static_cast<int64_t>(bytes)}, at::kByte);
    return {hold.data_ptr(), bytes};
  }
};

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

void* ptr(const OptTensor& x) { return x ? x->data_ptr() : nullptr; }
float* fptr(const Tensor& x) { return static_cast<float*>(x.data_ptr()); }
float* fptr(const OptTensor& x) { return static_cast<float*>(ptr(x)); }
int32_t* iptr(const Tensor& x) { return static_cast<int32_t*>(x.data_ptr()); }
int32_t* iptr(const OptTensor& x) { return static_cast<int32_t*>(ptr(x)); }
// a size as the C ABI's int; one that does not fit is refused there as out of range
int c_int(const char* where, int64_t x) {
  if (x > INT32_MAX || x < INT32_MIN) refuse(where, "the size ", x, " does not fit");
  return static_cast<int>(x);
}

// A tensor [..., H, d] whose leading axes step through its tokens with one stride.
struct Rows {
  int64_t tokens, heads, d, tok, head;
};
Rows rows(const char* where, const Tensor& x) {
  const auto size = x.sizes(), stride = x.strides();
  const int64_t n = x.dim();
  if (n < 3 || stride[n - 1] != 1) refuse(where, "expected [..., H, d] with adjacent values in a head, got ", size);
  int64_t tokens = 1, step = 0;
  for (int64_t i = n - 3; i >= 0; --i) {
    if (size[i] == 1) continue;
    if (tokens == 1) step = stride[i];
    else if (tokens > 0 && stride[i] != step * tokens) refuse(where, "tokens must lie at one stride, got ", stride);
    tokens *= size[i];
  }
  // the stride of an axis with one entry means nothing
  return {tokens, size[n - 2], size[n - 1], tokens > 1 ? step : 0, size[n - 2] > 1 ? stride[n - 2] : 0};
}

// positions, inv_freq and the pairs of each axis
struct Angles {
  int32_t sections[8];
  int n_axes, rotary_dim;
};
Angles angles(const Place& at_, const Tensor& positions, const Tensor& inv_freq,
              const std::optional<std::vector<int64_t>>& sections, int64_t T) {
  at_.need(positions, kI32);
  at_.need(inv_freq, kF32);
  Angles a = {};
  a.rotary_dim = c_int(at_.where, 2 * inv_freq.numel());
  a.n_axes = sections ? static_cast<int>(std::min<size_t>(sections->size(), 8)) : 1;
  a.sections[0] = a.rotary_dim / 2;
  for (int i = 0; sections && i < a.n_axes; ++i) a.sections[i] = c_int(at_.where, (*sections)[i]);
  // (as many values in another layout, a token's axes side by side, say, would be read as other positions)
  if (positions.numel() != a.n_axes * T || (a.n_axes > 1 && positions.dim() > 1 && positions.size(0) != a.n_axes))
    refuse(at_.where, "positions must be [", a.n_axes, ", ", T, "], got ", positions.sizes());
  return a;
}

using Three = std::tuple<OptTensor, OptTensor, OptTensor>;

Three rope(const OptTensor& q, const OptTensor& k, const OptTensor& v, const Tensor& positions, const Tensor& inv_freq,
           const std::optional<std::vector<int64_t>>& sections, unsigned flags, const std::optional<Three>& out,
           const py::object& stream) {
  const char* where = "mala_rope";
  const OptTensor* in[3] = {&q, &k, &v};
  const OptTensor& first = q ? q : k ? k : v;
  if (!first) refuse(where, "no tensor given");
  const Place place(where, *first, stream);
  OptTensor to[3];
  if (out) std::tie(to[0], to[1], to[2]) = *out;
  int64_t strides[12] = {}, T = -1, d = 0, heads[3] = {1, 1, 1};
  for (int w = 0; w < 3; ++w) {
    if (!*in[w] && !to[w]) continue;
    if (!*in[w] || (out && !to[w])) refuse(where, "each of q, k and v needs both its input and its output");
    const Tensor& x = **in[w];
    place.need(x, kBf16, false);
    if (!out) to[w] = place.empty(x.sizes(), kBf16);
    place.need(*to[w], kBf16, false);
    const Rows a = rows(where, x), b = rows(where, *to[w]);
    if (a.tokens != b.tokens || a.heads != b.heads || a.d != b.d) refuse(where, "an output's shape is not its input's");
    if (T >= 0 && (a.tokens != T || a.d != d)) refuse(where, "q, k and v disagree in tokens or head size");
    T = a.tokens;
    d = a.d;
    heads[w] = a.heads;
    strides[2 * w] = a.tok;
    strides[2 * w + 1] = a.head;
    strides[6 + 2 * w] = b.tok;
    strides[7 + 2 * w] = b.head;
  }
  if (k && v && heads[1] != heads[2]) refuse(where, "k and v disagree in heads");
  const Angles an = angles(place, positions, inv_freq, sections, T);
  check(mala_rope(ptr(q), ptr(k), ptr(v), ptr(to[0]), ptr(to[1]), ptr(to[2]), strides, iptr(positions), fptr(inv_freq),
                  c_int(where, T), c_int(where, heads[0]), c_int(where, k ? heads[1] : heads[2]), c_int(where, d),
                  an.rotary_dim, an.sections, an.n_axes, flags, place.handle()),
        where);
  return {to[0], to[1], to[2]};
}

OptTensor rope_append(const OptTensor& q, const Tensor& k, const Tensor& v, const Tensor& positions,
                      const Tensor& inv_freq, const Tensor& k_pages, const Tensor& v_pages, const Tensor& block_table,
                      const Tensor& seqlens_k, const OptTensor& cu_seqlens,
                      const std::optional<std::vector<int64_t>>& sections, unsigned flags, const OptTensor& out,
                      const py::object& stream) {
  const char* where = "mala_rope_append";
  const Place place(where, k, stream);
  place.need(q, kBf16, false);
  place.need(k, kBf16, false);
  place.need(v, kBf16, false);
  place.need(out, kBf16, false);
  place.need(k_pages, kBf16);
  place.need(v_pages, kBf16);
  place.need(block_table, kI32);
  place.need(seqlens_k, kI32);
  place.need(cu_seqlens, kI32);
  const Rows rk = rows(where, k), rv = rows(where, v);
  if (rk.tokens != rv.tokens || rk.heads != rv.heads || rk.d != rv.d)
    refuse(where, "k and v disagree in tokens, heads or head size");
  const int64_t S = seqlens_k.numel();
  if (k_pages.dim() != 4 || k_pages.size(2) != rk.heads || k_pages.size(3) != rk.d || v_pages.sizes() != k_pages.sizes())
    refuse(where, "pools must be [num_pages, page, ", rk.heads, ", ", rk.d, "], got ", k_pages.sizes(), " and ",
           v_pages.sizes());
  if (block_table.dim() != 2 || block_table.size(0) != S) refuse(where, "block_table must be [", S, ", max_pages]");
  if (cu_seqlens) place.shape(*cu_seqlens, "cu_seqlens", {S + 1});
  OptTensor to = out;
  int64_t strides[8] = {0, 0, rk.tok, rk.head, rv.tok, rv.head, 0, 0}, Hq = 1;
  if (q) {
    if (!to) to = place.empty(q->sizes(), kBf16);
    const Rows a = rows(where, *q), b = rows(where, *to);
    if (a.tokens != rk.tokens || a.d != rk.d || b.tokens != a.tokens || b.heads != a.heads || b.d != a.d)
      refuse(where, "q, out and k disagree in tokens, heads or head size");
    Hq = a.heads;
    strides[0] = a.tok;
    strides[1] = a.head;
    strides[6] = b.tok;
    strides[7] = b.head;
  } else if (out) {
    refuse(where, "out without q");
  }
  const Angles an = angles(place, positions, inv_freq, sections, rk.tokens);
  check(mala_rope_append(ptr(q), k.data_ptr(), v.data_ptr(), ptr(to), strides, iptr(positions), fptr(inv_freq),
                         k_pages.data_ptr(), v_pages.data_ptr(), iptr(block_table), iptr(seqlens_k), iptr(cu_seqlens),
                         c_int(where, S), c_int(where, rk.tokens), c_int(where, Hq), c_int(where, rk.heads),
                         c_int(where, k_pages.size(0)), c_int(where, k_pages.size(1)), c_int(where, block_table.size(1)),
                         c_int(where, rk.d), an.rotary_dim, an.sections, an.n_axes, flags, place.handle()),
        where);
  return to;
}

// The masses to write: the output given, or a new one as long as the input (or `ld`).
Tensor mass_out(const Place& place, const OptTensor& mass, const OptTensor& out, int64_t B, int64_t Hkv, int64_t ld) {
  place.need(mass, kF32);
  place.need(out, kF32);
  if (mass) ld = mass->size(-1);
  else if (out) ld = out->size(-1);
  if (mass) place.shape(*mass, "mass", {B, Hkv, ld});
  if (!out) return place.empty({B, Hkv, ld}, kF32);
  place.shape(*out, "out", {B, Hkv, ld});
  return *out;
}

Tensor key_mass(const Tensor& q, const Tensor& k, const Tensor& lse, double scale, int64_t window, const OptTensor& mass,
                double decay, const OptTensor& out, const OptTensor& workspace, const py::object& stream) {
  const char* where = "mala_key_mass";
  const Place place(where, q, stream);
  place.need(q, kBf16);
  place.need(k, kBf16);
  place.need(lse, kF32);
  if (q.dim() != 4 || k.dim() != 4) refuse(where, "q and k must be [B, L, H, d], got ", q.sizes(), " and ", k.sizes());
  const int64_t B = q.size(0), Lq = q.size(1), Hq = q.size(2), d = q.size(3), Lk = k.size(1), Hkv = k.size(2);
  place.shape(k, "k", {B, Lk, Hkv, d});
  place.shape(lse, "lse", {B, Hq, Lq});
  const Tensor to = mass_out(place, mass, out, B, Hkv, Lk);
  const int b = c_int(where, B), hq = c_int(where, Hq), hkv = c_int(where, Hkv), lq = c_int(where, Lq),
            lk = c_int(where, Lk), w = c_int(where, window);
  Tensor hold;
  const auto ws = place.scratch(workspace, workspace ? 0 : mala_key_mass_workspace_size(b, hq, hkv, lq, lk, w), hold);
  check(mala_key_mass(q.data_ptr(), k.data_ptr(), fptr(lse), fptr(mass), fptr(to), b, hq, hkv, lq, lk, c_int(where, d),
                      static_cast<float>(scale), w, static_cast<float>(decay), c_int(where, to.size(2)), ws.first,
                      ws.second, place.handle()),
        where);
  return to;
}

Tensor key_mass_varlen(const Tensor& q, const Tensor& k, const Tensor& lse, const Tensor& cu_q, const Tensor& cu_k,
                       int64_t max_q, int64_t max_k, double scale, int64_t window, const OptTensor& mass, double decay,
                       const OptTensor& out, const OptTensor& workspace, const py::object& stream) {
  const char* where = "mala_key_mass_varlen";
  const Place place(where, q, stream);
  place.need(q, kBf16);
  place.need(k, kBf16);
  place.need(lse, kF32);
  place.need(cu_q, kI32);
  place.need(cu_k, kI32);
  if (q.dim() != 3 || k.dim() != 3) refuse(where, "q and k must be [rows, H, d], got ", q.sizes(), " and ", k.sizes());
  const int64_t tq = q.size(0), Hq = q.size(1), d = q.size(2), tk = k.size(0), Hkv = k.size(1), S = cu_q.numel() - 1;
  place.shape(k, "k", {tk, Hkv, d});
  place.shape(lse, "lse", {Hq, tq});
  place.shape(cu_k, "cu_seqlens_k", {S + 1});
  const Tensor to = mass_out(place, mass, out, S, Hkv, max_k);
  const int s = c_int(where, S), hq = c_int(where, Hq), hkv = c_int(where, Hkv), mq = c_int(where, max_q),
            mk = c_int(where, max_k), w = c_int(where, window), n_q = c_int(where, tq);
  Tensor hold;
  const auto ws = place.scratch(
      workspace, workspace ? 0 : mala_key_mass_varlen_workspace_size(s, hq, hkv, mq, mk, n_q, w), hold);
  check(mala_key_mass_varlen(q.data_ptr(), k.data_ptr(), fptr(lse), iptr(cu_q), iptr(cu_k), fptr(mass), fptr(to), s, mq,
                             mk, n_q, c_int(where, tk), hq, hkv, c_int(where, d), static_cast<float>(scale), w,
                             static_cast<float>(decay), c_int(where, to.size(2)), ws.first, ws.second, place.handle()),
        where);
  return to;
}

std::tuple<Tensor, Tensor, Tensor, OptTensor, int, Tensor> decode_paged_mass(
    const Tensor& q, const Tensor& k_pages, const Tensor& v_pages, const Tensor& block_table, const Tensor& seqlens_k,
    double scale, double tau, const OptTensor& mass, double decay, const OptTensor& out, int n_splits, bool keep_map,
    const OptTensor& workspace, const py::object& stream) {
  const char* where = "mala_decode_paged_mass";
  const Place place(where, q, stream);
  place.need(q, kBf16);
  place.need(k_pages, kBf16);
  place.need(v_pages, kBf16);
  place.need(block_table, kI32);
  place.need(seqlens_k, kI32);
  if (q.dim() != 3) refuse(where, "q must be [B, Hq, d], got ", q.sizes());
  const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2);
  if (k_pages.dim() != 4 || k_pages.size(3) != d || v_pages.sizes() != k_pages.sizes())
    refuse(where, "pools must be [num_pages, page, Hkv, ", d, "], got ", k_pages.sizes(), " and ", v_pages.sizes());
  if (block_table.dim() != 2 || block_table.size(0) != B) refuse(where, "block_table must be [", B, ", max_pages]");
  place.shape(seqlens_k, "seqlens_k", {B});
  const int64_t page = k_pages.size(1), Hkv = k_pages.size(2), maxp = block_table.size(1);
  const Tensor to = mass_out(place, mass, out, B, Hkv, maxp * page);
  const int b = c_int(where, B), hq = c_int(where, Hq), hkv = c_int(where, Hkv), di = c_int(where, d),
            pg = c_int(where, page), mp = c_int(where, maxp);
  if (!(tau > 0)) n_splits = 0;  // nothing is split by count
  else if (n_splits == 0) n_splits = mala_decode_default_splits(b, hkv, c_int(where, maxp * page), pg);
  const Tensor o = place.empty(q.sizes(), kBf16), lse = place.empty({B, Hq}, kF32), kept = place.empty({B * Hq}, kI32);
  OptTensor km;
  if (keep_map) {
    km = place.empty({B, Hq, maxp}, at::kByte);
    c10::cuda::CUDAStreamGuard guard(place.stream);
    km->fill_(255);
  }
  Tensor hold;
  const auto ws =
      place.scratch(workspace, workspace ? 0 : mala_decode_mass_workspace_size(b, hq, hkv, di, pg, mp, n_splits), hold);
  check(mala_decode_paged_mass(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), iptr(block_table), iptr(seqlens_k),
                               o.data_ptr(), fptr(lse), fptr(mass), fptr(to), b, hq, hkv, c_int(where, k_pages.size(0)),
                               pg, mp, di, static_cast<float>(scale), static_cast<float>(tau),
                               static_cast<float>(decay), c_int(where, to.size(2)), n_splits, ws.first, ws.second,
                               iptr(kept), static_cast<uint8_t*>(ptr(km)), place.handle()),
        where);
  return {o, lse, kept, km, n_splits, to};
}

std::tuple<Tensor, Tensor, Tensor> evict_select(const Tensor& mass, const Tensor& seqlens_k, int64_t budget,
                                                int64_t n_sink, int64_t n_recent, const OptTensor& mass_to,
                                                const py::object& stream) {
  const char* where = "mala_evict_select";
  const Place place(where, mass, stream);
  place.need(mass, kF32);
  place.need(seqlens_k, kI32);
  if (mass.dim() != 3) refuse(where, "mass must be [B, Hkv, ld], got ", mass.sizes());
  const int64_t B = mass.size(0), Hkv = mass.size(1);
  place.shape(seqlens_k, "seqlens_k", {B});
  if (budget < 1) refuse(where, "budget must be at least 1, got ", budget);
  const Tensor index = place.empty({B, Hkv, budget}, kI32), fresh = place.empty({B}, kI32);
  place.need(mass_to, kF32);
  const Tensor out = mass_to ? *mass_to : place.empty({B, Hkv, budget}, kF32);
  if (out.dim() != 3 || out.size(0) != B || out.size(1) != Hkv) refuse(where, "mass_out must be [", B, ", ", Hkv, ", ld]");
  check(mala_evict_select(fptr(mass), iptr(seqlens_k), iptr(index), iptr(fresh), fptr(out), c_int(where, B),
                          c_int(where, Hkv), c_int(where, mass.size(2)), c_int(where, budget), c_int(where, n_sink),
                          c_int(where, n_recent), c_int(where, out.size(2)), place.handle()),
        where);
  return {index, fresh, out};
}

// The pools and tables of a copy of [B, Hkv, budget] rows, checked.
struct Copy {
  const Tensor &k, &v, &table, &to, &ko, &vo;
  int B, Hkv, budget, pages, out_pages, page, max_pages, max_out, d;

  Copy(const Place& at_, int64_t B_, int64_t Hkv_, int64_t budget_, const Tensor& k_, const Tensor& v_,
       const Tensor& table_, const Tensor& to_, const OptTensor& k_out, const OptTensor& v_out)
      : k(k_), v(v_), table(table_), to(to_), ko(k_out ? *k_out : k_), vo(v_out ? *v_out : v_) {
    const char* where = at_.where;
    for (const Tensor* x : {&table, &to}) at_.need(*x, kI32);
    for (const Tensor* x : {&k, &v, &ko, &vo}) at_.need(*x, kBf16);
    const auto pool = k.sizes(), out = ko.sizes();
    if (pool.size() != 4 || out.size() != 4 || pool[2] != Hkv_ || pool.slice(1) != out.slice(1) || v.sizes() != pool ||
        vo.sizes() != out)
      refuse(where, "pools must be [num_pages, page, ", Hkv_, ", d], got ", pool, ", ", v.sizes(), ", ", out, " and ",
             vo.sizes());
    if (table.dim() != 2 || table.size(0) != B_ || to.dim() != 2 || to.size(0) != B_)
      refuse(where, "block_table and out_table must be [", B_, ", pages]");
    B = c_int(where, B_);
    Hkv = c_int(where, Hkv_);
    budget = c_int(where, budget_);
    pages = c_int(where, pool[0]);
    out_pages = c_int(where, out[0]);
    page = c_int(where, pool[1]);
    d = c_int(where, pool[3]);
    max_pages = c_int(where, table.size(1));
    max_out = c_int(where, to.size(1));
  }
  void run(const Place& at_, const Tensor& index, const Tensor& lens) const {
    check(mala_evict_gather(k.data_ptr(), v.data_ptr(), iptr(table), iptr(index), iptr(lens), ko.data_ptr(),
                            vo.data_ptr(), iptr(to), B, Hkv, budget, pages, out_pages, page, max_pages, max_out, d,
                            at_.handle()),
          at_.where);
  }
};

std::tuple<Tensor, Tensor> evict_gather(const Tensor& index, const Tensor& new_seqlens, const Tensor& k_pages,
                                        const Tensor& v_pages, const Tensor& block_table, const Tensor& out_table,
                                        const OptTensor& k_out, const OptTensor& v_out, const py::object& stream) {
  const char* where = "mala_evict_gather";
  const Place place(where, index, stream);
  for (const Tensor* x : {&index, &new_seqlens}) place.need(*x, kI32);
  if (index.dim() != 3) refuse(where, "index must be [B, Hkv, budget], got ", index.sizes());
  place.shape(new_seqlens, "new_seqlens", {index.size(0)});
  const Copy copy(place, index.size(0), index.size(1), index.size(2), k_pages, v_pages, block_table, out_table, k_out,
                  v_out);
  copy.run(place, index, new_seqlens);
  return {copy.ko, copy.vo};
}

std::tuple<Tensor, Tensor, Tensor> evict(const Tensor& mass, const Tensor& seqlens_k, int64_t budget,
                                         const Tensor& k_pages, const Tensor& v_pages, const Tensor& block_table,
                                         const Tensor& out_table, int64_t n_sink, int64_t n_recent,
                                         const OptTensor& k_out, const OptTensor& v_out, const OptTensor& mass_to,
                                         const py::object& stream) {
  const char* where = "mala_evict_gather";
  const Place place(where, mass, stream);
  if (mass.dim() != 3) refuse(where, "mass must be [B, Hkv, ld], got ", mass.sizes());
  // what the copy would refuse is refused before the selection writes anything
  const Copy copy(place, mass.size(0), mass.size(1), budget, k_pages, v_pages, block_table, out_table, k_out, v_out);
  if (budget >= 1)  // (the selection refuses others; its lists have no pointers yet, so the masses' stand for them)
    check(mala::check_gather(k_pages.data_ptr(), v_pages.data_ptr(), iptr(block_table), fptr(mass), fptr(mass),
                             copy.ko.data_ptr(), copy.vo.data_ptr(), iptr(out_table), copy.B, copy.Hkv, copy.budget,
                             copy.pages, copy.out_pages, copy.page, copy.max_pages, copy.max_out, copy.d),
          where);
  auto rows_left = evict_select(mass, seqlens_k, budget, n_sink, n_recent, mass_to, stream);
  copy.run(place, std::get<0>(rows_left), std::get<1>(rows_left));
  return rows_left;
}

}  // namespace

PYBIND11_MODULE(mala_torch, m) {
  m.def("set_error_class", [](const py::object& cls) { error_class = py::object(cls).release().ptr(); });
  m.def("rows", [](const Tensor& x) {
    const Rows r = rows("rows", x);
    return py::make_tuple(r.tokens, r.heads, r.d, r.tok, r.head);
  });
  m.def("rope", &rope);
  m.def("rope_append", &rope_append);
  m.def("key_mass", &key_mass);
  m.def("key_mass_varlen", &key_mass_varlen);
  m.def("decode_paged_mass", &decode_paged_mass);
  m.def("evict_select", &evict_select);
  m.def("evict_gather", &evict_gather);
  m.def("evict", &evict);
}
