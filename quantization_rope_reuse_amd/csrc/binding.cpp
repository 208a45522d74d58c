// Native part of the Python binding (hkv.py) for calls whose GPU time is a
// few microseconds: tensor checks, structures and the library call in one
// step.  It computes nothing; every call goes to the C ABI through the
// addresses that hkv.py hands over from the loaded library.
//
// Each function returns the library's status, with the outputs where it makes
// them; what the C ABI cannot see (types, shapes, devices) raises ValueError.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "hkv.h"
#include "hkv_serve.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

struct Calls {
  decltype(&hkv_plan_step) plan = nullptr;
  decltype(&hkv_rope_heads) rope = nullptr;
  decltype(&hkv_append_tokens) append = nullptr;
  decltype(&hkv_attend_records) attend = nullptr;
  decltype(&hkv_attend_workspace_bytes) attend_bytes = nullptr;
  decltype(&hkv_fetch_dequant_rope_shift) fetch = nullptr;
  decltype(&hkv_fetch_dequant_rope_shift_tokens) fetch_tokens = nullptr;
  decltype(&hkv_record_bytes) record_bytes = nullptr;
} calls;

void bind(const py::dict& at) {
  auto set = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(py::cast<uintptr_t>(at[name]));
  };
  set(calls.plan, "hkv_plan_step");
  set(calls.rope, "hkv_rope_heads");
  set(calls.append, "hkv_append_tokens");
  set(calls.attend, "hkv_attend_records");
  set(calls.attend_bytes, "hkv_attend_workspace_bytes");
  set(calls.fetch, "hkv_fetch_dequant_rope_shift");
  set(calls.fetch_tokens, "hkv_fetch_dequant_rope_shift_tokens");
  set(calls.record_bytes, "hkv_record_bytes");
}

// A library call, without the interpreter's lock: a launch waits where the
// stream's queue is full.
template <class Call, class... Args>
int launch(Call call, Args... args) {
  py::gil_scoped_release unlocked;
  return call(args...);
}

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

// Every tensor of a call on one GPU: the kernels dereference their addresses.
class OneGpu {
 public:
  explicit OneGpu(const char* call) : call_(call) {}
  OneGpu& operator()(const Tensor& t) {
    if (!t.is_cuda())
      refuse(std::string(call_) + ": tensor arguments must be on a GPU, got one on " + t.device().str());
    if (!device_)
      device_ = t.device();
    else if (t.device() != *device_)
      refuse(std::string(call_) + ": tensor arguments on " + device_->str() + " and " + t.device().str());
    return *this;
  }
  OneGpu& operator()(const Maybe& t) { return t ? (*this)(*t) : *this; }
  at::Device device() const { return *device_; }

 private:
  const char* call_;
  std::optional<at::Device> device_;
};

c10::hip::HIPStream stream_of(const py::object& stream, at::Device device) {
  if (stream.is_none()) return c10::hip::getCurrentHIPStream(device.index());
  // a torch stream, or a handle: any whole number
  const py::object handle =
      PyIndex_Check(stream.ptr()) ? stream : py::getattr(stream, "cuda_stream", py::none());
  if (!PyIndex_Check(handle.ptr())) refuse("stream must be a torch stream or a stream's handle");
  const uintptr_t at = py::cast<uintptr_t>(py::reinterpret_steal<py::object>(PyNumber_Index(handle.ptr())));
  return c10::hip::getStreamFromExternal(reinterpret_cast<hipStream_t>(at), device.index());
}

// A tensor that a call on `stream` makes for itself.  The allocator orders
// the use of a block on the stream that was current when it was handed out
// alone: one from another stream's pool may still be in use there when the
// call writes it, and handed out there again while the call still works.
Tensor made_on(at::IntArrayRef sizes, const at::TensorOptions& options, c10::hip::HIPStream stream) {
  const c10::hip::HIPStream before = c10::hip::getCurrentHIPStream(stream.device_index());
  if (before.stream() == stream.stream()) return at::empty(sizes, options);
  struct Current {
    c10::hip::HIPStream before;
    ~Current() { c10::hip::setCurrentHIPStream(before); }
  } restore{before};
  c10::hip::setCurrentHIPStream(stream);
  return at::empty(sizes, options);
}

int32_t small(int64_t x, const char* what) {
  if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return static_cast<int32_t>(x);
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return HKV_F32;
    case at::kHalf: return HKV_F16;
    case at::kBFloat16: return HKV_BF16;
    default: return -1;
  }
}

std::string dtype_name(const Tensor& t) {
  return py::cast<std::string>(py::str(py::cast(t).attr("dtype")));
}

int32_t* ints(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kInt || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous int32 tensor");
  return static_cast<int32_t*>(t.data_ptr());
}

// Entries per row and row stride of an int32 [n_requests, max_blocks] tensor;
// strides that address nothing may be anything.
struct Table {
  int32_t* data;
  int64_t blocks, stride;
};
Table table_of(const Tensor& t) {
  if (t.dim() != 2 || t.scalar_type() != at::kInt ||
      (t.numel() > 0 && t.size(1) > 1 && t.stride(1) != 1))
    refuse("block_table must be an int32 [n_requests, max_blocks] tensor, last axis contiguous");
  return {static_cast<int32_t*>(t.data_ptr()), t.size(1),
          t.size(0) > 1 && t.numel() > 0 ? t.stride(0) : t.size(1)};
}

hkv_heads heads_of(const Tensor& t, const char* name) {
  if (t.dim() != 3 || t.size(2) != HKV_HEAD_DIM || t.stride(2) != 1)
    refuse(std::string(name) + " must be a [n_tokens, n_heads, 128] tensor, last axis contiguous");
  if (dtype_of(t) < 0) refuse("unsupported dtype " + dtype_name(t) + " of " + name);
  // the stride of an axis of one entry addresses nothing and may be anything
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0,
          small(t.size(1), "n_heads")};
}

// Records [L, n_blocks, bytes]: the last axis must hold a whole record, since
// the library can only compare strides.
hkv_records records_of(const Tensor& r, int fmt, int64_t block_tokens, int64_t heads) {
  if (r.scalar_type() != at::kByte || r.dim() != 3 || r.stride(2) != 1)
    refuse("records must be a uint8 [L, n_blocks, bytes] tensor, last axis contiguous");
  const int64_t bytes = calls.record_bytes(fmt, small(block_tokens, "block_tokens"),
                                           small(heads, "n_kv_heads"), HKV_HEAD_DIM);
  if (r.size(2) < bytes)
    refuse("records hold " + std::to_string(r.size(2)) + " bytes per block; a " +
           (fmt == HKV_INT4 ? "int4" : "fp8") + " record of " + std::to_string(block_tokens) +
           " tokens x " + std::to_string(heads) + " heads needs " + std::to_string(bytes));
  return {r.data_ptr(), r.stride(0), r.stride(1)};
}

// One layer's records, [n_blocks, bytes] or [1, n_blocks, bytes].
struct Pool {
  hkv_shape shape;
  hkv_records records;
};
Pool pool_of(const Tensor& records, int fmt, int64_t block_tokens, int64_t heads) {
  const Tensor r = records.dim() == 3 ? records : records.unsqueeze(0);
  if (r.dim() != 3 || r.size(0) != 1)
    refuse("records must be one layer's uint8 [n_blocks, bytes] tensor");
  return {{1, small(r.size(1), "n_blocks"), small(block_tokens, "block_tokens"),
           small(heads, "n_kv_heads"), HKV_HEAD_DIM},
          records_of(r, fmt, block_tokens, heads)};
}

// out: the six tensors of a plan, or none to make them.
py::tuple plan_step(const Tensor& kv_len, const Tensor& new_tokens, const Tensor& block_table,
                    const Tensor& free_blocks, const Tensor& free_count, int64_t block_tokens,
                    int64_t n_tokens, const std::optional<std::vector<Tensor>>& out,
                    const py::object& stream) {
  OneGpu on("plan_step");
  on(kv_len)(new_tokens)(block_table)(free_blocks)(free_count);
  const auto at_stream = stream_of(stream, on.device());
  const int64_t R = kv_len.numel();
  need(n_tokens >= 0, "n_tokens must not be negative");
  std::vector<Tensor> o;
  if (out) {
    need(out->size() == 6, "out must be a StepPlan");
    o = *out;
    for (const Tensor& t : o) on(t);
  } else {
    const auto i32 = kv_len.options().dtype(at::kInt);
    const auto ints_of = [&](int64_t n) { return made_on({n}, i32, at_stream); };
    o = {ints_of(R), ints_of(R + 1), ints_of(n_tokens),
         made_on({n_tokens}, i32.dtype(at::kLong), at_stream), ints_of(R), ints_of(1)};
  }
  const Tensor &len_out = o[0], &q_start = o[1], &positions = o[2], &slots = o[3], &refused = o[4],
               &count_out = o[5];
  need(positions.numel() == n_tokens, "out must hold n_tokens positions");
  const Table table = table_of(block_table);
  need(block_table.size(0) == R && new_tokens.numel() == R && len_out.numel() == R &&
           refused.numel() == R && q_start.numel() == R + 1,
       "kv_len, new_tokens, block_table, refused [n_requests] and q_start [n_requests + 1] must agree");
  need(free_count.numel() == 1 && count_out.numel() == 1, "free_count must hold one element");
  need(slots.scalar_type() == at::kLong && slots.is_contiguous() && slots.numel() == positions.numel(),
       "slots must be a contiguous int64 tensor as long as positions");
  hkv_step s;
  s.n_requests = small(R, "n_requests");
  s.block_tokens = small(block_tokens, "block_tokens");
  s.max_blocks = small(table.blocks, "max_blocks");
  s.n_tokens = small(n_tokens, "n_tokens");
  s.kv_len = ints(kv_len, "kv_len");
  s.new_tokens = ints(new_tokens, "new_tokens");
  s.block_table = table.data;
  s.table_stride = table.stride;
  s.free_blocks = ints(free_blocks, "free_blocks");
  s.free_capacity = small(free_blocks.numel(), "free_capacity");
  s.free_count = ints(free_count, "free_count");
  s.free_count_out = ints(count_out, "free_count");
  s.kv_len_out = ints(len_out, "kv_len");
  s.q_start = ints(q_start, "q_start");
  s.positions = ints(positions, "positions");
  s.slots = static_cast<int64_t*>(slots.data_ptr());
  s.refused = ints(refused, "refused");
  const int st = launch(calls.plan, &s, at_stream.stream());
  return py::make_tuple(st, o[0], o[1], o[2], o[3], o[4], o[5]);
}

// axes: address of an hkv_rope_axes.
py::tuple rope_heads(const Tensor& q, const Maybe& k, const Tensor& positions, uintptr_t axes,
                     bool inverse, const Maybe& q_out, const Maybe& k_out, const py::object& stream) {
  OneGpu on("rope_heads");
  on(q)(k)(positions)(q_out)(k_out);
  const auto at_stream = stream_of(stream, on.device());
  const auto* a = reinterpret_cast<const hkv_rope_axes*>(axes);
  const hkv_heads qh = heads_of(q, "q");
  const int64_t n = q.size(0);
  const int64_t rows = positions.dim() == 1 ? 1 : positions.size(0);
  if ((positions.dim() != 1 && positions.dim() != 2) || positions.scalar_type() != at::kInt ||
      rows != a->n_axes || positions.size(-1) != n || (n > 1 && positions.stride(-1) != 1))
    refuse("positions must be int32 [" + std::to_string(a->n_axes) + ", n_tokens], last axis contiguous");
  const Tensor qo = q_out ? *q_out : made_on(q.sizes(), q.options(), at_stream);
  const hkv_heads qoh = heads_of(qo, "q_out");
  hkv_heads kh = {}, koh = {};
  Maybe ko = k_out;
  bool same = qo.sizes() == q.sizes() && qo.scalar_type() == q.scalar_type();
  if (k) {
    if (!ko) ko = made_on(k->sizes(), k->options(), at_stream);
    kh = heads_of(*k, "k");
    koh = heads_of(*ko, "k_out");
    same = same && k->size(0) == n && ko->sizes() == k->sizes() &&
           k->scalar_type() == q.scalar_type() && ko->scalar_type() == q.scalar_type();
  }
  need(same, "q, k and their outputs must share dtype and n_tokens, each output its input's shape");
  const int st = launch(calls.rope, a, static_cast<const int32_t*>(positions.data_ptr()),
                        rows > 1 ? positions.stride(0) : 0, small(n, "n_tokens"), &qh, &kh, &qoh,
                        &koh, dtype_of(q), inverse ? 1 : 0, at_stream.stream());
  return py::make_tuple(st, qo, ko);
}

int append_tokens(const Tensor& k, const Tensor& v, const Tensor& slots, const Tensor& records,
                  int fmt, int64_t block_tokens, const py::object& stream) {
  OneGpu on("append_tokens");
  on(k)(v)(slots)(records);
  need(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type(), "k and v must share shape and dtype");
  const hkv_heads kh = heads_of(k, "k"), vh = heads_of(v, "v");
  need(slots.scalar_type() == at::kLong && slots.is_contiguous() && slots.numel() == k.size(0),
       "slots must be a contiguous int64 tensor of n_tokens elements");
  const Pool pool = pool_of(records, fmt, block_tokens, k.size(1));
  return launch(calls.append, &pool.shape, fmt, &kh, &vh, dtype_of(k), small(k.size(0), "n_tokens"),
                static_cast<const int64_t*>(slots.data_ptr()), &pool.records,
                stream_of(stream, on.device()).stream());
}

// workspace: True (made here where one is needed), None or a uint8 tensor.
// max_queries: -1 for the default.
py::tuple attend_records(const Tensor& q, const Tensor& records, int fmt, int64_t block_tokens,
                         int64_t n_kv_heads, const Tensor& block_table, const Tensor& kv_len,
                         const Maybe& q_start, int64_t max_queries, double sm_scale, bool causal,
                         const Maybe& delta_m, double rope_base, int pairs, const Maybe& out_,
                         const Maybe& lse_, const py::object& workspace, const py::object& stream) {
  OneGpu on("attend_records");
  on(q)(records)(block_table)(kv_len)(q_start)(delta_m)(out_)(lse_);
  Maybe ws;
  const bool make = workspace.is(py::bool_(true));
  if (!make && !workspace.is_none()) ws = py::cast<Tensor>(workspace);
  on(ws);
  const auto at_stream = stream_of(stream, on.device());
  const hkv_heads qh = heads_of(q, "q");
  const int64_t n = q.size(0), hq = q.size(1);
  const Table table = table_of(block_table);
  const int64_t R = block_table.size(0);
  need(kv_len.numel() == R && (q_start ? q_start->numel() == R + 1 : n == R),
       "kv_len [n_requests], q_start [n_requests + 1] (or one query per request) and block_table must agree");
  if (max_queries < 0) max_queries = q_start ? (n > 1 ? n : 1) : 1;
  const Tensor out = out_ ? *out_ : made_on(q.sizes(), q.options(), at_stream);
  need(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type(), "out must have q's shape and dtype");
  const Tensor lse = lse_ ? *lse_ : made_on({n, hq}, q.options().dtype(at::kFloat), at_stream);
  need(lse.dim() == 2 && lse.size(0) == n && lse.size(1) == hq && lse.scalar_type() == at::kFloat &&
           lse.is_contiguous(),
       "lse must be a contiguous float32 [n_tokens, n_q_heads] tensor");
  hkv_key_shift shift;
  if (delta_m) {
    need(delta_m->sizes() == block_table.sizes(), "delta_m must have block_table's shape, type and strides");
    const Table d = table_of(*delta_m);
    need(d.stride == table.stride, "delta_m must have block_table's shape, type and strides");
    shift = {d.data, rope_base, pairs};
  }
  const Pool pool = pool_of(records, fmt, block_tokens, n_kv_heads);
  const hkv_requests req = {small(R, "n_requests"), small(table.blocks, "max_blocks"),
                            small(max_queries, "max_queries"), table.data, table.stride,
                            ints(kv_len, "kv_len"), q_start ? ints(*q_start, "q_start") : nullptr};
  const int dtype = dtype_of(q);
  if (make) {
    const int64_t bytes = calls.attend_bytes(&pool.shape, &req, small(n, "n_tokens"), qh.n_heads, dtype);
    if (bytes > 0) ws = made_on({bytes}, q.options().dtype(at::kByte), at_stream);
  }
  if (ws) need(ws->scalar_type() == at::kByte && ws->is_contiguous(), "workspace must be a contiguous uint8 tensor");
  const hkv_heads oh = heads_of(out, "out");
  const int st = launch(calls.attend, &pool.shape, fmt, &pool.records, &req, &qh, dtype,
                        small(n, "n_tokens"), sm_scale, causal ? 1 : 0,
                        delta_m ? &shift : nullptr, &oh, static_cast<float*>(lse.data_ptr()),
                        ws ? ws->data_ptr() : nullptr, ws ? ws->numel() : 0, at_stream.stream());
  return py::make_tuple(st, out, lse);
}

// Pages [L, P, T_b, H, 128]; a 4-D tensor is one layer.
Tensor as_5d(const Tensor& t) {
  if (t.dim() == 4) return t.unsqueeze(0);
  if (t.dim() != 5) refuse("pages must be [L, P, T_b, H, 128] or [P, T_b, H, 128]");
  return t;
}

int fetch(bool per_token, const Tensor& records, int fmt, const Tensor& block_table,
          const Tensor& delta, double rope_base, int pairs, const Tensor& k_pages,
          const Tensor& v_pages, const Maybe& visit_order, const py::object& stream) {
  OneGpu on(per_token ? "fetch_dequant_rope_shift_tokens" : "fetch_dequant_rope_shift");
  on(records)(block_table)(delta)(k_pages)(v_pages)(visit_order);
  const Tensor k = as_5d(k_pages), v = as_5d(v_pages);
  need(k.sizes() == v.sizes() && k.strides() == v.strides() && k.scalar_type() == v.scalar_type(),
       "K and V pages must share shape, strides and dtype");
  need(k.size(4) == HKV_HEAD_DIM && k.stride(4) == 1,
       "the last (head_dim=128) axis of the pages must be contiguous");
  if (dtype_of(k) < 0) refuse("unsupported page dtype " + dtype_name(k));
  const int64_t nb = block_table.numel(), tb = k.size(2);
  need(records.dim() >= 2 && records.size(0) == k.size(0) && records.size(1) == nb &&
           delta.numel() == (per_token ? nb * tb : nb),
       "records [L, n_blocks, bytes], table and deltas must agree");
  need(!visit_order || visit_order->numel() == nb, "visit_order must hold n_blocks entries");
  const hkv_shape shape = {small(k.size(0), "n_layers"), small(nb, "n_blocks"),
                           small(tb, "block_tokens"), small(k.size(3), "n_kv_heads"), HKV_HEAD_DIM};
  const hkv_records rec = records_of(records, fmt, tb, k.size(3));
  const hkv_pages pages = {k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                           k.stride(3), small(k.size(1), "num_pages")};
  const int32_t* order = visit_order ? ints(*visit_order, "visit_order") : nullptr;
  return launch(per_token ? calls.fetch_tokens : calls.fetch, &shape, fmt, &rec,
                ints(block_table, "block_table"), ints(delta, "delta_m"), order, rope_base, pairs,
                &pages, dtype_of(k), stream_of(stream, on.device()).stream());
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("bind", &bind);
  m.def("plan_step", &plan_step);
  m.def("rope_heads", &rope_heads);
  m.def("append_tokens", &append_tokens);
  m.def("attend_records", &attend_records);
  m.def("fetch", &fetch);
}
