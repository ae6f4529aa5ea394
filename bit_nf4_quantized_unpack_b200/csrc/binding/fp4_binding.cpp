// fp4_binding.cpp -- Python calls of the microscaled 4-bit operators: checks, output allocation
// and marshalling to the C ABI, in C++ because at a few tokens the host bounds these calls
// (quantizing 16 x 4096 takes 2 us on the GPU; the same steps in Python took 13 us).
//
// The library's functions are looked up in the libqlora.so that the Python module has loaded.
#include <dlfcn.h>

#include <optional>
#include <string>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include "../../../include/qlora.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

struct Library {
  decltype(&qlora_last_error) last_error;
  decltype(&qlora_fp4_scales_bytes) scales_bytes;
  decltype(&qlora_fp4_quantize) quantize;
  decltype(&qlora_fp4_quantize_weight_workspace_size) weight_workspace;
  decltype(&qlora_fp4_quantize_weight) quantize_weight;
  decltype(&qlora_fp4_dequant) dequant;
  decltype(&qlora_fp4_matmul) matmul;
  decltype(&qlora_fp4_linear_fwd_workspace_size) fwd_workspace;
  decltype(&qlora_fp4_linear_fwd) fwd;
  decltype(&qlora_fp4_linear_bwd_workspace_size) bwd_workspace;
  decltype(&qlora_fp4_linear_bwd) bwd;
} L;

PyObject* g_error = nullptr;  // the Python class QLoraError(status, where, detail)

void open(const std::string& path, py::object error) {
  void* h = dlopen(path.c_str(), RTLD_NOW);
  if (!h) throw std::runtime_error(std::string("cannot load ") + path + ": " + dlerror());
  auto get = [&](auto& fn, const char* name) {
    fn = reinterpret_cast<std::decay_t<decltype(fn)>>(dlsym(h, name));
    if (!fn) throw std::runtime_error(path + " has no " + name);
  };
  get(L.last_error, "qlora_last_error");
  get(L.scales_bytes, "qlora_fp4_scales_bytes");
  get(L.quantize, "qlora_fp4_quantize");
  get(L.weight_workspace, "qlora_fp4_quantize_weight_workspace_size");
  get(L.quantize_weight, "qlora_fp4_quantize_weight");
  get(L.dequant, "qlora_fp4_dequant");
  get(L.matmul, "qlora_fp4_matmul");
  get(L.fwd_workspace, "qlora_fp4_linear_fwd_workspace_size");
  get(L.fwd, "qlora_fp4_linear_fwd");
  get(L.bwd_workspace, "qlora_fp4_linear_bwd_workspace_size");
  get(L.bwd, "qlora_fp4_linear_bwd");
  g_error = error.release().ptr();
}

void check(qlora_status status, const char* where) {
  if (status == QLORA_OK) return;
  const py::object cls = py::reinterpret_borrow<py::object>(g_error);
  const py::object e = cls(static_cast<int>(status), where, L.last_error());
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// The device index of the operand that the others have to share.
c10::DeviceIndex device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw py::value_error(std::string(name) + ": expected a CUDA tensor");
  return t.device().index();
}

// The address of a dense tensor on device `dev` with this dtype and shape.
void* dense(const Tensor& t, const char* name, c10::DeviceIndex dev, at::ScalarType dtype,
            at::IntArrayRef shape) {
  if (t.scalar_type() != dtype)
    throw py::type_error(std::string(name) + ": expected " + c10::toString(dtype) + ", got " +
                         c10::toString(t.scalar_type()));
  if (!t.is_contiguous() || t.sizes() != shape)
    throw py::value_error(std::string(name) + ": expected a contiguous tensor of shape " +
                          shape_text(shape) + ", got " + shape_text(t.sizes()) + " with strides " +
                          shape_text(t.strides()));
  if (!t.is_cuda() || t.device().index() != dev)
    throw py::value_error(std::string(name) + ": on " + t.device().str() + ", expected cuda:" +
                          std::to_string(dev));
  return t.data_ptr();
}

qlora_dtype dtype_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return QLORA_F32;
  if (t.scalar_type() == at::kBFloat16) return QLORA_BF16;
  throw py::type_error(std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()));
}

Tensor make(at::IntArrayRef shape, at::ScalarType dtype, c10::DeviceIndex dev) {
  const at::AutoDispatchBelowADInplaceOrView guard;
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(c10::Device(c10::kCUDA, dev)));
}

// `bytes` of one allocation, handed out as uint8 tensors at multiples of 256 bytes (an
// allocation costs the host a microsecond). All of one type, as tensors of different types on one
// storage cannot be saved together.
struct Bytes {
  Tensor all;
  int64_t off = 0;
  static int64_t room(int64_t n) { return (n + 255) / 256 * 256; }
  Bytes(int64_t bytes, c10::DeviceIndex dev) : all(make({bytes}, at::kByte, dev)) {}
  Tensor take(at::IntArrayRef shape) {
    auto t = c10::make_intrusive<at::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    t->set_storage_offset(off);
    t->set_sizes_contiguous(shape);
    off += room(t->numel());
    return Tensor(std::move(t));
  }
};

// The operands' device made current, and its current stream.
struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(c10::DeviceIndex dev)
      : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev).stream()) {}
};

// A matrix as Python passes it: its buffers hold what the sizes say, so that no kernel reads
// past them.
qlora_fp4_matrix matrix(const Tensor& codes, const Tensor& scales, const OptTensor& gscale,
                        int64_t rows, int64_t cols, int fmt, const char* name, c10::DeviceIndex dev) {
  qlora_fp4_matrix m;
  const std::string n(name);
  if (rows < 0 || cols < 0) throw py::value_error(n + ": negative sizes");
  m.codes = static_cast<uint8_t*>(dense(codes, (n + ".codes").c_str(), dev, at::kByte, {rows, cols / 2}));
  m.scales = static_cast<uint8_t*>(dense(scales, (n + ".scales").c_str(), dev, at::kByte,
                                         {static_cast<int64_t>(L.scales_bytes(rows, cols, fmt))}));
  m.gscale = nullptr;
  m.gscale_rows = 0;
  if (gscale) {
    m.gscale_rows = gscale->numel() == 1 ? 1 : rows;
    m.gscale = static_cast<float*>(dense(*gscale, (n + ".gscale").c_str(), dev, at::kFloat, {m.gscale_rows}));
  }
  m.rows = rows;
  m.cols = cols;
  m.format = fmt;
  return m;
}

struct Workspace {
  Tensor t;
  void* ptr;
  size_t bytes;
  Workspace(const OptTensor& given, size_t need, c10::DeviceIndex dev) {
    t = given ? *given : make({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, dev);
    if (given) dense(t, "workspace", dev, at::kByte, t.sizes());
    ptr = t.data_ptr();
    bytes = static_cast<size_t>(t.numel());
  }
};

Tensor or_make(const OptTensor& given, at::IntArrayRef shape, at::ScalarType dtype, c10::DeviceIndex dev) {
  return given ? *given : make(shape, dtype, dev);
}

void check_2d(const Tensor& t, const char* name) {
  if (t.dim() != 2) throw py::value_error(std::string(name) + " must be 2-D");
}

// (codes, scales, gscale or None) of X [rows, cols]
py::tuple quantize(const Tensor& X, int fmt) {
  const qlora_dtype dt = dtype_of(X, "X");
  const auto dev = device_of(X, "X");
  check_2d(X, "X");
  const int64_t rows = X.size(0), cols = X.size(1);
  const void* x = dense(X, "X", dev, X.scalar_type(), X.sizes());
  const size_t nsc = L.scales_bytes(rows, cols, fmt);
  if (nsc == 0 && rows != 0)  // no such format or shape: the entry point says which
    check(L.quantize(x, dt, rows, cols, fmt, nullptr, nullptr, nullptr, nullptr), "qlora_fp4_quantize");
  const int64_t sc = static_cast<int64_t>(nsc);
  Bytes b(Bytes::room(rows * (cols / 2)) + sc, dev);
  const Tensor codes = b.take({rows, cols / 2}), scales = b.take({sc});
  Tensor g;
  if (fmt == QLORA_FP4_NV) g = make({rows}, at::kFloat, dev);
  const Launch l(dev);
  check(L.quantize(x, dt, rows, cols, fmt, codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(),
                   g.defined() ? g.data_ptr<float>() : nullptr, l.stream),
        "qlora_fp4_quantize");
  return py::make_tuple(codes, scales, g.defined() ? py::cast(g) : py::none());
}

void quantize_out(const Tensor& X, int fmt, const Tensor& codes, const Tensor& scales,
                  const OptTensor& gscale) {
  const qlora_dtype dt = dtype_of(X, "X");
  const auto dev = device_of(X, "X");
  check_2d(X, "X");
  const int64_t rows = X.size(0), cols = X.size(1);
  const void* x = dense(X, "X", dev, X.scalar_type(), X.sizes());
  const qlora_fp4_matrix m = matrix(codes, scales, gscale, rows, cols, fmt, "out", dev);
  if (fmt == QLORA_FP4_NV && (!m.gscale || m.gscale_rows != rows))
    throw py::value_error("out.gscale: expected one value per row");
  const Launch l(dev);
  check(L.quantize(x, dt, rows, cols, fmt, const_cast<uint8_t*>(m.codes), const_cast<uint8_t*>(m.scales),
                   const_cast<float*>(m.gscale), l.stream),
        "qlora_fp4_quantize");
}

void weight_out(const Tensor& W, int fmt, const Tensor& codes, const Tensor& scales,
                const OptTensor& gscale, const OptTensor& t_codes, const OptTensor& t_scales,
                const OptTensor& workspace) {
  const qlora_dtype dt = dtype_of(W, "W");
  const auto dev = device_of(W, "W");
  check_2d(W, "W");
  const int64_t n = W.size(0), k = W.size(1);
  const void* src = dense(W, "W", dev, W.scalar_type(), W.sizes());
  const qlora_fp4_matrix m = matrix(codes, scales, gscale, n, k, fmt, "out.w", dev);
  if (fmt == QLORA_FP4_NV && (!m.gscale || m.gscale_rows != 1))
    throw py::value_error("out.w.gscale: expected one value");
  qlora_fp4_matrix t = {};
  if (t_codes && t_scales) t = matrix(*t_codes, *t_scales, std::nullopt, k, n, fmt, "out.wt", dev);
  const Launch l(dev);
  const Workspace ws(workspace, L.weight_workspace(), dev);
  check(L.quantize_weight(src, dt, n, k, fmt, const_cast<uint8_t*>(m.codes), const_cast<uint8_t*>(m.scales),
                          const_cast<float*>(m.gscale), const_cast<uint8_t*>(t.codes),
                          const_cast<uint8_t*>(t.scales), ws.ptr, ws.bytes, l.stream),
        "qlora_fp4_quantize_weight");
}

// (codes, scales, gscale or None, t_codes or None, t_scales or None) of W [n, k]
py::tuple weight(const Tensor& W, int fmt, bool transposed, const OptTensor& workspace) {
  const qlora_dtype dt = dtype_of(W, "W");
  const auto dev = device_of(W, "W");
  check_2d(W, "W");
  const int64_t n = W.size(0), k = W.size(1);
  const size_t nsc = L.scales_bytes(n, k, fmt), tsc = L.scales_bytes(k, n, fmt);
  if (nsc == 0 || (transposed && tsc == 0)) {  // no such format or shape: the entry point says which
    check(L.quantize_weight(nullptr, dt, n, k, fmt, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
          "qlora_fp4_quantize_weight");
  }
  const int64_t sc = static_cast<int64_t>(nsc), st = static_cast<int64_t>(tsc);
  const int64_t wsb = workspace ? 0 : static_cast<int64_t>(L.weight_workspace());
  Bytes b(Bytes::room(n * (k / 2)) + Bytes::room(sc) + wsb, dev);
  const Tensor codes = b.take({n, k / 2}), scales = b.take({sc});
  OptTensor g, tc, ts, ws = workspace;
  if (!ws) ws = b.take({wsb});
  if (fmt == QLORA_FP4_NV) g = make({1}, at::kFloat, dev);
  if (transposed) {  // an allocation of its own: it may be dropped by itself
    Bytes t(Bytes::room(k * (n / 2)) + st, dev);
    tc = t.take({k, n / 2});
    ts = t.take({st});
  }
  weight_out(W, fmt, codes, scales, g, tc, ts, ws);
  return py::make_tuple(codes, scales, g, tc, ts);
}

Tensor dequant(const Tensor& codes, const Tensor& scales, const OptTensor& gscale, int64_t rows,
               int64_t cols, int fmt, bool bf16, const OptTensor& out) {
  const auto dev = device_of(codes, "q.codes");
  const qlora_fp4_matrix m = matrix(codes, scales, gscale, rows, cols, fmt, "q", dev);
  Tensor o = or_make(out, {rows, cols}, bf16 ? at::kBFloat16 : at::kFloat, dev);
  const qlora_dtype dt = dtype_of(o, "out");
  void* p = dense(o, "out", dev, o.scalar_type(), {rows, cols});
  const Launch l(dev);
  check(L.dequant(m, dt, p, l.stream), "qlora_fp4_dequant");
  return o;
}

Tensor matmul(const Tensor& ac, const Tensor& as, const OptTensor& ag, int64_t ar, int64_t acols, int af,
              const Tensor& bc, const Tensor& bs, const OptTensor& bg, int64_t br, int64_t bcols, int bf,
              bool bf16, const OptTensor& out) {
  const auto dev = device_of(ac, "a.codes");
  const qlora_fp4_matrix a = matrix(ac, as, ag, ar, acols, af, "a", dev);
  const qlora_fp4_matrix b = matrix(bc, bs, bg, br, bcols, bf, "b", dev);
  Tensor o = or_make(out, {ar, br}, bf16 ? at::kBFloat16 : at::kFloat, dev);
  const qlora_dtype dt = dtype_of(o, "out");
  void* p = dense(o, "out", dev, o.scalar_type(), {ar, br});
  const Launch l(dev);
  check(L.matmul(a, b, dt, p, l.stream), "qlora_fp4_matmul");
  return o;
}

const uint16_t* bf16_in(const Tensor& t, const char* name, c10::DeviceIndex dev, at::IntArrayRef shape) {
  return static_cast<const uint16_t*>(dense(t, name, dev, at::kBFloat16, shape));
}

// (Y, T or None)
py::tuple linear_fwd(const Tensor& X, const Tensor& wc, const Tensor& ws_, const OptTensor& wg, int64_t n,
                     int64_t k, int fmt, const Tensor& A, const Tensor& B, double scale, bool save_T,
                     const OptTensor& Y_, const OptTensor& T_, const OptTensor& workspace) {
  const auto dev = device_of(X, "X");
  check_2d(X, "X");
  check_2d(A, "A");
  const qlora_fp4_matrix w = matrix(wc, ws_, wg, n, k, fmt, "w", dev);
  const int64_t M = X.size(0), r = A.size(1);
  const uint16_t *x = bf16_in(X, "X", dev, {M, k}), *a = bf16_in(A, "A", dev, {k, r}),
                 *b = bf16_in(B, "B", dev, {r, n});
  Tensor Y = or_make(Y_, {M, n}, at::kBFloat16, dev), T;
  auto* y = static_cast<uint16_t*>(dense(Y, "Y", dev, at::kBFloat16, {M, n}));
  float* t = nullptr;
  if (save_T) {
    T = or_make(T_, {M, r}, at::kFloat, dev);
    t = static_cast<float*>(dense(T, "T", dev, at::kFloat, {M, r}));
  }
  const int ri = static_cast<int>(r > 1 << 20 ? 1 << 20 : r);
  const Launch l(dev);  // before the query: the rank-r products' splits go by the device's SMs
  const Workspace ws(workspace, L.fwd_workspace(M, n, k, ri, fmt), dev);
  check(L.fwd(x, M, w, a, b, ri, static_cast<float>(scale), y, t, ws.ptr, ws.bytes, l.stream),
        "qlora_fp4_linear_fwd");
  return py::make_tuple(Y, save_T ? py::cast(T) : py::none());
}

// (dX or None, dA, dB)
py::tuple linear_bwd(const Tensor& dY, const Tensor& X, const OptTensor& T, const Tensor& wc,
                     const Tensor& ws_, const OptTensor& wg, int64_t k, int64_t n, int fmt, const Tensor& A,
                     const Tensor& B, double scale, bool need_dX, const OptTensor& dX_,
                     const OptTensor& dA_, const OptTensor& dB_, const OptTensor& workspace) {
  const auto dev = device_of(X, "X");
  check_2d(X, "X");
  check_2d(A, "A");
  const qlora_fp4_matrix wt = matrix(wc, ws_, wg, k, n, fmt, "w.wt", dev);
  const int64_t M = X.size(0), r = A.size(1);
  const uint16_t *dy = bf16_in(dY, "dY", dev, {M, n}), *x = bf16_in(X, "X", dev, {M, k}),
                 *a = bf16_in(A, "A", dev, {k, r}), *b = bf16_in(B, "B", dev, {r, n});
  const float* t = T ? static_cast<const float*>(dense(*T, "T", dev, at::kFloat, {M, r})) : nullptr;
  Tensor dX;
  uint16_t* dx = nullptr;
  if (need_dX) {
    dX = or_make(dX_, {M, k}, at::kBFloat16, dev);
    dx = static_cast<uint16_t*>(dense(dX, "dX", dev, at::kBFloat16, {M, k}));
  }
  Tensor dA = or_make(dA_, {k, r}, at::kFloat, dev), dB = or_make(dB_, {r, n}, at::kFloat, dev);
  auto* da = static_cast<float*>(dense(dA, "dA", dev, at::kFloat, {k, r}));
  auto* db = static_cast<float*>(dense(dB, "dB", dev, at::kFloat, {r, n}));
  const int ri = static_cast<int>(r > 1 << 20 ? 1 << 20 : r);
  const Launch l(dev);
  const Workspace ws(workspace, L.bwd_workspace(M, n, k, ri, fmt), dev);
  check(L.bwd(dy, x, t, M, wt, a, b, ri, static_cast<float>(scale), dx, da, db, ws.ptr, ws.bytes, l.stream),
        "qlora_fp4_linear_bwd");
  return py::make_tuple(need_dX ? py::cast(dX) : py::none(), dA, dB);
}

}  // namespace

PYBIND11_MODULE(qlora_binding, m) {
  m.attr("torch_version") = QLORA_TORCH_VERSION;  // tensors of another torch may be laid out otherwise
  m.def("open", &open);
  m.def("quantize", &quantize);
  m.def("quantize_out", &quantize_out);
  m.def("weight", &weight);
  m.def("weight_out", &weight_out);
  m.def("dequant", &dequant);
  m.def("matmul", &matmul);
  m.def("linear_fwd", &linear_fwd);
  m.def("linear_bwd", &linear_bwd);
}
