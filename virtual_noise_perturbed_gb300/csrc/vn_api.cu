// vn_api.cu -- the C ABI declared in include/vn.h: host-side validation,
// path selection and launch. Every argument is checked here, before anything
// touches the device; a failing check returns its status and launches nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <memory>
#include <mutex>
#include <new>

#include "vn.h"
#include "vn_internal.h"

namespace vn {

cudaError_t device_info(DeviceInfo* info) {
  static DeviceInfo cache[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  DeviceInfo& c = cache[dev];
  if (c.device != dev) {
    DeviceInfo d;
    d.device = dev;
    if ((err = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess)
      return err;
    c = d;
  }
  *info = c;
  return cudaSuccess;
}

}  // namespace vn

namespace {

thread_local char g_last_error[256] = "";

vn_status cuda_failure(cudaError_t err) {
  std::snprintf(g_last_error, sizeof(g_last_error), "%s: %s", cudaGetErrorName(err),
                cudaGetErrorString(err));
  return VN_ERR_CUDA;
}

vn_status launched(cudaError_t err) { return err == cudaSuccess ? VN_OK : cuda_failure(err); }

bool dtype_ok(vn_dtype d) { return d == VN_F32 || d == VN_BF16; }
size_t dtype_size(vn_dtype d) { return d == VN_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// r = a * b, false when it does not fit in int64 (inputs are >= 0).
bool mul(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

// The byte ranges [p, p + pb) and [q, q + qb) share a byte (an empty range shares none).
bool overlap(const void* p, int64_t pb, const void* q, int64_t qb) {
  if (p == nullptr || q == nullptr || pb <= 0 || qb <= 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + static_cast<uintptr_t>(qb) && b < a + static_cast<uintptr_t>(pb);
}

bool float_sigma(double sigma, float* out) {
  if (!std::isfinite(sigma)) return false;
  const float f = static_cast<float>(sigma);
  if (!std::isfinite(f)) return false;
  *out = f;
  return true;
}

bool device_is_cc10(const vn::DeviceInfo& d) { return d.cc_major == 10; }

// VN_PATH_AUTO takes the tensor-core path from this per-individual batch on:
// below it the MMA's N of 16 would be mostly padding.
constexpr int64_t kAutoTcMinBatch = 16;

// The checks of a perturbed linear call (vn_perturbed_linear_kind and the test
// hook share them): dtypes, enums, sizes, sigma, size products, nulls,
// alignment and overlaps, in that order. On VN_OK, *empty tells whether the
// output has no elements (nothing to launch) and *a holds the arguments.
vn_status check_linear(const void* x, vn_dtype x_dt, int x_shared, const void* w, vn_dtype w_dt,
                       const void* b, vn_dtype b_dt, const int64_t* seeds, int64_t pop,
                       int64_t batch, int64_t in, int64_t out, double sigma, uint64_t offset,
                       void* y, vn_dtype y_dt, vn_act act, vn_noise kind, vn::LinearArgs* a,
                       bool* empty) {
  if (kind != VN_NOISE_UNIFORM && kind != VN_NOISE_GAUSSIAN) return VN_ERR_VALUE;
  if (!dtype_ok(x_dt) || !dtype_ok(w_dt) || (b != nullptr && !dtype_ok(b_dt)) || !dtype_ok(y_dt))
    return VN_ERR_DTYPE;
  const vn_dtype want_y = (x_dt == VN_BF16 && w_dt == VN_BF16) ? VN_BF16 : VN_F32;
  if (y_dt != want_y) return VN_ERR_DTYPE;
  if (act != VN_ACT_NONE && act != VN_ACT_TANH) return VN_ERR_VALUE;
  if (pop < 0 || batch < 0 || in < 0 || out < 0) return VN_ERR_SHAPE;
  float sig;
  if (!float_sigma(sigma, &sig)) return VN_ERR_VALUE;
  int64_t x_elems, y_elems, w_elems, t;
  if (!mul(batch, in, &x_elems) || (!x_shared && !mul(x_elems, pop, &x_elems)) ||
      !mul(pop, batch, &t) || !mul(t, out, &y_elems) || !mul(out, in, &w_elems))
    return VN_ERR_OVERFLOW;
  *empty = y_elems == 0;
  if (*empty) return VN_OK;
  if (seeds == nullptr || y == nullptr || (x_elems > 0 && x == nullptr) ||
      (w_elems > 0 && w == nullptr))
    return VN_ERR_NULL;
  if (!aligned(seeds, 8) || !aligned(y, dtype_size(y_dt)) || !aligned(x, dtype_size(x_dt)) ||
      !aligned(w, dtype_size(w_dt)) || (b != nullptr && !aligned(b, dtype_size(b_dt))))
    return VN_ERR_ALIGN;
  int64_t yb, xb, wb, bb, sb;
  if (!mul(y_elems, dtype_size(y_dt), &yb) || !mul(x_elems, dtype_size(x_dt), &xb) ||
      !mul(w_elems, dtype_size(w_dt), &wb) || !mul(out, dtype_size(b_dt), &bb) ||
      !mul(pop, 8, &sb))
    return VN_ERR_OVERFLOW;
  if (overlap(y, yb, x, xb) || overlap(y, yb, w, wb) || overlap(y, yb, b, bb) ||
      overlap(y, yb, seeds, sb))
    return VN_ERR_VALUE;
  a->x = x; a->x_dt = x_dt; a->x_shared = x_shared ? 1 : 0;
  a->w = w; a->w_dt = w_dt; a->b = b; a->b_dt = b_dt;
  a->seeds = seeds; a->pop = pop; a->batch = batch; a->in = in; a->out = out;
  a->sigma = sig; a->offset = offset; a->y = y; a->y_dt = y_dt; a->act = act; a->kind = kind;
  return VN_OK;
}

// The activations of the centre network's linear layer.
bool linear_act_ok(vn_act act) { return act >= VN_ACT_NONE && act <= VN_ACT_SILU; }

// rows x n elements of dt in bytes; false when the product does not fit in int64.
bool bytes_of(int64_t rows, int64_t n, vn_dtype dt, int64_t* bytes) {
  return mul(rows, n, bytes) && mul(*bytes, static_cast<int64_t>(dtype_size(dt)), bytes);
}

// A range of device memory that a call reads or writes.
struct Range {
  const void* p;
  int64_t bytes;
};
// No output shares a byte with an input or with another output.
template <int kOut, int kIn>
bool disjoint(const Range (&outs)[kOut], const Range (&ins)[kIn]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < kIn; ++j)
      if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return false;
    for (int j = i + 1; j < kOut; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return false;
  }
  return true;
}

// The sizes of a linear layer: every matrix fits in 2^60 bytes, so that the workspace
// sums of a few such matrices do not overflow.
vn_status check_sizes(int64_t rows, int64_t in, int64_t out, vn_dtype dt) {
  if (!dtype_ok(dt)) return VN_ERR_DTYPE;
  if (rows < 0 || in < 0 || out < 0) return VN_ERR_SHAPE;
  const int64_t most = int64_t{1} << 57;
  int64_t t;
  if (rows > most || in > most || out > most || !mul(rows, in, &t) || t > most || !mul(rows, out, &t) ||
      t > most || !mul(out, in, &t) || t > most)
    return VN_ERR_OVERFLOW;
  return VN_OK;
}

// Few rows take any number of features; other kernels' coordinates have 32 bits.
bool features_ok(int64_t rows, int64_t in, int64_t out) {
  return rows <= 8 || (in <= vn::kDenseMost && out <= vn::kDenseMost);
}

// The memory of a call over many tensors: whether anything that is written shares a byte with anything else.
struct Span {
  uintptr_t start, end;
  bool written;
};
class Spans {
 public:
  explicit Spans(int64_t most) : s_(new (std::nothrow) Span[static_cast<size_t>(most)]) {}
  bool ok() const { return s_ != nullptr; }
  void add(const void* p, int64_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (p != nullptr && bytes > 0) s_[count_++] = {a, a + static_cast<uintptr_t>(bytes), written};
  }
  bool clash() {
    std::sort(s_.get(), s_.get() + count_, [](const Span& a, const Span& b) { return a.start < b.start; });
    uintptr_t any = 0, written = 0;  // ends of those so far
    for (int64_t i = 0; i < count_; ++i) {
      const Span& s = s_[i];
      if (s.start < (s.written ? any : written)) return true;
      any = std::max(any, s.end);
      if (s.written) written = std::max(written, s.end);
    }
    return false;
  }

 private:
  std::unique_ptr<Span[]> s_;
  int64_t count_ = 0;
};
class Pieces {
 public:
  explicit Pieces(int64_t count) : p_(new (std::nothrow) vn_gradient[static_cast<size_t>(count)]) {}
  bool ok() const { return p_ != nullptr; }
  vn_gradient& operator[](int64_t i) { return p_[i]; }
  const vn_gradient* get() const { return p_.get(); }

 private:
  std::unique_ptr<vn_gradient[]> p_;
};

constexpr int64_t kMostFeatures = int64_t{1} << 40;  // of packed weights
constexpr int64_t kMostTensors = int64_t{1} << 32;

vn_status check_norm(int64_t n_tensors, double max_norm, const float* norm, const void* workspace, int64_t workspace_bytes) {
  if (!(max_norm >= 0.0)) return VN_ERR_VALUE;
  if (n_tensors > kMostTensors) return VN_ERR_OVERFLOW;
  if (norm == nullptr) return VN_ERR_NULL;
  if (!aligned(norm, 4) || !aligned(workspace, 256)) return VN_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < vn::clip_workspace(n_tensors)) return VN_ERR_WORKSPACE;
  return VN_OK;
}

vn_status clip(const vn_gradient* tensors, int64_t n_tensors, vn_dtype dt, double max_norm, float* norm, void* workspace,
               int64_t workspace_bytes, bool scale, void* stream) {
  if (!dtype_ok(dt)) return VN_ERR_DTYPE;
  if (n_tensors < 0) return VN_ERR_SHAPE;
  const vn_status st = check_norm(n_tensors, max_norm, norm, workspace, workspace_bytes);
  if (st != VN_OK) return st;
  if (n_tensors > 0 && tensors == nullptr) return VN_ERR_NULL;
  Spans spans(2 * n_tensors + 2);
  if (!spans.ok()) return VN_ERR_OVERFLOW;
  spans.add(norm, 4, true);
  spans.add(workspace, vn::clip_workspace(n_tensors), true);
  const int64_t size = static_cast<int64_t>(dtype_size(dt));
  for (int64_t i = 0; i < n_tensors; ++i) {
    const vn_gradient& t = tensors[i];
    if (t.n < 0) return VN_ERR_SHAPE;
    if (t.n > (int64_t{1} << 59)) return VN_ERR_OVERFLOW;
    if (t.n == 0) continue;
    if (t.grad == nullptr || (scale && t.out == nullptr)) return VN_ERR_NULL;
    if (!aligned(t.grad, size) || (scale && !aligned(t.out, size))) return VN_ERR_ALIGN;
    if (scale) spans.add(t.out, t.n * size, true);
    if (!scale || t.out != t.grad) spans.add(t.grad, t.n * size, false);
  }
  if (spans.clash()) return VN_ERR_VALUE;
  vn::ClipArgs c = {tensors, n_tensors, dt, max_norm, norm, scale, workspace};
  return launched(vn::launch_clip(c, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

const char* vn_status_string(vn_status s) {
  switch (s) {
    case VN_OK: return "VN_OK";
    case VN_ERR_NULL: return "VN_ERR_NULL: a required pointer is NULL";
    case VN_ERR_SHAPE: return "VN_ERR_SHAPE: invalid size";
    case VN_ERR_DTYPE: return "VN_ERR_DTYPE: unsupported dtype or dtype combination";
    case VN_ERR_VALUE: return "VN_ERR_VALUE: invalid value (sigma, enum)";
    case VN_ERR_ALIGN: return "VN_ERR_ALIGN: pointer not aligned to its element size";
    case VN_ERR_OVERFLOW: return "VN_ERR_OVERFLOW: size product does not fit in int64";
    case VN_ERR_TIMEOUT: return "VN_ERR_TIMEOUT: a device-side bounded wait ran out";
    case VN_ERR_CUDA: return "VN_ERR_CUDA: a CUDA runtime call failed";
    case VN_ERR_DEVICE: return "VN_ERR_DEVICE: this path needs a compute capability 10.x GPU";
    case VN_ERR_PATH: return "VN_ERR_PATH: the forced path cannot run these arguments";
    case VN_ERR_WORKSPACE: return "VN_ERR_WORKSPACE: the workspace is too small";
  }
  return "unknown vn_status";
}

const char* vn_last_error_message(void) { return g_last_error; }

int vn_version(void) { return (1 << 16) | 0; }

vn_status vn_noise_dump(const int64_t* seeds, int64_t pop, int64_t n, uint64_t offset,
                        float* out, void* stream) {
  return vn_noise_dump_ex(seeds, pop, n, offset, VN_NOISE_UNIFORM, out, stream);
}

vn_status vn_noise_dump_ex(const int64_t* seeds, int64_t pop, int64_t n, uint64_t offset,
                           vn_noise kind, float* out, void* stream) {
  if (kind != VN_NOISE_UNIFORM && kind != VN_NOISE_GAUSSIAN) return VN_ERR_VALUE;
  if (pop < 0 || n < 0) return VN_ERR_SHAPE;
  int64_t total;
  if (!mul(pop, n, &total)) return VN_ERR_OVERFLOW;
  if (total == 0) return VN_OK;
  if (seeds == nullptr || out == nullptr) return VN_ERR_NULL;
  if (!aligned(seeds, 8) || !aligned(out, 4)) return VN_ERR_ALIGN;
  int64_t out_bytes, seed_bytes;
  if (!mul(total, 4, &out_bytes) || !mul(pop, 8, &seed_bytes)) return VN_ERR_OVERFLOW;
  if (overlap(out, out_bytes, seeds, seed_bytes)) return VN_ERR_VALUE;
  return launched(vn::launch_noise_dump(seeds, pop, n, offset, kind, out,
                                        static_cast<cudaStream_t>(stream)));
}

static vn_status gradient(const float* fitness, const int64_t* seeds, int64_t pop, int64_t m_rows,
                          int64_t m_cols, double sigma, uint64_t offset, vn_noise kind,
                          float* grad, void* stream, float* theta = nullptr, double lr = 0.0) {
  if (kind != VN_NOISE_UNIFORM && kind != VN_NOISE_GAUSSIAN) return VN_ERR_VALUE;
  if (pop < 1 || m_rows < 0 || m_cols < 0) return VN_ERR_SHAPE;
  int64_t m;
  if (!mul(m_rows, m_cols, &m)) return VN_ERR_OVERFLOW;
  float sig;
  if (!float_sigma(sigma, &sig) || sig == 0.f) return VN_ERR_VALUE;
  const double inv = 1.0 / (static_cast<double>(pop) * sigma);
  const float scale = static_cast<float>(inv);
  if (!std::isfinite(scale) || scale == 0.f) return VN_ERR_VALUE;
  float lr_f = 0.f;
  if (theta != nullptr && !float_sigma(lr, &lr_f)) return VN_ERR_VALUE;
  if (m == 0) return VN_OK;
  if (fitness == nullptr || seeds == nullptr || grad == nullptr) return VN_ERR_NULL;
  if (!aligned(fitness, 4) || !aligned(seeds, 8) || !aligned(grad, 4)) return VN_ERR_ALIGN;
  if (theta != nullptr && !aligned(theta, 4)) return VN_ERR_ALIGN;
  int64_t m_bytes, seed_bytes;
  if (!mul(m, 4, &m_bytes) || !mul(pop, 8, &seed_bytes)) return VN_ERR_OVERFLOW;
  const int64_t fit_bytes = pop * 4;
  // The outputs (grad, and theta when given) may not share memory with an input or each other.
  if (overlap(grad, m_bytes, fitness, fit_bytes) || overlap(grad, m_bytes, seeds, seed_bytes))
    return VN_ERR_VALUE;
  if (theta != nullptr &&
      (overlap(theta, m_bytes, grad, m_bytes) || overlap(theta, m_bytes, fitness, fit_bytes) ||
       overlap(theta, m_bytes, seeds, seed_bytes)))
    return VN_ERR_VALUE;
  return launched(vn::launch_grad(fitness, seeds, pop, m, offset, scale, kind, grad,
                                  static_cast<cudaStream_t>(stream), theta, lr_f));
}

vn_status vn_weight_gradient(const float* fitness, const int64_t* seeds, int64_t pop,
                             int64_t out, int64_t in, double sigma, uint64_t offset,
                             float* grad_w, void* stream) {
  return gradient(fitness, seeds, pop, out, in, sigma, offset, VN_NOISE_UNIFORM, grad_w, stream);
}

vn_status vn_bias_gradient(const float* fitness, const int64_t* seeds, int64_t pop,
                           int64_t out, double sigma, uint64_t offset, float* grad_b,
                           void* stream) {
  return gradient(fitness, seeds, pop, out, 1, sigma, offset, VN_NOISE_UNIFORM, grad_b, stream);
}

vn_status vn_gradient_ex(const float* fitness, const int64_t* seeds, int64_t pop, int64_t n,
                         double sigma, uint64_t offset, vn_noise kind, float* grad, void* stream) {
  return gradient(fitness, seeds, pop, n, 1, sigma, offset, kind, grad, stream);
}

vn_status vn_gradient_update(const float* fitness, const int64_t* seeds, int64_t pop, int64_t n,
                             double sigma, uint64_t offset, vn_noise kind, double lr, float* grad,
                             float* theta, void* stream) {
  if (n > 0 && theta == nullptr) return VN_ERR_NULL;
  if (theta == nullptr) {  // n == 0: validate as the plain estimate does, launch nothing
    float lr_f;
    if (!float_sigma(lr, &lr_f)) return VN_ERR_VALUE;
    return gradient(fitness, seeds, pop, n, 1, sigma, offset, kind, grad, stream);
  }
  return gradient(fitness, seeds, pop, n, 1, sigma, offset, kind, grad, stream, theta, lr);
}

vn_status vn_reduce_metric(const float* center, const int64_t* seeds, int64_t pop,
                           int64_t n_params, double sigma, uint64_t offset, float* fitness,
                           void* stream) {
  if (pop < 0 || n_params < 1) return VN_ERR_SHAPE;
  float sig;
  if (!float_sigma(sigma, &sig)) return VN_ERR_VALUE;
  int64_t total;
  if (!mul(pop, n_params, &total)) return VN_ERR_OVERFLOW;
  if (pop == 0) return VN_OK;
  if (center == nullptr || seeds == nullptr || fitness == nullptr) return VN_ERR_NULL;
  if (!aligned(center, 4) || !aligned(seeds, 8) || !aligned(fitness, 4)) return VN_ERR_ALIGN;
  int64_t center_bytes, seed_bytes;
  if (!mul(n_params, 4, &center_bytes) || !mul(pop, 8, &seed_bytes)) return VN_ERR_OVERFLOW;
  const int64_t fit_bytes = pop * 4;  // fits: pop * 8 does
  if (overlap(fitness, fit_bytes, center, center_bytes) || overlap(fitness, fit_bytes, seeds, seed_bytes))
    return VN_ERR_VALUE;
  const float inv_n = static_cast<float>(1.0 / static_cast<double>(n_params));
  return launched(vn::launch_reduce_metric(center, seeds, pop, n_params, sig, inv_n, offset,
                                           fitness, static_cast<cudaStream_t>(stream)));
}

vn_path vn_perturbed_linear_path(const void* x, vn_dtype x_dt, int x_shared, const void* w,
                                 vn_dtype w_dt, int64_t batch, int64_t in, int64_t out) {
  (void)x_shared;
  vn::DeviceInfo dev;
  if (vn::device_info(&dev) != cudaSuccess || !device_is_cc10(dev)) return VN_PATH_FFMA;
  return (batch >= kAutoTcMinBatch && vn::linear_tc_applies(x, x_dt, w, w_dt, batch, in, out))
             ? VN_PATH_TC
             : VN_PATH_FFMA;
}

vn_status vn_perturbed_linear_ex(const void* x, vn_dtype x_dt, int x_shared, const void* w,
                                 vn_dtype w_dt, const void* b, vn_dtype b_dt,
                                 const int64_t* seeds, int64_t pop, int64_t batch, int64_t in,
                                 int64_t out, double sigma, uint64_t offset, void* y,
                                 vn_dtype y_dt, vn_path path, vn_act act, void* stream) {
  return vn_perturbed_linear_kind(x, x_dt, x_shared, w, w_dt, b, b_dt, seeds, pop, batch, in, out,
                                  sigma, offset, y, y_dt, path, act, VN_NOISE_UNIFORM, stream);
}

vn_status vn_perturbed_linear_kind(const void* x, vn_dtype x_dt, int x_shared, const void* w,
                                   vn_dtype w_dt, const void* b, vn_dtype b_dt,
                                   const int64_t* seeds, int64_t pop, int64_t batch, int64_t in,
                                   int64_t out, double sigma, uint64_t offset, void* y,
                                   vn_dtype y_dt, vn_path path, vn_act act, vn_noise kind,
                                   void* stream) {
  if (path != VN_PATH_AUTO && path != VN_PATH_FFMA && path != VN_PATH_TC) return VN_ERR_PATH;
  vn::LinearArgs a;
  bool empty = false;
  const vn_status st = check_linear(x, x_dt, x_shared, w, w_dt, b, b_dt, seeds, pop, batch, in,
                                    out, sigma, offset, y, y_dt, act, kind, &a, &empty);
  if (st != VN_OK || empty) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool gaussian = kind == VN_NOISE_GAUSSIAN;

  if (path == VN_PATH_FFMA && !gaussian) return launched(vn::launch_linear_ffma(a, s));
  vn::DeviceInfo dev;
  cudaError_t err = vn::device_info(&dev);
  if (err != cudaSuccess) return cuda_failure(err);
  const bool tc_ok = vn::linear_tc_applies(x, x_dt, w, w_dt, batch, in, out);
  if (path == VN_PATH_TC) {
    if (!device_is_cc10(dev)) return VN_ERR_DEVICE;
    if (!tc_ok) return VN_ERR_PATH;
    return launched(vn::launch_linear_tc(a, s));
  }
  if (path == VN_PATH_AUTO && tc_ok && batch >= kAutoTcMinBatch && device_is_cc10(dev))
    return launched(vn::launch_linear_tc(a, s));
  // fp32 W (and bias), a policy-sized batch and enough individuals to give every
  // SM a group of them: the one-launch chain kernel with one layer (its
  // individuals share each loaded W chunk, which the single-layer CUDA-core
  // kernel does not), when the layer fits its shared memory. It is also the
  // CUDA-core kernel of the Gaussian kind, for any population.
  if (w_dt == VN_F32 && (b == nullptr || b_dt == VN_F32) && batch >= 1 &&
      batch <= vn::kMlpMaxBatch && (pop >= dev.sm_count || gaussian) && in < (int64_t{1} << 31) &&
      out < (int64_t{1} << 31)) {
    const int64_t dims[2] = {in, out};
    const size_t buf = vn::mlp_buffer_floats(1, dims);
    if (vn::mlp_bytes_per_individual(batch, buf) <= static_cast<size_t>(dev.smem_optin)) {
      const float* wl[1] = {static_cast<const float*>(w)};
      const float* bl[1] = {static_cast<const float*>(b)};
      const uint64_t offs[1] = {offset};
      vn::MlpArgs m;
      m.x = x; m.x_dt = x_dt; m.x_shared = x_shared ? 1 : 0;
      m.n_layers = 1;
      m.dims = dims; m.w = wl; m.b = bl; m.offsets = offs;
      m.seeds = seeds; m.pop = pop; m.batch = batch; m.sigma = a.sigma; m.act = VN_ACT_NONE;
      m.y = static_cast<float*>(y);
      m.act_last = act;
      m.kind = kind;
      return launched(vn::launch_mlp(m, s));
    }
  }
  // The single-layer CUDA-core kernel has the uniform kind only.
  if (gaussian) return VN_ERR_PATH;
  return launched(vn::launch_linear_ffma(a, s));
}

vn_status vn_perturbed_linear(const void* x, vn_dtype x_dt, int x_shared, const void* w,
                              vn_dtype w_dt, const void* b, vn_dtype b_dt, const int64_t* seeds,
                              int64_t pop, int64_t batch, int64_t in, int64_t out, double sigma,
                              uint64_t offset, void* y, vn_dtype y_dt, void* stream) {
  return vn_perturbed_linear_ex(x, x_dt, x_shared, w, w_dt, b, b_dt, seeds, pop, batch, in, out,
                                sigma, offset, y, y_dt, VN_PATH_AUTO, VN_ACT_NONE, stream);
}

vn_status vn_testhook_linear_tc_withhold(const void* x, vn_dtype x_dt, int x_shared, const void* w,
                                         vn_dtype w_dt, const void* b, vn_dtype b_dt,
                                         const int64_t* seeds, int64_t pop, int64_t batch,
                                         int64_t in, int64_t out, double sigma, uint64_t offset,
                                         void* y, vn_dtype y_dt, int64_t withhold_stage,
                                         double timeout_ms, void* stream) {
  if (!(timeout_ms > 0.0) || !(timeout_ms <= 60000.0) || withhold_stage < 0) return VN_ERR_VALUE;
  if (w_dt != VN_BF16 || y_dt != VN_BF16) return VN_ERR_DTYPE;  // the hook's one instance
  // The same checks as a forced tensor-core call, with the real population.
  vn::LinearArgs a;
  bool empty = false;
  const vn_status st = check_linear(x, x_dt, x_shared, w, w_dt, b, b_dt, seeds, pop, batch, in,
                                    out, sigma, offset, y, y_dt, VN_ACT_NONE, VN_NOISE_UNIFORM,
                                    &a, &empty);
  if (st != VN_OK) return st;
  if (empty) return VN_ERR_SHAPE;  // the hook needs a kernel to withhold an arrive in
  vn::DeviceInfo dev;
  cudaError_t err = vn::device_info(&dev);
  if (err != cudaSuccess) return cuda_failure(err);
  if (!device_is_cc10(dev)) return VN_ERR_DEVICE;
  if (!vn::linear_tc_applies(x, x_dt, w, w_dt, batch, in, out) || pop > (int64_t{1} << 31) - 1)
    return VN_ERR_PATH;
  return launched(vn::launch_linear_tc_hook(a, static_cast<cudaStream_t>(stream), withhold_stage,
                                            static_cast<unsigned long long>(timeout_ms * 1e6)));
}

vn_status vn_perturbed_mlp(const void* x, vn_dtype x_dt, int x_shared, int64_t n_layers,
                           const int64_t* dims, const float* const* w, const float* const* b,
                           const uint64_t* offsets, const int64_t* seeds, int64_t pop,
                           int64_t batch, double sigma, vn_act act, float* y, void* stream) {
  return vn_perturbed_mlp_ex(x, x_dt, x_shared, n_layers, dims, w, b, offsets, seeds, pop, batch,
                             sigma, act, VN_NOISE_UNIFORM, y, stream);
}

vn_status vn_perturbed_mlp_ex(const void* x, vn_dtype x_dt, int x_shared, int64_t n_layers,
                              const int64_t* dims, const float* const* w, const float* const* b,
                              const uint64_t* offsets, const int64_t* seeds, int64_t pop,
                              int64_t batch, double sigma, vn_act act, vn_noise kind, float* y,
                              void* stream) {
  if (kind != VN_NOISE_UNIFORM && kind != VN_NOISE_GAUSSIAN) return VN_ERR_VALUE;
  if (!dtype_ok(x_dt)) return VN_ERR_DTYPE;
  if (act != VN_ACT_NONE && act != VN_ACT_TANH) return VN_ERR_VALUE;
  if (n_layers < 1 || n_layers > vn::kMlpMaxLayers) return VN_ERR_SHAPE;
  if (dims == nullptr || w == nullptr || offsets == nullptr) return VN_ERR_NULL;
  if (pop < 0 || batch < 0 || batch > vn::kMlpMaxBatch) return VN_ERR_SHAPE;
  constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
  for (int64_t l = 0; l <= n_layers; ++l)
    if (dims[l] < 0 || dims[l] > kMaxDim) return VN_ERR_SHAPE;
  float sig;
  if (!float_sigma(sigma, &sig)) return VN_ERR_VALUE;
  int64_t x_elems, y_elems, t;
  if (!mul(batch, dims[0], &x_elems) || (!x_shared && !mul(x_elems, pop, &x_elems)) ||
      !mul(pop, batch, &t) || !mul(t, dims[n_layers], &y_elems))
    return VN_ERR_OVERFLOW;
  for (int64_t l = 0; l < n_layers; ++l) {
    int64_t we;
    if (!mul(dims[l], dims[l + 1], &we)) return VN_ERR_OVERFLOW;
    if (we > 0 && w[l] == nullptr) return VN_ERR_NULL;
    if (!aligned(w[l], 4) || (b != nullptr && !aligned(b[l], 4))) return VN_ERR_ALIGN;
  }
  if (y_elems == 0) return VN_OK;
  if (seeds == nullptr || y == nullptr || (x_elems > 0 && x == nullptr)) return VN_ERR_NULL;
  if (!aligned(seeds, 8) || !aligned(y, 4) || !aligned(x, dtype_size(x_dt))) return VN_ERR_ALIGN;
  {
    int64_t yb, xb, sb;
    if (!mul(y_elems, 4, &yb) || !mul(x_elems, dtype_size(x_dt), &xb) || !mul(pop, 8, &sb))
      return VN_ERR_OVERFLOW;
    if (overlap(y, yb, x, xb) || overlap(y, yb, seeds, sb)) return VN_ERR_VALUE;
    for (int64_t l = 0; l < n_layers; ++l) {
      int64_t wb;
      if (!mul(dims[l] * dims[l + 1], 4, &wb)) return VN_ERR_OVERFLOW;  // the product fits: checked above
      if (overlap(y, yb, w[l], wb) || (b != nullptr && overlap(y, yb, b[l], dims[l + 1] * 4)))
        return VN_ERR_VALUE;
    }
  }
  // The one device-dependent check: both activation buffers of one individual
  // must fit in the device's shared memory.
  const size_t buf = vn::mlp_buffer_floats(static_cast<int>(n_layers), dims);
  vn::DeviceInfo dev;
  cudaError_t err = vn::device_info(&dev);
  if (err != cudaSuccess) return cuda_failure(err);
  if (vn::mlp_bytes_per_individual(batch, buf) > static_cast<size_t>(dev.smem_optin))
    return VN_ERR_SHAPE;

  static const float* const kNoBias[vn::kMlpMaxLayers] = {};
  vn::MlpArgs m;
  m.x = x; m.x_dt = x_dt; m.x_shared = x_shared ? 1 : 0;
  m.n_layers = static_cast<int>(n_layers);
  m.dims = dims; m.w = w; m.b = b != nullptr ? b : kNoBias; m.offsets = offsets;
  m.seeds = seeds; m.pop = pop; m.batch = batch; m.sigma = sig; m.act = act; m.y = y;
  m.kind = kind;
  return launched(vn::launch_mlp(m, static_cast<cudaStream_t>(stream)));
}

vn_status vn_centered_ranks(const float* fitness, int64_t pop, float* out, void* stream) {
  if (pop < 0 || pop > (int64_t{1} << 31) - 1) return VN_ERR_SHAPE;
  if (pop == 0) return VN_OK;
  if (fitness == nullptr || out == nullptr) return VN_ERR_NULL;
  if (!aligned(fitness, 4) || !aligned(out, 4)) return VN_ERR_ALIGN;
  if (overlap(out, pop * 4, fitness, pop * 4)) return VN_ERR_VALUE;  // pop < 2^31: no overflow
  return launched(vn::launch_centered_ranks(fitness, pop, out, static_cast<cudaStream_t>(stream)));
}

vn_status vn_es_update(float* theta, const float* grad, int64_t n, double lr, void* stream) {
  if (n < 0) return VN_ERR_SHAPE;
  float lr_f;
  if (!float_sigma(lr, &lr_f)) return VN_ERR_VALUE;
  if (n == 0) return VN_OK;
  if (theta == nullptr || grad == nullptr) return VN_ERR_NULL;
  if (!aligned(theta, 4) || !aligned(grad, 4)) return VN_ERR_ALIGN;
  int64_t bytes;
  if (!mul(n, 4, &bytes)) return VN_ERR_OVERFLOW;
  if (overlap(theta, bytes, grad, bytes)) return VN_ERR_VALUE;
  return launched(vn::launch_es_update(theta, grad, n, lr_f, static_cast<cudaStream_t>(stream)));
}

vn_status vn_hash_probe(int64_t seed, uint64_t offset, int64_t n_sums, int64_t m, float* sums,
                        void* stream) {
  if (n_sums < 0 || n_sums > (int64_t{1} << 31) || m < 0) return VN_ERR_SHAPE;
  int64_t elems;
  if (!mul(n_sums, m, &elems)) return VN_ERR_OVERFLOW;
  if (n_sums == 0) return VN_OK;
  if (sums == nullptr) return VN_ERR_NULL;
  if (!aligned(sums, 4)) return VN_ERR_ALIGN;
  return launched(vn::launch_hash_probe(static_cast<uint64_t>(seed), offset, n_sums, m, sums,
                                        static_cast<cudaStream_t>(stream)));
}

int64_t vn_linear_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, int al) {
  if (check_sizes(rows, in, out, dt) != VN_OK || !features_ok(rows, in, out)) return -1;
  return vn::dense_workspace(rows, in, out, dt, al != 0);
}

vn_status vn_linear(const void* x, const void* w, vn_dtype dt, const void* b, vn_dtype b_dt,
                    const void* residual, int64_t rows, int64_t in, int64_t out, vn_act act,
                    void* y, void* preact, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  if (!dtype_ok(dt) || (b != nullptr && !dtype_ok(b_dt))) return VN_ERR_DTYPE;
  if (!linear_act_ok(act)) return VN_ERR_VALUE;
  const vn_status st = check_sizes(rows, in, out, dt);
  if (st != VN_OK) return st;
  if (rows == 0 || out == 0) return VN_OK;
  if (!features_ok(rows, in, out)) return VN_ERR_OVERFLOW;
  if (y == nullptr || (in > 0 && (x == nullptr || w == nullptr))) return VN_ERR_NULL;
  const size_t es = dtype_size(dt);
  if (!aligned(x, es) || !aligned(w, es) || !aligned(y, es) || !aligned(preact, es) ||
      !aligned(residual, es) || (b != nullptr && !aligned(b, dtype_size(b_dt))) || !aligned(workspace, 256))
    return VN_ERR_ALIGN;
  int64_t xb, wb, yb;
  if (!bytes_of(rows, in, dt, &xb) || !bytes_of(out, in, dt, &wb) || !bytes_of(rows, out, dt, &yb))
    return VN_ERR_OVERFLOW;
  const int64_t need =
      vn::dense_workspace(rows, in, out, dt, aligned(x, 16) && aligned(w, 16));
  if (need > 0 && workspace == nullptr) return VN_ERR_WORKSPACE;
  if (workspace_bytes < need) return VN_ERR_WORKSPACE;
  const int64_t bb = b != nullptr ? out * static_cast<int64_t>(dtype_size(b_dt)) : 0;
  const Range outs[] = {{y, yb}, {preact, yb}, {workspace, need}};
  const Range ins[] = {{x, xb}, {w, wb}, {b, bb}, {residual, yb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::DenseArgs a;
  a.x = x; a.w = w; a.dt = dt; a.b = b; a.b_dt = b_dt; a.residual = residual;
  a.rows = rows; a.in = in; a.out = out; a.act = act; a.y = y; a.preact = preact;
  a.workspace = workspace;
  return launched(vn::launch_dense(a, static_cast<cudaStream_t>(stream)));
}

vn_status vn_testhook_linear_plan(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, int al, int backward,
                                  int32_t* plan) {
  const vn_status st = check_sizes(rows, in, out, dt);
  if (st != VN_OK) return st;
  if (!linear_act_ok(act)) return VN_ERR_VALUE;
  if (rows > vn::kDenseMost || !features_ok(backward ? 9 : rows, in, out)) return VN_ERR_OVERFLOW;
  if (plan == nullptr) return VN_ERR_NULL;
  int32_t p[10];
  vn::dense_plan(rows, in, out, dt, act, al != 0, backward != 0, p);
  std::copy(p, p + 10, plan);
  return VN_OK;
}

vn_status vn_testhook_linear_withhold(int kernel, const void* x, const void* w, const void* residual, int64_t rows,
                                      int64_t in, int64_t out, void* y, void* preact, int64_t withhold,
                                      double timeout_ms, void* stream) {
  if (kernel < 0 || kernel == 3 || kernel > 6 || !(timeout_ms > 0.0) || !(timeout_ms <= 60000.0) || withhold < 0 || withhold > (1 << 30))
    return VN_ERR_VALUE;
  const vn_status st = check_sizes(rows, in, out, VN_BF16);
  if (st != VN_OK) return st;
  const int64_t most = int64_t{1} << 30;
  if (rows < 1 || out < 1 || in < 128 || in % 8 != 0 || out % 8 != 0 || rows > most || in > most || out > most)
    return VN_ERR_SHAPE;
  if (x == nullptr || w == nullptr || y == nullptr) return VN_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(preact, 16))
    return VN_ERR_ALIGN;
  const bool fp32 = kernel > 2;
  const int64_t es = fp32 ? 4 : 2, is = kernel > 4 ? 6 : es;  // of results and of operands
  const int64_t xb = rows * in * is, wb = out * in * is, yb = rows * out * es;
  const Range outs[] = {{y, yb}, {preact, yb}};
  const Range ins[] = {{x, xb}, {w, wb}, {residual, yb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::DenseArgs a = {};
  a.x = x; a.w = w; a.dt = fp32 ? VN_F32 : VN_BF16; a.residual = residual;
  a.rows = rows; a.in = in; a.out = out; a.act = VN_ACT_NONE; a.y = y; a.preact = preact;
  return launched(vn::launch_dense_hook(a, kernel, static_cast<int>(withhold),
                                        static_cast<unsigned long long>(timeout_ms * 1e6), static_cast<cudaStream_t>(stream)));
}

int64_t vn_linear_backward_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt,
                                     vn_act act, int al) {
  if (check_sizes(rows, in, out, dt) != VN_OK || !features_ok(9, in, out) || !linear_act_ok(act)) return -1;
  return vn::dense_backward_workspace(rows, in, out, dt, act, al != 0);
}

vn_status vn_linear_backward(const void* grad, const void* x, const void* w, const void* preact,
                             vn_dtype dt, int64_t rows, int64_t in, int64_t out, vn_act act,
                             void* grad_x, void* grad_w, void* grad_b, vn_dtype gb_dt,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt) || (grad_b != nullptr && !dtype_ok(gb_dt))) return VN_ERR_DTYPE;
  if (!linear_act_ok(act)) return VN_ERR_VALUE;
  const vn_status st = check_sizes(rows, in, out, dt);
  if (st != VN_OK) return st;
  const bool no_x = grad_x == nullptr || rows == 0 || in == 0;
  const bool no_w = grad_w == nullptr || out == 0 || in == 0;
  const bool no_b = grad_b == nullptr || out == 0;
  if (no_x && no_w && no_b) return VN_OK;
  if (!features_ok(9, in, out) || (rows > vn::kDenseMost && !(no_w && no_b))) return VN_ERR_OVERFLOW;
  const bool some = rows > 0 && out > 0;  // d has elements
  if (some && (grad == nullptr || (act != VN_ACT_NONE && preact == nullptr) || (!no_x && w == nullptr) ||
               (!no_w && x == nullptr)))
    return VN_ERR_NULL;
  const size_t es = dtype_size(dt);
  if (!aligned(grad, es) || !aligned(x, es) || !aligned(w, es) || !aligned(preact, es) ||
      !aligned(grad_x, es) || !aligned(grad_w, es) ||
      (grad_b != nullptr && !aligned(grad_b, dtype_size(gb_dt))) || !aligned(workspace, 256))
    return VN_ERR_ALIGN;
  int64_t xb, wb, yb;
  if (!bytes_of(rows, in, dt, &xb) || !bytes_of(out, in, dt, &wb) || !bytes_of(rows, out, dt, &yb))
    return VN_ERR_OVERFLOW;
  const int64_t need = vn::dense_backward_workspace(
      rows, in, out, dt, act, aligned(grad, 16) && aligned(x, 16) && aligned(w, 16));
  if (need > 0 && workspace == nullptr) return VN_ERR_WORKSPACE;
  if (workspace_bytes < need) return VN_ERR_WORKSPACE;
  const int64_t bb = grad_b != nullptr ? out * static_cast<int64_t>(dtype_size(gb_dt)) : 0;
  const Range outs[] = {{grad_x, xb}, {grad_w, wb}, {grad_b, bb}, {workspace, need}};
  const Range ins[] = {{grad, yb}, {x, xb}, {w, wb}, {act != VN_ACT_NONE ? preact : nullptr, yb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::DenseGradArgs a;
  a.grad = grad; a.x = x; a.w = w; a.preact = preact; a.dt = dt;
  a.rows = rows; a.in = in; a.out = out; a.act = act;
  a.grad_x = no_x ? nullptr : grad_x;
  a.grad_w = no_w ? nullptr : grad_w;
  a.grad_b = no_b ? nullptr : grad_b;
  a.gb_dt = gb_dt; a.workspace = workspace;
  return launched(vn::launch_dense_backward(a, static_cast<cudaStream_t>(stream)));
}

vn_status vn_layer_norm(const void* x, vn_dtype dt, const void* w, const void* b, vn_dtype w_dt,
                        int64_t rows, int64_t n, double eps, void* y, float* mean, float* rstd,
                        void* stream) {
  if (!dtype_ok(dt) || ((w != nullptr || b != nullptr) && !dtype_ok(w_dt))) return VN_ERR_DTYPE;
  float eps_f;
  if (!float_sigma(eps, &eps_f) || eps_f < 0.f) return VN_ERR_VALUE;
  if (rows < 0 || n < 1) return VN_ERR_SHAPE;
  int64_t xb, wb, sb;
  if (!bytes_of(rows, n, dt, &xb) || !bytes_of(1, n, w_dt, &wb) || !mul(rows, 4, &sb)) return VN_ERR_OVERFLOW;
  if (rows == 0) return VN_OK;
  if (x == nullptr || y == nullptr) return VN_ERR_NULL;
  const size_t es = dtype_size(dt), ws = dtype_size(w_dt);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(w, ws) || !aligned(b, ws) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return VN_ERR_ALIGN;
  const Range outs[] = {{y, xb}, {mean, sb}, {rstd, sb}};
  const Range ins[] = {{x, xb}, {w, wb}, {b, wb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::NormArgs a;
  a.x = x; a.dt = dt; a.w = w; a.b = b; a.w_dt = w_dt; a.rows = rows; a.n = n; a.eps = eps_f;
  a.y = y; a.mean = mean; a.rstd = rstd;
  return launched(vn::launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

int64_t vn_layer_norm_backward_workspace(int64_t rows, int64_t n) {
  int64_t bytes;
  if (rows < 0 || n < 1 || !mul(vn::layer_norm_parts(rows), n, &bytes) || !mul(bytes, 8, &bytes)) return -1;
  return bytes;
}

vn_status vn_layer_norm_backward(const void* grad, const void* x, vn_dtype dt, const float* mean,
                                 const float* rstd, const void* w, vn_dtype w_dt, int64_t rows,
                                 int64_t n, void* grad_x, void* grad_w, void* grad_b,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt) || !dtype_ok(w_dt)) return VN_ERR_DTYPE;
  if (rows < 0 || n < 1) return VN_ERR_SHAPE;
  int64_t xb, wb, sb;
  const int64_t need_sums = vn_layer_norm_backward_workspace(rows, n);
  if (!bytes_of(rows, n, dt, &xb) || !bytes_of(1, n, w_dt, &wb) || !mul(rows, 4, &sb) || need_sums < 0)
    return VN_ERR_OVERFLOW;
  const bool sums = grad_w != nullptr || grad_b != nullptr;
  if (rows == 0 && !sums) return VN_OK;
  if (rows > 0 && (grad == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || grad_x == nullptr))
    return VN_ERR_NULL;
  const size_t es = dtype_size(dt), ws = dtype_size(w_dt);
  if (!aligned(grad, es) || !aligned(x, es) || !aligned(grad_x, es) || !aligned(w, ws) ||
      !aligned(grad_w, ws) || !aligned(grad_b, ws) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 256))
    return VN_ERR_ALIGN;
  const int64_t need = sums ? need_sums : 0;
  if (sums && workspace == nullptr) return VN_ERR_WORKSPACE;
  if (workspace_bytes < need) return VN_ERR_WORKSPACE;
  const Range outs[] = {{grad_x, xb}, {grad_w, wb}, {grad_b, wb}, {workspace, need}};
  const Range ins[] = {{grad, xb}, {x, xb}, {mean, sb}, {rstd, sb}, {w, wb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::NormGradArgs a;
  a.grad = grad; a.x = x; a.dt = dt; a.mean = mean; a.rstd = rstd; a.w = w; a.w_dt = w_dt;
  a.rows = rows; a.n = n; a.grad_x = grad_x; a.grad_w = grad_w; a.grad_b = grad_b;
  a.part = static_cast<float*>(workspace);
  return launched(vn::launch_layer_norm_backward(a, static_cast<cudaStream_t>(stream)));
}

static vn_status check_adamw(const vn_adamw_tensor* tensors, int64_t n_tensors, vn_dtype param_dt, vn_dtype grad_dt,
                             int state_bits, double lr, double beta1, double beta2, double eps, int64_t step) {
  if (!dtype_ok(param_dt) || !dtype_ok(grad_dt)) return VN_ERR_DTYPE;
  if (state_bits != 8 && state_bits != 32) return VN_ERR_VALUE;
  float f;
  if (!float_sigma(lr, &f) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
      !float_sigma(eps, &f) || eps < 0.0 || step < 1)
    return VN_ERR_VALUE;
  if (n_tensors < 0) return VN_ERR_SHAPE;
  if (n_tensors == 0) return VN_OK;
  if (tensors == nullptr) return VN_ERR_NULL;
  const bool eight = state_bits == 8;
  const int64_t ps = static_cast<int64_t>(dtype_size(param_dt)), gs = static_cast<int64_t>(dtype_size(grad_dt));
  for (int64_t i = 0; i < n_tensors; ++i) {
    const vn_adamw_tensor& t = tensors[i];
    if (t.n < 0) return VN_ERR_SHAPE;
    if (!float_sigma(1.0 - lr * t.weight_decay, &f)) return VN_ERR_VALUE;
    if (t.n > (int64_t{1} << 59)) return VN_ERR_OVERFLOW;
    if (t.n == 0) continue;
    if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
        (eight && (t.exp_avg_scale == nullptr || t.exp_avg_sq_scale == nullptr)))
      return VN_ERR_NULL;
    const size_t ss = eight ? 1 : 4;
    if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.exp_avg, ss) ||
        !aligned(t.exp_avg_sq, ss) || (eight && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))))
      return VN_ERR_ALIGN;
    const int64_t sb = t.n * static_cast<int64_t>(ss), cb = eight ? (t.n + 255) / 256 * 4 : 0;
    const Range outs[] = {{t.param, t.n * ps}, {t.exp_avg, sb}, {t.exp_avg_sq, sb},
                          {t.exp_avg_scale, cb}, {t.exp_avg_sq_scale, cb}};
    const Range ins[] = {{t.grad, t.n * gs}};
    if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  }
  return VN_OK;
}

static vn::AdamwArgs adamw_args(const vn_adamw_tensor* tensors, int64_t n_tensors, vn_dtype param_dt, vn_dtype grad_dt,
                                int state_bits, double lr, double beta1, double beta2, double eps, int64_t step,
                                int maximize) {
  vn::AdamwArgs a;
  a.tensors = tensors; a.count = n_tensors; a.param_dt = param_dt; a.grad_dt = grad_dt;
  a.state_bits = state_bits; a.lr = lr; a.beta1 = beta1; a.beta2 = beta2; a.eps = eps;
  a.step = step; a.maximize = maximize ? 1 : 0;
  return a;
}

vn_status vn_adamw(const vn_adamw_tensor* tensors, int64_t n_tensors, vn_dtype param_dt,
                   vn_dtype grad_dt, int state_bits, double lr, double beta1, double beta2,
                   double eps, int64_t step, int maximize, void* stream) {
  const vn_status st = check_adamw(tensors, n_tensors, param_dt, grad_dt, state_bits, lr, beta1, beta2, eps, step);
  if (st != VN_OK || n_tensors == 0) return st;
  return launched(vn::launch_adamw(adamw_args(tensors, n_tensors, param_dt, grad_dt, state_bits, lr, beta1, beta2, eps, step,
                                              maximize),
                                   static_cast<cudaStream_t>(stream)));
}

vn_status vn_adamw_clipped(const vn_adamw_tensor* tensors, int64_t n_tensors, vn_dtype param_dt, vn_dtype grad_dt,
                           int state_bits, double lr, double beta1, double beta2, double eps, int64_t step, int maximize,
                           double max_norm, float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  vn_status st = check_adamw(tensors, n_tensors, param_dt, grad_dt, state_bits, lr, beta1, beta2, eps, step);
  if (st != VN_OK) return st;
  st = check_norm(n_tensors, max_norm, norm, workspace, workspace_bytes);
  if (st != VN_OK) return st;
  Spans spans(6 * n_tensors + 2);
  Pieces pieces(n_tensors);
  if (!spans.ok() || !pieces.ok()) return VN_ERR_OVERFLOW;
  const int64_t ps = static_cast<int64_t>(dtype_size(param_dt)), gs = static_cast<int64_t>(dtype_size(grad_dt));
  spans.add(norm, 4, true);
  spans.add(workspace, vn::clip_workspace(n_tensors), true);
  for (int64_t i = 0; i < n_tensors; ++i) {
    const vn_adamw_tensor& t = tensors[i];
    pieces[i] = {t.grad, nullptr, t.n};
    spans.add(t.grad, t.n * gs, false);
    spans.add(t.param, t.n * ps, true);
    const int64_t sb = t.n * (state_bits == 8 ? 1 : 4);
    spans.add(t.exp_avg, sb, true);
    spans.add(t.exp_avg_sq, sb, true);
    if (state_bits == 8) {
      spans.add(t.exp_avg_scale, (t.n + 255) / 256 * 4, true);
      spans.add(t.exp_avg_sq_scale, (t.n + 255) / 256 * 4, true);
    }
  }
  if (spans.clash()) return VN_ERR_VALUE;
  vn::ClipArgs c = {pieces.get(), n_tensors, grad_dt, max_norm, norm, false, workspace};
  const cudaError_t err = vn::launch_clip(c, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess || n_tensors == 0) return launched(err);
  vn::AdamwArgs a = adamw_args(tensors, n_tensors, param_dt, grad_dt, state_bits, lr, beta1, beta2, eps, step, maximize);
  a.factor = static_cast<const float*>(workspace);
  return launched(vn::launch_adamw(a, static_cast<cudaStream_t>(stream)));
}

int64_t vn_gradient_norm_workspace(int64_t n_tensors) {
  return n_tensors < 0 || n_tensors > kMostTensors ? -1 : vn::clip_workspace(n_tensors);
}

vn_status vn_gradient_norm(const vn_gradient* tensors, int64_t n_tensors, vn_dtype dt, float* norm, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  return clip(tensors, n_tensors, dt, HUGE_VAL, norm, workspace, workspace_bytes, false, stream);
}

vn_status vn_clip_gradients(const vn_gradient* tensors, int64_t n_tensors, vn_dtype dt, double max_norm, float* norm,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  return clip(tensors, n_tensors, dt, max_norm, norm, workspace, workspace_bytes, true, stream);
}

vn_status vn_adamw_moments(const void* exp_avg, const void* exp_avg_sq, const float* exp_avg_scale,
                           const float* exp_avg_sq_scale, int64_t n, float* m, float* v,
                           void* stream) {
  if (n < 0) return VN_ERR_SHAPE;
  if (n > (int64_t{1} << 59)) return VN_ERR_OVERFLOW;
  if (n == 0) return VN_OK;
  if (exp_avg == nullptr || exp_avg_sq == nullptr || exp_avg_scale == nullptr || exp_avg_sq_scale == nullptr ||
      m == nullptr || v == nullptr)
    return VN_ERR_NULL;
  if (!aligned(exp_avg_scale, 4) || !aligned(exp_avg_sq_scale, 4) || !aligned(m, 4) || !aligned(v, 4))
    return VN_ERR_ALIGN;
  const int64_t cb = (n + 255) / 256 * 4;
  const Range outs[] = {{m, n * 4}, {v, n * 4}};
  const Range ins[] = {{exp_avg, n}, {exp_avg_sq, n}, {exp_avg_scale, cb}, {exp_avg_sq_scale, cb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  return launched(vn::launch_adamw_moments(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, n, m, v,
                                           static_cast<cudaStream_t>(stream)));
}

int64_t vn_packed_row_bytes(int64_t in) { return in < 0 || in > kMostFeatures ? -1 : vn::packed_row_bytes(in); }

// The sizes of packed weights, and the bytes of their arrays.
static vn_status packed_sizes(int64_t out, int64_t in, int group, vn_dtype dt, int64_t* wb, int64_t* cb, int64_t* sb) {
  if (!dtype_ok(dt)) return VN_ERR_DTYPE;
  if (group != 32 && group != 64 && group != 128) return VN_ERR_VALUE;
  if (out < 0 || in < 0) return VN_ERR_SHAPE;
  if (in > kMostFeatures || !bytes_of(out, in, dt, wb) || !mul(out, vn::packed_row_bytes(in), cb) ||
      !bytes_of(out, (in + group - 1) / group, dt, sb))
    return VN_ERR_OVERFLOW;
  return VN_OK;
}

vn_status vn_pack_weight(const void* w, vn_dtype dt, int64_t out, int64_t in, int group, void* codes, void* scales,
                         void* stream) {
  int64_t wb, cb, sb;
  const vn_status st = packed_sizes(out, in, group, dt, &wb, &cb, &sb);
  if (st != VN_OK || wb == 0) return st;
  if (w == nullptr || codes == nullptr || scales == nullptr) return VN_ERR_NULL;
  if (!aligned(w, dtype_size(dt)) || !aligned(codes, 16) || !aligned(scales, dtype_size(dt))) return VN_ERR_ALIGN;
  const Range outs[] = {{codes, cb}, {scales, sb}};
  const Range ins[] = {{w, wb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  return launched(vn::launch_pack(w, dt, out, in, group, static_cast<uint8_t*>(codes), scales, static_cast<cudaStream_t>(stream)));
}

vn_status vn_unpack_weight(const void* codes, const void* scales, vn_dtype dt, int64_t out, int64_t in, int group, void* w,
                           void* stream) {
  int64_t wb, cb, sb;
  const vn_status st = packed_sizes(out, in, group, dt, &wb, &cb, &sb);
  if (st != VN_OK || wb == 0) return st;
  if (w == nullptr || codes == nullptr || scales == nullptr) return VN_ERR_NULL;
  if (!aligned(w, dtype_size(dt)) || !aligned(codes, 16) || !aligned(scales, dtype_size(dt))) return VN_ERR_ALIGN;
  const Range outs[] = {{w, wb}};
  const Range ins[] = {{codes, cb}, {scales, sb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  return launched(vn::launch_unpack(static_cast<const uint8_t*>(codes), scales, dt, out, in, group, w, static_cast<cudaStream_t>(stream)));
}

int64_t vn_linear_packed_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, int al) {
  if (check_sizes(rows, in, out, dt) != VN_OK || !features_ok(rows, in, out) || in > kMostFeatures) return -1;
  return vn::packed_workspace(rows, in, out, dt, al != 0);
}

vn_status vn_linear_packed(const void* x, const void* codes, const void* scales, vn_dtype dt, int group, const void* b,
                           vn_dtype b_dt, const void* residual, int64_t rows, int64_t in, int64_t out, vn_act act, void* y,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt) || (b != nullptr && !dtype_ok(b_dt))) return VN_ERR_DTYPE;
  if (!linear_act_ok(act)) return VN_ERR_VALUE;
  int64_t wb, cb, sb, xb, yb;
  vn_status st = packed_sizes(out, in, group, dt, &wb, &cb, &sb);
  if (st != VN_OK) return st;
  st = check_sizes(rows, in, out, dt);
  if (st != VN_OK) return st;
  if (rows == 0 || out == 0) return VN_OK;
  if (!features_ok(rows, in, out)) return VN_ERR_OVERFLOW;
  if (y == nullptr || (in > 0 && (x == nullptr || codes == nullptr || scales == nullptr))) return VN_ERR_NULL;
  const size_t es = dtype_size(dt);
  if (!aligned(x, es) || !aligned(codes, 16) || !aligned(scales, es) || !aligned(y, es) || !aligned(residual, es) ||
      (b != nullptr && !aligned(b, dtype_size(b_dt))) || !aligned(workspace, 256))
    return VN_ERR_ALIGN;
  if (!bytes_of(rows, in, dt, &xb) || !bytes_of(rows, out, dt, &yb)) return VN_ERR_OVERFLOW;
  const int64_t need = vn::packed_workspace(rows, in, out, dt, aligned(x, 16));
  if ((need > 0 && workspace == nullptr) || workspace_bytes < need) return VN_ERR_WORKSPACE;
  const int64_t bb = b != nullptr ? out * static_cast<int64_t>(dtype_size(b_dt)) : 0;
  const Range outs[] = {{y, yb}, {workspace, need}};
  const Range ins[] = {{x, xb}, {codes, cb}, {scales, sb}, {b, bb}, {residual, yb}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::PackedArgs a;
  a.x = x; a.codes = static_cast<const uint8_t*>(codes); a.scales = scales; a.dt = dt; a.group = group; a.b = b; a.b_dt = b_dt;
  a.residual = residual; a.rows = rows; a.in = in; a.out = out; a.act = act; a.y = y; a.workspace = workspace;
  return launched(vn::launch_packed(a, static_cast<cudaStream_t>(stream)));
}

vn_status vn_sample(const void* logits, vn_dtype dt, int64_t rows, int64_t n, const float* u, double temperature,
                    const float* temperatures, int64_t top_k, const int64_t* top_ks, double top_p, const float* top_ps,
                    double min_p, const float* min_ps, int64_t* index, float* logprob, void* stream) {
  if (!dtype_ok(dt)) return VN_ERR_DTYPE;
  if (!std::isfinite(temperature) || !std::isfinite(top_p) || !std::isfinite(min_p)) return VN_ERR_VALUE;
  if (rows < 0 || n < 1 || n > vn::kSampleMost) return VN_ERR_SHAPE;
  int64_t xb, r8;
  if (!bytes_of(rows, n, dt, &xb) || !mul(rows, 8, &r8)) return VN_ERR_OVERFLOW;
  if (rows == 0) return VN_OK;
  if (logits == nullptr || u == nullptr || index == nullptr) return VN_ERR_NULL;
  if (!aligned(logits, dtype_size(dt)) || !aligned(u, 4) || !aligned(temperatures, 4) || !aligned(top_ks, 8) ||
      !aligned(top_ps, 4) || !aligned(min_ps, 4) || !aligned(index, 8) || !aligned(logprob, 4))
    return VN_ERR_ALIGN;
  const Range outs[] = {{index, r8}, {logprob, r8 / 2}};
  const Range ins[] = {{logits, xb}, {u, r8 / 2}, {temperatures, r8 / 2}, {top_ks, r8}, {top_ps, r8 / 2}, {min_ps, r8 / 2}};
  if (!disjoint(outs, ins)) return VN_ERR_VALUE;
  vn::SampleArgs a;
  a.logits = logits; a.dt = dt; a.rows = rows; a.n = n; a.u = u;
  a.temperature = temperature; a.top_p = top_p; a.min_p = min_p; a.top_k = top_k;
  a.temperatures = temperatures; a.top_ks = top_ks; a.top_ps = top_ps; a.min_ps = min_ps;
  a.index = index; a.logprob = logprob;
  return launched(dt == VN_BF16 ? vn::launch_sample_bf16(a, static_cast<cudaStream_t>(stream))
                                : vn::launch_sample_f32(a, static_cast<cudaStream_t>(stream)));
}

vn_status vn_device_status(void* stream) {
  cudaError_t err = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_failure(err);
  unsigned int status = 0;
  err = vn::take_device_status(&status, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return cuda_failure(err);
  return status ? VN_ERR_TIMEOUT : VN_OK;
}

}  // extern "C"
