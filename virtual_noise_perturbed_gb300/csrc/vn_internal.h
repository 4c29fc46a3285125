// vn_internal.h -- launchers shared between the C-ABI layer (vn_api.cu) and
// the kernel translation units. Arguments reaching these functions have been
// validated by the C-ABI layer: pointers non-null and aligned, sizes >= 1 and
// their products below 2^63.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "vn.h"
#include "vn_smem.h"

namespace vn {

// Cached per-device facts (SM count, compute capability, opt-in shared memory).
struct DeviceInfo {
  int device = -1;
  int sm_count = 0;
  int cc_major = 0;
  int cc_minor = 0;
  int smem_optin = 0;
};
cudaError_t device_info(DeviceInfo* info);

// out[i, t] = PRNG(seed_i, offset + t), t < n; kind: VN_NOISE_UNIFORM (the
// centered uniform, exact) or VN_NOISE_GAUSSIAN (the Box-Muller variant).
cudaError_t launch_noise_dump(const int64_t* seeds, int64_t pop, int64_t n, uint64_t offset,
                              int kind, float* out, cudaStream_t stream);

// out[e] = scale * sum_i fitness[i] * PRNG(seed_i, offset + e), e < m, with the noise of `kind`;
// with theta != NULL also theta[e] = fma(lr, out[e], theta[e]).
cudaError_t launch_grad(const float* fitness, const int64_t* seeds, int64_t pop, int64_t m,
                        uint64_t offset, float scale, int kind, float* out, cudaStream_t stream,
                        float* theta = nullptr, float lr = 0.f);

// fitness[i] = inv_n * sum_k |center[k] + sigma * PRNG(seed_i, offset + k)|.
cudaError_t launch_reduce_metric(const float* center, const int64_t* seeds, int64_t pop,
                                 int64_t n, float sigma, float inv_n, uint64_t offset,
                                 float* fitness, cudaStream_t stream);

struct LinearArgs {
  const void* x;
  vn_dtype x_dt;
  int x_shared;
  const void* w;
  vn_dtype w_dt;
  const void* b;  // may be null
  vn_dtype b_dt;
  const int64_t* seeds;
  int64_t pop, batch, in, out;
  float sigma;
  uint64_t offset;
  void* y;
  vn_dtype y_dt;
  vn_act act;
  int kind = 0;  // noise kind: 0 the centered uniform, 1 the Gaussian variant
};

// CUDA-core forward: any dtypes, any batch.
cudaError_t launch_linear_ffma(const LinearArgs& a, cudaStream_t stream);

// Whether the tcgen05 forward can run these arguments (shape/alignment/dtype).
bool linear_tc_applies(const void* x, vn_dtype x_dt, const void* w, vn_dtype w_dt,
                       int64_t batch, int64_t in, int64_t out);
// tcgen05/TMEM forward (x bf16).
cudaError_t launch_linear_tc(const LinearArgs& a, cudaStream_t stream);
// The same with every barrier wait bounded by timeout_ns and, when
// withhold_stage >= 0, one hashing thread of CTA 0 skipping its arrive at that
// stage (test hook for the bounded-wait path).
cudaError_t launch_linear_tc_hook(const LinearArgs& a, cudaStream_t stream, long long withhold_stage,
                                  unsigned long long timeout_ns);

// A chain of perturbed linear layers in one launch (fp32 weights, batch <= 8).
constexpr int kMlpMaxLayers = 8;
constexpr int64_t kMlpMaxBatch = 8;
struct MlpArgs {
  const void* x;
  vn_dtype x_dt;
  int x_shared;
  int n_layers;
  const int64_t* dims;       // host, n_layers + 1
  const float* const* w;     // host array of device pointers
  const float* const* b;     // host array of device pointers (entries may be null)
  const uint64_t* offsets;   // host, n_layers
  const int64_t* seeds;
  int64_t pop, batch;
  float sigma;
  vn_act act;        // between layers
  float* y;
  vn_act act_last = VN_ACT_NONE;  // after the last layer (a single perturbed linear's own)
  int kind = 0;                   // noise kind: 0 the centered uniform, 1 the Gaussian variant
};
// Floats per (individual, batch row) of one activation buffer for these dims.
size_t mlp_buffer_floats(int n_layers, const int64_t* dims);
// Shared memory the kernel needs for one individual at this batch (both buffers).
inline size_t mlp_bytes_per_individual(int64_t batch, size_t buf_floats) {
  const int64_t nb = batch <= 1 ? 1 : batch <= 2 ? 2 : batch <= 4 ? 4 : 8;
  return 2 * static_cast<size_t>(nb) * buf_floats * sizeof(float) + 64;
}
cudaError_t launch_mlp(const MlpArgs& m, cudaStream_t stream);

// out[i] = rank of fitness[i] (ascending, ties by index) / (pop - 1) - 0.5.
cudaError_t launch_centered_ranks(const float* fitness, int64_t pop, float* out,
                                  cudaStream_t stream);
// theta[k] += lr * grad[k], k < n.
cudaError_t launch_es_update(float* theta, const float* grad, int64_t n, float lr,
                             cudaStream_t stream);

// sums[t] = sum_{e < m} PRNG(seed, offset + t*m + e), t < n_sums: the hash alone.
cudaError_t launch_hash_probe(uint64_t seed, uint64_t offset, int64_t n_sums, int64_t m,
                              float* sums, cudaStream_t stream);

// The centre network (arguments as in vn.h; sizes may be zero where it says so).
// The most features of a layer of more than 8 rows, and the most rows that its gradients sum over: the kernels'
// coordinates have 32 bits.
constexpr int64_t kDenseMost = (int64_t{1} << 31) - 512;
struct DenseArgs {
  const void* x;
  const void* w;
  vn_dtype dt;
  const void* b;  // may be null
  vn_dtype b_dt;
  const void* residual;  // may be null
  int64_t rows, in, out;
  vn_act act;
  void* y;
  void* preact;  // may be null
  void* workspace;
};
struct DenseGradArgs {
  const void* grad;
  const void* x;
  const void* w;
  const void* preact;  // null without an activation
  vn_dtype dt;
  int64_t rows, in, out;
  vn_act act;
  void* grad_x;  // may be null, and the other two
  void* grad_w;
  void* grad_b;
  vn_dtype gb_dt;
  void* workspace;
};
// Bytes of workspace; sizes have been checked (products of bytes fit in int64).
int64_t dense_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned);
int64_t dense_backward_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act,
                                 bool aligned);
cudaError_t launch_dense(const DenseArgs& a, cudaStream_t stream);
cudaError_t launch_dense_backward(const DenseGradArgs& a, cudaStream_t stream);
// The test hook of vn_testhook_linear_plan (vn.h).
void dense_plan(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned, bool backward, int32_t (&p)[10]);
// The test hook of vn_testhook_linear_withhold (vn.h): in a multiple of 8 and at least 128, out a
// multiple of 8, every pointer on 16 bytes.
cudaError_t launch_dense_hook(const DenseArgs& a, int kernel, int at, unsigned long long timeout_ns, cudaStream_t stream);

struct NormArgs {
  const void* x;
  vn_dtype dt;
  const void* w;  // may be null, and b, mean and rstd
  const void* b;
  vn_dtype w_dt;
  int64_t rows, n;
  float eps;
  void* y;
  float* mean;
  float* rstd;
};
struct NormGradArgs {
  const void* grad;
  const void* x;
  vn_dtype dt;
  const float* mean;
  const float* rstd;
  const void* w;  // may be null, and grad_w and grad_b
  vn_dtype w_dt;
  int64_t rows, n;
  void* grad_x;
  void* grad_w;
  void* grad_b;
  float* part;  // [layer_norm_parts(rows)][2][n]
};
cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t stream);
int64_t layer_norm_parts(int64_t rows);
cudaError_t launch_layer_norm_backward(const NormGradArgs& a, cudaStream_t stream);
// o1[c] = sum_p part[p][c] for c < n, o2[c - n] for the columns from n on (width of them in
// all), in fixed order, rounded to dt; o1 and o2 may be null.
cudaError_t launch_column_sum(const float* part, int64_t parts, int64_t width, int64_t n, void* o1,
                              void* o2, vn_dtype dt, cudaStream_t stream);

// The norm of a gradient, and what is done with it.
constexpr int kClipParts = 1216;  // partial sums of a launch at most
struct ClipArgs {
  const vn_gradient* tensors;  // host
  int64_t count;
  vn_dtype dt;
  double bound;
  float* norm;
  bool scale;       // write each tensor's out
  void* workspace;  // clip_workspace(count) bytes; the factor is left as its first float
};
int64_t clip_workspace(int64_t count);
cudaError_t launch_clip(const ClipArgs& a, cudaStream_t stream);

struct AdamwArgs {
  const vn_adamw_tensor* tensors;  // host
  int64_t count;
  vn_dtype param_dt, grad_dt;
  int state_bits;
  double lr, beta1, beta2, eps;
  int64_t step;
  int maximize;
  const float* factor = nullptr;  // device: what gradients are multiplied by, 1 if null
};
cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t stream);
cudaError_t launch_adamw_moments(const void* exp_avg, const void* exp_avg_sq, const float* exp_avg_scale,
                                 const float* exp_avg_sq_scale, int64_t n, float* m, float* v,
                                 cudaStream_t stream);

// Weights in 4 bits, and the linear layer on them.
struct PackedArgs {
  const void* x;
  const uint8_t* codes;
  const void* scales;
  vn_dtype dt;
  int group;
  const void* b;  // may be null
  vn_dtype b_dt;
  const void* residual;  // may be null
  int64_t rows, in, out;
  vn_act act;
  void* y;
  void* workspace;
};
int64_t packed_row_bytes(int64_t in);
cudaError_t launch_pack(const void* w, vn_dtype dt, int64_t out, int64_t in, int group, uint8_t* codes, void* scales, cudaStream_t stream);
cudaError_t launch_unpack(const uint8_t* codes, const void* scales, vn_dtype dt, int64_t out, int64_t in, int group, void* w,
                          cudaStream_t stream);
int64_t packed_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned);
cudaError_t launch_packed(const PackedArgs& a, cudaStream_t stream);

// An index for each row of logits.
constexpr int64_t kSampleMost = int64_t{1} << 19;  // logits of a row: what a cluster of 16 CTAs holds in shared memory
struct SampleArgs {
  const void* logits;
  vn_dtype dt;
  int64_t rows, n;
  const float* u;
  double temperature, top_p, min_p;
  int64_t top_k;
  const float* temperatures;  // of each row, in the scalar's place; may be null, and the other three
  const int64_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  int64_t* index;
  float* logprob;  // may be null
};
cudaError_t launch_sample_f32(const SampleArgs& a, cudaStream_t stream);
cudaError_t launch_sample_bf16(const SampleArgs& a, cudaStream_t stream);

// The current device's status word, which every bounded wait that runs out sets.
cudaError_t device_status_word(unsigned int** word);
// Reads and clears the device status word of the bounded-wait kernels (0 = fine).
cudaError_t take_device_status(unsigned int* status, cudaStream_t stream);

}  // namespace vn
