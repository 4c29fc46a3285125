// vn_dense.h -- the product that the centre network's linear layer and its gradients are
// made of, shared by its dispatcher (vn_dense.cu) and its tensor-core kernels (vn_dense_tc.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "vn.h"

namespace vn {

// How a product is tiled, and its time on a GB300 as the dispatcher reckons it (vn_dense.cu). bn: the
// tile's columns; log_split: log2 of the CTAs that share a tile's k loop.
struct TilePlan {
  double us = 1e30;
  bool pair = false;  // pairs of CTAs on 256 x bn tiles, else single CTAs on 128 x bn
  int bn = 64;
  int log_split = 0;
};
struct GatherPlan {
  double us = 1e30;
  int bn = 64;
  int log_split[2] = {0, 0};  // of the forward product, or of grad_x's; of grad_w's
};

// A bf16 operand of the tensor-core kernels: [planes][rows][pitch], of which the first `cols`
// of each row count. mn: the contiguous dimension is p (or q), the rows are k; otherwise k is
// contiguous. p is 16-byte aligned, pitch a multiple of 8, plane (elements) too.
struct TcOperand {
  const void* p;
  int64_t rows, cols, pitch, plane;
  int planes;  // 1, or 3: an fp32 matrix as the sum of three
  bool mn;
};

// out[q, p] = act(sum_k A(p, k) B(q, k) + bias[p]) + residual[q, p], preact before act.
// Layouts (a.mn, b.mn): (false, false), (true, false) and (true, true). nk >= 1; np, nq and nk
// below 2^31 - 256.
struct TcProduct {
  TcOperand a, b;
  int64_t np, nq, nk;
  vn_dtype dt;  // of residual, out and preact
  const void* bias;
  int bias_bf16, act;
  const void* residual;
  void* out;
  void* preact;
};
// A test's limit on every wait of a launch, and what it withholds so that one of them runs out: of the
// first CTA's handovers of operands to the MMAs that number `at` (from 0).
struct Withhold {
  int at;
  unsigned long long timeout_ns;
};
// hook: k-contiguous operands only; single tiles of 64 columns, pairs whose rows TMA can store.
cudaError_t launch_tc_product(const TcProduct& d, const TilePlan& plan, cudaStream_t stream, const Withhold* hook = nullptr);

// A layer, or all its gradients, in one launch, for any alignment and no workspace
// (vn_dense_gather.cu). At least one of grad_x and grad_w is asked for, and grad_b only with
// grad_w; rows, in and out up to 2^31 - 512. A sum over nothing is zero: in may be 0 in the forward
// product, rows or out in the gradients.
struct DenseArgs;
struct DenseGradArgs;
cudaError_t launch_rows_forward(const DenseArgs& a, cudaStream_t stream);  // rows <= 8 (vn_dense_rows.cu)
// hook: rows that start on 16 bytes, on 16 columns, fp32 in pieces. Beyond a CTA's last chunk, `at` is the commit
// that the epilogue waits for.
cudaError_t launch_gather_forward(const DenseArgs& a, const GatherPlan& plan, cudaStream_t stream,
                                  const Withhold* hook = nullptr);
cudaError_t launch_gather_backward(const DenseGradArgs& a, const GatherPlan& plan, cudaStream_t stream);

}  // namespace vn
