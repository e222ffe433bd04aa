// Row kernels of the stack update (declarations shared by stack.cu and api.cu).
#pragma once

#include "internal.h"

namespace muon {

// One stack of `count` rows x cols matrices in a batched launch; matrix b,
// row r of W starts at W + b * w_stride + r * w_ld (the others alike). X is
// the operand buffer: [count][planes][rows][ldx].
struct StackMat {
  void* W;
  float* M;
  const void* G;  // NULL: M already holds this step's gradient
  void* copy;     // NULL: none
  void* X;
  int64_t w_stride, w_ld, m_stride, m_ld, g_stride, g_ld, c_stride, c_ld;
  int64_t ldx;
  int32_t rows, cols, count;
  int32_t w_type, g_type, c_type;  // muon_dtype
  int32_t vec;                     // four-element accesses are aligned in every array
  int32_t row_begin, mat_begin;    // first row and matrix of the stack in the launch
  float kappa;                     // storage scale of the operands
};

constexpr int kMaxStacks = 64;  // per launch; the table travels in the kernel parameters

struct StackLaunch {
  StackMat m[kMaxStacks];
  int count;
  int total_rows, total_mats;
  double* rsum;   // per row: sum of squares of the update's target
  float* scale;   // per matrix: 1 / (norm + eps)
  float* xscale;  // per matrix: true X_0 = xscale * stored operand
  float mu, step, keep;  // W <- keep W - step O
  float eps;
  int nesterov;
  int folded;     // the operand is stored unscaled, scale enters the first products
  int sums;       // the cast adds the row sums itself (no launch_stack_norm)
  int clear;      // the momentum launch sets *status to MUON_OK
  int* status;
};
static_assert(sizeof(StackLaunch) <= 32764, "kernel parameters are limited to 32764 bytes");

// M <- mu M + G; rsum <- row sums of squares of the target (M, or G + mu M);
// with `cast` also X <- target, unscaled (type t).
muon_status launch_stack_momentum(const StackLaunch& L, Op t, bool cast, cudaStream_t s);
// scale, xscale of every matrix from rsum.
muon_status launch_stack_norm(const StackLaunch& L, cudaStream_t s);
// X <- kappa * scale * target in type t and one or two planes.
muon_status launch_stack_cast(const StackLaunch& L, Op t, int planes, cudaStream_t s);
// W <- keep W - step O (and its copy), O = X / kappa where two planes, else X.
muon_status launch_stack_update(const StackLaunch& L, Op t, int planes, cudaStream_t s);

// The whole update of one stack (L.m[0]) of small matrices in one launch
// (resident.cu): whether that is the faster way for T steps on this device
// (and the CTAs per matrix), and the launch. kappa and rho are the storage
// scales of X and of the n x n matrices.
bool resident_fits(int64_t rows, int64_t cols, int64_t count, int T, int planes, int* C_out);
muon_status launch_stack_resident(const StackLaunch& L, const muon_ns_params& ns, Op t, int planes, float kappa, float rho,
                                  uint64_t timeout_ns, cudaStream_t s);

}  // namespace muon
