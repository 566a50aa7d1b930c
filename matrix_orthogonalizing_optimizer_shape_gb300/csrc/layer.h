// Internal launcher interface of the layer operators (RMS norm, linear layer,
// 8-bit checkpoints).  Nothing here crosses the C ABI (include/dion3.h).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"

namespace dion3 {

constexpr int kPackBlock = 32;  // columns that share one scale byte

// Row-major matrix, row pitch in elements; null data: absent.
struct Mat {
  void* p = nullptr;
  long long ld = 0;
};
// 8-bit blocks: codes [rows][ldq], scale bytes [rows][lds]; null: absent.
struct Pack8 {
  int8_t* q = nullptr;
  long long ldq = 0;
  uint8_t* s = nullptr;
  long long lds = 0;
};

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

// SMs of the current device.
int sm_count();

// ---------------------------------------------------------------------------
// Memory-bound kernels (layer_mem.cu)
// ---------------------------------------------------------------------------
cudaError_t launch_pack8(int rows, int cols, int dtype, Mat x, Pack8 out, cudaStream_t s);
cudaError_t launch_unpack8(int rows, int cols, Pack8 in, int dtype, Mat out, cudaStream_t s);

struct NormArgs {
  int rows, cols, dtype;      // dtype of x, residual, h and y
  Mat x, residual, h, y;      // residual, h, y may be absent
  const void* w; int w_dtype;
  float eps;
  Pack8 y8;                   // may be absent
  float* rstd;                // may be null
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s);

// Widest row the norm's kernels take: 32-bit column sums of a row in shared
// memory.
constexpr int kNormMaxCols = 49152;
// Rows of 32-bit column-sum partials at most (rows of a workspace).
constexpr int kMaxPartials = 608;
struct NormGradArgs {
  int rows, cols, dtype;      // dtype of dy, h, dh and dx
  Mat dy, h, dh, dx;          // dh may be absent
  const void* w; int w_dtype;
  const float* rstd;
  float* dw;                  // null: not wanted
  int accumulate;
  float* partials;            // [<= kMaxPartials][cols]
  int strips = 0;             // blocks that give dw themselves
};
cudaError_t launch_rms_norm_grad(const NormGradArgs& a, cudaStream_t s);

// dz = dy act'(z) in the 16-bit type, and column sums of the unrounded dz.
struct ActGradArgs {
  int rows, cols, dtype, act;
  Mat dy, z;                  // z absent: z8, or no activation
  Pack8 z8;
  Mat dz;                     // absent: column sums only
  float* db;                  // null: not wanted
  int accumulate;
  float* partials;            // [<= kMaxPartials][cols]
};
cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s);
// Up to this many rows one block takes all of a strip of columns.
constexpr int kFewRowsOfDz = 256;

// 16-bit matrices (n = 1 or 2) copied to a pitch that TMA takes.
struct Repitch {
  int rows, cols;
  Mat src, dst;
};
cudaError_t launch_repitch(const Repitch* jobs, int n, cudaStream_t s);
// launch_act_grad, launch_repitch and, if x8 is given, launch_unpack8 into x
// (16-byte aligned, whole pieces) in one launch, for small matrices.
cudaError_t launch_prepare(const ActGradArgs& act, const Repitch* copies, int ncopies, int rows, int cols, Pack8 x8,
                           Mat x, cudaStream_t s);
// out[rows][cols] = 0 (32- or 16-bit elements, dense), or a 32-bit vector.
cudaError_t launch_zero(int rows, int cols, int elem_bytes, Mat out, cudaStream_t s);

// ---------------------------------------------------------------------------
// Products (layer_gemm.cu), 16-bit operands, 32-bit accumulation:
//   out[t][m] = sum_k A(m, k) B(t, k)
// A(m, k) = A[m][k], or A[k][m] when a_mn; B likewise.  All pointers 16-byte
// aligned and pitches multiples of 8 elements (launch_repitch otherwise).
// ---------------------------------------------------------------------------
struct Product {
  int M, N, K;                // M contiguous in the outputs, N rows of the outputs
  int elem;                   // kBF16 or kF16: operands, 16-bit outputs, residual
  Mat A, B;
  bool a_mn, b_mn;
  Mat out; int out_dtype;     // elem; of a gradient (a_mn, b_mn) any dtype
  int accumulate;             // out += ...
  // Forward epilogue: z = v + bias, out = act(z) + residual.
  const void* bias; int bias_dtype;
  int act;
  Mat residual, z;
  Pack8 z8, out8;
};
cudaError_t launch_product(const Product& g, unsigned* status, cudaStream_t s);

}  // namespace dion3
