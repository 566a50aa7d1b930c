// Memory-bound kernels of the layer operators on sm_103a: 8-bit checkpoints,
// the RMS norm with the residual's addition and its gradient, and the
// activation's gradient with the bias gradient's column sums.
#include <algorithm>
#include <type_traits>

#include "layer_math.cuh"

namespace dion3 {
namespace {

using namespace lm;

__device__ __forceinline__ float load_w(const void* w, int dtype, int c) {
  if (dtype == kF32) return static_cast<const float*>(w)[c];
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  return __half2float(static_cast<const __half*>(w)[c]);
}

// Largest |v| bits over the lanes that share a block of 32 columns (VEC
// columns a lane).  Magnitudes compare as unsigned integers; a NaN compares
// above every number.
template <int VEC>
__device__ __forceinline__ uint32_t block_amax(const float (&v)[VEC]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < kPackBlock / VEC; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Codes (and, from the block's first lane, its scale byte) of VEC columns at
// column c of a row.  Lanes of a warp hold consecutive columns from a multiple
// of 32; values of columns past the end are 0 and not written.
template <int VEC>
__device__ __forceinline__ void store_block(const Pack8& o, long long row, int c, int cols, float (&v)[VEC]) {
  const uint32_t byte = scale_byte(block_amax<VEC>(v));
  const float inv = inv_scale(byte);
  saturate_block(byte, v);
  if (c >= cols) return;
  int8_t* q = o.q + row * o.ldq + c;
  if constexpr (VEC == 8) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j / 4] |= code_of(v[j], inv) << (8 * (j % 4));
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  } else {
    *q = static_cast<int8_t>(code_of(v[0], inv));
  }
  if (c % kPackBlock == 0) o.s[row * o.lds + c / kPackBlock] = static_cast<uint8_t>(byte);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_cols(const Mat& m, long long row, int c, int cols, float (&v)[VEC]) {
  if (c < cols) {
    load_vec<T, VEC>(static_cast<const T*>(m.p) + row * m.ld + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = 0.f;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_cols(const Mat& m, long long row, int c, int cols, const float (&v)[VEC]) {
  if (c < cols) store_vec<T, VEC>(static_cast<T*>(m.p) + row * m.ld + c, v);
}

// Sum over the CTA, the same bits in every thread (blockDim.x a multiple of
// 32).  `red` alternates between two halves so one barrier a call is enough.
__device__ __forceinline__ float cta_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int nw = blockDim.x / 32;
  if (nw == 1) return v;
  float* r = red + 32 * flip;
  flip ^= 1;
  if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = v;
  __syncthreads();
  v = threadIdx.x % 32 < nw ? r[threadIdx.x % 32] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// --------------------------------------------------------------------------
// 8-bit checkpoints
// --------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void __launch_bounds__(256) pack8_kernel(int rows, int cols, Mat x, Pack8 o) {
  const int per_row = (cols + kPackBlock - 1) / kPackBlock * (kPackBlock / VEC);  // lanes of a row, whole blocks
  const long long total = (static_cast<long long>(rows) * per_row + 31) / 32 * 32;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / per_row;
    const int c = row < rows ? static_cast<int>(i - row * per_row) * VEC : cols;
    float v[VEC];
    load_cols<T, VEC>(x, row, c, cols, v);
    store_block<VEC>(o, row, c, cols, v);
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) unpack8_kernel(int rows, int cols, Pack8 in, Mat out) {
  const int per_row = (cols + VEC - 1) / VEC;
  const long long total = static_cast<long long>(rows) * per_row;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / per_row;
    const int c = static_cast<int>(i - row * per_row) * VEC;
    const float sc = scale_of(in.s[row * in.lds + c / kPackBlock]);
    float v[VEC];
    if constexpr (VEC == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(in.q + row * in.ldq + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? w.x : w.y) >> (8 * (j % 4)))) * sc;
    } else {
      v[0] = static_cast<float>(in.q[row * in.ldq + c]) * sc;
    }
    store_cols<T, VEC>(out, row, c, cols, v);
  }
}

// --------------------------------------------------------------------------
// RMS norm: one CTA a row at a time, the row read twice (the second time from
// cache).  h = x + r; rstd = 1 / sqrt(mean(h^2) + eps); y = h rstd w, from the
// unrounded h.
// --------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void rms_norm_kernel(NormArgs a) {
  __shared__ float red[64];
  int flip = 0;
  const int span = blockDim.x * VEC;
  const int padded = (a.cols + span - 1) / span * span;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.f;
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      float v[VEC], r[VEC];
      load_cols<T, VEC>(a.x, row, c, a.cols, v);
      if (a.residual.p) {
        load_cols<T, VEC>(a.residual, row, c, a.cols, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(v[j], v[j], ss);
    }
    ss = cta_sum(ss, red, flip);
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int c = threadIdx.x * VEC; c < padded; c += span) {
      float v[VEC], r[VEC];
      load_cols<T, VEC>(a.x, row, c, a.cols, v);
      if (a.residual.p) {
        load_cols<T, VEC>(a.residual, row, c, a.cols, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += r[j];
      }
      if (a.h.p) store_cols<T, VEC>(a.h, row, c, a.cols, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = c < a.cols ? v[j] * rstd * load_w(a.w, a.w_dtype, c + j) : 0.f;
      if (a.y.p) store_cols<T, VEC>(a.y, row, c, a.cols, v);
      if (a.y8.q) store_block<VEC>(a.y8, row, c, a.cols, v);
    }
  }
}

// Gradient: hn = h rstd, g = dy w; dx = dh + rstd (g - hn mean(g hn)),
// dw = sum over rows of dy hn.  A CTA takes rows in turn and keeps its column
// sums of dw in shared memory; column_sum_kernel adds the CTAs' sums in order.
template <typename T, int VEC>
__global__ void rms_norm_grad_kernel(NormGradArgs a) {
  extern __shared__ float colsum[];
  __shared__ float red[64];
  int flip = 0;
  const int span = blockDim.x * VEC;
  if (a.dw != nullptr)
    for (int c = threadIdx.x * VEC; c < a.cols; c += span)
#pragma unroll
      for (int j = 0; j < VEC; ++j) colsum[c + j] = 0.f;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float s = 0.f;
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      float dy[VEC], h[VEC];
      load_cols<T, VEC>(a.dy, row, c, a.cols, dy);
      load_cols<T, VEC>(a.h, row, c, a.cols, h);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(__fmul_rn(dy[j], load_w(a.w, a.w_dtype, c + j)), __fmul_rn(h[j], rstd), s);
    }
    s = cta_sum(s, red, flip) / static_cast<float>(a.cols);
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      float dy[VEC], h[VEC], d[VEC];
      load_cols<T, VEC>(a.dy, row, c, a.cols, dy);
      load_cols<T, VEC>(a.h, row, c, a.cols, h);
      if (a.dh.p) load_cols<T, VEC>(a.dh, row, c, a.cols, d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float hn = __fmul_rn(h[j], rstd);
        const float g = fmaf(-hn, s, __fmul_rn(dy[j], load_w(a.w, a.w_dtype, c + j)));
        d[j] = a.dh.p ? fmaf(rstd, g, d[j]) : __fmul_rn(rstd, g);
        if (a.dw != nullptr) colsum[c + j] = fmaf(dy[j], hn, colsum[c + j]);
      }
      store_cols<T, VEC>(a.dx, row, c, a.cols, d);
    }
  }
  if (a.dw != nullptr)
    for (int c = threadIdx.x * VEC; c < a.cols; c += span)
#pragma unroll
      for (int j = 0; j < VEC; ++j) a.partials[static_cast<long long>(blockIdx.x) * a.cols + c + j] = colsum[c + j];
}

// out[c] (+)= sum over p of partials[p][c], in order of p within each of 8
// interleaved chains and of the chains after that: the same bits every call.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partials, int nparts, int cols, float* out,
                                                         int accumulate) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = w; p < nparts; p += 8) s += partials[static_cast<long long>(p) * cols + c];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    s = red[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

// --------------------------------------------------------------------------
// Activation gradient and bias gradient: a CTA takes 32 VEC columns (one warp
// wide) of every 8 gridDim.y-th rows; its 8 warps' column sums meet in shared
// memory and go to one row of the partials.
// --------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void __launch_bounds__(256) act_grad_kernel(ActGradArgs a) {
  __shared__ float red[8][32 * VEC];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = (blockIdx.x * 32 + lane) * VEC;
  float sum[VEC] = {};
  for (long long row = blockIdx.y * 8 + w; row < a.rows; row += gridDim.y * 8) {
    float d[VEC], z[VEC];
    if (c >= a.cols) break;
    load_cols<T, VEC>(a.dy, row, c, a.cols, d);
    if (a.act != kActNone) {
      if (a.z.p) {
        load_cols<T, VEC>(a.z, row, c, a.cols, z);
      } else {
        const float sc = scale_of(a.z8.s[row * a.z8.lds + c / kPackBlock]);
        const int8_t* q = a.z8.q + row * a.z8.ldq + c;
        if constexpr (VEC == 8) {
          const uint2 u = *reinterpret_cast<const uint2*>(q);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            z[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? u.x : u.y) >> (8 * (j % 4)))) * sc;
        } else {
          z[0] = static_cast<float>(*q) * sc;
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] *= act_grad(a.act, z[j]);
    }
    if (a.dz.p) store_cols<T, VEC>(a.dz, row, c, a.cols, d);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] += d[j];
  }
  if (a.db == nullptr) return;
#pragma unroll
  for (int j = 0; j < VEC; ++j) red[w][lane + 32 * j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VEC; i += 256) {
    float s = red[0][i];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][i];
    const int col = (blockIdx.x * 32 + i % 32) * VEC + i / 32;
    if (col < a.cols) a.partials[static_cast<long long>(blockIdx.y) * a.cols + col] = s;
  }
}

__global__ void __launch_bounds__(256) repitch_kernel(int rows, int cols, const uint16_t* src, long long ld_src,
                                                      uint16_t* dst, long long ld_dst) {
  const long long total = static_cast<long long>(rows) * cols;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long r = i / cols;
    const int c = static_cast<int>(i - r * cols);
    dst[r * ld_dst + c] = src[r * ld_src + c];
  }
}

__global__ void __launch_bounds__(256) zero_kernel(int rows, int cols, int elem_bytes, uint8_t* out, long long ld) {
  const long long total = static_cast<long long>(rows) * cols;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long r = i / cols, at = r * ld + (i - r * cols);
    if (elem_bytes == 4)
      reinterpret_cast<uint32_t*>(out)[at] = 0u;
    else
      reinterpret_cast<uint16_t*>(out)[at] = 0u;
  }
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (cached[dev & 63] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev & 63] = n > 0 ? n : 1;
  }
  return cached[dev & 63];
}

// Blocks for `work` items of 256 threads, enough to fill the device.
unsigned flat_grid(long long threads) {
  const long long want = (threads + 255) / 256;
  return static_cast<unsigned>(std::max(1ll, std::min(want, 16ll * sm_count())));
}

// Whether rows of a matrix can be read as vectors of 8 elements.
bool vec_mat(const Mat& m, int elem_bytes) {
  return m.p == nullptr || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (m.ld * elem_bytes) % 16 == 0);
}
bool vec_pack(const Pack8& p) {
  return p.q == nullptr || (reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && p.ldq % 8 == 0);
}
int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

template <typename F>
cudaError_t by_dtype(int dtype, F&& f) {
  if (dtype == kF32) return f(float{});
  if (dtype == kBF16) return f(__nv_bfloat16{});
  return f(__half{});
}

}  // namespace

cudaError_t launch_pack8(int rows, int cols, int dtype, Mat x, Pack8 out, cudaStream_t s) {
  const bool vec = cols % 8 == 0 && vec_mat(x, elem_bytes(dtype)) && vec_pack(out);
  const long long lanes = static_cast<long long>(rows) * ((cols + kPackBlock - 1) / kPackBlock) *
                          (vec ? kPackBlock / 8 : kPackBlock);
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    auto k = vec ? pack8_kernel<T, 8> : pack8_kernel<T, 1>;
    return launch_kernel(false, k, dim3(flat_grid(lanes)), dim3(256), 0, s, rows, cols, x, out);
  });
}

cudaError_t launch_unpack8(int rows, int cols, Pack8 in, int dtype, Mat out, cudaStream_t s) {
  const bool vec = cols % 8 == 0 && vec_mat(out, elem_bytes(dtype)) && vec_pack(in);
  const long long lanes = static_cast<long long>(rows) * (vec ? cols / 8 : cols);
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    auto k = vec ? unpack8_kernel<T, 8> : unpack8_kernel<T, 1>;
    return launch_kernel(false, k, dim3(flat_grid(lanes)), dim3(256), 0, s, rows, cols, in, out);
  });
}

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.x, eb) && vec_mat(a.residual, eb) && vec_mat(a.h, eb) &&
                   vec_mat(a.y, eb) && vec_pack(a.y8);
  const int lanes = vec ? a.cols / 8 : a.cols;
  const int threads = std::min(1024, (lanes + 31) / 32 * 32);
  return by_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto k = vec ? rms_norm_kernel<T, 8> : rms_norm_kernel<T, 1>;
    return launch_kernel(false, k, dim3(std::min(a.rows, 8 * sm_count())), dim3(threads), 0, s, a);
  });
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, eb) && vec_mat(a.h, eb) && vec_mat(a.dh, eb) && vec_mat(a.dx, eb);
  const int lanes = vec ? a.cols / 8 : a.cols;
  const int threads = std::min(1024, (lanes + 31) / 32 * 32);
  const int grid = std::max(1, std::min(a.rows, std::min(kMaxPartials, 4 * sm_count())));
  const size_t smem = a.dw != nullptr ? static_cast<size_t>(a.cols) * 4 : 0;
  cudaError_t e = by_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto k = vec ? rms_norm_grad_kernel<T, 8> : rms_norm_grad_kernel<T, 1>;
    cudaError_t se = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxCols * 4);
    if (se != cudaSuccess) return se;
    return launch_kernel(false, k, dim3(grid), dim3(threads), smem, s, a);
  });
  if (e != cudaSuccess || a.dw == nullptr) return e;
  return launch_kernel(false, column_sum_kernel, dim3((a.cols + 31) / 32), dim3(256), 0, s,
                       static_cast<const float*>(a.partials), grid, a.cols, a.dw, a.accumulate);
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, 2) && vec_mat(a.z, 2) && vec_mat(a.dz, 2) && vec_pack(a.z8);
  const int wide = vec ? 256 : 32;
  const int gx = (a.cols + wide - 1) / wide;
  const int gy = std::max(1, std::min({kMaxPartials, (a.rows + 7) / 8, (8 * sm_count() + gx - 1) / gx}));
  cudaError_t e = by_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    if constexpr (std::is_same<T, float>::value) {
      return cudaErrorInvalidValue;  // 16-bit types only
    } else {
      auto k = vec ? act_grad_kernel<T, 8> : act_grad_kernel<T, 1>;
      return launch_kernel(false, k, dim3(gx, gy), dim3(256), 0, s, a);
    }
  });
  if (e != cudaSuccess || a.db == nullptr) return e;
  return launch_kernel(false, column_sum_kernel, dim3((a.cols + 31) / 32), dim3(256), 0, s,
                       static_cast<const float*>(a.partials), gy, a.cols, a.db, a.accumulate);
}

cudaError_t launch_repitch(int rows, int cols, Mat src, Mat dst, cudaStream_t s) {
  return launch_kernel(false, repitch_kernel, dim3(flat_grid(static_cast<long long>(rows) * cols)), dim3(256), 0, s,
                       rows, cols, static_cast<const uint16_t*>(src.p), src.ld, static_cast<uint16_t*>(dst.p), dst.ld);
}

cudaError_t launch_zero(int rows, int cols, int elem_bytes, Mat out, cudaStream_t s) {
  return launch_kernel(false, zero_kernel, dim3(flat_grid(static_cast<long long>(rows) * cols)), dim3(256), 0, s, rows,
                       cols, elem_bytes, static_cast<uint8_t*>(out.p), out.ld);
}

}  // namespace dion3
