// Memory-bound kernels of the layer operators on sm_103a: 8-bit checkpoints,
// the RMS norm with the residual's addition and its gradient, and the
// activation's gradient with the bias gradient's column sums.
//
// All are launched with programmatic stream serialization like the products:
// a kernel's blocks may be placed while the one before it drains, and read
// nothing before it has completed (pdl_wait).  The calls of a layer's step are
// short chains of small kernels, where that takes a microsecond or two off each.
#include <algorithm>
#include <atomic>
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

// Bits of the largest |v| over the lanes that share a block of 32 columns (VEC
// columns a lane); a NaN is larger than every number.
template <int VEC>
__device__ __forceinline__ uint32_t block_amax(const float (&v)[VEC]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < VEC; ++j) m = max_mag(m, v[j]);
#pragma unroll
  for (int d = 1; d < kPackBlock / VEC; d *= 2) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, d));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Codes (and, from the block's first lane, its scale byte) of VEC columns to q
// (and sb).  Lanes of a warp hold consecutive columns from a multiple of 32;
// `in` is false past the last column, where the values are 0.  amax: the bits
// of the block's largest magnitude.  Called by all lanes of a warp together.
template <int VEC>
__device__ __forceinline__ void store_block(int8_t* q, uint8_t* sb, bool in, bool first, uint32_t amax,
                                            float (&v)[VEC]) {
  const uint32_t byte = scale_byte(amax);
  const float inv = inv_scale(byte);
  if (__any_sync(0xffffffffu, byte == kTopByte)) saturate_block(byte, v);  // skipped by the whole warp
  if (!in) return;
  if constexpr (VEC == 8)
    *reinterpret_cast<uint2*>(q) =
        make_uint2(codes4(v[0], v[1], v[2], v[3], inv), codes4(v[4], v[5], v[6], v[7], inv));
  else
    *q = static_cast<int8_t>(code_of(v[0], inv));
  if (first) *sb = static_cast<uint8_t>(byte);
}
template <int VEC>
__device__ __forceinline__ void store_block(const Pack8& o, long long row, int c, int cols, float (&v)[VEC]) {
  store_block<VEC>(o.q + row * o.ldq + c, o.s + row * o.lds + c / kPackBlock, c < cols, c % kPackBlock == 0,
                   block_amax<VEC>(v), v);
}

// Raw codes and scale byte of VEC columns, and their values.
template <int VEC>
struct Codes {
  uint2 w;
  uint32_t byte;
  __device__ __forceinline__ void load(const int8_t* q, const uint8_t* s, bool in) {
    if (!in) return;
    if constexpr (VEC == 8)
      w = *reinterpret_cast<const uint2*>(q);
    else
      w.x = static_cast<uint32_t>(static_cast<uint8_t>(*q));
    byte = *s;
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) const {
    const float sc = scale_of(byte);
    float a[4];
    values4(w.x, sc, a);
    if constexpr (VEC == 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j];
      values4(w.y, sc, a);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 + j] = a[j];
    } else {
      v[0] = a[0];
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_cols(const Mat& m, long long row, int c, int cols, const float (&v)[VEC]) {
  if (c < cols) store_vec<T, VEC>(static_cast<T*>(m.p) + row * m.ld + c, v);
}
// VEC elements as they lie in memory (loaded ahead of their use), zeros past
// the last column.
template <typename T, int VEC>
struct Raw {
  static constexpr int kWords = VEC == 1 ? 1 : VEC * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const Mat& m, long long row, int c, int cols) {
    load(static_cast<const T*>(m.p) + row * m.ld + c, c < cols);
  }
  __device__ __forceinline__ void load(const T* p, bool in) {
    if (!in) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0u;
      return;
    }
    if constexpr (VEC == 1) {
      if constexpr (sizeof(T) == 2)
        w[0] = *reinterpret_cast<const uint16_t*>(p);
      else
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) const {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(w[j]);
    } else if constexpr (VEC == 1) {
      v[0] = unpack1<kBf>(static_cast<uint16_t>(w[0]));
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 f = unpack2<kBf>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};
// Bits of the block's largest magnitude, from the elements as loaded.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t raw_amax(const Raw<T, VEC>& r) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    uint32_t m = max_mag2<kBf>(max_mag2<kBf>(r.w[0], r.w[1]), max_mag2<kBf>(r.w[2], r.w[3]));
    m = max_mag2<kBf>(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_mag2<kBf>(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float2 f = unpack2<kBf>(m);
    return __float_as_uint(max_mag(f.x, f.y)) & 0x7FFFFFFFu;
  } else {
    float v[VEC];
    r.values(v);
    return block_amax<VEC>(v);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void load_cols(const Mat& m, long long row, int c, int cols, float (&v)[VEC]) {
  Raw<T, VEC> raw;
  raw.load(m, row, c, cols);
  raw.values(v);
}

// Sum over the threads of a row (blockDim.x, a multiple of 32), the same bits in
// every one.  `red` (16-byte aligned) alternates between two halves so one
// barrier a call is enough; every thread adds the warps' sums itself.
__device__ __forceinline__ float cta_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int nw = blockDim.x / 32;
  if (nw == 1) return v;
  float* r = red + 32 * flip;
  flip ^= 1;
  if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < nw; w += 4) {
    const float4 x = *reinterpret_cast<const float4*>(r + w);
    v += x.x + (w + 1 < nw ? x.y : 0.f) + (w + 2 < nw ? x.z : 0.f) + (w + 3 < nw ? x.w : 0.f);
  }
  return v;
}

// --------------------------------------------------------------------------
// 8-bit checkpoints.  Bound by HBM.  blockDim = (lanes along a row, rows): a
// thread keeps its columns and walks the rows kWalk at a time, all their loads
// issued before the first is used.
// --------------------------------------------------------------------------
constexpr int kWalk = 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(256, 4) pack8_kernel(int rows, int cols, Mat x, Pack8 o) {
  pdl_trigger();
  pdl_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
  const int step = gridDim.y * blockDim.y;
  int row = blockIdx.y * blockDim.y + threadIdx.y;
  const T* px = static_cast<const T*>(x.p) + row * x.ld + c;
  int8_t* pq = o.q + row * o.ldq + c;
  uint8_t* ps = o.s + row * o.lds + c / kPackBlock;
  const long long dx = step * x.ld, dq = step * o.ldq, ds = step * o.lds;
  const bool first = c % kPackBlock == 0;
  for (; row < rows; row += kWalk * step) {
    Raw<T, VEC> raw[kWalk];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, px += dx) raw[i].load(px, c < cols && row + i * step < rows);
#pragma unroll
    for (int i = 0; i < kWalk; ++i, pq += dq, ps += ds) {
      float v[VEC];
      raw[i].values(v);
      store_block<VEC>(pq, ps, c < cols && row + i * step < rows, first, raw_amax(raw[i]), v);
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256, 4) unpack8_kernel(int rows, int cols, Pack8 in, Mat out) {
  pdl_trigger();
  pdl_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
  if (c >= cols) return;
  const int step = gridDim.y * blockDim.y;
  int row = blockIdx.y * blockDim.y + threadIdx.y;
  const int8_t* pq = in.q + row * in.ldq + c;
  const uint8_t* ps = in.s + row * in.lds + c / kPackBlock;
  T* po = static_cast<T*>(out.p) + row * out.ld + c;
  const long long dq = step * in.ldq, ds = step * in.lds, dst = step * out.ld;
  for (; row < rows; row += kWalk * step) {
    Codes<VEC> q[kWalk];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, pq += dq, ps += ds) q[i].load(pq, ps, row + i * step < rows);
#pragma unroll
    for (int i = 0; i < kWalk; ++i, po += dst) {
      if (row + i * step >= rows) break;
      float v[VEC];
      q[i].values(v);
      store_vec<T, VEC>(po, v);
    }
  }
}

// --------------------------------------------------------------------------
// RMS norm: h = x + r; rstd = 1 / sqrt(mean(h^2) + eps); y = h rstd w, from the
// unrounded h.  Bound by HBM.  blockDim = (lanes of a row, rows): a thread holds
// NV pieces of VEC columns of its row in registers from the load to the last
// store and loads the next row's pieces before it waits for this row's sum.
// The gain stays in registers over the rows.
// --------------------------------------------------------------------------
constexpr int kRowThreads = 512;  // most of a row kernel's block (128 registers a thread)

template <typename T, int VEC, int NV, bool RES>
__global__ void __launch_bounds__(kRowThreads) rms_norm_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = threadIdx.x * VEC + i * span + j;
      w[i][j] = c < a.cols ? load_w(a.w, a.w_dtype, c) : 0.f;
    }
  Raw<T, VEC> x[NV], r[RES ? NV : 1];
  auto load_row = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = row < a.rows ? static_cast<int>(threadIdx.x) * VEC + i * span : a.cols;
      x[i].load(a.x, row, c, a.cols);
      if constexpr (RES) r[i].load(a.residual, row, c, a.cols);
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  load_row(row);
  for (; row < a.rows; row += step) {
    float v[NV][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i].values(v[i]);
      if constexpr (RES) {
        float t[VEC];
        r[i].values(t);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] += t[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    load_row(row + step);
    ss = cta_sum(ss, red, flip);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x * VEC + i * span;
      if (a.h.p) store_cols<T, VEC>(a.h, row, c, a.cols, v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = c < a.cols ? v[i][j] * rstd * w[i][j] : 0.f;
      if (a.y.p) store_cols<T, VEC>(a.y, row, c, a.cols, v[i]);
      if (a.y8.q) store_block<VEC>(a.y8, row, c, a.cols, v[i]);
    }
  }
}

// The same for rows too wide for that: the row is read twice, the second time
// from cache.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  const int padded = (a.cols + span - 1) / span * span;
  auto load_h = [&](long long row, int c, float (&v)[VEC]) {
    load_cols<T, VEC>(a.x, row, c, a.cols, v);
    if (a.residual.p) {
      float r[VEC];
      load_cols<T, VEC>(a.residual, row, c, a.cols, r);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] += r[j];
    }
  };
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.f, v[VEC];
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      load_h(row, c, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(v[j], v[j], ss);
    }
    ss = cta_sum(ss, red, flip);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int c = threadIdx.x * VEC; c < padded; c += span) {
      load_h(row, c, v);
      if (a.h.p) store_cols<T, VEC>(a.h, row, c, a.cols, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = c < a.cols ? v[j] * rstd * load_w(a.w, a.w_dtype, c + j) : 0.f;
      if (a.y.p) store_cols<T, VEC>(a.y, row, c, a.cols, v);
      if (a.y8.q) store_block<VEC>(a.y8, row, c, a.cols, v);
    }
  }
}

// Gradient: hn = h rstd, g = dy w; dx = dh + rstd (g - hn mean(g hn)), dw = sum
// over rows of dy hn.  Bound by HBM.  As the forward kernel, with dw's column
// sums of the CTA's rows in registers; column_sum_kernel adds the CTAs' sums in
// order.
__device__ __forceinline__ float norm_dx(float dy, float w, float hn, float mean, float rstd, float dh) {
  return fmaf(rstd, fmaf(-hn, mean, __fmul_rn(dy, w)), dh);
}

template <typename T, int VEC, int NV, bool DH>
__global__ void __launch_bounds__(kRowThreads, NV == 1 && sizeof(T) == 2 ? 2 : 1) rms_norm_grad_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  extern __shared__ float rows_sum[];  // [blockDim.y][span * NV], blockDim.y > 1
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  float w[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = threadIdx.x * VEC + i * span + j;
      w[i][j] = c < a.cols ? load_w(a.w, a.w_dtype, c) : 0.f;
      dw[i][j] = 0.f;
    }
  Raw<T, VEC> dy[NV], h[NV], dh[DH ? NV : 1];
  float rstd_next = 0.f;
  auto load_row = [&](long long row) {
    if (row < a.rows) rstd_next = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = row < a.rows ? static_cast<int>(threadIdx.x) * VEC + i * span : a.cols;
      dy[i].load(a.dy, row, c, a.cols);
      h[i].load(a.h, row, c, a.cols);
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  load_row(row);
  for (; row < a.rows; row += step) {
    const float rstd = rstd_next;
    float g[NV][VEC], hn[NV][VEC], s = 0.f;
    if constexpr (DH) {  // not needed before the sum is known
#pragma unroll
      for (int i = 0; i < NV; ++i) dh[i].load(a.dh, row, static_cast<int>(threadIdx.x) * VEC + i * span, a.cols);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i].values(g[i]);
      h[i].values(hn[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        hn[i][j] = __fmul_rn(hn[i][j], rstd);
        dw[i][j] = fmaf(g[i][j], hn[i][j], dw[i][j]);
        s = fmaf(__fmul_rn(g[i][j], w[i][j]), hn[i][j], s);
      }
    }
    load_row(row + step);
    s = cta_sum(s, red, flip) * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[VEC] = {};
      if constexpr (DH) dh[i].values(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = norm_dx(g[i][j], w[i][j], hn[i][j], s, rstd, d[j]);
      store_cols<T, VEC>(a.dx, row, static_cast<int>(threadIdx.x) * VEC + i * span, a.cols, d);
    }
  }
  if (a.dw == nullptr) return;
  // The rows of the block first, in order.
  if (blockDim.y > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) rows_sum[(threadIdx.y * NV + i) * span + threadIdx.x * VEC + j] = dw[i][j];
    __syncthreads();
    if (threadIdx.y > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        for (int y = 1; y < blockDim.y; ++y) dw[i][j] += rows_sum[(y * NV + i) * span + threadIdx.x * VEC + j];
  }
  float* part = a.partials + static_cast<long long>(blockIdx.x) * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x * VEC + i * span;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < a.cols) part[c + j] = dw[i][j];
  }
}

// The same for rows too wide for that: read twice, column sums in shared memory.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) rms_norm_grad_wide_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float colsum[];
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  if (a.dw != nullptr)
    for (int c = threadIdx.x * VEC; c < a.cols; c += span)
#pragma unroll
      for (int j = 0; j < VEC; ++j) colsum[c + j] = 0.f;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float s = 0.f, dy[VEC], h[VEC];
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      load_cols<T, VEC>(a.dy, row, c, a.cols, dy);
      load_cols<T, VEC>(a.h, row, c, a.cols, h);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        s = fmaf(__fmul_rn(dy[j], load_w(a.w, a.w_dtype, c + j)), __fmul_rn(h[j], rstd), s);
    }
    s = cta_sum(s, red, flip) * inv_cols;
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      float d[VEC];
      load_cols<T, VEC>(a.dy, row, c, a.cols, dy);
      load_cols<T, VEC>(a.h, row, c, a.cols, h);
      if (a.dh.p) load_cols<T, VEC>(a.dh, row, c, a.cols, d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float hn = __fmul_rn(h[j], rstd);
        d[j] = norm_dx(dy[j], load_w(a.w, a.w_dtype, c + j), hn, s, rstd, a.dh.p ? d[j] : 0.f);
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

// out[c] (+)= sum over p of partials[p][c], in order of p within each of
// kChains interleaved chains and of the chains after that: the same bits every
// call.
constexpr int kChains = 32;
__global__ void __launch_bounds__(32 * kChains) column_sum_kernel(const float* partials, int nparts, int cols,
                                                                  float* out, int accumulate) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[kChains][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int p = w; p < nparts; p += kChains) s += partials[static_cast<long long>(p) * cols + c];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    s = red[0][lane];
#pragma unroll
    for (int i = 1; i < kChains; ++i) s += red[i][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

// --------------------------------------------------------------------------
// Activation gradient and bias gradient.  Bound by HBM.  A warp takes 32 VEC
// columns and walks the rows kWalk at a time; the 8 warps' column sums of a CTA
// meet in shared memory and go to one row of the partials.
// --------------------------------------------------------------------------
template <typename T, int VEC, int ACT, bool Z8>
__global__ void __launch_bounds__(256, 3) act_grad_kernel(ActGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[8][32 * VEC];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = (blockIdx.x * 32 + lane) * VEC;
  const int step = gridDim.y * 8;
  int row = blockIdx.y * 8 + w;
  const T* py = static_cast<const T*>(a.dy.p) + row * a.dy.ld + c;
  const T* pz = static_cast<const T*>(a.z.p) + row * a.z.ld + c;
  const int8_t* pq = a.z8.q + row * a.z8.ldq + c;
  const uint8_t* ps = a.z8.s + row * a.z8.lds + c / kPackBlock;
  T* pd = static_cast<T*>(a.dz.p) + row * a.dz.ld + c;
  const long long sy = step * a.dy.ld, sz = step * a.z.ld, sq = step * a.z8.ldq, ss = step * a.z8.lds,
                  sd = step * a.dz.ld;
  float sum[VEC] = {};
  for (; row < a.rows && c < a.cols; row += kWalk * step) {
    Raw<T, VEC> dy[kWalk], z[ACT != kActNone && !Z8 ? kWalk : 1];
    Codes<VEC> z8[Z8 ? kWalk : 1];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, py += sy, pz += sz, pq += sq, ps += ss) {
      const bool in = row + i * step < a.rows;
      dy[i].load(py, in);
      if constexpr (ACT != kActNone && Z8)
        z8[i].load(pq, ps, in);
      else if constexpr (ACT != kActNone)
        z[i].load(pz, in);
    }
#pragma unroll
    for (int i = 0; i < kWalk; ++i, pd += sd) {
      if (row + i * step >= a.rows) break;
      float d[VEC];
      dy[i].values(d);
      if constexpr (ACT != kActNone) {
        float t[VEC];
        if constexpr (Z8)
          z8[i].values(t);
        else
          z[i].values(t);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = __fmul_rn(d[j], act_grad<ACT>(t[j]));
      }
      if (a.dz.p) store_vec<T, VEC>(pd, d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] += d[j];
    }
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
    if (col >= a.cols) continue;
    if (gridDim.y > 1)
      a.partials[static_cast<long long>(blockIdx.y) * a.cols + col] = s;
    else
      a.db[col] = a.accumulate ? a.db[col] + s : s;
  }
}

// Copies up to two matrices (blockIdx.z).  One element a lane, neighbouring lanes
// neighbouring elements: source rows may start anywhere.
struct RepitchArgs {
  Repitch job[2];
};
__global__ void __launch_bounds__(256) repitch_kernel(RepitchArgs a) {
  pdl_trigger();
  pdl_wait();
  const Repitch& g = a.job[blockIdx.z];
  const uint16_t* src = static_cast<const uint16_t*>(g.src.p);
  uint16_t* dst = static_cast<uint16_t*>(g.dst.p);
  const long long step = static_cast<long long>(gridDim.y) * blockDim.y;
  constexpr int kCols = 4;
  const int c0 = blockIdx.x * blockDim.x * kCols + threadIdx.x;
  if (c0 >= g.cols) return;
  for (long long row = blockIdx.y * blockDim.y + threadIdx.y; row < g.rows; row += 2 * step) {
    uint16_t v[2][kCols];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + j * blockDim.x;
        if (row + i * step < g.rows && c < g.cols) v[i][j] = src[(row + i * step) * g.src.ld + c];
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + j * blockDim.x;
        if (row + i * step < g.rows && c < g.cols) dst[(row + i * step) * g.dst.ld + c] = v[i][j];
      }
  }
}

__global__ void __launch_bounds__(256) zero_kernel(int rows, int cols, int elem_bytes, uint8_t* out, long long ld) {
  pdl_trigger();
  pdl_wait();
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

// Row kernels: pieces a thread (NV), lanes along a row and rows of a block; at
// most few_threads lanes if that can be.  The gradient does best with 256 (its
// row sum is spread over fewer warps: 16384 x 4096 in 95 us against 114 with
// 512), the forward kernel with as many as there are (100 us against 103).
struct RowShape {
  int nv = 0;  // 0: too wide
  dim3 block;
};
RowShape row_shape(int lanes, int few_threads, int max_threads, int max_nv) {
  RowShape r;
  for (int most : {few_threads, max_threads}) {
    for (int nv = 1; nv <= max_nv; nv *= 2) {
      const int tx = ((lanes + nv - 1) / nv + 31) / 32 * 32;
      if (tx > most) continue;
      r.nv = nv;
      r.block = dim3(tx, tx == 32 ? 4 : 1);
      return r;
    }
  }
  return r;
}
// Blocks of a kernel that the device holds at once (kept per block size).
template <typename K>
int resident(K k, int threads, size_t smem, std::atomic<int>* cache) {
  std::atomic<int>& c = cache[threads / 32];
  int n = c.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, threads, smem) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = 1;
    }
    c.store(n, std::memory_order_relaxed);
  }
  return n * sm_count();
}

// Blocks of 8 warps over rows x lanes: a warp takes 32 lanes of a row, the
// block's warps neighbouring rows, `walk` of them at a time.  One wave: the
// last blocks of a second one would run alone.
const dim3 kWalkBlock(32, 8);
template <typename K>
dim3 walk_grid(K k, int rows, int lanes, int walk, std::atomic<int>* cache) {
  const int gx = (lanes + 31) / 32;
  const int most = (rows + 8 * walk - 1) / (8 * walk);
  return dim3(gx, std::max(1, std::min({most, resident(k, 256, 0, cache) / gx, 65535})));
}

// Calls f with nv as a constant.
template <int MAX, typename F>
cudaError_t by_nv(int nv, F&& f) {
  if constexpr (MAX > 1) {
    if (nv < MAX) return by_nv<MAX / 2>(nv, f);
  }
  return f(std::integral_constant<int, MAX>{});
}
template <typename F>
cudaError_t by_act(int act, F&& f) {
  if (act == kActRelu) return f(std::integral_constant<int, kActRelu>{});
  if (act == kActGelu) return f(std::integral_constant<int, kActGelu>{});
  if (act == kActSilu) return f(std::integral_constant<int, kActSilu>{});
  return f(std::integral_constant<int, kActNone>{});
}

}  // namespace

cudaError_t launch_pack8(int rows, int cols, int dtype, Mat x, Pack8 out, cudaStream_t s) {
  const bool vec = cols % 8 == 0 && vec_mat(x, elem_bytes(dtype)) && vec_pack(out);
  const int lanes = (cols + kPackBlock - 1) / kPackBlock * (vec ? kPackBlock / 8 : kPackBlock);  // whole blocks
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    static std::atomic<int> cache[2][9];
    auto k = vec ? pack8_kernel<T, 8> : pack8_kernel<T, 1>;
    return launch_kernel(pdl_enabled(), k, walk_grid(k, rows, lanes, kWalk, cache[vec]), kWalkBlock, 0, s, rows, cols, x, out);
  });
}

cudaError_t launch_unpack8(int rows, int cols, Pack8 in, int dtype, Mat out, cudaStream_t s) {
  const bool vec = cols % 8 == 0 && vec_mat(out, elem_bytes(dtype)) && vec_pack(in);
  const int lanes = vec ? cols / 8 : cols;
  return by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    static std::atomic<int> cache[2][9];
    auto k = vec ? unpack8_kernel<T, 8> : unpack8_kernel<T, 1>;
    return launch_kernel(pdl_enabled(), k, walk_grid(k, rows, lanes, kWalk, cache[vec]), kWalkBlock, 0, s, rows, cols, in, out);
  });
}

// Columns of a thread in the register kernels: pieces of 8, or single elements
// where pitch, base or width rules vectors out.
template <typename T, int VEC>
constexpr int kMaxPieces = VEC == 8 ? 2 : 8;

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.x, eb) && vec_mat(a.residual, eb) && vec_mat(a.h, eb) &&
                   vec_mat(a.y, eb) && vec_pack(a.y8);
  const int lanes = vec ? a.cols / 8 : a.cols;
  auto run = [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int VEC = decltype(v)::value, MAXV = kMaxPieces<T, VEC>;
    const RowShape r = row_shape(lanes, kRowThreads, kRowThreads, MAXV);
    if (r.nv == 0)
      return launch_kernel(pdl_enabled(), rms_norm_wide_kernel<T, VEC>, dim3(std::min(a.rows, 2 * sm_count())), dim3(1024), 0,
                           s, a);
    return by_nv<MAXV>(r.nv, [&](auto n) {
      constexpr int NV = decltype(n)::value;
      static std::atomic<int> cache[2][kRowThreads / 32 + 1];
      const bool res = a.residual.p != nullptr;
      auto k = res ? rms_norm_kernel<T, VEC, NV, true> : rms_norm_kernel<T, VEC, NV, false>;
      const int threads = r.block.x * r.block.y;
      const long long blocks = (static_cast<long long>(a.rows) + r.block.y - 1) / r.block.y;
      const int grid = static_cast<int>(std::min<long long>(blocks, resident(k, threads, 0, cache[res])));
      return launch_kernel(pdl_enabled(), k, dim3(grid), r.block, 0, s, a);
    });
  };
  return by_dtype(a.dtype, [&](auto t) {
    return vec ? run(t, std::integral_constant<int, 8>{}) : run(t, std::integral_constant<int, 1>{});
  });
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, eb) && vec_mat(a.h, eb) && vec_mat(a.dh, eb) && vec_mat(a.dx, eb);
  const int lanes = vec ? a.cols / 8 : a.cols;
  int parts = 0;  // rows of partial column sums
  auto run = [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int VEC = decltype(v)::value, MAXV = kMaxPieces<T, VEC>;
    const RowShape r = row_shape(lanes, 256, kRowThreads, MAXV);
    if (r.nv == 0) {
      auto k = rms_norm_grad_wide_kernel<T, VEC>;
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxCols * 4);
      if (e != cudaSuccess) return e;
      parts = std::min(a.rows, sm_count());
      return launch_kernel(pdl_enabled(), k, dim3(parts), dim3(1024), a.dw != nullptr ? static_cast<size_t>(a.cols) * 4 : 0, s,
                           a);
    }
    return by_nv<MAXV>(r.nv, [&](auto n) {
      constexpr int NV = decltype(n)::value;
      static std::atomic<int> cache[2][kRowThreads / 32 + 1];
      const bool dh = a.dh.p != nullptr;
      auto k = dh ? rms_norm_grad_kernel<T, VEC, NV, true> : rms_norm_grad_kernel<T, VEC, NV, false>;
      const int ty = r.block.y, threads = r.block.x * ty;
      const size_t smem = ty > 1 ? static_cast<size_t>(threads) * VEC * NV * 4 : 0;
      const long long blocks = (static_cast<long long>(a.rows) + ty - 1) / ty;
      // One row of partials a block, as many at most as the workspace holds.
      parts = static_cast<int>(std::min({blocks, static_cast<long long>(resident(k, threads, smem, cache[dh])),
                                         static_cast<long long>(kMaxPartials)}));
      return launch_kernel(pdl_enabled(), k, dim3(parts), r.block, smem, s, a);
    });
  };
  const cudaError_t e = by_dtype(a.dtype, [&](auto t) {
    return vec ? run(t, std::integral_constant<int, 8>{}) : run(t, std::integral_constant<int, 1>{});
  });
  if (e != cudaSuccess || a.dw == nullptr) return e;
  return launch_kernel(pdl_enabled(), column_sum_kernel, dim3((a.cols + 31) / 32), dim3(32 * kChains), 0, s,
                       static_cast<const float*>(a.partials), parts, a.cols, a.dw, a.accumulate);
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, 2) && vec_mat(a.z, 2) && vec_mat(a.dz, 2) && vec_pack(a.z8);
  int parts = 0;
  const cudaError_t e = by_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    if constexpr (std::is_same<T, float>::value) {
      return cudaErrorInvalidValue;  // 16-bit types only
    } else {
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        auto k = a.z8.q != nullptr ? (vec ? act_grad_kernel<T, 8, ACT, true> : act_grad_kernel<T, 1, ACT, true>)
                                   : (vec ? act_grad_kernel<T, 8, ACT, false> : act_grad_kernel<T, 1, ACT, false>);
        static std::atomic<int> cache[2][2][9];
        dim3 grid = walk_grid(k, a.rows, vec ? a.cols / 8 : a.cols, kWalk, cache[a.z8.q != nullptr][vec]);
        // Few rows: one block a column strip, which writes db itself (a second
        // kernel takes longer than the rows the strip's warps walk instead).
        grid.y = a.db != nullptr && a.rows <= 256 ? 1 : std::min<unsigned>(grid.y, kMaxPartials);
        parts = static_cast<int>(grid.y);
        return launch_kernel(pdl_enabled(), k, grid, dim3(256), 0, s, a);
      });
    }
  });
  if (e != cudaSuccess || a.db == nullptr || parts == 1) return e;
  return launch_kernel(pdl_enabled(), column_sum_kernel, dim3((a.cols + 31) / 32), dim3(32 * kChains), 0, s,
                       static_cast<const float*>(a.partials), parts, a.cols, a.db, a.accumulate);
}

cudaError_t launch_repitch(const Repitch* jobs, int n, cudaStream_t s) {
  static std::atomic<int> cache[9];
  RepitchArgs a{};
  dim3 grid(1, 1, n);
  for (int i = 0; i < n; ++i) {
    a.job[i] = jobs[i];
    const dim3 g = walk_grid(repitch_kernel, jobs[i].rows, (jobs[i].cols + 3) / 4, 2, cache);
    grid.x = std::max(grid.x, g.x);
    grid.y = std::max(grid.y, g.y);
  }
  return launch_kernel(pdl_enabled(), repitch_kernel, grid, kWalkBlock, 0, s, a);
}

cudaError_t launch_zero(int rows, int cols, int elem_bytes, Mat out, cudaStream_t s) {
  return launch_kernel(pdl_enabled(), zero_kernel, dim3(flat_grid(static_cast<long long>(rows) * cols)), dim3(256), 0, s, rows,
                       cols, elem_bytes, static_cast<uint8_t*>(out.p), out.ld);
}

}  // namespace dion3
