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
#include <mutex>
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

// The gain of VEC columns from c, 0 outside the row.
template <int VEC>
__device__ __forceinline__ void load_gain(const void* w, int dtype, int c, int cols, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    if (c + 8 <= cols && ((reinterpret_cast<uintptr_t>(w) | static_cast<uintptr_t>(c)) & 7u) == 0 &&
        (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
      if (dtype == kF32)
        load_vec<float, 8>(static_cast<const float*>(w) + c, v);
      else if (dtype == kBF16)
        load_vec<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16*>(w) + c, v);
      else
        load_vec<__half, 8>(static_cast<const __half*>(w) + c, v);
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = c + j >= 0 && c + j < cols ? load_w(w, dtype, c + j) : 0.f;
}

// --------------------------------------------------------------------------
// Access.  A thread holds VEC consecutive columns: 8, or 1 for fp32 rows that
// are not a multiple of 8 columns or not 16-byte aligned.  16-bit rows of any
// width and alignment are taken 8 columns a thread too (ANY): a thread reads the
// two aligned 16-byte pieces that its columns lie in and shifts, and a warp
// writes its 256 columns through shared memory as consecutive 4-byte words.
// --------------------------------------------------------------------------

// A matrix that is read, and (ANY) the bytes that its rows span: 16-byte pieces
// inside it may be read whole, whatever columns they hold.
template <typename T, bool ANY>
struct Reader {
  const T* p;
  long long ld;
  uintptr_t lo = 0, hi = 0;
  __device__ __forceinline__ Reader(const Mat& m, int rows, int cols) : p(static_cast<const T*>(m.p)), ld(m.ld) {
    if constexpr (ANY) {
      lo = reinterpret_cast<uintptr_t>(p);
      hi = lo + ((static_cast<long long>(rows) - 1) * ld + cols) * sizeof(T);
    }
  }
  __device__ __forceinline__ const T* at(long long row, int c) const { return p + row * ld + c; }
};

// VEC elements as they lie in memory, loaded ahead of their use.
template <typename T, int VEC, bool ANY>
struct Raw {
  static constexpr int kWords = VEC == 1 ? 1 : (ANY ? 2 : 1) * VEC * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  uint32_t meta;  // ANY: elements to shift by, and columns inside the row << 8
  // p: the element at column c of the row; `in` false or c past the end: zeros.
  __device__ __forceinline__ void load(const Reader<T, ANY>& r, const T* p, int c, int cols, bool in) {
    if (!in || c >= cols) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0u;
      meta = 0u;
      return;
    }
    if constexpr (ANY) {
      static_assert(VEC == 8 && sizeof(T) == 2, "16-bit types, 8 columns");
      const uintptr_t at = reinterpret_cast<uintptr_t>(p), lo = at & ~static_cast<uintptr_t>(15);
      const uint32_t n = static_cast<uint32_t>(min(8, cols - c));
      if (lo >= r.lo && lo + 32 <= r.hi) {
        const uint4 u = reinterpret_cast<const uint4*>(lo)[0], v = reinterpret_cast<const uint4*>(lo)[1];
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
        meta = static_cast<uint32_t>(at & 15) / 2 | n << 8;
      } else {  // the first or last columns of the whole matrix
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(q[2 * i + 1]) << 16 : 0u);
        w[4] = w[5] = w[6] = w[7] = 0u;
        meta = n << 8;
      }
    } else if constexpr (VEC == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void load(const Reader<T, ANY>& r, long long row, int c, int cols, bool in = true) {
    load(r, r.at(row, c), c, cols, in);
  }
  // ANY: the elements in the first four words, zeros past the end of the row.
  __device__ __forceinline__ void align() {
    if constexpr (ANY) {
      const uint32_t n = meta >> 8;
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = meta & 4 ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = meta & 2 ? w[i + 1] : w[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = meta & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
      if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xFFFFu : 0u;
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) {
    align();
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(w[j]);
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
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void load_cols(const Reader<T, ANY>& r, long long row, int c, int cols, float (&v)[VEC]) {
  Raw<T, VEC, ANY> raw;
  raw.load(r, row, c, cols);
  raw.values(v);
}

// Writes VEC columns from p (the element at column c; nothing past the end of
// the row).  ANY: called by all lanes of a warp, which hold consecutive columns
// of one row; buf is the warp's 33 pieces of shared memory.
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void store_cols(T* p, int c, int cols, const float (&v)[VEC], uint4* buf) {
  if constexpr (!ANY) {
    if (c < cols) store_vec<T, VEC>(p, v);
  } else {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    const int lane = threadIdx.x % 32;
    const int n = min(256, cols - (c - 8 * lane));  // columns of the warp
    uint16_t* out = reinterpret_cast<uint16_t*>(p) - 8 * lane;
    __syncwarp();
    buf[lane] = make_uint4(pack2<kBf>(v[0], v[1]), pack2<kBf>(v[2], v[3]), pack2<kBf>(v[4], v[5]),
                           pack2<kBf>(v[6], v[7]));
    __syncwarp();
    const uint32_t* w = reinterpret_cast<const uint32_t*>(buf);
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(out) >> 1) & 1;  // the same in every lane
    if (odd && lane == 0 && n > 0) out[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 32 * j + lane, e = 2 * i + odd;
      const uint32_t x = odd ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];  // w[128] is beyond the row's data
      if (e + 1 < n)
        *reinterpret_cast<uint32_t*>(out + e) = x;
      else if (e < n)
        out[e] = static_cast<uint16_t>(x);
    }
  }
}
// Its shared memory.
template <bool ANY, int WARPS>
struct StoreBuf {
  uint4 piece[ANY ? WARPS : 1][33];
  __device__ __forceinline__ uint4* mine() {
    return ANY ? piece[(threadIdx.y * blockDim.x + threadIdx.x) / 32] : piece[0];
  }
};

// --------------------------------------------------------------------------
// 8-bit blocks
// --------------------------------------------------------------------------

// Bits of the largest |v| over the lanes that share a block of 32 columns (VEC
// columns a lane); a NaN is larger than every number.
template <int VEC>
__device__ __forceinline__ uint32_t block_amax(const float (&v)[VEC]) {
  if constexpr (VEC == 1) return __reduce_max_sync(0xffffffffu, __float_as_uint(v[0]) & 0x7FFFFFFFu);
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < VEC; ++j) m = max_mag(m, v[j]);
#pragma unroll
  for (int d = 1; d < kPackBlock / VEC; d *= 2) m = max_mag(m, __shfl_xor_sync(0xffffffffu, m, d));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}
// The same from 16-bit elements as loaded (and aligned).
template <bool BF16>
__device__ __forceinline__ uint32_t block_amax16(const uint32_t* w) {
  uint32_t m = max_mag2<BF16>(max_mag2<BF16>(w[0], w[1]), max_mag2<BF16>(w[2], w[3]));
  m = max_mag2<BF16>(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_mag2<BF16>(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float2 f = unpack2<BF16>(m);
  return __float_as_uint(max_mag(f.x, f.y)) & 0x7FFFFFFFu;
}

// Codes (and, from the block's first lane, its scale byte) of VEC columns from
// column c to q (and sb).  Lanes of a warp hold consecutive columns from a
// multiple of 32; n: how many of the thread's columns are in the row (the values
// of the others are 0).  amax: the bits of the block's largest magnitude.
// Without ANY eight codes are one aligned piece; with it `aligned` says whether
// they are where the row has them all.  Called by all lanes of a warp together.
template <int VEC, bool ANY>
__device__ __forceinline__ void store_block(int8_t* q, uint8_t* sb, int n, bool first, bool aligned, uint32_t amax,
                                            float (&v)[VEC]) {
  const uint32_t byte = scale_byte(amax);
  const float inv = inv_scale(byte);
  if (__any_sync(0xffffffffu, byte == kTopByte)) saturate_block(byte, v);  // skipped by the whole warp
  if (n <= 0) return;
  if constexpr (VEC == 8) {
    const uint32_t w[2] = {codes4(v[0], v[1], v[2], v[3], inv), codes4(v[4], v[5], v[6], v[7], inv)};
    if (!ANY || (aligned && n >= 8)) {
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)));
    }
  } else {
    *q = static_cast<int8_t>(code_of(v[0], inv));
  }
  if (first) *sb = static_cast<uint8_t>(byte);
}
__device__ __forceinline__ bool codes_aligned(const Pack8& p) {
  return ((reinterpret_cast<uintptr_t>(p.q) | static_cast<uintptr_t>(p.ldq)) & 7u) == 0;
}
template <int VEC, bool ANY>
__device__ __forceinline__ void store_block(const Pack8& o, long long row, int c, int cols, bool aligned,
                                            float (&v)[VEC]) {
  store_block<VEC, ANY>(o.q + row * o.ldq + c, o.s + row * o.lds + c / kPackBlock, cols - c, c % kPackBlock == 0, aligned,
                   block_amax<VEC>(v), v);
}

// Raw codes and scale byte of VEC columns, and their values.
template <int VEC, bool ANY>
struct Codes {
  uint2 w;
  uint32_t byte;
  // n: columns in the row from this one; ANY and `aligned` as for store_block.
  __device__ __forceinline__ void load(const int8_t* q, const uint8_t* s, int n, bool aligned) {
    if (n <= 0) return;
    if constexpr (VEC == 1) {
      w.x = static_cast<uint8_t>(*q);
    } else if (!ANY || (aligned && n >= 8)) {
      w = *reinterpret_cast<const uint2*>(q);
    } else {
      w = make_uint2(0u, 0u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = j < n ? static_cast<uint8_t>(q[j]) : 0u;
        (j < 4 ? w.x : w.y) |= x << (8 * (j % 4));
      }
    }
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

// Sum over the threads of a row (blockDim.x, a multiple of 32), the same bits in
// every one.  `red` (16-byte aligned) alternates between two halves so one
// barrier a call is enough; every thread adds the warps' sums itself.  ROWS: the
// rows of a block (threadIdx.y) wait for their own threads alone, at barriers of
// their own (of which an SM has few: only where few blocks are wanted).
template <bool ROWS = false>
__device__ __forceinline__ float cta_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int nw = blockDim.x / 32;
  if (nw == 1) return v;
  float* r = red + 32 * flip + (ROWS ? threadIdx.y * ((nw + 3) / 4 * 4) : 0);
  flip ^= 1;
  if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = v;
  if constexpr (ROWS)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
  else
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
// issued before the first is used.  16384 x 11008 bf16: 94 us written (5.8 TB/s),
// 89 us read back (6.1 TB/s).
// --------------------------------------------------------------------------
constexpr int kWalk = 4;

template <typename T, int VEC, bool ANY>
__global__ void __launch_bounds__(256, ANY ? 3 : 4) pack8_kernel(int rows, int cols, Mat x, Pack8 o) {
  pdl_trigger();
  pdl_wait();
  const Reader<T, ANY> rx(x, rows, cols);
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
  const int step = gridDim.y * blockDim.y;
  int row = blockIdx.y * blockDim.y + threadIdx.y;
  const T* px = rx.at(row, c);
  int8_t* pq = o.q + row * o.ldq + c;
  uint8_t* ps = o.s + row * o.lds + c / kPackBlock;
  const long long dx = step * x.ld, dq = step * o.ldq, ds = step * o.lds;
  const bool first = c % kPackBlock == 0, aligned = codes_aligned(o);
  for (; row < rows; row += kWalk * step) {
    Raw<T, VEC, ANY> raw[kWalk];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, px += dx) raw[i].load(rx, px, c, cols, row + i * step < rows);
#pragma unroll
    for (int i = 0; i < kWalk; ++i, pq += dq, ps += ds) {
      float v[VEC];
      raw[i].values(v);
      uint32_t amax;
      if constexpr (sizeof(T) == 2)
        amax = block_amax16<std::is_same<T, __nv_bfloat16>::value>(raw[i].w);
      else
        amax = block_amax<VEC>(v);
      store_block<VEC, ANY>(pq, ps, row + i * step < rows ? cols - c : 0, first, aligned, amax, v);
    }
  }
}

// Blocks of 8 warps in x strips of 32 VEC columns, y deep in rows.
template <typename T, int VEC, bool ANY, bool ANY_CODES>
__device__ __forceinline__ void unpack_rows(int rows, int cols, const Pack8& in, const Mat& out, int x, int y, int ny,
                                            uint4* buf) {
  const int c = (x * 32 + threadIdx.x % 32) * VEC;
  const int step = ny * 8;
  int row = y * 8 + (threadIdx.y * blockDim.x + threadIdx.x) / 32;
  const int8_t* pq = in.q + row * in.ldq + c;
  const uint8_t* ps = in.s + row * in.lds + c / kPackBlock;
  T* po = static_cast<T*>(out.p) + row * out.ld + c;
  const long long dq = step * in.ldq, ds = step * in.lds, dst = step * out.ld;
  const bool aligned = codes_aligned(in);
  for (; row < rows; row += kWalk * step) {
    Codes<VEC, ANY_CODES> q[kWalk];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, pq += dq, ps += ds)
      q[i].load(pq, ps, row + i * step < rows ? cols - c : 0, aligned);
#pragma unroll
    for (int i = 0; i < kWalk; ++i, po += dst) {
      if (row + i * step >= rows) break;
      float v[VEC];
      q[i].values(v);
      store_cols<T, VEC, ANY>(po, c, cols, v, buf);
    }
  }
}
template <typename T, int VEC, bool ANY>
__global__ void __launch_bounds__(256, 4) unpack8_kernel(int rows, int cols, Pack8 in, Mat out) {
  pdl_trigger();
  pdl_wait();
  __shared__ StoreBuf<ANY, 8> sbuf;
  unpack_rows<T, VEC, ANY, ANY>(rows, cols, in, out, blockIdx.x, blockIdx.y, gridDim.y, sbuf.mine());
}

// --------------------------------------------------------------------------
// RMS norm: h = x + r; rstd = 1 / sqrt(mean(h^2) + eps); y = h rstd w, from the
// unrounded h.  Bound by HBM.  blockDim = (lanes of a row, rows): a thread holds
// NV pieces of VEC columns of its row in registers from the load to the last
// store and loads the next row's pieces before it waits for this row's sum.
// The gain stays in registers over the rows.  16384 x 4096 bf16 with residual
// and blocks: 100 us, 6.1 TB/s.
// --------------------------------------------------------------------------
constexpr int kRowThreads = 512;  // most of a row kernel's block (128 registers a thread)

template <typename T, int VEC, bool ANY, int NV, bool RES>
__global__ void __launch_bounds__(kRowThreads) rms_norm_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  // Where registers are short (twice the words a piece), the gain is read again
  // for each row and the next row's pieces after this one.
  constexpr bool kAhead = !(ANY && NV > 1);
  float w[kAhead ? NV : 1][VEC];
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load_gain<VEC>(a.w, a.w_dtype, threadIdx.x * VEC + i * span, a.cols, w[i]);
  }
  __shared__ StoreBuf<ANY, kRowThreads / 32> sbuf;
  const Reader<T, ANY> rx(a.x, a.rows, a.cols), rr(a.residual, a.rows, a.cols);
  const bool aligned = codes_aligned(a.y8);
  Raw<T, VEC, ANY> x[NV], r[RES ? NV : 1];
  auto load_row = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = static_cast<int>(threadIdx.x) * VEC + i * span;
      x[i].load(rx, row, c, a.cols, row < a.rows);
      if constexpr (RES) r[i].load(rr, row, c, a.cols, row < a.rows);
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
    if constexpr (kAhead) load_row(row + step);
    ss = cta_sum(ss, red, flip);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x * VEC + i * span;
      if (a.h.p)
        store_cols<T, VEC, ANY>(static_cast<T*>(a.h.p) + row * a.h.ld + c, c, a.cols, v[i], sbuf.mine());
      float (&g)[VEC] = w[kAhead ? i : 0];
      if constexpr (!kAhead) load_gain<VEC>(a.w, a.w_dtype, c, a.cols, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = c + j < a.cols ? v[i][j] * rstd * g[j] : 0.f;
      if (a.y.p)
        store_cols<T, VEC, ANY>(static_cast<T*>(a.y.p) + row * a.y.ld + c, c, a.cols, v[i], sbuf.mine());
      if (a.y8.q) store_block<VEC, ANY>(a.y8, row, c, a.cols, aligned, v[i]);
    }
    if constexpr (!kAhead) load_row(row + step);
  }
}

// The same for rows too wide for that: the row is read twice, the second time
// from cache.
template <typename T, int VEC, bool ANY>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(NormArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  const int padded = (a.cols + span - 1) / span * span;
  __shared__ StoreBuf<ANY, 32> sbuf;
  const Reader<T, ANY> rx(a.x, a.rows, a.cols), rr(a.residual, a.rows, a.cols);
  const bool aligned = codes_aligned(a.y8);
  auto load_h = [&](long long row, int c, float (&v)[VEC]) {
    load_cols<T, VEC, ANY>(rx, row, c, a.cols, v);
    if (a.residual.p) {
      float r[VEC];
      load_cols<T, VEC, ANY>(rr, row, c, a.cols, r);
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
      if (a.h.p) store_cols<T, VEC, ANY>(static_cast<T*>(a.h.p) + row * a.h.ld + c, c, a.cols, v, sbuf.mine());
      float g[VEC];
      load_gain<VEC>(a.w, a.w_dtype, c, a.cols, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = c + j < a.cols ? v[j] * rstd * g[j] : 0.f;
      if (a.y.p) store_cols<T, VEC, ANY>(static_cast<T*>(a.y.p) + row * a.y.ld + c, c, a.cols, v, sbuf.mine());
      if (a.y8.q) store_block<VEC, ANY>(a.y8, row, c, a.cols, aligned, v);
    }
  }
}

// Gradient: hn = h rstd, g = dy w; dx = dh + rstd (g - hn mean(g hn)), dw = sum
// over rows of dy hn.  Bound by HBM.  As the forward kernel, with dw's column
// sums of the CTA's rows in registers; column_sum_kernel adds the CTAs' sums in
// order.  16384 x 4096 bf16 with dh: 91 us, 5.9 TB/s.
__device__ __forceinline__ float norm_dx(float g, float hn, float mean, float rstd, float dh) {
  return fmaf(rstd, fmaf(-hn, mean, g), dh);
}

// dw of a strip of columns over all rows, by a block: it does not need the rows'
// sums, so that few rows' dw comes from blocks beside those of dx, which read the
// rows once more (from L2), and not from a second launch.
constexpr int kStripLanes = 8;  // of VEC = 8; a warp's lanes for single columns
template <int VEC>
__host__ __device__ constexpr int strip_cols() {
  return VEC == 8 ? 8 * kStripLanes : 32;
}
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void strip_dw(const NormGradArgs& a, const Reader<T, ANY>& ry, const Reader<T, ANY>& rh,
                                         int strip, float* sums) {
  constexpr int kCols = strip_cols<VEC>(), kLanes = kCols / VEC, kRows = 4;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, groups = blockDim.x * blockDim.y / kLanes;
  const int c = strip * kCols + tid % kLanes * VEC;
  float dw[VEC] = {};
  for (int row = tid / kLanes; row < a.rows; row += kRows * groups) {
    Raw<T, VEC, ANY> dy[kRows], h[kRows];
    float rstd[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row + i * groups;
      dy[i].load(ry, r, c, a.cols, r < a.rows);
      h[i].load(rh, r, c, a.cols, r < a.rows);
      rstd[i] = r < a.rows ? a.rstd[r] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float g[VEC], hn[VEC];
      dy[i].values(g);
      h[i].values(hn);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dw[j] = fmaf(g[j], __fmul_rn(hn[j], rstd[i]), dw[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) sums[tid * VEC + j] = dw[j];
  __syncthreads();
  const int col = strip * kCols + tid;
  if (tid >= kCols || col >= a.cols) return;
  float v = 0.f;
  for (int k = 0; k < groups; ++k) v += sums[k * kCols + tid];
  a.dw[col] = a.accumulate ? a.dw[col] + v : v;
}

template <typename T, int VEC, bool ANY, int NV, bool DH>
__global__ void __launch_bounds__(kRowThreads, NV == 1 && sizeof(T) == 2 && !ANY ? 2 : 1)
    rms_norm_grad_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  extern __shared__ float rows_sum[];  // [blockDim.y][span * NV], blockDim.y > 1, or a strip's
  const Reader<T, ANY> ry(a.dy, a.rows, a.cols), rh(a.h, a.rows, a.cols), rd(a.dh, a.rows, a.cols);
  if (static_cast<int>(blockIdx.x) < a.strips) {
    strip_dw<T, VEC, ANY>(a, ry, rh, blockIdx.x, rows_sum);
    return;
  }
  const int block = blockIdx.x - a.strips;
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * VEC;
  constexpr bool kAhead = !(ANY && NV > 1);  // as in the forward kernel
  float w[kAhead ? NV : 1][VEC], dw[NV][VEC] = {};
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < NV; ++i) load_gain<VEC>(a.w, a.w_dtype, threadIdx.x * VEC + i * span, a.cols, w[i]);
  }
  __shared__ StoreBuf<ANY, kRowThreads / 32> sbuf;
  Raw<T, VEC, ANY> dy[NV], h[NV], dh[DH ? NV : 1];
  float rstd_next = 0.f;
  auto load_row = [&](long long row) {
    if (row < a.rows) rstd_next = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = static_cast<int>(threadIdx.x) * VEC + i * span;
      dy[i].load(ry, row, c, a.cols, row < a.rows);
      h[i].load(rh, row, c, a.cols, row < a.rows);
    }
  };
  const long long step = static_cast<long long>(gridDim.x - a.strips) * blockDim.y;
  long long row = static_cast<long long>(block) * blockDim.y + threadIdx.y;
  load_row(row);
  for (; row < a.rows; row += step) {
    const float rstd = rstd_next;
    float g[NV][VEC], hn[NV][VEC], s = 0.f;
    if constexpr (DH) {  // not needed before the sum is known
#pragma unroll
      for (int i = 0; i < NV; ++i) dh[i].load(rd, row, static_cast<int>(threadIdx.x) * VEC + i * span, a.cols);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i].values(g[i]);
      h[i].values(hn[i]);
      float (&gain)[VEC] = w[kAhead ? i : 0];
      if constexpr (!kAhead) load_gain<VEC>(a.w, a.w_dtype, threadIdx.x * VEC + i * span, a.cols, gain);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        hn[i][j] = __fmul_rn(hn[i][j], rstd);
        dw[i][j] = fmaf(g[i][j], hn[i][j], dw[i][j]);
        g[i][j] = __fmul_rn(g[i][j], gain[j]);
        s = fmaf(g[i][j], hn[i][j], s);
      }
    }
    if constexpr (kAhead) load_row(row + step);
    s = cta_sum<true>(s, red, flip) * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d[VEC] = {};
      if constexpr (DH) dh[i].values(d);
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[j] = norm_dx(g[i][j], hn[i][j], s, rstd, d[j]);
      const int c = static_cast<int>(threadIdx.x) * VEC + i * span;
      store_cols<T, VEC, ANY>(static_cast<T*>(a.dx.p) + row * a.dx.ld + c, c, a.cols, d, sbuf.mine());
    }
    if constexpr (!kAhead) load_row(row + step);
  }
  if (a.dw == nullptr || a.strips > 0) return;
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
  float* part = a.partials + static_cast<long long>(block) * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x * VEC + i * span;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < a.cols) part[c + j] = dw[i][j];
  }
}

// --------------------------------------------------------------------------
// Norms of rows through shared memory: rows are copied ahead of their use, as the
// aligned 16-byte pieces of memory that they lie in, so that registers hold no
// row but the block's own.  A thread holds columns 8 t - lead and the seven after
// it, where lead is what the rows begin after a 16-byte boundary: whole pieces of
// memory, of which only a row's first and last are taken element by element.  All
// matrices have to be misaligned alike (tensors of one shape are), and a block's
// rows are a multiple of 8 apart, which keeps its lead the same.  bf16, against
// the shifted access of the kernels above: 16384 x 4095 with residual 97 us for
// 161, 12000 x 11007 193 for 387; gradient of 6568 x 4353 52 for 107, of 12000 x
// 11007 216 for 734.  The gradient is held up by its instructions and barriers
// (62 % of the issue slots used): two pieces a thread do better than one (9000 x
// 2041 35 us for 41, the norm itself 21 for 25) and than four (47), at 96 registers,
// with which two blocks of up to 320 threads share an SM (6568 x 4353 52 us; 67 at
// 118).
// --------------------------------------------------------------------------
__device__ __forceinline__ void copy_piece(uint4* dst, uintptr_t src, int bytes) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `behind` (0 to 2) of the thread's groups are unfinished.
__device__ __forceinline__ void copies_wait(int behind) {
  if (behind == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (behind == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// Rows of up to three matrices in a ring of `depth` (2 to 4) in shared memory.
template <typename T, int MATS>
struct Staged {
  uintptr_t base[MATS];
  long long step[MATS];  // bytes from a row of the block to the next
  uintptr_t next[MATS];  // the next row to copy
  long long ahead;       // its number
  int rows, bytes, depth, pitch, to = 0, from = 0;
  uint4* ring;  // [depth][MATS][pitch]
  __device__ __forceinline__ Staged(uint4* ring_, int depth_, int pitch_, int rows_, int cols)
      : ahead(blockIdx.x), rows(rows_), bytes(cols * static_cast<int>(sizeof(T))), depth(depth_), pitch(pitch_),
        ring(ring_) {}
  __device__ __forceinline__ void add(int k, const Mat& m) {
    base[k] = reinterpret_cast<uintptr_t>(m.p);
    next[k] = base[k] + blockIdx.x * m.ld * static_cast<long long>(sizeof(T));
    step[k] = gridDim.x * m.ld * static_cast<long long>(sizeof(T));
  }
  // Begins the copy of the block's next row; nothing outside the matrix is read.
  __device__ __forceinline__ void copy() {
    if (ahead < rows) {
#pragma unroll
      for (int k = 0; k < MATS; ++k) {
        uint4* dst = ring + (to * MATS + k) * pitch;
        const int lead = static_cast<int>(next[k] & 15u), all = lead + bytes;
        const uintptr_t lo = next[k] - lead;
        // Past the row's last element is another row, but for the last row.
        const int end = ahead + 1 < rows ? (all + 15) / 16 * 16 : all;
        for (int o = static_cast<int>(threadIdx.x) * 16; o < all; o += static_cast<int>(blockDim.x) * 16) {
          if (lo + o >= base[k]) {
            copy_piece(dst + o / 16, lo + o, min(16, end - o));
          } else {  // the first row of an unaligned matrix
            for (int j = lead; j < 16 && j < all; j += sizeof(T))
              reinterpret_cast<T*>(dst)[j / sizeof(T)] = *reinterpret_cast<const T*>(lo + j);
          }
        }
        next[k] += step[k];
      }
    }
    copies_commit();
    ahead += gridDim.x;
    to = to + 1 == depth ? 0 : to + 1;
  }
  __device__ __forceinline__ void begin() {
    for (int i = 1; i < depth; ++i) copy();
  }
  // Waits for the block's next row, frees the one before it and copies ahead.
  __device__ __forceinline__ const uint4* row() {
    copies_wait(depth - 2);
    __syncthreads();
    copy();
    const uint4* r = ring + from * MATS * pitch;
    from = from + 1 == depth ? 0 : from + 1;
    return r;
  }
};
// The eight columns from c of a copied row, zeros outside it (without EDGE: the
// row begins on a boundary and is a multiple of 8 columns long).
template <typename T, bool EDGE>
__device__ __forceinline__ void staged_cols(const uint4* row, int c, int lead, int cols, float (&v)[8]) {
  Raw<T, 8, false> raw;
  const uint4* p = row + (c + lead) * static_cast<int>(sizeof(T)) / 16;
#pragma unroll
  for (int i = 0; i < Raw<T, 8, false>::kWords / 4; ++i) {
    const uint4 u = c < cols ? p[i] : make_uint4(0u, 0u, 0u, 0u);
    raw.w[4 * i] = u.x, raw.w[4 * i + 1] = u.y, raw.w[4 * i + 2] = u.z, raw.w[4 * i + 3] = u.w;
  }
  raw.values(v);
  if (!EDGE || (c >= 0 && c + 8 <= cols)) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < 0 || c + j >= cols) v[j] = 0.f;
}
template <typename T, bool EDGE>
__device__ __forceinline__ void store_staged(const Mat& m, long long row, int c, int cols, const float (&v)[8]) {
  T* p = static_cast<T*>(m.p) + row * m.ld + c;
  if (c >= 0 && c + 8 <= cols) {
    store_vec<T, 8>(p, v);
    return;
  }
  if (!EDGE) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < cols) p[j] = from_f32<T>(v[j]);
}
// Elements between a 16-byte boundary and the block's rows.
template <typename T>
__device__ __forceinline__ int lead_of(const Mat& m) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(m.p) + blockIdx.x * m.ld) % 16 / sizeof(T));
}

template <typename T, int NV, bool RES>
__global__ void __launch_bounds__(kRowThreads) rms_norm_staged_kernel(const __grid_constant__ NormArgs a, int depth,
                                                                      int pitch) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  extern __shared__ uint4 ring[];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * 8, lead = lead_of<T>(a.x), first = static_cast<int>(threadIdx.x) * 8 - lead;
  Staged<T, 1 + RES> rows(ring, depth, pitch, a.rows, a.cols);
  rows.add(0, a.x);
  if constexpr (RES) rows.add(1, a.residual);
  rows.begin();
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_gain<8>(a.w, a.w_dtype, first + i * span, a.cols, w[i]);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint4* st = rows.row();
    float v[NV][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * span;
      staged_cols<T, true>(st, c, lead, a.cols, v[i]);
      if constexpr (RES) {
        float t[8];
        staged_cols<T, true>(st + pitch, c, lead, a.cols, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += t[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    ss = cta_sum(ss, red, flip);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * span;
      if (a.h.p) store_staged<T, true>(a.h, row, c, a.cols, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[i][j];
      if (a.y.p) store_staged<T, true>(a.y, row, c, a.cols, v[i]);
    }
  }
  copies_wait(0);
}

template <typename T, bool EDGE, int NV, bool DH>
__global__ void __maxnreg__(NV == 2 ? 96 : 128) rms_norm_grad_staged_kernel(const __grid_constant__ NormGradArgs a,
                                                                           int depth, int pitch) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) float red[64];
  extern __shared__ uint4 ring[];
  constexpr bool kKeep = NV <= 2;  // the row's values stay in registers until its sum is known
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  const int span = blockDim.x * 8, lead = EDGE ? lead_of<T>(a.h) : 0, first = static_cast<int>(threadIdx.x) * 8 - lead;
  Staged<T, 2 + DH> rows(ring, depth, pitch, a.rows, a.cols);
  rows.add(0, a.dy);
  rows.add(1, a.h);
  if constexpr (DH) rows.add(2, a.dh);
  rows.begin();
  float w[NV][8], dw[NV][8] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) load_gain<8>(a.w, a.w_dtype, first + i * span, a.cols, w[i]);
  float rstd_next = a.rstd[blockIdx.x];
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = rstd_next;
    if (row + gridDim.x < a.rows) rstd_next = a.rstd[row + gridDim.x];
    const uint4* st = rows.row();
    float g[kKeep ? NV : 1][8], hn[kKeep ? NV : 1][8], s = 0.f;
    auto load = [&](int i, float (&gi)[8], float (&hi)[8]) {
      const int c = first + i * span;
      staged_cols<T, EDGE>(st, c, lead, a.cols, gi);
      staged_cols<T, EDGE>(st + pitch, c, lead, a.cols, hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) hi[j] = __fmul_rn(hi[j], rstd);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&gi)[8] = g[kKeep ? i : 0], (&hi)[8] = hn[kKeep ? i : 0];
      load(i, gi, hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] = fmaf(gi[j], hi[j], dw[i][j]);
        gi[j] = __fmul_rn(gi[j], w[i][j]);
        s = fmaf(gi[j], hi[j], s);
      }
    }
    s = cta_sum(s, red, flip) * inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * span;
      float (&gi)[8] = g[kKeep ? i : 0], (&hi)[8] = hn[kKeep ? i : 0], d[8] = {};
      if constexpr (!kKeep) {
        load(i, gi, hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) gi[j] = __fmul_rn(gi[j], w[i][j]);
      }
      if constexpr (DH) staged_cols<T, EDGE>(st + 2 * pitch, c, lead, a.cols, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = norm_dx(gi[j], hi[j], s, rstd, d[j]);
      store_staged<T, EDGE>(a.dx, row, c, a.cols, d);
    }
  }
  copies_wait(0);
  if (a.dw == nullptr) return;
  float* part = a.partials + static_cast<long long>(blockIdx.x) * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * span;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j >= 0 && c + j < a.cols) part[c + j] = dw[i][j];
  }
}

// The same for rows too wide for that: read twice, column sums in shared memory.
template <typename T, int VEC, bool ANY>
__global__ void __launch_bounds__(1024) rms_norm_grad_wide_kernel(NormGradArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float colsum[];
  __shared__ __align__(16) float red[64];
  int flip = 0;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  __shared__ StoreBuf<ANY, 32> sbuf;
  const Reader<T, ANY> ry(a.dy, a.rows, a.cols), rh(a.h, a.rows, a.cols), rd(a.dh, a.rows, a.cols);
  const int span = blockDim.x * VEC;
  const int padded = (a.cols + span - 1) / span * span;
  // A thread's own slots: the words of a piece blockDim.x apart.
  if (a.dw != nullptr)
    for (int c = threadIdx.x; c < padded; c += blockDim.x) colsum[c] = 0.f;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float s = 0.f, dy[VEC], h[VEC], w[VEC];
    for (int c = threadIdx.x * VEC; c < a.cols; c += span) {
      load_cols<T, VEC, ANY>(ry, row, c, a.cols, dy);
      load_cols<T, VEC, ANY>(rh, row, c, a.cols, h);
      load_gain<VEC>(a.w, a.w_dtype, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(__fmul_rn(dy[j], w[j]), __fmul_rn(h[j], rstd), s);
    }
    s = cta_sum(s, red, flip) * inv_cols;
    for (int c = threadIdx.x * VEC; c < padded; c += span) {
      float d[VEC] = {}, *sums = colsum + (c - threadIdx.x * VEC) + threadIdx.x;
      load_cols<T, VEC, ANY>(ry, row, c, a.cols, dy);
      load_cols<T, VEC, ANY>(rh, row, c, a.cols, h);
      if (a.dh.p) load_cols<T, VEC, ANY>(rd, row, c, a.cols, d);
      load_gain<VEC>(a.w, a.w_dtype, c, a.cols, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float hn = __fmul_rn(h[j], rstd);
        d[j] = norm_dx(__fmul_rn(dy[j], w[j]), hn, s, rstd, d[j]);
        if (a.dw != nullptr) sums[j * blockDim.x] = fmaf(dy[j], hn, sums[j * blockDim.x]);
      }
      store_cols<T, VEC, ANY>(static_cast<T*>(a.dx.p) + row * a.dx.ld + c, c, a.cols, d, sbuf.mine());
    }
  }
  if (a.dw == nullptr) return;
  for (int c = threadIdx.x * VEC; c < a.cols; c += span)
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < a.cols)
        a.partials[static_cast<long long>(blockIdx.x) * a.cols + c + j] =
            colsum[(c - threadIdx.x * VEC) + threadIdx.x + j * blockDim.x];
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
// meet in shared memory and go to one row of the partials.  16384 x 11008, silu
// from blocks: 152 us, 6.0 TB/s.  The arguments are read where the launch put
// them: with a copy of them, rows of any alignment take 231 us instead of 139
// (15448 x 7164, silu).
// --------------------------------------------------------------------------
struct StripSums {
  float warp[8][256];
};
template <typename T, bool ANY, int ACT, bool Z8>
__device__ __forceinline__ void act_grad_rows(const ActGradArgs& a, int x, int y, int ny, StripSums& sums) {
  constexpr int VEC = 8;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = (x * 32 + lane) * VEC;
  const int step = ny * 8;
  int row = y * 8 + w;
  const Reader<T, ANY> ry(a.dy, a.rows, a.cols), rz(a.z, a.rows, a.cols);
  const T *py = ry.at(row, c), *pz = rz.at(row, c);
  const bool aligned = codes_aligned(a.z8);
  const int8_t* pq = a.z8.q + row * a.z8.ldq + c;
  const uint8_t* ps = a.z8.s + row * a.z8.lds + c / kPackBlock;
  T* pd = static_cast<T*>(a.dz.p) + row * a.dz.ld + c;
  const long long sy = step * a.dy.ld, sz = step * a.z.ld, sq = step * a.z8.ldq, ss = step * a.z8.lds,
                  sd = step * a.dz.ld;
  float sum[VEC] = {};
  for (; row < a.rows && c < a.cols; row += kWalk * step) {
    Raw<T, VEC, ANY> dy[kWalk], z[ACT != kActNone && !Z8 ? kWalk : 1];
    Codes<VEC, ANY> z8[Z8 ? kWalk : 1];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, py += sy, pz += sz, pq += sq, ps += ss) {
      const bool in = row + i * step < a.rows;
      dy[i].load(ry, py, c, a.cols, in);
      if constexpr (ACT != kActNone && Z8)
        z8[i].load(pq, ps, in ? a.cols - c : 0, aligned);
      else if constexpr (ACT != kActNone)
        z[i].load(rz, pz, c, a.cols, in);
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
      if (a.dz.p) store_vec<T, VEC>(pd, d);  // the workspace's pitch holds whole pieces
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] += d[j];
    }
  }
  if (a.db == nullptr) return;
#pragma unroll
  for (int j = 0; j < VEC; ++j) sums.warp[w][lane + 32 * j] = sum[j];
  __syncthreads();
  const int i = threadIdx.x;
  float s = sums.warp[0][i];
#pragma unroll
  for (int k = 1; k < 8; ++k) s += sums.warp[k][i];
  const int col = (x * 32 + i % 32) * VEC + i / 32;
  if (col >= a.cols) return;
  if (ny > 1)
    a.partials[static_cast<long long>(y) * a.cols + col] = s;
  else
    a.db[col] = a.accumulate ? a.db[col] + s : s;
}
template <typename T, bool ANY, int ACT, bool Z8>
__global__ void __launch_bounds__(256, ANY ? 2 : 3) act_grad_kernel(const __grid_constant__ ActGradArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ StripSums sums;
  act_grad_rows<T, ANY, ACT, Z8>(a, blockIdx.x, blockIdx.y, gridDim.y, sums);
}

// Copies a matrix to a pitch that holds whole 16-byte pieces.  Bound by HBM:
// 15448 x 7164 in 70 us, 6.3 TB/s.
__device__ __forceinline__ void repitch_rows(const Repitch& g, int x, int y, int ny) {
  using T = __nv_bfloat16;  // any 16-bit type: nothing is computed
  const int rows = g.rows, cols = g.cols;
  const Reader<T, true> r(g.src, rows, cols);
  const int c = (x * 32 + threadIdx.x % 32) * 8;
  if (c >= cols) return;
  const int step = ny * 8;
  int row = y * 8 + (threadIdx.y * blockDim.x + threadIdx.x) / 32;
  const T* p = r.at(row, c);
  T* d = static_cast<T*>(g.dst.p) + row * g.dst.ld + c;
  const long long ds = step * g.src.ld, dd = step * g.dst.ld;
  for (; row < rows; row += kWalk * step) {
    Raw<T, 8, true> raw[kWalk];
#pragma unroll
    for (int i = 0; i < kWalk; ++i, p += ds) raw[i].load(r, p, c, cols, row + i * step < rows);
#pragma unroll
    for (int i = 0; i < kWalk; ++i, d += dd) {
      if (row + i * step >= rows) break;
      raw[i].align();
      *reinterpret_cast<uint4*>(d) = make_uint4(raw[i].w[0], raw[i].w[1], raw[i].w[2], raw[i].w[3]);
    }
  }
}
struct RepitchArgs {
  Repitch job[2];  // by blockIdx.z
};
__global__ void __launch_bounds__(256, 4) repitch_kernel(const __grid_constant__ RepitchArgs a) {
  pdl_trigger();
  pdl_wait();
  repitch_rows(a.job[blockIdx.z], blockIdx.x, blockIdx.y, gridDim.y);
}

// What a small gradient needs before its products, in one launch (each launch
// less takes some 3 us off it): dz and db, the copies, and x from its blocks,
// every one over its own run of blocks.
struct PrepareArgs {
  ActGradArgs act;
  Repitch copy[2];
  int rows, cols;   // x
  Pack8 x8;
  Mat x;
  int first[5];     // blocks before dz, the copies, x, and in all
  int strips[4];    // strips of each
};
template <typename T, int ACT, bool Z8>
__global__ void __launch_bounds__(256, 2) prepare_kernel(const __grid_constant__ PrepareArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ StripSums sums;
  int k = 0;
  while (static_cast<int>(blockIdx.x) >= a.first[k + 1]) ++k;
  const int at = blockIdx.x - a.first[k], n = a.first[k + 1] - a.first[k];
  const int x = at % a.strips[k], y = at / a.strips[k], ny = n / a.strips[k];
  if (k == 0)
    act_grad_rows<T, true, ACT, Z8>(a.act, x, y, ny, sums);
  else if (k < 3)
    repitch_rows(a.copy[k - 1], x, y, ny);
  else
    unpack_rows<T, 8, false, true>(a.rows, a.cols, a.x8, a.x, x, y, ny, nullptr);
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
}  // namespace

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::atomic<int>& c = cached[dev & 63];
  int n = c.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    n = n > 0 ? n : 1;
    c.store(n, std::memory_order_relaxed);
  }
  return n;
}

namespace {
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

// How the columns are taken: type, columns a thread, any alignment.
template <typename T_, int VEC_, bool ANY_>
struct Access {
  using T = T_;
  static constexpr int VEC = VEC_;
  static constexpr bool ANY = ANY_;
  // Pieces a thread of the norm's kernels (and its gradient's) holds at most.
  static constexpr int kPieces = VEC == 8 ? 4 : 8, kGradPieces = VEC == 8 ? 2 : 8;
  static int lanes(int cols) { return (cols + VEC - 1) / VEC; }
};
// Calls f with the access for rows of `dtype`; vec: all of them are 16-byte
// aligned and a multiple of 8 columns long.
template <typename F>
cudaError_t by_access(int dtype, bool vec, F&& f) {
  if (dtype == kF32) return vec ? f(Access<float, 8, false>{}) : f(Access<float, 1, false>{});
  if (dtype == kBF16) return vec ? f(Access<__nv_bfloat16, 8, false>{}) : f(Access<__nv_bfloat16, 8, true>{});
  return vec ? f(Access<__half, 8, false>{}) : f(Access<__half, 8, true>{});
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
  return by_access(dtype, cols % 8 == 0 && vec_mat(x, elem_bytes(dtype)) && vec_pack(out), [&](auto acc) {
    using A = decltype(acc);
    static std::atomic<int> cache[9];
    auto k = pack8_kernel<typename A::T, A::VEC, A::ANY>;
    return launch_kernel(pdl_enabled(), k, walk_grid(k, rows, A::lanes(cols), kWalk, cache), kWalkBlock, 0, s, rows,
                         cols, x, out);
  });
}

cudaError_t launch_unpack8(int rows, int cols, Pack8 in, int dtype, Mat out, cudaStream_t s) {
  return by_access(dtype, cols % 8 == 0 && vec_mat(out, elem_bytes(dtype)) && vec_pack(in), [&](auto acc) {
    using A = decltype(acc);
    static std::atomic<int> cache[9];
    auto k = unpack8_kernel<typename A::T, A::VEC, A::ANY>;
    return launch_kernel(pdl_enabled(), k, walk_grid(k, rows, A::lanes(cols), kWalk, cache), kWalkBlock, 0, s, rows,
                         cols, in, out);
  });
}

namespace {
// Raises a kernel's dynamic shared memory limit, once per device.
template <typename K>
cudaError_t allow_smem(K k, int bytes, std::once_flag* once) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess)
    std::call_once(once[dev & 63],
                   [&] { err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  return err;
}

// Whether rows of both are misaligned alike.
bool alike(const Mat& a, const Mat& b, int elem_bytes) {
  return b.p == nullptr || ((reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p)) % 16 == 0 &&
                            (a.ld - b.ld) * elem_bytes % 16 == 0);
}

// Whether the memory of two of a gradient's matrices may overlap.
bool overlap(const NormGradArgs& a, const Mat& x, const Mat& y, int elem_bytes) {
  const auto end = [&](const Mat& m) {
    return reinterpret_cast<uintptr_t>(m.p) + ((a.rows - 1LL) * m.ld + a.cols) * elem_bytes;
  };
  return reinterpret_cast<uintptr_t>(x.p) < end(y) && reinterpret_cast<uintptr_t>(y.p) < end(x);
}

// Rows of `mats` matrices through shared memory: pieces a thread (NV, 0: they do
// not fit), threads, rows in shared memory and pieces of a row there.
constexpr int kStagedBytes = 220 * 1024;  // of a block at most
struct StagedPlan {
  int nv = 0, threads, depth, pitch, row;
  StagedPlan(int cols, int elem_bytes, int mats) {
    pitch = cols * elem_bytes / 16 + 3;
    row = mats * pitch * 16;
    const int lanes = (cols + 16 / elem_bytes - 1 + 7) / 8;
    for (int k : {2, 4}) {
      threads = ((lanes + k - 1) / k + 31) / 32 * 32;
      if (threads <= kRowThreads) {
        if (2 * row <= kStagedBytes) nv = k;
        return;
      }
    }
  }
  // Blocks the device holds, of the most an SM has registers for: as many as
  // leave each two rows.
  int blocks(int most) {
    for (int n = std::max(1, most / sm_count());; --n) {
      depth = std::min(4, (kStagedBytes / n - 2 * 1024) / row);
      if (depth >= 2 || n == 1) {
        depth = std::max(depth, 2);
        return n * sm_count();
      }
    }
  }
};
template <typename F>
cudaError_t by_staged_nv(int nv, F&& f) {
  return nv == 2 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 4>{});
}
template <typename F>
cudaError_t by_type(int dtype, F&& f) {
  if (dtype == kF32) return f(0.f);
  if (dtype == kBF16) return f(__nv_bfloat16{});
  return f(__half{});
}
// Launches kernel k (one of nkernels) over rows of a staged plan; `grid` gets
// the blocks: a multiple of 8 that are at most `most`, unless every row has one.
template <typename K, typename A>
cudaError_t launch_staged(K k, StagedPlan p, const A& a, int most, int* grid, std::once_flag* once,
                          std::atomic<int>* cache, cudaStream_t s) {
  const cudaError_t e = allow_smem(k, kStagedBytes, once);
  if (e != cudaSuccess) return e;
  *grid = std::min(p.blocks(resident(k, p.threads, 0, cache)), most);
  *grid = a.rows <= *grid ? a.rows : std::max(8, *grid / 8 * 8);
  return launch_kernel(pdl_enabled(), k, dim3(*grid), dim3(p.threads), static_cast<size_t>(p.depth) * p.row, s, a,
                       p.depth, p.pitch);
}
}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.x, eb) && vec_mat(a.residual, eb) && vec_mat(a.h, eb) &&
                   vec_mat(a.y, eb) && vec_pack(a.y8);
  const bool res = a.residual.p != nullptr;
  // Misaligned rows (up to 240 columns no faster).  Blocks of 8 bits are 32 columns
  // of a row, wherever it begins.
  const StagedPlan p(a.cols, eb, 1 + res);
  if (!vec && a.y8.q == nullptr && a.cols > 240 && p.nv > 0 && alike(a.x, a.residual, eb) && alike(a.x, a.h, eb) &&
      alike(a.x, a.y, eb))
    return by_type(a.dtype, [&](auto t) {
      return by_staged_nv(p.nv, [&](auto n) {
        using T = decltype(t);
        constexpr int NV = decltype(n)::value;
        static std::once_flag once[2][64];
        static std::atomic<int> cache[2][kRowThreads / 32 + 1];
        auto k = res ? rms_norm_staged_kernel<T, NV, true> : rms_norm_staged_kernel<T, NV, false>;
        int grid;
        return launch_staged(k, p, a, 1 << 30, &grid, once[res], cache[res], s);
      });
    });
  return by_access(a.dtype, vec, [&](auto acc) {
    using A = decltype(acc);
    using T = typename A::T;
    const RowShape r = row_shape(A::lanes(a.cols), kRowThreads, kRowThreads, A::kPieces);
    if (r.nv == 0)
      return launch_kernel(pdl_enabled(), rms_norm_wide_kernel<T, A::VEC, A::ANY>,
                           dim3(std::min(a.rows, 2 * sm_count())), dim3(1024), 0, s, a);
    return by_nv<A::kPieces>(r.nv, [&](auto n) {
      constexpr int NV = decltype(n)::value;
      static std::atomic<int> cache[2][kRowThreads / 32 + 1];
      auto k = res ? rms_norm_kernel<T, A::VEC, A::ANY, NV, true> : rms_norm_kernel<T, A::VEC, A::ANY, NV, false>;
      const int threads = r.block.x * r.block.y;
      const long long blocks = (static_cast<long long>(a.rows) + r.block.y - 1) / r.block.y;
      const int grid = static_cast<int>(std::min<long long>(blocks, resident(k, threads, 0, cache[res])));
      return launch_kernel(pdl_enabled(), k, dim3(grid), r.block, 0, s, a);
    });
  });
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, cudaStream_t s) {
  const int eb = elem_bytes(a.dtype);
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, eb) && vec_mat(a.h, eb) && vec_mat(a.dh, eb) && vec_mat(a.dx, eb);
  const bool dh = a.dh.p != nullptr;
  const StagedPlan p(a.cols, eb, 2 + dh);
  // Misaligned rows that registers hold only with many instructions, where there
  // are enough of them to be copied ahead.  bf16: 9000 x 1531 33 us for 36, but 16384
  // x 1009 43 for 37; 5000 x 8005 70 for 102, but 608 x 8005 27 for 23; 9001 columns,
  // which registers do not hold: 8 rows 14.8 for 17.0, 608 24.9 for 37.4.  fp32: 16384
  // x 4095 152 for 154, but 1500 x 4089 27 for 19; 2500 x 6001 49 for 89.
  const bool some = a.rows >= 6 * sm_count();
  const bool edge = !vec && (eb == 2 ? a.cols > 16 * kRowThreads || (a.cols > 1280 && some) : a.cols > 4096 && some) &&
                    alike(a.h, a.dy, eb) && alike(a.h, a.dh, eb) && alike(a.h, a.dx, eb);
  int parts = 0;  // rows of partial column sums, as many at most as the workspace holds
  cudaError_t e;
  // Aligned rows of more than two pieces a thread: 16384 x 11008 230 us, read twice
  // from memory and cache 678.
  if (p.nv > 0 && (edge || (vec && a.cols > 16 * kRowThreads)))
    e = by_type(a.dtype, [&](auto t) {
      return by_staged_nv(p.nv, [&](auto n) {
        using T = decltype(t);
        constexpr int NV = decltype(n)::value;
        static std::once_flag once[4][64];
        static std::atomic<int> cache[4][kRowThreads / 32 + 1];
        const auto launch = [&](auto k, int i) {
          return launch_staged(k, p, a, kMaxPartials, &parts, once[i], cache[i], s);
        };
        if constexpr (NV == 4)
          if (vec)
            return dh ? launch(rms_norm_grad_staged_kernel<T, false, NV, true>, 0)
                      : launch(rms_norm_grad_staged_kernel<T, false, NV, false>, 1);
        return dh ? launch(rms_norm_grad_staged_kernel<T, true, NV, true>, 2)
                  : launch(rms_norm_grad_staged_kernel<T, true, NV, false>, 3);
      });
    });
  else
    e = by_access(a.dtype, vec, [&](auto acc) {
      using A = decltype(acc);
      using T = typename A::T;
      const RowShape r = row_shape(A::lanes(a.cols), 256, kRowThreads, A::kGradPieces);
      if (r.nv == 0) {
        auto k = rms_norm_grad_wide_kernel<T, A::VEC, A::ANY>;
        static std::once_flag once[64];
        const cudaError_t e = allow_smem(k, kNormMaxCols * 4, once);
        if (e != cudaSuccess) return e;
        const int span = 1024 * A::VEC;
        parts = std::min(a.rows, sm_count());
        return launch_kernel(pdl_enabled(), k, dim3(parts), dim3(1024),
                             a.dw != nullptr ? static_cast<size_t>(a.cols + span - 1) / span * span * 4 : 0, s, a);
      }
      return by_nv<A::kGradPieces>(r.nv, [&](auto n) {
        constexpr int NV = decltype(n)::value;
        static std::atomic<int> cache[2][kRowThreads / 32 + 1];
        auto k = dh ? rms_norm_grad_kernel<T, A::VEC, A::ANY, NV, true> : rms_norm_grad_kernel<T, A::VEC, A::ANY, NV, false>;
        // Rows of a block: what makes it 256 threads, as the partials allow few blocks
        // (16384 x 1024 bf16: 27.5 us against 33.5), where there are rows for it.
        // Few rows in one launch: 512 x 4096 bf16 9.8 us for 15.4, as much at 640 x 8000
        // (16.4 for 17.7).  Misaligned 512 x 2047 12.4 us for 13.3, but 512 x 301 12.3
        // for 10.4, where few strips have it all to shift (304 x 301 10.3 for 9.6).
        // What is written must not be what the strips' blocks read.
        const int few = vec ? 640 : eb == 2 && a.cols >= 1000 ? 512 : 256;
        const bool strips = a.dw != nullptr && a.rows <= few && !overlap(a, a.dx, a.dy, eb) && !overlap(a, a.dx, a.h, eb);
        const int tx = r.block.x,
                  ty = std::max<int>(r.block.y, strips ? 256 / tx : std::min(256 / tx, a.rows / (2 * sm_count())));
        const int threads = tx * ty;
        const long long blocks = (static_cast<long long>(a.rows) + ty - 1) / ty;
        if (strips) {
          NormGradArgs b = a;
          b.strips = (a.cols + strip_cols<A::VEC>() - 1) / strip_cols<A::VEC>();
          const size_t smem = static_cast<size_t>(threads) * A::VEC * 4;
          return launch_kernel(pdl_enabled(), k, dim3(b.strips + static_cast<unsigned>(blocks)), dim3(tx, ty), smem, s, b);
        }
        const size_t smem = ty > 1 ? static_cast<size_t>(threads) * A::VEC * NV * 4 : 0;
        parts = static_cast<int>(std::min({blocks, static_cast<long long>(resident(k, threads, smem, cache[dh])),
                                           static_cast<long long>(kMaxPartials)}));
        return launch_kernel(pdl_enabled(), k, dim3(parts), dim3(tx, ty), smem, s, a);
      });
    });
  if (e != cudaSuccess || a.dw == nullptr || parts == 0) return e;
  return launch_kernel(pdl_enabled(), column_sum_kernel, dim3((a.cols + 31) / 32), dim3(32 * kChains), 0, s,
                       static_cast<const float*>(a.partials), parts, a.cols, a.dw, a.accumulate);
}

namespace {
// db from the activation gradient's partials; one row of them was written to db.
cudaError_t sum_columns(const float* partials, int parts, int cols, float* db, int accumulate, cudaStream_t s) {
  if (parts == 1) return cudaSuccess;
  return launch_kernel(pdl_enabled(), column_sum_kernel, dim3((cols + 31) / 32), dim3(32 * kChains), 0, s, partials,
                       parts, cols, db, accumulate);
}
}  // namespace

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && vec_mat(a.dy, 2) && vec_mat(a.z, 2) && vec_pack(a.z8);
  int parts = 0;
  const cudaError_t e = by_access(a.dtype, vec, [&](auto acc) {
    using A = decltype(acc);
    if constexpr (sizeof(typename A::T) == 4) {
      return cudaErrorInvalidValue;  // 16-bit types only
    } else {
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        const bool z8 = a.z8.q != nullptr;
        auto k = z8 ? act_grad_kernel<typename A::T, A::ANY, ACT, true> : act_grad_kernel<typename A::T, A::ANY, ACT, false>;
        static std::atomic<int> cache[2][9];
        dim3 grid = walk_grid(k, a.rows, A::lanes(a.cols), kWalk, cache[z8]);
        // Few rows: one block a column strip, which writes db itself (a second
        // kernel takes longer than the rows the strip's warps walk instead).
        grid.y = a.db != nullptr && a.rows <= kFewRowsOfDz ? 1 : std::min<unsigned>(grid.y, kMaxPartials);
        parts = static_cast<int>(grid.y);
        return launch_kernel(pdl_enabled(), k, grid, dim3(256), 0, s, a);
      });
    }
  });
  return e != cudaSuccess || a.db == nullptr ? e : sum_columns(a.partials, parts, a.cols, a.db, a.accumulate, s);
}

cudaError_t launch_prepare(const ActGradArgs& act, const Repitch* copies, int ncopies, int rows, int cols, Pack8 x8,
                           Mat x, cudaStream_t s) {
  PrepareArgs a{};
  a.act = act;
  a.rows = rows;
  a.cols = cols;
  a.x8 = x8;
  a.x = x;
  // Blocks of a job: whole strips, a wave of the device at most.
  int n = 0;
  const auto add = [&](int k, int r, int c, int most) {
    if (r > 0) {
      a.strips[k] = (c + 255) / 256;
      n += a.strips[k] * std::max(1, std::min({(r + 8 * kWalk - 1) / (8 * kWalk), 2 * sm_count() / a.strips[k], most}));
    }
    a.first[k + 1] = n;
  };
  add(0, act.rows, act.cols, act.db != nullptr && act.rows <= kFewRowsOfDz ? 1 : kMaxPartials);
  const int parts = n / a.strips[0];
  for (int k = 0; k < 2; ++k) {
    if (k < ncopies) a.copy[k] = copies[k];
    add(1 + k, k < ncopies ? copies[k].rows : 0, k < ncopies ? copies[k].cols : 0, 1 << 30);
  }
  add(3, x8.q != nullptr ? rows : 0, cols, 1 << 30);
  const cudaError_t e = by_act(act.act, [&](auto t) {
    constexpr int ACT = decltype(t)::value;
    const bool z8 = act.z8.q != nullptr;
    auto run = [&](auto v) {
      using T = decltype(v);
      auto k = z8 ? prepare_kernel<T, ACT, ACT != kActNone> : prepare_kernel<T, ACT, false>;
      return launch_kernel(pdl_enabled(), k, dim3(n), dim3(256), 0, s, a);
    };
    return act.dtype == kBF16 ? run(__nv_bfloat16{}) : run(__half{});
  });
  return e != cudaSuccess || act.db == nullptr ? e : sum_columns(act.partials, parts, act.cols, act.db, act.accumulate, s);
}

cudaError_t launch_repitch(const Repitch* jobs, int n, cudaStream_t s) {
  static std::atomic<int> cache[9];
  RepitchArgs a{};
  dim3 grid(1, 1, n);
  for (int i = 0; i < n; ++i) {
    a.job[i] = jobs[i];
    const dim3 g = walk_grid(repitch_kernel, jobs[i].rows, (jobs[i].cols + 7) / 8, kWalk, cache);
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
