// The norm over all gradients and their clipping, on sm_103a.  Bound by HBM: the
// norm reads every gradient once, clipping reads and writes each once more (what
// the norm read last still comes from L2, since clipping walks backwards).
//
// Tensors are divided into chunks of kChunk bytes, which the blocks of one launch
// take in turn: a table of the tensors travels in the kernel's parameters.  Each
// block leaves one partial sum, and every block that needs the norm adds them in
// the same order.
//
// Squares are summed in fp32 over a thread's few pieces and those sums in fp64.  A
// sum outside [2^-70, 2^110], where squares may have left fp32's range, is formed
// again from scaled values, so the norm is right for every finite gradient.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cluster.cuh"
#include "layer_math.cuh"
#include "model.h"

namespace dion3 {
namespace {

using namespace lm;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 16384;  // bytes of a chunk that is read
constexpr int kSquareBlocks = 6, kScaleBlocks = 5;  // of an SM
constexpr int kBatch = 4;      // pieces of 16 bytes a thread has in flight: a chunk in one go

template <typename T>
constexpr int kPer = 16 / sizeof(T);

template <int N>
struct Table {
  GradTensor t[N];
};
constexpr int kFew = 16, kMany = 448;
static_assert(sizeof(Table<kMany>) < 32000, "kernel parameters");

template <typename T>
__device__ __forceinline__ void piece_values(const uint4& u, float (&v)[kPer<T>]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = unpack2<std::is_same<T, __nv_bfloat16>::value>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// A chunk: n elements from `in`, to `out`.
struct Chunk {
  const GradTensor* t;
  long long row, at;  // its row and its first element's column
  int n;
};
// Which one number c is: the last tensor whose first chunk is not behind it.
template <int N>
__device__ __forceinline__ Chunk chunk_of(const Table<N>& tab, int count, unsigned c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].first <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  const GradTensor& t = tab.t[lo];
  const unsigned k = c - t.first, row = k / t.per_row;
  const int len = kChunk / (t.dtype == kF32 ? 4 : 2);
  const long long at = static_cast<long long>(k - row * t.per_row) * len;
  return {&t, static_cast<long long>(row), at, static_cast<int>(min(static_cast<long long>(len), t.cols - at))};
}

// Sum of squares of n values, as a double; s: their plain fp32 sum.
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) s = fmaf(v[j], v[j], s);
  if (s >= 0x1p-70f && s <= 0x1p110f) return static_cast<double>(s);
  const float up = s < 1.f ? 0x1p90f : 0x1p-70f;  // too small, or too large (or NaN)
  float r = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float x = v[j] * up;
    r = fmaf(x, x, r);
  }
  return static_cast<double>(r) * (s < 1.f ? 0x1p-180 : 0x1p140);
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const Chunk& c) {
  const T* p = static_cast<const T*>(c.t->in) + c.row * c.t->ld_in + c.at;
  const int head = min(c.n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) % 16 / sizeof(T)));
  const int pieces = (c.n - head) / kPer<T>, tail = c.n - head - pieces * kPer<T>;
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  float v[kBatch * kPer<T>];
  static_assert(kBatch * 16 * kThreads == kChunk, "a chunk in one go");
  uint4 u[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int i = threadIdx.x + b * kThreads;
    u[b] = i < pieces ? body[i] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    float f[kPer<T>];
    piece_values<T>(u[b], f);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) v[b * kPer<T> + j] = f[j];
  }
  double sum = squares(v);
  if (threadIdx.x < head + tail) {
    const int at = threadIdx.x < head ? threadIdx.x : head + pieces * kPer<T> + threadIdx.x - head;
    const float e[1] = {to_f32<T>(p[at])};
    sum += squares(e);
  }
  return sum;
}

// The sum over a block's threads, in thread 0.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kWarps ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int d = kWarps / 2; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// A thread's part of the squares of the chunks that its block takes.
template <int N>
__device__ __forceinline__ double squares_of_chunks(const Table<N>& tab, int count, unsigned chunks) {
  double sum = 0.0;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = chunk_of(tab, count, c);
    if (k.t->dtype == kF32)
      sum += chunk_squares<float>(k);
    else if (k.t->dtype == kBF16)
      sum += chunk_squares<__nv_bfloat16>(k);
    else
      sum += chunk_squares<__half>(k);
  }
  return sum;
}

// partials[block] = (of an earlier launch: +=) the block's sum; `kept`: partials that earlier launches left.
template <int N>
__global__ void __launch_bounds__(kThreads, kSquareBlocks) grad_squares_kernel(const __grid_constant__ Table<N> tab, int count,
                                                                  unsigned chunks, double* partials, int kept) {
  pdl_trigger();
  pdl_wait();
  __shared__ double red[kWarps];
  const double sum = block_sum(squares_of_chunks(tab, count, chunks), red);
  if (threadIdx.x == 0) partials[blockIdx.x] = sum + (static_cast<int>(blockIdx.x) < kept ? partials[blockIdx.x] : 0.0);
}

// The norm from the partials, the same bits in every block (in thread 0).
__device__ __forceinline__ float norm_of(const double* partials, int n, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += partials[i];
  v = block_sum(v, red);
  return static_cast<float>(sqrt(v));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* partials, int n, float* norm) {
  pdl_trigger();
  pdl_wait();
  __shared__ double red[kWarps];
  const float v = norm_of(partials, n, red);
  if (threadIdx.x == 0) *norm = v;
}

// Scales a chunk, kBatch pieces of a thread (or eight elements) in flight.
template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const Chunk& c, float coef) {
  const T* p = static_cast<const T*>(c.t->in) + c.row * c.t->ld_in + c.at;
  O* q = static_cast<O*>(c.t->out) + c.row * c.t->ld_out + c.at;
  const int head = min(c.n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) % 16 / sizeof(T)));
  constexpr int kBytes = kPer<T> * static_cast<int>(sizeof(O));  // what a piece becomes: 8, 16 or 32
  const bool together = (reinterpret_cast<uintptr_t>(q + head) & (std::min(kBytes, 16) - 1)) == 0;
  if (!together) {
    constexpr int kAhead = 8;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < c.n; i0 += kAhead * kThreads) {
      T v[kAhead];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) v[b] = p[min(i0 + b * kThreads, c.n - 1)];
#pragma unroll
      for (int b = 0; b < kAhead; ++b)
        if (i0 + b * kThreads < c.n) q[i0 + b * kThreads] = from_f32<O>(to_f32<T>(v[b]) * coef);
    }
    return;
  }
  const int pieces = (c.n - head) / kPer<T>, tail = c.n - head - pieces * kPer<T>;
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  O* to = q + head;
  if (threadIdx.x < head + tail) {
    const int at = threadIdx.x < head ? threadIdx.x : head + pieces * kPer<T> + threadIdx.x - head;
    q[at] = from_f32<O>(to_f32<T>(p[at]) * coef);
  }
  {
    uint4 u[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      u[b] = threadIdx.x + b * kThreads < pieces ? body[threadIdx.x + b * kThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = threadIdx.x + b * kThreads;
      if (i >= pieces) break;
      uint4* at = reinterpret_cast<uint4*>(to + i * kPer<T>);
      float f[kPer<T>];
      piece_values<T>(u[b], f);
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j) f[j] *= coef;
      constexpr bool kBf = std::is_same<O, __nv_bfloat16>::value;
      if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(at) = make_uint2(pack2<kBf>(f[0], f[1]), pack2<kBf>(f[2], f[3]));
      } else if constexpr (sizeof(O) == 4) {
#pragma unroll
        for (int j = 0; j < kPer<T> / 4; ++j)
          at[j] = make_uint4(__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]),
                             __float_as_uint(f[4 * j + 3]));
      } else {
        *at = make_uint4(pack2<kBf>(f[0], f[1]), pack2<kBf>(f[2], f[3]), pack2<kBf>(f[4], f[5]), pack2<kBf>(f[6], f[7]));
      }
    }
  }
}

__device__ __forceinline__ float factor(float norm, float max_norm) {
  if (max_norm == INFINITY) return 1.f;  // clips nothing, though a norm may be infinite too
  const float r = max_norm / (norm + 1e-6f);
  return r > 1.f ? 1.f : r;  // NaN stays NaN
}
// The factor from the partials, the same bits in every block and thread.
__device__ __forceinline__ float factor_of(const double* partials, int n, float max_norm, float* norm) {
  __shared__ double red[kWarps];
  __shared__ float coef;
  const float total = norm_of(partials, n, red);
  if (threadIdx.x == 0) {
    coef = factor(total, max_norm);
    if (norm != nullptr && blockIdx.x == 0) *norm = total;
  }
  __syncthreads();
  return coef;
}

// Clipping, out = min(1, max_norm / (norm + 1e-6)) in; in place a factor of 1 leaves
// everything as it is.  Chunks run from the last to the first.  Tensors whose rows are
// aligned pieces that keep their type go through this kernel, the next chunk's loads in
// flight while one is scaled; the others through the kernels below, one a pair of types
// (all in one needed more registers than its blocks have).
template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4& u, float coef) {
  float f[kPer<T>];
  piece_values<T>(u, f);
#pragma unroll
  for (int j = 0; j < kPer<T>; ++j) f[j] *= coef;
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    return make_uint4(pack2<kBf>(f[0], f[1]), pack2<kBf>(f[2], f[3]), pack2<kBf>(f[4], f[5]), pack2<kBf>(f[6], f[7]));
  }
}
struct Pieces {
  const char* in;
  char* out;
  int bytes, dtype;
  __device__ __forceinline__ explicit Pieces(const Chunk& c) : dtype(c.t->dtype) {
    const int es = dtype == kF32 ? 4 : 2;
    in = static_cast<const char*>(c.t->in) + (c.row * c.t->ld_in + c.at) * es;
    out = static_cast<char*>(c.t->out) + (c.row * c.t->ld_out + c.at) * es;
    bytes = c.n * es;
  }
  __device__ __forceinline__ void load(uint4 (&u)[kBatch]) const {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = 16 * (threadIdx.x + b * kThreads);
      u[b] = at + 16 <= bytes ? *reinterpret_cast<const uint4*>(in + at) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(const uint4 (&u)[kBatch], float coef) const {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = 16 * (threadIdx.x + b * kThreads);
      if (at + 16 <= bytes) *reinterpret_cast<uint4*>(out + at) = scaled<T>(u[b], coef);
    }
    const int tail = bytes / 16 * 16 + static_cast<int>(threadIdx.x * sizeof(T));
    if (tail < bytes)
      *reinterpret_cast<T*>(out + tail) = from_f32<T>(to_f32<T>(*reinterpret_cast<const T*>(in + tail)) * coef);
  }
};
// A thread's part of chunk after chunk of its block, from the last to the first.
template <int N>
__device__ __forceinline__ void scale_chunks(const Table<N>& tab, int count, unsigned chunks, float coef) {
  unsigned i = blockIdx.x;
  if (i >= chunks) return;
  Pieces p(chunk_of(tab, count, chunks - 1 - i));
  uint4 u[kBatch];
  p.load(u);
  for (;;) {
    i += gridDim.x;
    const bool more = i < chunks;
    Pieces next = p;
    uint4 v[kBatch];
    if (more) {
      next = Pieces(chunk_of(tab, count, chunks - 1 - i));
      next.load(v);
    }
    if (p.dtype == kF32)
      p.store<float>(u, coef);
    else if (p.dtype == kBF16)
      p.store<__nv_bfloat16>(u, coef);
    else
      p.store<__half>(u, coef);
    if (!more) return;
    p = next;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) u[b] = v[b];
  }
}
template <int N>
__global__ void __launch_bounds__(kThreads, kScaleBlocks) grad_scale_kernel(const __grid_constant__ Table<N> tab,
                                                                           int count, unsigned chunks,
                                                                           const double* partials, int n, float max_norm,
                                                                           bool in_place, float* norm) {
  pdl_trigger();
  pdl_wait();
  const float coef = factor_of(partials, n, max_norm, norm);
  if (in_place && coef == 1.f) return;
  scale_chunks(tab, count, chunks, coef);
}

// Norm and clipping of a few chunks by one cluster: one launch, whose second reads come
// from cache.  Seven matrices and two vectors of a small layer: 21 us a call for 24 with
// two launches, where the host's side is what counts (on the device 7.7 for 5.8).
constexpr int kSmallCluster = 16, kSmallChunks = 4 * kSmallCluster;
__global__ void __launch_bounds__(kThreads) grad_clip_small_kernel(const __grid_constant__ Table<kFew> tab, int count,
                                                                   unsigned chunks, float max_norm, bool in_place,
                                                                   float* norm) {
  pdl_trigger();
  pdl_wait();
  __shared__ double red[kWarps];
  __shared__ unsigned long long sums[kSmallCluster];  // of the cluster's blocks
  cl::arrive();  // waited for before the first store to another block
  const int rank = cl::rank();
  const double sum = block_sum(squares_of_chunks(tab, count, chunks), red);
  cl::wait();
  if (threadIdx.x == 0)
    for (int r = 0; r < kSmallCluster; ++r)
      cl::store(cl::peer(&sums[rank], r), static_cast<unsigned long long>(__double_as_longlong(sum)));
  __syncwarp();
  cl::arrive();
  cl::wait();
  double all = 0.0;
  for (int r = 0; r < kSmallCluster; ++r) all += __longlong_as_double(static_cast<long long>(sums[r]));
  const float total = static_cast<float>(sqrt(all)), coef = factor(total, max_norm);
  if (norm != nullptr && rank == 0 && threadIdx.x == 0) *norm = total;
  if (in_place && coef == 1.f) return;
  scale_chunks(tab, count, chunks, coef);
}

template <int N, typename T, typename O>
__global__ void __launch_bounds__(kThreads, kScaleBlocks) grad_scale_other_kernel(const __grid_constant__ Table<N> tab,
                                                                                 int count, unsigned chunks,
                                                                                 const double* partials, int n,
                                                                                 float max_norm, bool in_place, float* norm) {
  pdl_trigger();
  pdl_wait();
  const float coef = factor_of(partials, n, max_norm, norm);
  if (in_place && coef == 1.f) return;
  for (unsigned i = blockIdx.x; i < chunks; i += gridDim.x) scale_chunk<T, O>(chunk_of(tab, count, chunks - 1 - i), coef);
}
// Whether a tensor goes through the first of the two.
bool keeps_pieces(const GradTensor& t) {
  const int es = t.dtype == kF32 ? 4 : 2;
  return t.dtype == t.out_dtype && ((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0 &&
         (t.rows == 1 || (t.ld_in * es % 16 == 0 && t.ld_out * es % 16 == 0));
}

// Calls f(table, tensors, chunks) for groups of the wanted tensors that fit a launch's
// parameters: kFew (a kilobyte) or kMany.

template <class P, class F>
cudaError_t for_groups(const GradTensor* t, int n, P&& wanted, F&& f) {
  int i = 0;
  while (i < n) {
    // The tensors of a group have fewer than 2^31 chunks together.
    Table<kMany> tab;
    int k = 0;
    unsigned long long chunks = 0;
    for (; i < n && k < kMany; ++i) {
      const long long len = kChunk / (t[i].dtype == kF32 ? 4 : 2), per = (t[i].cols + len - 1) / len;
      const unsigned long long all = static_cast<unsigned long long>(per) * t[i].rows;
      if (all == 0 || !wanted(t[i])) continue;
      if (chunks + all >= (1ull << 31)) {
        if (k == 0) return cudaErrorInvalidValue;
        break;
      }
      GradTensor& g = tab.t[k++] = t[i];
      g.first = static_cast<unsigned>(chunks);
      g.per_row = static_cast<unsigned>(per);
      chunks += all;
    }
    if (k == 0) break;
    cudaError_t e;
    if (k <= kFew) {
      Table<kFew> few;
      std::copy(tab.t, tab.t + k, few.t);
      e = f(few, k, static_cast<unsigned>(chunks));
    } else {
      e = f(tab, k, static_cast<unsigned>(chunks));
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
int dtype_of() {
  return std::is_same<T, float>::value ? kF32 : std::is_same<T, __nv_bfloat16>::value ? kBF16 : kF16;
}
int blocks_for(unsigned chunks, int per_sm) {
  return static_cast<int>(std::min<unsigned>(chunks, static_cast<unsigned>(std::min(per_sm * sm_count(), kMaxGradPartials))));
}

// Whether the current device holds a cluster past 8 blocks of the kernel for small sets: a
// part of a device may not, and takes the other launches.  Asked once a device, with the
// attribute that its launches need.
bool holds_small_cluster(const cudaLaunchConfig_t& cfg) {
  constexpr int kDevices = 64;
  static std::atomic<signed char> known[kDevices];  // 0: not asked, 1: yes, -1: no
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  if (device < kDevices && known[device].load(std::memory_order_acquire) != 0) return known[device].load() > 0;
  int clusters = 0;
  const bool holds =
      cudaFuncSetAttribute(grad_clip_small_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, grad_clip_small_kernel, &cfg) == cudaSuccess && clusters > 0;
  if (!holds) cudaGetLastError();
  if (device < kDevices) known[device].store(holds ? 1 : -1, std::memory_order_release);
  return holds;
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* t, int n, bool clip, float max_norm, bool in_place, float* norm,
                             double* partials, cudaStream_t s) {
  if (clip && n <= kFew) {  // all in one launch?
    bool done = false;
    const bool plain = std::all_of(t, t + n, keeps_pieces);
    const cudaError_t e = !plain ? cudaSuccess : for_groups(t, n, [](const GradTensor&) { return true; },
                                                           [&](const auto& tab, int count, unsigned chunks) {
      if constexpr (sizeof(tab.t) == sizeof(Table<kFew>)) {
        if (chunks > kSmallChunks) return cudaSuccess;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSmallCluster);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {kSmallCluster, 1u, 1u};
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (!holds_small_cluster(cfg)) return cudaSuccess;
        cfg.numAttrs = pdl_enabled() ? 2 : 1;
        done = true;
        return cudaLaunchKernelEx(&cfg, grad_clip_small_kernel, tab, count, chunks, max_norm, in_place, norm);
      }
      return cudaSuccess;
    });
    if (e != cudaSuccess || done) return e;
  }
  int kept = 0;
  cudaError_t e = for_groups(t, n, [](const GradTensor&) { return true; }, [&](const auto& tab, int count, unsigned chunks) {
    constexpr int N = sizeof(tab.t) / sizeof(GradTensor);
    const int blocks = blocks_for(chunks, kSquareBlocks);
    const cudaError_t r = launch_kernel(pdl_enabled(), grad_squares_kernel<N>, dim3(blocks), dim3(kThreads), 0, s, tab,
                                        count, chunks, partials, kept);
    kept = std::max(kept, blocks);
    return r;
  });
  if (e != cudaSuccess) return e;
  if (!clip || kept == 0)
    return norm == nullptr ? cudaSuccess
                           : launch_kernel(pdl_enabled(), grad_norm_kernel, dim3(1), dim3(kThreads), 0, s,
                                           static_cast<const double*>(partials), kept, norm);
  // One launch for the tensors whose pieces keep their type, and one for each pair of
  // types among the others.
  auto launch = [&](auto wanted, auto kernel_of) {
    return for_groups(t, n, wanted, [&](const auto& tab, int count, unsigned chunks) {
      constexpr int N = sizeof(tab.t) / sizeof(GradTensor);
      const cudaError_t r = launch_kernel(pdl_enabled(), kernel_of(std::integral_constant<int, N>{}),
                                          dim3(blocks_for(chunks, kScaleBlocks)), dim3(kThreads), 0, s, tab, count,
                                          chunks, static_cast<const double*>(partials), kept, max_norm, in_place, norm);
      norm = nullptr;  // written by the first launch
      return r;
    });
  };
  e = launch([](const GradTensor& g) { return keeps_pieces(g); }, [](auto N) { return grad_scale_kernel<N()>; });
  auto pair = [&](auto* from, auto* to) {
    using T = std::remove_pointer_t<decltype(from)>;
    using O = std::remove_pointer_t<decltype(to)>;
    if (e == cudaSuccess)
      e = launch([](const GradTensor& g) { return !keeps_pieces(g) && g.dtype == dtype_of<T>() && g.out_dtype == dtype_of<O>(); },
                 [](auto N) { return grad_scale_other_kernel<N(), T, O>; });
  };
  float* f = nullptr;
  __nv_bfloat16* b = nullptr;
  __half* h = nullptr;
  pair(f, f), pair(f, b), pair(f, h), pair(b, f), pair(b, b), pair(b, h), pair(h, f), pair(h, b), pair(h, h);
  return e;
}

}  // namespace dion3
