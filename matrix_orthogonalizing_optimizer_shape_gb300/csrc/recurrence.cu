// Gated linear recurrence on sm_103a, h_t = a_t h_{t-1} + (1 - a_t) x_t with
// a = sigmoid(z), and its gradient.  Both are bound by HBM: every row is read
// once and written once, the scan happens in registers.
//
// A step h -> a h + b is an affine map, and maps compose: (A, B) after (A', B')
// is (A A', A B' + B).  A block takes a tile of channels (a lane VEC of them) and
// kSpan consecutive rows, kRows a warp: each thread composes its rows' maps in
// order, the warps' maps are composed through shared memory and those of a
// cluster's blocks, which take the spans after one another, through the cluster's.
// The cluster then walks down the rows, keeping the state; a row waits for one
// block barrier and one cluster barrier, while the next rows' loads are in flight.
//
// Packed sequences: a map whose factor is set to 0 cuts, so that rows are divided
// evenly whatever the sequences' lengths; nothing of the rows before a cut, NaN
// included, passes it.  Where the channels are few, groups of whole sequences go
// to different clusters.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "cluster.cuh"
#include "layer_math.cuh"
#include "model.h"

namespace dion3 {
namespace {

using namespace lm;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 8;                // rows of a warp in a step
constexpr int kSpan = kWarps * kRows;   // rows of a block in a step
constexpr int kMaxCluster = 8;
constexpr int kSharedOffsets = 1024;

// --------------------------------------------------------------------------
// Elements and maps.  VEC = 2 channels a lane where they are aligned, else 1.
// --------------------------------------------------------------------------
template <typename T, int VEC>
struct Word {
  using type = std::conditional_t<sizeof(T) * VEC == 8, uint2, std::conditional_t<sizeof(T) * VEC == 4, uint32_t, uint16_t>>;
};
template <typename T, int VEC>
struct Cell {
  typename Word<T, VEC>::type w;
  __device__ __forceinline__ void load(const T* p, bool in) {
    if (in)
      w = *reinterpret_cast<const typename Word<T, VEC>::type*>(p);
    else
      w = {};
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) const {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    if constexpr (sizeof(T) == 4 && VEC == 2) {
      v[0] = __uint_as_float(w.x);
      v[1] = __uint_as_float(w.y);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w);
    } else if constexpr (VEC == 2) {
      const float2 f = unpack2<kBf>(w);
      v[0] = f.x;
      v[1] = f.y;
    } else {
      v[0] = unpack1<kBf>(w);
    }
  }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_cell(T* p, const float (&v)[VEC]) {
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  if constexpr (sizeof(T) == 4 && VEC == 2)
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else if constexpr (sizeof(T) == 2 && VEC == 2)
    *reinterpret_cast<uint32_t*>(p) = pack2<kBf>(v[0], v[1]);
  else
    *p = from_f32<T>(v[0]);
}
// State vectors are fp32 with the channels' alignment unknown: element by element.
template <int VEC>
__device__ __forceinline__ void load_state(const float* p, float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = p[j];
}
template <int VEC>
__device__ __forceinline__ void store_state(float* p, const float (&v)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[j] = v[j];
}

// Maps h -> A h + B.  Where A is at least a half, F holds -(1 - A) with its sign
// bit set, else A itself: a factor near 1 that were rounded would decay the state
// at a rate that is off in every one of thousands of rows.  F = +0 cuts: nothing
// of h passes, NaN and infinity included.
__device__ __forceinline__ bool near_one(float F) { return static_cast<int>(__float_as_uint(F)) < 0; }
__device__ __forceinline__ float through(float F, float B, float h) {
  const float r = fmaf(F, h, B) + (near_one(F) ? h : 0.f);
  return __float_as_uint(F) == 0u ? B : r;
}
// The factor of F2 after F1: with both below 1 by D, D1 + D2 - D1 D2.
__device__ __forceinline__ float after(float F2, float F1) {
  const bool n1 = near_one(F1), n2 = near_one(F2);
  const float r = fmaf(F2, F1, (n2 ? F1 : 0.f) + (n1 ? F2 : 0.f));
  if (!(n1 && n2)) return r;
  return r < -0.5f ? 1.f + r : -fabsf(r);
}
__device__ __forceinline__ float encode(float A, float D) { return D < 0.5f ? -D : A; }
// A row's state from its thread's map up to it: not passed on, so a plain factor.
__device__ __forceinline__ float reach(float A, float B, float h) { return A == 0.f ? B : fmaf(A, h, B); }

// w = the smaller of a = sigmoid(z) and 1 - a, computed without cancellation;
// the larger is 1 - w.  A state that is nearly kept or nearly replaced is then
// h + w (x - h) or x + w (h - x), off by a rounding of the result, where a rounded
// factor a near 1 would change the decay over thousands of rows.
struct Gate {
  float w, big;  // small and large of a, 1 - a
  bool keep;     // a is the larger
  __device__ __forceinline__ explicit Gate(float z) : keep(z >= 0.f) {
    float u;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(-kLog2E * fabsf(z)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(big) : "f"(1.f + u));
    w = u * big;
  }
  __device__ __forceinline__ float step(float h, float x) const {
    const float p = keep ? h : x, q = keep ? x : h;
    return fmaf(w, q - p, p);
  }
  __device__ __forceinline__ float decay(float A) const {  // a A
    const float t = w * A;
    return keep ? A - t : t;
  }
  __device__ __forceinline__ void decay(float& A, float& D) const {  // and D = 1 - A
    const float t = w * A;
    A = keep ? A - t : t;
    D = keep ? D + t : 1.f - t;
  }
};

// --------------------------------------------------------------------------
// Sequences: off[0 .. n], rows [off[i], off[i + 1]) are sequence i.
// --------------------------------------------------------------------------
struct Sequences {
  const int* off;
  int n;
  // Numbers of starts below row (or up to it).
  __device__ __forceinline__ int starts_below(int row, bool inclusive) const {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      const int v = off[mid];
      if (inclusive ? v <= row : v < row)
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo;
  }
  // The sequence that holds a row of the sequences' rows.
  __device__ __forceinline__ int of(int row) const { return max(starts_below(row, true) - 1, 0); }
  // The next and the previous one that has rows.
  __device__ __forceinline__ int next(int q) const {
    q = min(q + 1, n - 1);
    while (q < n - 1 && off[q + 1] <= off[q]) ++q;
    return q;
  }
  __device__ __forceinline__ int prev(int q) const {
    q = max(q - 1, 0);
    while (q > 0 && off[q + 1] <= off[q]) --q;
    return q;
  }
};

// What a block works on: the sequences (their offsets in shared memory where they
// fit) and the rows [r0, r1) of its group, sequences [s0, s1).
struct Span {
  Sequences seq;
  int s0, s1, r0, r1;
};
__device__ __forceinline__ Span span_of(const RecurrenceArgs& a, int group, int groups, int* shared) {
  Span p;
  p.seq.n = a.sequences;
  if (a.offsets == nullptr) {
    if (threadIdx.x == 0) shared[0] = 0, shared[1] = a.tokens;
    p.seq.off = shared;
  } else if (a.sequences < kSharedOffsets) {
    for (int i = threadIdx.x; i <= a.sequences; i += kThreads) shared[i] = a.offsets[i];
    p.seq.off = shared;
  } else {
    p.seq.off = a.offsets;
  }
  __syncthreads();
  const long long t = a.tokens;
  p.s0 = group == 0 ? 0 : p.seq.starts_below(static_cast<int>(t * group / groups), false);
  p.s1 = group == groups - 1 ? a.sequences : p.seq.starts_below(static_cast<int>(t * (group + 1) / groups), false);
  p.r0 = min(max(p.seq.off[p.s0], 0), a.tokens);
  p.r1 = min(max(p.seq.off[p.s1], p.r0), a.tokens);
  return p;
}

// to[i] = from[i] (0 without one) for the sequences without rows.
template <int VEC>
__device__ __forceinline__ void copy_empty(const Span& p, const float* from, float* to, int channels, int c, bool in) {
  for (int q = p.s0 + static_cast<int>(threadIdx.x) / 32; q < p.s1; q += kWarps) {
    if (p.seq.off[q + 1] > p.seq.off[q] || !in) continue;
    float v[VEC] = {};
    if (from != nullptr) load_state<VEC>(from + static_cast<long long>(q) * channels + c, v);
    store_state<VEC>(to + static_cast<long long>(q) * channels + c, v);
  }
}

// The maps of a block's warps and a cluster's blocks, in turn in two halves.
struct Maps {
  float4 warp[2][kWarps][32];
  float4 block[2][kMaxCluster][32];
};

// From the map (F, B) of this warp's rows and the state before the cluster's rows
// (which becomes the state after them): the state before this warp's rows.  A
// thread's call number is `step`.
template <int VEC>
__device__ __forceinline__ void enter(Maps& m, int step, int rank, int size, const float (&F)[VEC], const float (&B)[VEC],
                                      float (&carry)[VEC], float (&h)[VEC]) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, half = step & 1;
  m.warp[half][warp][lane] = make_float4(F[0], B[0], F[VEC - 1], B[VEC - 1]);
  __syncthreads();
  auto apply = [&](const float4& v, float (&to)[VEC]) {
    to[0] = through(v.x, v.y, to[0]);
    if constexpr (VEC == 2) to[1] = through(v.z, v.w, to[1]);
  };
  if (size > 1) {
    if (warp == kWarps - 1) {
      float4 all = m.warp[half][0][lane];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 v = m.warp[half][w][lane];
        all = make_float4(after(v.x, all.x), through(v.x, v.y, all.y), after(v.z, all.z), through(v.z, v.w, all.w));
      }
      for (int r = 0; r < size; ++r) cl::store(cl::peer(&m.block[half][rank][lane], r), all);
    }
    cl::arrive();
    cl::wait();
    for (int r = 0; r < size; ++r) {
      if (r == rank) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = carry[j];
      }
      apply(m.block[half][r][lane], carry);
    }
    for (int w = 0; w < warp; ++w) apply(m.warp[half][w][lane], h);
  } else {
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = carry[j];
      }
      apply(m.warp[half][w][lane], carry);
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) recurrence_kernel(RecurrenceArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ Maps maps;
  __shared__ int shared_off[kSharedOffsets];
  const int size = cl::size(), rank = cl::rank(), groups = gridDim.x / size;
  const Span p = span_of(a, blockIdx.x / size, groups, shared_off);
  if (size > 1) cl::arrive(), cl::wait();  // every block has begun before one writes to another
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = (blockIdx.y * 32 + lane) * VEC;
  const bool in = c < a.channels;
  if (a.last != nullptr && rank == 0) copy_empty<VEC>(p, a.first, a.last, a.channels, c, in);

  const T* pz = static_cast<const T*>(a.z.p) + c;
  const T* px = static_cast<const T*>(a.x.p) + c;
  T* ph = static_cast<T*>(a.h.p) + c;
  Cell<T, VEC> z[kRows], x[kRows];
  auto load = [&](long long row0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool ok = in && row0 + i < p.r1;
      z[i].load(pz + (row0 + i) * a.z.ld, ok);
      x[i].load(px + (row0 + i) * a.x.ld, ok);
    }
  };
  float carry[VEC] = {};
  const int stride = size * kSpan;
  long long base = p.r0 + (rank * kWarps + warp) * kRows;
  load(base);
  int step = 0;
  for (long long top = p.r0; top < p.r1; top += stride, base += stride, ++step) {
    const int row0 = static_cast<int>(min(base, static_cast<long long>(INT_MAX - kRows)));
    // Which rows begin a sequence, and the states that those begin with.
    unsigned begins = 0, ends = 0;
    float f[kRows][VEC];
    int q0 = 0;
    if (row0 < p.r1) {
      int q = q0 = p.seq.of(row0);
      int begin = p.seq.off[q], end = p.seq.off[q + 1];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (row0 + i == begin) {
          begins |= 1u << i;
          if (a.first != nullptr && in) load_state<VEC>(a.first + static_cast<long long>(q) * a.channels + c, f[i]);
        }
        if (row0 + i + 1 == end && row0 + i < p.r1) {
          ends |= 1u << i;
          q = p.seq.next(q);
          begin = p.seq.off[q], end = p.seq.off[q + 1];
        }
      }
    }
    float A[kRows][VEC], B[kRows][VEC], F[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float ra = 1.f, rd = 0.f, rb = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (begins >> i & 1) {
          ra = 0.f;
          rd = 1.f;
          rb = a.first != nullptr ? f[i][j] : 0.f;
        }
        float zv[VEC], xv[VEC];
        z[i].values(zv);
        x[i].values(xv);
        if (row0 + i < p.r1) {
          const Gate g(zv[j]);
          rb = g.step(rb, xv[j]);
          g.decay(ra, rd);
        }
        A[i][j] = ra;
        B[i][j] = rb;
      }
      F[j] = encode(ra, rd);
    }
    load(base + stride);
    float h[VEC];
    enter<VEC>(maps, step, rank, size, F, B[kRows - 1], carry, h);
    if (!in || row0 >= p.r1) continue;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (row0 + i >= p.r1) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) B[i][j] = reach(A[i][j], B[i][j], h[j]);
      store_cell<T, VEC>(ph + static_cast<long long>(row0 + i) * a.h.ld, B[i]);
    }
    if (a.last != nullptr && ends != 0u) {
      int q = q0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (ends >> i & 1) {
          store_state<VEC>(a.last + static_cast<long long>(q) * a.channels + c, B[i]);
          q = p.seq.next(q);
        }
      }
    }
  }
}

// --------------------------------------------------------------------------
// Gradient: g_t = dh_t + s_{t+1}, s_t = a_t g_t, dx = (1 - a) g and
// dz = g (h_{t-1} - x) a (1 - a).  The scan runs from the last row to the first;
// a row's map is s -> a s + a dh.  Row i of a warp is the i-th from its end.
// --------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) recurrence_grad_kernel(RecurrenceArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ Maps maps;
  __shared__ int shared_off[kSharedOffsets];
  const int size = cl::size(), rank = cl::rank(), groups = gridDim.x / size;
  const Span p = span_of(a, blockIdx.x / size, groups, shared_off);
  if (size > 1) cl::arrive(), cl::wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = (blockIdx.y * 32 + lane) * VEC;
  const bool in = c < a.channels;
  if (a.dfirst != nullptr && rank == 0) copy_empty<VEC>(p, a.dlast, a.dfirst, a.channels, c, in);

  const T* pz = static_cast<const T*>(a.z.p) + c;
  const T* px = static_cast<const T*>(a.x.p) + c;
  const T* ph = static_cast<const T*>(a.h.p) + c;
  const T* pd = static_cast<const T*>(a.dh.p) + c;
  T* pdz = static_cast<T*>(a.dz.p) + c;
  T* pdx = static_cast<T*>(a.dx.p) + c;
  float carry[VEC] = {};
  const int stride = size * kSpan;
  long long base = static_cast<long long>(p.r1) - 1 - (rank * kWarps + warp) * kRows;
  int step = 0;
  for (long long top = p.r1; top > p.r0; top -= stride, base -= stride, ++step) {
    Cell<T, VEC> z[kRows], x[kRows], hp[kRows], d[kRows];
    const bool any = base >= p.r0;
    const int row0 = any ? static_cast<int>(base) : p.r0;
    unsigned begins = 0, ends = 0;
    float f[kRows][VEC], dl[kRows][VEC];
    int q0 = 0;
    if (any) {
      int q = q0 = p.seq.of(row0);
      int begin = p.seq.off[q], end = p.seq.off[q + 1];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = row0 - i;
        if (row + 1 == end) {
          ends |= 1u << i;
          if (a.dlast != nullptr && in) load_state<VEC>(a.dlast + static_cast<long long>(q) * a.channels + c, dl[i]);
        }
        if (row == begin) {
          begins |= 1u << i;
          if (a.first != nullptr && in) load_state<VEC>(a.first + static_cast<long long>(q) * a.channels + c, f[i]);
          q = p.seq.prev(q);
          begin = p.seq.off[q], end = p.seq.off[q + 1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long row = row0 - i;
      const bool ok = in && any && row >= p.r0;
      z[i].load(pz + row * a.z.ld, ok);
      d[i].load(pd + row * a.dh.ld, ok);
      x[i].load(px + row * a.x.ld, ok);
      hp[i].load(ph + (row - 1) * a.h.ld, ok && row > p.r0 && !(begins >> i & 1));
    }
    float A[VEC], D[VEC], B[VEC], dv[kRows][VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) A[j] = 1.f, D[j] = B[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      d[i].values(dv[i]);
      float zv[VEC];
      z[i].values(zv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (ends >> i & 1) {
          A[j] = B[j] = 0.f;
          D[j] = 1.f;
          if (a.dlast != nullptr) dv[i][j] += dl[i][j];
        }
        if (any && row0 - i >= p.r0) {
          const Gate g(zv[j]);
          B[j] = g.decay(dv[i][j] + B[j]);
          g.decay(A[j], D[j]);
        }
      }
    }
    float F[VEC], s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) F[j] = encode(A[j], D[j]);
    enter<VEC>(maps, step, rank, size, F, B, carry, s);
    if (!in || !any) continue;
    int q = q0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const long long row = row0 - i;
      if (row < p.r0) break;
      float zv[VEC], xv[VEC], hv[VEC], dz[VEC], dx[VEC];
      z[i].values(zv);
      x[i].values(xv);
      hp[i].values(hv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (ends >> i & 1) s[j] = 0.f;
        if ((begins >> i & 1) && a.first != nullptr) hv[j] = f[i][j];
        const Gate g(zv[j]);
        const float gr = dv[i][j] + s[j], t = g.w * gr;
        dx[j] = g.keep ? t : gr - t;
        dz[j] = t * g.big * (hv[j] - xv[j]);
        s[j] = g.keep ? gr - t : t;
      }
      store_cell<T, VEC>(pdz + row * a.dz.ld, dz);
      store_cell<T, VEC>(pdx + row * a.dx.ld, dx);
      if (begins >> i & 1) {
        if (a.dfirst != nullptr) store_state<VEC>(a.dfirst + static_cast<long long>(q) * a.channels + c, s);
        q = p.seq.prev(q);
      }
    }
  }
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
bool pairs(const Mat& m, int dtype) {  // two channels at an aligned address in every row
  const int es = dtype == kF32 ? 4 : 2;
  return m.p == nullptr || (m.ld % 2 == 0 && reinterpret_cast<uintptr_t>(m.p) % (2 * es) == 0);
}

template <class K>
cudaError_t launch_scan(K kernel, const RecurrenceArgs& a, int vec, cudaStream_t s) {
  const int tiles = (a.channels + 32 * vec - 1) / (32 * vec);
  const int want = 2 * sm_count();  // blocks
  int size = 1;
  while (size < kMaxCluster && 2 * size * tiles <= want && size * kSpan < a.tokens) size *= 2;
  const int groups = std::max(1, std::min({a.sequences, want / (tiles * size), 65535 / kMaxCluster}));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * groups, tiles);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(size), 1u, 1u};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t launch_typed(const RecurrenceArgs& a, bool vec2, cudaStream_t s) {
  if (a.grad)
    return launch_scan(vec2 ? recurrence_grad_kernel<T, 2> : recurrence_grad_kernel<T, 1>, a, vec2 ? 2 : 1, s);
  return launch_scan(vec2 ? recurrence_kernel<T, 2> : recurrence_kernel<T, 1>, a, vec2 ? 2 : 1, s);
}

}  // namespace

cudaError_t launch_recurrence(const RecurrenceArgs& a, cudaStream_t s) {
  bool vec2 = a.channels % 2 == 0;
  for (const Mat* m : {&a.z, &a.x, &a.h, &a.dh, &a.dz, &a.dx}) vec2 = vec2 && pairs(*m, a.dtype);
  if (a.dtype == kF32) return launch_typed<float>(a, vec2, s);
  if (a.dtype == kBF16) return launch_typed<__nv_bfloat16>(a, vec2, s);
  return launch_typed<__half>(a, vec2, s);
}

}  // namespace dion3
