// Log probabilities of given tokens, entropy and top alternatives, and their
// gradient, on sm_103a.  Both passes are bound by HBM.
//
// A thread keeps the largest logit m it has seen, S = sum e^(s (l - m)) and
// Q = sum e^(s (l - m)) (l - m); two such triples join with one exponential each.
// Then log p = s (l - m) - log S and the entropy is log S - s Q / S.  Differences
// to m are taken before the scale, so that a logit's error does not grow with its
// size.  A row is split over a cluster's blocks where there are few.  8192 x 131072
// bf16: 331 us, 6.5 TB/s; its gradient 641 us, 6.7 TB/s.
//
// The k largest logits are found after the same single pass over memory: a thread
// whose own largest is below the k-th largest of the threads' holds none of them,
// so only the elements of the others, k threads where no two are equal, are read
// again (from L2) and put into a warp's sorted list: 453 us with 20 of them, at five
// blocks an SM (541 at three).  One row of 131072 takes 8.4 us.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "layer_math.cuh"
#include "model.h"

namespace dion3 {
namespace {

using namespace lm;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 4;  // pieces of 16 bytes that a thread has in flight
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster <= kWarps, "a warp a block");
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -1e30f;  // of a masked logit: its exponential is 0, and 0 times it too

using Key = unsigned long long;

__device__ __forceinline__ long long target_at(const Ids& ids, long long i) {
  if (ids.p == nullptr) return -1;
  return ids.bytes == 8 ? static_cast<const long long*>(ids.p)[i] : static_cast<const int*>(ids.p)[i];
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp, 0 below 2^-126
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 16 bytes as fp32 values.
template <typename T>
constexpr int kPer = 16 / sizeof(T);
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

// A slice [c0, c1) of a row: `head` elements before the first aligned piece,
// `pieces` pieces, `tail` elements.
template <typename T>
struct Slice {
  const T* p;  // element c0
  int head, pieces, tail;
  __device__ __forceinline__ Slice(const T* row, int c0, int c1) : p(row + c0) {
    const int n = max(c1 - c0, 0);
    head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) % 16 / sizeof(T)));
    pieces = (n - head) / kPer<T>;
    tail = n - head - pieces * kPer<T>;
  }
  __device__ __forceinline__ const uint4* body() const { return reinterpret_cast<const uint4*>(p + head); }
  // Offset from c0 of piece i's first element and of tail element i.
  __device__ __forceinline__ int piece_at(int i) const { return head + i * kPer<T>; }
  __device__ __forceinline__ int tail_at(int i) const { return head + pieces * kPer<T> + i; }
};

// --------------------------------------------------------------------------
// Softmax statistics
// --------------------------------------------------------------------------
struct Stat {
  float m = kLowest, s = 0.f, q = 0.f;
  // To a larger maximum; c = scale log2 e.
  __device__ __forceinline__ void raise(float to, float c) {
    const float d = max_nan(m - to, kFar), e = exp2_fast(d * c);
    q = fmaf(s, d, q) * e;
    s *= e;
    m = to;
  }
  __device__ __forceinline__ void add(float v, float c) {
    const float d = max_nan(v - m, kFar), e = exp2_fast(d * c);
    s += e;
    q = fmaf(e, d, q);
  }
  __device__ __forceinline__ void join(Stat o, float c) {
    const float to = fmaxf(m, o.m);
    raise(to, c);
    o.raise(to, c);
    s += o.s;
    q += o.q;
  }
  __device__ __forceinline__ Stat shuffled(int d) const {
    Stat o;
    o.m = __shfl_xor_sync(0xffffffffu, m, d);
    o.s = __shfl_xor_sync(0xffffffffu, s, d);
    o.q = __shfl_xor_sync(0xffffffffu, q, d);
    return o;
  }
};

// --------------------------------------------------------------------------
// Sorted lists: lane i of a warp holds the i-th largest.  Keys are a logit's
// order and, among equals, its column from the right; 0 is no entry, and NaN
// comes behind everything.
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return v != v ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return o == 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(float v, int column) {
  return static_cast<Key>(order_of(v)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(column));
}
template <typename K>
__device__ __forceinline__ K exchange(K a, int d, bool larger) {  // with the lane at distance d
  const K b = __shfl_xor_sync(0xffffffffu, a, d);
  return larger ? max(a, b) : min(a, b);
}
// A bitonic sequence, then any, into descending order.
template <typename K>
__device__ __forceinline__ K merge_lanes(K a) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) a = exchange(a, d, (lane & d) == 0);
  return a;
}
template <typename K>
__device__ __forceinline__ K sort_lanes(K a) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int d = n / 2; d > 0; d /= 2) a = exchange(a, d, ((lane & d) == 0) == ((lane & n) == 0));
  return a;
}
// The 32 largest of two descending lists; b_reversed: the other list's entry 31 - lane.
template <typename K>
__device__ __forceinline__ K merge_lists(K a, K b_reversed) { return merge_lanes(max(a, b_reversed)); }

// Puts each lane's key (0: none) into the list if it is among the k largest.
__device__ __forceinline__ void insert(Key key, int k, Key& list) {
  const int lane = threadIdx.x % 32;
  unsigned todo = __ballot_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, list, k - 1));
  while (todo != 0u) {
    const Key x = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
    todo &= todo - 1;
    const int at = __popc(__ballot_sync(0xffffffffu, list > x));
    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
    if (lane == at) list = x;
    if (lane > at) list = up;
  }
}

// The lists of a block's warps, written and waited for, into one in warp 0: by halves.
template <typename K>
__device__ __forceinline__ K merge_warps(K (&lists)[kWarps][32], K mine) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int n = kWarps / 2; n > 0; n /= 2) {
    if (warp < n) {
      mine = merge_lists(mine, lists[warp + n][31 - lane]);
      lists[warp][lane] = mine;
    }
    __syncthreads();
  }
  return mine;
}

struct Shared {
  Stat warp[kWarps];
  float4 block[kMaxCluster];          // of the cluster's blocks, in block 0
  uint32_t order[kWarps][32];         // the threads' maxima, sorted by warp
  uint32_t least;                     // the k-th largest of them
  int ncand;
  short cand[kThreads];
  Key list[kWarps][32];
  Key lists[kWarps][32];              // of the cluster's blocks, in block 0; others empty
};

// The block's k largest elements of its slice, in warp 0's lanes.
template <typename T>
__device__ __forceinline__ Key block_top(Shared& sh, const Slice<T>& sl, int c0, int k, float mine, bool any) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t order = any ? order_of(mine) : 0u;
  sh.order[warp][lane] = sort_lanes(order);
  if (tid == 0) sh.ncand = 0;
  __syncthreads();
  const uint32_t top = merge_warps(sh.order, sh.order[warp][lane]);
  if (warp == 0 && lane == k - 1) sh.least = max(top, 1u);
  __syncthreads();
  const uint32_t least = sh.least;
  // Many threads whose maximum equals the least (masked rows, for instance): of those
  // elements only the first columns count, and they are found from the left (64 rows
  // with three tokens allowed: 29 us, by reading all threads' elements again 110).
  const bool dense = __syncthreads_count(any && order >= least) > 2 * 32;
  if (any && (dense ? order > least : order >= least)) sh.cand[atomicAdd(&sh.ncand, 1)] = static_cast<short>(tid);
  __syncthreads();
  const int n = sh.ncand;
  Key list = 0;
  // Elements of order lo and above up to hi among a piece (p < sl.pieces) of each lane.
  auto offer_piece = [&](int p, uint32_t lo, uint32_t hi) {
    const bool in = p < sl.pieces;
    float v[kPer<T>];
    piece_values<T>(in ? sl.body()[p] : make_uint4(0u, 0u, 0u, 0u), v);
    int some = 0;
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) some += order_of(v[j]) >= lo && order_of(v[j]) <= hi;
    some = in ? some : 0;
    if (__any_sync(0xffffffffu, some)) {
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j) {
        const uint32_t o = order_of(v[j]);
        insert(in && o >= lo && o <= hi ? key_of(v[j], c0 + sl.piece_at(p) + j) : 0, k, list);
      }
    }
    return some;
  };
  for (int i = warp; i < n; i += kWarps)
    for (int p0 = sh.cand[i]; p0 < sl.pieces; p0 += 32 * kThreads)  // a lane takes one of the thread's pieces
      offer_piece(p0 + lane * kThreads, dense ? least + 1 : least, 0xFFFFFFFFu);
  if (dense) {
    int found = 0;
    for (int p0 = 0; p0 < sl.pieces && found < k; p0 += kThreads) {
      const int some = offer_piece(p0 + tid, least, least);
      found += __syncthreads_count(some > 0);  // of that many elements at least
    }
  }
  if (warp == 0) {  // the elements outside the pieces
    const bool in = lane < sl.head + sl.tail;
    const int at = lane < sl.head ? lane : sl.tail_at(lane - sl.head);
    const float v = in ? to_f32<T>(sl.p[at]) : 0.f;
    insert(in && order_of(v) >= least ? key_of(v, c0 + at) : 0, k, list);
  }
  sh.list[warp][lane] = list;
  __syncthreads();
  return merge_warps(sh.list, list);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, TOP ? 5 : 4) logprob_kernel(LogProbArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int size = cl::size(), rank = cl::rank();
  if constexpr (TOP) sh.lists[warp][lane] = 0;
  __syncwarp();
  if (size > 1) cl::arrive();  // waited for before the first store to another block
  const long long row = blockIdx.x / size;
  const T* p = static_cast<const T*>(a.logits.p) + row * a.logits.ld;
  const int per = (a.vocab + size - 1) / size;
  const int c0 = min(rank * per, a.vocab), c1 = min(c0 + per, a.vocab);
  const Slice<T> sl(p, c0, c1);
  const float c = a.scale * kLog2E;
  const uint4* body = sl.body();

  Stat st;
  float best = __uint_as_float(0x7FC00000u);  // the largest element, NaN while there is none
  float loose = kLowest;
  if (tid < sl.head + sl.tail) loose = to_f32<T>(sl.p[tid < sl.head ? tid : sl.tail_at(tid - sl.head)]);
  for (int i = tid; i < sl.pieces; i += kBatch * kThreads) {
    uint4 u[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i + b * kThreads < sl.pieces) u[b] = body[i + b * kThreads];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i + b * kThreads >= sl.pieces) break;
      float v[kPer<T>];
      piece_values<T>(u[b], v);
      float top = v[0];
#pragma unroll
      for (int j = 1; j < kPer<T>; ++j) top = fmaxf(top, v[j]);
      if (top > st.m) st.raise(top, c);
      if constexpr (TOP) best = fmaxf(best, top);
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j) st.add(v[j], c);
    }
  }
  if (tid < sl.head + sl.tail) {
    if (loose > st.m) st.raise(loose, c);
    st.add(loose, c);
    best = fmaxf(best, loose);
  }
  Key list = 0;
  if constexpr (TOP) list = block_top<T>(sh, sl, c0, a.top, best, tid < sl.pieces || tid < sl.head + sl.tail);

#pragma unroll
  for (int d = 16; d > 0; d /= 2) st.join(st.shuffled(d), c);
  if (lane == 0) sh.warp[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = lane < kWarps ? sh.warp[lane] : Stat{};
#pragma unroll
    for (int d = kWarps / 2; d > 0; d /= 2) st.join(st.shuffled(d), c);
  }
  if (size > 1) {
    cl::wait();
    if (warp == 0) {
      if (lane == 0) cl::store(cl::peer(&sh.block[rank], 0), make_float4(st.m, st.s, st.q, 0.f));
      if constexpr (TOP) cl::store(cl::peer(&sh.lists[rank][lane], 0), list);
    }
    __syncwarp();
    cl::arrive();
    cl::wait();
    if (rank != 0) return;
    if constexpr (TOP) {
      list = warp < size ? sh.lists[warp][lane] : 0;  // a warp a block
      list = merge_warps(sh.lists, list);
    }
    if (warp != 0) return;
    st = Stat{};
    if (lane < size) st.m = sh.block[lane].x, st.s = sh.block[lane].y, st.q = sh.block[lane].z;
#pragma unroll
    for (int d = kMaxCluster / 2; d > 0; d /= 2) st.join(st.shuffled(d), c);
  }
  if (warp != 0) return;
  // Lane 0 has them all.  A row without a logit above -infinity has no distribution.
  const float m = __shfl_sync(0xffffffffu, st.m, 0), s = __shfl_sync(0xffffffffu, st.s, 0);
  const float logs = s == 0.f ? INFINITY : logf(s);
  if (lane == 0) {
    const float entropy = s == 0.f ? 0.f : logs - a.scale * (st.q / s);
    if (a.logp != nullptr) {
      const long long y = target_at(a.targets, row);
      a.logp[row] = y >= 0 && y < a.vocab ? fmaf(a.scale, to_f32<T>(p[y]) - m, -logs) : 0.f;
    }
    if (a.entropy != nullptr) a.entropy[row] = entropy;
    if (a.stats != nullptr) {
      a.stats[3 * row] = m;
      a.stats[3 * row + 1] = logs;
      a.stats[3 * row + 2] = entropy;
    }
  }
  if constexpr (TOP) {
    if (lane < a.top) {
      const long long at = row * a.top + lane;
      if (a.top_values != nullptr)
        a.top_values[at] = fmaf(a.scale, of_order(static_cast<uint32_t>(list >> 32)) - m, -logs);
      if (a.top_ids != nullptr) a.top_ids[at] = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(list));
    }
  }
}

// --------------------------------------------------------------------------
// Gradient: with g = dlogp, e = dentropy and p_j = e^(s (l_j - m)) / S,
//   dl_j = s (g [j = y] - p_j (g + e (log p_j + H))).
// A block takes kBatch pieces a thread of one row.
// --------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void put(T* p, float v) { *p = from_f32<T>(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_grad_kernel(LogProbGradArgs a, int slices, int per) {
  pdl_trigger();
  pdl_wait();
  const long long row = blockIdx.x / slices;
  const int c0 = static_cast<int>(blockIdx.x % slices) * per, c1 = min(c0 + per, a.vocab);
  const T* in = static_cast<const T*>(a.logits.p) + row * a.logits.ld;
  T* out = static_cast<T*>(a.dlogits.p) + row * a.dlogits.ld;
  const long long yt = target_at(a.targets, row);
  const int y = yt >= 0 && yt < a.vocab ? static_cast<int>(yt) : -1;
  const float m = a.stats[3 * row], logs = a.stats[3 * row + 1], entropy = a.stats[3 * row + 2];
  const bool empty = logs == INFINITY;
  const float g = y >= 0 && a.dlogp != nullptr && !empty ? a.scale * a.dlogp[row] : 0.f;
  const float e = a.dentropy != nullptr && !empty ? a.scale * a.dentropy[row] : 0.f;
  const bool zero = g == 0.f && e == 0.f;
  auto value = [&](float l, int column) {
    const float lp = max_nan(fmaf(a.scale, l - m, -logs), -200.f), pj = exp2_fast(lp * kLog2E);  // e^-200 is 0
    const float v = -pj * (e == 0.f ? g : fmaf(e, lp + entropy, g));
    return column == y ? v + g : v;
  };
  const Slice<T> sl(in, c0, c1);
  const bool together = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  if (!together) {  // rows that begin at different places of a 16-byte piece: by elements, eight in flight
    constexpr int kAhead = 8;
#pragma unroll 1
    for (int j0 = c0 + threadIdx.x; j0 < c1; j0 += kAhead * kThreads) {
      T l[kAhead];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) l[b] = zero ? from_f32<T>(0.f) : in[min(j0 + b * kThreads, c1 - 1)];
#pragma unroll
      for (int b = 0; b < kAhead; ++b) {
        const int j = j0 + b * kThreads;
        if (j < c1) put<T>(out + j, zero ? 0.f : value(to_f32<T>(l[b]), j));
      }
    }
    return;
  }
  if (threadIdx.x < sl.head + sl.tail) {
    const int j = c0 + (threadIdx.x < sl.head ? threadIdx.x : sl.tail_at(threadIdx.x - sl.head));
    put<T>(out + j, zero ? 0.f : value(to_f32<T>(in[j]), j));
  }
  uint4* to = reinterpret_cast<uint4*>(out + c0 + sl.head);
  uint4 u[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int i = threadIdx.x + b * kThreads;
    if (i < sl.pieces) u[b] = zero ? make_uint4(0u, 0u, 0u, 0u) : sl.body()[i];
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int i = threadIdx.x + b * kThreads;
    if (i >= sl.pieces) break;
    if (!zero) {
      float v[kPer<T>];
      piece_values<T>(u[b], v);
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j) v[j] = value(v[j], c0 + sl.piece_at(i) + j);
      if constexpr (sizeof(T) == 4) {
        u[b] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      } else {
        constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
        u[b] = make_uint4(pack2<kBf>(v[0], v[1]), pack2<kBf>(v[2], v[3]), pack2<kBf>(v[4], v[5]),
                          pack2<kBf>(v[6], v[7]));
      }
    }
    to[i] = u[b];
  }
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
template <typename T>
cudaError_t forward(const LogProbArgs& a, cudaStream_t s) {
  // Blocks for several warps a scheduler, as long as one has some pieces a thread.
  int size = 1;
  while (size < kMaxCluster && static_cast<long long>(a.rows) * size < 6ll * sm_count() &&
         a.vocab / (2 * size) >= 2 * kThreads * kPer<T>)
    size *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * size);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(size), 1u, 1u};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, a.top > 0 ? logprob_kernel<T, true> : logprob_kernel<T, false>, a);
}
template <typename T>
cudaError_t backward(const LogProbGradArgs& a, cudaStream_t s) {
  const int per = kBatch * kThreads * kPer<T>;
  const int slices = (a.vocab + per - 1) / per;
  return launch_kernel(pdl_enabled(), logprob_grad_kernel<T>, dim3(static_cast<unsigned>(a.rows) * slices),
                       dim3(kThreads), 0, s, a, slices, per);
}

}  // namespace

cudaError_t launch_log_probs(const LogProbArgs& a, cudaStream_t s) {
  if (a.dtype == kF32) return forward<float>(a, s);
  if (a.dtype == kBF16) return forward<__nv_bfloat16>(a, s);
  return forward<__half>(a, s);
}
cudaError_t launch_log_probs_grad(const LogProbGradArgs& a, cudaStream_t s) {
  if (a.dtype == kF32) return backward<float>(a, s);
  if (a.dtype == kBF16) return backward<__nv_bfloat16>(a, s);
  return backward<__half>(a, s);
}

}  // namespace dion3
