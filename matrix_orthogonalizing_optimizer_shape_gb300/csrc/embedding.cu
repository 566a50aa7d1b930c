// Token embedding and its gradient on sm_103a.  Both are bound by HBM.
//
// The gradient sums the rows of dy that belong to one token.  Which rows those
// are is found without a sort of the whole vocabulary: the tokens are grouped by
// the low bits of their number, a block a group (group_kernel), then summed in
// windows of equal numbers of positions (window_kernel), so that a token that
// makes up a tenth of the batch costs no block more than any other; runs that cross
// windows are joined in order by the last block of them.  No atomic touches a sum:
// the result's bits depend on the ids alone.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "layer_math.cuh"
#include "model.h"

namespace dion3 {
namespace {

using namespace lm;

__device__ __forceinline__ long long id_at(const Ids& ids, long long i) {
  return ids.bytes == 8 ? static_cast<const long long*>(ids.p)[i] : static_cast<const int*>(ids.p)[i];
}

// VEC elements as they lie in memory: loads of several are in flight before the
// first is unpacked (unpacking each behind its own condition made them wait for one
// another, 72 us instead of 25 for the sums of 16384 x 4096).
template <typename T, int VEC>
struct Raw {
  static constexpr int kPieces = VEC == 8 ? static_cast<int>(sizeof(T)) / 2 : 1;
  std::conditional_t<VEC == 8, uint4, T> w[kPieces];
  __device__ __forceinline__ void load(const T* p, bool in = true) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (VEC == 8)
        w[i] = in ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
      else
        w[i] = in ? *p : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void values(float (&v)[VEC]) const {
    if constexpr (VEC == 1) {
      v[0] = to_f32<T>(w[0]);
    } else {
      constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            v[4 * i + j] = __uint_as_float(x[j]);
          } else {
            const float2 f = unpack2<kBf>(x[j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
          }
        }
      }
    }
  }
};

// --------------------------------------------------------------------------
// Lookup.  blockDim = (lanes along a row, rows); a thread keeps its columns and
// walks kWalk rows, all their loads issued before the first is used.  VEC = 8
// columns at a time, or 1 where rows are not whole aligned pieces.  16384 x 4096
// bf16 of 131072 rows: 46 us, 5.9 TB/s.
// --------------------------------------------------------------------------
constexpr int kWalk = 4;
template <int VEC>
constexpr int kStrips = VEC == 8 ? 1 : 4;  // of blockDim.x columns that a thread takes of a row

template <typename W, typename T, int VEC>
__global__ void __launch_bounds__(256) embedding_kernel(EmbedArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int S = kStrips<VEC>;
  const int c0 = (blockIdx.x * blockDim.x * S + threadIdx.x) * VEC, apart = blockDim.x * VEC;
  const long long step = static_cast<long long>(gridDim.y) * blockDim.y;
  for (long long t = static_cast<long long>(blockIdx.y) * blockDim.y + threadIdx.y; t < a.tokens; t += kWalk * step) {
    long long id[kWalk];
    Raw<W, VEC> raw[kWalk][S];
#pragma unroll
    for (int i = 0; i < kWalk; ++i) id[i] = t + i * step < a.tokens ? id_at(a.ids, t + i * step) : -1;
#pragma unroll
    for (int i = 0; i < kWalk; ++i) {
      const bool ok = id[i] >= 0 && id[i] < a.vocab;
      const W* p = static_cast<const W*>(a.table.p) + id[i] * a.table.ld + c0;
#pragma unroll
      for (int j = 0; j < S; ++j) raw[i][j].load(p + j * apart, ok && c0 + j * apart < a.cols);
    }
#pragma unroll
    for (int i = 0; i < kWalk; ++i) {
      if (t + i * step >= a.tokens) break;
      T* y = static_cast<T*>(a.y.p) + (t + i * step) * a.y.ld + c0;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (c0 + j * apart >= a.cols) break;
        float v[VEC];
        raw[i][j].values(v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] *= a.scale;
        store_vec<T, VEC>(y + j * apart, v);
      }
    }
  }
}

// --------------------------------------------------------------------------
// Groups.  Block b takes the tokens with id mod blocks = b (a power of two):
// frequent tokens have neighbouring numbers in most vocabularies, and land in
// different blocks.  Every block reads all ids (from L2: 64 kB at 16384 tokens),
// counts its own by token and warp, and lays their positions out behind those of
// the blocks before it, which it counts on the way.  A warp takes a contiguous
// part of the positions in order, so a token's positions end up ascending; it
// keeps those of its block in shared memory, and reads the ids again only where
// they are too many.
// --------------------------------------------------------------------------
constexpr int kGroupWarps = 16, kGroupThreads = 32 * kGroupWarps;
constexpr int kMaxLocals = 512;  // tokens of a block: counters in 34 kB of shared memory
constexpr int kMinGroups = 256;

constexpr int kIdsAhead = 16;    // ids a lane has in flight
constexpr int kListed = 64;      // of a warp's own positions kept from the first walk

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

__global__ void __launch_bounds__(kGroupThreads) group_kernel(EmbedGradArgs a, int log_groups, int locals, int counters) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ int cnt[];  // [kGroupWarps][locals]
  __shared__ int2 listed[kGroupWarps][kListed];  // position, token
  __shared__ int before_s, wsum[kGroupWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int mine = blockIdx.x, mask = (1 << log_groups) - 1;
  for (int i = threadIdx.x; i < kGroupWarps * locals; i += kGroupThreads) cnt[i] = 0;
  for (int i = blockIdx.x * kGroupThreads + threadIdx.x; i < counters; i += gridDim.x * kGroupThreads) a.arrived[i] = 0;
  if (threadIdx.x == 0) before_s = 0;
  __syncthreads();

  constexpr int kStep = 32 * kIdsAhead;
  const int slice = ((a.tokens + kGroupWarps - 1) / kGroupWarps + kStep - 1) / kStep * kStep;
  const int lo = static_cast<int>(min(static_cast<long long>(warp) * slice, static_cast<long long>(a.tokens)));
  const int hi = static_cast<int>(min(static_cast<long long>(lo) + slice, static_cast<long long>(a.tokens)));
  int* own = cnt + warp * locals;
  // The tokens at i0 + 32 u + lane, -1 where there is none.
  auto load = [&](int i0, int (&id)[kIdsAhead]) {
    if (a.ids.bytes == 8) {
      int2 v[kIdsAhead];
#pragma unroll
      for (int u = 0; u < kIdsAhead; ++u)
        v[u] = i0 + 32 * u + lane < hi ? static_cast<const int2*>(a.ids.p)[i0 + 32 * u + lane] : make_int2(-1, -1);
#pragma unroll
      for (int u = 0; u < kIdsAhead; ++u)
        id[u] = v[u].y == 0 && static_cast<unsigned>(v[u].x) < static_cast<unsigned>(a.vocab) ? v[u].x : -1;
    } else {
      int v[kIdsAhead];
#pragma unroll
      for (int u = 0; u < kIdsAhead; ++u)
        v[u] = i0 + 32 * u + lane < hi ? static_cast<const int*>(a.ids.p)[i0 + 32 * u + lane] : -1;
#pragma unroll
      for (int u = 0; u < kIdsAhead; ++u) id[u] = static_cast<unsigned>(v[u]) < static_cast<unsigned>(a.vocab) ? v[u] : -1;
    }
  };
  int before = 0, found = 0;
  for (int i0 = lo; i0 < hi; i0 += kStep) {
    int id[kIdsAhead];
    load(i0, id);
#pragma unroll
    for (int u = 0; u < kIdsAhead; ++u) {
      const int g = id[u] < 0 ? INT_MAX : id[u] & mask;
      before += g < mine;
      const bool hit = g == mine;
      const unsigned hits = __ballot_sync(0xffffffffu, hit);
      if (hits == 0u) continue;
      if (hit) {
        atomicAdd(own + (id[u] >> log_groups), 1);
        const int at = found + __popc(hits & ((1u << lane) - 1u));
        if (at < kListed) listed[warp][at] = make_int2(i0 + 32 * u + lane, id[u]);
      }
      found += __popc(hits);
    }
  }
  before = warp_sum(before);
  if (lane == 0) atomicAdd(&before_s, before);
  __syncthreads();

  // Where each warp's part of each token starts.
  int sum = 0;
  if (threadIdx.x < locals) {
    for (int w = 0; w < kGroupWarps; ++w) {
      const int n = cnt[w * locals + threadIdx.x];
      cnt[w * locals + threadIdx.x] = sum;
      sum += n;
    }
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int n = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += n;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int base = before_s + incl - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  if (threadIdx.x < locals)
    for (int w = 0; w < kGroupWarps; ++w) cnt[w * locals + threadIdx.x] += base;
  if (threadIdx.x == kGroupThreads - 1 && mine == mask) *a.count = base + sum;
  __syncthreads();

  if (threadIdx.x < locals && !a.accumulate) a.occurs[static_cast<long long>(mine) * locals + threadIdx.x] = sum != 0;

  auto lay = [&](bool hit, int position, int id) {
    const unsigned hits = __ballot_sync(0xffffffffu, hit);
    if (hits == 0u) return;
    if (hit) {
      const int local = id >> log_groups;
      const unsigned same = __match_any_sync(hits, local);
      const int at = own[local] + __popc(same & ((1u << lane) - 1u));
      a.order[at] = position;
      a.token[at] = id;
      __syncwarp(hits);
      if ((same >> lane) == 1u) own[local] = at + 1;  // the last of them
    }
    __syncwarp();
  };
  if (found <= kListed) {
    for (int i = 0; i < found; i += 32) {
      const int2 e = i + lane < found ? listed[warp][i + lane] : make_int2(0, 0);
      lay(i + lane < found, e.x, e.y);
    }
  } else {
    for (int i0 = lo; i0 < hi; i0 += kStep) {
      int id[kIdsAhead];
      load(i0, id);
#pragma unroll
      for (int u = 0; u < kIdsAhead; ++u) lay(id[u] >= 0 && (id[u] & mask) == mine, i0 + 32 * u + lane, id[u]);
    }
  }
}

// --------------------------------------------------------------------------
// Sums.  A window is `window` grouped positions; a block takes one window of one
// strip of columns, walks its rows kBatch at a time with all their loads in
// flight, and writes a token's row when its run ends.  Each warp also writes
// zeros to its share of the rows of tokens that do not occur, some at every batch: the
// memory takes no more than 6.4 TB/s of writes alone, and reads wait behind as many as
// are sent ahead of them (16384 x 4096 under 131072 tokens: 212 us; with all zeros sent
// at once 400, in a launch of their own before the sums 260).  A run that reaches over
// the window's first or last position leaves its sum in fp32 instead: slot 0 of
// the window if it began before, else slot 1 (joined in a launch of its own the
// gradient of 216 x 1054 took 13.4 us on the device).
// --------------------------------------------------------------------------
constexpr int kMaxWindow = 512;
constexpr int kZeros = 8192;    // bytes of shared zeros
constexpr int kZerosAhead = 16;  // rows of a warp being written: enough of short ones

// A warp's share of the rows of tokens that do not occur, written by bulk copies of
// shared zeros, some at a time.
struct ZeroRows {
  const EmbedGradArgs& a;
  int log_groups, locals, lane;
  long long r0, hi;   // the rows whose bits are in todo begin at r0; all end at hi
  unsigned todo = 0;
  long long bytes, pitch;
  uint8_t* out;
  uint32_t from;
  bool pieces;
  __device__ __forceinline__ ZeroRows(const EmbedGradArgs& args, int log_g, int l, const uint4* zeros)
      : a(args), log_groups(log_g), locals(l), lane(threadIdx.x % 32) {
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    hi = a.accumulate ? 0 : a.vocab * (warp + 1) / warps;
    r0 = (a.accumulate ? 0 : a.vocab * warp / warps) - 32;
    const int es = a.table_dtype == kF32 ? 4 : 2;
    bytes = static_cast<long long>(a.cols) * es, pitch = a.dtable.ld * es;
    out = static_cast<uint8_t*>(a.dtable.p);
    from = static_cast<uint32_t>(__cvta_generic_to_shared(zeros));
    pieces = ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(bytes) | static_cast<uintptr_t>(pitch)) & 15u) == 0;
  }
  // Up to `most` rows; false: none is left.
  __device__ __forceinline__ bool some(int most) {
    while (most > 0) {
      while (todo == 0u) {
        r0 += 32;
        if (r0 >= hi) return false;
        const long long row = r0 + lane, slot = (row & ((1 << log_groups) - 1)) * locals + (row >> log_groups);
        todo = __ballot_sync(0xffffffffu, row < hi && a.occurs[row < hi ? slot : 0] == 0);
      }
      uint8_t* p = out + (r0 + __ffs(todo) - 1) * pitch;
      todo &= todo - 1;
      --most;
      if (pieces) {
        if (lane == 0) {
          for (long long i = 0; i < bytes; i += kZeros)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p + i), "r"(from),
                         "r"(static_cast<int>(min(bytes - i, static_cast<long long>(kZeros))))
                         : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group %0;" ::"n"(kZerosAhead - 1) : "memory");
        }
      } else {  // elements up to an aligned piece, pieces, elements
        const int es = a.table_dtype == kF32 ? 4 : 2;
        const long long head = min(bytes, static_cast<long long>(-reinterpret_cast<uintptr_t>(p) & 15u));
        const long long body = (bytes - head) / 16, tail = head + 16 * body;
        for (long long i = lane; i < body; i += 32) reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0u, 0u, 0u, 0u);
        const int i = lane * es, j = i - static_cast<int>(head);  // of the head, else of the tail
        uint8_t* e = i < head ? p + i : tail + j < bytes ? p + tail + j : nullptr;
        if (e != nullptr) {
          if (es == 4)
            *reinterpret_cast<uint32_t*>(e) = 0u;
          else
            *reinterpret_cast<uint16_t*>(e) = 0u;
        }
      }
    }
    return true;
  }
  __device__ __forceinline__ void finish() {
    while (some(kZerosAhead)) {
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
};

template <int VEC>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, int token, int c, const float (&sum)[VEC]) {
  const long long at = static_cast<long long>(token) * a.dtable.ld + c;
  auto put = [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    float v[VEC];
    if (a.accumulate) {
      load_vec<T, VEC>(p + at, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = fmaf(sum[j], a.scale, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = sum[j] * a.scale;
    }
    store_vec<T, VEC>(p + at, v);
  };
  if (a.table_dtype == kF32)
    put(static_cast<float*>(a.dtable.p));
  else if (a.table_dtype == kBF16)
    put(static_cast<__nv_bfloat16*>(a.dtable.p));
  else
    put(static_cast<__half*>(a.dtable.p));
}

// A run over several windows: each of them that has left its sum counts itself at the
// first one's counter, and the last to do so adds them all, in the windows' order
// whichever it is.  Called by all threads of a block, `index` being its window.
template <int VEC>
__device__ __forceinline__ void contribute(const EmbedGradArgs& a, int window, int n, int index, int strips, int strip,
                                           int t, bool began_before, bool goes_on, int c) {
  __shared__ int last;
  int first = index, end = index;  // windows of the run
  if (began_before) {
    for (first = index - 1;;) {
      const int w = first - static_cast<int>(threadIdx.x);  // a window that the run may have come into from before
      const int got = __syncthreads_count(w > 0 && a.token[max(w, 1) * window - 1] == t);
      first -= got;
      if (got < static_cast<int>(blockDim.x)) break;
    }
  }
  if (goes_on) {
    for (;;) {
      const int w = end + 1 + static_cast<int>(threadIdx.x);
      const long long at = static_cast<long long>(w) * window;
      const int got = __syncthreads_count(at < n && a.token[min(at, n - 1ll)] == t);
      end += got;
      if (got < static_cast<int>(blockDim.x)) break;
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.arrived + static_cast<long long>(first) * strips + strip, 1) == end - first;
  __syncthreads();
  const bool mine = last != 0;
  __syncthreads();
  if (!mine || c >= a.cols) return;
  __threadfence();
  float sum[VEC] = {};
  constexpr int kParts = 8;  // in flight
  for (int w0 = first; w0 <= end; w0 += kParts) {
    float v[kParts][VEC];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int w = min(w0 + i, end);
      const float* p = a.partials + (2ll * w + (w == first)) * a.cols + c;
      if constexpr (VEC == 8) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p)), y = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        v[i][4] = y.x, v[i][5] = y.y, v[i][6] = y.z, v[i][7] = y.w;
      } else {
        v[i][0] = __ldcg(p);
      }
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      if (w0 + i > end) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] += v[i][j];
    }
  }
  put_row<VEC>(a, t, c, sum);
}

template <typename T, int VEC>
constexpr int kBatch = VEC == 8 && sizeof(T) == 4 ? 4 : 8;

template <typename T, int VEC>
__global__ void __launch_bounds__(VEC == 8 ? 128 : 256, VEC == 8 ? 5 : 4) window_kernel(EmbedGradArgs a, int window, int strips, int log_groups,
                                                                                   int locals) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(128) uint4 zeros[kZeros / 16];
  __shared__ int pos[kMaxWindow], tok[kMaxWindow + 2];
  const int index = static_cast<int>(blockIdx.x) / strips, strip = static_cast<int>(blockIdx.x) % strips;
  const int n = *a.count, s0 = min(index * window, n), s1 = min(s0 + window, n), len = s1 - s0;
  for (int i = threadIdx.x; i < kZeros / 16; i += blockDim.x) zeros[i] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  for (int i = threadIdx.x; i < len; i += blockDim.x) pos[i] = a.order[s0 + i];
  for (int i = static_cast<int>(threadIdx.x) - 1; i <= len; i += blockDim.x)
    tok[i + 1] = s0 + i >= 0 && s0 + i < n ? a.token[s0 + i] : -1;
  __syncthreads();
  ZeroRows zero(a, log_groups, locals, zeros);
  const int each = static_cast<int>(min((zero.hi - zero.r0 - 32) * kBatch<T, VEC> / window + 1, 1ll << 20));  // at a batch
  const int c = (strip * blockDim.x + threadIdx.x) * VEC;
  const bool in = c < a.cols;
  const T* dy = static_cast<const T*>(a.dy.p) + (in ? c : 0);
  float* part = a.partials + 2ll * index * a.cols + c;
  bool began_before = tok[0] == tok[1];
  const bool head = len > 0 && began_before, tail = len > 0 && tok[len] == tok[len + 1];
  float sum[VEC] = {};
  for (int i0 = 0; i0 < len; i0 += kBatch<T, VEC>) {
    Raw<T, VEC> raw[kBatch<T, VEC>];
#pragma unroll
    for (int i = 0; i < kBatch<T, VEC>; ++i) raw[i].load(dy + static_cast<long long>(pos[min(i0 + i, len - 1)]) * a.dy.ld);
    zero.some(each);
#pragma unroll
    for (int i = 0; i < kBatch<T, VEC>; ++i) {
      if (i0 + i >= len) break;
      float v[VEC];
      raw[i].values(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] += v[j];
      const int t = tok[i0 + i + 1];
      const bool last = i0 + i == len - 1, goes_on = t == tok[i0 + i + 2];
      if (goes_on && !last) continue;
      if (in) {
        if (!goes_on && !began_before)
          put_row<VEC>(a, t, c, sum);
        else
          store_vec<float, VEC>(part + (began_before ? 0 : a.cols), sum);
      }
      began_before = false;
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] = 0.f;
    }
  }
  if (head || tail) {
    const bool through = tail && tok[1] == tok[len];  // one run takes the whole window
    if (head) contribute<VEC>(a, window, n, index, strips, strip, tok[1], true, through, c);
    if (tail && !(head && through)) contribute<VEC>(a, window, n, index, strips, strip, tok[len], false, true, c);
  }
  zero.finish();
}


// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
bool pieces_of(const Mat& m, int dtype, int cols) {  // whole aligned pieces of 8 columns
  const int es = dtype == kF32 ? 4 : 2;
  return cols % 8 == 0 && (reinterpret_cast<uintptr_t>(m.p) & 15u) == 0 && m.ld * es % 16 == 0;
}
int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Calls f with a null pointer of the element type.
template <class F>
cudaError_t with_type(int dtype, F&& f) {
  if (dtype == kF32) return f(static_cast<float*>(nullptr));
  if (dtype == kBF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  return f(static_cast<__half*>(nullptr));
}

}  // namespace

cudaError_t launch_embedding(const EmbedArgs& a, cudaStream_t s) {
  const bool vec = pieces_of(a.table, a.table_dtype, a.cols) && pieces_of(a.y, a.dtype, a.cols);
  const int pieces = ceil_div(a.cols, vec ? 8 * kStrips<8> : kStrips<1>);  // threads of a row
  int lanes = 32;
  while (lanes < 256 && lanes < pieces) lanes *= 2;
  const dim3 block(lanes, 256 / lanes);
  const dim3 grid(ceil_div(pieces, lanes), std::min(65535, ceil_div(a.tokens, kWalk * block.y)));
  return with_type(a.table_dtype, [&](auto* w) {
    return with_type(a.dtype, [&](auto* t) {
      using W = std::remove_pointer_t<decltype(w)>;
      using T = std::remove_pointer_t<decltype(t)>;
      return launch_kernel(pdl_enabled(), vec ? embedding_kernel<W, T, 8> : embedding_kernel<W, T, 1>, grid, block, 0, s,
                           a);
    });
  });
}

// Windows enough for every SM, sums of several rows each: 32 positions at 16384 (more and
// shorter ones leave more partial sums of frequent tokens to add: 14136 x 448 in 39 us,
// in 55 with windows of 8).
int embed_window(int tokens) {
  int w = 8;
  while (w < kMaxWindow && w < (tokens + 511) / 512) w *= 2;
  return w;
}

static int log_groups_of(int vocab) {
  int n = 8;
  static_assert(kMinGroups == 1 << 8, "256 blocks");
  while (ceil_div(vocab, 1ll << n) > kMaxLocals) ++n;
  return n;
}
int embed_counters(int tokens, int cols) { return ceil_div(tokens, embed_window(tokens)) * ceil_div(cols, 256); }
int embed_slots(int vocab) {
  const int n = log_groups_of(vocab);
  return ceil_div(vocab, 1ll << n) << n;
}

cudaError_t launch_embedding_grad(const EmbedGradArgs& a, cudaStream_t s) {
  const int log_groups = log_groups_of(a.vocab), locals = ceil_div(a.vocab, 1ll << log_groups);
  const bool vec = pieces_of(a.dy, a.dtype, a.cols) && pieces_of(a.dtable, a.table_dtype, a.cols);
  const int window = embed_window(a.tokens), windows = ceil_div(a.tokens, window);
  const int pieces = vec ? a.cols / 8 : a.cols;
  const int threads = vec ? 128 : 256, strips = ceil_div(pieces, threads);
  cudaError_t e = launch_kernel(pdl_enabled(), group_kernel, dim3(1u << log_groups), dim3(kGroupThreads),
                                kGroupWarps * locals * sizeof(int), s, a, log_groups, locals, windows * strips);
  if (e != cudaSuccess) return e;
  // Enough blocks for the zeros of a large vocabulary, too.
  const int blocks = a.accumulate ? windows * strips : std::max(windows * strips, 5 * sm_count());
  return with_type(a.dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_kernel(pdl_enabled(), vec ? window_kernel<T, 8> : window_kernel<T, 1>, dim3(blocks), dim3(threads),
                         0, s, a, window, strips, log_groups, locals);
  });
}

}  // namespace dion3
