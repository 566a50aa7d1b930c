// Gated linear recurrence on sm_103a, h_t = a_t h_{t-1} + (1 - a_t) x_t with
// a = sigmoid(z), and its gradient.  Every row is read once and written once; the
// scan happens in registers.
//
// A step h -> a h + b is an affine map, and maps compose: (A, B) after (A', B')
// is (A A', A B' + B).  The blocks of a cluster take 16 VEC channels and walk down the
// rows together, one span of rows behind the other: each thread composes the maps of R
// rows of VEC channels, a few lanes a channel compose those of a block's threads, the
// blocks exchange theirs, and each thread runs through its rows again from the state
// before them, the next rows' loads in flight.  Arithmetic is on pairs of channels
// (one instruction for two).  16384 x 4096 bf16: 80 us by boxes of 32 channels in
// clusters of two (by cp.async of 64 channels in clusters of four 95; of 128 in clusters
// of eight, where more blocks wait for one another, 120; of 16 in none, whose rows are
// sectors of 32 bytes, 157), the gradient 148: 74 and 80 % of what their bytes take.
// What bounds both is latency: 128 registers leave two blocks, 16 warps, an SM (on two
// thirds of the SMs), which stand at two barriers and an exchange a step; 23 and 45
// instructions an element keep the issue slots 53 and 58 % and DRAM 56 and 66 % busy.
// Four rows a thread with three blocks an SM: 125.
//
// Packed sequences: a map that begins a sequence cuts, so that rows are divided
// evenly whatever the sequences' lengths; nothing of the rows before a cut, NaN
// included, passes it.  Warps whose rows hold a boundary pick by it in each row, without
// a branch (64 sequences: 98 us; row by row behind conditions 120).  Where the
// channels are few, groups of whole sequences go to different clusters.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "cluster.cuh"
#include "layer_math.cuh"
#include "model.h"
#include "tc_ops.cuh"

namespace dion3 {
namespace {

using namespace lm;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxCluster = 16;                // past 8 a kernel has to ask
constexpr int kAcross = 16;                    // threads along a block's channels
constexpr int kGroups = kThreads / kAcross;    // groups of rows
constexpr int kSharedOffsets = 1024;

// --------------------------------------------------------------------------
// Vectors of VEC channels, 4 or 2 where they are aligned and else 1.
// --------------------------------------------------------------------------
template <int VEC>
struct Vec {
  float v[VEC];
  __device__ __forceinline__ float& operator[](int j) { return v[j]; }
  __device__ __forceinline__ float operator[](int j) const { return v[j]; }
};
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> fma(const Vec<VEC>& a, const Vec<VEC>& b, const Vec<VEC>& c) {
  Vec<VEC> r;
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      unsigned long long d;
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])),
          "l"(pair(c[j], c[j + 1])));
      unpair(d, r[j], r[j + 1]);
    }
  } else {
    r[0] = fmaf(a[0], b[0], c[0]);
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> mul(const Vec<VEC>& a, const Vec<VEC>& b) {
  Vec<VEC> r;
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      unsigned long long d;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
      unpair(d, r[j], r[j + 1]);
    }
  } else {
    r[0] = a[0] * b[0];
  }
  return r;
}
// a / 2, 0 where that is below 2^-126.
template <int VEC>
__device__ __forceinline__ Vec<VEC> half_of(const Vec<VEC>& a) {
  Vec<VEC> r;
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      unsigned long long d;
      asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(0.5f, 0.5f)));
      unpair(d, r[j], r[j + 1]);
    }
  } else {
    asm("mul.rn.ftz.f32 %0, %1, 0f3F000000;" : "=f"(r[0]) : "f"(a[0]));
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> add(const Vec<VEC>& a, const Vec<VEC>& b) {
  Vec<VEC> r;
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      unsigned long long d;
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a[j], a[j + 1])), "l"(pair(b[j], b[j + 1])));
      unpair(d, r[j], r[j + 1]);
    }
  } else {
    r[0] = a[0] + b[0];
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> all(float x) {
  Vec<VEC> r;
#pragma unroll
  for (int j = 0; j < VEC; ++j) r[j] = x;
  return r;
}

// VEC elements as they lie in memory.
template <typename T, int VEC>
struct Cell {
  static constexpr int kWords = (VEC * static_cast<int>(sizeof(T)) + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC * sizeof(T) == 16) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (VEC * sizeof(T) == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else if constexpr (VEC * sizeof(T) == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ Vec<VEC> values() const {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    Vec<VEC> v;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(w[j]);
    } else if constexpr (VEC == 1) {
      v[0] = unpack1<kBf>(static_cast<uint16_t>(w[0]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j += 2) {
        const float2 f = unpack2<kBf>(w[j / 2]);
        v[j] = f.x;
        v[j + 1] = f.y;
      }
    }
    return v;
  }
};
// What a block has in flight: R cells a thread of each of N matrices, for kAhead steps.
//   kTma    the block's rows as one box of a matrix, where bases and pitches are
//           multiples of 16 bytes and there are steps enough to pay for the maps;
//   kCells  cells of 4 bytes or more by cp.async, to a place of its own for each thread
//           (8 instructions a row and matrix with their addresses);
//   kRegs   in registers, for one step.
// DOWN: a thread's row i is the i-th from its last (the gradient).
enum Way { kTma, kCells, kRegs };
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if (bytes == 16)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
struct TileMaps {
  CUtensorMap m[4];
};
struct NoMaps {};
template <Way WAY>
using MapsOf = std::conditional_t<WAY == kTma, TileMaps, NoMaps>;

template <typename T, int VEC, int R, int N, Way WAY, bool DOWN>
struct Flight {
  static constexpr int kAhead = WAY == kRegs ? 1 : 2;
  static constexpr int kCell = VEC * static_cast<int>(sizeof(T));
  static constexpr int kBox = R * kThreads * kCell;  // bytes of a step's cells of a matrix
  static constexpr size_t kBytes = WAY == kRegs ? 0 : static_cast<size_t>(kAhead) * N * kBox;
  Cell<T, VEC> reg[WAY == kRegs ? N : 1][WAY == kRegs ? R : 1];
  char* mem;
  uint32_t at, bar;
  __device__ __forceinline__ Flight(char* shared, const unsigned long long* full) {
    const int group = threadIdx.x / kAcross, first = DOWN ? kGroups * R - 1 - group * R : group * R;
    mem = shared + (WAY == kTma ? (first * kAcross + threadIdx.x % kAcross) * kCell : threadIdx.x * kCell);
    at = static_cast<uint32_t>(__cvta_generic_to_shared(WAY == kTma ? shared : mem));
    bar = static_cast<uint32_t>(__cvta_generic_to_shared(full));
    if constexpr (WAY == kRegs) {
#pragma unroll
      for (auto& r : reg)
#pragma unroll
        for (auto& cell : r) cell = {};
    }
  }
  // Cell i of matrix n for step `step`.
  __device__ __forceinline__ void load(int step, int n, int i, const T* p) {
    if constexpr (WAY == kCells)
      copy_async(at + ((step % kAhead) * N + n) * kBox + i * kThreads * kCell, p, kCell);
    else if constexpr (WAY == kRegs)
      reg[n][i].load(p);
  }
  __device__ __forceinline__ void loaded() const {  // after the loads of a step
    if constexpr (WAY == kCells) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // kTma, by one thread: the boxes of a step, from row y and channel x (of matrix 2 from the row before).
  __device__ __forceinline__ void issue(int step, const MapsOf<WAY>& maps, int x, int y) const {
    if constexpr (WAY == kTma) {
      const uint32_t b = bar + 8 * (step % kAhead);
      tc::mbar_expect(b, N * kBox);
#pragma unroll
      for (int n = 0; n < N; ++n) tc::tma_load(at + ((step % kAhead) * N + n) * kBox, &maps.m[n], b, x, n == 2 ? y - 1 : y);
    }
  }
  // For a step's cells; false: the wait ran out.
  __device__ __forceinline__ bool wait(int step, unsigned* status) const {
    if constexpr (WAY == kTma) return tc::mbar_wait_warp(bar + 8 * (step % kAhead), step / kAhead & 1, status);
    if constexpr (WAY == kCells) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    return true;
  }
  __device__ __forceinline__ Vec<VEC> values(int step, int n, int i) const {
    if constexpr (WAY == kRegs) {
      return reg[n][i].values();
    } else {
      constexpr int kRow = WAY == kTma ? (DOWN ? -1 : 1) * kAcross * kCell : kThreads * kCell;  // from row to row of a thread
      Cell<T, VEC> c;
      c.load(reinterpret_cast<const T*>(mem + ((step % kAhead) * N + n) * kBox + i * kRow));
      return c.values();
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_cell(T* p, const Vec<VEC>& v) {
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  if constexpr (VEC == 1)
    *p = from_f32<T>(v[0]);
  else if constexpr (sizeof(T) == 4 && VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<kBf>(v[0], v[1]), pack2<kBf>(v[2], v[3]));
  else
    *reinterpret_cast<uint32_t*>(p) = pack2<kBf>(v[0], v[1]);
}
// State vectors are fp32 with the channels' alignment unknown: element by element.
template <int VEC>
__device__ __forceinline__ Vec<VEC> load_state(const float* p) {
  Vec<VEC> v;
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = p[j];
  return v;
}
template <int VEC>
__device__ __forceinline__ void store_state(float* p, const Vec<VEC>& v) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) p[j] = v[j];
}

template <int VEC>
__device__ __forceinline__ Vec<VEC> pick(bool first, const Vec<VEC>& a, const Vec<VEC>& b) {
  Vec<VEC> r;
#pragma unroll
  for (int j = 0; j < VEC; ++j) r[j] = first ? a[j] : b[j];
  return r;
}
// to[i] = the state of a sequence at the rows whose bits are in `at`, else 0; the first
// is q's, and bits of `past` step to the next one.
template <int VEC, int R, class Next>
__device__ __forceinline__ void load_states(Vec<VEC> (&to)[R], const float* from, unsigned at, unsigned past, int q,
                                            Next&& next, int channels, int c) {
#pragma unroll
  for (int i = 0; i < R; ++i) to[i] = all<VEC>(0.f);
  if (from == nullptr || at == 0u) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (at >> i & 1) to[i] = load_state<VEC>(from + static_cast<long long>(q) * channels + c);
    if (past >> i & 1) q = next(q);
  }
}

// --------------------------------------------------------------------------
// Gates.  With u = e^-z / 2 and r = 1 / (u + 1/2), by two special function
// instructions, a = r / 2 and 1 - a = u r: each accurate relative to itself, to some
// units of 2^-23 for small |z| and to 6e-6 at |z| = 87, where the exponent's argument is
// rounded at 2^-18.  u stops at 2^126, where r is 2^-126 and the product still 1; halving
// flushes, so that a is 0 there (as everywhere below 2^-126; 1 - a is below 2^-125):
// z = -infinity forgets.
// --------------------------------------------------------------------------
template <int VEC>
struct Gate {
  Vec<VEC> a, na;
  __device__ __forceinline__ explicit Gate(const Vec<VEC>& z) {
    const Vec<VEC> e = fma(z, all<VEC>(-kLog2E), all<VEC>(-1.f));
    Vec<VEC> u, r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(u[j]) : "f"(e[j]));
      asm("min.NaN.f32 %0, %1, 0f7E800000;" : "=f"(u[j]) : "f"(u[j]));
    }
    const Vec<VEC> s = add(u, all<VEC>(0.5f));
#pragma unroll
    for (int j = 0; j < VEC; ++j) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[j]) : "f"(s[j]));
    na = mul(u, r);
    a = half_of(r);
  }
};

// --------------------------------------------------------------------------
// Maps h -> A h + B, with D = 1 - A summed for itself: where A is above a half a
// map is applied as h - D h + B, since a factor near 1 that were rounded would decay
// the state at a rate that is off in every one of thousands of rows.  D = 2 cuts:
// nothing passes.  Between blocks a map's factor is one number: A up to a half, else
// -D with its sign bit set, or 2.  An infinite h stays infinite by A and becomes NaN by
// -D, and by an A that has underflowed: never finite, which is all that is promised (a
// select by |h| could not tell an underflowed A from a gate of 0).
// --------------------------------------------------------------------------
constexpr float kCut = 2.f;
__device__ __forceinline__ float through(float A, float D, float B, float h) {
  const bool near = D < 0.5f;
  const float r = fmaf(near ? -D : A, h, B) + (near ? h : 0.f);
  return D == kCut ? B : r;
}
__device__ __forceinline__ float encode(float A, float D) { return D == kCut ? kCut : D < 0.5f ? -D : A; }
__device__ __forceinline__ float pass_block(float F, float B, float h) {
  const float r = fmaf(F, h, B) + (static_cast<int>(__float_as_uint(F)) < 0 ? h : 0.f);
  return F == kCut ? B : r;
}
// A thread's map.
template <int VEC>
struct Map {
  Vec<VEC> A = all<VEC>(1.f), D = all<VEC>(0.f), B = all<VEC>(0.f);
  __device__ __forceinline__ void factor(const Gate<VEC>& g) {
    D = fma(g.na, A, D);
    A = mul(g.a, A);
  }
  // The product's factors are rounded numbers near 1, the same in row after row of a
  // steady gate: taken from D, A is off by less than one of those roundings.
  __device__ __forceinline__ Vec<VEC> kept() const {
    Vec<VEC> r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = D[j] < 0.875f ? 1.f - D[j] : A[j];
    return r;
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
  __device__ __forceinline__ int of(int row) const { return n == 1 ? 0 : max(starts_below(row, true) - 1, 0); }
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
__device__ __forceinline__ void copy_empty(const Span& p, const float* from, float* to, int channels, int c, int group,
                                           bool in) {
  for (int q = p.s0 + group; q < p.s1; q += kGroups) {
    if (p.seq.off[q + 1] > p.seq.off[q] || !in) continue;
    const long long at = static_cast<long long>(q) * channels + c;
    store_state<VEC>(to + at, from != nullptr ? load_state<VEC>(from + at) : all<VEC>(0.f));
  }
}

// The sequence of a warp's row, kept from step to step.
struct Place {
  int q = 0, begin = INT_MAX, end = INT_MIN;
  __device__ __forceinline__ void set(const Sequences& s, int to) { q = to, begin = s.off[to], end = s.off[to + 1]; }
  __device__ __forceinline__ void find(const Sequences& s, int row) {
    if (row < begin || row >= end) set(s, s.of(row));
  }
};

// --------------------------------------------------------------------------
// The states before each thread's rows, from the maps of all and the state before
// the cluster's rows, which kLanes neighbouring lanes a channel keep.  A block's map
// goes to the others of the cluster by stores that complete on an mbarrier of theirs,
// so that no fence waits for this block's own stores of rows.
// --------------------------------------------------------------------------
template <int VEC>
struct Shared {
  static constexpr int kTile = kAcross * VEC;        // channels of a block
  static constexpr int kLanes = kThreads / kTile;    // that compose a channel's maps
  static constexpr int kMaps = kGroups / kLanes;     // of each of them
  float A[kGroups][kTile], D[kGroups][kTile], B[kGroups][kTile];  // the groups' maps, columns by at()
  float enter[kGroups][kTile];                                    // the states
  float2 block[2][kMaxCluster][kTile];                            // of the cluster's blocks, in turn in two halves
  unsigned long long bar[2];                                      // of the halves
  unsigned long long full[2];                                     // of the boxes in flight
  // Waits that ran out: for rows, written before a step's first barrier and read behind
  // it, and for maps, written between its two barriers and read behind the second.  No
  // warp can write one while another of the block has yet to read it, so that all threads
  // leave at the same step.
  int late, stop;
  int off[kSharedOffsets];
  // A warp reads 32 / kLanes channels of kLanes groups at once: each from other banks.
  static __device__ __forceinline__ int at(int group, int c) { return (c + group / kMaps * (32 / kLanes)) % kTile; }
};
template <int VEC>
__device__ __forceinline__ void put(float* p, const Vec<VEC>& v) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else if constexpr (VEC == 2)
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else
    *p = v[0];
}
template <int VEC>
__device__ __forceinline__ Vec<VEC> get(const float* p) {
  Vec<VEC> v;
  if constexpr (VEC == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else if constexpr (VEC == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x, v[1] = f.y;
  } else {
    v[0] = *p;
  }
  return v;
}
// Before the first step, by all threads.
template <int VEC>
__device__ __forceinline__ void begin_steps(Shared<VEC>& sh, int size) {
  if (threadIdx.x == 0) {
    sh.late = sh.stop = 0;
    for (unsigned long long& b : sh.bar) tc::mbar_init(tc::smem_u32(&b), 1);
    for (unsigned long long& b : sh.full) tc::mbar_init(tc::smem_u32(&b), 1);
    tc::mbar_init_fence();
  }
  __syncthreads();
  if (size > 1) cl::arrive(), cl::wait();  // every block has begun before one writes to another
}
// After the last: no block leaves while another may write to it.
__device__ __forceinline__ void end_steps(int size) {
  __syncwarp();
  if (size > 1) cl::arrive(), cl::wait();
}
// (A, D, B) after (A1, D1, B1).
__device__ __forceinline__ void compose(float& A, float& D, float& B, float A1, float D1, float B1) {
  const bool cut = D == kCut;
  B = through(A, D, B, B1);
  D = cut ? kCut : fmaf(D, A1, D1);
  A = cut ? 0.f : A * A1;  // whatever was before a cut, NaN too
}
template <int VEC, class Then>
__device__ __forceinline__ Vec<VEC> enter(Shared<VEC>& sh, int step, int rank, int size, const Map<VEC>& m, bool cut,
                                          float& carry, unsigned* status, bool& stop,
                                          Then&& then) {  // once all have their rows
  using S = Shared<VEC>;
  constexpr int kTile = S::kTile, kLanes = S::kLanes;
  const int group = threadIdx.x / kAcross, own = S::at(group, threadIdx.x % kAcross * VEC), half = step & 1;
  put<VEC>(&sh.A[group][own], cut ? all<VEC>(0.f) : m.kept());
  put<VEC>(&sh.D[group][own], cut ? all<VEC>(kCut) : m.D);
  put<VEC>(&sh.B[group][own], m.B);
  __syncthreads();
  const bool late = sh.late;
  then();
  const int c = threadIdx.x / kLanes, k = threadIdx.x % kLanes;
  float a[S::kMaps], d[S::kMaps], b[S::kMaps];
#pragma unroll
  for (int i = 0; i < S::kMaps; ++i) {
    const int w = k * S::kMaps + i;
    a[i] = sh.A[w][S::at(w, c)], d[i] = sh.D[w][S::at(w, c)], b[i] = sh.B[w][S::at(w, c)];
  }
  float A = a[0], D = d[0], B = b[0];
#pragma unroll
  for (int i = 1; i < S::kMaps; ++i) {
    float A2 = a[i], D2 = d[i], B2 = b[i];
    compose(A2, D2, B2, A, D, B);
    A = A2, D = D2, B = B2;
  }
#pragma unroll
  for (int n = 1; n < kLanes; n *= 2) {  // of the channel's lanes up to this one
    const float A1 = __shfl_up_sync(0xffffffffu, A, n, kLanes), D1 = __shfl_up_sync(0xffffffffu, D, n, kLanes),
                B1 = __shfl_up_sync(0xffffffffu, B, n, kLanes);
    if (k >= n) compose(A, D, B, A1, D1, B1);
  }
  const float F = encode(A, D);
  const float allF = __shfl_sync(0xffffffffu, F, kLanes - 1, kLanes);
  const float allB = __shfl_sync(0xffffffffu, B, kLanes - 1, kLanes);
  const float F1 = __shfl_up_sync(0xffffffffu, F, 1, kLanes), B1 = __shfl_up_sync(0xffffffffu, B, 1, kLanes);
  float h = carry;
  if (size > 1) {
    if (threadIdx.x == 0) tc::mbar_expect(tc::smem_u32(&sh.bar[half]), size * kTile * sizeof(float2));
    for (int r = k; r < size; r += kLanes)
      cl::store_async(cl::peer(&sh.block[half][rank][c], r), make_float2(allF, allB), cl::peer(&sh.bar[half], r));
    if (!tc::mbar_wait_warp(tc::smem_u32(&sh.bar[half]), (step >> 1) & 1, status)) sh.stop = 1;
    for (int r = 0; r < size; ++r) {
      if (r == rank) h = carry;
      const float2 f = sh.block[half][r][c];
      carry = pass_block(f.x, f.y, carry);
    }
  } else {
    carry = pass_block(allF, allB, carry);
  }
  if (k > 0) h = pass_block(F1, B1, h);
#pragma unroll
  for (int i = 0; i < S::kMaps; ++i) {
    sh.enter[k * S::kMaps + i][S::at(k * S::kMaps + i, c)] = h;
    if (i + 1 < S::kMaps) h = through(a[i], d[i], b[i], h);
  }
  __syncthreads();
  stop = late || sh.stop;
  return get<VEC>(&sh.enter[group][own]);
}

template <typename T, int VEC, int R, Way WAY>
__global__ void __launch_bounds__(kThreads, 2) recurrence_kernel(RecurrenceArgs a, const __grid_constant__ MapsOf<WAY> boxes) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) Shared<VEC> sh;
  const int size = cl::size(), rank = cl::rank(), groups = gridDim.x / size;
  const Span p = span_of(a, blockIdx.x / size, groups, sh.off);
  begin_steps<VEC>(sh, size);
  const int group = threadIdx.x / kAcross;
  const int c = (blockIdx.y * kAcross + threadIdx.x % kAcross) * VEC, cr = c < a.channels ? c : 0;
  const bool in = c < a.channels;
  if (a.last != nullptr && rank == 0) copy_empty<VEC>(p, a.first, a.last, a.channels, c, group, in);

  const T* pz = static_cast<const T*>(a.z.p) + cr;
  const T* px = static_cast<const T*>(a.x.p) + cr;
  T* ph = static_cast<T*>(a.h.p) + cr;
  extern __shared__ __align__(128) char flight_mem[];
  using F = Flight<T, VEC, R, 2, WAY, false>;
  F in_flight(flight_mem, sh.full);
  auto load = [&](int step, int row0) {
    const int n = min(p.r1 - row0, R);
    const T *qz = pz + row0 * a.z.ld, *qx = px + row0 * a.x.ld;
    if (n == R) {
#pragma unroll
      for (int i = 0; i < R; ++i, qz += a.z.ld, qx += a.x.ld) {
        in_flight.load(step, 0, i, qz);
        in_flight.load(step, 1, i, qx);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i, qz += a.z.ld, qx += a.x.ld) {
        if (i >= n) break;
        in_flight.load(step, 0, i, qz);
        in_flight.load(step, 1, i, qx);
      }
    }
    in_flight.loaded();
  };
  float carry = 0.f;
  const int stride = size * kGroups * R;
  int row0 = p.r0 + (rank * kGroups + group) * R;
  const int start = row0, x = blockIdx.y * kAcross * VEC;
  auto fetch = [&](int to) {  // what step `to` reads
    if constexpr (WAY != kTma)
      load(to, start + to * stride);
    else if (threadIdx.x == 0 && p.r0 + to * stride < p.r1)
      in_flight.issue(to, boxes, x, p.r0 + rank * kGroups * R + to * stride);
  };
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) fetch(i);
  Place at;
  int step = 0;
  for (int top = p.r0; top < p.r1; top += stride, row0 += stride, ++step) {
    if (!in_flight.wait(step, a.status)) sh.late = 1;
    Map<VEC> m;
    Vec<VEC> f[R];  // a and (1 - a) x of the rows
    Vec<VEC> g[R];
    unsigned begins = 0, ends = 0;
    int q0 = 0;
    bool whole = false;  // whole rows of one sequence, neither its first nor (where that is asked for) its last
    if (row0 < p.r1) {
      at.find(p.seq, row0);
      q0 = at.q;
      whole = row0 + R <= p.r1 && row0 != at.begin && (a.last == nullptr ? row0 + R <= at.end : row0 + R < at.end);
    }
    whole = __all_sync(0xffffffffu, whole);
    if (row0 < p.r1) {
      if (whole) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Gate<VEC> k(in_flight.values(step, 0, i));
          f[i] = k.a;
          g[i] = mul(k.na, in_flight.values(step, 1, i));
          m.factor(k);
          m.B = fma(f[i], m.B, g[i]);
        }
      } else {
        for (int n = 0; n < R; ++n) {  // the sequences of the rows
          if (static_cast<unsigned>(at.begin) - row0 < R) begins |= 1u << (at.begin - row0);
          if (static_cast<unsigned>(at.end) - 1 - row0 >= R) break;
          ends |= 1u << (at.end - 1 - row0);
          if (at.end >= p.r1) break;
          at.set(p.seq, p.seq.next(at.q));
        }
        load_states<VEC, R>(g, a.first, begins, ends, q0, [&](int q) { return p.seq.next(q); }, a.channels, cr);
#pragma unroll
        for (int i = 0; i < R; ++i) {  // rows behind the last are nobody's past
          const Gate<VEC> k(in_flight.values(step, 0, i));
          const bool cut = begins >> i & 1;
          const Vec<VEC> b = mul(k.na, in_flight.values(step, 1, i));
          f[i] = k.a;
          m.B = fma(f[i], pick(cut, g[i], m.B), b);  // the state before a sequence is in g
          g[i] = pick(cut, m.B, b);
          m.factor(k);
        }
      }
    }
    if constexpr (WAY != kTma) fetch(step + F::kAhead);
    bool stop;
    Vec<VEC> h = enter<VEC>(sh, step, rank, size, m, begins != 0u, carry, a.status, stop, [&] {
      if constexpr (WAY == kTma) fetch(step + F::kAhead);
    });
    if (stop) {
      for (int i = 1; i <= F::kAhead && WAY == kTma && top + i * stride < p.r1; ++i) in_flight.wait(step + i, a.status);
      break;
    }
    T* q = ph + static_cast<long long>(row0) * a.h.ld;
    if (whole) {
#pragma unroll
      for (int i = 0; i < R; ++i, q += a.h.ld) {
        h = fma(f[i], h, g[i]);
        if (in) store_cell<T, VEC>(q, h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i, q += a.h.ld) {
        h = pick(begins >> i & 1, g[i], fma(f[i], h, g[i]));
        if (in && row0 + i < p.r1) store_cell<T, VEC>(q, h);
        if (a.last != nullptr && (ends >> i & 1)) {
          if (in) store_state<VEC>(a.last + static_cast<long long>(q0) * a.channels + c, h);
          q0 = p.seq.next(q0);
        }
      }
    }
  }
  end_steps(size);
}

// --------------------------------------------------------------------------
// Gradient: g_t = dh_t + s_{t+1}, s_t = a_t g_t, dx = (1 - a) g and
// dz = dx a (h_{t-1} - x).  The scan runs from the last row to the first; a row's
// map is s -> a s + a dh.  Row i of a warp is the i-th from its end.
// --------------------------------------------------------------------------
template <typename T, int VEC, int R, Way WAY>
__global__ void __launch_bounds__(kThreads, 2) recurrence_grad_kernel(RecurrenceArgs a,
                                                                    const __grid_constant__ MapsOf<WAY> boxes) {
  pdl_trigger();
  pdl_wait();
  __shared__ __align__(16) Shared<VEC> sh;
  const int size = cl::size(), rank = cl::rank(), groups = gridDim.x / size;
  const Span p = span_of(a, blockIdx.x / size, groups, sh.off);
  begin_steps<VEC>(sh, size);
  const int group = threadIdx.x / kAcross;
  const int c = (blockIdx.y * kAcross + threadIdx.x % kAcross) * VEC, cr = c < a.channels ? c : 0;
  const bool in = c < a.channels;
  if (a.dfirst != nullptr && rank == 0) copy_empty<VEC>(p, a.dlast, a.dfirst, a.channels, c, group, in);

  const T* pz = static_cast<const T*>(a.z.p) + cr;
  const T* px = static_cast<const T*>(a.x.p) + cr;
  const T* ph = static_cast<const T*>(a.h.p) + cr;
  const T* pd = static_cast<const T*>(a.dh.p) + cr;
  T* pdz = static_cast<T*>(a.dz.p) + cr;
  T* pdx = static_cast<T*>(a.dx.p) + cr;
  extern __shared__ __align__(128) char flight_mem[];
  using F = Flight<T, VEC, R, 4, WAY, true>;
  F in_flight(flight_mem, sh.full);
  auto load = [&](int step, int row0) {  // of h the row before, where there is one
    const int n = min(row0 - p.r0 + 1, R + 1);
    const T *qz = pz + row0 * a.z.ld, *qx = px + row0 * a.x.ld, *qh = ph + (row0 - 1) * a.h.ld, *qd = pd + row0 * a.dh.ld;
    if (n > R) {
#pragma unroll
      for (int i = 0; i < R; ++i, qz -= a.z.ld, qx -= a.x.ld, qh -= a.h.ld, qd -= a.dh.ld) {
        in_flight.load(step, 0, i, qz);
        in_flight.load(step, 1, i, qx);
        in_flight.load(step, 2, i, qh);
        in_flight.load(step, 3, i, qd);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i, qz -= a.z.ld, qx -= a.x.ld, qh -= a.h.ld, qd -= a.dh.ld) {
        if (i >= n) break;
        in_flight.load(step, 0, i, qz);
        in_flight.load(step, 1, i, qx);
        if (i + 1 < n) in_flight.load(step, 2, i, qh);
        in_flight.load(step, 3, i, qd);
      }
    }
    in_flight.loaded();
  };
  float carry = 0.f;
  const int stride = size * kGroups * R;
  int base = p.r1 - 1 - (rank * kGroups + group) * R;
  const int start = base, x = blockIdx.y * kAcross * VEC;
  auto fetch = [&](int to) {  // what step `to` reads
    if constexpr (WAY != kTma)
      load(to, start - to * stride);
    else if (threadIdx.x == 0 && p.r1 - to * stride > p.r0)
      in_flight.issue(to, boxes, x, p.r1 - (rank + 1) * kGroups * R - to * stride);
  };
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) fetch(i);
  Place at;
  int step = 0;
  for (int top = p.r1; top > p.r0; top -= stride, base -= stride, ++step) {
    const bool any = base >= p.r0;
    if (!in_flight.wait(step, a.status)) sh.late = 1;
    const int row0 = any ? base : p.r0;
    Map<VEC> m;
    Vec<VEC> ga[R], gn[R], dv[R], diff[R];  // a, 1 - a, dh and h_{t-1} - x of the rows
    unsigned begins = 0, ends = 0;
    int q0 = 0;
    bool whole = false;
    if (any) {
      at.find(p.seq, row0);
      q0 = at.q;
      whole = row0 - R >= p.r0 && row0 + 1 != at.end && row0 - R >= at.begin;
    }
    whole = __all_sync(0xffffffffu, whole);
    if (any) {
      if (whole) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const Gate<VEC> k(in_flight.values(step, 0, i));
          ga[i] = k.a;
          gn[i] = k.na;
          dv[i] = in_flight.values(step, 3, i);
          diff[i] = fma(in_flight.values(step, 1, i), all<VEC>(-1.f), in_flight.values(step, 2, i));
          m.factor(k);
          m.B = mul(ga[i], add(dv[i], m.B));
        }
      } else {
        for (int n = 0; n < R; ++n) {  // the sequences of the rows
          if (static_cast<unsigned>(row0) - at.end + 1 < R) ends |= 1u << (row0 - at.end + 1);
          if (static_cast<unsigned>(row0) - at.begin >= R) break;
          begins |= 1u << (row0 - at.begin);
          if (at.begin <= p.r0) break;
          at.set(p.seq, p.seq.prev(at.q));
        }
        const auto prev = [&](int q) { return p.seq.prev(q); };
        load_states<VEC, R>(dv, a.dlast, ends, begins, q0, prev, a.channels, cr);
        load_states<VEC, R>(diff, a.first, begins, begins, q0, prev, a.channels, cr);
#pragma unroll
        for (int i = 0; i < R; ++i) {  // rows before the first are nobody's future
          const Gate<VEC> k(in_flight.values(step, 0, i));
          ga[i] = k.a;
          gn[i] = k.na;
          dv[i] = add(in_flight.values(step, 3, i), dv[i]);
          diff[i] = fma(in_flight.values(step, 1, i), all<VEC>(-1.f),
                        pick(begins >> i & 1, diff[i], in_flight.values(step, 2, i)));
          m.factor(k);
          m.B = mul(ga[i], add(dv[i], pick(ends >> i & 1, all<VEC>(0.f), m.B)));
        }
      }
    }
    if constexpr (WAY != kTma) fetch(step + F::kAhead);
    bool stop;
    Vec<VEC> s = enter<VEC>(sh, step, rank, size, m, ends != 0u, carry, a.status, stop, [&] {
      if constexpr (WAY == kTma) fetch(step + F::kAhead);
    });
    if (stop) {
      for (int i = 1; i <= F::kAhead && WAY == kTma && top - i * stride > p.r0; ++i) in_flight.wait(step + i, a.status);
      break;
    }
    if (!any) continue;
    T *qz = pdz + static_cast<long long>(row0) * a.dz.ld, *qx = pdx + static_cast<long long>(row0) * a.dx.ld;
#pragma unroll
    for (int i = 0; i < R; ++i, qz -= a.dz.ld, qx -= a.dx.ld) {
      const Vec<VEC> g = add(dv[i], pick(ends >> i & 1, all<VEC>(0.f), s)), dx = mul(gn[i], g);
      s = mul(ga[i], g);
      if (in && row0 - i >= p.r0) {
        store_cell<T, VEC>(qx, dx);
        store_cell<T, VEC>(qz, mul(mul(dx, ga[i]), diff[i]));
      }
      if (a.dfirst != nullptr && (begins >> i & 1)) {
        if (in) store_state<VEC>(a.dfirst + static_cast<long long>(q0) * a.channels + c, s);
        q0 = p.seq.prev(q0);
      }
    }
  }
  end_steps(size);
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
// Channels at an aligned address in every row: 4, 2 or 1.
int aligned_channels(const Mat& m, int dtype) {
  if (m.p == nullptr) return 4;
  const int es = dtype == kF32 ? 4 : 2;
  for (int v : {4, 2})
    if (m.ld % v == 0 && reinterpret_cast<uintptr_t>(m.p) % (v * es) == 0) return v;
  return 1;
}

// Channels of a thread that the matrices allow.
int vector_of(const RecurrenceArgs& a) {
  int vec = a.channels % 4 == 0 ? 4 : a.channels % 2 == 0 ? 2 : 1;
  for (const Mat* m : {&a.z, &a.x, &a.h, &a.dh, &a.dz, &a.dx}) vec = std::min(vec, aligned_channels(*m, a.dtype));
  return vec;
}
// Tiles of 64 channels, where they give every SM a block in clusters of 8 (16384 x 1024 in
// tiles of 32: 28 us for 46).
bool wide(const RecurrenceArgs& a) {
  return vector_of(a) == 4 && (a.channels + 4 * kAcross - 1) / (4 * kAcross) * 8 >= sm_count();
}

// Whether one row a thread takes all of it in a step (the gradient) or two: single tokens
// of many sequences.  With eight, a thread walks through the boundaries of as many rows
// while others have none: 64 tokens x 4096 in as many sequences 4.1 us for 6.8, one token
// 2.7 for 3.9; 256 tokens, in four steps, 9.5 for 7.8.
bool is_short(const RecurrenceArgs& a) {
  const int vec = wide(a) ? 4 : std::min(2, vector_of(a)), tiles = (a.channels + vec * kAcross - 1) / (vec * kAcross);
  const int groups = std::max(1, std::min(a.sequences, 2 * sm_count() / tiles));
  return a.tokens <= (a.grad ? 1 : 2) * kGroups * groups;
}

// A launch of clusters.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(dim3 grid, int size, size_t shared, cudaStream_t s) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(size), 1u, 1u};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
  }
  Launch(const Launch&) = delete;
};

// How many clusters of each size run side by side (0: none): what the groups of SMs that
// hold a cluster leave of two blocks an SM, 296 blocks in clusters of 4 and 266 of 7 on
// 152 SMs.  Asked once a kernel and device, with the attributes that its launches need.
template <auto kernel>
cudaError_t resident_of(size_t shared, int (&clusters)[kMaxCluster + 1]) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];  // [0]: 1 when the others are there
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::atomic<int>* r = device < kDevices ? known[device] : nullptr;
  if (r != nullptr && r[0].load(std::memory_order_acquire)) {
    for (int n = 1; n <= kMaxCluster; ++n) clusters[n] = r[n].load(std::memory_order_relaxed);
    return cudaSuccess;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int n = 1; n <= kMaxCluster && e == cudaSuccess; ++n) {
    Launch l(dim3(n), n, shared, nullptr);
    l.cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters[n], kernel, &l.cfg);
    if (r != nullptr) r[n].store(clusters[n], std::memory_order_relaxed);
  }
  if (r != nullptr && e == cudaSuccess) r[0].store(1, std::memory_order_release);
  return e;
}

// Blocks of a cluster, and clusters side by side for groups of sequences.
struct Plan {
  int tiles, size, groups;
};
Plan plan_scan(const RecurrenceArgs& a, int vec, int rows, const int (&clusters)[kMaxCluster + 1]) {  // rows of a block's step
  Plan p;
  p.tiles = (a.channels + kAcross * vec - 1) / (kAcross * vec);
  // Clusters for the length that two sequences have on the average, groups of sequences
  // beyond that (16384 x 512 in 64 sequences: 22 us for 44 in clusters of 16).  16
  // blocks wait for one another longer than 8: where they have four steps at least
  // (16384 x 256: 16 us for 23; 2048 x 512, gradient: 12.9 for 10.5).  All clusters run
  // at once: a second wave costs as much as the first.
  const long long length = std::min<long long>(a.tokens, 2ll * a.tokens / a.sequences);
  for (p.size = kMaxCluster; p.size > 1; --p.size) {
    int half = 1;  // of the next power of two
    while (2 * half < p.size) half *= 2;
    if (p.tiles <= clusters[p.size] &&
        (half < 8 ? static_cast<long long>(half) * rows < length : 8ll * half * rows <= length))
      break;
  }
  p.groups = std::max(1, std::min({a.sequences, clusters[p.size] / p.tiles, 65535 / kMaxCluster}));
  return p;
}

// Boxes of all matrices that are read; false where TMA cannot read one.
bool boxes_of(const RecurrenceArgs& a, int rows, int cols, TileMaps* boxes) {
  const Mat* m[4] = {&a.z, &a.x, &a.h, &a.dh};
  const int es = a.dtype == kF32 ? 4 : 2;
  for (int i = 0; i < (a.grad ? 4 : 2); ++i) {
    if (reinterpret_cast<uintptr_t>(m[i]->p) % 16 != 0 || m[i]->ld * es % 16 != 0) return false;
    if (!plain_box_map(&boxes->m[i], *m[i], a.tokens, a.channels, a.dtype, rows, cols)) return false;
  }
  return true;
}

template <typename T, int VEC, Way WAY, bool GRAD, bool SHORT = false>
cudaError_t launch_way(const RecurrenceArgs& a, cudaStream_t s) {
  // Rows of a thread, one or: 32 (forward) and 16 elements of each matrix fill the registers,
  // half of them where the next rows' wait there too, and half in fp32, whose cells
  // would not leave two blocks the shared memory.
  constexpr int kElements = sizeof(T) == 4 || WAY == kRegs ? 16 : 32;
  constexpr int R = SHORT ? 1 : kElements / VEC / (GRAD ? 2 : 1), kRows = kGroups * R;
  constexpr size_t kBytes = Flight<T, VEC, R, GRAD ? 4 : 2, WAY, GRAD>::kBytes;
  constexpr auto kernel = [] {
    if constexpr (GRAD)
      return recurrence_grad_kernel<T, VEC, R, WAY>;
    else
      return recurrence_kernel<T, VEC, R, WAY>;
  }();
  int clusters[kMaxCluster + 1];
  const cudaError_t e = resident_of<kernel>(kBytes, clusters);
  if (e != cudaSuccess) return e;
  const Plan p = plan_scan(a, VEC, kRows, clusters);
  MapsOf<WAY> boxes;
  if constexpr (WAY == kTma) {
    // A map costs the host half a microsecond: for some steps of the clusters at least.
    if (a.tokens < 4 * kRows * p.size || !boxes_of(a, kRows, kAcross * VEC, &boxes)) {
      // Cells of two channels are copied by twice the instructions.
      constexpr int kWide = VEC == 2 && !GRAD && sizeof(T) == 2 ? 4 : VEC;
      if (kWide != VEC && wide(a)) return launch_way<T, kWide, kCells, GRAD>(a, s);
      return launch_way<T, VEC, kCells, GRAD>(a, s);
    }
  }
  const Launch l(dim3(p.size * p.groups, p.tiles), p.size, kBytes, s);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, boxes);
}
template <typename T, bool GRAD>
cudaError_t launch_typed(const RecurrenceArgs& a, cudaStream_t s) {
  // Boxes of 32 channels and 16 rows a thread compose half as many maps as 64 and 8, by
  // as many blocks in smaller clusters: 16384 x 4096 bf16 83 us for 87, x 8192 138 for
  // 158.  The gradient has no registers for that (157 for 148), fp32 loads halve (65 for
  // 64).
  if (is_short(a)) {
    if (wide(a)) return launch_way<T, 4, kRegs, GRAD, true>(a, s);
    if (vector_of(a) >= 2) return launch_way<T, 2, kRegs, GRAD, true>(a, s);
    return launch_way<T, 1, kRegs, GRAD, true>(a, s);
  }
  if (wide(a) && (GRAD || sizeof(T) == 4)) return launch_way<T, 4, kTma, GRAD>(a, s);
  if (vector_of(a) >= 2) return launch_way<T, 2, kTma, GRAD>(a, s);
  return launch_way<T, 1, sizeof(T) == 4 ? kCells : kRegs, GRAD>(a, s);
}

}  // namespace

cudaError_t launch_recurrence(const RecurrenceArgs& a, cudaStream_t s) {
  const auto launch = [&](auto grad) {
    if (a.dtype == kF32) return launch_typed<float, grad()>(a, s);
    if (a.dtype == kBF16) return launch_typed<__nv_bfloat16, grad()>(a, s);
    return launch_typed<__half, grad()>(a, s);
  };
  return a.grad ? launch(std::true_type{}) : launch(std::false_type{});
}

}  // namespace dion3
