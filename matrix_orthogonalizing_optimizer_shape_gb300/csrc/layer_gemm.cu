// Tensor-core products of the linear layer on sm_103a (see Product in
// layer.h): out[t][m] = sum_k A(m, k) B(t, k), fp32 accumulation in tensor
// memory, operands K-major or MN-major in 16 bits.
//   forward:  A = W,   B = x:   z = v + bias, y = act(z) + residual, with z
//             and y also in 8-bit blocks
//   dx:       A = W^T, B = dz
//   dW:       A = x^T, B = dz^T
//
// Small products (tile_kernel): one CTA computes a tile of 128 m x BN t.  m runs along the TMEM
// lanes, so the 32 lanes of a warp hold 32 consecutive columns of an output
// row: 16-bit rows are written in 64-byte pieces, and the 32 columns of an
// 8-bit block are one warp's lanes.  Warp 0 fills a ring of 64-wide K slabs
// by TMA, warp 1 issues the MMAs, warps 2..5 (one per TMEM lane quadrant) are
// the epilogue.  Every wait is bounded (about a second) and records
// kDevTimeout in the status word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "layer_math.cuh"
#include "model.h"
#include "tc_ops.cuh"

namespace dion3 {
namespace {

using namespace tc;
using namespace lm;

constexpr int BM = 128;
constexpr int BK = 64;  // 16-bit elements of one 128-byte swizzle row

struct Epilogue {
  int M, N;
  void* out; long long ld_out; int out_f32, out_bf16, accumulate;
  const void* bias; int bias_dtype;
  int act;
  const uint16_t* res; long long ld_res;
  uint16_t* z; long long ld_z;
  Pack8 z8, out8;
};

__device__ __forceinline__ float load_bias(const void* b, int dtype, int c) {
  if (dtype == kF32) return static_cast<const float*>(b)[c];
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(b)[c]);
  return __half2float(static_cast<const __half*>(b)[c]);
}

template <int N>
__device__ __forceinline__ void apply_act(int act, float (&v)[N]) {
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_fwd<kActRelu>(v[j]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_fwd<kActGelu>(v[j]);
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_fwd<kActSilu>(v[j]);
  }
}

// The 8-bit blocks of n rows held by a warp: lane = column of the block, 0 past
// the last column (`in` false there).
template <int C>
__device__ __forceinline__ void store_blocks_warp(const Pack8& o, int t0, int n, int m, bool in, const float (&v)[C]) {
  int8_t* q = o.q + static_cast<long long>(t0) * o.ldq + m;
  uint8_t* s = o.s + static_cast<long long>(t0) * o.lds + m / kPackBlock;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if (j >= n) break;
    const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7FFFFFFFu));
    float u[1] = {v[j]};
    saturate_block(byte, u);
    if (in) q[j * o.ldq] = static_cast<int8_t>(code_of(u[0], inv_scale(byte)));
    if (in && m % kPackBlock == 0) s[j * o.lds] = static_cast<uint8_t>(byte);
  }
}

// Values v[0..C) of output rows t0.. at column m (in: m < M).  Run by a whole
// warp whose lanes hold 32 consecutive columns.
template <bool BF16, bool FWD, int C>
__device__ __forceinline__ void epilogue_rows(const Epilogue& e, int t0, int m, bool in, float bias, float (&v)[C]) {
  const int n = min(C, e.N - t0);
  const int nw = in ? n : 0;  // rows this lane writes
  const long long o = static_cast<long long>(t0) * e.ld_out + m;
  if constexpr (FWD) {
    uint16_t r[C];
    if (e.res != nullptr) {
      const uint16_t* p = e.res + static_cast<long long>(t0) * e.ld_res + m;
#pragma unroll
      for (int j = 0; j < C; ++j) r[j] = j < nw ? p[j * e.ld_res] : uint16_t(0);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = in ? v[j] + bias : 0.f;
    if (e.z != nullptr) {
      uint16_t* p = e.z + static_cast<long long>(t0) * e.ld_z + m;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j < nw) p[j * e.ld_z] = pack1<BF16>(v[j]);
    }
    if (e.z8.q != nullptr) store_blocks_warp(e.z8, t0, n, m, in, v);
    apply_act(e.act, v);
    if (e.res != nullptr) {
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] += unpack1<BF16>(r[j]);
    }
    uint16_t* p = static_cast<uint16_t*>(e.out) + o;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (j < nw) p[j * e.ld_out] = pack1<BF16>(v[j]);
    if (e.out8.q != nullptr) store_blocks_warp(e.out8, t0, n, m, in, v);
  } else if (e.out_f32) {
    float* p = static_cast<float*>(e.out) + o;
    if (e.accumulate) {
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] += j < nw ? p[j * e.ld_out] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (j < nw) p[j * e.ld_out] = v[j];
  } else {
    uint16_t* p = static_cast<uint16_t*>(e.out) + o;
    if (e.accumulate) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const uint16_t old = j < nw ? p[j * e.ld_out] : uint16_t(0);
        v[j] += e.out_bf16 ? unpack1<true>(old) : unpack1<false>(old);
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (j < nw) p[j * e.ld_out] = e.out_bf16 ? pack1<true>(v[j]) : pack1<false>(v[j]);
  }
}

// A 32-bit result is summed in pieces of kPiece K slabs: the tensor cores
// truncate each addition to the accumulator, an error that grows with their
// number (relative 1.9e-5 over 16384 tokens in one piece, 4.4e-6 over 4096,
// 1.0e-6 over 1024).  The pieces are added in fp32, rounded to nearest, in order:
// by the tile kernel to a second set of TMEM columns, by the paired kernel, which
// has none to spare, to the output in place, by bulk reductions that find the tile
// in L2.  Their traffic is why a piece is no shorter: dW of 16384 x 4096 x 11008
// takes 818 us in one piece and 1060 in pieces of 16 slabs.  A 16-bit result does
// not show the error.
constexpr int kPiece = 64;

template <int BN, bool DEEP, bool SUM>  // DEEP: one CTA an SM, the ring takes all of it; SUM: a sum of pieces
struct TileCfg {
  static constexpr int kABytes = BM * BK * 2;
  static constexpr int kBBytes = BN * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = (DEEP ? 200 : 96) * 1024 / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  // Two CTAs of an SM hold 512 columns at most: all there are, so that a CTA
  // placed early never keeps them from one that has to finish first.
  static constexpr int kTmemCols = SUM ? 2 * BN : BN < 32 ? 32 : BN;
  static constexpr int kBars = (2 * kStages + 3) * 8;
  static constexpr int kDyn = 1024 + kRing + kBars + 16;
  static_assert(BN * BM * 4 <= kRing, "a tile's partial sums take the ring's place");
};
constexpr int kTileThreads = 6 * 32;
constexpr int kTurn = 8;  // output rows an epilogue warp finishes at a time

// v += eight TMEM columns of the thread's lane.
__device__ __forceinline__ void add_columns(uint32_t taddr, float (&v)[kTurn]) {
  uint32_t u[kTurn];
  tmem_ld8(taddr, u);
  tmem_ld_done(u);
#pragma unroll
  for (int j = 0; j < kTurn; ++j) v[j] += __uint_as_float(u[j]);
}
// Adds all pieces but the last, n columns each, from the accumulator at tb to the
// sum BN columns after it.  True (to every lane) once the last is in the accumulator.
template <int BN>
__device__ __forceinline__ bool take_pieces(uint32_t tb, int pieces, int n, uint32_t bar_done, uint32_t bar_taken,
                                            unsigned* status) {
  for (int p = 0;; ++p) {
    if (!mbar_wait_warp(bar_done, p & 1u, status)) return false;
    fence_after();
    if (p == pieces - 1) return true;
#pragma unroll 1
    for (int c = 0; c < n; c += kTurn) {
      float v[kTurn] = {};
      add_columns(tb + c, v);
      if (p > 0) add_columns(tb + BN + c, v);
      uint32_t u[kTurn];
#pragma unroll
      for (int j = 0; j < kTurn; ++j) u[j] = __float_as_uint(v[j]);
      tmem_st8(tb + BN + c, u);
    }
    tmem_st_done();
    fence_before();
    mbar_arrive(bar_taken);
  }
}

// K is split over the CTAs of a cluster when there are few tiles: each CTA
// multiplies its share of the K slabs, the partial tiles meet in distributed
// shared memory, and every CTA adds the partials of its share of the rows in
// rank order (the same bits every call) and finishes them.  SUM: a share of
// more than kPiece slabs, for a 32-bit output.  After each piece the epilogue warps
// add the accumulator to the running sum in the BN columns beside it, while the
// MMAs wait: 65536 x 1024 x 1024 (dW) takes 116 us where one piece takes 114.  (A
// form of its own: shares of one piece take 0.8 us more with its code.)
template <bool BF16, bool AT, bool BT, int BN, bool FWD, bool DEEP, bool SUM>
__global__ void __launch_bounds__(kTileThreads)
    tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, int nkb_all,
                int tiles_m, int split, Epilogue e, unsigned* status) {
  using C = TileCfg<BN, DEEP, SUM>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sA = base, sB = base + C::kStages * C::kABytes;
  const uint32_t bar_full = base + C::kRing, bar_empty = bar_full + 8 * C::kStages,
                 bar_done = bar_empty + 8 * C::kStages, bar_drain = bar_done + 8, bar_taken = bar_drain + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (base - raw) + C::kRing + C::kBars);
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmB);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);    // a piece is in the accumulator
    mbar_init(bar_drain, 1);
    mbar_init(bar_taken, 128);  // the epilogue's threads have added it to the sum
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), C::kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / split;
  const int m0 = (tile % tiles_m) * BM, t0 = (tile / tiles_m) * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(nkb_all) * rank / split);
  const int nkb = static_cast<int>(static_cast<long long>(nkb_all) * (rank + 1) / split) - kb0;
  const int pieces = SUM ? (nkb + kPiece - 1) / kPiece : 1;
  const int quad = warp % 4;
  const int m = m0 + quad * 32 + lane;
  const bool in = m < e.M;

  if (warp == 0) {
    int kb = 0;
    for (; kb < nkb; ++kb) {
      const uint32_t s = kb % C::kStages, ph = (kb / C::kStages) & 1u;
      if (!mbar_wait_warp(bar_empty + 8 * s, ph ^ 1u, status)) break;
      const uint32_t a = sA + s * C::kABytes, b = sB + s * C::kBBytes, full = bar_full + 8 * s;
      const int k0 = (kb0 + kb) * BK;
      if (elect_one()) {
        mbar_expect(full, C::kStageBytes);
        if constexpr (AT) {
          tma_load(a, &tmA, full, m0, k0);
          tma_load(a + C::kABytes / 2, &tmA, full, m0 + 64, k0);
        } else {
          tma_load(a, &tmA, full, k0, m0);
        }
        if constexpr (BT) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) tma_load(b + i * 8192, &tmB, full, t0 + 64 * i, k0);
        } else {
          tma_load(b, &tmB, full, k0, t0);
        }
      }
      __syncwarp();
    }
    // Wait (bounded) for the last copies, so none is in flight when the CTA
    // exits even if the MMA warp gave up.
    for (int i = kb > C::kStages ? kb - C::kStages : 0; i < kb; ++i)
      mbar_wait_warp(bar_full + 8 * (i % C::kStages), (i / C::kStages) & 1u, status);
  } else if (warp == 1) {
    constexpr uint32_t id = instr_desc<BF16, AT, BT>(BM, BN);
    int at = 0, piece = 0;  // slabs in the accumulator, pieces before it
    for (int kb = 0; kb < nkb; ++kb) {
      const uint32_t s = kb % C::kStages, ph = (kb / C::kStages) & 1u;
      if (SUM && at == kPiece) {
        if (!mbar_wait_warp(bar_taken, piece & 1u, status)) break;
        at = 0, ++piece;
      }
      if (!mbar_wait_warp(bar_full + 8 * s, ph, status)) break;
      fence_after();
      const uint64_t da = smem_desc<AT>(sA + s * C::kABytes), db = smem_desc<BT>(sB + s * C::kBBytes);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_f16<1>(tmem, da + kDescStep<AT> * kk, db + kDescStep<BT> * kk, id, (at > 0 || kk > 0) ? 1u : 0u);
        mma_commit(bar_empty + 8 * s);
        if (kb == nkb - 1 || (SUM && at + 1 == kPiece)) mma_commit(bar_done);
      }
      ++at;
      __syncwarp();
    }
    // All MMAs have completed before TMEM is freed.
    if (elect_one()) mma_commit(bar_drain);
    __syncwarp();
    mbar_wait_warp(bar_drain, 0u, status);
  } else if (SUM ? take_pieces<BN>(tmem + (static_cast<uint32_t>(quad * 32) << 16), pieces, min(BN, e.N - t0), bar_done,
                                   bar_taken, status)
                 : mbar_wait_warp(bar_done, 0u, status)) {
    fence_after();
    const float bias = FWD && e.bias != nullptr && in ? load_bias(e.bias, e.bias_dtype, m) : 0.f;
    const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // Eight rows a turn, rolled: this code runs once or a few times a launch,
    // and fetching it unrolled took longer than running it.  A turn's loads
    // run under the turn before.
    uint32_t u[kTurn];
    tmem_ld8(tb, u);
    const int n = min(BN, e.N - t0);
#pragma unroll 1
    for (int c = 0; c < n; c += kTurn) {
      tmem_ld_done(u);
      float v[kTurn];
#pragma unroll
      for (int j = 0; j < kTurn; ++j) v[j] = __uint_as_float(u[j]);
      if (SUM && pieces > 1) add_columns(tb + BN + c, v);
      if (c + kTurn < n) tmem_ld8(tb + c + kTurn, u);
      if (split > 1) {  // every slab has been consumed: the ring is free
#pragma unroll
        for (int j = 0; j < kTurn; ++j) st_shared_f32(base + ((c + j) * BM + quad * 32 + lane) * 4, v[j]);
      } else {
        epilogue_rows<BF16, FWD, kTurn>(e, t0 + c, m, in, bias, v);
      }
    }
  }
  if (split > 1) {
    cluster_sync();
    if (warp >= 2) {
      const float bias = FWD && e.bias != nullptr && in ? load_bias(e.bias, e.bias_dtype, m) : 0.f;
      const int valid = min(BN, e.N - t0), per = (valid + split - 1) / split;
      const int j1 = min(valid, (rank + 1) * per);
#pragma unroll 1
      for (int j0 = rank * per; j0 < j1; j0 += kTurn) {
        float v[kTurn] = {};
        const uint32_t at = base + (j0 * BM + quad * 32 + lane) * 4;
        for (int r = 0; r < split; ++r) {
          const uint32_t peer = map_to_rank(at, r);
#pragma unroll
          for (int j = 0; j < kTurn; ++j)
            if (j0 + j < j1) v[j] += ld_cluster_f32(peer + j * BM * 4);
        }
        // Rows past this CTA's share end at e.N for the epilogue.
        Epilogue part = e;
        part.N = t0 + j1;
        epilogue_rows<BF16, FWD, kTurn>(part, t0 + j0, m, in, bias, v);
      }
    }
  }
  fence_before();
  // With a split, no CTA leaves while a peer may still read its partials.
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<1>(tmem, C::kTmemCols);
  }
}

// --------------------------------------------------------------------------
// Forward products of one to four tokens: the weights' bytes are the time.  A
// warp reads four rows of W along their length (TMA's 128-byte pieces of 128 rows
// reach 4.8 TB/s where this reaches 5.8: 1 x 4096 x 11008 in 15.7 us against
// 18.9), multiplies them on the fp32 units and adds up its lanes; the 32 columns
// of a block's 8 warps meet in shared memory, where one warp a token finishes
// them like a tile's rows.
// --------------------------------------------------------------------------
constexpr int kFewTokens = 4;
constexpr int kFewRows = 4;  // rows of W a warp

template <bool BF16, int T>
__global__ void __launch_bounds__(256)
    few_tokens_kernel(const uint16_t* w, long long ldw, const uint16_t* x, long long ldx, int K, Epilogue e) {
  pdl_trigger();
  pdl_wait();
  __shared__ float res[T][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint16_t* rows[kFewRows];
#pragma unroll
  for (int r = 0; r < kFewRows; ++r) {
    const int m = blockIdx.x * 32 + warp * kFewRows + r;
    rows[r] = w + static_cast<long long>(min(m, e.M - 1)) * ldw;  // past the last row: its values again, not used
  }
  float acc[kFewRows][T] = {};
#pragma unroll 4
  for (int k = lane * 8; k < K; k += 256) {
    uint4 wv[kFewRows], xv[T];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) wv[r] = __ldcs(reinterpret_cast<const uint4*>(rows[r] + k));
#pragma unroll
    for (int t = 0; t < T; ++t) xv[t] = __ldg(reinterpret_cast<const uint4*>(x + t * ldx + k));
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
      const uint32_t a[4] = {wv[r].x, wv[r].y, wv[r].z, wv[r].w};
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint32_t b[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = unpack2<BF16>(a[i]), v = unpack2<BF16>(b[i]);
          acc[r][t] = fmaf(u.x, v.x, acc[r][t]);
          acc[r][t] = fmaf(u.y, v.y, acc[r][t]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kFewRows; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o /= 2) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (lane == 0) res[t][warp * kFewRows + r] = acc[r][t];
    }
  __syncthreads();
  if (warp >= T) return;
  const int m = blockIdx.x * 32 + lane;
  const bool in = m < e.M;
  const float bias = e.bias != nullptr && in ? load_bias(e.bias, e.bias_dtype, m) : 0.f;
  float v[1] = {res[warp][lane]};
  epilogue_rows<BF16, true, 1>(e, warp, m, in, bias, v);
}

// --------------------------------------------------------------------------
// Large products: bound by the tensor cores, and back to back by the board's
// power.  16384 x 4096 x 11008 forward (silu, pre-activation kept): 0.79 ms on a
// cool board (1.87 PFLOP/s), 0.88 under the power cap; dx 0.77, dW 0.80.
// Persistent clusters of two CTAs on two SMs, each cluster a
// 256 x 256 (or 256 x 128) tile of the output at a time with the paired-SM MMA
// (M = 256, K = 16).  Here the TMEM lanes are output rows: CTA rank r holds rows
// 128 r .. of the tile and every epilogue thread one row, 32 contiguous
// columns at a time, so an 8-bit block is one thread's registers.  Two
// accumulators let the epilogue of a tile run under the next
// tile's MMAs.  Warps: 0 TMA producer, 1 MMA issuer (even CTA), 2..9 epilogue
// (two per TMEM lane quadrant, each half of the columns).  Each CTA loads its own
// rows of both operands: what an SM's copy engine can issue (a 128-byte row every
// 2.2 cycles, measured) bounds the narrow tiles.
// --------------------------------------------------------------------------
constexpr int kPairEpiWarps = 8;
constexpr int kBox = 2048;  // staging box: 32 rows of 64 bytes
constexpr int kBand = 8;  // row tiles walked together, column by column: operand panels shared through L2

// kOutOther: 16 bits, of the type that the operands do not have.
enum PairOut : int { kOutFwd = 0, kOut16 = 1, kOut32 = 2, kOutOther = 3 };

struct PairParams {
  int rows, cols, nkb;         // output rows and columns, K slabs
  int tiles_r, tiles_c;        // tiles of 256 rows
  int tma_out, tma_z;          // the output has a store map
  int vec_res;                 // residual (or the accumulated output) readable in 16-byte pieces
  Epilogue e;
  unsigned* status;
};

template <int PN>  // tile width: 256, or 128 where there are few tiles
struct PairCfg {
  static constexpr int kA = 128 * BK * 2;       // one CTA's rows of A, one slab: 16 KB
  static constexpr int kB = PN / 2 * BK * 2;    // and its half of B
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = PN == 256 ? 6 : 8;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kStaging = kPairEpiWarps * 2 * kBox;
  static constexpr int kBars = (2 * kStages + 5) * 8;
  static constexpr int kDyn = 1024 + kRing + kStaging + kBars + 16;
  static constexpr int kTmem = 2 * PN;          // two accumulators
  static constexpr int kThreads = 32 * (2 + kPairEpiWarps);
};

__device__ __forceinline__ void pair_tile(const PairParams& p, int u, int& R, int& C) {
  const int per_band = kBand * p.tiles_c;
  const int band = u / per_band, in = u - band * per_band;
  const int h = min(kBand, p.tiles_r - band * kBand);
  C = in / h;
  R = band * kBand + in - C * h;
}

// Staging boxes of one epilogue warp and the bulk stores that read them.
struct Stager {
  uint32_t buf;    // two boxes
  uint32_t count;  // boxes staged so far
  int lane;
  bool bulk;       // every box is read by a bulk store
  // Writes the thread's row of the next box (64 bytes); returns its address.
  __device__ __forceinline__ uint32_t fill(const uint32_t (&w)[16]) {
    const uint32_t b = buf + (count & 1u) * kBox;
    const uint32_t sw = static_cast<uint32_t>((lane >> 1) & 3);
    if (lane == 0) {  // the store two boxes back has read its box
      if (bulk)
        bulk_wait_read<1>();
      else
        bulk_wait_read<0>();
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st_shared_v4(b + lane * 64 + ((static_cast<uint32_t>(q) ^ sw) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2],
                   w[4 * q + 3]);
    ++count;
    return b;
  }
  __device__ __forceinline__ void store(const CUtensorMap* map, const uint32_t (&w)[16], int x, int y, bool add) {
    const uint32_t b = fill(w);
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (add)
        tma_reduce_add(map, b, x, y);
      else
        tma_store(map, b, x, y);
      bulk_commit();
    }
  }
  // The same box by plain stores, for outputs whose base or pitch TMA cannot
  // take: the warp reads the box back row by row, so each row is one
  // contiguous piece.
  template <int BYTES>
  __device__ __forceinline__ void store_plain(void* out, long long ld, int rows, int cols, const uint32_t (&w)[16],
                                              int x, int y, bool add) {
    const uint32_t b = fill(w);
    __syncwarp();
    constexpr int kCols = 64 / BYTES, kPass = 32 / kCols;  // columns of the box, rows a pass
    const int c = lane % kCols, r0 = lane / kCols, n = x + c < cols ? rows - y - r0 : 0;
    const uint32_t sw = static_cast<uint32_t>(c * BYTES), at = b + r0 * 64;
    uint8_t* d = static_cast<uint8_t*>(out) + (static_cast<long long>(y + r0) * ld + x + c) * BYTES;
    const long long step = ld * (kPass * BYTES);
#pragma unroll 1
    for (int r = 0; r < 32; r += 8) {
#pragma unroll
      for (int j = 0; j < 8; j += kPass, d += step) {
        if (r + j >= n) continue;
        const uint32_t src = at + (r + j) * 64 + (sw ^ ((j / 2 & 3) << 4));
        if constexpr (BYTES == 2) {
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src) : "memory");
          *reinterpret_cast<uint16_t*>(d) = v;
        } else {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(src) : "memory");
          float* f = reinterpret_cast<float*>(d);
          *f = add ? *f + v : v;
        }
      }
    }
    __syncwarp();
  }
};

// 32 columns of one row, as fp32, to 16-bit words.
template <bool BF16>
__device__ __forceinline__ void to_words(const float (&f)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack2<BF16>(f[2 * j], f[2 * j + 1]);
}

// 16-bit values of one row's 32 columns (a residual, or an output to add to):
// read in 16-byte pieces ahead of their use where that is possible.
struct RowPiece {
  uint4 v[4];
  template <typename P>
  __device__ __forceinline__ void load(const uint16_t* base, long long ld, const P& p, int r, int c0) {
    if (base == nullptr || r >= p.rows) return;
    const uint16_t* row = base + static_cast<long long>(r) * ld + c0;
    if (p.vec_res && c0 + 32 <= p.cols) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(row + 8 * q);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t a = c0 + 2 * j < p.cols ? row[2 * j] : 0u, b = c0 + 2 * j + 1 < p.cols ? row[2 * j + 1] : 0u;
        w[j] = a | (b << 16);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  }
  template <bool BF16>
  __device__ __forceinline__ void add(float (&f)[32]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = unpack2<BF16>(w[i]);
        f[8 * q + 2 * i] += x.x;
        f[8 * q + 2 * i + 1] += x.y;
      }
    }
  }
};

__device__ __forceinline__ void add_bias(const Epilogue& e, int c0, int cols, float (&f)[32]) {
  const int bytes = e.bias_dtype == kF32 ? 4 : 2;
  const bool vec = c0 + 32 <= cols && (reinterpret_cast<uintptr_t>(e.bias) & 15u) == 0;
  if (vec && bytes == 4) {
    const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(e.bias) + c0);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 x = __ldg(b + q);
      f[4 * q] += x.x, f[4 * q + 1] += x.y, f[4 * q + 2] += x.z, f[4 * q + 3] += x.w;
    }
  } else if (vec) {
    const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.bias) + c0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 x = __ldg(b + q);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = e.bias_dtype == kBF16 ? unpack2<true>(w[i]) : unpack2<false>(w[i]);
        f[8 * q + 2 * i] += y.x;
        f[8 * q + 2 * i + 1] += y.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c0 + j < cols) f[j] += load_bias(e.bias, e.bias_dtype, c0 + j);
  }
}

// One block of 32 columns held by a thread (0 past the last column).
__device__ __forceinline__ void store_block_row(const Pack8& o, long long r, int c0, int cols, const float (&f)[32]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 32; ++j) m = max_mag(m, f[j]);
  const uint32_t byte = scale_byte(__float_as_uint(m) & 0x7FFFFFFFu);
  const float inv = inv_scale(byte);
  float v[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = f[j];
  saturate_block(byte, v);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = codes4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], inv);
  int8_t* q = o.q + r * o.ldq + c0;
  if (c0 + 32 <= cols && ((reinterpret_cast<uintptr_t>(q) & 15u) == 0)) {
    *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(q + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c0 + j < cols) q[j] = static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)));
  }
  o.s[r * o.lds + c0 / kPackBlock] = static_cast<uint8_t>(byte);
}

template <bool BF16, bool AT, bool BT, int OUT, int PN>
__global__ void __launch_bounds__(PairCfg<PN>::kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmZ,
                const __grid_constant__ PairParams p) {
  using C = PairCfg<PN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sA = base, sB = base + C::kStages * C::kA, staging = base + C::kRing;
  const uint32_t bar_full = staging + C::kStaging, bar_empty = bar_full + 8 * C::kStages;
  const uint32_t bar_tfull = bar_empty + 8 * C::kStages, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (base - raw) + C::kRing + C::kStaging + C::kBars);
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr uint32_t even = 0;    // rank of the CTA that issues the MMAs
  constexpr uint16_t both = 0x3;  // the CTAs of the pair
  const uint32_t rank = cluster_rank();
  const bool leader = rank == even;
  const int cluster = blockIdx.x / 2, nclusters = gridDim.x / 2;
  const int total = p.tiles_r * p.tiles_c;
  const int depth = OUT == kOut32 ? kPiece : p.nkb;  // K slabs of one accumulation
  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmB);
    if (p.tma_out) prefetch_map(&tmOut);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);   // in the even CTA: its producer, and both CTAs' bytes
      mbar_init(bar_empty + 8 * s, 1);  // the MMA commit that frees the slot
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_tfull + 8 * a, 1);
      mbar_init(bar_tempty + 8 * a, 2 * 32 * kPairEpiWarps);  // in the even CTA: both CTAs' epilogue threads
    }
    mbar_init(bar_drain, 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), C::kTmem);
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    uint32_t kc = 0;
    bool ok = true;
    for (int u = cluster; u < total && ok; u += nclusters) {
      int R, Cc;
      pair_tile(p, u, R, Cc);
      const int a_row = R * 256 + static_cast<int>(rank) * 128, b_row = Cc * PN + static_cast<int>(rank) * (PN / 2);
      for (int kb = 0; kb < p.nkb; ++kb, ++kc) {
        const uint32_t s = kc % C::kStages, ph = (kc / C::kStages) & 1u;
        if (!(ok = mbar_wait_warp(bar_empty + 8 * s, ph ^ 1u, p.status))) break;
        const uint32_t a = sA + s * C::kA, b = sB + s * C::kB;
        const int k0 = kb * BK;
        if (elect_one()) {
          if (leader) mbar_expect(bar_full + 8 * s, 2 * C::kStage);
          const uint32_t full = map_to_rank(bar_full + 8 * s, even);
          if constexpr (AT) {
            tma_load_pair(a, &tmA, full, a_row, k0);
            tma_load_pair(a + C::kA / 2, &tmA, full, a_row + 64, k0);
          } else {
            tma_load_pair(a, &tmA, full, k0, a_row);
          }
          if constexpr (BT) {
            tma_load_pair(b, &tmB, full, b_row, k0);
            if constexpr (PN == 256) tma_load_pair(b + C::kB / 2, &tmB, full, b_row + 64, k0);
          } else {
            tma_load_pair(b, &tmB, full, k0, b_row);
          }
        }
        __syncwarp();
      }
    }
    // Every copy has landed (bounded) before the pair exits; the even CTA's
    // barriers count the bytes of both.
    for (uint32_t i = 0; leader && i < C::kStages && i < kc; ++i) {
      const uint32_t last = kc - 1 - i;
      mbar_wait_warp(bar_full + 8 * (last % C::kStages), (last / C::kStages) & 1u, p.status);
    }
  } else if (warp == 1) {
    if (leader) {
      constexpr uint32_t id = instr_desc<BF16, AT, BT>(256, PN);
      uint32_t kc = 0, tc = 0;
      bool ok = true;
      for (int u = cluster, kb0 = 0; u < total && ok; ++tc) {
        const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
        if (!mbar_wait_warp(bar_tempty + 8 * acc, aph ^ 1u, p.status)) break;
        fence_after();
        const uint32_t d = tmem + acc * PN;
        const int kb1 = min(p.nkb, kb0 + depth);
        for (int kb = kb0; kb < kb1; ++kb, ++kc) {
          const uint32_t s = kc % C::kStages, ph = (kc / C::kStages) & 1u;
          if (!(ok = mbar_wait_warp(bar_full + 8 * s, ph, p.status))) break;
          fence_after();
          const uint64_t da = smem_desc<AT>(sA + s * C::kA), db = smem_desc<BT>(sB + s * C::kB);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_f16<2>(d, da + kDescStep<AT> * kk, db + kDescStep<BT> * kk, id, (kb > kb0 || kk > 0) ? 1u : 0u);
            mma_commit_pair(bar_empty + 8 * s, both);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair(bar_tfull + 8 * acc, both);
        __syncwarp();
        kb0 = kb1;
        if (kb0 == p.nkb) kb0 = 0, u += nclusters;
      }
      // All MMAs have completed before TMEM is freed.
      if (elect_one()) mma_commit_pair(bar_drain, 1u << even);
      __syncwarp();
      mbar_wait_warp(bar_drain, 0u, p.status);
    }
  } else {
    const int quad = warp % 4;
    const int col_lo = ((warp - 2) / 4) * (PN / 2);
    const Epilogue& e = p.e;
    constexpr bool kOutBf = OUT == kOutOther ? !BF16 : BF16;
    Stager st{staging + static_cast<uint32_t>(warp - 2) * 2 * kBox, 0u, lane,
              p.tma_out && (e.z == nullptr || p.tma_z)};
    // What is added to the row before it is rounded: the residual, or the
    // output itself.
    const uint16_t* addend =
        OUT == kOutFwd ? e.res : (OUT != kOut32 && e.accumulate ? static_cast<const uint16_t*>(e.out) : nullptr);
    const long long ld_add = OUT == kOutFwd ? e.ld_res : e.ld_out;
    uint32_t tc = 0;
    for (int u = cluster, kb0 = 0; u < total; ++tc) {
      int R, Cc;
      pair_tile(p, u, R, Cc);
      const uint32_t acc = tc & 1u, aph = (tc >> 1) & 1u;
      const bool add = OUT == kOut32 && (e.accumulate != 0 || kb0 > 0);
      const int row0 = R * 256 + static_cast<int>(rank) * 128 + quad * 32, r = row0 + lane;
      const int cbase = Cc * PN + col_lo;
      const int nch = row0 < p.rows ? min(PN / 64, (p.cols - cbase + 31) / 32) : 0;  // chunks with something to write
      const uint32_t tb = tmem + acc * PN + col_lo + (static_cast<uint32_t>(quad * 32) << 16);
      RowPiece piece, next;
      if (nch > 0) piece.load(addend, ld_add, p, r, cbase);
      if (!mbar_wait_warp(bar_tfull + 8 * acc, aph, p.status)) break;
      fence_after();
      // The previous piece of this tile is in place before this one is added.
      if (OUT == kOut32 && kb0 > 0 && lane == 0) bulk_wait_all();
      uint32_t v[32];
      if (nch > 0) {
        tmem_ld32(tb, v);
        tmem_ld_done(v);
      }
#pragma unroll 1
      for (int i = 0; i < nch; ++i) {
        const int c0 = cbase + 32 * i;
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
        if (i + 1 < nch) {  // the next chunk's loads run under this chunk's work
          tmem_ld32(tb + 32 * (i + 1), v);
          next.load(addend, ld_add, p, r, c0 + 32);
        }
        uint32_t w[16];
        if constexpr (OUT == kOutFwd) {
          if (e.bias != nullptr) add_bias(e, c0, p.cols, f);
          if (e.z != nullptr) {
            to_words<BF16>(f, w);
            if (p.tma_z)
              st.store(&tmZ, w, c0, row0, false);
            else
              st.store_plain<2>(e.z, e.ld_z, p.rows, p.cols, w, c0, row0, false);
          }
          if (e.z8.q != nullptr && r < p.rows) store_block_row(e.z8, r, c0, p.cols, f);
          apply_act(e.act, f);
        }
        if (addend != nullptr && r < p.rows) piece.add<kOutBf>(f);
        if constexpr (OUT == kOut32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 columns a box
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(f[16 * h + j]);
            if (p.tma_out)
              st.store(&tmOut, w, c0 + 16 * h, row0, add);
            else
              st.store_plain<4>(e.out, e.ld_out, p.rows, p.cols, w, c0 + 16 * h, row0, add);
          }
        } else {
          to_words<kOutBf>(f, w);
          if (p.tma_out)
            st.store(&tmOut, w, c0, row0, false);
          else
            st.store_plain<2>(e.out, e.ld_out, p.rows, p.cols, w, c0, row0, false);
          if constexpr (OUT == kOutFwd) {
            if (e.out8.q != nullptr && r < p.rows) store_block_row(e.out8, r, c0, p.cols, f);
          }
        }
        if (i + 1 < nch) tmem_ld_done(v);
        piece = next;
      }
      fence_before();
      mbar_arrive_remote_cta(map_to_rank(bar_tempty + 8 * acc, even));
      kb0 += depth;
      if (kb0 >= p.nkb) kb0 = 0, u += nclusters;
    }
    // Every bulk store has read its box before shared memory goes away.
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  fence_before();
  // No CTA leaves while a peer may still write into its shared memory or arrive
  // on its barriers.
  cluster_sync();
  if (warp == 1) {
    fence_after();
    tmem_free<2>(tmem, C::kTmem);
  }
}

// --------------------------------------------------------------------------
// Host side
// --------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// 16-bit operand [rows][cols], boxes of 64 columns x box_rows rows, 128-byte
// swizzle, zeros outside.
bool operand_map(CUtensorMap* map, const Mat& m, int rows, int cols, int box_rows, int elem) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m.ld) * 2u};
  const cuuint32_t box[2] = {BK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, elem == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, m.p, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [rows][cols] for the epilogue's bulk stores: boxes of 64 bytes x 32
// rows in the 64-byte swizzle of the staging boxes.  False: base or pitch is
// not a multiple of 16 bytes.
bool store_map(CUtensorMap* map, void* p, long long ld, int rows, int cols, int dtype) {
  const int bytes = dtype == kF32 ? 4 : 2;
  if (p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 || (ld * bytes) % 16) return false;
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * bytes};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / bytes), 32u};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType dt = dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, dt, 2, p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::once_flag* once, int dev) {
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63],
                 [&] { err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  return err;
}

// A launch of clusters of `size` CTAs; attr has room for two.
cudaLaunchConfig_t cluster_config(int ctas, int threads, int smem, int size, bool pdl, cudaStream_t s,
                                  cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  if (size > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = size;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cfg;
}

// Clusters of `kern` that the device runs at once.
template <typename K>
int resident_clusters(K kern, int threads, int smem, int size, int dev, std::atomic<int>* cached) {
  std::atomic<int>& c = cached[dev & 63];
  int n = c.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(size, threads, smem, size, false, nullptr, attr);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = std::max(1, sm_count() / size);
    }
    c.store(n, std::memory_order_relaxed);
  }
  return n;
}

// The pair kernel's A is the operand of the output's rows (Product::B) and its
// B that of the columns (Product::A).
template <bool BF16, bool AT, bool BT, int OUT, int PN>
cudaError_t run_pair(const Product& g, const Epilogue& e, unsigned* status, cudaStream_t s) {
  using C = PairCfg<PN>;
  auto kern = pair_kernel<BF16, AT, BT, OUT, PN>;
  static std::once_flag once[64];
  static std::atomic<int> pairs[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t err = allow_smem(kern, C::kDyn, once, dev);
  if (err != cudaSuccess) return err;
  CUtensorMap ta, tb, to, tz;
  if (!operand_map(&ta, g.B, AT ? g.K : g.N, AT ? g.N : g.K, AT ? BK : 128, g.elem)) return cudaErrorInvalidValue;
  if (!operand_map(&tb, g.A, BT ? g.K : g.M, BT ? g.M : g.K, BT ? BK : PN / 2, g.elem)) return cudaErrorInvalidValue;
  memset(&to, 0, sizeof to);
  memset(&tz, 0, sizeof tz);
  PairParams p{};
  p.rows = g.N;
  p.cols = g.M;
  p.nkb = (g.K + BK - 1) / BK;
  p.tiles_r = (g.N + 255) / 256;
  p.tiles_c = (g.M + PN - 1) / PN;
  p.tma_out = store_map(&to, e.out, e.ld_out, g.N, g.M, g.out_dtype);
  p.tma_z = store_map(&tz, e.z, e.ld_z, g.N, g.M, g.elem);
  const uintptr_t add = reinterpret_cast<uintptr_t>(OUT == kOutFwd ? static_cast<const void*>(e.res) : e.out);
  p.vec_res = add % 16 == 0 && (OUT == kOutFwd ? e.ld_res : e.ld_out) % 8 == 0;
  p.e = e;
  p.status = status;
  const long long total = static_cast<long long>(p.tiles_r) * p.tiles_c;
  if (total > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
  const int clusters = static_cast<int>(
      std::min<long long>(total, resident_clusters(kern, C::kThreads, C::kDyn, 2, dev, pairs)));
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = cluster_config(2 * clusters, C::kThreads, C::kDyn, 2, pdl_enabled(), s, attr);
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, to, tz, p);
}

template <bool BF16, bool AT, bool BT, int BN, bool FWD, bool DEEP, bool SUM>
cudaError_t run_tile(const Product& g, const Epilogue& e, int split, unsigned* status, cudaStream_t s) {
  using C = TileCfg<BN, DEEP, SUM>;
  auto kern = tile_kernel<BF16, AT, BT, BN, FWD, DEEP, SUM>;
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t err = allow_smem(kern, C::kDyn, once, dev);
  if (err != cudaSuccess) return err;
  CUtensorMap ta, tb;
  if (!operand_map(&ta, g.A, AT ? g.K : g.M, AT ? g.M : g.K, AT ? BK : BM, g.elem)) return cudaErrorInvalidValue;
  if (!operand_map(&tb, g.B, BT ? g.K : g.N, BT ? g.N : g.K, BT ? BK : BN, g.elem)) return cudaErrorInvalidValue;
  const int tiles_m = (g.M + BM - 1) / BM, nkb = (g.K + BK - 1) / BK;
  const long long ctas = static_cast<long long>(tiles_m) * ((g.N + BN - 1) / BN) * split;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      cluster_config(static_cast<int>(ctas), kTileThreads, C::kDyn, split, pdl_enabled(), s, attr);
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, nkb, tiles_m, split, e, status);
}

// Which kernel a product takes, and how.
struct Plan {
  bool pair;
  int bn, split;  // tile width; CTAs that share a tile's K (tile kernel)
  bool deep;      // one CTA an SM with a deeper ring (tile kernel)
};

// The cheapest by an estimate in microseconds.  Short of large products every
// variant is bound by what the copy engines bring an SM: about 105 KB a
// microsecond with one CTA or a pair's half on it, 135 with two CTAs, while all
// SMs together take 6500 KB a microsecond from HBM.  An operand whose rows do
// not start on 128-byte lines costs more, two of them a good deal more (each
// 128-byte row of a box then lies in two lines).  To that come a launch's fixed
// part, the rows that a tile's epilogue writes, and the join of a split.
// Measured over 64 products of 1 .. 16384 rows and 512 .. 11008 columns, the
// choice is mostly within 10 % of the best of the up to 18 variants that each
// can take: at 256 x 2048 x 2048 (dx) a 64-wide tile with K over 4 CTAs, 11.1 us,
// where a pair a tile takes 15.9; at 16384 x 512 x 512 (dW) K over 8 CTAs, 22 us,
// where a pair takes 77.
Plan plan_product(const Product& g) {
  const int sms = sm_count(), pairs = sms / 2;
  const long long nkb = (g.K + BK - 1) / BK, tm = (g.M + BM - 1) / BM;
  const auto ceil_div = [](long long a, long long b) { return (a + b - 1) / b; };
  const auto off_line = [](const Mat& m) { return m.ld % 64 != 0 || reinterpret_cast<uintptr_t>(m.p) % 128 != 0; };
  const int off = off_line(g.A) + off_line(g.B);
  const double slow256[3] = {1.0, 1.08, 1.4}, slow128[3] = {1.0, 1.05, 1.22}, slow_tile[3] = {1.0, 1.15, 1.35};
  const double hbm = 2.0 * (1.0 * g.M * g.K + 1.0 * g.N * g.K + 1.0 * g.M * g.N) / 1024 / 6500;
  Plan best{};
  double least = 1e30;
  for (int bn : {256, 128}) {
    const long long waves = ceil_div(ceil_div(g.N, 256) * ceil_div(g.M, bn), pairs);
    const double kb = static_cast<double>(waves) * nkb * (16 + bn / 16) * (bn == 256 ? slow256 : slow128)[off];
    const double t = 6.0 + std::max(hbm, kb / (waves > 1 ? 116.0 : 105.0));
    if (t < least) least = t, best = {true, bn, 1, false};
  }
  for (int bn : {128, 64, 32, 16}) {
    if (g.b_mn && bn < 64) break;
    if (bn > 16 && g.N <= bn / 2 && !(g.b_mn && bn == 64)) continue;  // a narrower tile holds every row
    const long long tiles = tm * ceil_div(g.N, bn);
    if (tiles > 16 * sms) continue;
    for (int split = 1; split <= 8 && split * 2 <= std::max(nkb, 2ll); split *= 2) {
      const long long ctas = tiles * split, rounds = ceil_div(ctas, 2 * sms);
      const long long on_sm = rounds > 1 ? 2 * rounds : ceil_div(ctas, sms);
      const double kb = static_cast<double>(on_sm) * ceil_div(nkb, split) * (16 + bn / 8) * slow_tile[off];
      const double t = 5.0 + 3.0 * (rounds - 1) + std::max(hbm, kb / (on_sm > 1 ? 135.0 : 105.0)) +
                       (split > 1 ? 0.6 + 0.02 * bn : 0.0) + (split > 4 ? 3.0 : 0.0) +
                       std::min<long long>(g.N, bn) / split * (g.a_mn ? 0.015 : 0.03);
      if (t < least) least = t, best = {false, bn, split, ctas <= sms && split <= 4};
    }
  }
  return best;
}

template <bool BF16, bool AT, bool BT, int BN, bool FWD>
cudaError_t run_tile_d(const Product& g, const Epilogue& e, const Plan& p, unsigned* status, cudaStream_t s) {
  if constexpr (BT) {
    if (e.out_f32 && g.K > kPiece * BK * p.split)  // a share is longer than a piece
      return p.deep ? run_tile<BF16, AT, BT, BN, FWD, true, true>(g, e, p.split, status, s)
                    : run_tile<BF16, AT, BT, BN, FWD, false, true>(g, e, p.split, status, s);
  }
  return p.deep ? run_tile<BF16, AT, BT, BN, FWD, true, false>(g, e, p.split, status, s)
                : run_tile<BF16, AT, BT, BN, FWD, false, false>(g, e, p.split, status, s);
}
template <bool BF16, bool AT, bool BT, bool FWD>
cudaError_t run_tile_n(const Product& g, const Epilogue& e, const Plan& p, unsigned* status, cudaStream_t s) {
  if constexpr (!BT) {
    if (p.bn == 16) return run_tile_d<BF16, AT, BT, 16, FWD>(g, e, p, status, s);
    if (p.bn == 32) return run_tile_d<BF16, AT, BT, 32, FWD>(g, e, p, status, s);
  }
  if (p.bn <= 64) return run_tile_d<BF16, AT, BT, 64, FWD>(g, e, p, status, s);
  return run_tile_d<BF16, AT, BT, 128, FWD>(g, e, p, status, s);
}

template <bool BF16, bool AT, bool BT, int OUT>
cudaError_t run_pair_n(const Product& g, const Epilogue& e, const Plan& p, unsigned* status, cudaStream_t s) {
  return p.bn == 128 ? run_pair<BF16, AT, BT, OUT, 128>(g, e, status, s)
                     : run_pair<BF16, AT, BT, OUT, 256>(g, e, status, s);
}

// Whether a forward product goes to few_tokens_kernel: enough rows of W for its
// blocks to reach most SMs.
bool few_tokens(const Product& g) {
  return !g.a_mn && g.N <= kFewTokens && g.M >= 2048 && g.K % 8 == 0;
}
template <bool BF16>
cudaError_t run_few(const Product& g, const Epilogue& e, cudaStream_t s) {
  auto kern = g.N == 1   ? few_tokens_kernel<BF16, 1>
              : g.N == 2 ? few_tokens_kernel<BF16, 2>
              : g.N == 3 ? few_tokens_kernel<BF16, 3>
                         : few_tokens_kernel<BF16, 4>;
  return launch_kernel(pdl_enabled(), kern, dim3((g.M + 31) / 32), dim3(256), 0, s,
                       static_cast<const uint16_t*>(g.A.p), g.A.ld, static_cast<const uint16_t*>(g.B.p), g.B.ld, g.K, e);
}

template <bool BF16>
cudaError_t run_product(const Product& g, const Epilogue& e, unsigned* status, cudaStream_t s) {
  if (few_tokens(g)) return run_few<BF16>(g, e, s);
  const Plan p = plan_product(g);
  if (!g.a_mn && !g.b_mn)
    return p.pair ? run_pair_n<BF16, false, false, kOutFwd>(g, e, p, status, s)
                  : run_tile_n<BF16, false, false, true>(g, e, p, status, s);
  if (g.a_mn && !g.b_mn)
    return p.pair ? run_pair_n<BF16, false, true, kOut16>(g, e, p, status, s)
                  : run_tile_n<BF16, true, false, false>(g, e, p, status, s);
  if (g.a_mn && g.b_mn) {
    if (!p.pair) return run_tile_n<BF16, true, true, false>(g, e, p, status, s);
    if (e.out_f32) return run_pair_n<BF16, true, true, kOut32>(g, e, p, status, s);
    return g.out_dtype == g.elem ? run_pair_n<BF16, true, true, kOut16>(g, e, p, status, s)
                                 : run_pair_n<BF16, true, true, kOutOther>(g, e, p, status, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

bool plain_box_map(CUtensorMap* map, const Mat& m, int rows, int cols, int dtype, int box_rows, int box_cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const int bytes = dtype == kF32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m.ld) * bytes};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType dt = dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(map, dt, 2, m.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_product(const Product& g, unsigned* status, cudaStream_t s) {
  Epilogue e{};
  e.M = g.M;
  e.N = g.N;
  e.out = g.out.p;
  e.ld_out = g.out.ld;
  e.out_f32 = g.out_dtype == kF32;
  e.out_bf16 = g.out_dtype == kBF16;
  e.accumulate = g.accumulate;
  e.bias = g.bias;
  e.bias_dtype = g.bias_dtype;
  e.act = g.act;
  e.res = static_cast<const uint16_t*>(g.residual.p);
  e.ld_res = g.residual.ld;
  e.z = static_cast<uint16_t*>(g.z.p);
  e.ld_z = g.z.ld;
  e.z8 = g.z8;
  e.out8 = g.out8;
  return g.elem == kBF16 ? run_product<true>(g, e, status, s) : run_product<false>(g, e, status, s);
}

}  // namespace dion3
