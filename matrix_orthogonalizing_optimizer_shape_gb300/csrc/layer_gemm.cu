// Tensor-core products of the linear layer on sm_103a (see Product in
// layer.h): out[t][m] = sum_k A(m, k) B(t, k), fp32 accumulation in tensor
// memory, operands K-major or MN-major in 16 bits.
//   forward:  A = W,   B = x:   z = v + bias, y = act(z) + residual, with z
//             and y also in 8-bit blocks
//   dx:       A = W^T, B = dz
//   dW:       A = x^T, B = dz^T
//
// Kernel: one CTA computes a tile of 128 m x BN t.  m runs along the TMEM
// lanes, so the 32 lanes of a warp hold 32 consecutive columns of an output
// row: 16-bit rows are written in 64-byte pieces, and the 32 columns of an
// 8-bit block are one warp's lanes.  Warp 0 fills a ring of 64-wide K slabs
// by TMA, warp 1 issues the MMAs, warps 2..5 (one per TMEM lane quadrant) are
// the epilogue.  Every wait is bounded (about a second) and records
// kDevTimeout in the status word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "layer_math.cuh"
#include "tc_ops.cuh"

namespace dion3 {
namespace {

using namespace tc;
using namespace lm;

constexpr int BM = 128;
constexpr int BK = 64;  // 16-bit elements of one 128-byte swizzle row

struct Epilogue {
  int M, N;
  void* out; long long ld_out; int out_f32, accumulate;
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

// One 8-bit block held by a warp: lane = column of the block (0 past the end).
__device__ __forceinline__ void store_block_warp(const Pack8& o, long long t, int m, bool in, float v) {
  const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
  if (!in) return;
  float u[1] = {v};
  saturate_block(byte, u);
  o.q[t * o.ldq + m] = static_cast<int8_t>(code_of(u[0], inv_scale(byte)));
  if (m % kPackBlock == 0) o.s[t * o.lds + m / kPackBlock] = static_cast<uint8_t>(byte);
}

// Values v[0..C) of output rows t0.. at column m (in: m < M).  Run by a whole
// warp whose lanes hold 32 consecutive columns.
template <bool BF16, bool FWD, int C>
__device__ __forceinline__ void epilogue_rows(const Epilogue& e, int t0, int m, bool in, float bias, float (&v)[C]) {
  if constexpr (FWD) {
    uint16_t r[C];
    if (e.res != nullptr) {
#pragma unroll
      for (int j = 0; j < C; ++j)
        r[j] = in && t0 + j < e.N ? e.res[static_cast<long long>(t0 + j) * e.ld_res + m] : uint16_t(0);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (t0 + j >= e.N) break;
      const long long t = t0 + j;
      const float z = in ? v[j] + bias : 0.f;
      if (e.z != nullptr && in) e.z[t * e.ld_z + m] = pack1<BF16>(z);
      if (e.z8.q != nullptr) store_block_warp(e.z8, t, m, in, z);
      float y = act_fwd(e.act, z);
      if (e.res != nullptr) y += unpack1<BF16>(r[j]);
      if (in) static_cast<uint16_t*>(e.out)[t * e.ld_out + m] = pack1<BF16>(y);
      if (e.out8.q != nullptr) store_block_warp(e.out8, t, m, in, in ? y : 0.f);
    }
  } else if (e.out_f32) {
    float* o = static_cast<float*>(e.out) + static_cast<long long>(t0) * e.ld_out + m;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (in && t0 + j < e.N) o[j * e.ld_out] = e.accumulate ? o[j * e.ld_out] + v[j] : v[j];
  } else {
    uint16_t* o = static_cast<uint16_t*>(e.out) + static_cast<long long>(t0) * e.ld_out + m;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (in && t0 + j < e.N)
        o[j * e.ld_out] = pack1<BF16>(e.accumulate ? unpack1<BF16>(o[j * e.ld_out]) + v[j] : v[j]);
  }
}

template <int BN>
struct TileCfg {
  static constexpr int kABytes = BM * BK * 2;
  static constexpr int kBBytes = BN * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 96 * 1024 / kStageBytes;  // two CTAs an SM
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kTmemCols = BN < 32 ? 32 : BN;
  static constexpr int kBars = (2 * kStages + 2) * 8;
  static constexpr int kDyn = 1024 + kRing + kBars + 16;
};
constexpr int kTileThreads = 6 * 32;

template <bool BF16, bool AT, bool BT, int BN, bool FWD>
__global__ void __launch_bounds__(kTileThreads)
    tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, int nkb, int tiles_m,
                Epilogue e, unsigned* status) {
  using C = TileCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sA = base, sB = base + C::kStages * C::kABytes;
  const uint32_t bar_full = base + C::kRing, bar_empty = bar_full + 8 * C::kStages, bar_done = bar_empty + 8 * C::kStages,
                 bar_drain = bar_done + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (base - raw) + C::kRing + C::kBars);
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_done, 1);
    mbar_init(bar_drain, 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), C::kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int m0 = (blockIdx.x % tiles_m) * BM, t0 = (blockIdx.x / tiles_m) * BN;

  if (warp == 0) {
    int kb = 0;
    for (; kb < nkb; ++kb) {
      const uint32_t s = kb % C::kStages, ph = (kb / C::kStages) & 1u;
      if (!mbar_wait_warp(bar_empty + 8 * s, ph ^ 1u, status)) break;
      const uint32_t a = sA + s * C::kABytes, b = sB + s * C::kBBytes, full = bar_full + 8 * s;
      const int k0 = kb * BK;
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
    bool ok = true;
    for (int kb = 0; kb < nkb && ok; ++kb) {
      const uint32_t s = kb % C::kStages, ph = (kb / C::kStages) & 1u;
      if (!(ok = mbar_wait_warp(bar_full + 8 * s, ph, status))) break;
      fence_after();
      const uint64_t da = smem_desc<AT>(sA + s * C::kABytes), db = smem_desc<BT>(sB + s * C::kBBytes);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_f16<1>(tmem, da + kDescStep<AT> * kk, db + kDescStep<BT> * kk, id, (kb > 0 || kk > 0) ? 1u : 0u);
        mma_commit(bar_empty + 8 * s);
        if (kb == nkb - 1) mma_commit(bar_done);
      }
      __syncwarp();
    }
    // All MMAs have completed before TMEM is freed.
    if (elect_one()) mma_commit(bar_drain);
    __syncwarp();
    mbar_wait_warp(bar_drain, 0u, status);
  } else {
    const int quad = warp % 4;
    const int m = m0 + quad * 32 + lane;
    const bool in = m < e.M;
    const float bias = FWD && e.bias != nullptr && in ? load_bias(e.bias, e.bias_dtype, m) : 0.f;
    if (mbar_wait_warp(bar_done, 0u, status)) {
      fence_after();
      constexpr int CH = BN < 32 ? 16 : 32;
      const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN; c += CH) {
        if (t0 + c >= e.N) break;
        uint32_t u[CH];
        if constexpr (CH == 16)
          tmem_ld16(tb + c, u);
        else
          tmem_ld32(tb + c, u);
        tmem_ld_done(u);
        float v[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) v[j] = __uint_as_float(u[j]);
        epilogue_rows<BF16, FWD, CH>(e, t0 + c, m, in, bias, v);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<1>(tmem, C::kTmemCols);
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

template <bool BF16, bool AT, bool BT, int BN, bool FWD>
cudaError_t run_tile(const Product& g, const Epilogue& e, unsigned* status, cudaStream_t s) {
  using C = TileCfg<BN>;
  auto kern = tile_kernel<BF16, AT, BT, BN, FWD>;
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDyn);
  });
  if (err != cudaSuccess) return err;
  CUtensorMap ta, tb;
  if (!operand_map(&ta, g.A, AT ? g.K : g.M, AT ? g.M : g.K, AT ? BK : BM, g.elem)) return cudaErrorInvalidValue;
  if (!operand_map(&tb, g.B, BT ? g.K : g.N, BT ? g.N : g.K, BT ? BK : BN, g.elem)) return cudaErrorInvalidValue;
  const int tiles_m = (g.M + BM - 1) / BM;
  const long long tiles = static_cast<long long>(tiles_m) * ((g.N + BN - 1) / BN);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_kernel(pdl_enabled(), kern, dim3(static_cast<unsigned>(tiles)), dim3(kTileThreads), C::kDyn, s, ta, tb,
                       (g.K + BK - 1) / BK, tiles_m, e, status);
}

template <bool BF16>
cudaError_t run_product(const Product& g, const Epilogue& e, bool fwd, unsigned* status, cudaStream_t s) {
  if (fwd) return run_tile<BF16, false, false, 128, true>(g, e, status, s);
  if (g.a_mn && !g.b_mn) return run_tile<BF16, true, false, 128, false>(g, e, status, s);
  if (g.a_mn && g.b_mn) return run_tile<BF16, true, true, 128, false>(g, e, status, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_product(const Product& g, unsigned* status, cudaStream_t s) {
  Epilogue e{};
  e.M = g.M;
  e.N = g.N;
  e.out = g.out.p;
  e.ld_out = g.out.ld;
  e.out_f32 = g.out_dtype == kF32;
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
  const bool fwd = !g.a_mn && !g.b_mn;
  return g.elem == kBF16 ? run_product<true>(g, e, fwd, status, s) : run_product<false>(g, e, fwd, status, s);
}

}  // namespace dion3
