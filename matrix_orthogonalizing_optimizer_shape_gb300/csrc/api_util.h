// What the entry points of the layer and model operators share: errors,
// argument checks and workspace carving.
#pragma once

#include <cstdarg>
#include <cstdio>
#include <numeric>

#include "../../include/dion3.h"
#include "layer.h"

namespace dion3 {

inline dion3_status fail(dion3_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline dion3_status fail(dion3_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error_message(buf);
  return st;
}
inline dion3_status ok() {
  set_last_error_message("");
  return DION3_OK;
}
inline dion3_status cuda_fail(cudaError_t e, const char* what) {
  return fail(DION3_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int32_t kMaxRows = 1 << 30, kMaxCols = 1 << 24;

inline bool known_dtype(int32_t d) { return d == DION3_F32 || d == DION3_BF16 || d == DION3_F16; }
inline int bytes_of(int32_t d) { return d == DION3_F32 ? 4 : 2; }

inline dion3_status check_dims(int32_t rows, int32_t cols, int32_t max_cols) {
  if (rows < 0 || cols < 1) return fail(DION3_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (got %d x %d)", rows, cols);
  if (rows > kMaxRows || cols > max_cols)
    return fail(DION3_ERR_UNSUPPORTED, "%d x %d is larger than this operator takes (%d x %d)", rows, cols, kMaxRows,
                max_cols);
  return DION3_OK;
}

// A matrix of `rows` rows that must be there (its data may be NULL if it has
// no rows).
inline dion3_status check_mat(const char* name, const dion3_matrix& m, int32_t rows, int32_t cols, int32_t dtype) {
  if (rows == 0) return DION3_OK;
  if (m.data == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s is NULL", name);
  if (m.dtype != dtype) return fail(DION3_ERR_INVALID_ARG, "%s has dtype %d, %d is wanted", name, m.dtype, dtype);
  if (m.ld < cols) return fail(DION3_ERR_INVALID_ARG, "%s: pitch %lld is smaller than its row of %d", name,
                               static_cast<long long>(m.ld), cols);
  if (m.ld > (1ll << 38)) return fail(DION3_ERR_INVALID_ARG, "%s: pitch too large", name);
  if (reinterpret_cast<uintptr_t>(m.data) % bytes_of(dtype))
    return fail(DION3_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  return DION3_OK;
}
inline dion3_status check_opt(const char* name, const dion3_matrix* m, int32_t rows, int32_t cols, int32_t dtype) {
  return m == nullptr || m->data == nullptr ? DION3_OK : check_mat(name, *m, rows, cols, dtype);
}
inline dion3_status check_vector(const char* name, const void* w, int32_t dtype) {
  if (!known_dtype(dtype)) return fail(DION3_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
  if (w == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(w) % bytes_of(dtype))
    return fail(DION3_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  return DION3_OK;
}
inline dion3_status check_f32(const char* name, const float* p) {
  if (reinterpret_cast<uintptr_t>(p) % 4) return fail(DION3_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  return DION3_OK;
}
inline dion3_status check_ws(void* ws, size_t bytes, size_t need) {
  if (need == 0) return DION3_OK;
  if (ws == nullptr) return fail(DION3_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(DION3_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < need) return fail(DION3_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", bytes, need);
  return DION3_OK;
}
inline dion3_status check_inject() {
  return inject_launch_failure() ? fail(DION3_ERR_CUDA, "injected launch failure (DION3_INJECT=launch_fail)")
                                 : DION3_OK;
}


inline Mat mat(const dion3_matrix& m) { return {m.data, m.ld}; }
inline Mat mat(const dion3_matrix* m) { return m == nullptr ? Mat{} : mat(*m); }

// The memory of an argument: rows of `row` bytes, `pitch` bytes apart (0: one row, as
// dense ones are together).
struct Extent {
  uintptr_t lo = 0, hi = 0;  // both 0: nothing
  unsigned long long pitch = 0, row = 0;
};
inline Extent extent_of(const void* p, long long rows, long long cols, long long ld, int bytes) {
  if (p == nullptr || rows <= 0 || cols <= 0) return {};
  using ull = unsigned long long;
  const bool one = rows == 1 || ld == cols;
  const ull row = static_cast<ull>(cols) * bytes * (one ? rows : 1), pitch = one ? 0 : static_cast<ull>(ld) * bytes;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, static_cast<uintptr_t>(lo + (rows - 1) * pitch + row), pitch, row};
}
inline Extent extent_of(const dion3_matrix* m, int32_t rows, int32_t cols) {
  return m == nullptr ? Extent{} : extent_of(m->data, rows, cols, m->ld, bytes_of(m->dtype));
}
inline Extent extent_of(const float* p, int32_t rows, int32_t cols) { return extent_of(p, rows, cols, cols, 4); }
// Whether two may share elements: they overlap and are not different columns or rows of
// one matrix, apart modulo what both pitches are multiples of.
inline bool meet(const Extent& a, const Extent& b) {
  if (a.lo > b.lo) return meet(b, a);
  if (b.lo >= a.hi || b.lo == b.hi) return false;
  const unsigned long long pitch = std::gcd(a.pitch, b.pitch);
  if (pitch == 0) return true;
  const unsigned long long at = (b.lo - a.lo) % pitch;
  return !(at >= a.row && at + b.row <= pitch);
}
inline bool same_place(const Extent& a, const Extent& b) {
  return a.lo == b.lo && a.hi == b.hi && a.pitch == b.pitch && a.row == b.row;
}

// What a call reads or writes.  `may`: bits of the arguments before this one whose place
// (all of their memory, at the same pitch) it may take.
struct Arg {
  const char* name;
  Extent e;
  bool written;
  unsigned may = 0;
};
// Refuses results that share memory with other arguments: some rows would be read behind
// the writes of others.
template <size_t N>
inline dion3_status check_args_apart(const Arg (&a)[N]) {
  for (size_t j = 1; j < N; ++j)
    for (size_t i = 0; i < j; ++i)
      if ((a[i].written || a[j].written) && meet(a[i].e, a[j].e) && !((a[j].may >> i & 1) && same_place(a[i].e, a[j].e)))
        return fail(DION3_ERR_INVALID_ARG, "%s and %s share memory", a[i].name, a[j].name);
  return DION3_OK;
}

// Hands out 256-byte aligned pieces of a workspace (base NULL: sizes only).
struct Carve {
  char* base;
  size_t off = 0;
  void* take(size_t bytes) {
    off = (off + 255) / 256 * 256;
    void* p = base != nullptr ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

}  // namespace dion3

#define DION3_TRY(call)                    \
  do {                                     \
    const dion3_status rc_ = (call);       \
    if (rc_ != DION3_OK) return rc_;       \
  } while (0)
#define DION3_CUDA(call, what)                       \
  do {                                               \
    const cudaError_t e_ = (call);                   \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)
