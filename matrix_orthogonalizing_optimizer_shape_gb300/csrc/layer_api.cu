// C ABI of the layer operators (include/dion3.h): argument validation,
// workspace carving and launch order.
#include "api_util.h"

#include <algorithm>

namespace dion3 {
namespace {

// Pitch of a 16-bit matrix in the workspace: rows start on 128-byte lines, which
// TMA reads fastest.
long long line_pitch(long long n) { return (n + 63) / 64 * 64; }
size_t matrix_bytes(long long rows, long long cols) { return static_cast<size_t>(rows) * line_pitch(cols) * 2; }

dion3_status check_pack(const char* name, const dion3_packed8& p, int32_t rows, int32_t cols) {
  if (rows == 0) return DION3_OK;
  if (p.codes == nullptr || p.scales == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s: codes or scales NULL", name);
  const int32_t nb = (cols + kPackBlock - 1) / kPackBlock;
  if (p.ld_codes < cols || p.ld_scales < nb)
    return fail(DION3_ERR_INVALID_ARG, "%s: pitches %lld and %lld are smaller than its rows of %d codes and %d scales",
                name, static_cast<long long>(p.ld_codes), static_cast<long long>(p.ld_scales), cols, nb);
  if (p.ld_codes > (1ll << 38) || p.ld_scales > (1ll << 38))
    return fail(DION3_ERR_INVALID_ARG, "%s: pitch too large", name);
  return DION3_OK;
}
bool present(const dion3_packed8* p) { return p != nullptr && (p->codes != nullptr || p->scales != nullptr); }

Pack8 pack(const dion3_packed8& p) { return {p.codes, p.ld_codes, p.scales, p.ld_scales}; }
Pack8 pack(const dion3_packed8* p) { return p == nullptr ? Pack8{} : pack(*p); }

// An operand of a product as TMA takes it (16-byte base and pitch), and as it
// reads it fastest.
bool tma_ready(const Mat& m) { return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % 8 == 0; }
bool on_lines(const Mat& m) { return reinterpret_cast<uintptr_t>(m.p) % 128 == 0 && m.ld % 64 == 0; }
// Whether an operand off the 128-byte lines is worth a copy onto them: a product
// with two such operands takes about a fifth longer than with one (5576 x 1688 x
// 8344: 119 us against 97), a copy what its bytes take at 6 TB/s and a launch.
bool worth_copy(const Mat& m, int rows, int cols, int other) {
  const double n = static_cast<double>(rows) * cols;
  return !on_lines(m) && 0.2 * (2.0 * n * other / 1.7e9) > 1.3 * (4.0 * n / 6.0e6 + 2.5);
}

// The operands of a call that have to be copied first.
struct Staging {
  Repitch job[2];
  int n = 0;
  // m as the products can read it: itself, or its copy in the workspace (if TMA
  // cannot read it, or `anyway`).
  Mat add(Carve& c, const Mat& m, int rows, int cols, bool anyway = false) {
    if (tma_ready(m) && !anyway) return m;
    const Mat dst{c.take(matrix_bytes(rows, cols)), line_pitch(cols)};
    job[n++] = {rows, cols, m, dst};
    return dst;
  }
  double bytes() const {
    double b = 0.0;
    for (int i = 0; i < n; ++i) b += 4.0 * job[i].rows * job[i].cols;
    return b;
  }
  cudaError_t run(cudaStream_t s) const {
    if (n == 0) return cudaSuccess;
    return traced_launch("repitch", 0.0, bytes(), s, [&] { return launch_repitch(job, n, s); });
  }
};

// Results of the layer operators may take any place that no check by name refuses.
constexpr unsigned kAnyPlace = ~0u;

dion3_status check_act(int32_t act) {
  return act < DION3_ACT_NONE || act > DION3_ACT_SILU ? fail(DION3_ERR_INVALID_ARG, "unknown activation %d", act)
                                                      : DION3_OK;
}
dion3_status check_linear_dims(int32_t tokens, int32_t in, int32_t out, int32_t dtype) {
  if (!known_dtype(dtype)) return fail(DION3_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (dtype == DION3_F32) return fail(DION3_ERR_UNSUPPORTED, "the linear layer takes bf16 and fp16 (got fp32)");
  dion3_status rc = check_dims(tokens, in, kMaxCols);
  return rc != DION3_OK ? rc : check_dims(tokens, out, kMaxCols);
}

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

dion3_status dion3_pack8(int32_t rows, int32_t cols, const dion3_matrix* x, const dion3_packed8* out,
                         dion3_stream_t stream) {
  if (x == nullptr || out == nullptr) return fail(DION3_ERR_INVALID_ARG, "x or out is NULL");
  if (!known_dtype(x->dtype)) return fail(DION3_ERR_INVALID_ARG, "x: unknown dtype %d", x->dtype);
  DION3_TRY(check_dims(rows, cols, kMaxCols));
  DION3_TRY(check_mat("x", *x, rows, cols, x->dtype));
  DION3_TRY(check_pack("out", *out, rows, cols));
  DION3_TRY(check_inject());
  if (rows == 0) return ok();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("pack8", 0.0, static_cast<double>(rows) * cols * (bytes_of(x->dtype) + 33.0 / 32), s,
                           [&] { return launch_pack8(rows, cols, x->dtype, mat(x), pack(out), s); }),
             "pack8 launch");
  return ok();
}

dion3_status dion3_unpack8(int32_t rows, int32_t cols, const dion3_packed8* in, const dion3_matrix* out,
                           dion3_stream_t stream) {
  if (in == nullptr || out == nullptr) return fail(DION3_ERR_INVALID_ARG, "in or out is NULL");
  if (!known_dtype(out->dtype)) return fail(DION3_ERR_INVALID_ARG, "out: unknown dtype %d", out->dtype);
  DION3_TRY(check_dims(rows, cols, kMaxCols));
  DION3_TRY(check_pack("in", *in, rows, cols));
  DION3_TRY(check_mat("out", *out, rows, cols, out->dtype));
  DION3_TRY(check_inject());
  if (rows == 0) return ok();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("unpack8", 0.0, static_cast<double>(rows) * cols * (bytes_of(out->dtype) + 33.0 / 32), s,
                           [&] { return launch_unpack8(rows, cols, pack(in), out->dtype, mat(out), s); }),
             "unpack8 launch");
  return ok();
}

dion3_status dion3_rms_norm(int32_t rows, int32_t cols, const dion3_matrix* x, const dion3_matrix* residual,
                            const void* weight, int32_t weight_dtype, float eps, const dion3_matrix* h,
                            const dion3_matrix* y, const dion3_packed8* y8, float* rstd, dion3_stream_t stream) {
  if (x == nullptr) return fail(DION3_ERR_INVALID_ARG, "x is NULL");
  if (!known_dtype(x->dtype)) return fail(DION3_ERR_INVALID_ARG, "x: unknown dtype %d", x->dtype);
  DION3_TRY(check_dims(rows, cols, kNormMaxCols));
  DION3_TRY(check_mat("x", *x, rows, cols, x->dtype));
  DION3_TRY(check_opt("residual", residual, rows, cols, x->dtype));
  DION3_TRY(check_opt("h", h, rows, cols, x->dtype));
  DION3_TRY(check_opt("y", y, rows, cols, x->dtype));
  DION3_TRY(check_vector("weight", weight, weight_dtype));
  DION3_TRY(check_f32("rstd", rstd));
  if (!(eps >= 0.f)) return fail(DION3_ERR_INVALID_ARG, "eps must be >= 0");
  if (present(y8)) DION3_TRY(check_pack("y8", *y8, rows, cols));
  if (rows > 0 && (y == nullptr || y->data == nullptr) && !present(y8))
    return fail(DION3_ERR_INVALID_ARG, "neither y nor y8 is given");
  const Arg args[] = {{"x", extent_of(x, rows, cols), false},
                      {"residual", extent_of(residual, rows, cols), false},
                      {"h", extent_of(h, rows, cols), true, kAnyPlace},
                      {"y", extent_of(y, rows, cols), true, kAnyPlace}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (rows == 0) return ok();
  NormArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.dtype = x->dtype;
  a.x = mat(x);
  a.residual = mat(residual);
  a.h = mat(h);
  a.y = mat(y);
  a.w = weight;
  a.w_dtype = weight_dtype;
  a.eps = eps;
  a.y8 = pack(y8);
  a.rstd = rstd;
  const double n = static_cast<double>(rows) * cols;
  const double bytes = n * bytes_of(x->dtype) * (1 + (a.residual.p != nullptr) + (a.h.p != nullptr) + (a.y.p != nullptr)) +
                       (a.y8.q != nullptr ? n * 33.0 / 32 : 0.0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("rms_norm", 0.0, bytes, s, [&] { return launch_rms_norm(a, s); }), "rms_norm launch");
  return ok();
}

dion3_status dion3_rms_norm_backward_workspace_size(int32_t rows, int32_t cols, size_t* bytes) {
  if (bytes == nullptr) return fail(DION3_ERR_INVALID_ARG, "bytes is NULL");
  DION3_TRY(check_dims(rows, cols, kNormMaxCols));
  *bytes = static_cast<size_t>(std::min(rows, kMaxPartials)) * cols * 4;
  return ok();
}

dion3_status dion3_rms_norm_backward(int32_t rows, int32_t cols, const dion3_matrix* dy, const dion3_matrix* h,
                                     const void* weight, int32_t weight_dtype, const float* rstd,
                                     const dion3_matrix* dh, const dion3_matrix* dx, float* dw, int32_t accumulate,
                                     void* ws, size_t ws_bytes, dion3_stream_t stream) {
  if (dy == nullptr || h == nullptr || dx == nullptr) return fail(DION3_ERR_INVALID_ARG, "dy, h or dx is NULL");
  if (!known_dtype(dy->dtype)) return fail(DION3_ERR_INVALID_ARG, "dy: unknown dtype %d", dy->dtype);
  DION3_TRY(check_dims(rows, cols, kNormMaxCols));
  DION3_TRY(check_mat("dy", *dy, rows, cols, dy->dtype));
  DION3_TRY(check_mat("h", *h, rows, cols, dy->dtype));
  DION3_TRY(check_mat("dx", *dx, rows, cols, dy->dtype));
  DION3_TRY(check_opt("dh", dh, rows, cols, dy->dtype));
  DION3_TRY(check_vector("weight", weight, weight_dtype));
  DION3_TRY(check_f32("rstd", rstd));
  DION3_TRY(check_f32("dw", dw));
  if (rows > 0 && rstd == nullptr) return fail(DION3_ERR_INVALID_ARG, "rstd is NULL");
  const Arg args[] = {{"dy", extent_of(dy, rows, cols), false},
                      {"h", extent_of(h, rows, cols), false},
                      {"dh", extent_of(dh, rows, cols), false},
                      {"dx", extent_of(dx, rows, cols), true, kAnyPlace}};
  DION3_TRY(check_args_apart(args));
  size_t need = 0;
  DION3_TRY(dion3_rms_norm_backward_workspace_size(rows, cols, &need));
  DION3_TRY(check_ws(ws, ws_bytes, dw != nullptr ? need : 0));
  DION3_TRY(check_inject());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dw != nullptr && !accumulate) DION3_CUDA(launch_zero(1, cols, 4, {dw, cols}, s), "zero launch");
    return ok();
  }
  NormGradArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.dtype = dy->dtype;
  a.dy = mat(dy);
  a.h = mat(h);
  a.dh = mat(dh);
  a.dx = mat(dx);
  a.w = weight;
  a.w_dtype = weight_dtype;
  a.rstd = rstd;
  a.dw = dw;
  a.accumulate = accumulate != 0;
  a.partials = static_cast<float*>(ws);
  const double bytes = static_cast<double>(rows) * cols * bytes_of(dy->dtype) * (a.dh.p != nullptr ? 4 : 3);
  DION3_CUDA(traced_launch("rms_norm_backward", 0.0, bytes, s, [&] { return launch_rms_norm_grad(a, s); }),
             "rms_norm_backward launch");
  return ok();
}

dion3_status dion3_linear_workspace_size(int32_t tokens, int32_t in_features, int32_t out_features, int32_t dtype,
                                         int32_t strided, size_t* bytes) {
  if (bytes == nullptr) return fail(DION3_ERR_INVALID_ARG, "bytes is NULL");
  DION3_TRY(check_linear_dims(tokens, in_features, out_features, dtype));
  Carve c{nullptr};
  if (strided || in_features % 8) {
    c.take(matrix_bytes(tokens, in_features));
    c.take(matrix_bytes(out_features, in_features));
  } else if (in_features % 64) {
    c.take(matrix_bytes(std::min(tokens, out_features), in_features));
  }
  *bytes = c.off;
  return ok();
}

dion3_status dion3_linear(const dion3_linear_args* g, void* ws, size_t ws_bytes, dion3_stream_t stream) {
  if (g == nullptr) return fail(DION3_ERR_INVALID_ARG, "args is NULL");
  const int32_t T = g->tokens, K = g->in_features, N = g->out_features, dt = g->w.dtype;
  DION3_TRY(check_linear_dims(T, K, N, dt));
  DION3_TRY(check_act(g->act));
  DION3_TRY(check_mat("x", g->x, T, K, dt));
  DION3_TRY(check_mat("w", g->w, N, K, dt));
  DION3_TRY(check_mat("y", g->y, T, N, dt));
  DION3_TRY(check_opt("residual", &g->residual, T, N, dt));
  DION3_TRY(check_opt("z", &g->z, T, N, dt));
  if (present(&g->z8)) DION3_TRY(check_pack("z8", g->z8, T, N));
  if (present(&g->y8)) DION3_TRY(check_pack("y8", g->y8, T, N));
  if (g->bias != nullptr) DION3_TRY(check_vector("bias", g->bias, g->bias_dtype));
  if (T > 0 && (g->y.data == g->x.data || g->y.data == g->w.data))
    return fail(DION3_ERR_INVALID_ARG, "y may not be x or w");
  Carve c{static_cast<char*>(ws)};
  Staging copies;
  // The copies that there have to be; else one operand of two off the lines, if
  // that pays and the workspace has the room.
  Mat x = copies.add(c, mat(g->x), T, K), w = copies.add(c, mat(g->w), N, K);
  DION3_TRY(check_ws(ws, ws_bytes, T > 0 ? c.off : 0));
  if (T > 0 && copies.n == 0 && !on_lines(x) && !on_lines(w) && ws != nullptr &&
      (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && ws_bytes >= matrix_bytes(std::min(T, N), K)) {
    if (T <= N && worth_copy(x, T, K, N)) x = copies.add(c, x, T, K, true);
    if (T > N && worth_copy(w, N, K, T)) w = copies.add(c, w, N, K, true);
  }
  const Arg args[] = {{"x", extent_of(x.p, T, K, x.ld, 2), false},  // what the product reads: x or its copy
                      {"residual", extent_of(&g->residual, T, N), false},
                      {"y", extent_of(&g->y, T, N), true, kAnyPlace},
                      {"z", extent_of(&g->z, T, N), true, kAnyPlace}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (T == 0) return ok();
  unsigned* st = device_status_ptr();
  if (st == nullptr) return fail(DION3_ERR_CUDA, "cannot resolve the device status word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(copies.run(s), "repitch launch");
  Product p{};
  p.M = N;
  p.N = T;
  p.K = K;
  p.elem = dt;
  p.A = w;
  p.B = x;
  p.out = mat(g->y);
  p.out_dtype = dt;
  p.bias = g->bias;
  p.bias_dtype = g->bias_dtype;
  p.act = g->act;
  p.residual = mat(g->residual);
  p.z = mat(g->z);
  p.z8 = pack(g->z8);
  p.out8 = pack(g->y8);
  DION3_CUDA(traced_launch("linear", 2.0 * T * N * K, 2.0 * (1.0 * T * K + 1.0 * N * K + 1.0 * T * N), s,
                           [&] { return launch_product(p, st, s); }),
             "linear launch");
  return ok();
}

dion3_status dion3_linear_backward_workspace_size(int32_t tokens, int32_t in_features, int32_t out_features,
                                                  int32_t dtype, int32_t strided, size_t* bytes) {
  if (bytes == nullptr) return fail(DION3_ERR_INVALID_ARG, "bytes is NULL");
  DION3_TRY(check_linear_dims(tokens, in_features, out_features, dtype));
  Carve c{nullptr};
  c.take(static_cast<size_t>(std::min(tokens, kMaxPartials)) * out_features * 4);  // column sums of db
  c.take(matrix_bytes(tokens, out_features));                                      // dz
  c.take(matrix_bytes(tokens, in_features));                                       // x from its 8-bit blocks
  if (strided || in_features % 8) c.take(matrix_bytes(out_features, in_features));  // w
  *bytes = c.off;
  return ok();
}

dion3_status dion3_linear_backward(const dion3_linear_grad_args* g, void* ws, size_t ws_bytes,
                                   dion3_stream_t stream) {
  if (g == nullptr) return fail(DION3_ERR_INVALID_ARG, "args is NULL");
  const int32_t T = g->tokens, K = g->in_features, N = g->out_features, dt = g->w.dtype;
  const bool want_dx = g->dx.data != nullptr, want_dw = g->dw.data != nullptr;
  const bool x8 = present(&g->x8), z8 = present(&g->z8), act = g->act != DION3_ACT_NONE;
  DION3_TRY(check_linear_dims(T, K, N, dt));
  DION3_TRY(check_act(g->act));
  DION3_TRY(check_mat("dy", g->dy, T, N, dt));
  DION3_TRY(check_mat("w", g->w, N, K, dt));
  if (want_dx) DION3_TRY(check_mat("dx", g->dx, T, K, dt));
  if (want_dw) {
    if (!known_dtype(g->dw.dtype)) return fail(DION3_ERR_INVALID_ARG, "dw: unknown dtype %d", g->dw.dtype);
    DION3_TRY(check_mat("dw", g->dw, N, K, g->dw.dtype));
    if (x8 && g->x.data != nullptr) return fail(DION3_ERR_INVALID_ARG, "x and x8 are both given");
    if (x8) {
      DION3_TRY(check_pack("x8", g->x8, T, K));
    } else {
      DION3_TRY(check_mat("x", g->x, T, K, dt));
    }
  }
  if (act) {
    if (z8 && g->z.data != nullptr) return fail(DION3_ERR_INVALID_ARG, "z and z8 are both given");
    if (z8) {
      DION3_TRY(check_pack("z8", g->z8, T, N));
    } else {
      DION3_TRY(check_mat("z", g->z, T, N, dt));
    }
  }
  DION3_TRY(check_f32("db", g->db));
  if (T > 0 && want_dx && (g->dx.data == g->dy.data || g->dx.data == g->w.data || (want_dw && g->dx.data == g->x.data)))
    return fail(DION3_ERR_INVALID_ARG, "dx may not be dy, w or (with dw) x");

  // dz is dy itself without an activation, if the products can read it well.
  const bool products = want_dx || want_dw;
  const bool own_dz =
      products && (act || !tma_ready(mat(g->dy)) || (T > 0 && worth_copy(mat(g->dy), T, N, (want_dx + want_dw) * K)));
  Carve c{static_cast<char*>(ws)};
  float* partials = g->db != nullptr
                        ? static_cast<float*>(c.take(static_cast<size_t>(std::min(T, kMaxPartials)) * N * 4))
                        : nullptr;
  Mat dz = mat(g->dy);
  if (own_dz) dz = {c.take(matrix_bytes(T, N)), line_pitch(N)};
  Staging copies;
  Mat x{}, w{};
  if (want_dw && x8) {
    x = {c.take(matrix_bytes(T, K)), line_pitch(K)};
  } else if (want_dw) {
    x = copies.add(c, mat(g->x), T, K, T > 0 && worth_copy(mat(g->x), T, K, N));
  }
  if (want_dx) w = copies.add(c, mat(g->w), N, K);
  DION3_TRY(check_ws(ws, ws_bytes, T > 0 ? c.off : 0));
  const Arg args[] = {{"dy", extent_of(dz.p, T, N, dz.ld, 2), false},  // what the products read, each or its copy
                      {"x", extent_of(x.p, T, K, x.ld, 2), false},
                      {"dx", extent_of(&g->dx, T, K), true, kAnyPlace}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!g->accumulate && want_dw)
      DION3_CUDA(launch_zero(N, K, bytes_of(g->dw.dtype), mat(g->dw), s), "zero launch");
    if (!g->accumulate && g->db != nullptr) DION3_CUDA(launch_zero(1, N, 4, {g->db, N}, s), "zero launch");
    return ok();
  }
  unsigned* st = device_status_ptr();
  if (st == nullptr) return fail(DION3_ERR_CUDA, "cannot resolve the device status word");

  const bool unpack = want_dw && x8;
  bool unpacked = false;
  if (own_dz || g->db != nullptr) {
    ActGradArgs a{};
    a.rows = T;
    a.cols = N;
    a.dtype = dt;
    a.act = g->act;
    a.dy = mat(g->dy);
    if (act && z8) a.z8 = pack(g->z8);
    if (act && !z8) a.z = mat(g->z);
    if (own_dz) a.dz = dz;
    a.db = g->db;
    a.accumulate = g->accumulate != 0;
    a.partials = partials;
    const double n = static_cast<double>(T) * N, xn = unpack ? static_cast<double>(T) * K : 0.0;
    const double bytes = n * (2 + (act ? (z8 ? 33.0 / 32 : 2.0) : 0.0) + (own_dz ? 2 : 0));
    // Small ones in one launch (x8, z8: 1003 x 1544 x 988 24.5 -> 21.7 us, 9864 x
    // 493 x 81 37.4 -> 32.8); at 16 M elements each in its own kernel, whose
    // registers and grid are for what it reads (4000 x 2000 x 2000 65.2 against
    // 67.0, 15448 x 7164 x 88 260 against 306).
    const bool small = T <= kFewRowsOfDz || n + xn + copies.bytes() / 4 < 12e6;
    if (small && (copies.n > 0 || unpack)) {
      const Pack8 none{};
      DION3_CUDA(traced_launch("prepare", 0.0, bytes + copies.bytes() + xn * (2 + 33.0 / 32), s,
                               [&] {
                                 return launch_prepare(a, copies.job, copies.n, T, K, unpack ? pack(g->x8) : none, x,
                                                       s);
                               }),
                 "gradient preparation launch");
      copies.n = 0;
      unpacked = true;
    } else {
      DION3_CUDA(traced_launch("act_grad", 0.0, bytes, s, [&] { return launch_act_grad(a, s); }),
                 "activation gradient launch");
    }
  }
  DION3_CUDA(copies.run(s), "repitch launch");
  if (want_dx) {
    Product p{};
    p.M = K;
    p.N = T;
    p.K = N;
    p.elem = dt;
    p.A = w;
    p.a_mn = true;
    p.B = dz;
    p.out = mat(g->dx);
    p.out_dtype = dt;
    DION3_CUDA(traced_launch("linear_dx", 2.0 * T * N * K, 2.0 * (1.0 * T * K + 1.0 * N * K + 1.0 * T * N), s,
                             [&] { return launch_product(p, st, s); }),
               "dx launch");
  }
  if (want_dw) {
    if (unpack && !unpacked)
      DION3_CUDA(traced_launch("unpack8", 0.0, static_cast<double>(T) * K * (2 + 33.0 / 32), s,
                               [&] { return launch_unpack8(T, K, pack(g->x8), dt, x, s); }),
                 "unpack8 launch");
    Product p{};
    p.M = K;
    p.N = N;
    p.K = T;
    p.elem = dt;
    p.A = x;
    p.a_mn = true;
    p.B = dz;
    p.b_mn = true;
    p.out = mat(g->dw);
    p.out_dtype = g->dw.dtype;
    p.accumulate = g->accumulate != 0;
    DION3_CUDA(traced_launch("linear_dw", 2.0 * T * N * K,
                             (x8 ? 33.0 / 32 : 2.0) * T * K + 2.0 * T * N + 1.0 * bytes_of(g->dw.dtype) * N * K, s,
                             [&] { return launch_product(p, st, s); }),
               "dw launch");
  }
  return ok();
}

}  // extern "C"
