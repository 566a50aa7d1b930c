// C ABI of the model operators (include/dion3.h): argument validation,
// workspace carving and launch order.
#include "api_util.h"
#include "model.h"

#include <algorithm>
#include <memory>
#include <new>

namespace dion3 {
namespace {

constexpr int32_t kMaxGrouped = 1 << 27;    // tokens whose positions are grouped
constexpr int32_t kMaxGroupedVocab = 1 << 24;  // every group's block reads all ids
constexpr int32_t kMaxEmbedCols = 1 << 20;
constexpr int32_t kMaxChannels = 1 << 19;
constexpr int32_t kMaxSequences = 1 << 27;
constexpr int32_t kMaxLogRows = 1 << 21, kMaxVocab = 1 << 21;

dion3_status check_any(const char* name, const dion3_matrix* m, int32_t rows, int32_t cols) {
  if (m == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s is NULL", name);
  if (!known_dtype(m->dtype)) return fail(DION3_ERR_INVALID_ARG, "%s: unknown dtype %d", name, m->dtype);
  return check_mat(name, *m, rows, cols, m->dtype);
}
dion3_status check_ids(const char* name, const void* p, int32_t bytes, int32_t n) {
  if (bytes != 4 && bytes != 8) return fail(DION3_ERR_INVALID_ARG, "%s: numbers of %d bytes, 4 or 8 are wanted", name, bytes);
  if (n > 0 && p == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % bytes)
    return fail(DION3_ERR_INVALID_ARG, "%s is not aligned to its element", name);
  return DION3_OK;
}
dion3_status check_finite(const char* name, float v) {
  return v - v == 0.f ? DION3_OK : fail(DION3_ERR_INVALID_ARG, "%s must be finite", name);
}

dion3_status check_mat_ptr(const char* name, const dion3_matrix* m, int32_t rows, int32_t cols, int32_t dtype) {
  if (m == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s is NULL", name);
  return check_mat(name, *m, rows, cols, dtype);
}
dion3_status check_sequences(const int32_t* offsets, int32_t sequences) {
  if (sequences < 0) return fail(DION3_ERR_INVALID_ARG, "sequences must be >= 0 (got %d)", sequences);
  if (sequences > kMaxSequences) return fail(DION3_ERR_UNSUPPORTED, "more than %d sequences", kMaxSequences);
  if (offsets == nullptr && sequences != 1)
    return fail(DION3_ERR_INVALID_ARG, "offsets is NULL with %d sequences", sequences);
  if (reinterpret_cast<uintptr_t>(offsets) % 4) return fail(DION3_ERR_INVALID_ARG, "offsets is not aligned to its element");
  return DION3_OK;
}
dion3_status check_log_probs(int32_t rows, int32_t vocab, const dion3_matrix* logits, float scale, const void* targets,
                             int32_t target_bytes) {
  DION3_TRY(check_dims(rows, vocab, kMaxVocab));
  if (rows > kMaxLogRows) return fail(DION3_ERR_UNSUPPORTED, "more than %d rows", kMaxLogRows);
  DION3_TRY(check_any("logits", logits, rows, vocab));
  if (!(scale >= 0x1p-20f && scale <= 0x1p20f)) return fail(DION3_ERR_INVALID_ARG, "scale must lie in [2^-20, 2^20]");
  return targets != nullptr ? check_ids("targets", targets, target_bytes, rows) : DION3_OK;
}
dion3_status check_tensor(const char* name, int32_t i, const dion3_tensor& t) {
  if (!known_dtype(t.dtype)) return fail(DION3_ERR_INVALID_ARG, "%s[%d]: unknown dtype %d", name, i, t.dtype);
  if (t.rows < 0 || t.cols < 0) return fail(DION3_ERR_INVALID_ARG, "%s[%d]: negative size", name, i);
  if (t.rows == 0 || t.cols == 0) return DION3_OK;
  if (t.rows > kMaxRows || t.cols > (1ll << 40) || t.ld > (1ll << 40))
    return fail(DION3_ERR_UNSUPPORTED, "%s[%d] is larger than 2^30 rows of 2^40", name, i);
  if (t.data == nullptr) return fail(DION3_ERR_INVALID_ARG, "%s[%d] is NULL", name, i);
  if (t.rows > 1 && t.ld < t.cols)
    return fail(DION3_ERR_INVALID_ARG, "%s[%d]: pitch %lld is smaller than its row of %lld", name, i,
                static_cast<long long>(t.ld), static_cast<long long>(t.cols));
  if (reinterpret_cast<uintptr_t>(t.data) % bytes_of(t.dtype))
    return fail(DION3_ERR_INVALID_ARG, "%s[%d] is not aligned to its element", name, i);
  return DION3_OK;
}

// A tensor of a call that clips.
struct Part : Extent {
  int32_t i;
  bool written;
};
Part part_of(const dion3_tensor& t, int32_t i, bool written) {
  return {extent_of(t.data, t.rows, t.cols, t.ld, bytes_of(t.dtype)), i, written};
}
// Refuses tensors whose elements several would write, or one write and another read.
dion3_status check_apart(const dion3_tensor* in, const dion3_tensor* out, int32_t n) {
  std::unique_ptr<Part[]> all(new (std::nothrow) Part[2 * static_cast<size_t>(n)]);
  if (all == nullptr) return fail(DION3_ERR_UNSUPPORTED, "no host memory for %d tensors", n);
  size_t m = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (in[i].rows == 0 || in[i].cols == 0) continue;
    if (out == nullptr) {
      all[m++] = part_of(in[i], i, true);
      continue;
    }
    const Part a = part_of(in[i], i, false), b = part_of(out[i], i, true);
    all[m++] = b;
    if (a.lo != b.lo || in[i].dtype != out[i].dtype || (in[i].rows > 1 && in[i].ld != out[i].ld)) all[m++] = a;
  }
  std::sort(all.get(), all.get() + m, [](const Part& a, const Part& b) { return a.lo < b.lo; });
  for (size_t j = 0; j < m; ++j)
    for (size_t k = j + 1; k < m && all[k].lo < all[j].hi; ++k)
      if ((all[j].written || all[k].written) && meet(all[j], all[k]))
        return fail(DION3_ERR_INVALID_ARG, "tensors %d and %d share elements", std::min(all[j].i, all[k].i),
                    std::max(all[j].i, all[k].i));
  return DION3_OK;
}

dion3_status grad_norm(const dion3_tensor* in, const dion3_tensor* out, int32_t n, bool clip, float max_norm, float* norm,
                       void* ws, size_t ws_bytes, dion3_stream_t stream) {
  if (n < 0) return fail(DION3_ERR_INVALID_ARG, "n must be >= 0 (got %d)", n);
  if (n > 0 && in == nullptr) return fail(DION3_ERR_INVALID_ARG, "tensors is NULL");
  if (!clip && norm == nullptr) return fail(DION3_ERR_INVALID_ARG, "norm is NULL");
  if (clip && !(max_norm >= 0.f)) return fail(DION3_ERR_INVALID_ARG, "max_norm must be >= 0");
  DION3_TRY(check_f32("norm", norm));
  for (int32_t i = 0; i < n; ++i) {
    DION3_TRY(check_tensor("tensors", i, in[i]));
    if (out == nullptr) continue;
    DION3_TRY(check_tensor("out", i, out[i]));
    if (out[i].rows != in[i].rows || out[i].cols != in[i].cols)
      return fail(DION3_ERR_INVALID_ARG, "out[%d] is not of the size of tensors[%d]", i, i);
  }
  if (clip) DION3_TRY(check_apart(in, out, n));
  DION3_TRY(check_ws(ws, ws_bytes, kMaxGradPartials * sizeof(double)));
  std::unique_ptr<GradTensor[]> t(new (std::nothrow) GradTensor[static_cast<size_t>(n) + 1]);
  if (t == nullptr) return fail(DION3_ERR_UNSUPPORTED, "no host memory for %d tensors", n);
  double bytes = 0.0;
  for (int32_t i = 0; i < n; ++i) {
    const dion3_tensor &a = in[i], &b = out != nullptr ? out[i] : in[i];
    const bool dense = a.rows == 1 || (a.ld == a.cols && b.ld == b.cols);
    t[i] = {a.data, b.data, a.ld, b.ld, dense ? a.rows * a.cols : a.cols, dense ? std::min<int>(a.rows, 1) : static_cast<int>(a.rows),
            0u, 0u, static_cast<short>(a.dtype), static_cast<short>(b.dtype)};
    bytes += static_cast<double>(a.rows) * a.cols * (bytes_of(a.dtype) * (clip ? 2 : 1) + (clip ? bytes_of(b.dtype) : 0));
  }
  DION3_TRY(check_inject());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch(clip ? "clip_grad_norm" : "grad_norm", 0.0, bytes, s,
                           [&] {
                             return launch_grad_norm(t.get(), n, clip, max_norm, out == nullptr, norm,
                                                     static_cast<double*>(ws), s);
                           }),
             clip ? "clip_grad_norm launch" : "grad_norm launch");
  return ok();
}

// Whether two matrices of a call start at the same address.
bool same(const dion3_matrix* a, const dion3_matrix* b) { return a->data != nullptr && a->data == b->data; }

}  // namespace
}  // namespace dion3

using namespace dion3;

extern "C" {

dion3_status dion3_embedding(int32_t tokens, int32_t vocab, int32_t cols, const void* ids, int32_t id_bytes,
                             const dion3_matrix* table, float scale, const dion3_matrix* y, dion3_stream_t stream) {
  DION3_TRY(check_dims(tokens, cols, kMaxEmbedCols));
  DION3_TRY(check_dims(vocab, cols, kMaxEmbedCols));
  DION3_TRY(check_ids("ids", ids, id_bytes, tokens));
  DION3_TRY(check_any("table", table, vocab, cols));
  DION3_TRY(check_any("y", y, tokens, cols));
  DION3_TRY(check_finite("scale", scale));
  if (tokens > 0 && y->data == table->data) return fail(DION3_ERR_INVALID_ARG, "y may not be table");
  const Arg args[] = {{"ids", extent_of(ids, 1, tokens, tokens, id_bytes), false},
                      {"table", extent_of(table, vocab, cols), false},
                      {"y", extent_of(y, tokens, cols), true}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (tokens == 0) return ok();
  EmbedArgs a{tokens, vocab, cols, {ids, id_bytes}, mat(table), table->dtype, mat(y), y->dtype, scale};
  const double n = static_cast<double>(tokens) * cols;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("embedding", 0.0, n * (bytes_of(table->dtype) + bytes_of(y->dtype)), s,
                           [&] { return launch_embedding(a, s); }),
             "embedding launch");
  return ok();
}

dion3_status dion3_embedding_backward_workspace_size(int32_t tokens, int32_t vocab, int32_t cols, size_t* bytes) {
  if (bytes == nullptr) return fail(DION3_ERR_INVALID_ARG, "bytes is NULL");
  DION3_TRY(check_dims(tokens, cols, kMaxEmbedCols));
  DION3_TRY(check_dims(vocab, cols, kMaxEmbedCols));
  if (tokens > kMaxGrouped) return fail(DION3_ERR_UNSUPPORTED, "more than %d tokens", kMaxGrouped);
  if (vocab > kMaxGroupedVocab) return fail(DION3_ERR_UNSUPPORTED, "a vocabulary of more than %d", kMaxGroupedVocab);
  Carve c{nullptr};
  if (tokens > 0) {
    const size_t n = tokens, w = embed_window(tokens);
    c.take(4 * n);
    c.take(4 * n);
    c.take(4);
    c.take(embed_slots(vocab));
    c.take(2 * ((n + w - 1) / w) * cols * 4);
    c.take(4 * static_cast<size_t>(embed_counters(tokens, cols)));
  }
  *bytes = c.off;
  return ok();
}

dion3_status dion3_embedding_backward(int32_t tokens, int32_t vocab, int32_t cols, const dion3_matrix* dy,
                                      const void* ids, int32_t id_bytes, float scale, const dion3_matrix* dtable,
                                      int32_t accumulate, void* ws, size_t ws_bytes, dion3_stream_t stream) {
  size_t need = 0;
  DION3_TRY(dion3_embedding_backward_workspace_size(tokens, vocab, cols, &need));
  DION3_TRY(check_ids("ids", ids, id_bytes, tokens));
  DION3_TRY(check_any("dy", dy, tokens, cols));
  DION3_TRY(check_any("dtable", dtable, vocab, cols));
  DION3_TRY(check_finite("scale", scale));
  if (tokens > 0 && dtable->data != nullptr && dy->data == dtable->data)
    return fail(DION3_ERR_INVALID_ARG, "dtable may not be dy");
  const Arg args[] = {{"ids", extent_of(ids, 1, tokens, tokens, id_bytes), false},
                      {"dy", extent_of(dy, tokens, cols), false},
                      {"dtable", extent_of(dtable, vocab, cols), true},
                      {"workspace", extent_of(ws, 1, need, need, 1), true}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_ws(ws, ws_bytes, need));
  DION3_TRY(check_inject());
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (vocab == 0) return ok();
  if (tokens == 0) {
    if (!accumulate)
      DION3_CUDA(launch_zero(vocab, cols, bytes_of(dtable->dtype), mat(dtable), s), "zero launch");
    return ok();
  }
  EmbedGradArgs a{tokens, vocab,         cols, {ids, id_bytes}, mat(dy), dy->dtype, mat(dtable), dtable->dtype,
                  scale,  accumulate != 0};
  const size_t n = tokens, w = embed_window(tokens);
  Carve c{static_cast<char*>(ws)};
  a.order = static_cast<int*>(c.take(4 * n));
  a.token = static_cast<int*>(c.take(4 * n));
  a.count = static_cast<int*>(c.take(4));
  a.occurs = static_cast<uint8_t*>(c.take(embed_slots(vocab)));
  a.partials = static_cast<float*>(c.take(2 * ((n + w - 1) / w) * cols * 4));
  a.arrived = static_cast<int*>(c.take(4 * static_cast<size_t>(embed_counters(tokens, cols))));
  DION3_CUDA(traced_launch("embedding_backward", 0.0,
                           1.0 * tokens * cols * bytes_of(dy->dtype) + 1.0 * vocab * cols * bytes_of(dtable->dtype), s,
                           [&] { return launch_embedding_grad(a, s); }),
             "embedding_backward launch");
  return ok();
}

dion3_status dion3_recurrence(int32_t tokens, int32_t channels, const dion3_matrix* z, const dion3_matrix* x,
                              const int32_t* offsets, int32_t sequences, const float* first, const dion3_matrix* h,
                              float* last, dion3_stream_t stream) {
  DION3_TRY(check_dims(tokens, channels, kMaxChannels));
  DION3_TRY(check_any("z", z, tokens, channels));
  DION3_TRY(check_mat_ptr("x", x, tokens, channels, z->dtype));
  DION3_TRY(check_mat_ptr("h", h, tokens, channels, z->dtype));
  DION3_TRY(check_sequences(offsets, sequences));
  DION3_TRY(check_f32("first", first));
  DION3_TRY(check_f32("last", last));
  if ((same(h, z) && h->ld != z->ld) || (same(h, x) && h->ld != x->ld))
    return fail(DION3_ERR_INVALID_ARG, "h in the place of z or x needs its pitch");
  const Arg args[] = {{"z", extent_of(z, tokens, channels), false},
                      {"x", extent_of(x, tokens, channels), false},
                      {"first", extent_of(first, sequences, channels), false},
                      {"h", extent_of(h, tokens, channels), true, 3u},
                      {"last", extent_of(last, sequences, channels), true, 4u}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (sequences == 0 || (tokens == 0 && last == nullptr)) return ok();
  RecurrenceArgs a{};
  a.tokens = tokens;
  a.channels = channels;
  a.dtype = z->dtype;
  a.z = mat(z);
  a.x = mat(x);
  a.h = mat(h);
  a.offsets = offsets;
  a.sequences = sequences;
  a.first = first;
  a.last = last;
  a.status = device_status_ptr();
  if (a.status == nullptr) return fail(DION3_ERR_CUDA, "cannot resolve the device status word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("recurrence", 0.0, 3.0 * tokens * channels * bytes_of(z->dtype), s,
                           [&] { return launch_recurrence(a, s); }),
             "recurrence launch");
  return ok();
}

dion3_status dion3_recurrence_backward(int32_t tokens, int32_t channels, const dion3_matrix* dh, const dion3_matrix* z,
                                       const dion3_matrix* x, const dion3_matrix* h, const int32_t* offsets,
                                       int32_t sequences, const float* first, const float* dlast,
                                       const dion3_matrix* dz, const dion3_matrix* dx, float* dfirst,
                                       dion3_stream_t stream) {
  DION3_TRY(check_dims(tokens, channels, kMaxChannels));
  DION3_TRY(check_any("dh", dh, tokens, channels));
  const struct {
    const char* name;
    const dion3_matrix* m;
  } rest[] = {{"z", z}, {"x", x}, {"h", h}, {"dz", dz}, {"dx", dx}};
  for (const auto& r : rest) DION3_TRY(check_mat_ptr(r.name, r.m, tokens, channels, dh->dtype));
  DION3_TRY(check_sequences(offsets, sequences));
  DION3_TRY(check_f32("first", first));
  DION3_TRY(check_f32("dlast", dlast));
  DION3_TRY(check_f32("dfirst", dfirst));
  if (same(dz, h) || same(dx, h) || same(dz, dx))
    return fail(DION3_ERR_INVALID_ARG, "dz and dx may not be h nor one another");
  for (const dion3_matrix* in : {z, x, dh})
    for (const dion3_matrix* o : {dz, dx})
      if (same(in, o) && in->ld != o->ld)
        return fail(DION3_ERR_INVALID_ARG, "dz or dx in the place of an input needs its pitch");
  if (first != nullptr && (first == dfirst))
    return fail(DION3_ERR_INVALID_ARG, "dfirst may not be first");
  const Arg args[] = {{"dh", extent_of(dh, tokens, channels), false},
                      {"z", extent_of(z, tokens, channels), false},
                      {"x", extent_of(x, tokens, channels), false},
                      {"h", extent_of(h, tokens, channels), false},
                      {"first", extent_of(first, sequences, channels), false},
                      {"dlast", extent_of(dlast, sequences, channels), false},
                      {"dz", extent_of(dz, tokens, channels), true, 7u},
                      {"dx", extent_of(dx, tokens, channels), true, 7u},
                      {"dfirst", extent_of(dfirst, sequences, channels), true, 1u << 5}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (sequences == 0 || (tokens == 0 && dfirst == nullptr)) return ok();
  RecurrenceArgs a{};
  a.tokens = tokens;
  a.channels = channels;
  a.dtype = dh->dtype;
  a.z = mat(z);
  a.x = mat(x);
  a.h = mat(h);
  a.offsets = offsets;
  a.sequences = sequences;
  a.first = first;
  a.dh = mat(dh);
  a.dz = mat(dz);
  a.dx = mat(dx);
  a.dlast = dlast;
  a.dfirst = dfirst;
  a.grad = true;
  a.status = device_status_ptr();
  if (a.status == nullptr) return fail(DION3_ERR_CUDA, "cannot resolve the device status word");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("recurrence_backward", 0.0, 6.0 * tokens * channels * bytes_of(dh->dtype), s,
                           [&] { return launch_recurrence(a, s); }),
             "recurrence_backward launch");
  return ok();
}

dion3_status dion3_log_probs(int32_t rows, int32_t vocab, const dion3_matrix* logits, float scale, const void* targets,
                             int32_t target_bytes, float* logp, float* entropy, float* stats, int32_t top,
                             float* top_values, int32_t* top_ids, dion3_stream_t stream) {
  DION3_TRY(check_log_probs(rows, vocab, logits, scale, targets, target_bytes));
  DION3_TRY(check_f32("logp", logp));
  DION3_TRY(check_f32("entropy", entropy));
  DION3_TRY(check_f32("stats", stats));
  DION3_TRY(check_f32("top_values", top_values));
  DION3_TRY(check_f32("top_ids", reinterpret_cast<const float*>(top_ids)));
  if (rows > 0 && logp != nullptr && targets == nullptr) return fail(DION3_ERR_INVALID_ARG, "logp is given without targets");
  if (top < 0 || top > kMaxTop || top > vocab)
    return fail(DION3_ERR_INVALID_ARG, "top must lie in [0, %d] (got %d)", std::min(kMaxTop, vocab), top);
  const Arg args[] = {{"logits", extent_of(logits, rows, vocab), false},
                      {"logp", extent_of(logp, rows, 1), true},
                      {"entropy", extent_of(entropy, rows, 1), true},
                      {"stats", extent_of(stats, rows, 3), true},
                      {"top_values", extent_of(top_values, rows, top), true},
                      {"top_ids", extent_of(top_ids, rows, top, top, 4), true}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (rows == 0) return ok();
  LogProbArgs a{};
  a.rows = rows;
  a.vocab = vocab;
  a.dtype = logits->dtype;
  a.logits = mat(logits);
  a.scale = scale;
  a.targets = {targets, target_bytes};
  a.logp = logp;
  a.entropy = entropy;
  a.stats = stats;
  a.top = top_values != nullptr || top_ids != nullptr ? top : 0;
  a.top_values = top_values;
  a.top_ids = top_ids;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("log_probs", 0.0, 1.0 * rows * vocab * bytes_of(logits->dtype), s,
                           [&] { return launch_log_probs(a, s); }),
             "log_probs launch");
  return ok();
}

dion3_status dion3_log_probs_backward(int32_t rows, int32_t vocab, const dion3_matrix* logits, float scale,
                                      const void* targets, int32_t target_bytes, const float* stats,
                                      const float* dlogp, const float* dentropy, const dion3_matrix* dlogits,
                                      dion3_stream_t stream) {
  DION3_TRY(check_log_probs(rows, vocab, logits, scale, targets, target_bytes));
  DION3_TRY(check_mat_ptr("dlogits", dlogits, rows, vocab, logits->dtype));
  DION3_TRY(check_f32("stats", stats));
  DION3_TRY(check_f32("dlogp", dlogp));
  DION3_TRY(check_f32("dentropy", dentropy));
  if (rows > 0 && stats == nullptr) return fail(DION3_ERR_INVALID_ARG, "stats is NULL");
  if (rows > 0 && dlogp != nullptr && targets == nullptr) return fail(DION3_ERR_INVALID_ARG, "dlogp is given without targets");
  if (same(logits, dlogits) && logits->ld != dlogits->ld)
    return fail(DION3_ERR_INVALID_ARG, "dlogits in the place of logits needs its pitch");
  const Arg args[] = {{"logits", extent_of(logits, rows, vocab), false},
                      {"targets", targets == nullptr ? Extent{} : extent_of(targets, 1, rows, rows, target_bytes), false},
                      {"stats", extent_of(stats, rows, 3), false},
                      {"dlogp", extent_of(dlogp, rows, 1), false},
                      {"dentropy", extent_of(dentropy, rows, 1), false},
                      {"dlogits", extent_of(dlogits, rows, vocab), true, 1u}};
  DION3_TRY(check_args_apart(args));
  DION3_TRY(check_inject());
  if (rows == 0) return ok();
  LogProbGradArgs a{rows,  vocab, logits->dtype, mat(logits), scale, {targets, target_bytes},
                    stats, dlogp, dentropy,      mat(dlogits)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DION3_CUDA(traced_launch("log_probs_backward", 0.0, 2.0 * rows * vocab * bytes_of(logits->dtype), s,
                           [&] { return launch_log_probs_grad(a, s); }),
             "log_probs_backward launch");
  return ok();
}

dion3_status dion3_grad_norm_workspace_size(size_t* bytes) {
  if (bytes == nullptr) return fail(DION3_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = kMaxGradPartials * sizeof(double);
  return ok();
}

dion3_status dion3_grad_norm(const dion3_tensor* tensors, int32_t n, float* norm, void* ws, size_t ws_bytes,
                             dion3_stream_t stream) {
  return grad_norm(tensors, nullptr, n, false, 0.f, norm, ws, ws_bytes, stream);
}

dion3_status dion3_clip_grad_norm(const dion3_tensor* tensors, const dion3_tensor* out, int32_t n, float max_norm,
                                  float* norm, void* ws, size_t ws_bytes, dion3_stream_t stream) {
  return grad_norm(tensors, out, n, true, max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
