// Internal launcher interface of the model operators (embedding, recurrence,
// log probabilities, gradient norm).  Nothing here crosses the C ABI.
#pragma once

#include <cuda.h>

#include "layer.h"

namespace dion3 {

// Token numbers: signed integers of 4 or 8 bytes.
struct Ids {
  const void* p = nullptr;
  int bytes = 8;
};

// ---------------------------------------------------------------------------
// Embedding (embedding.cu)
// ---------------------------------------------------------------------------
struct EmbedArgs {
  int tokens, vocab, cols;
  Ids ids;
  Mat table; int table_dtype;
  Mat y; int dtype;
  float scale;
};
cudaError_t launch_embedding(const EmbedArgs& a, cudaStream_t s);

// Positions of a window of the grouped tokens, and the workspace's pieces.
int embed_window(int tokens);
struct EmbedGradArgs {
  int tokens, vocab, cols;
  Ids ids;
  Mat dy; int dtype;
  Mat dtable; int table_dtype;
  float scale;
  int accumulate;
  int* order;       // [tokens] positions, grouped by token
  int* token;       // [tokens] their tokens
  int* count;       // [1] positions that have a token
  uint8_t* occurs;  // [embed_slots(vocab)] whether a token does, by its group
  float* partials;  // [2 windows][cols]
  int* arrived;     // [windows][strips of columns] of the runs that begin there
};
int embed_slots(int vocab);
int embed_counters(int tokens, int cols);  // at most
cudaError_t launch_embedding_grad(const EmbedGradArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Recurrence (recurrence.cu): the forward pass, or the gradient.
// ---------------------------------------------------------------------------
struct RecurrenceArgs {
  int tokens, channels, dtype;
  Mat z, x, h;
  const int* offsets;  // [sequences + 1], or null: one sequence
  int sequences;       // >= 1
  const float* first;  // [sequences][channels], may be null
  float* last;         // forward, may be null
  Mat dh, dz, dx;      // gradient
  const float* dlast;  // may be null
  float* dfirst;       // may be null
  bool grad;
  unsigned* status;    // device status word
};
cudaError_t launch_recurrence(const RecurrenceArgs& a, cudaStream_t s);
// Boxes of box_rows x box_cols of a matrix [rows][cols] whose base and pitch are
// multiples of 16 bytes, as they lie in memory, zeros outside (layer_gemm.cu).
bool plain_box_map(CUtensorMap* map, const Mat& m, int rows, int cols, int dtype, int box_rows, int box_cols);

// ---------------------------------------------------------------------------
// Log probabilities (logprob.cu)
// ---------------------------------------------------------------------------
constexpr int kMaxTop = 32;  // alternatives: a list in a warp's lanes
struct LogProbArgs {
  int rows, vocab, dtype;
  Mat logits;
  float scale;
  Ids targets;        // p null: none
  float* logp;        // [rows], may be null
  float* entropy;     // [rows], may be null
  float* stats;       // [rows][3], may be null
  int top;            // 0 .. kMaxTop
  float* top_values;  // [rows][top], may be null
  int* top_ids;       // [rows][top], may be null
};
cudaError_t launch_log_probs(const LogProbArgs& a, cudaStream_t s);

struct LogProbGradArgs {
  int rows, vocab, dtype;
  Mat logits;
  float scale;
  Ids targets;
  const float* stats;
  const float* dlogp;     // [rows], may be null
  const float* dentropy;  // [rows], may be null
  Mat dlogits;            // may be logits
};
cudaError_t launch_log_probs_grad(const LogProbGradArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Gradient norm and clipping (grad_norm.cu)
// ---------------------------------------------------------------------------
struct GradTensor {
  const void* in;
  void* out;
  long long ld_in, ld_out, cols;  // in elements
  int rows;
  unsigned first, per_row;        // chunks before the tensor, and of a row (set by the launcher)
  short dtype, out_dtype;
};
constexpr int kMaxGradPartials = 1024;
// The norm of n tensors (norm: may be null when clipping) and, with clip, out =
// min(1, max_norm / (norm + 1e-6)) in.  partials: [kMaxGradPartials].
cudaError_t launch_grad_norm(const GradTensor* t, int n, bool clip, float max_norm, bool in_place, float* norm,
                             double* partials, cudaStream_t s);

}  // namespace dion3
