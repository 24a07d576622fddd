// C ABI of the language-model operators: argument checks, workspace layout and
// launches.  See include/mpopt.h for the contract of every entry point.

#include <cmath>

#include "../../include/mpopt.h"
#include "checks.h"
#include "internal.h"

namespace mpopt {
namespace {

bool index_dtype(int32_t d) { return d == OPT_INDEX_INT32 || d == OPT_INDEX_INT64; }

int index_size(int32_t d) { return d == OPT_INDEX_INT32 ? 4 : 8; }

bool extent(int64_t n, int64_t least) { return n >= least && n <= kMaxExtent; }

int64_t blocks_of(int64_t cols) { return (cols + OPT_CHECKPOINT_BLOCK - 1) / OPT_CHECKPOINT_BLOCK; }

// An output that starts where an input does has to be the same matrix.
bool same_or_apart(const void* out, int64_t out_ld, const void* in, int64_t in_ld) { return out != in || out_ld == in_ld; }

bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a && b && p < q + bytes && q < p + bytes;
}

size_t key_bytes(int64_t rows) { return round_up(static_cast<size_t>(rows) * 4, 256); }

template <typename Launch>
opt_status run(int kernel, int64_t a, int64_t b, cudaStream_t st, const char* where, Launch&& launch) {
  prof_begin(kernel, 1, a, b, st);
  const cudaError_t e = launch();
  prof_end(st);
  return cuda_status(e, where);
}

// What the forward and the backward recurrence have in common.
opt_status check_sequences(int64_t rows, int64_t cols, int64_t sequences, const int32_t* starts, const float* h0) {
  if (!extent(rows, 0) || !extent(cols, 1) || !extent(sequences, 1)) return OPT_ERR_INVALID_ARG;
  if (!starts && rows % sequences) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_vector(starts, true, 4));
  return check_vector(h0, true, 4);
}

size_t state_bytes(int64_t sequences, int64_t cols) { return static_cast<size_t>(sequences) * static_cast<size_t>(cols) * 4; }

// dst <- src or zeros: the states behind sequences that have no rows.
opt_status copy_states(float* dst, const float* src, size_t bytes, cudaStream_t st) {
  if (!dst || dst == src) return OPT_OK;
  return cuda_status(src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(dst, 0, bytes, st),
                     "recurrence states");
}

}  // namespace
}  // namespace mpopt

using namespace mpopt;

extern "C" {

opt_status opt_embedding_forward(const opt_embedding_args* a, void* stream) {
  if (!a || !extent(a->rows, 0) || !extent(a->vocab, 1) || !extent(a->cols, 1)) return OPT_ERR_INVALID_ARG;
  if (!index_dtype(a->index_dtype) || !float_dtype(a->dtype) || !float_dtype(a->y_dtype)) return OPT_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return OPT_ERR_INVALID_ARG;
  if (a->rows == 0) return OPT_OK;
  MPOPT_TRY(check_vector(a->tokens, false, index_size(a->index_dtype)));
  MPOPT_TRY(check_matrix(a->table, false, a->table_ld, a->vocab, a->cols, elem_size(a->dtype)));
  MPOPT_TRY(check_matrix(a->y, false, a->y_ld, a->rows, a->cols, elem_size(a->y_dtype)));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(OPT_KERNEL_EMBEDDING, a->rows, a->cols, st, "embedding launch", [&] { return launch_embedding(*a, st); });
}

size_t opt_embedding_workspace_size(int64_t rows, int64_t vocab, int64_t cols) {
  if (!extent(rows, 1) || !extent(vocab, 1) || !extent(cols, 1)) return 0;
  return 4 * key_bytes(rows) + static_cast<size_t>(embedding_most_pieces(rows)) * 2 * static_cast<size_t>(cols) * 4;
}

opt_status opt_embedding_backward(const opt_embedding_grad_args* a, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  if (!a || !extent(a->rows, 0) || !extent(a->vocab, 1) || !extent(a->cols, 1)) return OPT_ERR_INVALID_ARG;
  if (!index_dtype(a->index_dtype) || !float_dtype(a->dtype) || !std::isfinite(a->scale)) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_vector(a->dtable, false, 4));
  if (a->rows > 0) {
    MPOPT_TRY(check_vector(a->tokens, false, index_size(a->index_dtype)));
    MPOPT_TRY(check_matrix(a->dy, false, a->dy_ld, a->rows, a->cols, elem_size(a->dtype)));
    MPOPT_TRY(check_workspace(workspace, workspace_bytes, opt_embedding_workspace_size(a->rows, a->vocab, a->cols)));
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!a->accumulate)
    MPOPT_TRY(cuda_status(cudaMemsetAsync(a->dtable, 0, static_cast<size_t>(a->vocab) * static_cast<size_t>(a->cols) * 4, st),
                          "embedding gradient clear"));
  if (a->rows == 0) return OPT_OK;
  EmbeddingScratch ws;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  const size_t kb = key_bytes(a->rows);
  for (int i = 0; i < 2; ++i) {
    ws.key[i] = reinterpret_cast<uint32_t*>(p + 2 * i * kb);
    ws.row[i] = reinterpret_cast<uint32_t*>(p + (2 * i + 1) * kb);
  }
  ws.partial = reinterpret_cast<float*>(p + 4 * kb);
  int sorted = 0;
  MPOPT_TRY(run(OPT_KERNEL_EMBEDDING_SORT, a->rows, a->vocab, st, "embedding sort launch",
                [&] { return launch_embedding_sort(*a, ws, &sorted, st); }));
  MPOPT_TRY(run(OPT_KERNEL_EMBEDDING_GRAD, a->rows, a->cols, st, "embedding gradient launch",
                [&] { return launch_embedding_sums(*a, ws, sorted, st); }));
  if (embedding_pieces(a->rows) == 1) return OPT_OK;
  return run(OPT_KERNEL_EMBEDDING_JOIN, a->rows, a->cols, st, "embedding join launch",
             [&] { return launch_embedding_join(*a, ws, sorted, st); });
}

int64_t opt_recurrence_state_rows(int32_t dtype) { return float_dtype(dtype) ? kRecurrenceStateRows : 0; }

opt_status opt_recurrence_forward(const opt_recurrence_args* a, void* stream) {
  if (!a || !float_dtype(a->dtype)) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_sequences(a->rows, a->cols, a->sequences, a->starts, a->h0));
  MPOPT_TRY(check_vector(a->hT, true, 4));
  MPOPT_TRY(check_vector(a->states, true, 4));
  const size_t bytes = state_bytes(a->sequences, a->cols);
  const bool single = !a->starts && (a->rows == a->sequences || a->rows == 0);
  if (overlap(a->hT, a->h0, bytes) && !(a->hT == a->h0 && single)) return OPT_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) return copy_states(a->hT, a->h0, bytes, st);
  const int es = elem_size(a->dtype);
  MPOPT_TRY(check_matrix(a->x, false, a->x_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->gate, false, a->gate_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->y, false, a->y_ld, a->rows, a->cols, es));
  if (a->rows > 1 && (!same_or_apart(a->y, a->y_ld, a->x, a->x_ld) || !same_or_apart(a->y, a->y_ld, a->gate, a->gate_ld)))
    return OPT_ERR_INVALID_ARG;
  return run(OPT_KERNEL_RECURRENCE, a->rows, a->cols, st, "recurrence launch", [&] { return launch_recurrence(*a, st); });
}

opt_status opt_recurrence_backward(const opt_recurrence_grad_args* a, void* stream) {
  if (!a || !float_dtype(a->dtype)) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_sequences(a->rows, a->cols, a->sequences, a->starts, a->h0));
  MPOPT_TRY(check_vector(a->dhT, true, 4));
  MPOPT_TRY(check_vector(a->dh0, true, 4));
  const size_t bytes = state_bytes(a->sequences, a->cols);
  if (overlap(a->dh0, a->dhT, bytes) || overlap(a->dh0, a->h0, bytes)) return OPT_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) return copy_states(a->dh0, a->dhT, bytes, st);
  const int es = elem_size(a->dtype);
  MPOPT_TRY(check_vector(a->states, false, 4));
  MPOPT_TRY(check_matrix(a->dy, false, a->dy_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->x, false, a->x_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->gate, false, a->gate_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->dx, false, a->dx_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->dgate, false, a->dgate_ld, a->rows, a->cols, es));
  if (a->dx == a->dgate) return OPT_ERR_INVALID_ARG;
  if (a->rows > 1) {
    const void* in[3] = {a->dy, a->x, a->gate};
    const int64_t ld[3] = {a->dy_ld, a->x_ld, a->gate_ld};
    for (int i = 0; i < 3; ++i)
      if (!same_or_apart(a->dx, a->dx_ld, in[i], ld[i]) || !same_or_apart(a->dgate, a->dgate_ld, in[i], ld[i]))
        return OPT_ERR_INVALID_ARG;
  }
  return run(OPT_KERNEL_RECURRENCE_GRAD, a->rows, a->cols, st, "recurrence gradient launch",
             [&] { return launch_recurrence_grad(*a, st); });
}

opt_status opt_checkpoint_save(const void* x, int64_t x_ld, int32_t dtype, int64_t rows, int64_t cols, uint8_t* q,
                               int64_t q_ld, uint8_t* scale, int64_t scale_ld, void* stream) {
  if (!extent(rows, 0) || !extent(cols, 1) || !float_dtype(dtype)) return OPT_ERR_INVALID_ARG;
  if (rows == 0) return OPT_OK;
  MPOPT_TRY(check_matrix(x, false, x_ld, rows, cols, elem_size(dtype)));
  MPOPT_TRY(check_matrix(q, false, q_ld, rows, cols, 1));
  MPOPT_TRY(check_matrix(scale, false, scale_ld, rows, blocks_of(cols), 1));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(OPT_KERNEL_CHECKPOINT_SAVE, rows, cols, st, "checkpoint launch",
             [&] { return launch_checkpoint_save(x, x_ld, dtype, rows, cols, q, q_ld, scale, scale_ld, st); });
}

opt_status opt_checkpoint_restore(const opt_checkpoint_args* a, void* stream) {
  if (!a || !extent(a->rows, 0) || !extent(a->cols, 1)) return OPT_ERR_INVALID_ARG;
  if (a->act < OPT_ACT_NONE || a->act > OPT_ACT_SILU) return OPT_ERR_INVALID_ARG;
  if (a->rows == 0) return OPT_OK;
  if (!a->dy != !a->dz) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_matrix(a->q, false, a->q_ld, a->rows, a->cols, 1));
  MPOPT_TRY(check_matrix(a->scale, false, a->scale_ld, a->rows, blocks_of(a->cols), 1));
  MPOPT_TRY(check_matrix(a->dy, true, a->dy_ld, a->rows, a->cols, 2));
  MPOPT_TRY(check_matrix(a->z, true, a->z_ld, a->rows, a->cols, 2));
  MPOPT_TRY(check_matrix(a->y, true, a->y_ld, a->rows, a->cols, 2));
  MPOPT_TRY(check_matrix(a->dz, true, a->dz_ld, a->rows, a->cols, 2));
  if (a->dz && a->rows > 1 && !same_or_apart(a->dz, a->dz_ld, a->dy, a->dy_ld)) return OPT_ERR_INVALID_ARG;
  if (!a->z && !a->y && !a->dz) return OPT_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(OPT_KERNEL_CHECKPOINT_RESTORE, a->rows, a->cols, st, "checkpoint restore launch",
             [&] { return launch_checkpoint_restore(*a, st); });
}

opt_status opt_cross_entropy(const opt_cross_entropy_args* a, void* stream) {
  if (!a || !extent(a->rows, 0) || !extent(a->cols, 1)) return OPT_ERR_INVALID_ARG;
  if (!float_dtype(a->dtype) || !index_dtype(a->index_dtype) || !std::isfinite(a->scale)) return OPT_ERR_INVALID_ARG;
  if (a->rows == 0) return OPT_OK;
  const int es = elem_size(a->dtype);
  MPOPT_TRY(check_matrix(a->logits, false, a->logits_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_vector(a->labels, false, index_size(a->index_dtype)));
  MPOPT_TRY(check_vector(a->weight, true, 4));
  MPOPT_TRY(check_vector(a->loss, true, 4));
  MPOPT_TRY(check_vector(a->lse, true, 4));
  MPOPT_TRY(check_matrix(a->dlogits, true, a->dlogits_ld, a->rows, a->cols, es));
  if (a->rows > 1 && !same_or_apart(a->dlogits, a->dlogits_ld, a->logits, a->logits_ld)) return OPT_ERR_INVALID_ARG;
  if (!a->loss && !a->lse && !a->dlogits) return OPT_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(OPT_KERNEL_CROSS_ENTROPY, a->rows, a->cols, st, "cross-entropy launch", [&] { return launch_cross_entropy(*a, st); });
}

opt_status opt_selftest_mail(float* sums, int32_t ctas, int32_t messages, int32_t held_back, void* stream) {
  if (ctas < 2 || ctas > 8 || messages < 1 || messages > 64 || held_back < -1 || held_back >= messages) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_vector(sums, false, 4));
  return cuda_status(launch_mail_selftest(sums, ctas, messages, held_back, static_cast<cudaStream_t>(stream)), "mail self-test launch");
}

}  // extern "C"
