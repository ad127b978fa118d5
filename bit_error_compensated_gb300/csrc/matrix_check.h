// matrix_check.h -- argument checks of calls on batches of matrices
// (echo_matrix of include/echo.h): sizes, strides, alignment and overlaps.
#pragma once

#include "ops_common.h"

#define ECHO_TRY(call)                  \
  do {                                  \
    const int rc_ = (call);             \
    if (rc_ != ECHO_OK) return rc_;     \
  } while (0)

namespace echo {

// Sizes whose products stay far inside 64 bits (and grids inside CUDA's limits).
constexpr int64_t kMaxExtent = (int64_t)1 << 40;
constexpr int64_t kMaxRows = ECHO_MATMUL_MAX_ROWS;

inline int check_sizes(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth) {
  if (ranks < 1 || ranks > ECHO_MAX_RANKS) return ECHO_ERR_ARG;
  if (tokens < 0 || channels < 0 || depth < 0) return ECHO_ERR_SHAPE;
  if (tokens > kMaxRows || channels > kMaxRows) return ECHO_ERR_UNSUPPORTED;
  if (depth > ECHO_MATMUL_MAX_DEPTH) return ECHO_ERR_UNSUPPORTED;
  return ECHO_OK;
}

inline int check_matrix(const echo_matrix* m, int64_t ranks, int64_t rows, int64_t cols, int size, bool output) {
  if (m == nullptr) return ECHO_ERR_ARG;
  if (rows == 0 || cols == 0) return ECHO_OK;
  if (m->data == nullptr) return ECHO_ERR_ARG;
  if (!on_boundary(m->data, size)) return ECHO_ERR_ALIGN;
  if (rows > 1 && (m->ld < cols || m->ld > kMaxExtent)) return ECHO_ERR_SHAPE;
  if (ranks > 1 && (m->rank_stride < (output ? 1 : 0) || m->rank_stride > kMaxExtent)) return ECHO_ERR_SHAPE;
  return ECHO_OK;
}

inline Region of_rank(const echo_matrix* m, int64_t rank, int64_t rows, int64_t cols, int size) {
  if (m->data == nullptr) return Region();
  return region(static_cast<char*>(m->data) + rank * m->rank_stride * size, rows, cols, m->ld, size);
}

// Each rank's part of an output overlaps no other rank's and no input.
inline bool clear_of(const echo_matrix* out, int64_t ranks, int64_t rows, int64_t cols, int size,
              const Region* in, int n) {
  for (int64_t p = 0; p < ranks; ++p) {
    const Region mine = of_rank(out, p, rows, cols, size);
    for (int64_t q = 0; q < p; ++q)
      if (overlaps(mine, of_rank(out, q, rows, cols, size))) return false;
    for (int i = 0; i < n; ++i)
      if (overlaps(mine, in[i])) return false;
  }
  return true;
}

// All ranks' parts of an input as regions; `at` is advanced.
inline void add_regions(const echo_matrix* m, int64_t ranks, int64_t rows, int64_t cols, int size, Region* in, int* n) {
  for (int64_t p = 0; p < (m->rank_stride ? ranks : 1); ++p) in[(*n)++] = of_rank(m, p, rows, cols, size);
}

}  // namespace echo
