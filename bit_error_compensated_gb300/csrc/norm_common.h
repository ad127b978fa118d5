// norm_common.h -- launch arguments of the residual join (norm_fwd.cu,
// norm_bwd.cu) and its block-wide sums.  The operator is described in
// include/echo.h (echo_norm_plan).
#pragma once

#include "ops_common.h"

namespace echo {

struct NormArgs {
  int64_t rows;
  int width;
  const void *x, *y, *gate;
  int64_t ld_x, ld_y;
  int64_t gate_span;             // rows that share a gate row
  const void *w_post, *b_post, *w_pre, *b_pre;
  void *r, *h;
  int64_t ld_r, ld_h;
  int8_t* codes;
  int64_t ld_codes;
  float *scales, *stats;
  float eps, scale;
  int gate_scalar;               // one gate value a row instead of `width`
  int post;                      // the norm after the block is there (and y is)
  int params_f32;                // parameters and gate are fp32 (else the rows' type)
};

struct NormGradArgs {
  int64_t rows;
  int width;
  const void *x, *y, *gate;
  int64_t ld_x, ld_y;
  int64_t gate_span;
  const void *w_post, *b_post, *w_pre;
  const float* stats;
  const void *dr, *dh;
  int64_t ld_dr, ld_dh;
  void *dx, *dy, *dgate;
  int64_t ld_dx, ld_dy;
  void* dparam[4];               // w_post, b_post, w_pre, b_pre
  float* partial[4];             // [workers][width] sums of each, or nullptr
  float* gate_partial;           // [workers][2][width or 1], see norm_bwd.cu
  int64_t span;                  // rows a worker takes
  int64_t workers;
  float scale;
  int gate_scalar, post, params_f32;
  int folded;                    // partial[0], [1] are without scale and gate (norm_bwd.cu)
};

// N floats of a parameter vector (or gate row) of either type, from element `col`.
template <typename T, int N>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t col, float (&out)[N]) {
  if (sizeof(T) == 4 || f32) {
    const Pack<float, N> v = load_pack<float, N>(static_cast<const float*>(p) + col);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = v.v[i];
  } else {
    to_floats<T, N>(load_pack<T, N>(static_cast<const T*>(p) + col), out);
  }
}
// The same, `missing` where there is no vector.
template <typename T, int N>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t col, float missing,
                                           float (&out)[N]) {
  if (p != nullptr) return load_param<T, N>(p, f32, col, out);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = missing;
}

// Launchers, one instantiation per element type (norm_fwd.cu and norm_bwd.cu
// are compiled once for each).  `vec`: 16-byte accesses are possible.
template <typename T>
cudaError_t launch_norm(const NormArgs& a, int layer, bool vec, int sms, cudaStream_t s);
template <typename T>
cudaError_t launch_norm_grad(NormGradArgs a, int layer, bool vec, int sms, cudaStream_t s);
// Threads that the backward kernel gives a row of `cols` columns of a block, at
// `each` elements a thread.
inline int norm_grad_threads(int cols, int each) { return ((cols + each - 1) / each + 31) / 32 * 32; }
// Threads of a block, at most, and of an SM: at 128 registers a thread.  (64 and
// twice the threads spill: 143 us with 8 elements a thread, where this takes 92,
// 8192 x 4096 bf16.)
constexpr int kNormGradThreads = 512;
// How the backward kernel lays rows on blocks, at `each` elements a thread: a
// row's columns over `blocks`, or `rows` narrow rows on one.
struct NormGradShape {
  int blocks, block_cols, threads, rows;
  NormGradShape(int width, int each) {
    blocks = (width + each * kNormGradThreads - 1) / (each * kNormGradThreads);
    block_cols = ((width + blocks - 1) / blocks + 7) / 8 * 8;
    threads = norm_grad_threads(block_cols, each);
    rows = threads < 128 ? 128 / threads : 1;
  }
  // Workers (row ranges with their own partial sums) of a call, where an SM
  // holds the blocks that registers let it and at most `room`.
  int64_t workers(int sms, int room) const {
    int at_once = kNormGradThreads / (threads * rows);
    at_once = at_once > room ? room : at_once;
    const int64_t most = (int64_t)((at_once < 1 ? 1 : at_once) * sms / blocks) * rows;
    return most < 1 ? 1 : most;
  }
};
// Workers a backward call may have at most, whichever form it takes.
inline int64_t norm_grad_max_workers(int width, int sms) {
  const int64_t a = NormGradShape(width, 8).workers(sms, kNormGradThreads);
  const int64_t b = NormGradShape(width, 16).workers(sms, kNormGradThreads);
  return a > b ? a : b;
}

}  // namespace echo

#if ECHO_T == 0
#define ECHO_ELEM float
#elif ECHO_T == 1
#define ECHO_ELEM __nv_bfloat16
#elif ECHO_T == 2
#define ECHO_ELEM __half
#endif
