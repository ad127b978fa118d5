// int8_api.cu -- host side of the 8-bit product and its token quantizer:
// argument checks and launches (contract in include/echo.h).
#include <cstring>

#include "int8_common.h"

namespace {
using namespace echo;

#define ECHO_TRY(call)                  \
  do {                                  \
    const int rc_ = (call);             \
    if (rc_ != ECHO_OK) return rc_;     \
  } while (0)

// Sizes whose products stay far inside 64 bits (and grids inside CUDA's limits).
constexpr int64_t kMaxExtent = (int64_t)1 << 40;
constexpr int64_t kMaxRows = ECHO_MATMUL_MAX_ROWS;

int check_sizes(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth) {
  if (ranks < 1 || ranks > ECHO_MAX_RANKS) return ECHO_ERR_ARG;
  if (tokens < 0 || channels < 0 || depth < 0) return ECHO_ERR_SHAPE;
  if (tokens > kMaxRows || channels > kMaxRows) return ECHO_ERR_UNSUPPORTED;
  if (depth > ECHO_MATMUL_MAX_DEPTH) return ECHO_ERR_UNSUPPORTED;
  return ECHO_OK;
}

int check_matrix(const echo_matrix* m, int64_t ranks, int64_t rows, int64_t cols, int size, bool output) {
  if (m == nullptr) return ECHO_ERR_ARG;
  if (rows == 0 || cols == 0) return ECHO_OK;
  if (m->data == nullptr) return ECHO_ERR_ARG;
  if (!on_boundary(m->data, size)) return ECHO_ERR_ALIGN;
  if (rows > 1 && (m->ld < cols || m->ld > kMaxExtent)) return ECHO_ERR_SHAPE;
  if (ranks > 1 && (m->rank_stride < (output ? 1 : 0) || m->rank_stride > kMaxExtent)) return ECHO_ERR_SHAPE;
  return ECHO_OK;
}

Region of_rank(const echo_matrix* m, int64_t rank, int64_t rows, int64_t cols, int size) {
  if (m->data == nullptr) return Region();
  return region(static_cast<char*>(m->data) + rank * m->rank_stride * size, rows, cols, m->ld, size);
}

// Each rank's part of an output overlaps no other rank's and no input.
bool clear_of(const echo_matrix* out, int64_t ranks, int64_t rows, int64_t cols, int size,
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
void add_regions(const echo_matrix* m, int64_t ranks, int64_t rows, int64_t cols, int size, Region* in, int* n) {
  for (int64_t p = 0; p < (m->rank_stride ? ranks : 1); ++p) in[(*n)++] = of_rank(m, p, rows, cols, size);
}

int check_quantize(int64_t ranks, int64_t tokens, int64_t depth, int dtype, const echo_matrix* x,
                   const echo_matrix* codes, const float* scales) {
  if (!known_dtype(dtype)) return ECHO_ERR_UNSUPPORTED;
  const int size = elem_size(dtype);
  ECHO_TRY(check_matrix(x, ranks, tokens, depth, size, false));
  ECHO_TRY(check_matrix(codes, ranks, tokens, depth, 1, true));
  if (tokens == 0) return ECHO_OK;
  if (scales == nullptr) return ECHO_ERR_ARG;
  if (!on_boundary(scales, 4)) return ECHO_ERR_ALIGN;
  Region in[ECHO_MAX_RANKS + 1];
  int n = 0;
  add_regions(x, ranks, tokens, depth, size, in, &n);
  const Region sc = region(scales, 1, ranks * tokens, ranks * tokens, 4);
  for (int i = 0; i < n; ++i)
    if (overlaps(sc, in[i])) return ECHO_ERR_ARG;
  in[n++] = sc;
  return clear_of(codes, ranks, tokens, depth, 1, in, n) ? ECHO_OK : ECHO_ERR_ARG;
}

// `a` and a_scales as the product reads them.
int check_product(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth, const echo_matrix* a,
                  const float* a_scales, int64_t a_scale_stride, const echo_matrix* w,
                  const float* w_scales, int64_t w_scale_stride, int out_dtype, const echo_matrix* out) {
  if (!known_dtype(out_dtype)) return ECHO_ERR_UNSUPPORTED;
  const int size = elem_size(out_dtype);
  ECHO_TRY(check_matrix(a, ranks, tokens, depth, 1, false));
  ECHO_TRY(check_matrix(w, ranks, channels, depth, 1, false));
  ECHO_TRY(check_matrix(out, ranks, tokens, channels, size, true));
  if (tokens == 0 || channels == 0) return ECHO_OK;
  if (a_scales == nullptr || w_scales == nullptr) return ECHO_ERR_ARG;
  if (!on_boundary(a_scales, 4) || !on_boundary(w_scales, 4)) return ECHO_ERR_ALIGN;
  if (ranks > 1 && w_scale_stride != 0 && (w_scale_stride < channels || w_scale_stride > kMaxExtent))
    return ECHO_ERR_SHAPE;
  if (ranks > 1 && a_scale_stride != 0 && (a_scale_stride < tokens || a_scale_stride > kMaxExtent))
    return ECHO_ERR_SHAPE;
  Region in[4 * ECHO_MAX_RANKS];
  int n = 0;
  add_regions(a, ranks, tokens, depth, 1, in, &n);
  add_regions(w, ranks, channels, depth, 1, in, &n);
  const echo_matrix at = {const_cast<float*>(a_scales), tokens, a_scale_stride};
  const echo_matrix wt = {const_cast<float*>(w_scales), channels, w_scale_stride};
  add_regions(&at, ranks, 1, tokens, 4, in, &n);
  add_regions(&wt, ranks, 1, channels, 4, in, &n);
  return clear_of(out, ranks, tokens, channels, size, in, n) ? ECHO_OK : ECHO_ERR_ARG;
}

int check_workspace(const ProductArgs& p, size_t bytes) {
  const size_t need = product_workspace(p).bytes();
  if (need == 0) return ECHO_OK;
  if (p.wide == nullptr || bytes < need) return ECHO_ERR_TOO_LARGE;
  return on_boundary(p.wide, 16) ? ECHO_OK : ECHO_ERR_ALIGN;
}

QuantArgs quant_args(int64_t ranks, int64_t tokens, int64_t depth, const echo_matrix* x,
                     const echo_matrix* codes, float* scales, void* wide) {
  QuantArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x->data; a.ld_x = x->ld; a.rank_x = x->rank_stride;
  a.codes = static_cast<int8_t*>(codes->data);
  a.ld_codes = codes->ld; a.rank_codes = codes->rank_stride;
  a.scales = scales;
  a.wide = static_cast<uint8_t*>(wide);
  a.ranks = ranks; a.tokens = tokens; a.depth = depth;
  return a;
}

ProductArgs product_args(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth,
                         const echo_matrix* a, const float* a_scales, int64_t a_scale_stride,
                         const echo_matrix* w, const float* w_scales, int64_t w_scale_stride,
                         int out_dtype, const echo_matrix* out, void* wide) {
  ProductArgs p;
  std::memset(&p, 0, sizeof(p));
  p.a = static_cast<const int8_t*>(a->data); p.ld_a = a->ld; p.rank_a = a->rank_stride;
  p.a_scales = a_scales; p.rank_a_scales = a_scale_stride;
  p.w = static_cast<const int8_t*>(w->data); p.ld_w = w->ld; p.rank_w = w->rank_stride;
  p.w_scales = w_scales; p.rank_w_scales = w_scale_stride;
  p.out = out->data; p.ld_out = out->ld; p.rank_out = out->rank_stride;
  p.ranks = ranks; p.tokens = tokens; p.channels = channels; p.depth = depth;
  p.out_dtype = out_dtype;
  p.wide = static_cast<uint8_t*>(wide);
  return p;
}

}  // namespace

extern "C" {

int echo_quantize_tokens(int64_t ranks, int64_t tokens, int64_t depth, int dtype,
                         const echo_matrix* x, const echo_matrix* codes, float* scales,
                         void* stream) {
  ECHO_TRY(check_sizes(ranks, tokens, 0, depth));
  ECHO_TRY(check_quantize(ranks, tokens, depth, dtype, x, codes, scales));
  if (tokens == 0) return ECHO_OK;
  ECHO_OPS_CUDA(launch_quantize(quant_args(ranks, tokens, depth, x, codes, scales, nullptr), dtype,
                                static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

int echo_matmul_int8(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth,
                     const echo_matrix* a, const float* a_scales, int64_t a_scale_stride,
                     const echo_matrix* w, const float* w_scales, int64_t w_scale_stride,
                     int out_dtype, const echo_matrix* out, void* workspace, size_t workspace_bytes,
                     void* stream) {
  ECHO_TRY(check_sizes(ranks, tokens, channels, depth));
  ECHO_TRY(check_product(ranks, tokens, channels, depth, a, a_scales, a_scale_stride, w, w_scales,
                         w_scale_stride, out_dtype, out));
  if (tokens == 0 || channels == 0) return ECHO_OK;
  const ProductArgs p = product_args(ranks, tokens, channels, depth, a, a_scales, a_scale_stride, w, w_scales,
                                     w_scale_stride, out_dtype, out, workspace);
  ECHO_TRY(check_workspace(p, workspace_bytes));
  ECHO_OPS_CUDA(launch_product(p, false, static_cast<cudaStream_t>(stream)));
  return ECHO_OK;
}

size_t echo_matmul_workspace_bytes(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth,
                                   const echo_matrix* a, const echo_matrix* w) {
  if (check_sizes(ranks, tokens, channels, depth) != ECHO_OK || a == nullptr || w == nullptr) return 0;
  const echo_matrix none = {nullptr, 0, 0};
  return product_workspace(product_args(ranks, tokens, channels, depth, a, nullptr, 0, w, nullptr, 0, ECHO_F32,
                                        &none, nullptr)).bytes();
}

int echo_matmul_status(void* stream, int* status) {
  if (status == nullptr) return ECHO_ERR_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int word[3] = {0, 0, 0};
  ECHO_OPS_CUDA(read_gave_up<float>(word, s));
  ECHO_OPS_CUDA(read_gave_up<__nv_bfloat16>(word + 1, s));
  ECHO_OPS_CUDA(read_gave_up<__half>(word + 2, s));
  ECHO_OPS_CUDA(cudaStreamSynchronize(s));
  // Only a word that was set is cleared: one that a product on another stream
  // sets right now is the next call's to report.
  if (word[0]) ECHO_OPS_CUDA(clear_gave_up<float>(s));
  if (word[1]) ECHO_OPS_CUDA(clear_gave_up<__nv_bfloat16>(s));
  if (word[2]) ECHO_OPS_CUDA(clear_gave_up<__half>(s));
  if (word[0] | word[1] | word[2]) ECHO_OPS_CUDA(cudaStreamSynchronize(s));
  *status = word[0] | word[1] | word[2] ? ECHO_ERR_TIMEOUT : ECHO_OK;
  return ECHO_OK;
}

int echo_debug_hold_product(int on) {
  if (on != 0 && on != 1) return ECHO_ERR_ARG;
  set_product_hold(on);
  return ECHO_OK;
}

int echo_linear_int8(int64_t ranks, int64_t tokens, int64_t channels, int64_t depth, int dtype,
                     const echo_matrix* x, const echo_matrix* w, const float* w_scales,
                     int64_t w_scale_stride, const echo_matrix* codes, float* a_scales,
                     const echo_matrix* out, void* workspace, size_t workspace_bytes, void* stream) {
  ECHO_TRY(check_sizes(ranks, tokens, channels, depth));
  ECHO_TRY(check_quantize(ranks, tokens, depth, dtype, x, codes, a_scales));
  ECHO_TRY(check_product(ranks, tokens, channels, depth, codes, a_scales, tokens, w, w_scales,
                         w_scale_stride, dtype, out));
  if (tokens == 0) return ECHO_OK;
  {
    // The quantizer must not write what the product takes as given.
    Region given[2 * ECHO_MAX_RANKS];
    int n = 0;
    const echo_matrix wt = {const_cast<float*>(w_scales), channels, w_scale_stride};
    add_regions(w, ranks, channels, depth, 1, given, &n);
    add_regions(&wt, ranks, 1, channels, 4, given, &n);
    const Region scales = region(a_scales, 1, ranks * tokens, ranks * tokens, 4);
    if (!clear_of(codes, ranks, tokens, depth, 1, given, n)) return ECHO_ERR_ARG;
    for (int i = 0; i < n; ++i)
      if (overlaps(scales, given[i])) return ECHO_ERR_ARG;
  }
  const ProductArgs p = product_args(ranks, tokens, channels, depth, codes, a_scales, tokens, w, w_scales,
                                     w_scale_stride, dtype, out, workspace);
  ECHO_TRY(check_workspace(p, workspace_bytes));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool many = product_workspace(p).tokens > 0;
  ECHO_OPS_CUDA(launch_quantize(quant_args(ranks, tokens, depth, x, codes, a_scales, many ? workspace : nullptr),
                                dtype, s));
  if (channels > 0) ECHO_OPS_CUDA(launch_product(p, true, s));
  return ECHO_OK;
}

}  // extern "C"
