// int8_common.h -- launch arguments of the 8-bit product and its token
// quantizer (int8_*.cu).  The operators are described in include/echo.h.
#pragma once

#include "ops_common.h"

namespace echo {

struct QuantArgs {
  const void* x;
  int64_t ld_x, rank_x;
  int8_t* codes;
  int64_t ld_codes, rank_codes;
  float* scales;                 // [ranks][tokens]
  uint8_t* wide;                 // the codes as f16 too (int8_load.h), or nullptr
  int64_t ranks, tokens, depth;
};

struct ProductArgs {
  const int8_t* a;               // [ranks][tokens][depth]
  int64_t ld_a, rank_a;
  const float* a_scales;
  int64_t rank_a_scales;
  const int8_t* w;               // [ranks][channels][depth]
  int64_t ld_w, rank_w;
  const float* w_scales;
  int64_t rank_w_scales;
  void* out;                     // [ranks][tokens][channels]
  int64_t ld_out, rank_out;
  int64_t ranks, tokens, channels, depth;
  int out_dtype;
  uint8_t* wide;                 // workspace: the tokens' codes as f16 (int8_load.h), many tokens only
};

// Products of more tokens than this run in tiles (int8_pair.cu), from f16
// codes in a workspace, which those of fewer (int8_few.cu) do not need.  Both
// product_workspace and launch_product go by it.  Depth 4096, 4096 and 14336
// channels: tiles take 21 and 26 us for 33 to 96 tokens, these kernels 8 and 23
// for 32, 14 and 43 for 48, 22 and 67 for 96.
constexpr int64_t kFewTokens = 32;
// Ranks of the tokens' codes: one where all share them.
inline int64_t token_ranks(const ProductArgs& p) { return p.rank_a == 0 ? 1 : p.ranks; }
// Whether a matrix' rows of codes all start on 16-byte boundaries.
inline bool rows_aligned(const void* data, int64_t ld, int64_t rank_stride, int64_t rows, int64_t ranks) {
  return on_boundary(data, 16) && (rows == 1 || ld % 16 == 0) && (ranks == 1 || rank_stride % 16 == 0);
}
// The workspace of a product of many tokens: their f16 codes, then a copy of
// the channels' codes if their rows are not aligned (TMA takes no others).
struct Workspace {
  size_t tokens = 0, channels = 0;
  size_t bytes() const { return tokens + channels; }
};
Workspace product_workspace(const ProductArgs& p);

// The value of an exact sum: fp32 products by the token's, then the channel's
// scale, in this order everywhere, so that every kernel gives the same bits.
__device__ __forceinline__ float scaled_sum(float sum, float token, float channel) {
  return __fmul_rn(__fmul_rn(sum, token), channel);
}

struct ProductLayout {
  int out_align;                 // rows of out start on multiples of 32, 16, 4 or (1) fewer bytes
  int sms;
  int hold;                      // echo_debug_hold_product
};

cudaError_t launch_quantize(const QuantArgs& a, int dtype, cudaStream_t s);
// The f16 codes of tokens that are in int8 already.
cudaError_t launch_widen(const ProductArgs& p, cudaStream_t s);
// Copies the channels' codes to rows of `ld` bytes, aligned, rank after rank.
cudaError_t launch_realign(const ProductArgs& p, int8_t* to, int64_t ld, cudaStream_t s);
// `quantized`: this call's quantizer ran just before, and has left the tokens'
// f16 codes in the workspace where the product needs them.
cudaError_t launch_product(const ProductArgs& a, bool quantized, cudaStream_t s);
// Test hook: whether later products of many tokens hold a report back.
void set_product_hold(int on);
// `early`: the kernel before is this call's quantizer, see int8_few.cu.
cudaError_t launch_few(const ProductArgs& p, bool aligned, bool early, int sms, cudaStream_t s);
// One instantiation per type of out (the sources are compiled once for each).
template <typename T>
cudaError_t launch_pair(const ProductArgs& p, const ProductLayout& l, cudaStream_t s);
// Reads, and clears, the word that a wait that gave up has set.
template <typename T> cudaError_t read_gave_up(int* word, cudaStream_t s);
template <typename T> cudaError_t clear_gave_up(cudaStream_t s);

}  // namespace echo

#if ECHO_T == 0
#define ECHO_ELEM float
#elif ECHO_T == 1
#define ECHO_ELEM __nv_bfloat16
#elif ECHO_T == 2
#define ECHO_ELEM __half
#endif
