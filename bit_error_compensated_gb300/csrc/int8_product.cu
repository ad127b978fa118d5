// int8_product.cu -- which kernel a product runs on.
#include "int8_load.h"

namespace echo {

size_t product_workspace(int64_t ranks, int64_t tokens, int64_t depth) {
  if (tokens <= kFewTokens || depth == 0) return 0;
  return (size_t)(ranks * wide_blocks(tokens) * wide_blocks(depth)) * kBlockBytes;
}

cudaError_t launch_product(const ProductArgs& p, bool quantized, cudaStream_t s) {
  ProductLayout l;
  cudaError_t e = device_sms(&l.sms);
  if (e != cudaSuccess) return e;
  const int64_t size = elem_size(p.out_dtype);
  l.aligned = on_boundary(p.a, 16) && on_boundary(p.w, 16) && (p.tokens == 1 || p.ld_a % 16 == 0) &&
              (p.channels == 1 || p.ld_w % 16 == 0) &&
              (p.ranks == 1 || (p.rank_a % 16 == 0 && p.rank_w % 16 == 0));
  l.wide = on_boundary(p.out, 16) && (p.tokens == 1 || p.ld_out * size % 16 == 0) &&
           (p.ranks == 1 || p.rank_out * size % 16 == 0);
  if (p.tokens <= kFewTokens || p.depth == 0) return launch_few(p, l.aligned, quantized, s);
  if (!quantized && (e = launch_widen(p, l.aligned, s)) != cudaSuccess) return e;
  return p.out_dtype == ECHO_F32    ? launch_pair<float>(p, l, s)
         : p.out_dtype == ECHO_BF16 ? launch_pair<__nv_bfloat16>(p, l, s) : launch_pair<__half>(p, l, s);
}

}  // namespace echo
