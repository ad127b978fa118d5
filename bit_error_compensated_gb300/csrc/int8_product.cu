// int8_product.cu -- which kernel a product runs on.
#include "int8_load.h"

namespace echo {

Workspace product_workspace(const ProductArgs& p) {
  Workspace w;
  if (p.tokens <= kFewTokens || p.depth == 0 || p.channels == 0) return w;
  w.tokens = (size_t)(token_ranks(p) * wide_blocks(p.tokens) * wide_blocks(p.depth)) * kBlockBytes;
  if (!rows_aligned(p.w, p.ld_w, p.rank_w, p.channels, p.ranks))
    w.channels = (size_t)((p.rank_w == 0 ? 1 : p.ranks) * p.channels) * (size_t)((p.depth + 15) / 16 * 16);
  return w;
}

namespace {
std::atomic<int> g_hold{0};
}

void set_product_hold(int on) { g_hold.store(on, std::memory_order_relaxed); }

cudaError_t launch_product(const ProductArgs& given, bool quantized, cudaStream_t s) {
  ProductArgs p = given;
  ProductLayout l;
  l.hold = g_hold.load(std::memory_order_relaxed);
  cudaError_t e = device_sms(&l.sms);
  if (e != cudaSuccess) return e;
  const bool w_aligned = rows_aligned(p.w, p.ld_w, p.rank_w, p.channels, p.ranks);
  if (p.tokens <= kFewTokens || p.depth == 0)
    return launch_few(p, w_aligned && rows_aligned(p.a, p.ld_a, p.rank_a, p.tokens, p.ranks), quantized, l.sms, s);
  const int64_t size = elem_size(p.out_dtype);
  for (l.out_align = 32; l.out_align > 1; l.out_align = l.out_align == 32 ? 16 : l.out_align == 16 ? 4 : 1)
    if (on_boundary(p.out, l.out_align) && (p.tokens == 1 || p.ld_out * size % l.out_align == 0) &&
        (p.ranks == 1 || p.rank_out * size % l.out_align == 0))
      break;
  if (!quantized && (e = launch_widen(p, s)) != cudaSuccess) return e;
  if (!w_aligned) {
    int8_t* copy = reinterpret_cast<int8_t*>(p.wide + product_workspace(given).tokens);
    const int64_t ld = (p.depth + 15) / 16 * 16;
    if ((e = launch_realign(p, copy, ld, s)) != cudaSuccess) return e;
    p.w = copy;
    p.ld_w = ld;
    if (p.rank_w != 0) p.rank_w = p.channels * ld;
  }
  return p.out_dtype == ECHO_F32    ? launch_pair<float>(p, l, s)
         : p.out_dtype == ECHO_BF16 ? launch_pair<__nv_bfloat16>(p, l, s) : launch_pair<__half>(p, l, s);
}

}  // namespace echo
