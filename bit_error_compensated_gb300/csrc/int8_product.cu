// int8_product.cu -- echo_matmul_int8 (include/echo.h): a plain tile kernel.
// A block computes 64 tokens x 64 channels; 64 codes of each row at a time
// pass through shared memory and every thread sums 4 x 4 results with dp4a.
#include "int8_load.h"

namespace echo {
namespace {

constexpr int kTile = 64, kDepth = 64, kPitch = kDepth / 4 + 1;

template <typename T>
__global__ void __launch_bounds__(256)
product_tile_kernel(const ProductArgs p) {
  __shared__ int sa[kTile][kPitch], sw[kTile][kPitch];
  const int64_t t0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
  const int64_t rank = blockIdx.z;
  const int8_t* a = p.a + rank * p.rank_a;
  const int8_t* w = p.w + rank * p.rank_w;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int sum[4][4] = {};
  pdl_wait();
  for (int64_t k0 = 0; k0 < p.depth; k0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
      const int row = i / kDepth, k = i % kDepth;
      const bool deep = k0 + k < p.depth;
      reinterpret_cast<int8_t*>(sa[row])[k] =
          deep && t0 + row < p.tokens ? a[(t0 + row) * p.ld_a + k0 + k] : (int8_t)0;
      reinterpret_cast<int8_t*>(sw[row])[k] =
          deep && c0 + row < p.channels ? w[(c0 + row) * p.ld_w + k0 + k] : (int8_t)0;
    }
    __syncthreads();
    for (int k = 0; k < kDepth / 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = __dp4a(sa[ty + 16 * i][k], sw[tx + 16 * j][k], sum[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty + 16 * i;
    if (t >= p.tokens) continue;
    const float token = p.a_scales[rank * p.rank_a_scales + t];
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + tx + 16 * j;
      if (c < p.channels)
        static_cast<T*>(p.out)[rank * p.rank_out + t * p.ld_out + c] =
            from_float<T>(scaled_sum(sum[i][j], token, p.w_scales[rank * p.rank_w_scales + c]));
    }
  }
}

template <typename T>
cudaError_t launch(const ProductArgs& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.channels + kTile - 1) / kTile),
                     (unsigned)((p.tokens + kTile - 1) / kTile), (unsigned)p.ranks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, product_tile_kernel<T>, p);
}

}  // namespace

size_t product_workspace(int64_t ranks, int64_t tokens, int64_t depth) {
  if (tokens <= kFewTokens || depth == 0) return 0;
  return (size_t)(ranks * wide_blocks(tokens) * wide_blocks(depth)) * kBlockBytes;
}

cudaError_t launch_product(const ProductArgs& p, bool widened, cudaStream_t s) {
  ProductLayout l;
  cudaError_t e = device_sms(&l.sms);
  if (e != cudaSuccess) return e;
  const int64_t size = elem_size(p.out_dtype);
  l.aligned = on_boundary(p.a, 16) && on_boundary(p.w, 16) && (p.tokens == 1 || p.ld_a % 16 == 0) &&
              (p.channels == 1 || p.ld_w % 16 == 0) &&
              (p.ranks == 1 || (p.rank_a % 16 == 0 && p.rank_w % 16 == 0));
  l.wide = on_boundary(p.out, 16) && (p.tokens == 1 || p.ld_out * size % 16 == 0) &&
           (p.ranks == 1 || p.rank_out * size % 16 == 0);
  if (p.tokens > kFewTokens && p.depth > 0) {
    if (!widened && (e = launch_widen(p, l.aligned, s)) != cudaSuccess) return e;
    return p.out_dtype == ECHO_F32    ? launch_pair<float>(p, l, s)
           : p.out_dtype == ECHO_BF16 ? launch_pair<__nv_bfloat16>(p, l, s) : launch_pair<__half>(p, l, s);
  }
  return p.out_dtype == ECHO_F32    ? launch<float>(p, s)
         : p.out_dtype == ECHO_BF16 ? launch<__nv_bfloat16>(p, s) : launch<__half>(p, s);
}

}  // namespace echo
