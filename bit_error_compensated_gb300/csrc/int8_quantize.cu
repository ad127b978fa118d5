// int8_quantize.cu -- echo_quantize_tokens: one int8 scale a token
// (include/echo.h).
//
//     amax = max(2^-110, max |x|),  codes = rint(x * (127 / amax)),  scale = amax / 127
//
// One block a row.  The row is read once: its elements wait for the maximum in
// registers; a row longer than the block's registers is read again instead.
// It is bound by those bytes.
#include "int8_load.h"

namespace echo {
namespace {

constexpr int kPieces = 4;             // 16-byte pieces (or elements) a thread holds

template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
quantize_kernel(const QuantArgs a) {
  __shared__ uint32_t maxima[32];
  const int64_t token = blockIdx.x, rank = blockIdx.y;
  const T* x = static_cast<const T*>(a.x) + rank * a.rank_x + token * a.ld_x;
  int8_t* codes = a.codes + rank * a.rank_codes + token * a.ld_codes;
  const int64_t step = (int64_t)blockDim.x * VEC;
  const int64_t col0 = (int64_t)threadIdx.x * VEC;
  pdl_wait();
  pdl_trigger();

  Pack<T, VEC> held[kPieces];
  uint32_t amax = __float_as_uint(kTinyAmax);
  auto take = [&](const Pack<T, VEC>& p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) amax = max(amax, abs_bits(to_float(p.v[i])));
  };
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (col0 + j * step < a.depth) held[j] = load_pack<T, VEC>(x + col0 + j * step);
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (col0 + j * step < a.depth) take(held[j]);
  for (int64_t c = col0 + kPieces * step; c < a.depth; c += step) take(load_pack<T, VEC>(x + c));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
  if ((threadIdx.x & 31) == 0) maxima[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int i = 0; i < (int)blockDim.x / 32; ++i) amax = max(amax, maxima[i]);
  const float top = __uint_as_float(amax), inv = __fdiv_rn(127.f, top);

  auto put = [&](int64_t c, const Pack<T, VEC>& p) {
    Pack<int8_t, VEC> q;
#pragma unroll
    for (int i = 0; i < VEC; ++i) q.v[i] = (int8_t)quantize_code(to_float(p.v[i]), inv);
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + c) = *reinterpret_cast<const uint2*>(&q);
    else if constexpr (VEC == 4)
      *reinterpret_cast<uint32_t*>(codes + c) = *reinterpret_cast<const uint32_t*>(&q);
    else codes[c] = q.v[0];
    if (a.wide) {
      Pack<__half, VEC> h;
#pragma unroll
      for (int i = 0; i < VEC; ++i) h.v[i] = __int2half_rn(q.v[i]);
      uint8_t* to = a.wide + wide_offset(rank, token, c & ~(int64_t)7, a.tokens, a.depth) + 2 * (c & 7);
      if constexpr (VEC == 8) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(&h);
      else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(&h);
      else *reinterpret_cast<__half*>(to) = h.v[0];
    }
  };
#pragma unroll
  for (int j = 0; j < kPieces; ++j)
    if (col0 + j * step < a.depth) put(col0 + j * step, held[j]);
  for (int64_t c = col0 + kPieces * step; c < a.depth; c += step) put(c, load_pack<T, VEC>(x + c));
  if (a.wide)                          // zeros up to the last block's end
    for (int64_t c = a.depth + threadIdx.x; c < wide_blocks(a.depth) * kBlockCodes; c += blockDim.x)
      *reinterpret_cast<uint16_t*>(a.wide + wide_offset(rank, token, c & ~(int64_t)7, a.tokens, a.depth) + 2 * (c & 7)) = 0;
  if (threadIdx.x == 0) a.scales[rank * a.tokens + token] = __fdiv_rn(top, 127.f);
}

// Codes that are in int8 already, as f16: a thread turns 16 of a row (x, z: the
// token and its rank).
template <bool ALIGNED>
__global__ void __launch_bounds__(256)
widen_kernel(const ProductArgs p) {
  pdl_wait();
  pdl_trigger();
  const int64_t k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 16, token = blockIdx.x, rank = blockIdx.z;
  if (k >= wide_blocks(p.depth) * kBlockCodes) return;
  const uint4 v = k < p.depth ? load_codes<ALIGNED>(pinned(p.a + rank * p.rank_a + token * p.ld_a), k, p.depth)
                              : make_uint4(0, 0, 0, 0);
  uint32_t h[8];
  codes_to_f16(v.x, h[0], h[1]);
  codes_to_f16(v.y, h[2], h[3]);
  codes_to_f16(v.z, h[4], h[5]);
  codes_to_f16(v.w, h[6], h[7]);
  uint8_t* base = p.wide;
  *reinterpret_cast<uint4*>(base + wide_offset(rank, token, k, p.tokens, p.depth)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(base + wide_offset(rank, token, k + 8, p.tokens, p.depth)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// Channels' codes into rows that start on 16-byte boundaries, a thread 16 of a row.
__global__ void __launch_bounds__(256)
realign_kernel(const ProductArgs p, int8_t* to, int64_t ld) {
  pdl_wait();
  pdl_trigger();
  const int64_t k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 16, channel = blockIdx.x, rank = blockIdx.z;
  if (k >= ld) return;
  *reinterpret_cast<uint4*>(to + (rank * p.channels + channel) * ld + k) =
      load_codes<false>(pinned(p.w + rank * p.rank_w + channel * p.ld_w), k, p.depth);
}

template <typename T, int VEC>
cudaError_t launch(const QuantArgs& a, cudaStream_t s) {
  int64_t threads = (a.depth + 2 * VEC - 1) / (2 * VEC);
  threads = threads > 1024 ? 1024 : threads < 32 ? 32 : (threads + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.tokens, (unsigned)a.ranks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, quantize_kernel<T, VEC>, a);
}

template <typename T>
cudaError_t pick(const QuantArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t size = sizeof(T);
  const bool vec = on_boundary(a.x, 16) && on_boundary(a.codes, V) && a.depth % V == 0 &&
                   (a.tokens == 1 || (a.ld_x * size % 16 == 0 && a.ld_codes % V == 0)) &&
                   (a.ranks == 1 || (a.rank_x * size % 16 == 0 && a.rank_codes % V == 0));
  return vec ? launch<T, V>(a, s) : launch<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_widen(const ProductArgs& p, cudaStream_t s) {
  const int64_t pieces = wide_blocks(p.depth) * (kBlockCodes / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tokens, (unsigned)((pieces + 255) / 256), (unsigned)token_ranks(p));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return rows_aligned(p.a, p.ld_a, p.rank_a, p.tokens, p.ranks) ? cudaLaunchKernelEx(&cfg, widen_kernel<true>, p)
                                                                : cudaLaunchKernelEx(&cfg, widen_kernel<false>, p);
}

cudaError_t launch_realign(const ProductArgs& p, int8_t* to, int64_t ld, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.channels, (unsigned)((ld / 16 + 255) / 256), (unsigned)(p.rank_w == 0 ? 1 : p.ranks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, realign_kernel, p, to, ld);
}

cudaError_t launch_quantize(const QuantArgs& a, int dtype, cudaStream_t s) {
  return dtype == ECHO_F32 ? pick<float>(a, s) : dtype == ECHO_BF16 ? pick<__nv_bfloat16>(a, s) : pick<__half>(a, s);
}

}  // namespace echo
