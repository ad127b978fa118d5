// int8_few.cu -- echo_matmul_int8 for few tokens (include/echo.h): decode.
//
// The channels' codes are read once (per 32 tokens) and everything else is
// small, so the kernel streams them: a block takes 16 (or 32) channels, its
// warps take windows of 64 codes in turn, and each thread's 16-byte loads go
// straight into the operand registers of a matrix instruction.  (A sum does
// not mind the order of its terms: as long as channels and tokens are cut the
// same way, the 16 codes that a thread loads can be any of the instruction's
// k positions.)  Up to 8 tokens the instruction is the integer one, 251
// products a cycle and SM here (measured), which is what 8 tokens need at the
// full memory rate and nothing has to be turned; for more the codes become
// f16 in registers (int8_load.h) and the f16 instruction does 1023.  Its fp32
// sums are exact for 1024 codes; after those, and at the end, a warp adds its
// sums to the block's in shared memory as int32, whose order does not matter.
//
// One GB300, GPU time a call: 1 x 4096 x 4096 in 4.4 us (3.8 TB/s: its 2.5 us
// of bytes and about 2.2 of a launch), 8 x 14336 x 4096 in 9.9 us (6.0 TB/s), 16
// in 15, 32 in 23.  The last are bound by latency: 136 registers a thread leave
// eight warps an SM, whose loads and products take turns (memory, matrix pipe and
// issue slots are each busy less than a third of the time).
#include "int8_load.h"

namespace echo {
namespace {

constexpr int kWarps = 8, kWindow = 64;
constexpr int kExactWindows = 1024 / kWindow;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(int (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma_s8(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma_s8(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// 16 codes as f16, in the pairs of the f16 instruction's operands.
struct Turned {
  uint32_t h[8];
};
__device__ __forceinline__ Turned turn(const uint4& v) {
  Turned t;
  codes_to_f16(v.x, t.h[0], t.h[1]);
  codes_to_f16(v.y, t.h[2], t.h[3]);
  codes_to_f16(v.z, t.h[4], t.h[5]);
  codes_to_f16(v.w, t.h[6], t.h[7]);
  return t;
}

// OCTETS: of tokens; TALL: 16-channel groups of a block; DEEP: windows loaded
// at once.
template <int OCTETS, int TALL, int DEEP, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps)
product_few_kernel(const ProductArgs p, const int early) {
  constexpr bool kInteger = OCTETS == 1;
  constexpr int kRows = 16 * TALL, kCols = 8 * OCTETS;
  using Sum = typename std::conditional<kInteger, int, float>::type;
  __shared__ int total[kRows * kCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
  const int64_t rank = blockIdx.z, c0 = (int64_t)blockIdx.x * kRows, t0 = (int64_t)blockIdx.y * kCols;
  for (int i = threadIdx.x; i < kRows * kCols; i += 32 * kWarps) total[i] = 0;

  // Rows past the last channel or token repeat it: their results are dropped.
  const int8_t* w[2 * TALL];
#pragma unroll
  for (int i = 0; i < 2 * TALL; ++i) {
    const int64_t c = c0 + 8 * i + g;
    w[i] = p.w + rank * p.rank_w + (c < p.channels ? c : p.channels - 1) * p.ld_w;
  }
  const int8_t* a[OCTETS];
#pragma unroll
  for (int i = 0; i < OCTETS; ++i) {
    const int64_t t = t0 + 8 * i + g;
    a[i] = p.a + rank * p.rank_a + (t < p.tokens ? t : p.tokens - 1) * p.ld_a;
  }
  Sum sum[TALL][OCTETS][4];
  auto clear = [&]() {
#pragma unroll
    for (int r = 0; r < TALL; ++r)
#pragma unroll
      for (int o = 0; o < OCTETS; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[r][o][i] = 0;
  };
  auto flush = [&]() {
#pragma unroll
    for (int r = 0; r < TALL; ++r)
#pragma unroll
      for (int o = 0; o < OCTETS; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int v;
          if constexpr (kInteger) v = sum[r][o][i];
          else v = __float2int_rn(sum[r][o][i]);
          atomicAdd(&total[(8 * o + 2 * quad + (i & 1)) * kRows + 16 * r + g + 8 * (i >> 1)], v);
        }
  };
  clear();

  const int64_t windows = (p.depth + kWindow - 1) / kWindow;
  uint4 codes[DEEP][2 * TALL];
  // All loads of a turn stand in a row, without branches between them; where
  // the depth is ragged, the piece at its end is loaded again by itself (32 x
  // 14336 x 4096: 23 us, with a branch around every load 26).
  auto load = [&](auto& v, const auto& rows, int64_t first) {
    constexpr int kN = sizeof(rows) / sizeof(rows[0]);
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int64_t k = (first + d * kWarps) * kWindow + 16 * quad;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if constexpr (ALIGNED) v[d][i] = load_free16(rows[i] + k, k + 16 <= p.depth);
        else v[d][i] = k < p.depth ? load_codes<false>(rows[i], k, p.depth) : make_uint4(0, 0, 0, 0);
      }
    }
    if (ALIGNED && p.depth % 16 != 0)
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const int64_t k = (first + d * kWarps) * kWindow + 16 * quad;
        if (k >= p.depth || k + 16 <= p.depth) continue;
#pragma unroll
        for (int i = 0; i < kN; ++i) v[d][i] = load_codes<true>(rows[i], k, p.depth);
      }
  };
  // In echo_linear_int8 the launch before this one is the tokens' quantizer,
  // whose blocks let this one start only after all work before them has
  // ended: the channels' codes, which it does not write, can be read now.
  if (early) load(codes, w, warp);
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < 2 * TALL; ++i) w[i] = pinned(w[i]);
#pragma unroll
  for (int i = 0; i < OCTETS; ++i) a[i] = pinned(a[i]);
  __syncthreads();
  int exact = 0;                       // windows in sum
  for (int64_t first = warp; first < windows; first += DEEP * kWarps) {
    if (!early || first != warp) load(codes, w, first);
    uint4 tokens[DEEP][OCTETS];
    load(tokens, a, first);
    __syncwarp();                      // a row's ragged end parts the lanes; matrix instructions want them together
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      if constexpr (kInteger) {
#pragma unroll
        for (int r = 0; r < TALL; ++r) mma(sum[r][0], codes[d][2 * r], codes[d][2 * r + 1], tokens[d][0]);
      } else {
        Turned lo[TALL], hi[TALL];
#pragma unroll
        for (int r = 0; r < TALL; ++r) {
          lo[r] = turn(codes[d][2 * r]);
          hi[r] = turn(codes[d][2 * r + 1]);
        }
#pragma unroll
        for (int o = 0; o < OCTETS; ++o) {
          const Turned b = turn(tokens[d][o]);
#pragma unroll
          for (int r = 0; r < TALL; ++r)
#pragma unroll
            for (int j = 0; j < 8; j += 2)
              mma_f16(sum[r][o], lo[r].h[j], hi[r].h[j], lo[r].h[j + 1], hi[r].h[j + 1], b.h[j], b.h[j + 1]);
        }
      }
    }
    exact += DEEP;
    if (!kInteger && exact + DEEP > kExactWindows) {
      flush();
      clear();
      exact = 0;
    }
  }
  flush();
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += 32 * kWarps) {
    const int64_t c = c0 + i % kRows, t = t0 + i / kRows;
    if (c >= p.channels || t >= p.tokens) continue;
    const float v = scaled_sum(__int2float_rn(total[i]), p.a_scales[rank * p.rank_a_scales + t], p.w_scales[rank * p.rank_w_scales + c]);
    const int64_t at = rank * p.rank_out + t * p.ld_out + c;
    if (p.out_dtype == ECHO_F32) static_cast<float*>(p.out)[at] = v;
    else if (p.out_dtype == ECHO_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = from_float<__nv_bfloat16>(v);
    else static_cast<__half*>(p.out)[at] = from_float<__half>(v);
  }
}

template <int OCTETS, int TALL, int DEEP>
cudaError_t launch(const ProductArgs& p, bool aligned, bool early, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.channels + 16 * TALL - 1) / (16 * TALL)),
                     (unsigned)((p.tokens + 8 * OCTETS - 1) / (8 * OCTETS)), (unsigned)p.ranks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return aligned ? cudaLaunchKernelEx(&cfg, product_few_kernel<OCTETS, TALL, DEEP, true>, p, (int)early)
                 : cudaLaunchKernelEx(&cfg, product_few_kernel<OCTETS, TALL, DEEP, false>, p, (int)early);
}

}  // namespace

cudaError_t launch_few(const ProductArgs& p, bool aligned, bool early, int sms, cudaStream_t s) {
  // Eight windows at once leave registers for two blocks an SM: with no more
  // blocks than that, a block's time is its loads' latency (1 x 4096 x 4096:
  // 4.4 us, with four 5.5; 300 blocks, 1 x 4800 x 4096: 4.5, 5.5); with more,
  // three blocks an SM keep more loads in flight (8 x 6144 x 4096: 5.9 us, with
  // eight 6.4; 8 x 14336 x 4096: 9.9, 11.1).
  if (p.tokens <= 8)
    return (p.channels + 15) / 16 * p.ranks <= 2 * sms ? launch<1, 1, 8>(p, aligned, early, s)
                                                       : launch<1, 1, 4>(p, aligned, early, s);
  if (p.tokens <= 16) return launch<2, 1, 4>(p, aligned, early, s);
  return launch<4, 2, 2>(p, aligned, early, s);
}

}  // namespace echo
