// int4_few.cu -- echo_linear_int4 (include/echo.h): few tokens with 4-bit
// weights.
//
// The weights are read once for 32 tokens and streamed: a warp takes 16
// channels, and a thread's loads are the operands of matrix instructions: as
// long as weights and tokens are cut the same way, the codes that a thread has
// of a row can be any of the instruction's places.  A code behind the bits of
// 128 (bf16) or 1024 (f16) is that number plus the code; taking off that number
// plus the zero point leaves code - z, exact.  Products are exact, a window's
// sums (of one group) are multiplied by the group's step in fp32 and added up.
// fp32 tokens are three bf16 numbers each, which hold all their bits.
//
// The tokens of a window go through shared memory, turned into the order of the
// operands once for the block's eight warps: 32 tokens are eight times the bytes
// of a warp's codes, and read by every warp for itself they cost more than the
// weights (32 x 14336 x 4096: 51 us).  A cluster's blocks share the depth where
// channels are few, and add up their sums through each other's shared memory, in
// the order of the blocks.
//
// One GB300, GPU time a call: 1 x 4096 x 4096 in 5.7 us (2.2 of them a launch),
// 1, 8, 16, 32 x 14336 x 4096 in 11.5, 12.4, 21 and 31 us (2.7 to 1.0 TB/s): a
// block's loads, products and sums take turns, and the tokens' elements are as
// many bytes as the codes.
#include "serve_common.h"

namespace echo {
namespace {

constexpr int kWarps = 8;

template <typename T> struct Codes {                     // f16 tokens
  static constexpr uint32_t kBase = 0x64006400u;
  static __device__ __forceinline__ uint32_t base_and(float z) {         // 1024 + z, twice
    const __half2 h = __float2half2_rn(1024.0f + z);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t* lo, const uint32_t* hi, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(lo[0]), "r"(hi[0]), "r"(lo[1]), "r"(hi[1]), "r"(b0), "r"(b1));
  }
};
struct CodesBf16 {
  static constexpr uint32_t kBase = 0x43004300u;
  static __device__ __forceinline__ uint32_t base_and(float z) {
    const __nv_bfloat162 h = __float2bfloat162_rn(128.0f + z);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t* lo, const uint32_t* hi, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(lo[0]), "r"(hi[0]), "r"(lo[1]), "r"(hi[1]), "r"(b0), "r"(b1));
  }
};
template <> struct Codes<__nv_bfloat16> : CodesBf16 {};
template <> struct Codes<float> : CodesBf16 {};

// Eight codes of a word, less the zero point, as pairs of elements (0, 4),
// (1, 5), (2, 6), (3, 7).
template <typename T>
__device__ __forceinline__ void turn(uint32_t w, uint32_t base, uint32_t zero, uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = Codes<T>::less(masked<0x000F000Fu>(w >> (4 * i), base), zero);
}

// WORDS words of a row of `bytes` bytes from byte `at` (a multiple of 4 WORDS),
// zeros behind its end.  ALIGNED: rows start on multiples of 4 WORDS bytes.
template <int WORDS, bool ALIGNED>
__device__ __forceinline__ void load_codes(const uint8_t* row, int64_t at, int64_t bytes, uint32_t (&w)[WORDS]) {
  const uint8_t* p = row + at;
  if (ALIGNED && at + 4 * WORDS <= bytes) {
    if constexpr (WORDS == 4) {
      const uint4 v = load_free16(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      asm("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
    return;
  }
  if (!ALIGNED && at >= 3 && at + 4 * WORDS + 3 <= bytes) {
    // put together from the aligned words around it, all of them inside the row too
    const uint32_t shift = (uint32_t)((uintptr_t)p & 3) * 8;
    const uint32_t* from = reinterpret_cast<const uint32_t*>((uintptr_t)p & ~(uintptr_t)3);
    uint32_t v[WORDS + 1];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) v[i] = load_free4(from + i);
    v[WORDS] = shift ? load_free4(from + WORDS) : 0;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], shift);
    return;
  }
#pragma unroll
  for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
  for (int i = 0; i < 4 * WORDS; ++i)
    if (at + i < bytes) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
}

// Eight elements of a token's row from k, zeros behind its end, in the order of
// turn's pairs: PARTS operands of four registers, whose sum they are.
template <typename T> constexpr int parts() { return sizeof(T) == 4 ? 3 : 1; }
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_tokens(const T* row, int64_t k, int64_t depth, uint32_t (&h)[parts<T>()][4]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (ALIGNED && k + 8 <= depth) {
      const uint4 v = load_free16(row + k);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < depth) w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[k + i] << (16 * (i % 2));
    }
    h[0][0] = __byte_perm(w[0], w[2], 0x5410);
    h[0][1] = __byte_perm(w[0], w[2], 0x7632);
    h[0][2] = __byte_perm(w[1], w[3], 0x5410);
    h[0][3] = __byte_perm(w[1], w[3], 0x7632);
  } else {
    float v[8];
    if (ALIGNED && k + 8 <= depth) {
      const uint4 a = load_free16(row + k), b = load_free16(row + k + 4);
      v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < depth ? row[k + i] : 0.0f;
    }
    // The upper 8 bits of the significand, the next, and the rest; an infinity is
    // its own first part, and so is a NaN once the sum has made it CUDA's (one with
    // its bits set in the lower half only would leave an infinity).
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], 0.0f);
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __float_as_uint(v[i]), hi = __float_as_uint(v[i + 4]);
        h[part][i] = __byte_perm(lo, hi, 0x7632);
        if (part < 2) {
          const float rest = v[i] - __uint_as_float(lo & 0xFFFF0000u), rest4 = v[i + 4] - __uint_as_float(hi & 0xFFFF0000u);
          v[i] = isfinite(v[i]) ? rest : 0.0f;
          v[i + 4] = isfinite(v[i + 4]) ? rest4 : 0.0f;
        }
      }
  }
}

// Few tokens: each warp loads what it needs of them by itself.
// OCTETS: of tokens; TALL: 16-channel parts of a block; WORDS: of a row's
// window, a thread's (a window is 32 WORDS codes of one group).
template <typename T, int OCTETS, int TALL, int WORDS, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps, OCTETS * TALL == 1 ? 4 : OCTETS * TALL == 2 ? 3 : 2) linear4_kernel(const Linear4Args p) {
  constexpr int kRows = 16 * TALL, kCols = 8 * OCTETS, kWindow = 32 * WORDS, kParts = parts<T>();
  __shared__ float total[kWarps][kCols][kRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
  const int64_t rank = blockIdx.z, c0 = (int64_t)blockIdx.x * kRows, t0 = (int64_t)blockIdx.y * kCols;
  const int64_t bytes = (p.depth + 1) / 2;
  const uint32_t base = unknown(Codes<T>::kBase);
  pdl_wait();
  pdl_trigger();
  // Rows past the last channel or token repeat it: their results are dropped.
  const uint8_t* codes[2 * TALL];
  const uint32_t* meta[2 * TALL];
#pragma unroll
  for (int i = 0; i < 2 * TALL; ++i) {
    const int64_t c = c0 + 8 * i + g < p.channels ? c0 + 8 * i + g : p.channels - 1;
    codes[i] = pinned(p.codes + rank * p.rank_codes + c * p.ld_codes);
    meta[i] = pinned(p.meta + rank * p.rank_meta + c * p.ld_meta);
  }
  const T* x[OCTETS];
#pragma unroll
  for (int i = 0; i < OCTETS; ++i) {
    const int64_t t = t0 + 8 * i + g < p.tokens ? t0 + 8 * i + g : p.tokens - 1;
    x[i] = pinned(static_cast<const T*>(p.x) + rank * p.rank_x + t * p.ld_x);
  }
  float sum[TALL][OCTETS][4];
#pragma unroll
  for (int r = 0; r < TALL; ++r)
#pragma unroll
    for (int o = 0; o < OCTETS; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[r][o][i] = 0.0f;

  const int64_t windows = (p.depth + kWindow - 1) / kWindow;
#pragma unroll 1
  for (int64_t window = warp; window < windows; window += kWarps) {
    uint32_t w[2 * TALL][WORDS], word[2 * TALL];
#pragma unroll
    for (int i = 0; i < 2 * TALL; ++i) {
      load_codes<WORDS, ALIGNED>(codes[i], window * (kWindow / 2) + 4 * WORDS * quad, bytes, w[i]);
      word[i] = load_free4(meta[i] + window * kWindow / p.group);
    }
    // The tokens' loads follow the codes', before any of them is used (16-bit
    // ones: three parts of fp32 ones would not fit registers).
    constexpr bool kEarly = sizeof(T) == 2;
    const int64_t k = window * kWindow + 8 * WORDS * quad;
    uint32_t early[kEarly ? WORDS : 1][OCTETS][kParts][4];
    if constexpr (kEarly)
#pragma unroll
      for (int n = 0; n < WORDS; ++n)
#pragma unroll
        for (int o = 0; o < OCTETS; ++o) load_tokens<T, ALIGNED>(x[o], k + 8 * n, p.depth, early[n][o]);
    float part[TALL][OCTETS][4] = {};
    uint32_t zero[2 * TALL];
#pragma unroll
    for (int i = 0; i < 2 * TALL; ++i) zero[i] = Codes<T>::base_and(meta_zero(word[i]));
#pragma unroll
    for (int n = 0; n < WORDS; ++n) {
      uint32_t lo[TALL][4], hi[TALL][4];
#pragma unroll
      for (int r = 0; r < TALL; ++r) {
        turn<T>(w[2 * r][n], base, zero[2 * r], lo[r]);
        turn<T>(w[2 * r + 1][n], base, zero[2 * r + 1], hi[r]);
      }
#pragma unroll
      for (int o = 0; o < OCTETS; ++o) {
        uint32_t b[kParts][4];
        if constexpr (kEarly) {
#pragma unroll
          for (int i = 0; i < 4; ++i) b[0][i] = early[n][o][0][i];
        } else {
          load_tokens<T, ALIGNED>(x[o], k + 8 * n, p.depth, b);
        }
        __syncwarp();                                      // a row's ragged end parts the lanes; matrix instructions want them together
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int r = 0; r < TALL; ++r) {
            Codes<T>::mma(part[r][o], lo[r], hi[r], b[q][0], b[q][1]);
            Codes<T>::mma(part[r][o], lo[r] + 2, hi[r] + 2, b[q][2], b[q][3]);
          }
      }
    }
#pragma unroll
    for (int r = 0; r < TALL; ++r) {
      const float s0 = meta_step(word[2 * r]), s1 = meta_step(word[2 * r + 1]);
#pragma unroll
      for (int o = 0; o < OCTETS; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[r][o][i] = fmaf(part[r][o][i], i < 2 ? s0 : s1, sum[r][o][i]);
    }
  }
#pragma unroll
  for (int r = 0; r < TALL; ++r)
#pragma unroll
    for (int o = 0; o < OCTETS; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[warp][8 * o + 2 * quad + (i & 1)][16 * r + g + 8 * (i >> 1)] = sum[r][o][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += 32 * kWarps) {
    const int64_t c = c0 + i % kRows, t = t0 + i / kRows;
    if (c >= p.channels || t >= p.tokens) continue;
    float v = 0.0f;
#pragma unroll
    for (int n = 0; n < kWarps; ++n) v += total[n][i / kRows][i % kRows];
    static_cast<T*>(p.out)[rank * p.rank_out + t * p.ld_out + c] = from_float<T>(v);
  }
}

__device__ __forceinline__ float load_cluster(uint32_t at, uint32_t block) {
  float v;
  asm volatile("{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %1, %2;\n\tld.shared::cluster.f32 %0, [there];\n\t}"
               : "=f"(v) : "r"(at), "r"(block) : "memory");
  return v;
}

// OCTETS: of tokens; WORDS: of a row's window, a thread's (a window is 32 WORDS
// codes of one group).  `split`: blocks of the cluster, which share the depth.
template <typename T, int OCTETS, int WORDS>
struct Tiled {
  static constexpr int kChannels = 16 * kWarps, kCols = 8 * OCTETS, kWindow = 32 * WORDS;
  static constexpr int kSlab = sizeof(T) == 4 && OCTETS > 1 ? 4 : 8;       // windows of tokens in shared memory at once
  static constexpr int kPitch = 2 * kWindow + 64;          // bytes from token to token: two rows that are read together meet no bank twice
  static constexpr int kTokens = parts<T>() * kSlab * kCols * kPitch;
  static constexpr int kTotal = kCols * (kChannels + 4) * 4;
  static constexpr int kBytes = kTokens > kTotal ? kTokens : kTotal;
};
template <typename T, int OCTETS, int WORDS, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps, 2) linear4_tiled_kernel(const Linear4Args p, const int split) {
  using S = Tiled<T, OCTETS, WORDS>;
  constexpr int kChannels = S::kChannels, kCols = S::kCols, kWindow = S::kWindow, kSlab = S::kSlab, kPitch = S::kPitch;
  constexpr int kParts = parts<T>(), kAhead = 4;           // windows of codes loaded ahead
  constexpr int kEights = kCols * kWindow / 8;             // of a window of tokens
  extern __shared__ __align__(16) uint8_t tokens[];        // [parts][windows][tokens], then the sums
  float (*const total)[kChannels + 4] = reinterpret_cast<float (*)[kChannels + 4]>(tokens);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, quad = lane & 3;
  const int part_of = (int)(blockIdx.x % split);
  const int64_t rank = blockIdx.z, c0 = (int64_t)(blockIdx.x / split) * kChannels, t0 = (int64_t)blockIdx.y * kCols;
  const int64_t bytes = (p.depth + 1) / 2;
  const uint32_t base = unknown(Codes<T>::kBase);
  pdl_wait();
  pdl_trigger();
  // Rows past the last channel or token repeat it: their results are dropped.
  const uint8_t* codes[2];
  const uint32_t* meta[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t c = c0 + 16 * warp + 8 * i + g < p.channels ? c0 + 16 * warp + 8 * i + g : p.channels - 1;
    codes[i] = pinned(p.codes + rank * p.rank_codes + c * p.ld_codes);
    meta[i] = pinned(p.meta + rank * p.rank_meta + c * p.ld_meta);
  }
  const T* const x = pinned(static_cast<const T*>(p.x) + rank * p.rank_x);
  const int64_t all = (p.depth + kWindow - 1) / kWindow;
  const int64_t first = all * part_of / split, last = all * (part_of + 1) / split;
  const int groups = p.group / kWindow;                    // windows of a group
  uint32_t w[kAhead][2][WORDS], word[kAhead][2];
  auto load = [&](int slot, int64_t window) {
    const bool there = window < last;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_codes<WORDS, ALIGNED>(codes[i], there ? window * (kWindow / 2) + 4 * WORDS * quad : bytes, bytes, w[slot][i]);
      word[slot][i] = there ? load_free4(meta[i] + (uint32_t)window / (uint32_t)groups) : 0;
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, first + i);
  float sum[OCTETS][4] = {};
#pragma unroll 1
  for (int64_t slab = first; slab < last; slab += kSlab) {
    if (slab != first) __syncthreads();                    // the slab before has been read
    const int windows = last - slab < kSlab ? (int)(last - slab) : kSlab;
#pragma unroll 4
    for (int e = tid; e < windows * kEights; e += 32 * kWarps) {
      const int window = e / kEights, token = e % kEights / (kWindow / 8), eight = e % (kWindow / 8);
      const int64_t t = t0 + token < p.tokens ? t0 + token : p.tokens - 1;
      uint32_t h[kParts][4];
      load_tokens<T, ALIGNED>(x + t * p.ld_x, (slab + window) * kWindow + 8 * eight, p.depth, h);
#pragma unroll
      for (int q = 0; q < kParts; ++q)                     // eights that lanes read together lie side by side
        *reinterpret_cast<uint4*>(tokens + ((q * kSlab + window) * kCols + token) * kPitch + 16 * (eight % WORDS * 4 + eight / WORDS)) =
            make_uint4(h[q][0], h[q][1], h[q][2], h[q][3]);
    }
    __syncthreads();
#pragma unroll 1
    for (int w0 = 0; w0 < windows; w0 += kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (w0 + d >= windows) break;                      // the whole block
        float part[OCTETS][4] = {};
        uint32_t zero[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) zero[i] = Codes<T>::base_and(meta_zero(word[d][i]));
#pragma unroll
        for (int n = 0; n < WORDS; ++n) {
          uint32_t lo[4], hi[4];
          turn<T>(w[d][0][n], base, zero[0], lo);
          turn<T>(w[d][1][n], base, zero[1], hi);
#pragma unroll
          for (int o = 0; o < OCTETS; ++o)
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              const uint4 b = *reinterpret_cast<const uint4*>(tokens + ((q * kSlab + w0 + d) * kCols + 8 * o + g) * kPitch +
                                                              16 * (4 * n + quad));
              Codes<T>::mma(part[o], lo, hi, b.x, b.y);
              Codes<T>::mma(part[o], lo + 2, hi + 2, b.z, b.w);
            }
        }
        const float s0 = meta_step(word[d][0]), s1 = meta_step(word[d][1]);
#pragma unroll
        for (int o = 0; o < OCTETS; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[o][i] = fmaf(part[o][i], i < 2 ? s0 : s1, sum[o][i]);
        load(d, slab + w0 + d + kAhead);
      }
    }
  }
  __syncthreads();                                         // the tokens' place is free
#pragma unroll
  for (int o = 0; o < OCTETS; ++o)
#pragma unroll
    for (int i = 0; i < 4; ++i) total[8 * o + 2 * quad + (i & 1)][16 * warp + g + 8 * (i >> 1)] = sum[o][i];
  if (split > 1) cluster_barrier();
  else __syncthreads();
  const int here = p.tokens - t0 < kCols ? (int)(p.tokens - t0) : kCols;
  for (int i = tid + 32 * kWarps * part_of; i < here * kChannels; i += 32 * kWarps * split) {
    const int64_t c = c0 + i % kChannels, t = t0 + i / kChannels;
    if (c >= p.channels) continue;
    float v = 0.0f;
    if (split == 1) {
      v = total[i / kChannels][i % kChannels];
    } else {
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(&total[i / kChannels][i % kChannels]);
      for (int b = 0; b < split; ++b) v += load_cluster(at, b);
    }
    static_cast<T*>(p.out)[rank * p.rank_out + t * p.ld_out + c] = from_float<T>(v);
  }
  if (split > 1) cluster_barrier();                        // no block leaves while its sums are read
}

template <typename T>
bool rows_aligned(const Linear4Args& p) {
  const int64_t in16 = 16 / (int64_t)sizeof(T);
  return on_boundary(p.codes, 16) && (p.channels == 1 || p.ld_codes % 16 == 0) && (p.ranks == 1 || p.rank_codes % 16 == 0) &&
         on_boundary(p.x, 16) && (p.tokens == 1 || p.ld_x % in16 == 0) && (p.ranks == 1 || p.rank_x % in16 == 0);
}
template <typename T, int OCTETS, int TALL, int WORDS>
cudaError_t launch_direct(const Linear4Args& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.channels + 16 * TALL - 1) / (16 * TALL)),
                     (unsigned)((p.tokens + 8 * OCTETS - 1) / (8 * OCTETS)), (unsigned)p.ranks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return rows_aligned<T>(p) ? cudaLaunchKernelEx(&cfg, linear4_kernel<T, OCTETS, TALL, WORDS, true>, p)
                            : cudaLaunchKernelEx(&cfg, linear4_kernel<T, OCTETS, TALL, WORDS, false>, p);
}
template <typename T, int OCTETS, int WORDS>
cudaError_t launch_tiled(const Linear4Args& p, int sms, cudaStream_t s) {
  using S = Tiled<T, OCTETS, WORDS>;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    const cudaError_t one = cudaFuncSetAttribute(linear4_tiled_kernel<T, OCTETS, WORDS, true>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    return one != cudaSuccess ? one : cudaFuncSetAttribute(linear4_tiled_kernel<T, OCTETS, WORDS, false>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  // The depth is shared by as many blocks, up to 8, as all run at once (two an
  // SM) and leave each four windows.
  const int64_t blocks = (p.channels + S::kChannels - 1) / S::kChannels, windows = (p.depth + S::kWindow - 1) / S::kWindow;
  const int64_t columns = (p.tokens + S::kCols - 1) / S::kCols;
  int split = 1;
  while (split < 8 && blocks * columns * p.ranks * split <= sms && windows >= 8 * split) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * split), (unsigned)columns, (unsigned)p.ranks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0] = overlapped_launch();
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return rows_aligned<T>(p) ? cudaLaunchKernelEx(&cfg, linear4_tiled_kernel<T, OCTETS, WORDS, true>, p, split)
                            : cudaLaunchKernelEx(&cfg, linear4_tiled_kernel<T, OCTETS, WORDS, false>, p, split);
}
template <typename T, int WORDS>
cudaError_t launch(const Linear4Args& p, int sms, cudaStream_t s) {
  // 32 channels a block halve the loads of the tokens' elements, if there are
  // blocks enough (one token, 14336 x 4096: 11.4 us, with 16 channels 13.9; 7 x
  // 1111 x 2051: 5.6 us with 16, 8.1 with 32).  Of 9 to 16 tokens those loads
  // are as many as the codes' in each warp (in fp32 twice, and parts are made of
  // them), and of large weights they cost more than shared memory does.  16 tokens,
  // by themselves and through shared memory: 2^24 weights (4096 x 4096) 7.4 and
  // 9.7 us, 2^25 12.2 and 13.6, 14336 x 4096 23.1 and 21.2; in fp32 2^20 (1024 x
  // 1024) 4.6 and 9.3, 2^22 7.9 and 9.1, 2^24 14.6 and 12.6, 2^25 22.2 and 19.0.
  const int64_t blocks = (p.channels + 31) / 32 * p.ranks;
  const bool many = blocks * 4 >= 3 * sms;
  if (p.tokens <= 8) return many ? launch_direct<T, 1, 2, WORDS>(p, s) : launch_direct<T, 1, 1, WORDS>(p, s);
  if (p.tokens <= 16 && p.ranks * p.channels * p.depth <= (int64_t)1 << (sizeof(T) == 4 ? 23 : 25))
    return many ? launch_direct<T, 2, 2, WORDS>(p, s) : launch_direct<T, 2, 1, WORDS>(p, s);
  if (p.tokens <= 16) return launch_tiled<T, 2, WORDS>(p, sms, s);
  return launch_tiled<T, sizeof(T) == 4 ? 2 : 4, WORDS>(p, sms, s);      // (three parts of fp32 tokens: 16 at once)
}
template <typename T>
cudaError_t launch(const Linear4Args& p, int sms, cudaStream_t s) {
  return p.group == 64 ? launch<T, 2>(p, sms, s) : launch<T, 4>(p, sms, s);
}

}  // namespace

cudaError_t launch_linear4(const Linear4Args& p, int sms, cudaStream_t s) {
  if (p.dtype == ECHO_F32) return launch<float>(p, sms, s);
  if (p.dtype == ECHO_BF16) return launch<__nv_bfloat16>(p, sms, s);
  return launch<__half>(p, sms, s);
}

}  // namespace echo
