// serve_common.h -- shared by the operators of a serving step (cache_*.cu,
// attn_*.cu, int4_*.cu): launch arguments, a batch's geometry, and the group
// quantizer with exact quotients.  The operators are described in
// include/echo.h.
#pragma once

#include "ops_common.h"
#include "quant.cuh"

namespace echo {

// Places that a table may have (sums of places stay inside 32 bits).
constexpr int kMostPlaces = 1 << 30;
// Bits of the status words.
constexpr int kBadPage = 1, kBadRows = 2, kNaNGroup = 4, kGaveUp = 8;

struct CacheArgs {
  uint8_t* codes;
  uint32_t* meta;
  int64_t pages;
  int heads, head_dim, bits;
  int page_shift;                // log2 of page_size
};

struct BatchArgs {
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* table;
  int64_t ld_table;
  int sequences, tokens, table_pages;
};

struct HeadsArgs {
  void* data;
  int64_t ld, head_stride;
};

struct RowsArgs {
  CacheArgs cache;
  BatchArgs batch;
  HeadsArgs k, v;                // data nullptr: not read back
};

struct AttentionArgs {
  CacheArgs cache;
  BatchArgs batch;
  HeadsArgs q, out;
  float* lse;
  int heads, group;              // query heads, and to a head of the cache
  int dtype;
  float scale;
  int causal;
  int window;                    // 0: none
  float* partial;                // workspace
};

struct WeightsArgs {
  const void* w;
  int64_t ld_w, rank_w;
  uint8_t* codes;
  int64_t ld_codes, rank_codes;
  uint32_t* meta;
  int64_t ld_meta, rank_meta;
  int64_t ranks, channels, depth;
  int group;
};

struct Linear4Args {
  const void* x;
  int64_t ld_x, rank_x;
  const uint8_t* codes;
  int64_t ld_codes, rank_codes;
  const uint32_t* meta;
  int64_t ld_meta, rank_meta;
  void* out;
  int64_t ld_out, rank_out;
  int64_t ranks, tokens, channels, depth;
  int group, dtype;
};

cudaError_t launch_append(const RowsArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_read(const RowsArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_attention(const AttentionArgs& a, int sms, cudaStream_t s);
int64_t attention_bytes(int head_dim, int sms);        // of its workspace
cudaError_t launch_quantize_weights(const WeightsArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_linear4(const Linear4Args& a, int sms, cudaStream_t s);

// Each translation unit whose kernels report has a status word of its own:
// read copies it to the host on a stream, clear takes the bits that were read
// off it (one that a kernel sets meanwhile is the next call's to report).
struct StatusWord {
  cudaError_t (*read)(int* word, cudaStream_t s);
  cudaError_t (*clear)(int bits, cudaStream_t s);
};
StatusWord rows_status();
StatusWord attn_few_status();
StatusWord attn_many_status();
StatusWord weights_status();

#define ECHO_STATUS_WORD                                                              \
  __device__ int g_status;                                                            \
  __global__ void clear_status(int bits) { atomicAnd(&g_status, ~bits); }             \
  cudaError_t read_status(int* word, cudaStream_t s) {                                \
    return cudaMemcpyFromSymbolAsync(word, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s); \
  }                                                                                   \
  cudaError_t clear_status_bits(int bits, cudaStream_t s) {                           \
    clear_status<<<1, 1, 0, s>>>(bits);                                               \
    return cudaGetLastError();                                                        \
  }                                                                                   \
  __device__ __forceinline__ void report(int bits) { atomicOr(&g_status, bits); }

// a / b of no negative numbers, in 32 bits where they fit (a division in 64 takes
// five times as long).
__device__ __forceinline__ int64_t divided(int64_t a, int64_t b) {
  return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// ------------------------------------------------------------------ batches
// One sequence of a batch: its rows of the token tensors and its tokens in the
// cache, as far as the arrays make sense.
struct Sequence {
  int row, rows;                 // first of its rows, and how many
  int length;                    // as given (0 if negative, cut off far behind any table's end)
  int keys;                      // of these, that the table has room for
  int place;                     // of its first row, may be negative
};
__device__ __forceinline__ Sequence sequence_of(const BatchArgs& b, int page_shift, int i, int* bad) {
  Sequence s;
  const int first = b.starts[i], last = b.starts[i + 1], length = b.lengths[i];
  if (last < first || first < 0 || last > b.tokens) *bad |= kBadRows;
  const int from = first < 0 ? 0 : first, to = last > b.tokens ? b.tokens : last;
  s.row = from;
  s.rows = to > from ? to - from : 0;
  s.length = length < 0 ? 0 : length < kMostPlaces + (1 << 20) ? length : kMostPlaces + (1 << 20);
  const int64_t room = (int64_t)b.table_pages << page_shift;
  s.keys = s.length < room ? s.length : (int)room;
  if (s.rows > 0 && s.length > room) *bad |= kBadPage;
  // row `first` is at length - (last - first), whether or not it exists
  const int64_t place = (int64_t)s.length - ((int64_t)last - from);
  s.place = place < -(1 << 30) ? -(1 << 30) : (int)place;
  return s;
}

// The sequence whose rows hold row t (as far as starts rise), -1 or
// `sequences` where none does; of a whole warp, 32 probes a step.
__device__ __forceinline__ int sequence_at(const BatchArgs& b, int t, int lane) {
  int lo = 0, n = b.sequences + 1;
  for (;;) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool below = at < n && b.starts[lo + at] <= t;
    const int k = __popc(__ballot_sync(kFull, below));
    if (k == 0) return lo - 1;
    if (step == 1) return lo + k - 1;
    lo += (k - 1) * step;
    n = n - (k - 1) * step < step ? n - (k - 1) * step : step;
  }
}

// The page of a place, or -1 (reported) if the table or the cache has none.
__device__ __forceinline__ int page_of(const BatchArgs& b, const CacheArgs& c, int sequence, int place) {
  const int at = place >> c.page_shift;
  if (at >= b.table_pages) return -1;
  const int page = b.table[(int64_t)sequence * b.ld_table + at];
  return page >= 0 && page < c.pages ? page : -1;
}

// Where the groups of a page's place begin, in groups: keys, or values `heads << page_shift` later.
__device__ __forceinline__ int64_t group_index(const CacheArgs& c, int page, int head, int place) {
  return ((((int64_t)page * 2 * c.heads + head) << c.page_shift) + (place & ((1 << c.page_shift) - 1)));
}

// ------------------------------------------------------------------- groups
// The least fp16 number s with s * L >= hi - lo, exactly: from an approximate
// quotient, which is off by one step at most.  s * L has 19 bits, so it is
// exact in fp32; hi - lo is d + e exactly, and s * L - d is exact because the
// two are near each other.
__device__ __forceinline__ bool covers(unsigned short s, float L, float d, float e) {
  return __fsub_rn(__fmul_rn(__half2float(__ushort_as_half(s)), L), d) >= e;
}
struct GroupStep {
  float s, inv, zf;
  uint32_t meta;
  bool finite;
};
// rint(v / s) with the quotient exact, for |v / s| < 256 and inv within 2^-23 of
// 1 / s (so the product is within 256 * 3 * 2^-24 of the quotient, less than
// 2^-13): where the product with inv lies near a half, v is compared with s times that
// half, which has 21 bits at most and so is exact.
__device__ __forceinline__ float exact_rint(float v, float s, float inv) {
  const float t = __fmul_rn(v, inv), r = rint_small(t);
  if (fabsf(__fsub_rn(t, r)) < kFastRintLimit) return r;
  const float low = floorf(t), half = __fmul_rn(s, __fadd_rn(low, 0.5f));
  if (v != half) return v > half ? __fadd_rn(low, 1.0f) : low;
  return rintf(__fadd_rn(low, 0.5f));
}
__device__ __forceinline__ GroupStep group_step(float lo, float hi, float L) {
  GroupStep g;
  const float d = __fsub_rn(hi, lo), b = -lo, bb = __fsub_rn(d, hi);
  const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(d, bb)), __fsub_rn(b, bb));   // hi - lo is d + err
  unsigned short s = __half_as_ushort(__float2half_ru(__fmul_rn(d, 1.0f / L)));
  g.finite = isfinite(d);
  if (g.finite) {
    if (s > 0x7BFF) s = 0x7BFF;  // the quotient of 65504 L is beyond 65504 as fp32 has it
    if (!covers(s, L, d, err)) ++s;
    else if (s > 0 && covers(s - 1, L, d, err)) --s;
    if (s == 0) s = 0x3C00;      // 1, only for a group of zeros
    g.finite = s < 0x7C00;
  }
  g.s = __half2float(__ushort_as_half(s));
  asm("rcp.approx.f32 %0, %1;" : "=f"(g.inv) : "f"(g.s));
  g.zf = 0.0f;
  g.meta = 0x7E00u;              // a step of NaN
  if (g.finite) {
    g.zf = fminf(fmaxf(exact_rint(-lo, g.s, g.inv), 0.0f), L);
    g.meta = (uint32_t)s | ((uint32_t)__half_as_ushort(__float2half_rn(g.zf)) << 16);
  }
  return g;
}
// Codes of 8 values, packed as by pack8.  Quotients come from the product with
// inv unless one of the 8 lies near a half.  v >= lo, so rint(v / s) >= -z
// without a clamp (rint is monotonic and odd); only the upper one is applied.
template <int BITS>
__device__ __forceinline__ void group_codes8(const float (&v)[8], const GroupStep& g, uint32_t& w0, uint32_t& w1) {
  constexpr float L = BITS == 4 ? 15.0f : 255.0f, M = 12582912.0f;        // 1.5 * 2^23, see rint_small
  float t[8], r[8], e[8], c[8];
  mul_ns<8>(t, v, g.inv);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    add2(r[k], r[k + 1], t[k], t[k + 1], M, M);
    sub2(r[k], r[k + 1], r[k], r[k + 1], M, M);
  }
  sub_n<8>(e, t, r);
  float off = max3(fabsf(e[0]), fabsf(e[1]), fabsf(e[2]));
  off = max3(off, fabsf(e[3]), fabsf(e[4]));
  off = max3(off, fabsf(e[5]), fabsf(e[6]));
  off = fmaxf(off, fabsf(e[7]));
  if (off >= kFastRintLimit)
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = exact_rint(v[k], g.s, g.inv);
  const float most = __fsub_rn(L, g.zf);
#pragma unroll
  for (int k = 0; k < 8; ++k) c[k] = fminf(r[k], most);
#pragma unroll
  for (int k = 0; k < 8; k += 2) add2(c[k], c[k + 1], c[k], c[k + 1], g.zf, g.zf);
  pack8<BITS>(c, w0, w1);
  if (!g.finite) w0 = w1 = 0;
}
__device__ __forceinline__ float meta_step(uint32_t meta) {
  return __half2float(__ushort_as_half((unsigned short)(meta & 0xFFFFu)));
}
__device__ __forceinline__ float meta_zero(uint32_t meta) {
  return __half2float(__ushort_as_half((unsigned short)(meta >> 16)));
}

// Groups of which NL lanes have 16 values each.  A group's step takes more than a
// hundred instructions, so a warp that has G steps of 32 / NL groups lets lane q
// of NL find that of step q % G: lanes hand on half of their ranges at a time.
//
// The range of 16 values and 0.
template <typename T>
__device__ __forceinline__ void range_of(const Pack<T, 8> (&x)[2], float& lo, float& hi) {
  if constexpr (sizeof(T) == 4) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = x[k / 8].v[k % 8];
    group_range<1>(v, lo, hi);
  } else {
    using Two = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const Two* a = reinterpret_cast<const Two*>(&x[0]);
    const Two* b = reinterpret_cast<const Two*>(&x[1]);
    Two low[4], high[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      low[k] = __hmin2_nan(a[k], b[k]);
      high[k] = __hmax2_nan(a[k], b[k]);
    }
    const Two l = __hmin2_nan(__hmin2_nan(low[0], low[1]), __hmin2_nan(low[2], low[3]));
    const Two h = __hmax2_nan(__hmax2_nan(high[0], high[1]), __hmax2_nan(high[2], high[3]));
    lo = min3_nan(to_float(l.x), to_float(l.y), 0.0f);
    hi = max3_nan(to_float(h.x), to_float(h.y), 0.0f);
  }
}
// The step of step q % G's group, from the parts of all; of a whole warp.
template <int NL, int G>
__device__ __forceinline__ GroupStep shared_step(float (&lo)[G], float (&hi)[G], int q, float L) {
  int n = G;
#pragma unroll
  for (int off = 1; off < NL; off <<= 1) {
    if (n > 1) {                         // this lane keeps the steps whose next bit is its own
      const bool odd = q & off;
#pragma unroll
      for (int j = 0; j < n / 2; ++j) {
        const float l = __shfl_xor_sync(kFull, odd ? lo[2 * j] : lo[2 * j + 1], off);
        const float h = __shfl_xor_sync(kFull, odd ? hi[2 * j] : hi[2 * j + 1], off);
        lo[j] = min_nan(odd ? lo[2 * j + 1] : lo[2 * j], l);
        hi[j] = max_nan(odd ? hi[2 * j + 1] : hi[2 * j], h);
      }
      n /= 2;
    } else {
      lo[0] = min_nan(lo[0], __shfl_xor_sync(kFull, lo[0], off));
      hi[0] = max_nan(hi[0], __shfl_xor_sync(kFull, hi[0], off));
    }
  }
  return group_step(lo[0], hi[0], L);
}
// Step i's, from the lane that has it; of a whole warp.
template <int NL, int G>
__device__ __forceinline__ GroupStep step_at(const GroupStep& mine, int i) {
  if constexpr (G == 1) return mine;
  const int from = (threadIdx.x & 31 & ~(NL - 1)) | i;
  GroupStep g;
  g.meta = __shfl_sync(kFull, mine.meta, from);
  g.inv = __shfl_sync(kFull, mine.inv, from);
  g.s = meta_step(g.meta);
  g.zf = meta_zero(g.meta);
  g.finite = (g.meta & 0x7FFFu) < 0x7C00u;
  return g;
}

// (w & MASK) | base in one instruction: an instruction takes one constant, so
// the base is a register that the compiler does not know (it made two of them,
// and the codes' turning bounds these kernels).
__device__ __forceinline__ uint32_t unknown(uint32_t v) {
  uint32_t r;
  asm("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked(uint32_t w, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(base));
  return r;
}

}  // namespace echo
