// attn_few.cu -- echo_attention for few rows a sequence (include/echo.h):
// decode, drafted tokens.
//
// Every key is read once for 16 rows, so the kernel streams codes: each warp
// copies 16 keys and values at a time into a ring of its own (asynchronous
// copies, no barrier between warps) and feeds them to matrix instructions of 16
// rows.  A code c behind the bits of 1024 is the f16 number 1024 + c (of 4 bits
// at bit 4: 1024 + 16 c), from which one instruction for two codes takes c - z,
// exactly; steps are multiplied into scores and weights in fp32.  (f16 holds
// c * 2^-24 as it stands, as a subnormal, but the matrix instructions align
// their sums by exponents that leave such a number 14 bits.)  The step s of a
// value goes into the weight, p_j = exp(score_j + log s_j - m), whose running
// maximum m then bounds p_j by 2^8 whatever the steps are (it is raised only
// when a score passes it by 2^8), so that p_j has 11 bits in f16; the sum of
// weights takes p_j / s_j.
//
// Blocks take equal shares of the batch's tiles (attn_common.h); four warps
// take a tile's 64 keys and join at the unit's end, and parts of units that
// several blocks have had are joined by a second kernel.
#include "attn_common.h"

namespace echo {
namespace {

ECHO_STATUS_WORD

constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 16, kStep = 16, kTile = kStep * kWarps;
constexpr int kLeast = 2;                // tiles of a block: fewer parts to join where a batch is small
// Blocks an SM: what registers allow (of rows of 256, sums alone take 128 a thread).
template <int D> __host__ __device__ constexpr int few_blocks() { return D == 256 ? 2 : 3; }
constexpr float kAhead = 8.0f;           // a score may pass the maximum by this much, as a power of two

template <int D, int BITS>
struct Shape {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kStage = 2 * kStep * kRowBytes + 2 * kStep * 4;     // keys, values, meta of both
  static constexpr int kStages = kRowBytes >= 256 ? 3 : 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * kRows * D * 4;   // the warps' sums, in the ring's place
  static constexpr int kQuery = D / 16 * 32 * 16;        // rows as the instructions' operands
  static constexpr int kBytes = (kRing > kJoin ? kRing : kJoin) + kQuery;
  static constexpr int kKeyPiece = kRowBytes / 4 < 16 ? kRowBytes / 4 : 16;      // bytes a thread takes at once
  static constexpr int kValuePiece = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;
  static constexpr int kPerWord = 32 / BITS;
};

// Where 16-byte piece `piece` of row r lies in a stage: turned so that the lanes
// that load together meet no bank twice.  Values' rows are reordered: those of
// even keys of eight, then odd.
template <int ROW_BYTES>
__device__ __forceinline__ int key_at(int r, int piece) {
  return r * ROW_BYTES + (ROW_BYTES >= 128 ? piece ^ ((r & 1) << 2) : piece) * 16;
}
__device__ __forceinline__ int value_row(int r) { return (r & 8) + ((r & 7) >> 1) + 4 * (r & 1); }
template <int ROW_BYTES>
__device__ __forceinline__ int value_at(int at, int piece) {     // at: value_row
  return at * ROW_BYTES + (ROW_BYTES >= 128 ? piece ^ (2 * (at & 3)) : ROW_BYTES == 64 ? piece ^ (at & 2) : piece) * 16;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t at, uint32_t* w) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {         // a in the low half
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes less their zero points (of two rows, for values) as pairs of f16.
// `low` is 1024 + z, `high` 64 + z, twice.
struct Zero {
  uint32_t low, high, base;              // base: 1024, twice
};
__device__ __forceinline__ Zero zero_of(uint32_t zs, uint32_t base) {     // two fp16 zero points
  const __half2 z = *reinterpret_cast<const __half2*>(&zs);
  const __half2 low = __hadd2(z, __float2half2_rn(1024.0f)), high = __hneg2(__hadd2(z, __float2half2_rn(64.0f)));
  return {*reinterpret_cast<const uint32_t*>(&low), *reinterpret_cast<const uint32_t*>(&high), base};
}
__device__ __forceinline__ uint32_t less_low(uint32_t v, const Zero& z) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&z.low));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t less_high(uint32_t v, const Zero& z) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f),
                            *reinterpret_cast<const __half2*>(&z.high));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t low_codes(uint32_t w, const Zero& z) {        // at bits 0 and 16
  return less_low(masked<0x000F000Fu>(w, z.base), z);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, const Zero& z) {       // at bits 4 and 20
  return less_high(masked<0x00F000F0u>(w, z.base), z);
}
__device__ __forceinline__ uint32_t byte_codes(uint32_t w, uint32_t bytes, const Zero& z) {
  return less_low(__byte_perm(w, z.base, bytes), z);
}

// Loads the unit's rows as operands: for each matrix instruction and lane, the
// four registers in a row.  Element e of a row meets the code that the lane
// of its quarter finds at the same place of its words.  The rows' factors go to
// shared memory (NaN for a row with a non-finite element).
template <typename T, int D, int BITS>
__device__ __forceinline__ void load_queries(const AttentionArgs& a, const Sequence& s, const Unit& u, uint8_t* query,
                                             float* factor) {
  using S = Shape<D, BITS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kRows / kWarps; ++i) {
    const int r = warp * (kRows / kWarps) + i, row = u.first + r;
    float v[D / 32];
    uint32_t top = 0;
    if (r < u.rows) {
      const T* from = static_cast<const T*>(a.q.data) + (int64_t)(s.row + row / a.group) * a.q.ld +
                      (int64_t)(u.head * a.group + row % a.group) * a.q.head_stride;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v[k] = to_float(from[lane + 32 * k]);
    } else {
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v[k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) top = max(top, abs_bits(v[k]));
    top = __reduce_max_sync(kFull, top);
    const float f = row_factor(top);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int e = lane + 32 * k;
      constexpr int kPiece = S::kKeyPiece * 8 / BITS;      // elements
      const int piece = e / kPiece, in = e % kPiece, quad = piece & 3;
      const int word = (piece >> 2) * (S::kKeyPiece / 4) + in / S::kPerWord, c = in % S::kPerWord;
      const int instruction = BITS == 4 ? 2 * word + ((c >> 1) & 1) : word;
      const int half = BITS == 4 ? c >> 2 : c & 1, second = BITS == 4 ? c & 1 : c >> 1;
      const int at = ((instruction * 32 + (r & 7) * 4 + quad) * 4 + 2 * second + (r >> 3)) * 4 + 2 * half;
      *reinterpret_cast<__half*>(query + at) = __float2half_rn(v[k] * f);
    }
    if (lane == 0) factor[r] = top < 0x7F800000u ? a.scale * kLog2E / f : __int_as_float(0x7FC00000);
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, few_blocks<D>()) attention_few_kernel(const AttentionArgs a, const int vector_out) {
  using S = Shape<D, BITS>;
  constexpr int kCols = D / 8;                             // tiles of 8 columns
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ int64_t shared[kWarps + 3];
  __shared__ float factor[kRows], most[kWarps][kRows], weight[kWarps][kRows];
  uint8_t* const query = raw + (S::kBytes - S::kQuery);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, quad = lane & 3;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(raw) + warp * S::kStages * S::kStage;
  const uint32_t base1024 = unknown(0x64006400u);
  pdl_wait();
  pdl_trigger();
  if (tid == 0) joins(a)[blockIdx.x].blocks = 0;
  int bad = 0;
  const Range range = block_range<kRows, kTile, kThreads, kLeast>(a, shared, &bad);
  const int heads = a.cache.heads, page_size = 1 << a.cache.page_shift;
  Walk<kRows, kTile> walk;
  for (walk.start(a, range, &bad); walk.more(); walk.next(a, &bad)) {
    const Sequence& s = walk.s;
    const Unit& u = walk.unit;
    const int tiles = walk.take;
    const bool whole = walk.whole();
    __syncthreads();                                       // the last unit's sums have been read
    if (a.dtype == ECHO_BF16) load_queries<__nv_bfloat16, D, BITS>(a, s, u, query, factor);
    else load_queries<__half, D, BITS>(a, s, u, query, factor);
    __syncthreads();
    const bool tall = u.rows > 8;
    float row_scale[2];
    int from[2], to[2];                                    // keys that rows g and g + 8 see
    int all_from = 0, all_to = 0x7FFFFFFF, end = 0;        // that all rows see, and where the last that any sees ends
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h, place = s.place + (u.first + r) / a.group;
      row_scale[h] = factor[r];
      from[h] = r < u.rows ? keys_from(a, place) : 0;
      to[h] = r < u.rows ? keys_to(a, s, place) : 0;
    }
    {
      const int first = s.place + u.first / a.group, last = s.place + (u.first + u.rows - 1) / a.group;
      all_to = keys_to(a, s, first);
      all_from = keys_from(a, last);
      end = keys_to(a, s, last);
    }

    float sums[kCols][4], m[2] = {kLowest, kLowest}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) sums[c][k] = 0.0f;

    const int key0 = (u.tile + walk.in) * kTile + kStep * warp;            // of this warp's first step
    const int64_t values_on = (int64_t)heads << a.cache.page_shift;        // groups from a key's to its value's
    uint32_t missing = 0;                                  // stages without a page
    auto look_up = [&](int t) {
      const int key = key0 + t * kTile;
      return t < tiles && key < end ? page_of(a.batch, a.cache, u.sequence, key) : -1;
    };
    auto issue = [&](int t, int page, int stage) {
      const int key = key0 + t * kTile;
      missing &= ~(1u << stage);
      if (page >= 0) {
        const int64_t group = group_index(a.cache, page, u.head, key & (page_size - 1));
        const uint8_t* codes = a.cache.codes + group * S::kRowBytes;
        const uint32_t base = ring + stage * S::kStage;
        constexpr int kPieces = S::kRowBytes / 16;         // of a row; a stage's rows have 32 lanes' worth of them or more
#pragma unroll
        for (int n = 0; n < kPieces * kStep / 32; ++n) {
          const int piece = lane + 32 * n, r = piece / kPieces, p = piece % kPieces;
          copy16_async(base + key_at<S::kRowBytes>(r, p), codes + piece * 16);
          copy16_async(base + kStep * S::kRowBytes + value_at<S::kRowBytes>(value_row(r), p),
                       codes + values_on * S::kRowBytes + piece * 16);
        }
        if (lane < 8)
          copy16_async(base + 2 * kStep * S::kRowBytes + 16 * lane,
                       a.cache.meta + group + (lane < 4 ? 0 : values_on) + 4 * (lane & 3));
      } else if (t < tiles && key < end) {
        missing |= 1u << stage;
        bad |= kBadPage;
      }
      copies_commit();
    };
    int page = look_up(0);
#pragma unroll 1
    for (int t = 0; t < S::kStages - 1; ++t) {
      const int next = look_up(t + 1);
      issue(t, page, t);
      page = next;
    }
    int stage = 0, ahead = S::kStages - 1;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int key = key0 + t * kTile;
      copies_wait<S::kStages - 2>();
      __syncwarp();
      if (key < end && !(missing >> stage & 1)) {          // the whole warp
        const uint32_t base = ring + stage * S::kStage, meta = base + 2 * kStep * S::kRowBytes;
        float scores[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int k = 0; k < 4; ++k) scores[n][k] = 0.0f;
          constexpr int kWords = S::kRowBytes / 16, kPieceWords = S::kKeyPiece / 4;      // a thread's, of a row and at once
          uint32_t w[kWords];
#pragma unroll
          for (int p = 0; p < kWords / kPieceWords; ++p) {
            const int byte = (4 * p + quad) * S::kKeyPiece;
            load_words<S::kKeyPiece>(base + key_at<S::kRowBytes>(8 * n + g, byte / 16) + byte % 16, w + p * kPieceWords);
          }
          uint32_t word;
          load_words<4>(meta + (8 * n + g) * 4, &word);
          const Zero z = zero_of(__byte_perm(word, word, 0x3232), base1024);
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            if constexpr (BITS == 4) {
              const uint4 q0 = reinterpret_cast<const uint4*>(query)[2 * k * 32 + lane];
              const uint4 q1 = reinterpret_cast<const uint4*>(query)[(2 * k + 1) * 32 + lane];
              const uint32_t high = w[k] >> 8;
              mma_f16(scores[n], q0.x, q0.y, q0.z, q0.w, low_codes(w[k], z), high_codes(w[k], z));
              mma_f16(scores[n], q1.x, q1.y, q1.z, q1.w, low_codes(high, z), high_codes(high, z));
            } else {
              const uint4 q0 = reinterpret_cast<const uint4*>(query)[k * 32 + lane];
              mma_f16(scores[n], q0.x, q0.y, q0.z, q0.w, byte_codes(w[k], 0x5150, z), byte_codes(w[k], 0x5352, z));
            }
          }
        }
        // This thread's keys: 2 quad and 2 quad + 1 of each eight.
        uint32_t vmeta[2][2];
        const bool inside = key >= all_from && key + kStep <= all_to;      // every row sees all 16
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t kmeta[2];
          load_words<8>(meta + (8 * n + 2 * quad) * 4, kmeta);
          load_words<8>(meta + (kStep + 8 * n + 2 * quad) * 4, vmeta[n]);
          float ks[2], steps[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[e] = meta_step(kmeta[e]);
            steps[e] = log2_of(meta_step(vmeta[n][e]));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !tall) break;
            float *s0 = &scores[n][2 * h], *s1 = s0 + 1;
            mul2(*s0, *s1, *s0, *s1, row_scale[h], row_scale[h]);
            fma2(*s0, *s1, *s0, *s1, ks[0], ks[1], steps[0], steps[1]);
          }
        }
        if (!inside) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = key + 8 * n + 2 * quad + e;
              if (k >= end) vmeta[n][e] = 0x00003C00u;     // whatever lies there must not meet a weight of 0
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (k < from[h] || k >= to[h]) scores[n][2 * h + e] = kNone;
            }
        }
        // The maxima, where a score has passed them by far.
        float top[2];
        top[0] = fmaxf(fmaxf(scores[0][0], scores[0][1]), fmaxf(scores[1][0], scores[1][1]));
        top[1] = tall ? fmaxf(fmaxf(scores[0][2], scores[0][3]), fmaxf(scores[1][2], scores[1][3])) : kLowest;
        if (__any_sync(kFull, top[0] - kAhead > m[0] || top[1] - kAhead > m[1])) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
            top[h] = fmaxf(top[h], m[h]);
            const float f = exp2_of(m[h] - top[h]);
            m[h] = top[h];
            l[h] *= f;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              sums[c][2 * h] *= f;
              sums[c][2 * h + 1] *= f;
            }
          }
        }
        uint32_t p[2][2] = {{0, 0}, {0, 0}};               // weights of [keys' eight][rows' eight]
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float per[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) per[e] = reciprocal(meta_step(vmeta[n][e]));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && !tall) break;
            const float p0 = exp2_of(scores[n][2 * h] - m[h]), p1 = exp2_of(scores[n][2 * h + 1] - m[h]);
            if (inside) {
              l[h] = fmaf(p0, per[0], l[h]);
              l[h] = fmaf(p1, per[1], l[h]);
            } else {                                       // a hidden key's step may be anything
              if (scores[n][2 * h] != kNone) l[h] = fmaf(p0, per[0], l[h]);
              if (scores[n][2 * h + 1] != kNone) l[h] = fmaf(p1, per[1], l[h]);
            }
            p[n][h] = pack_f16(p0, p1);
          }
        }
        __syncwarp();                                      // hidden keys part the lanes; matrix instructions want them together
        // Values: columns of eight lanes' pieces, keys' pairs side by side.
        constexpr int kPieceWords = S::kValuePiece / 4, kPieces = S::kRowBytes / (8 * S::kValuePiece);
        const Zero zx = zero_of(__byte_perm(vmeta[0][0], vmeta[0][1], 0x7632), base1024);
        const Zero zy = zero_of(__byte_perm(vmeta[1][0], vmeta[1][1], 0x7632), base1024);
        const uint32_t values = base + kStep * S::kRowBytes;
#pragma unroll
        for (int piece = 0; piece < kPieces; ++piece) {
          const int byte = (8 * piece + g) * S::kValuePiece;
          uint32_t w[4][kPieceWords];                      // keys 2 quad, 2 quad + 1, and 8 on
#pragma unroll
          for (int k = 0; k < 4; ++k)
            load_words<S::kValuePiece>(
                values + value_at<S::kRowBytes>(8 * (k >> 1) + 4 * (k & 1) + quad, byte / 16) + byte % 16, w[k]);
#pragma unroll
          for (int k = 0; k < kPieceWords; ++k) {
            float(*out)[4] = &sums[(piece * kPieceWords + k) * S::kPerWord];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t x = __byte_perm(w[0][k], w[1][k], half ? 0x7632 : 0x5410);
              const uint32_t y = __byte_perm(w[2][k], w[3][k], half ? 0x7632 : 0x5410);
              auto add = [&](float(&to)[4], uint32_t b0, uint32_t b1) {
                mma_f16(to, p[0][0], p[0][1], p[1][0], p[1][1], b0, b1);
              };
              if constexpr (BITS == 4) {
                add(out[4 * half], low_codes(x, zx), low_codes(y, zy));
                add(out[4 * half + 1], high_codes(x, zx), high_codes(y, zy));
                add(out[4 * half + 2], low_codes(x >> 8, zx), low_codes(y >> 8, zy));
                add(out[4 * half + 3], high_codes(x >> 8, zx), high_codes(y >> 8, zy));
              } else {
                add(out[2 * half], byte_codes(x, 0x5250, zx), byte_codes(y, 0x5250, zy));
                add(out[2 * half + 1], byte_codes(x, 0x5351, zx), byte_codes(y, 0x5351, zy));
              }
            }
          }
        }
      }
      __syncwarp();                                        // before the stage is overwritten
      const int next = look_up(t + S::kStages);
      issue(t + S::kStages - 1, page, ahead);
      page = next;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
      ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
    }
    copies_wait<0>();
    __syncthreads();                                       // the rings are free

    // The warps' sums.
    float* const join = reinterpret_cast<float*>(raw);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kFull, l[h], 1);
      l[h] += __shfl_xor_sync(kFull, l[h], 2);
      if (quad == 0) {
        most[warp][g + 8 * h] = m[h];
        weight[warp][g + 8 * h] = l[h];
      }
      float* row = join + (warp * kRows + g + 8 * h) * D;
      constexpr int kPiece = S::kValuePiece * 8 / BITS;    // elements
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) row[(8 * (c / kPiece) + 2 * quad + e) * kPiece + c % kPiece] = sums[c][2 * h + e];
    }
    __syncthreads();
    float* const part = slot_at(a, gridDim.x, slot_of(walk, range), kRows, D);
    for (int n = tid; n < u.rows * (D / 4); n += kThreads) {
      const int r = n / (D / 4), d = n % (D / 4) * 4;
      float top = most[0][r], sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, most[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_of(most[w][r] - top);
        const float4 four = *reinterpret_cast<const float4*>(join + (w * kRows + r) * D + d);
        sum = fmaf(weight[w][r], f, sum);
        v[0] = fmaf(four.x, f, v[0]);
        v[1] = fmaf(four.y, f, v[1]);
        v[2] = fmaf(four.z, f, v[2]);
        v[3] = fmaf(four.w, f, v[3]);
      }
      if (whole) {
        const int row = u.first + r, token = s.row + row / a.group, head = u.head * a.group + row % a.group;
        const float per = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= per;
        store_values4(a, token * a.out.ld + head * a.out.head_stride + d, v, vector_out);
        if (a.lse && d == 0) a.lse[(int64_t)token * a.heads + head] = sum == 0.0f ? kNone : (top + log2_of(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = make_float4(v[0], v[1], v[2], v[3]);
        if (d == 0) {
          part[kRows * D + r] = top;
          part[kRows * D + kRows + r] = sum;
        }
      }
    }
    if (!whole && walk.in == 0 && tid == 0) name_parts(a, walk, range);
  }
  if (bad) report(bad);
}

// Joins the parts of the units that several blocks have had: a block for each
// block of the first kernel, by four rows.
__global__ void __launch_bounds__(128) attention_join_kernel(const AttentionArgs a, const int blocks, const int rows,
                                                             const int vector_out) {
  pdl_wait();
  pdl_trigger();
  const Join j = joins(a)[blockIdx.x];
  if (j.blocks == 0) return;
  const int dim = a.cache.head_dim;
  for (int n = blockIdx.y * 128 + threadIdx.x; n < j.rows * (dim / 4); n += 128 * gridDim.y) {
    const int r = n / (dim / 4), d = n % (dim / 4) * 4;
    float top = kLowest, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int b = 0; b < j.blocks; ++b) {
      const int slot = b == 0 ? j.slot : 2 * ((int)blockIdx.x + b);
      const float* part = slot_at(a, blocks, slot, rows, dim);
      const float m = part[rows * dim + r], l = part[rows * dim + rows + r];
      const float4 four = *reinterpret_cast<const float4*>(part + r * dim + d);
      const float t = fmaxf(top, m), f0 = exp2_of(top - t), f1 = exp2_of(m - t);
      sum = fmaf(l, f1, sum * f0);
      v[0] = fmaf(four.x, f1, v[0] * f0);
      v[1] = fmaf(four.y, f1, v[1] * f0);
      v[2] = fmaf(four.z, f1, v[2] * f0);
      v[3] = fmaf(four.w, f1, v[3] * f0);
      top = t;
    }
    const int row = j.first + r, token = j.row + row / a.group, head = j.head * a.group + row % a.group;
    const float per = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= per;
    store_values4(a, token * a.out.ld + head * a.out.head_stride + d, v, vector_out);
    if (a.lse && d == 0) a.lse[(int64_t)token * a.heads + head] = sum == 0.0f ? kNone : (top + log2_of(sum)) * kLn2;
  }
}

// Up to as many rows a sequence this kernel runs, for more attn_many.cu's.
constexpr int64_t kFewRows = 64;

template <int D, int BITS>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t s) {
  using S = Shape<D, BITS>;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(attention_few_kernel<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int blocks = few_blocks<D>() * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  const cudaError_t e2 = cudaLaunchKernelEx(&cfg, attention_few_kernel<D, BITS>, a, (int)vector_rows(a.out));
  return e2 != cudaSuccess ? e2 : launch_join(a, blocks, kRows, s);
}

}  // namespace

cudaError_t launch_join(const AttentionArgs& a, int blocks, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)(rows / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel, a, blocks, rows, (int)vector_rows(a.out));
}

cudaError_t launch_attention(const AttentionArgs& a, int sms, cudaStream_t s) {
  // Rows of an average sequence; which kernel runs changes no result beyond rounding.
  const int64_t rows = (int64_t)a.batch.tokens * a.group / a.batch.sequences;
  if (rows > kFewRows) return launch_attention_many(a, sms, s);
  const bool four = a.cache.bits == 4;
  if (a.cache.head_dim == 64) return four ? launch<64, 4>(a, sms, s) : launch<64, 8>(a, sms, s);
  if (a.cache.head_dim == 128) return four ? launch<128, 4>(a, sms, s) : launch<128, 8>(a, sms, s);
  return four ? launch<256, 4>(a, sms, s) : launch<256, 8>(a, sms, s);
}
int64_t attention_bytes(int head_dim, int sms) {
  const int64_t few = workspace_bytes((head_dim == 256 ? few_blocks<256>() : few_blocks<128>()) * sms, kRows, head_dim), many = attention_many_bytes(head_dim, sms);
  return few > many ? few : many;
}
StatusWord attn_few_status() { return {read_status, clear_status_bits}; }

}  // namespace echo
