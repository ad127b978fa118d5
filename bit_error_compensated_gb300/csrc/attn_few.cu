// attn_few.cu -- echo_attention for few rows a sequence (include/echo.h):
// decode, drafted tokens.
//
// Every key is read once for 8 to 48 rows, so the kernel streams codes:
// each warp copies 32 keys and values at a time into a ring of its own
// (asynchronous copies, no barrier between warps) and feeds them to matrix
// instructions whose 16 rows are keys, or columns of the values, and whose 8
// columns are rows of queries:
//     S^T[keys][rows] = K Q^T,    O^T[columns][rows] += V^T P^T
// (the other way round half of an instruction is idle where a head of the cache
// serves 8 queries or fewer).  A code c behind the bits of 1024 is the f16
// number 1024 + c (of 4 bits at bit 4: 1024 + 16 c), from which one instruction
// for two codes takes c - z, exactly.  (f16 holds c * 2^-24 as it stands, as a
// subnormal, but the matrix instructions align their sums by exponents that leave
// such a number 14 bits.)  A key's step is multiplied into its score in fp32; of a
// value's its power of two goes into the value and the rest, 1 to 2, into the
// weight, which is f16 below a bound on its row (attn_common.h).
//
// Blocks take equal shares of the batch's tiles (attn_common.h); four warps
// take a tile's keys and join at the unit's end, and parts of units that several
// blocks have had are joined by a second kernel.
//
// One GB300, 32 heads to 8 of 128, GPU time a call: 64 ragged sequences up to
// 16384, 4 bits, in 164 us (4.1 TB/s: bound by the instructions that turn
// codes), 4 x 131072 of 8 bits in 180 (6.2 TB/s: memory); one token over 2000
// keys in 10, 131000 in 47.
#include "attn_common.h"

namespace echo {
namespace {

ECHO_STATUS_WORD

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kLeast = 1;                // tiles of a block
constexpr int kAhead = 4;                // (8 is no faster)

// NR: eights of rows.
template <int D, int BITS, int NR>
struct Few {
  static constexpr int kRows = 8 * NR;
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kStep = kRowBytes >= 256 ? 16 : 32;                 // keys of a warp at once
  static constexpr int kTile = kStep * kWarps;
  static constexpr int kStage = 2 * kStep * kRowBytes + 2 * kStep * 4;     // keys, values, meta of both
  static constexpr int kStages = kRowBytes >= 128 ? 2 : 3;
  static constexpr int kPairBytes = BITS == 4 ? 16 : 8;  // of what turns the codes of two values
  static constexpr int kSteps = kStep * 8 + kStep / 2 * kPairBytes;        // a warp's, see prepare_values
  static constexpr int kRing = kWarps * (kStages * kStage + kSteps);
  static constexpr int kPitch = D + 4;                   // floats from row to row of the warps' sums
  static constexpr int kJoin = kWarps * kRows * kPitch * 4;                // which take the ring's place
  static constexpr int kQuery = D / 16 * NR * 32 * 8;    // rows as the instructions' operands
  static constexpr int kBytes = (kRing > kJoin ? kRing : kJoin) + kQuery;
  static constexpr int kKeyPiece = kRowBytes / 4 < 16 ? kRowBytes / 4 : 16;      // bytes a thread takes at once
  static constexpr int kValuePiece = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;
  static constexpr int kPerWord = 32 / BITS;
  // Blocks an SM: what registers (sums take D * NR / 4 a thread) and shared memory allow.
  static constexpr int kByRegs = D * NR <= 128 ? 4 : D * NR <= 256 ? 3 : 2, kBySmem = 227 * 1024 / (kBytes + 1152 + 44 * kRows);
  static constexpr int kBlocks = kByRegs < kBySmem ? kByRegs : kBySmem;
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
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
// 8 x 8 halves, a lane's two in row lane / 4, with rows and columns exchanged.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {         // a in the low half
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes less their zero points as pairs of f16: of a key, `low` is 1024 + z,
// `high` - 64 - z, twice; of two values, - (1024 + z) S and - (64 + z) S.
struct Zero {
  uint32_t low, high, base;              // base: 1024, twice
};
struct ScaledZero {
  uint32_t low, scale, high, high_scale; // scale: S, high_scale: S / 16
  uint32_t base;
};
__device__ __forceinline__ Zero zero_of(uint32_t zs, uint32_t base) {     // two fp16 zero points
  const __half2 z = *reinterpret_cast<const __half2*>(&zs);
  const __half2 low = __hadd2(z, __float2half2_rn(1024.0f)), high = __hneg2(__hadd2(z, __float2half2_rn(64.0f)));
  return {*reinterpret_cast<const uint32_t*>(&low), *reinterpret_cast<const uint32_t*>(&high), base};
}
__device__ __forceinline__ uint32_t scaled_sum(uint32_t v, uint32_t scale, uint32_t z) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&scale),
                            *reinterpret_cast<const __half2*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t less_low(uint32_t v, const ScaledZero& z) { return scaled_sum(v, z.scale, z.low); }
__device__ __forceinline__ uint32_t less_high(uint32_t v, const ScaledZero& z) { return scaled_sum(v, z.high_scale, z.high); }
__device__ __forceinline__ uint32_t less_low(uint32_t v, const Zero& z) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&z.low));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t less_high(uint32_t v, const Zero& z) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f),
                            *reinterpret_cast<const __half2*>(&z.high));
  return *reinterpret_cast<const uint32_t*>(&d);
}
template <typename Z>
__device__ __forceinline__ uint32_t low_codes(uint32_t w, const Z& z) {           // at bits 0 and 16
  return less_low(masked<0x000F000Fu>(w, z.base), z);
}
template <typename Z>
__device__ __forceinline__ uint32_t high_codes(uint32_t w, const Z& z) {          // at bits 4 and 20
  return less_high(masked<0x00F000F0u>(w, z.base), z);
}
template <typename Z>
__device__ __forceinline__ uint32_t byte_codes(uint32_t w, uint32_t bytes, const Z& z) {
  return less_low(__byte_perm(w, z.base, bytes), z);
}

// What a step's values are turned and weighted with, found once by the lane of
// each value for all that need it: at `to`, log2 f and 1 / f of each (its weight
// adds 0 to the sum of weights where no key is, or where f is NaN: whatever lies
// there must not meet a weight of 0, nor may a NaN that a row does not see reach
// its sum), then of each two a ScaledZero.
template <typename S, int BITS>
__device__ __forceinline__ void prepare_values(uint32_t metas, uint32_t to, bool there) {
  const int lane = threadIdx.x & 31;
  if (S::kStep == 32 || lane < S::kStep) {
    uint32_t meta;
    load_words<4>(metas + 4 * lane, &meta);
    if (!there) meta = 0;
    const float f = value_factor(meta), log = log2_of(f), per = there && f == f ? reciprocal(f) : 0.0f;
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" :: "r"(to + 8 * lane), "f"(log), "f"(per) : "memory");
    const uint32_t scale = value_scale(meta), scales = __byte_perm(scale, scale, 0x1010), zs = __byte_perm(meta, meta, 0x3232);
    const __half2 zero = __hmul2(__hsub2(__floats2half2_rn(-1024.0f, -64.0f), *reinterpret_cast<const __half2*>(&zs)),
                                 *reinterpret_cast<const __half2*>(&scales));
    const uint32_t zeros = *reinterpret_cast<const uint32_t*>(&zero), at = to + 8 * S::kStep + S::kPairBytes * (lane >> 1) + 2 * (lane & 1);
    asm volatile("st.shared.b16 [%0], %1;" :: "r"(at), "h"((unsigned short)zeros) : "memory");
    asm volatile("st.shared.b16 [%0], %1;" :: "r"(at + 4), "h"((unsigned short)scale) : "memory");
    if constexpr (BITS == 4) {
      const __half sixteenth = __hmul(__ushort_as_half((unsigned short)scale), __float2half_rn(0.0625f));
      asm volatile("st.shared.b16 [%0], %1;" :: "r"(at + 8), "h"((unsigned short)(zeros >> 16)) : "memory");
      asm volatile("st.shared.b16 [%0], %1;" :: "r"(at + 12), "h"(__half_as_ushort(sixteenth)) : "memory");
    }
  }
  __syncwarp();
}

// Loads the unit's rows as operands: for each matrix instruction, eight of rows
// and lane, its two registers.  Element e of a row meets the code that the lane
// of its quarter finds at the same place of its words.  The rows' factors go to
// shared memory (NaN for a row with a non-finite element).
template <typename T, int D, int BITS, int NR>
__device__ __forceinline__ void load_queries(const AttentionArgs& a, const Sequence& s, const Unit& u, uint8_t* query,
                                             float* factor) {
  using S = Few<D, BITS, NR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 2
  for (int i = 0; i < S::kRows / kWarps; ++i) {
    const int r = warp * (S::kRows / kWarps) + i, row = u.first + r;
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
      const int at = ((instruction * NR + (r >> 3)) * 32 + (r & 7) * 4 + quad) * 8 + 4 * second + 2 * half;
      *reinterpret_cast<__half*>(query + at) = __float2half_rn(v[k] * f);
    }
    if (lane == 0) factor[r] = top < 0x7F800000u ? a.scale * kLog2E / f : __int_as_float(0x7FC00000);
  }
}

template <int D, int BITS, int NR>
__global__ void __launch_bounds__(kThreads, (Few<D, BITS, NR>::kBlocks)) attention_few_kernel(const AttentionArgs a, const int vector_out) {
  using S = Few<D, BITS, NR>;
  constexpr int kRows = S::kRows, kStep = S::kStep, kTile = S::kTile, kSubs = kStep / 16;
  constexpr int kPairs = D / 16;                           // of columns that a thread has of O^T
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ int64_t shared[2 * kWarps + 3];
  __shared__ float factor[kRows], most[kWarps][kRows], weight[kWarps][kRows];
  __shared__ int2 seen[kRows];                             // keys [x, y) that a row sees
  uint8_t* const query = raw + (S::kBytes - S::kQuery);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, quad = lane & 3;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(raw) + warp * S::kStages * S::kStage;
  const uint32_t steps = (uint32_t)__cvta_generic_to_shared(raw) + kWarps * S::kStages * S::kStage + warp * S::kSteps;
  const uint32_t base1024 = unknown(0x64006400u);
  pdl_wait();
  pdl_trigger();
  if (tid == 0) joins(a)[blockIdx.x].blocks = 0;
  int bad = 0;
  const Range range = block_range<kRows, kTile, kThreads, kLeast>(a, shared, &bad);
  const int heads = a.cache.heads, page_size = 1 << a.cache.page_shift;
  Walk<kRows, kTile> walk;
  for (walk.start(a, range); walk.more(); walk.next(a, &bad)) {
    const Sequence& s = walk.s;
    const Unit& u = walk.unit;
    const int tiles = walk.take;
    const bool whole = walk.whole();

    __syncthreads();                                       // the last unit's sums have been read
    // Keys that all rows see, and where the last that any sees ends.
    const int first_place = s.place + u.first / a.group, last_place = s.place + (u.first + u.rows - 1) / a.group;
    const int all_to = keys_to(a, s, first_place), all_from = keys_from(a, last_place), end = keys_to(a, s, last_place);
    const int key0 = (u.tile + walk.in) * kTile + kStep * warp;            // of this warp's first step
    const int64_t values_on = (int64_t)heads << a.cache.page_shift;        // groups from a key's to its value's
    uint32_t missing = 0;                                  // 16 keys of a stage without a page, a bit each
    // The pages of a step's sixteens of keys (the same one where a page is larger),
    // as the table has them: what is there is looked at a step later, since a use
    // right away would wait for it.  Pages wholly behind the rows' window (`from` in the
    // first tile, 0 past it) may be gone.
    auto wanted = [&](int t, int key, int from) { return t < tiles && key < end && key + 16 > from; };
    struct Pages {
      int of[kSubs];
    };
    auto look_up = [&](int t, int from) {
      Pages p;
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub) {
        const int key = key0 + t * kTile + 16 * sub;
        const int at = key >> a.cache.page_shift;
        p.of[sub] = -1;
        if (wanted(t, key, from) && at < a.batch.table_pages)
          p.of[sub] = a.batch.table[(int64_t)u.sequence * a.batch.ld_table + at];
      }
      return p;
    };
    auto issue = [&](int t, const Pages& pages, int stage, int from) {
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub) {
        const int key = key0 + t * kTile + 16 * sub, page = pages.of[sub];
        const uint32_t bit = 1u << (stage * kSubs + sub);
        missing &= ~bit;
        if (page >= 0 && page < a.cache.pages) {
          const int64_t group = group_index(a.cache, page, u.head, key & (page_size - 1));
          const uint8_t* codes = a.cache.codes + group * S::kRowBytes + 16 * lane;
          const uint8_t* value_codes = codes + values_on * S::kRowBytes;
          const uint32_t base = ring + stage * S::kStage + sub * 16 * S::kRowBytes;
          constexpr int kPieces = S::kRowBytes / 16;       // of a row; 16 rows have 32 lanes' worth of them or more
#pragma unroll
          for (int n = 0; n < kPieces * 16 / 32; ++n) {
            const int piece = lane + 32 * n, r = piece / kPieces, p = piece % kPieces;
            copy16_async(base + key_at<S::kRowBytes>(r, p), codes + 512 * n);
            copy16_async(base + kStep * S::kRowBytes + value_at<S::kRowBytes>(value_row(r), p), value_codes + 512 * n);
          }
          if (lane < 8)
            copy16_async(ring + stage * S::kStage + 2 * kStep * S::kRowBytes + (lane < 4 ? 0 : 4 * kStep) + 64 * sub + 16 * (lane & 3),
                         a.cache.meta + group + (lane < 4 ? 0 : values_on) + 4 * (lane & 3));
        } else {
          missing |= bit;
          if (wanted(t, key, from)) bad |= kBadPage;
        }
      }
      copies_commit();
    };
    // (the first copies are under way before the rows are loaded)
    const int from = keys_from(a, first_place);
    Pages pages = look_up(0, from);
#pragma unroll 1
    for (int t = 0; t < S::kStages - 1; ++t) {
      issue(t, pages, t, t == 0 ? from : 0);
      pages = look_up(t + 1, 0);
    }
    if (a.dtype == ECHO_BF16) load_queries<__nv_bfloat16, D, BITS, NR>(a, s, u, query, factor);
    else load_queries<__half, D, BITS, NR>(a, s, u, query, factor);
    if (tid < kRows) {
      const int place = s.place + (u.first + tid) / a.group;
      // (rows past the last see all, so that they ask for nothing by themselves)
      seen[tid] = tid < u.rows ? make_int2(keys_from(a, place), keys_to(a, s, place)) : make_int2(0, 0x7FFFFFFF);
    }
    __syncthreads();
    float row_scale[NR][2];                                // of rows 8 o + 2 quad and the next
#pragma unroll
    for (int o = 0; o < NR; ++o)
#pragma unroll
      for (int e = 0; e < 2; ++e) row_scale[o][e] = factor[8 * o + 2 * quad + e];
    uint2 held[NR == 1 ? D / 16 : 1];                      // one eight of rows stays in registers
    if constexpr (NR == 1) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) held[k] = reinterpret_cast<const uint2*>(query)[k * 32 + lane];
    }

    float sums[kPairs][NR][4], m[NR][2], l[NR][2];
#pragma unroll
    for (int o = 0; o < NR; ++o) {
#pragma unroll
      for (int c = 0; c < kPairs; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) sums[c][o][k] = 0.0f;
      m[o][0] = m[o][1] = kLowest;
      l[o][0] = l[o][1] = 0.0f;
    }

    int stage = 0, ahead = S::kStages - 1;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int key = key0 + t * kTile;
      copies_wait<S::kStages - 2>();
      __syncwarp();
      const uint32_t absent = missing >> (stage * kSubs) & ((1u << kSubs) - 1);
      if (key < end && absent != (1u << kSubs) - 1) {      // the whole warp
        const uint32_t base = ring + stage * S::kStage, meta = base + 2 * kStep * S::kRowBytes;
        prepare_values<S, BITS>(meta + 4 * kStep, steps, key + lane < end && !(absent >> (lane >> 4) & 1));
        // S^T of keys 16 sub + g (+ 8) and rows 8 o + 2 quad (+ 1).
        float scores[kSubs][NR][4];
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int o = 0; o < NR; ++o)
#pragma unroll
            for (int k = 0; k < 4; ++k) scores[sub][o][k] = 0.0f;
        uint32_t kmeta[kSubs][2];
        Zero z[kSubs][2];
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            load_words<4>(meta + (16 * sub + 8 * h + g) * 4, &kmeta[sub][h]);
            z[sub][h] = zero_of(__byte_perm(kmeta[sub][h], kmeta[sub][h], 0x3232), base1024);
          }
        {
          constexpr int kPieceWords = S::kKeyPiece / 4, kPieces = S::kRowBytes / (4 * S::kKeyPiece);
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
            const int byte = (4 * p + quad) * S::kKeyPiece;
            uint32_t w[kSubs][2][kPieceWords];
#pragma unroll
            for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                load_words<S::kKeyPiece>(base + key_at<S::kRowBytes>(16 * sub + 8 * h + g, byte / 16) + byte % 16, w[sub][h]);
#pragma unroll
            for (int k = 0; k < kPieceWords; ++k)
#pragma unroll
              for (int part = 0; part < (BITS == 4 ? 2 : 1); ++part) {
                const int instruction = BITS == 4 ? 2 * (p * kPieceWords + k) + part : p * kPieceWords + k;
                uint2 q[NR];
#pragma unroll
                for (int o = 0; o < NR; ++o) {
                  if constexpr (NR == 1) q[o] = held[instruction];
                  else q[o] = reinterpret_cast<const uint2*>(query)[(instruction * NR + o) * 32 + lane];
                }
#pragma unroll
                for (int sub = 0; sub < kSubs; ++sub) {
                  uint32_t c[2][2];                        // of key g, g + 8: first and second pair
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t v = w[sub][h][k];
                    if constexpr (BITS == 4) {
                      c[h][0] = low_codes(part ? v >> 8 : v, z[sub][h]);
                      c[h][1] = high_codes(part ? v >> 8 : v, z[sub][h]);
                    } else {
                      c[h][0] = byte_codes(v, 0x5150, z[sub][h]);
                      c[h][1] = byte_codes(v, 0x5352, z[sub][h]);
                    }
                  }
#pragma unroll
                  for (int o = 0; o < NR; ++o) mma_f16(scores[sub][o], c[0][0], c[1][0], c[0][1], c[1][1], q[o].x, q[o].y);
                }
              }
          }
        }
        const bool inside = key >= all_from && key + kStep <= all_to && absent == 0;     // every row sees all
        float per[kSubs][2];                               // 1 / f of the values
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t two[2];
            load_words<8>(steps + 8 * (16 * sub + 8 * h + g), two);
            const float ks = meta_step(kmeta[sub][h]), log = __uint_as_float(two[0]);
            per[sub][h] = __uint_as_float(two[1]);
#pragma unroll
            for (int o = 0; o < NR; ++o) {
              float &s0 = scores[sub][o][2 * h], &s1 = scores[sub][o][2 * h + 1];
              mul2(s0, s1, s0, s1, row_scale[o][0], row_scale[o][1]);
              fma2(s0, s1, s0, s1, ks, ks, log, log);
            }
          }
        if (!inside) {
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = key + 16 * sub + 8 * h + g;
              const bool there = k < end && !(absent >> sub & 1);
#pragma unroll
              for (int o = 0; o < NR; ++o)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int2 see = seen[8 * o + 2 * quad + e];
                  if (!there || k < see.x || k >= see.y) scores[sub][o][2 * h + e] = kNone;
                }
            }
        }
        // The maxima, where a score has passed them by far.
        float top[NR][2];
        bool passed = false;
#pragma unroll
        for (int o = 0; o < NR; ++o)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[o][e] = m[o][e];
#pragma unroll
            for (int sub = 0; sub < kSubs; ++sub) top[o][e] = max3(top[o][e], scores[sub][o][e], scores[sub][o][2 + e]);
            passed |= top[o][e] - m[o][e] > kMostWeight;
          }
        if (__any_sync(kFull, passed)) {
#pragma unroll
          for (int o = 0; o < NR; ++o) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = top[o][e];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
              v = raised<kAhead>(m[o][e], v);
              top[o][e] = exp2_of(m[o][e] - v);
              m[o][e] = v;
              l[o][e] *= top[o][e];
            }
#pragma unroll
            for (int c = 0; c < kPairs; ++c) {
              mul2(sums[c][o][0], sums[c][o][1], sums[c][o][0], sums[c][o][1], top[o][0], top[o][1]);
              mul2(sums[c][o][2], sums[c][o][3], sums[c][o][2], sums[c][o][3], top[o][0], top[o][1]);
            }
          }
        }
        uint32_t p[kSubs][NR][2];                          // P^T as operands: keys 2 quad (+ 1) of each eight, row g
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int o = 0; o < NR; ++o)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float p0 = scores[sub][o][2 * h], p1 = scores[sub][o][2 * h + 1];
              sub2(p0, p1, p0, p1, m[o][0], m[o][1]);
              p0 = exp2_of(p0);
              p1 = exp2_of(p1);
              fma2(l[o][0], l[o][1], p0, p1, per[sub][h], per[sub][h], l[o][0], l[o][1]);
              p[sub][o][h] = pack_f16(p0, p1);
            }
        __syncwarp();                                      // hidden keys part the lanes; matrix instructions want them together
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
          for (int o = 0; o < NR; ++o)
#pragma unroll
            for (int h = 0; h < 2; ++h) p[sub][o][h] = transposed(p[sub][o][h]);
        // Values: a lane has its piece of every eighth of a row; pairs of keys side by side.
        constexpr int kPieceWords = S::kValuePiece / 4, kPieces = S::kRowBytes / (8 * S::kValuePiece);
        const uint32_t values = base + kStep * S::kRowBytes;
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) {
          ScaledZero zv[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t found[S::kPairBytes / 4];
            load_words<S::kPairBytes>(steps + 8 * kStep + S::kPairBytes * (8 * sub + 4 * h + quad), found);
            zv[h].low = found[0];
            zv[h].scale = found[1];
            if constexpr (BITS == 4) {
              zv[h].high = found[2];
              zv[h].high_scale = found[3];
            }
            zv[h].base = base1024;
          }
#pragma unroll
          for (int piece = 0; piece < kPieces; ++piece) {
            const int byte = (8 * piece + g) * S::kValuePiece;
            uint32_t w[4][kPieceWords];                    // keys 2 quad, 2 quad + 1, and 8 on
#pragma unroll
            for (int k = 0; k < 4; ++k)
              load_words<S::kValuePiece>(
                  values + value_at<S::kRowBytes>(16 * sub + 8 * (k >> 1) + 4 * (k & 1) + quad, byte / 16) + byte % 16, w[k]);
#pragma unroll
            for (int k = 0; k < kPieceWords; ++k)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t x = __byte_perm(w[0][k], w[1][k], half ? 0x7632 : 0x5410);
                const uint32_t y = __byte_perm(w[2][k], w[3][k], half ? 0x7632 : 0x5410);
                const int pair = (piece * kPieceWords + k) * (S::kPerWord / 2) + (BITS == 4 ? 2 * half : half);
                auto add = [&](int at, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                  for (int o = 0; o < NR; ++o) mma_f16(sums[at][o], a0, a1, a2, a3, p[sub][o][0], p[sub][o][1]);
                };
                if constexpr (BITS == 4) {
                  add(pair, low_codes(x, zv[0]), high_codes(x, zv[0]), low_codes(y, zv[1]), high_codes(y, zv[1]));
                  add(pair + 1, low_codes(x >> 8, zv[0]), high_codes(x >> 8, zv[0]), low_codes(y >> 8, zv[1]),
                      high_codes(y >> 8, zv[1]));
                } else {
                  add(pair, byte_codes(x, 0x5250, zv[0]), byte_codes(x, 0x5351, zv[0]), byte_codes(y, 0x5250, zv[1]),
                      byte_codes(y, 0x5351, zv[1]));
                }
              }
          }
        }
      }
      __syncwarp();                                        // before the stage is overwritten
      const Pages next = look_up(t + S::kStages, 0);
      issue(t + S::kStages - 1, pages, ahead, 0);
      pages = next;
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
      ahead = ahead + 1 == S::kStages ? 0 : ahead + 1;
    }
    copies_wait<0>();
    __syncthreads();                                       // the rings are free

    // The warps' sums.
    float* const join = reinterpret_cast<float*>(raw);
#pragma unroll
    for (int o = 0; o < NR; ++o)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * o + 2 * quad + e;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[o][e] += __shfl_xor_sync(kFull, l[o][e], off);
        if (g == 0) {
          most[warp][r] = m[o][e];
          weight[warp][r] = l[o][e];
        }
        float* row = join + (warp * kRows + r) * S::kPitch;
        constexpr int kPiece = S::kValuePiece * 8 / BITS;  // elements
#pragma unroll
        for (int c = 0; c < kPairs; ++c)
          *reinterpret_cast<float2*>(row + (8 * (2 * c / kPiece) + g) * kPiece + 2 * c % kPiece) =
              make_float2(sums[c][o][e], sums[c][o][2 + e]);
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
        const float4 four = *reinterpret_cast<const float4*>(join + (w * kRows + r) * S::kPitch + d);
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

// Joins the parts of the units that several blocks have had: blocks for each
// block of the first kernel, which take the unit's rows in turn.  DIM / 4 threads
// take a row's parts; where these are many, several such groups share them (one
// after the other, the 76 parts of 32000 keys took 20 us), where they are few,
// the groups take rows.
constexpr int kJoiners = 256;
template <int DIM>
__global__ void __launch_bounds__(kJoiners) attention_join_kernel(const AttentionArgs a, const int blocks, const int rows,
                                                                  const int vector_out) {
  constexpr int kWide = DIM / 4, kGroups = kJoiners / kWide;
  __shared__ float4 sums[kGroups][kWide];
  __shared__ float most[kGroups], weight[kGroups];
  pdl_wait();
  pdl_trigger();
  const Join j = joins(a)[blockIdx.x];
  if (j.blocks == 0) return;
  const int lane = threadIdx.x % kWide, group = threadIdx.x / kWide;
  const int wanted = j.blocks >= 16 ? 8 : j.blocks >= 6 ? 4 : 1, share = wanted < kGroups ? wanted : kGroups;
  const int step = kGroups / share, mine = group % share;  // rows at once; this group's number among its row's
  for (int r0 = blockIdx.y * step; r0 < j.rows; r0 += gridDim.y * step) {
    const int r = r0 + group / share;
    float top = kLowest, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto join = [&](float m, float l, const float4& w) {
      const float t = fmaxf(top, m), f0 = exp2_of(top - t), f1 = exp2_of(m - t);
      sum = fmaf(l, f1, sum * f0);
      v.x = fmaf(w.x, f1, v.x * f0);
      v.y = fmaf(w.y, f1, v.y * f0);
      v.z = fmaf(w.z, f1, v.z * f0);
      v.w = fmaf(w.w, f1, v.w * f0);
      top = t;
    };
    if (r < j.rows)
#pragma unroll 4
      for (int b = mine; b < j.blocks; b += share) {
        const float* part = slot_at(a, blocks, b == 0 ? j.slot : 2 * ((int)blockIdx.x + b), rows, DIM);
        join(part[rows * DIM + r], part[rows * DIM + rows + r], reinterpret_cast<const float4*>(part + r * DIM)[lane]);
      }
    if (share > 1) {                                       // the whole block
      __syncthreads();                                     // the row before has been read
      sums[group][lane] = v;
      if (lane == 0) {
        most[group] = top;
        weight[group] = sum;
      }
      __syncthreads();
      if (mine != 0) continue;
      for (int g = group + 1; g < group + share; ++g) join(most[g], weight[g], sums[g][lane]);
    }
    if (r >= j.rows) continue;
    const int row = j.first + r, token = j.row + row / a.group, head = j.head * a.group + row % a.group;
    const float per = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float out[4] = {v.x * per, v.y * per, v.z * per, v.w * per};
    store_values4(a, token * a.out.ld + head * a.out.head_stride + 4 * lane, out, vector_out);
    if (a.lse && lane == 0) a.lse[(int64_t)token * a.heads + head] = sum == 0.0f ? kNone : (top + log2_of(sum)) * kLn2;
  }
}

template <int D, int BITS, int NR>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t s) {
  using S = Few<D, BITS, NR>;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(attention_few_kernel<D, BITS, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int blocks = useful_blocks(a, S::kRows, S::kTile, S::kBlocks * sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  const cudaError_t e2 = cudaLaunchKernelEx(&cfg, attention_few_kernel<D, BITS, NR>, a, (int)vector_rows(a.out));
  return e2 != cudaSuccess ? e2 : launch_join(a, blocks, S::kRows, s);
}
template <int D, int NR>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t s) {
  return a.cache.bits == 4 ? launch<D, 4, NR>(a, sms, s) : launch<D, 8, NR>(a, sms, s);
}
// How many eights of rows a unit has: a unit's keys cost about as much as four
// eights do by themselves, so the fewest of units * (4 + eights), among what
// registers hold.  (16 sequences of 8000 keys, 8 heads, 4 bits, one unit of 2, 3 and
// 4 eights of rows of 128: 65, 76 and 92 us; of 2 to 6 eights of rows of 64: 49, 55,
// 70, 76 and 88; of 128 two units of 3 and of 4: 121 and 147.)
template <int D>
int eights(int64_t rows) {
  constexpr int kMost = D == 64 ? 6 : D == 128 ? 4 : 2;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMost; ++n) {
    const int64_t cost = (rows + 8 * n - 1) / (8 * n) * (4 + n);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}
template <int D>
cudaError_t launch(const AttentionArgs& a, int64_t rows, int sms, cudaStream_t s) {
  switch (eights<D>(rows)) {
    case 1: return launch<D, 1>(a, sms, s);
    case 2: return launch<D, 2>(a, sms, s);
    case 3: return launch<D, D <= 128 ? 3 : 2>(a, sms, s);
    case 4: return launch<D, D <= 128 ? 4 : 2>(a, sms, s);
    case 5: return launch<D, D <= 64 ? 5 : 2>(a, sms, s);
    default: return launch<D, D <= 64 ? 6 : 2>(a, sms, s);
  }
}
template <int D, int NR>
int64_t bytes(int sms) {
  constexpr int kMost = Few<D, 4, NR>::kBlocks > Few<D, 8, NR>::kBlocks ? Few<D, 4, NR>::kBlocks : Few<D, 8, NR>::kBlocks;
  return workspace_bytes(kMost * sms, 8 * NR, D);
}
template <int D>
int64_t bytes(int sms) {
  int64_t most = 0;
  for (int64_t n : {bytes<D, 1>(sms), bytes<D, 2>(sms), bytes<D, D <= 128 ? 3 : 2>(sms), bytes<D, D <= 128 ? 4 : 2>(sms),
                    bytes<D, D <= 64 ? 5 : 2>(sms), bytes<D, D <= 64 ? 6 : 2>(sms)})
    most = n > most ? n : most;
  return most;
}

}  // namespace

cudaError_t launch_join(const AttentionArgs& a, int blocks, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // (most of these find nothing to join: more of them, and they take as long as the joining)
  cfg.gridDim = dim3((unsigned)blocks, rows <= 32 ? 4 : 16);
  cfg.blockDim = dim3(kJoiners);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  const int vector = vector_rows(a.out);
  if (a.cache.head_dim == 64) return cudaLaunchKernelEx(&cfg, attention_join_kernel<64>, a, blocks, rows, vector);
  if (a.cache.head_dim == 128) return cudaLaunchKernelEx(&cfg, attention_join_kernel<128>, a, blocks, rows, vector);
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<256>, a, blocks, rows, vector);
}

// Up to as many rows a sequence this file's kernels run, for more attn_many.cu's.
// 16 sequences of 8000 keys, 4 bits, here and there: 64 rows of 64 107 and 157 us, 96
// 135 and 158, 128 193 and 160; of 128 147 and 176, 219 and 178, 270 and 180; of 256
// (4 heads; 48 rows 141 and 158) 176 and 158, 254 and 160, 322 and 166.
constexpr int64_t kFewRows = 64;

cudaError_t launch_attention(const AttentionArgs& a, int sms, cudaStream_t s) {
  // Rows of an average sequence, rounded up; which kernel runs changes no result beyond rounding.
  const int64_t rows = ((int64_t)a.batch.tokens * a.group + a.batch.sequences - 1) / a.batch.sequences;
  if (rows > kFewRows) return launch_attention_many(a, sms, s);
  if (a.cache.head_dim == 64) return launch<64>(a, rows, sms, s);
  if (a.cache.head_dim == 128) return launch<128>(a, rows, sms, s);
  return launch<256>(a, rows, sms, s);
}
int64_t attention_bytes(int head_dim, int sms) {
  const int64_t few = head_dim == 64 ? bytes<64>(sms) : head_dim == 128 ? bytes<128>(sms) : bytes<256>(sms);
  const int64_t many = attention_many_bytes(head_dim, sms);
  return few > many ? few : many;
}
StatusWord attn_few_status() { return {read_status, clear_status_bits}; }

}  // namespace echo
