// attn_many.cu -- echo_attention for many rows a sequence (include/echo.h):
// prompts, chunks of them, on the tensor cores.
//
// A block takes NT tiles of 128 rows of queries (two for rows of 64 and 128,
// one of 256) and KT keys at a time.  Scores and sums of values are matrix
// instructions with fp32 sums in TMEM:
//     S[128][KT] = Q K^T        Q and K in shared memory,
//     O[128][D] += P V          P in TMEM, in the place of S, V in shared memory,
// where K and V hold codes less their zero points, exact in f16.  Warps of the
// block:
//   8 a tile of rows   take S out of TMEM, turn scores into weights and put P
//                      back (attn_common.h says what of a value's step is in
//                      the weight and what in the value);
//   4 for the keys, 4 for the values
//                      turn a tile's codes, loaded one tile ahead;
//   1 issues the matrix instructions.
// What a row's weights are scaled by changes only when a score passes the ones
// before by 2^kAhead, so O in TMEM is rescaled a few times a row, and the weights are
// made in one pass over S.  While one tile's weights are made, the tensor cores work for the other (with one tile
// of rows: on the next tile's scores).
//
// A lane has two neighbouring keys of every eight and two rows of the warp's
// 16, so a quarter of the keys' steps are read by each lane, P's pairs go back
// as they are, and a row is one warp's alone.
//
// One GB300: 2048 tokens (32 heads to 8, of 128) over 32768 keys of 4 bits in
// 1217 us, 932 TFLOP/s; a prompt of 8192 in 741 us, 742.  A tile of 256 rows and
// 128 keys takes 5100 cycles, of which the matrix instructions need 2100.  What
// it is nearest to is shared memory: operands take 1536 cycles of it, the
// warps' accesses 3100 (steps 1600, codes turned 570, barriers, and loads of
// codes from L2); issue slots are 59% busy.  Four warps a tile of rows, with four
// rows a lane, load steps half as often and wait longer for each other: when that
// was measured 1172 us (1211), and 107 for a prompt of 2048 (95).
//
// Every wait is bounded; one that gives up ends the call with a status
// (echo_serving_status): the block's other warps leave at their next wait, and
// the issuing one first waits for what it has issued.
#include "attn_common.h"
#include "tensor.cuh"

namespace echo {
namespace {

ECHO_STATUS_WORD

constexpr int kRowTile = 128;
constexpr int kSlots = 4;                               // of steps: tiles whose weights are being made, or are next
// Registers: the block starts with 72 a thread (seven warpgroups of 504 in all).
constexpr int kWarpsWeights = 16, kWarpsKeys = 4, kWarpsValues = 4;
constexpr int kIssuer = kWarpsWeights + kWarpsKeys + kWarpsValues, kThreads = 32 * (kIssuer + 4);
constexpr int kWeightRegs = 88, kTurnRegs = 56, kIssueRegs = 40;
// (4, as attn_few.cu has it for nothing: a prompt of 8192 takes 6% longer, 6: 3%, 7: 1%)
constexpr int kAhead = 8;
static_assert(4 * kWeightRegs + 2 * kTurnRegs + kIssueRegs <= 7 * 72, "a split above the launch's registers never ends");

template <int D, int BITS>
struct Many {
  static constexpr int NT = D == 256 ? 1 : 2;            // tiles of rows
  static constexpr int KT = D == 256 ? 64 : 128;         // keys of a tile
  static constexpr int kRows = NT * kRowTile;
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kQuery = kRowTile * D * 2;        // bytes of a tile of rows
  static constexpr int kStage = KT * D * 2;              // of a tile of keys, or values
  static constexpr int kSteps = 3 * KT * 4;              // keys' steps, values' log steps and reciprocals
  static constexpr int kBytes = NT * kQuery + 4 * kStage + kSlots * kSteps + 1024;
  static constexpr int kSums = NT == 2 ? 256 : 128;      // TMEM column of O; S before it
};

// Values of V for the instruction's B operand: D contiguous, a row a key.  128-
// byte swizzle: 64 elements of eight rows are 1024 bytes, rows' eights follow
// each other, 64 elements on are KT rows on.
template <int KT>
__device__ __forceinline__ uint64_t value_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(KT * 128 / 16) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// One lane issues (`one`), but its warp stays together, and what the
// instructions take is known to be uniform: an instruction whose operands have
// to be moved to uniform registers first takes longer to issue than to run.
__device__ __forceinline__ void mma_shared(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(desc), "r"(add), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(desc), "r"(add), "r"(one) : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      :: "r"(bar), "r"(one) : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(kFull, v); }

// 16 rows x 32 columns of TMEM: v[4 n + k] is row lane / 4 (+ 8 for k >= 2),
// column 8 n + 2 (lane % 4) + k % 2.  (.aligned: hidden keys part the lanes.)
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_loaded(float (&v)[16]) {
  // the registers are inputs and outputs, so that none is used before the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :: "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const float (&v)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
         "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]) : "memory");
}
// 16 rows x 16 columns: w[2 n + k] is row lane / 4 + 8 k, column 4 n + lane % 4.
__device__ __forceinline__ void tmem_store_pairs(uint32_t at, const uint32_t* w) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
      :: "r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
__device__ __forceinline__ void tmem_load_pairs(uint32_t at, uint32_t (&w)[8]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {         // a in the low half
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 shared_pair(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void store_shared16(uint32_t at, const uint32_t (&h)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
}

// The barriers, as offsets from the first one's address.
template <int NT>
struct Bars {
  static constexpr int kQuery = 0;                       // NT tiles of rows are in shared memory
  static constexpr int kKeys = kQuery + 8, kKeysFree = kKeys + 16;
  static constexpr int kValues = kKeysFree + 16, kValuesFree = kValues + 16;
  static constexpr int kSteps = kValuesFree + 16;        // steps of a slot
  static constexpr int kScores = kSteps + 8 * kSlots;    // by tile of rows, or by buffer
  static constexpr int kWeights = kScores + 16;          // the same
  static constexpr int kSums = kWeights + 16;            // a unit's sums are complete, by tile of rows
  static constexpr int kLast = kSums + 16;
  static constexpr int kCount = kLast / 8 + 1;
};

// Eight codes of a word (4 bits) as (0, 4), (1, 5), (2, 6), (3, 7), or of two
// (8 bits) in order, less the zero point, times S (1 for keys).  low: -(1024 + z)
// S, high: -(64 + z) S, scale and high_scale S and S / 16, all twice.
__device__ __forceinline__ uint32_t less(uint32_t v, uint32_t scale, uint32_t z) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&scale),
                            *reinterpret_cast<const __half2*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t times_half(uint32_t a, float b) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void turn4(uint32_t w, uint32_t base, uint32_t scale, uint32_t low, uint32_t high_scale, uint32_t high,
                                      uint32_t (&h)[4]) {
  const uint32_t up = w >> 8;
  h[0] = less(masked<0x000F000Fu>(w, base), scale, low);
  h[1] = less(masked<0x00F000F0u>(w, base), high_scale, high);
  h[2] = less(masked<0x000F000Fu>(up, base), scale, low);
  h[3] = less(masked<0x00F000F0u>(up, base), high_scale, high);
}
__device__ __forceinline__ void turn8(uint32_t a, uint32_t b, uint32_t base, uint32_t scale, uint32_t low, uint32_t (&h)[4]) {
  h[0] = less(__byte_perm(a, base, 0x5150), scale, low);
  h[1] = less(__byte_perm(a, base, 0x5352), scale, low);
  h[2] = less(__byte_perm(b, base, 0x5150), scale, low);
  h[3] = less(__byte_perm(b, base, 0x5352), scale, low);
}
// The rows of tile t of a unit into shared memory, as the A operand (K-major);
// a warp takes 16 of them, from row0.  They are scaled by one power of two, from the
// largest of them, that takes f16's range into account; a row that is 2^-16 of
// it or less has one of its own, and what its scores then have to be multiplied
// by goes to `apart` (1 for the others).  A row with a non-finite element is
// made NaN.  Returns the inverse of the warp's factor, and whether any row is
// apart.
constexpr int kSpread = 16;
template <typename T, int D, int BITS>
__device__ __forceinline__ float load_rows(const AttentionArgs& a, const Sequence& s, const Unit& u, int t, int row0,
                                           uint32_t query, float* apart, bool* any_apart, bool aligned) {
  const int lane = threadIdx.x & 31;
  constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks == 0 ? 1 : 32 / kChunks;      // of a row, of eight elements; rows a step
  constexpr int kSteps = 16 * kChunks / 32;
  // A lane's chunks, one a step, come to where they stay, element by element as
  // they lie in memory; then they are read twice, for the largest and to be turned.
  auto row_of = [&](int n) { return kChunks <= 32 ? n * kAtOnce + lane / kChunks : n; };
  const int chunk = lane % kChunks;
  auto spot_of = [&](int n) {
    const int r = row0 + row_of(n);
    return query + (chunk >> 3) * (kRowTile * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
  };
  static_assert(kChunks <= 32, "a row is one step's at most");
  const T* my_row = nullptr;                               // row `lane`
  {
    const int r = t * kRowTile + row0 + lane, row = u.first + r;
    if (lane < 16 && r < u.rows)
      my_row = static_cast<const T*>(a.q.data) + (int64_t)(s.row + row / a.group) * a.q.ld +
               (int64_t)(u.head * a.group + row % a.group) * a.q.head_stride;
  }
#pragma unroll 2
  for (int n = 0; n < kSteps; ++n) {
    const T* from = reinterpret_cast<const T*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(my_row), row_of(n)));
    if (from != nullptr) {
      from += 8 * chunk;
      if (aligned) {
        copy16_async(spot_of(n), from);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(from)[e] << (16 * (e % 2));
        store_shared16(spot_of(n), w);
      }
    } else {
      const uint32_t none[4] = {0, 0, 0, 0};
      store_shared16(spot_of(n), none);
    }
  }
  copies_commit();
  copies_wait<0>();
  uint32_t most = 0;                                       // the largest |element| of the warp's finite rows
  uint32_t mine = 0;                                       // of row `lane`
#pragma unroll 2
  for (int n = 0; n < kSteps; ++n) {
    float v[8];
    to_floats<T, 8>(load_shared16<T, 8>(spot_of(n)), v);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
#pragma unroll
    for (int off = kChunks / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(kFull, top, off));
    // lane k of this step's row: hand the row's largest to the lane of its number
    const int first = n * kAtOnce;
    const uint32_t got = __shfl_sync(kFull, top, ((lane - first) & (kAtOnce - 1)) * kChunks);
    if (lane >= first && lane < first + kAtOnce) mine = got;
  }
  const bool finite = mine < 0x7F800000u;
  most = __reduce_max_sync(kFull, finite ? mine : 0u);
  const float factor = row_factor(most);
  const bool own = finite && mine != 0 && (int)(most >> 23) - (int)(mine >> 23) > kSpread;
  const float my_factor = own ? row_factor(mine) : factor;
  *any_apart = __any_sync(kFull, own);
  if (lane < 16) apart[t * kRowTile + row0 + lane] = factor / my_factor;  // powers of two
#pragma unroll 2
  for (int n = 0; n < kSteps; ++n) {
    const float f = __shfl_sync(kFull, my_factor, row_of(n));
    const bool bad = __shfl_sync(kFull, (int)!finite, row_of(n)) != 0;
    float v[8];
    to_floats<T, 8>(load_shared16<T, 8>(spot_of(n)), v);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // places 2 i and 2 i + 1
      const int e0 = BITS == 4 ? i : 2 * i, e1 = BITS == 4 ? i + 4 : 2 * i + 1;
      h[i] = bad ? 0x7E007E00u : pack_f16(v[e0] * f, v[e1] * f);
    }
    store_shared16(spot_of(n), h);
  }
  __syncwarp();
  return 1.0f / factor;
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) attention_many_kernel(const AttentionArgs a, const int wide_out, const int wide_in) {
  using S = Many<D, BITS>;
  constexpr int NT = S::NT, KT = S::KT;
  using B = Bars<NT>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[B::kCount];
  __shared__ int64_t shared[kThreads / 16 + 3];
  __shared__ float apart[S::kRows];
  __shared__ int2 seen[S::kRows];                        // keys [x, y) that a row sees
  __shared__ uint32_t tmem_at;
  __shared__ volatile int give_up;
  const uint32_t query = (smem_addr(raw) + 1023u) & ~1023u, keys = query + NT * S::kQuery, values = keys + 2 * S::kStage,
                 steps = values + 2 * S::kStage, bar = smem_addr(bars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    give_up = 0;
    mbar_init(bar + B::kQuery, 8 * NT);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B::kKeys + 8 * i, kWarpsKeys);
      mbar_init(bar + B::kKeysFree + 8 * i, 1);
      mbar_init(bar + B::kValues + 8 * i, kWarpsValues);
      mbar_init(bar + B::kValuesFree + 8 * i, 1);
      mbar_init(bar + B::kScores + 8 * i, 1);
      mbar_init(bar + B::kWeights + 8 * i, 8);
      mbar_init(bar + B::kSums + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(bar + B::kSteps + 8 * i, kWarpsKeys + kWarpsValues);
    mbar_init(bar + B::kLast, 1);
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_addr(&tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) joins(a)[blockIdx.x].blocks = 0;
  int bad = 0;
  const Range range = block_range<S::kRows, KT, kThreads, 1>(a, shared, &bad);
  Walk<S::kRows, KT> walk;
  walk.start(a, range);
  bool ok = true;

  if (warp >= kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssueRegs));
    if (warp == kIssuer) {
      const uint32_t one = elect_one();
      const uint32_t tm = uniform(tmem);
      constexpr uint32_t kInstrS = (1u << 4) | ((uint32_t)(KT / 8) << 17) | (8u << 24);                  // f16, fp32 sums
      constexpr uint32_t kInstrO = (1u << 4) | (1u << 16) | ((uint32_t)(D / 8) << 17) | (8u << 24);      // B with D contiguous
      auto wait = [&](uint32_t b, uint32_t parity) {
        ok = ok && __all_sync(0xFFFFFFFFu, wait_on(b, parity, &give_up));
        fence_after();
        return ok;
      };
      auto score = [&](int t, uint32_t i, uint32_t to) {               // S of tile i and rows' tile t
        const uint64_t da = smem_desc(query + t * S::kQuery), db = smem_desc(keys + (i & 1) * S::kStage);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_shared(one, to, da + (k / 4) * (kRowTile * 128 / 16) + 2 * (k % 4), db + (k / 4) * (KT * 128 / 16) + 2 * (k % 4),
                     kInstrS, k > 0);
      };
      auto weigh = [&](int t, uint32_t i, uint32_t from, bool add) {   // O of rows' tile t
        const uint64_t db = value_desc<KT>(values + (i & 1) * S::kStage);
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          mma_tmem(one, tm + S::kSums + t * D, from + 8 * k, db + k * (16 * 128 / 16), kInstrO, add || k > 0);
      };
      auto tell = [&](uint32_t b) { commit(one, b); };
      uint32_t i = 0, unit = 0;                            // tiles, units so far
      for (; __any_sync(kFull, walk.more()) && ok; walk.next(a, &bad), ++unit) {
        const uint32_t n = uniform(walk.take);
        if (!wait(bar + B::kQuery, unit & 1)) break;
        if (!wait(bar + B::kKeys + 8 * (i & 1), (i >> 1) & 1)) break;
        if constexpr (NT == 2) {
          for (int t = 0; t < 2; ++t) {
            score(t, i, tm + t * KT);
            tell(bar + B::kScores + 8 * t);
          }
          tell(bar + B::kKeysFree + 8 * (i & 1));
          for (uint32_t k = 0; k < n && ok; ++k, ++i) {
            const bool last = k + 1 == n;
            for (int t = 0; t < 2 && ok; ++t) {
              if (!wait(bar + B::kWeights + 8 * t, i & 1)) break;
              if (t == 0 && !wait(bar + B::kValues + 8 * (i & 1), (i >> 1) & 1)) break;
              weigh(t, i, tm + t * KT, k > 0);
              if (last) {
                tell(bar + B::kSums + 8 * t);
              } else {
                if (t == 0 && !wait(bar + B::kKeys + 8 * ((i + 1) & 1), ((i + 1) >> 1) & 1)) break;
                score(t, i + 1, tm + t * KT);
                tell(bar + B::kScores + 8 * t);
              }
            }
            if (!ok) break;
            tell(bar + B::kValuesFree + 8 * (i & 1));
            if (!last) tell(bar + B::kKeysFree + 8 * ((i + 1) & 1));
          }
        } else {
          score(0, i, tm + (i & 1) * KT);
          tell(bar + B::kScores + 8 * (i & 1));
          tell(bar + B::kKeysFree + 8 * (i & 1));
          for (uint32_t k = 0; k < n && ok; ++k, ++i) {
            const bool last = k + 1 == n;
            if (!last) {
              if (!wait(bar + B::kKeys + 8 * ((i + 1) & 1), ((i + 1) >> 1) & 1)) break;
              score(0, i + 1, tm + ((i + 1) & 1) * KT);
              tell(bar + B::kScores + 8 * ((i + 1) & 1));
              tell(bar + B::kKeysFree + 8 * ((i + 1) & 1));
            }
            if (!wait(bar + B::kWeights + 8 * (i & 1), (i >> 1) & 1)) break;
            if (!wait(bar + B::kValues + 8 * (i & 1), (i >> 1) & 1)) break;
            weigh(0, i, tm + (i & 1) * KT, k > 0);
            tell(bar + B::kValuesFree + 8 * (i & 1));
            if (last) tell(bar + B::kSums);
          }
        }
      }
      if (one) {                                           // instructions still running end before TMEM is freed
        commit(1, bar + B::kLast);
        mbar_wait_bounded(bar + B::kLast, 0);
      }
      __syncwarp();
    }
  } else if (warp >= kWarpsWeights) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kTurnRegs));
    // Keys, or values: a thread has a row of a tile (of KT 64, half of one).
    const bool value = warp >= kWarpsWeights + kWarpsKeys;
    const uint32_t base1024 = unknown(0x64006400u);
    // For loads a row's pieces of 16 bytes are neighbouring lanes', 32 * kWide of
    // which a warp takes at once; page and meta word of a row come from its lane.
    constexpr int kWarpRows = KT / 4, kPieces = S::kRowBytes / 16;         // rows of a warp; pieces of a row
    constexpr int kWide = 32 / kPieces;                                    // rows at once
    constexpr int kLoads = kWarpRows / kWide, kChunks = 16 / BITS;         // loads; eights of codes of a piece
    const int row0 = (warp & 3) * kWarpRows, r = row0 + lane;              // this lane's row, if it has one
    const bool row_lane = lane < kWarpRows;
    const int piece = lane % kPieces, in_row = lane / kPieces;
    const uint32_t stages = value ? values : keys, full = bar + (value ? B::kValues : B::kKeys),
                   empty = bar + (value ? B::kValuesFree : B::kKeysFree);
    const int64_t on = value ? (int64_t)a.cache.heads << a.cache.page_shift : 0;
    uint4 w[kLoads];
    uint32_t meta = 0;                                     // of this lane's row
    bool there = false;
    // A row's page is looked up two tiles ahead (and looked at one ahead: a use
    // right away would wait for it), its codes are loaded one ahead.
    int ahead = 0, page = 0, page_key = 0, page_head = 0;  // tiles into the unit of the page that is looked up next
    const uint32_t n = (uint32_t)(range.end - range.begin);
    auto look_up = [&]() {
      page_key = -1;                                       // no key for this lane
      if (!__any_sync(kFull, walk.more())) return;
      page_key = (walk.unit.tile + walk.in + ahead) * KT + r;
      page_head = walk.unit.head;
      if (!row_lane || page_key >= walk.s.keys) page_key = -1;
      // (pages wholly behind the window of the unit's first row may be gone)
      if (ahead == 0 && a.window && page_key < keys_from(a, walk.s.place + walk.unit.first / a.group)) page_key = -1;
      if (page_key >= 0) {
        const int at = page_key >> a.cache.page_shift;
        page = -1;
        if (at < a.batch.table_pages) page = a.batch.table[(int64_t)walk.unit.sequence * a.batch.ld_table + at];
      }
      if (++ahead == walk.take) {
        ahead = 0;
        walk.next(a, &bad);
      }
    };
    // Rows that are not there have codes of 0, less 0.
    auto load = [&]() {
      there = page_key >= 0 && page >= 0 && page < a.cache.pages;
      if (page_key >= 0 && !there) bad |= kBadPage;
      const int64_t group = there ? group_index(a.cache, page, page_head, page_key) + on : -1;
      meta = 0;
      if (there) meta = a.cache.meta[group];
#pragma unroll
      for (int p = 0; p < kLoads; ++p) {
        const int64_t of = __shfl_sync(kFull, group, p * kWide + in_row);
        w[p] = make_uint4(0, 0, 0, 0);
        if (of >= 0) w[p] = reinterpret_cast<const uint4*>(a.cache.codes + of * S::kRowBytes)[piece];
      }
    };
    look_up();
    load();
    look_up();
    for (uint32_t i = 0; i < n; ++i) {
      ok = __all_sync(0xFFFFFFFFu, wait_on(empty + 8 * (i & 1), ((i >> 1) & 1) ^ 1u, &give_up));
      if (!ok) break;
      // A value that is not there has a log of -infinity, so that its weight is 0,
      // which adds 0 to the sum.  So does a NaN to the sums of rows that do not
      // see it; its log spreads it to those that do.
      if (row_lane) {
        const uint32_t at = steps + (i & (kSlots - 1)) * S::kSteps + 4 * r;
        if (!value) {
          asm volatile("st.shared.f32 [%0], %1;" :: "r"(at), "f"(meta_step(meta)) : "memory");
        } else {
          const float of = value_factor(meta);
          const float log = there ? log2_of(of) : kNone, per = there && of == of ? reciprocal(of) : 0.0f;
          asm volatile("st.shared.f32 [%0], %1;" :: "r"(at + 4 * KT), "f"(log) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" :: "r"(at + 8 * KT), "f"(per) : "memory");
        }
      }
      __syncwarp();
      if (lane == 0) arrive_here(bar + B::kSteps + 8 * (i & (kSlots - 1)));
      // Of this lane's row: -(1024 + z) S and -(64 + z) S in one word, S in another
      // (with 8 bits in the first one's upper half).
      const uint32_t zs = __byte_perm(meta, meta, 0x3232), my_scale = value ? value_scale(meta) : 0x3C00u;
      const uint32_t scales = __byte_perm(my_scale, my_scale, 0x1010);
      const __half2 both = __hmul2(__hsub2(__floats2half2_rn(-1024.0f, -64.0f), *reinterpret_cast<const __half2*>(&zs)),
                                   *reinterpret_cast<const __half2*>(&scales));
      uint32_t my_zero = *reinterpret_cast<const uint32_t*>(&both);
      if constexpr (BITS == 8) my_zero = __byte_perm(my_zero, my_scale, 0x5410);
      const uint32_t to = stages + (i & 1) * S::kStage;
      // A piece's eights are stored in an order by piece, so that eight lanes that
      // store together (one, two or four rows) meet no bank twice.
      constexpr int kAtom = 8 / kChunks;                   // pieces of a row's 128 bytes
      const int turn = (piece / kAtom * (kPieces / kAtom == 2 && kChunks == 4 ? 2 : 1)) & (kChunks - 1);
#pragma unroll
      for (int p = 0; p < kLoads; ++p) {
        const int row = p * kWide + in_row;
        const uint32_t zero = __shfl_sync(kFull, my_zero, row), low = __byte_perm(zero, zero, 0x1010),
                       upper = __byte_perm(zero, zero, 0x3232);
        const uint32_t scale = BITS == 4 ? __shfl_sync(kFull, scales, row) : upper;
        const uint32_t high_scale = BITS == 4 ? times_half(scale, 0.0625f) : 0;
        const uint32_t at = to + (row0 + row) * 128;
        uint32_t words[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
        if constexpr (BITS == 4) {
          if (turn & 2) {
            uint32_t x = words[0];
            words[0] = words[2], words[2] = x, x = words[1], words[1] = words[3], words[3] = x;
          }
          if (turn & 1) {
            uint32_t x = words[0];
            words[0] = words[1], words[1] = x, x = words[2], words[2] = words[3], words[3] = x;
          }
        } else {
          if (turn & 1) {
            uint32_t x = words[0];
            words[0] = words[2], words[2] = x, x = words[1], words[1] = words[3], words[3] = x;
          }
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t h[4];
          if constexpr (BITS == 4) turn4(words[c], base1024, scale, low, high_scale, upper, h);
          else turn8(words[2 * c], words[2 * c + 1], base1024, scale, low, h);
          const int chunk = piece * kChunks + (c ^ turn);
          store_shared16(at + (chunk >> 3) * (KT * 128) + (((chunk & 7) ^ ((row0 + row) & 7)) << 4), h);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_here(full + 8 * (i & 1));
      load();                          // behind the fence, which would wait for it
      look_up();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kWeightRegs));
    const int t = warp >> 3;                               // tile of rows
    if (t < NT) {
      // Two warps have 16 each of the 32 rows that a warp of this number reaches.
      const int row0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
      const int g = lane >> 2, quad = lane & 3;
      const uint32_t lanes = tmem + ((uint32_t)row0 << 16);
      const uint32_t sums = lanes + S::kSums + t * D;
      uint32_t i = 0, unit = 0;
      float scale = 0.0f, next_scale = 0.0f;               // of the warp's scores
      bool any_apart = false, next_apart = false;
      auto take_rows = [&]() {
        const uint32_t to = query + t * S::kQuery;
        const float back = a.dtype == ECHO_BF16
                               ? load_rows<__nv_bfloat16, D, BITS>(a, walk.s, walk.unit, t, row0, to, apart, &next_apart, wide_in)
                               : load_rows<__half, D, BITS>(a, walk.s, walk.unit, t, row0, to, apart, &next_apart, wide_in);
        next_scale = a.scale * kLog2E * back;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_here(bar + B::kQuery);
      };
      if (walk.more()) take_rows();
      while (walk.more() && ok) {
        // This lane's rows: g and g + 8 of the warp's.
        float m[2], l[2][2];
        scale = next_scale;
        any_apart = next_apart;
        const int first = t * kRowTile + row0;             // of the unit's rows, the warp's first
        if (lane < 16) {
          const int r = first + lane, place = walk.s.place + (walk.unit.first + r) / a.group;
          // (rows past the last see all: one that sees nothing has no maximum)
          seen[r] = r < walk.unit.rows ? make_int2(keys_from(a, place), keys_to(a, walk.s, place)) : make_int2(0, 0x7FFFFFFF);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[h] = kLowest;
          l[h][0] = l[h][1] = 0.0f;
        }
        int all_from = 0, all_to = 0x7FFFFFFF;             // keys that all rows of the warp see
        if (first < walk.unit.rows) {
          const int end = first + 16 < walk.unit.rows ? first + 15 : walk.unit.rows - 1;
          all_from = keys_from(a, walk.s.place + (walk.unit.first + end) / a.group);
          all_to = keys_to(a, walk.s, walk.s.place + (walk.unit.first + first) / a.group);
        }
        int key = (walk.unit.tile + walk.in) * KT;
        for (int k = 0; k < walk.take; ++k, ++i, key += KT) {
          const uint32_t buffer = NT == 2 ? (uint32_t)t : i & 1;
          ok = __all_sync(0xFFFFFFFFu, wait_on(bar + B::kSteps + 8 * (i & (kSlots - 1)), (i / kSlots) & 1, &give_up) &&
                                           wait_on(bar + B::kScores + 8 * buffer, NT == 2 ? i & 1 : (i >> 1) & 1, &give_up));
          if (!ok) break;
          fence_after();
          const uint32_t s_at = lanes + buffer * KT, slot = steps + (i & (kSlots - 1)) * S::kSteps + 8 * quad;
          const bool inside = key >= all_from && key + KT <= all_to;
          // Raises the rows' maxima to `top` and scales what was made with the
          // old ones: the sums, and this tile's weights of the keys before c.
          auto raise = [&](float (&top)[2], int c) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
              top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
              top[h] = raised<kAhead>(m[h], top[h]);
              f[h] = exp2_of(m[h] - top[h]);
              m[h] = top[h];
              l[h][0] *= f[h];
              l[h][1] *= f[h];
            }
            if (k > 0) {
              if (NT == 1) {                               // (with two tiles of rows the scores came after the sums)
                ok = ok && __all_sync(0xFFFFFFFFu, wait_on(bar + B::kValuesFree + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, &give_up));
                fence_after();
              }
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                float v[16];
                tmem_load(sums + d, v);
                tmem_loaded(v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= f[(e >> 1) & 1];
                tmem_store(sums + d, v);
              }
            }
            if (c > 0) tmem_stored();
#pragma unroll 1
            for (int d = 0; d < c / 2; d += 16) {          // (pairs, read and written as 8 words of two rows)
              uint32_t w[8];
              tmem_load_pairs(s_at + d, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                w[e] = pack_f16(two.x * f[e & 1], two.y * f[e & 1]);
              }
              tmem_store_pairs(s_at + d, w);
            }
          };
          // Weights of the tile's keys, 32 at a time: u = s * scale * step_k + log
          // step_v, p = exp(u - m).  PLAIN: every row sees all, none is apart (a
          // branch a pair would leave the compiler nothing to interleave).
          auto weights = [&](auto plain) {
            constexpr bool kPlain = decltype(plain)::value;
            float v[2][16];                                // of these and of the next keys
            float f[2];
            int2 see[2];
            if (!kPlain) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                f[h] = apart[first + g + 8 * h];
                see[h] = seen[first + g + 8 * h];
              }
            }
            tmem_load(s_at, v[0]);
#pragma unroll 1                                           // (code that is fetched again costs as much as its work)
            for (int c0 = 0; c0 < KT; c0 += 64)
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {
                const int c = c0 + 32 * odd;
                float(&now)[16] = v[odd];
                tmem_loaded(now);
                if (c + 32 < KT) tmem_load(s_at + c + 32, v[odd ^ 1]);
                float top[2] = {m[0], m[1]};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  float2 ks = shared_pair(slot + 4 * (c + 8 * n));
                  const float2 log = shared_pair(slot + 4 * (KT + c + 8 * n));
                  mul2(ks.x, ks.y, ks.x, ks.y, scale, scale);
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float &v0 = now[4 * n + 2 * h], &v1 = now[4 * n + 2 * h + 1];
                    if (!kPlain) mul2(v0, v1, v0, v1, f[h], f[h]);
                    fma2(v0, v1, v0, v1, ks.x, ks.y, log.x, log.y);
                    if (!kPlain) {
                      const int at = key + c + 8 * n + 2 * quad;
                      v0 = at < see[h].x || at >= see[h].y ? kNone : v0;
                      v1 = at + 1 < see[h].x || at + 1 >= see[h].y ? kNone : v1;
                    }
                    top[h] = max3(top[h], v0, v1);
                  }
                }
                if (__any_sync(kFull, top[0] - m[0] > kMostWeight || top[1] - m[1] > kMostWeight)) raise(top, c);
                uint32_t w[8];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  const float2 per = shared_pair(slot + 4 * (2 * KT + c + 8 * n));
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float v0 = now[4 * n + 2 * h], v1 = now[4 * n + 2 * h + 1];
                    sub2(v0, v1, v0, v1, m[h], m[h]);
                    v0 = exp2_of(v0);
                    v1 = exp2_of(v1);
                    fma2(l[h][0], l[h][1], v0, v1, per.x, per.y, l[h][0], l[h][1]);
                    w[2 * n + h] = pack_f16(v0, v1);
                  }
                }
                // (in the place of scores that have been read: those of half as many keys)
                tmem_store_pairs(s_at + c / 2, w);
              }
          };
          if (inside && !any_apart) weights(std::true_type());
          else weights(std::false_type());
          if (!ok) break;
          tmem_stored();
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_here(bar + B::kWeights + 8 * buffer);
        }
        if (!ok) break;
        // The next unit's rows (this one's have been used), then this one's sums.
        const Walk<S::kRows, KT> done = walk;
        walk.next(a, &bad);
        if (walk.more()) take_rows();
        ok = __all_sync(0xFFFFFFFFu, wait_on(bar + B::kSums + 8 * t, unit & 1, &give_up));
        if (!ok) break;
        ++unit;
        fence_after();
        const bool whole = done.whole();
        float* const part = slot_at(a, gridDim.x, slot_of(done, range), S::kRows, D);
        float per[2];
        int64_t out[2];
        bool there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = l[h][0] + l[h][1];
          sum += __shfl_xor_sync(kFull, sum, 1);
          sum += __shfl_xor_sync(kFull, sum, 2);
          per[h] = sum == 0.0f ? 0.0f : 1.0f / sum;
          const int r = first + g + 8 * h, row = done.unit.first + r, token = done.s.row + row / a.group;
          const int head = done.unit.head * a.group + row % a.group;
          there[h] = r < done.unit.rows;
          out[h] = token * a.out.ld + head * a.out.head_stride + 8 * quad;
          if (quad == 0 && there[h]) {
            if (!whole) {
              part[S::kRows * D + r] = m[h];
              part[S::kRows * D + S::kRows + r] = sum;
            } else if (a.lse) {
              a.lse[(int64_t)token * a.heads + head] = sum == 0.0f ? kNone : (m[h] + log2_of(sum)) * kLn2;
            }
          }
        }
        if (!whole && done.in == 0 && tid == 0) name_parts(a, done, range);
        // Two rows of 32 columns at a time, in a rolled loop: code that runs once a
        // unit is fetched each time.
        {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[16];
            tmem_load(sums + c, v);
            tmem_loaded(v);
            // Of a row's four eights this lane has a pair each; after the exchange
            // it has all pairs of the eight of its own number.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float e[8];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float x[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) x[n] = v[4 * n + 2 * h + b];
#pragma unroll
                for (int step = 1; step < 4; step *= 2)
#pragma unroll
                  for (int n = 0; n < 4; ++n) {
                    if (n & step) continue;
                    const bool high = quad & step;
                    const float got = __shfl_xor_sync(kFull, high ? x[n] : x[n + step], step);
                    x[n] = high ? got : x[n];
                    x[n + step] = high ? x[n + step] : got;
                  }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const int place = 2 * q + b;             // in the eight, as TMEM has it
                  e[BITS == 4 ? (place & 1) * 4 + (place >> 1) : place] = x[q];
                }
              }
              if (!there[h]) continue;
              if (whole) {
#pragma unroll
                for (int n = 0; n < 8; ++n) e[n] *= per[h];
                if (wide_out) {
                  if (a.dtype == ECHO_BF16) store_floats<__nv_bfloat16, 8>(static_cast<__nv_bfloat16*>(a.out.data) + out[h] + c, e);
                  else store_floats<__half, 8>(static_cast<__half*>(a.out.data) + out[h] + c, e);
                } else {
#pragma unroll
                  for (int n = 0; n < 8; ++n) store_value(a, out[h] + c + n, e[n]);
                }
              } else {
                float* const to_part = part + (first + g + 8 * h) * D + c + 8 * quad;
                *reinterpret_cast<float4*>(to_part) = make_float4(e[0], e[1], e[2], e[3]);
                *reinterpret_cast<float4*>(to_part + 4) = make_float4(e[4], e[5], e[6], e[7]);
              }
            }
          }
        }
        fence_before();
      }
    }
  }
  if (!ok) bad |= kGaveUp;
  if (bad) report(bad);
  __syncthreads();
  if (warp == kIssuer) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem));
  }
}

template <int D, int BITS>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t s) {
  using S = Many<D, BITS>;
  static OncePerDevice once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(attention_many_kernel<D, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int blocks = useful_blocks(a, S::kRows, S::KT, sms);
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  auto wide = [](const HeadsArgs& h) { return (int)(on_boundary(h.data, 16) && h.ld % 8 == 0 && h.head_stride % 8 == 0); };
  const cudaError_t e2 = cudaLaunchKernelEx(&cfg, attention_many_kernel<D, BITS>, a, wide(a.out), wide(a.q));
  return e2 != cudaSuccess ? e2 : launch_join(a, blocks, S::kRows, s);
}

}  // namespace

cudaError_t launch_attention_many(const AttentionArgs& a, int sms, cudaStream_t s) {
  const bool four = a.cache.bits == 4;
  if (a.cache.head_dim == 64) return four ? launch<64, 4>(a, sms, s) : launch<64, 8>(a, sms, s);
  if (a.cache.head_dim == 128) return four ? launch<128, 4>(a, sms, s) : launch<128, 8>(a, sms, s);
  return four ? launch<256, 4>(a, sms, s) : launch<256, 8>(a, sms, s);
}
int64_t attention_many_bytes(int head_dim, int sms) { return workspace_bytes(sms, head_dim == 256 ? 128 : 256, head_dim); }
StatusWord attn_many_status() { return {read_status, clear_status_bits}; }

}  // namespace echo
