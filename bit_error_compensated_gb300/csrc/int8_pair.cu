// int8_pair.cu -- echo_matmul_int8 for many tokens, on the tensor cores.
//
// This GPU's tensor cores have no fast integer form, but an int8 code is an
// f16 number, the product of two is exact, and a sum of products is exact in
// fp32 while it stays within 2^24: for 1024 products of codes, whatever they
// are (128 * 128 * 1024 = 2^24).  So the codes are turned into f16 on their
// way into shared memory, f16 matrix instructions sum 1024 products deep
// chunks in TMEM, and each chunk's sums are added up as int32 in registers.
//
// Two SMs (a cluster of two blocks) share one tile of 256 tokens x BN channels
// (tcgen05 cta_group::2), 128 rows of tokens and BN / 2 of channels in each
// block's shared memory, which halves what goes through it per product.  The
// tokens' codes come as f16 from the workspace, a block of 128 x 128 per copy;
// turning those of the tokens once instead of in every tile costs 2 bytes a
// code, while turning the larger weights ahead would cost as much as the
// product of a thousand tokens.  So the channels' codes come as int8 by TMA,
// and warps turn them in shared memory.  A block's warps:
//   8  take chunks' sums out of TMEM, add them up and store the results;
//   8  turn codes, in two groups that take the stages (128 codes deep) in turn,
//      so that one group's fences and waits overlap the other's work;
//   3  issue: matrix instructions (first block), the tokens' copies, the
//      channels' copies.
// TMEM holds two chunks' sums, so one is taken out while the next is computed.
// A stage takes 1000 to 1100 cycles, 1024 of which its matrix instructions need.
//
// One GB300: 8192 x 14336 x 4096 in 491 to 506 us, 1900 to 1960 TFLOP/s of
// products (bound by the matrix instructions: a library's f16 product reaches
// 1920); 4 x 2048 x 4096 x 1024 in 54 us, 1280 (one chunk a tile: its 128 KB of
// results take the takers as long as its products take the tensor cores).
// Where tiles are few the machine is not full: a tile is always 256 x 256, so 64
// x 4096 x 4096 takes the 21 us of 256 tokens, of 2.5 us of bytes.
//
// Where there are fewer tiles than pairs of SMs, SPLIT pairs in a cluster share
// a tile's depth.  Their sums are int32, so their order does not matter: each
// pair writes those of the columns that it does not own into the owner's
// shared memory (the ring is free by then), and the owner adds and stores.  (With
// that exchange beside 128 sums, 136 to 316 bytes a thread are spilled.)
//
// Every wait is bounded; one that gives up ends the call with a status
// (echo_matmul_status).  The other warps of its block leave at their next wait,
// whose own flag stays set; each issuing warp first waits for what it has
// issued to end (mbar_wait_bounded, which looks at no flag), whether it gave up
// itself or finished and another did.
#include <cuda.h>

#include "int8_load.h"
#include "tensor.cuh"

namespace echo {
namespace {

constexpr int kRows = kBlockTokens;     // tokens a block holds of the pair's 256
constexpr int kStageDepth = kBlockCodes;
constexpr int kStages = 3;
constexpr int kChunkStages = 8;         // 1024 codes: exact in fp32
constexpr int kTakers = 8, kGroups = 2, kGroupWarps = 4, kTurners = kGroups * kGroupWarps;
constexpr int kIssuer = kTakers + kTurners;     // the first of the issuing warps
constexpr int kThreads = 32 * (kIssuer + 4);    // five warpgroups; of the last, three warps work
// Registers: the block starts with 96 a thread (five warpgroups of 480 in
// all); a taker holds up to 128 sums, a turner a stage's codes.
constexpr int kTakerRegs = 168, kTurnerRegs = 56, kIssuerRegs = 32;
static_assert(2 * kTakerRegs + 2 * kTurnerRegs + kIssuerRegs <= 5 * 96,
              "a split above the launch's registers never ends");

template <int BN> constexpr int code_bytes() { return BN / 2 * kStageDepth; }        // int8, one stage
template <int BN> constexpr int stage_bytes() { return kBlockBytes + 2 * code_bytes<BN>(); }
template <int BN> constexpr int smem_bytes() {
  return kStages * stage_bytes<BN>() + kGroups * code_bytes<BN>() + 1024;
}

// Set by a block whose wait gave up, until echo_matmul_status clears it.
__device__ int g_gave_up;

struct Tiles {
  int rows, cols, per_rank, total;      // of 256 tokens, BN channels
  int hold;                             // test hook: the first block never reports a stage
};

struct Place {
  int rank, row, col;
};
// Tiles in groups of eight along the tokens, so that the pairs at work at one
// time read few different rows of either operand.
__device__ __forceinline__ Place place_of(const Tiles& t, int tile) {
  Place p;
  p.rank = tile / t.per_rank;
  const int i = tile - p.rank * t.per_rank, group = i / (8 * t.cols);
  const int first = group * 8, high = t.rows - first < 8 ? t.rows - first : 8;
  const int j = i - group * 8 * t.cols;
  p.col = j / high;
  p.row = first + j - p.col * high;
  return p;
}

// Arrives on a barrier of the pair's first block, without a release to the
// cluster (which waits for everything the SM has in flight, over a thousand
// cycles).  What the arrival reports needs none: rows in this block's shared
// memory, which this SM's own matrix unit reads and the proxy fence before the
// arrival has made visible to it; copies that have landed there; and loads
// from TMEM that have returned.
__device__ __forceinline__ void arrive_first(uint32_t bar, uint32_t first_rank) {
  asm volatile(
      "{\n\t.reg .b32 at;\n\t"
      "mapa.shared::cluster.u32 at, %0, %1;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [at];\n\t}"
      :: "r"(bar), "r"(first_rank) : "memory");
}

// All matrix instructions issued so far will arrive on `bar` of both blocks.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint32_t first_rank) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" :: "r"(bar), "h"((uint16_t)(3u << first_rank)) : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(desc), "r"(add) : "memory");
}

// (.aligned: lanes that store rows and columns past the last ones leave a
// store early, so a warp's are brought together first.)
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// A box of the channels' codes: 128 codes from k of the rows from c of a rank.
__device__ __forceinline__ void load_box(uint32_t to, const CUtensorMap* map, int k, int c, int rank, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(to), "l"(map), "r"(k), "r"(c), "r"(rank), "r"(bar) : "memory");
}

// Among the takers' warps; whether all of them are fine.
__device__ __forceinline__ bool takers_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all) : "r"((uint32_t)ok), "n"(32 * kTakers) : "memory");
  return all != 0;
}

// 16 exact sums of this lane's token times its scale and the channels' (in
// shared memory), as out's type, into half (fp32: all) of 16 words.
template <typename T>
__device__ __forceinline__ void scale_sums(float (&sum)[16], uint32_t scales, float token, uint32_t* words) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    float w[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(scales + 4 * i) : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[i + k] = scaled_sum(sum[i + k], token, w[k]);
  }
  const Pack<T, 16> out = from_floats<T, 16>(sum);
#pragma unroll
  for (int i = 0; i < (int)sizeof(out) / 4; ++i) words[i] = reinterpret_cast<const uint32_t*>(&out)[i];
}

// Each lane has UNITS units of WORDS words of its own token's row; after this it
// has unit lane % UNITS of the rows of its UNITS lanes (in order), so that these
// store a row's part together: a store takes its time by the lines it touches,
// and lanes that each store their own row touch 32 (4 x 2048 x 4096 x 1024:
// 61 us, units of 32 bytes exchanged 57).
template <int UNITS, int WORDS>
__device__ __forceinline__ void exchange_units(uint32_t (&w)[WORDS * UNITS], int lane) {
#pragma unroll
  for (int step = 1; step < UNITS; step *= 2) {
    const bool high = lane & step;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if (u & step) continue;
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        uint32_t &a = w[WORDS * u + k], &b = w[WORDS * (u + step) + k];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? a : b, step);
        if (high) a = got;
        else b = got;
      }
    }
  }
}

// Stores the lanes' rows, 8 UNITS words of each from channel c, of which the
// first lane's is token t - lane.  `align`: the bytes on whose multiples out's
// rows start (32, 16, 4 or fewer).  Rows on 16 bytes go in units of 32 bytes;
// others, where a unit takes 16 stores that each touch a sector, BY_WORD with a
// row's words from neighbouring lanes (9578 x 7999 x 512: 528 us in units, 115
// by word).  A kernel that holds 128 sums a thread has no registers for that
// second way (8192 x 14336 x 4096: 490 us without it, 680 with) and less to win,
// as it stores once in several chunks (4 x 544 x 1587 x 8192: 144 us, 130).
template <typename T, int UNITS, bool BY_WORD>
__device__ __forceinline__ void store_rows(const ProductArgs& p, T* out, int64_t t, int64_t c, int lane,
                                           uint32_t (&w)[8 * UNITS], int align) {
  if (!BY_WORD || align >= 16) {
    constexpr int kUnit = 32 / sizeof(T);
    exchange_units<UNITS, 8>(w, lane);
    t -= lane % UNITS;
    c += lane % UNITS * kUnit;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (t + i >= p.tokens) break;
      T* to = out + (t + i) * p.ld_out + c;
      const bool whole = c + kUnit <= p.channels;
      if (whole && align == 32) {
        store32(to, reinterpret_cast<const uint32_t(*)[8]>(w)[i]);
      } else if (whole && align == 16) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          reinterpret_cast<uint4*>(to)[e] = make_uint4(w[8 * i + 4 * e], w[8 * i + 4 * e + 1], w[8 * i + 4 * e + 2],
                                                       w[8 * i + 4 * e + 3]);
      } else if (!BY_WORD && whole && align == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<uint32_t*>(to)[e] = w[8 * i + e];
      } else {
#pragma unroll
        for (int e = 0; e < kUnit; ++e)
          if (c + e < p.channels) to[e] = reinterpret_cast<const T*>(w)[i * kUnit + e];
      }
    }
  } else {
    constexpr int kWords = 8 * UNITS, kWord = 4 / sizeof(T);
    exchange_units<kWords, 1>(w, lane);
    t -= lane % kWords;
    c += lane % kWords * kWord;
    if (c >= p.channels) return;
    T* to = out + t * p.ld_out + c;
#pragma unroll
    for (int i = 0; i < kWords; ++i, to += p.ld_out) {
      if (t + i >= p.tokens) break;
      if (align == 4 && c + kWord <= p.channels) {
        *reinterpret_cast<uint32_t*>(to) = w[i];
      } else {
#pragma unroll
        for (int e = 0; e < kWord; ++e)
          if (c + e < p.channels) to[e] = reinterpret_cast<const T*>(w)[i * kWord + e];
      }
    }
  }
}

// ONE: a tile is one chunk (depth up to 1024), whose sums are stored as they
// come; SPLIT is 1.
template <typename T, int BN, int SPLIT, bool ONE>
__global__ void __cluster_dims__(2 * SPLIT, 1, 1) __launch_bounds__(kThreads, 1)
product_pair_kernel(const ProductArgs p, const Tiles tiles, const int out_align,
                    const __grid_constant__ CUtensorMap codes_map) {
  constexpr int kCols = BN / 2;                         // of a chunk's sums, a taker's
  // Units that lanes exchange before a store: with 128 sums in registers two
  // are what fits.
  constexpr int kUnits = ONE ? 4 : 2, kLine = kUnits * 32 / (int)sizeof(T);
  constexpr uint32_t kAtomA = kRows * 128, kAtomB = BN / 2 * 128;         // 64 codes of every row
  constexpr uint32_t kInstr = (1u << 4) | ((uint32_t)(BN / 8) << 17) | (16u << 24);  // f16, fp32 sums, 256 x BN
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[3 * kStages + 2 * kGroups + 5];
  __shared__ uint32_t tmem_at;
  __shared__ volatile int give_up;
  __shared__ __align__(16) float channel_scales[BN];
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u, codes = ring + kStages * stage_bytes<BN>();
  const uint32_t full = smem_addr(bars), landed = full + 8 * kStages, empty = landed + 8 * kStages,
                 codes_full = empty + 8 * kStages, codes_free = codes_full + 8 * kGroups,
                 sums_full = codes_free + 8 * kGroups, sums_empty = sums_full + 16, last = sums_empty + 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = (int)(blockIdx.x & 1);               // of the pair
  const int split = SPLIT == 1 ? 0 : (int)(blockIdx.x >> 1) % SPLIT;      // of the tile's depth, this pair's
  const uint32_t first_rank = 2 * split;                // in the cluster, of the pair's first block
  const int pair = (int)(blockIdx.x / (2 * SPLIT)), pairs = (int)(gridDim.x / (2 * SPLIT));   // (or cluster)
  const int tile_stages = (int)wide_blocks(p.depth);    // at least SPLIT
  const int first_stage = tile_stages * split / SPLIT;  // of a tile, this pair's
  const int stages = tile_stages * (split + 1) / SPLIT - first_stage;
  const int least = (stages + kChunkStages - 1) / kChunkStages;           // chunks, as even as can be
  const int chunk_stages = (stages + least - 1) / least, chunks = (stages + chunk_stages - 1) / chunk_stages;
  const int mine = pair < tiles.total ? (tiles.total - 1 - pair) / pairs + 1 : 0;

  if (tid == 0) {
    give_up = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 2 * kGroupWarps);
      mbar_init(landed + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int g = 0; g < kGroups; ++g) {
      mbar_init(codes_full + 8 * g, 1);
      mbar_init(codes_free + 8 * g, kGroupWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sums_full + 8 * b, 1);
      mbar_init(sums_empty + 8 * b, 2 * kTakers);
    }
    mbar_init(last, 1);
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(&tmem_at)), "r"(2 * BN) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_barrier();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_at;
  pdl_wait();
  pdl_trigger();

  if (warp >= kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssuerRegs));
    int slot = 0;
    uint32_t phase = 0;
    auto next = [&]() {
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
    };
    if (warp == kIssuer && half == 0) {
      // The pair's matrix instructions (one lane issues; the warp stays
      // together, so that addresses are uniform).
      const bool one = elect_one();
      uint32_t chunk = 0;
      bool ok = true;
      for (int t = 0; t < mine && ok; ++t) {
        for (int s0 = 0; s0 < stages && ok; s0 += chunk_stages, ++chunk) {
          const uint32_t b = chunk & 1, d = tmem + b * BN;
          const int n = stages - s0 < chunk_stages ? stages - s0 : chunk_stages;
          ok = __all_sync(0xFFFFFFFFu, wait_on(sums_empty + 8 * b, ((chunk >> 1) & 1) ^ 1u, &give_up));
          for (int s = 0; s < n && ok; ++s) {
            ok = __all_sync(0xFFFFFFFFu, wait_on(full + 8 * slot, phase, &give_up));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (one && ok) {
              const uint64_t da = smem_desc(ring + slot * stage_bytes<BN>());
              const uint64_t db = da + (2 * kAtomA >> 4);
#pragma unroll
              for (int k = 0; k < kStageDepth / 16; ++k)        // 16 codes: 32 bytes on
                mma_pair(d, da + (k / 4) * (kAtomA >> 4) + 2 * (k % 4),
                         db + (k / 4) * (kAtomB >> 4) + 2 * (k % 4), kInstr, s > 0 || k > 0);
              commit_pair(empty + 8 * slot, first_rank);
            }
            next();
          }
          if (one && ok) commit_pair(sums_full + 8 * b, first_rank);
        }
      }
      if (one) {                       // instructions still running end before TMEM is freed
        commit_pair(last, first_rank);
        mbar_wait_bounded(last, 0);
      }
    } else if (warp == kIssuer + 1 && lane == 0) {
      // The tokens' copies.
      const int64_t blocks = wide_blocks(p.tokens);
      const uint64_t policy = policy_evict_normal();
      int64_t issued = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles.total && ok; tile += pairs) {
        const Place at = place_of(tiles, tile);
        int64_t row = (int64_t)at.row * 2 + half;
        row = row < blocks ? row : blocks - 1;          // past the last token: its results are dropped
        const uint8_t* from =
            p.wide + (((p.rank_a == 0 ? 0 : at.rank) * blocks + row) * tile_stages + first_stage) * kBlockBytes;
        for (int s = 0; s < stages; ++s, from += kBlockBytes) {
          ok = wait_on(empty + 8 * slot, phase ^ 1u, &give_up);
          if (!ok) break;
          mbar_expect_tx(landed + 8 * slot, kBlockBytes);
          bulk_g2s(ring + slot * stage_bytes<BN>(), from, kBlockBytes, landed + 8 * slot, policy);
          ++issued;
          next();
        }
      }
      for (int n = 0; n < kStages && issued > 0; ++n, --issued) {         // no copy outlives the block
        slot = slot == 0 ? kStages - 1 : slot - 1;
        if (slot == kStages - 1) phase ^= 1;
        mbar_wait_bounded(landed + 8 * slot, phase);
      }
    } else if (warp == kIssuer + 2 && lane == 0) {
      // The channels' copies, a slot for each group of turners.
      int64_t g = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles.total && ok; tile += pairs) {
        const Place at = place_of(tiles, tile);
        for (int s = 0; s < stages; ++s, ++g) {
          const uint32_t bar = codes_full + 8 * (uint32_t)(g & 1);
          ok = wait_on(codes_free + 8 * (uint32_t)(g & 1), (uint32_t)((g >> 1) & 1) ^ 1u, &give_up);
          if (!ok) break;
          mbar_expect_tx(bar, code_bytes<BN>());
          load_box(codes + (uint32_t)(g & 1) * code_bytes<BN>(), &codes_map, (first_stage + s) * kStageDepth,
                   at.col * BN + half * (BN / 2), p.rank_w == 0 ? 0 : at.rank, bar);
        }
      }
      for (int n = 0; n < kGroups && g > 0; ++n) {                        // no copy outlives the block
        --g;
        mbar_wait_bounded(codes_full + 8 * (uint32_t)(g & 1), (uint32_t)((g >> 1) & 1));
      }
    }
    if (SPLIT > 1) {                   // the takers' exchange
      cluster_barrier();
      cluster_barrier();
    }
  } else if (warp >= kTakers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kTurnerRegs));
    // This thread's pieces: 16 codes from 16 * seg of a row.  Eight lanes
    // that load or store together have eight rows and one seg: swizzled, they
    // lie in different banks.
    constexpr int kPieces = BN / 32;                    // a thread turns of a stage
    const int group = (warp - kTakers) / kGroupWarps;
    const int r0 = (warp % kGroupWarps) * (BN / 8) + (lane & 7), seg0 = lane >> 3;
    const uint32_t from = codes + (uint32_t)group * code_bytes<BN>() + (uint32_t)r0 * 128;
    const uint32_t from0 = from + (uint32_t)((seg0 ^ (lane & 7)) << 4), from1 = from + (uint32_t)(((seg0 + 4) ^ (lane & 7)) << 4);
    const uint32_t put = 2 * kAtomA + (uint32_t)(r0 * 128 + (((2 * seg0) ^ (lane & 7)) << 4));
    int slot = group;
    uint32_t phase = 0, codes_phase = 0;
    int stage = group;
    bool ok = true;
    for (int tile = pair; tile < tiles.total && ok; tile += pairs, stage -= stages) {
      for (; stage < stages; stage += kGroups) {
        uint4 held[kPieces];
        ok = __all_sync(0xFFFFFFFFu, wait_on(codes_full + 8 * group, codes_phase, &give_up));
        if (!ok) break;
        codes_phase ^= 1;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)               // two pieces of each eighth row
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(held[i].x), "=r"(held[i].y), "=r"(held[i].z), "=r"(held[i].w)
                       : "r"((i & 1 ? from1 : from0) + (i >> 1) * 1024) : "memory");
        ok = __all_sync(0xFFFFFFFFu, wait_on(empty + 8 * slot, phase ^ 1u, &give_up));
        if (!ok) break;
        const uint32_t base = ring + slot * stage_bytes<BN>() + put;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
          const int i = kPieces - 1 - n;                // the last loaded first:
          const uint32_t to = base + (i >> 1) * 1024 + (i & 1 ? kAtomB : 0);
          uint32_t h[8];
          codes_to_f16(held[i].x, h[0], h[1]);
          codes_to_f16(held[i].y, h[2], h[3]);
          codes_to_f16(held[i].z, h[4], h[5]);
          codes_to_f16(held[i].w, h[6], h[7]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(to ^ 16u), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
          if (n == 0) {                 // where it has arrived, all have, and the slot can be filled
            __syncwarp();               // again (a copy overtakes loads that no one has used yet)
            if (lane == 0) arrive_here(codes_free + 8 * group);
          }
        }
        fence_proxy_async();
        if (warp % kGroupWarps == 0)    // one warp vouches for the tokens' copy too
          ok = __all_sync(0xFFFFFFFFu, wait_on(landed + 8 * slot, phase, &give_up));
        if (!ok) break;
        __syncwarp();
        if (lane == 0 && !(tiles.hold && blockIdx.x == 0 && warp == kTakers)) arrive_first(full + 8 * slot, first_rank);
        slot += kGroups;
        if (slot >= kStages) {
          slot -= kStages;
          phase ^= 1;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_gave_up, 1);
    if (SPLIT > 1) {
      cluster_barrier();
      cluster_barrier();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kTakerRegs));
    int sum[ONE ? 1 : kCols];
    uint32_t chunk = 0;
    bool ok = true;
    const uint32_t my_tmem = tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)(warp >> 2) * kCols;
    for (int tile = pair; tile < tiles.total; tile += pairs) {
      // The last tile's scales have been used; and if a warp has given up, all
      // leave here, so that no one waits for it at the barriers.
      ok = takers_all(ok);
      if (!ok) break;
      const Place at = place_of(tiles, tile);
      const int r = (warp & 3) * 32 + lane, col0 = (warp >> 2) * kCols;     // in the block's tile
      const int64_t t = (int64_t)at.row * 256 + half * kRows + r;
      const int64_t c0 = (int64_t)at.col * BN + col0;
      const bool there = t < p.tokens;
      // Read now, used after the sums: a channel's scale, this thread's token's.
      static_assert(BN == 32 * kTakers, "a channel each");
      const float channel = (int64_t)at.col * BN + tid < p.channels
                                ? p.w_scales[at.rank * p.rank_w_scales + (int64_t)at.col * BN + tid] : 0.f;
      const float token = there ? p.a_scales[at.rank * p.rank_a_scales + t] : 0.f;
      T* out = static_cast<T*>(p.out) + at.rank * p.rank_out;
      channel_scales[tid] = channel;
      takers_all(true);
      const uint32_t my_scales = smem_addr(channel_scales) + 4 * col0;
      for (int c = 0; c < chunks; ++c, ++chunk) {
        const uint32_t b = chunk & 1;
        ok = __all_sync(0xFFFFFFFFu, wait_on(sums_full + 8 * b, (chunk >> 1) & 1, &give_up));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (ONE) {
#pragma unroll 1
          for (int j = 0; j < kCols; j += kLine) {      // rolled: code that runs once a tile is fetched each time
            uint32_t words[8 * kUnits];
#pragma unroll
            for (int n = 0; n < kLine; n += 16) {
              float v[16];
              tmem_load16(my_tmem + b * BN + j + n, v);
              scale_sums<T>(v, my_scales + 4 * (j + n), token, words + n * sizeof(T) / 4);
            }
            store_rows<T, kUnits, ONE>(p, out, t, c0 + j, lane, words, out_align);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCols; j += 16) {
            float v[16];
            tmem_load16(my_tmem + b * BN + j, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int x = __float2int_rn(v[i]);
              sum[j + i] = c == 0 ? x : sum[j + i] + x;
            }
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_first(sums_empty + 8 * b, first_rank);
      }
      if constexpr (SPLIT > 1) {
        constexpr int kOwn = BN / SPLIT;                // columns of a pair
        cluster_barrier();                              // every ring is free
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          const int owner = (col0 + j) / kOwn;
          if (owner == split) continue;
          const int from = split < owner ? split : split - 1;
          const uint32_t to = ring + (uint32_t)((from * (kOwn / 4) + (col0 + j - owner * kOwn) / 4) * kRows + r) * 16u;
          asm volatile(
              "{\n\t.reg .b32 at;\n\t"
              "mapa.shared::cluster.u32 at, %0, %1;\n\t"
              "st.shared::cluster.v4.b32 [at], {%2, %3, %4, %5};\n\t}"
              :: "r"(to), "r"(2 * owner + half), "r"(sum[j]), "r"(sum[j + 1]), "r"(sum[j + 2]), "r"(sum[j + 3])
              : "memory");
        }
        cluster_barrier();
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          if ((col0 + j) / kOwn != split) continue;
#pragma unroll
          for (int from = 0; from < SPLIT - 1; ++from) {
            int v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(ring + (uint32_t)((from * (kOwn / 4) + (col0 + j - split * kOwn) / 4) * kRows + r) * 16u)
                         : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[j + i] += v[i];
          }
        }
      }
      if constexpr (!ONE) {
#pragma unroll
        for (int j = 0; j < kCols; j += kLine) {
          if (!ok) break;
          if (SPLIT > 1 && (col0 + j) / (BN / SPLIT) != split) continue;
          uint32_t words[8 * kUnits];
#pragma unroll
          for (int n = 0; n < kLine; n += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __int2float_rn(sum[j + n + i]);
            scale_sums<T>(v, my_scales + 4 * (j + n), token, words + n * sizeof(T) / 4);
          }
          store_rows<T, kUnits, ONE>(p, out, t, c0 + j, lane, words, out_align);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_gave_up, 1);
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_barrier();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kIssuer)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(2 * BN) : "memory");
}

// CUDA's encoder of tensor maps, looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t encoder(EncodeTiled* out) {
  static std::atomic<void*> known{nullptr};
  void* f = known.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || f == nullptr) return cudaErrorNotSupported;
    known.store(f, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeTiled>(f);
  return cudaSuccess;
}

// The channels' codes as a tensor of depth x channels x ranks, taken in boxes
// of 128 codes x BN / 2 channels, rows swizzled; zeros outside.
template <int BN>
cudaError_t channels_map(const ProductArgs& p, CUtensorMap* map) {
  EncodeTiled encode = nullptr;
  cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  const int64_t ranks = p.rank_w == 0 ? 1 : p.ranks;
  const int64_t ld = p.channels > 1 ? p.ld_w : (p.depth + 15) / 16 * 16;
  const cuuint64_t dims[3] = {(cuuint64_t)p.depth, (cuuint64_t)p.channels, (cuuint64_t)ranks};
  const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)(ranks > 1 ? p.rank_w : ld)};
  const cuuint32_t box[3] = {kStageDepth, BN / 2, 1}, every[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(p.w), dims, strides, box, every,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int BN, int SPLIT, bool ONE>
struct Launch {
  static cudaError_t prepare() {
    static OncePerDevice prepared;
    return prepared.run([] {
      return cudaFuncSetAttribute(product_pair_kernel<T, BN, SPLIT, ONE>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<BN>());
    });
  }
  static cudaLaunchConfig_t config(int clusters, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * SPLIT * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<BN>();
    cfg.stream = s;
    return cfg;
  }
  // Clusters that can run at once on the current device: clusters lie inside
  // a GPC, so fewer large ones fit than its SMs would hold.
  static cudaError_t at_once(int* clusters) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *clusters = known[dev & 63].load(std::memory_order_relaxed);
    if (*clusters) return cudaSuccess;
    if ((e = prepare()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = config(1, nullptr);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2 * SPLIT;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, product_pair_kernel<T, BN, SPLIT, ONE>, &cfg);
    if (e == cudaSuccess) known[dev & 63].store(*clusters, std::memory_order_relaxed);
    return e;
  }
  static cudaError_t run(const ProductArgs& p, const Tiles& t, const CUtensorMap& map, const ProductLayout& l,
                         cudaStream_t s) {
    cudaError_t e = prepare();
    if (e != cudaSuccess) return e;
    const int pairs = l.sms / 2;
    cudaLaunchConfig_t cfg = config(SPLIT > 1 || t.total < pairs ? t.total : pairs, s);
    cudaLaunchAttribute overlapped = overlapped_launch();
    cfg.attrs = &overlapped;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, product_pair_kernel<T, BN, SPLIT, ONE>, p, t, l.out_align, map);
  }
};

}  // namespace

template <>
cudaError_t launch_pair<ECHO_ELEM>(const ProductArgs& p, const ProductLayout& l, cudaStream_t s) {
  constexpr int BN = 256;
  using T = ECHO_ELEM;
  CUtensorMap map = {};
  cudaError_t e = channels_map<BN>(p, &map);
  if (e != cudaSuccess) return e;
  Tiles t;
  t.rows = (int)((p.tokens + 255) / 256);
  t.cols = (int)((p.channels + BN - 1) / BN);
  const int64_t total = (p.tokens + 255) / 256 * ((p.channels + BN - 1) / BN) * p.ranks;
  if (total > 0x7FFFFFFF) return cudaErrorInvalidValue;       // past any memory's results
  t.per_rank = t.rows * t.cols;
  t.total = (int)total;
  t.hold = l.hold;
  // Pairs that share a tile's depth, where the clusters all run at once and
  // each pair has two stages at least.  256 x 4096 x 4096, 16 tiles: alone
  // 25 us, two to a tile 21; four do not fit at once, and take 34.
  const int64_t stages = wide_blocks(p.depth);
  int room = 0;
  if (total * 2 <= l.sms / 2 && stages >= 8) {
    if ((e = Launch<T, BN, 4, false>::at_once(&room)) != cudaSuccess) return e;
    if (total <= room) return Launch<T, BN, 4, false>::run(p, t, map, l, s);
  }
  if (total * 2 <= l.sms / 2 && stages >= 4) {
    if ((e = Launch<T, BN, 2, false>::at_once(&room)) != cudaSuccess) return e;
    if (total <= room) return Launch<T, BN, 2, false>::run(p, t, map, l, s);
  }
  return stages <= kChunkStages ? Launch<T, BN, 1, true>::run(p, t, map, l, s)
                                : Launch<T, BN, 1, false>::run(p, t, map, l, s);
}

template <>
cudaError_t read_gave_up<ECHO_ELEM>(int* word, cudaStream_t s) {
  void* at = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  return e == cudaSuccess ? cudaMemcpyAsync(word, at, sizeof(int), cudaMemcpyDeviceToHost, s) : e;
}

template <>
cudaError_t clear_gave_up<ECHO_ELEM>(cudaStream_t s) {
  void* at = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  return e == cudaSuccess ? cudaMemsetAsync(at, 0, sizeof(int), s) : e;
}

}  // namespace echo
