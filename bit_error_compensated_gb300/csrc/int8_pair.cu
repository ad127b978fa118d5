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
// (tcgen05 cta_group::2): each block turns 128 rows of tokens and BN / 2 rows
// of channels, which halves what goes through its shared memory per product.
// In a block, eight warps load 16-byte pieces of codes a stage ahead into
// registers, turn and store them (the 128-byte-swizzled K-major layout the
// matrix instruction reads), and in between take the last chunk's sums out of
// TMEM, 32 columns a stage; one thread of the first block issues the matrix
// instructions.  TMEM holds two chunks' sums, so one is taken out while the
// next is computed.
//
// Every wait is bounded; one that gives up ends the call with a status
// (echo_matmul_status).
#include "int8_load.h"
#include "tma.cuh"

namespace echo {
namespace {

constexpr int kRows = 128;              // tokens a block holds of the pair's 256
constexpr int kStageDepth = 128;        // codes of a row per stage: two swizzle atoms of f16
constexpr int kStages = 3;
constexpr int kChunkStages = 8;         // 1024 codes: exact in fp32
constexpr int kWorkers = 8;             // warps that convert and store results
constexpr int kThreads = 32 * (kWorkers + 4);   // three warpgroups; of the last, one warp works
// Registers: the block starts with 168 a thread (three warpgroups of 504 in
// all); a worker holds 128 sums, two stages' codes and 16 columns.
constexpr int kWorkerRegs = 224, kIssuerRegs = 40;
static_assert(2 * kWorkerRegs + kIssuerRegs <= 3 * 168, "a split above the launch's registers never ends");
constexpr int kStep = 32;               // columns taken out of TMEM after a stage

template <int BN> constexpr int stage_bytes() { return (kRows + BN / 2) * 2 * kStageDepth; }
template <int BN> constexpr int smem_bytes() { return kStages * stage_bytes<BN>() + 1024; }

// Set by a block whose wait gave up, until echo_matmul_status clears it.
__device__ int g_gave_up;

struct Tiles {
  int64_t rows, cols, per_rank, total;  // of 256 tokens, BN channels
};

struct Place {
  int64_t rank, row, col;
};
// Tiles in groups of eight along the tokens, so that the pairs at work at one
// time read few different rows of either operand.
__device__ __forceinline__ Place place_of(const Tiles& t, int64_t tile) {
  Place p;
  p.rank = tile / t.per_rank;
  const int64_t i = tile - p.rank * t.per_rank, group = i / (8 * t.cols);
  const int64_t first = group * 8, high = t.rows - first < 8 ? t.rows - first : 8;
  const int64_t j = i - group * 8 * t.cols;
  p.col = j / high;
  p.row = first + j - p.col * high;
  return p;
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  // K-major, 128-byte swizzle: rows of 128 bytes in groups of eight, 1024 bytes apart
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* give_up) {
  uint64_t began = 0;
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    if (*give_up) return false;
    const uint64_t t = global_ns();
    if (began == 0) began = t;
    else if (t - began > kWaitLimitNs) {
      *give_up = 1;
      return false;
    }
  }
}

// Arrives on a barrier of this block; what its threads wrote is visible to
// the block's waiters.
__device__ __forceinline__ void arrive_here(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// Arrives on a barrier of the pair's first block.  Releasing to the cluster
// waits for the thread's loads in flight, so only the issuing warps do it.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 at;\n\t"
      "mapa.shared::cluster.u32 at, %0, 0;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [at];\n\t}"
      :: "r"(bar) : "memory");
}

// The same for a thread that has nothing in memory to publish.
__device__ __forceinline__ void arrive_first_relaxed(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 at;\n\t"
      "mapa.shared::cluster.u32 at, %0, 0;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [at];\n\t}"
      :: "r"(bar) : "memory");
}

// All matrix instructions issued so far will arrive on `bar` of both blocks.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" :: "r"(bar), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(desc), "r"(add) : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 results of one token, from channel c.
template <typename T>
__device__ __forceinline__ void store_results(const ProductArgs& p, int64_t rank, T* row, int64_t c,
                                              const int* sum, float token, bool wide) {
  const float* scales = p.w_scales + rank * p.rank_w_scales + c;
  if (wide && c + 16 <= p.channels) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < 16; j += N) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = scaled_sum(sum[j + i], token, __ldg(scales + j + i));
      store_floats<T, N>(row + c + j, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < p.channels) row[c + i] = from_float<T>(scaled_sum(sum[i], token, __ldg(scales + i)));
  }
}

template <typename T, int BN, bool ALIGNED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
product_pair_kernel(const ProductArgs p, const Tiles tiles, const int wide) {
  constexpr int kPieces = 4 + BN / 64;                  // a thread loads of a stage: tokens', channels' rows
  constexpr uint32_t kAtomA = kRows * 128, kAtomB = BN / 2 * 128;         // 64 codes of every row
  constexpr int kSteps = BN / 2 / kStep;                // to take out a chunk's sums
  constexpr uint32_t kInstr = (1u << 4) | ((uint32_t)(BN / 8) << 17) | (16u << 24);  // f16, fp32 sums, 256 x BN
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_at;
  __shared__ volatile int give_up;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, sums_full = empty + 8 * kStages,
                 sums_empty = sums_full + 16, last = sums_empty + 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = (int)(blockIdx.x & 1);               // of the pair
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int64_t stages = (p.depth + kStageDepth - 1) / kStageDepth;       // of a tile
  const int64_t chunks = (stages + kChunkStages - 1) / kChunkStages;
  const int64_t chunk_stages = (stages + chunks - 1) / chunks;            // the last may have fewer
  const int64_t mine = pair < tiles.total ? (tiles.total - 1 - pair) / pairs + 1 : 0;

  if (tid == 0) {
    give_up = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, kWorkers + (half == 0 ? 1 : 0));   // and the second block's word
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sums_full + 8 * b, 1);
      mbar_init(sums_empty + 8 * b, 2 * kWorkers);
    }
    mbar_init(last, 1);
    fence_barrier_init();
  }
  if (warp == kWorkers) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(&tmem_at)), "r"(2 * BN) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_at;
  pdl_wait();

  if (warp >= kWorkers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssuerRegs));
    if (warp == kWorkers && half == 0 && lane == 0) {
      // Issues the matrix instructions of the pair.
      int slot = 0;
      uint32_t phase = 0;
      int64_t chunk = 0;
      bool ok = true;
      for (int64_t t = 0; t < mine && ok; ++t) {
        for (int64_t s0 = 0; s0 < stages && ok; s0 += chunk_stages, ++chunk) {
          const int b = (int)(chunk & 1);
          const int64_t n = stages - s0 < chunk_stages ? stages - s0 : chunk_stages;
          ok = wait_on(sums_empty + 8 * b, (uint32_t)((chunk >> 1) & 1) ^ 1u, &give_up);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int64_t s = 0; s < n && ok; ++s) {
            ok = wait_on(full + 8 * slot, phase, &give_up);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t at = ring + slot * stage_bytes<BN>();
#pragma unroll
            for (int k = 0; k < kStageDepth / 16; ++k) {        // 16 codes: 32 bytes on
              const uint64_t da = smem_desc(at + (k / 4) * kAtomA) + 2 * (k % 4);
              const uint64_t db = smem_desc(at + 2 * kAtomA + (k / 4) * kAtomB) + 2 * (k % 4);
              mma_pair(tmem + b * BN, da, db, kInstr, s > 0 || k > 0);
            }
            commit_pair(empty + 8 * slot);
            if (++slot == kStages) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (ok) commit_pair(sums_full + 8 * b);
        }
      }
      if (!ok) {                       // instructions still running end before TMEM is freed
        commit_pair(last);
        give_up = 0;
        wait_on(last, 0, &give_up);
        give_up = 1;
      }
    }
    if (warp == kWorkers && half == 1 && lane == 0) {
      // Tells the first block of each stage that this block has stored.
      int slot = 0;
      uint32_t phase = 0;
      for (int64_t g = 0; g < mine * stages; ++g) {
        if (!wait_on(full + 8 * slot, phase, &give_up)) break;
        arrive_first(full + 8 * slot);
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kWorkerRegs));
    // This thread's pieces: 16 codes from 16 * seg of rows r0 + 32 i.  A
    // quarter of a warp stores four pieces of two rows of one atom: swizzled,
    // they lie in different banks; a row's eight pieces are one 128-byte line.
    const int seg = (lane & 3) + 4 * ((lane >> 3) & 1);
    const int r0 = warp * 4 + ((lane >> 2) & 1) + 2 * (lane >> 4);
    const uint32_t put = (uint32_t)(r0 * 128 + (((2 * (seg & 3)) ^ (r0 & 7)) << 4));
    const uint32_t put_a = put + (seg >> 2) * kAtomA, put_b = put + 2 * kAtomA + (seg >> 2) * kAtomB;
    // The stage to load next: its tile, its depth, its rows.
    int64_t load_tile = pair, load_k = 0;
    const int8_t* row[kPieces];
    // Rows past the last token or channel repeat it: their results are dropped.
    auto find_rows = [&]() {
      const Place at = place_of(tiles, load_tile < tiles.total ? load_tile : pair);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        if (i < 4) {
          const int64_t t = at.row * 256 + half * kRows + r0 + 32 * i;
          row[i] = p.a + at.rank * p.rank_a + (t < p.tokens ? t : p.tokens - 1) * p.ld_a;
        } else {
          const int64_t c = at.col * BN + half * (BN / 2) + r0 + 32 * (i - 4);
          row[i] = p.w + at.rank * p.rank_w + (c < p.channels ? c : p.channels - 1) * p.ld_w;
        }
      }
    };
    uint4 held[kPieces];
    auto load_stage = [&]() {
      const int64_t k = load_k + 16 * seg;
      if (ALIGNED && k + 16 <= p.depth) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) held[i] = __ldg(reinterpret_cast<const uint4*>(row[i] + k));
      } else {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) held[i] = load_codes<ALIGNED>(row[i], k, p.depth);
      }
      load_k += kStageDepth;
      if (load_k >= p.depth) {
        load_k = 0;
        load_tile += pairs;
        find_rows();
      }
    };

    // The chunk whose sums are being taken out.
    int sum[BN / 2];
    int step = kSteps, delay = 0;       // next columns; stages to wait before the first
    int64_t drained = 0;                // chunks taken out, or being so
    bool first = false, final = false;
    Place place = {0, 0, 0};
    bool ok = true;
    const uint32_t my_tmem = tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)(warp >> 2) * (BN / 2);
    auto take_step = [&]() {
      const int64_t chunk = drained - 1;
      const uint32_t b = (uint32_t)(chunk & 1);
      if (step == 0) {
        ok = __all_sync(0xFFFFFFFFu, wait_on(sums_full + 8 * b, (uint32_t)((chunk >> 1) & 1), &give_up));
        if (!ok) return;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s != step) continue;
#pragma unroll
        for (int j = s * kStep; j < (s + 1) * kStep; j += 16) {
          float v[16];
          tmem_load16(my_tmem + b * BN + j, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int x = __float2int_rn(v[i]);
            sum[j + i] = first ? x : sum[j + i] + x;
          }
          if (final) {
            const int64_t t = place.row * 256 + half * kRows + (warp & 3) * 32 + lane;
            const int64_t c = place.col * BN + (warp >> 2) * (BN / 2) + j;
            if (t < p.tokens && c < p.channels)
              store_results<T>(p, place.rank, static_cast<T*>(p.out) + place.rank * p.rank_out + t * p.ld_out,
                               c, sum + j, __ldg(p.a_scales + place.rank * p.rank_a_scales + t), wide);
          }
        }
      }
      if (++step == kSteps) {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_first_relaxed(sums_empty + 8 * b);   // the loads from TMEM are done
      }
    };

    find_rows();
    load_stage();
    int slot = 0;
    uint32_t phase = 0;
    int64_t tile = pair, s_tile = 0, s_chunk = 0;         // the stage being stored
    for (int64_t left = mine * stages; ok; --left) {      // and once more, for the last sums
      if (left > 0) {
        ok = __all_sync(0xFFFFFFFFu, wait_on(empty + 8 * slot, phase ^ 1u, &give_up));
        if (!ok) break;
        const uint32_t base = ring + slot * stage_bytes<BN>();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint32_t at = base + (i < 4 ? put_a + 4096 * i : put_b + 4096 * (i - 4));   // 32 rows on
          uint32_t h[8];
          codes_to_f16(held[i].x, h[0], h[1]);
          codes_to_f16(held[i].y, h[2], h[3]);
          codes_to_f16(held[i].z, h[4], h[5]);
          codes_to_f16(held[i].w, h[6], h[7]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       :: "r"(at ^ 16u), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_here(full + 8 * slot);
        load_stage();
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
        ++s_chunk;
        ++s_tile;
      }
      // A chunk is complete in the ring: the one before it must be out of
      // TMEM now, as the chunk after this one goes where it was.
      const bool end = left > 0 && (s_chunk == chunk_stages || s_tile == stages);
      int take = 1;
      if (end || left == 0) take = kSteps;
      else if (delay > 0) --delay, take = 0;
      for (; take > 0 && step < kSteps && ok; --take) take_step();
      if (left == 0) break;
      if (end) {
        first = s_tile <= chunk_stages;
        final = s_tile == stages;
        if (final) place = place_of(tiles, tile);
        ++drained;
        step = 0;
        delay = kStages;                // until the matrix instructions have caught up
        s_chunk = 0;
        if (final) {
          s_tile = 0;
          tile += pairs;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_gave_up, 1);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kWorkers)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(2 * BN) : "memory");
}

template <typename T, int BN, bool ALIGNED>
cudaError_t launch(const ProductArgs& p, const ProductLayout& l, cudaStream_t s) {
  static OncePerDevice prepared;
  cudaError_t e = prepared.run([] {
    return cudaFuncSetAttribute(product_pair_kernel<T, BN, ALIGNED>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<BN>());
  });
  if (e != cudaSuccess) return e;
  Tiles t;
  t.rows = (p.tokens + 255) / 256;
  t.cols = (p.channels + BN - 1) / BN;
  t.per_rank = t.rows * t.cols;
  t.total = t.per_rank * p.ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (t.total < l.sms / 2 ? t.total : l.sms / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<BN>();
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, product_pair_kernel<T, BN, ALIGNED>, p, t, (int)l.wide);
}

}  // namespace

template <>
cudaError_t launch_pair<ECHO_ELEM>(const ProductArgs& p, const ProductLayout& l, cudaStream_t s) {
  return l.aligned ? launch<ECHO_ELEM, 256, true>(p, l, s) : launch<ECHO_ELEM, 256, false>(p, l, s);
}

template <>
cudaError_t take_gave_up<ECHO_ELEM>(int* word, cudaStream_t s) {
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  if (e == cudaSuccess) e = cudaMemcpyAsync(word, at, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(at, 0, sizeof(int), s);
  return e;
}

}  // namespace echo
