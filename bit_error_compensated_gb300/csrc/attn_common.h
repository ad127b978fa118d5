// attn_common.h -- how echo_attention's work is cut (attn_*.cu): rows of
// queries into units, the keys that a unit sees into tiles, and the tiles of
// all units into one even range for each block.
#pragma once

#include "serve_common.h"

namespace echo {

constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.4028234663852886e38f;      // a maximum before any key
constexpr float kNone = -INFINITY;

// Rows of queries that share a head of the cache: row r of a sequence is query
// head r % group of its token r / group.  A unit is R consecutive rows of one
// sequence and head, its tiles are the TILE keys at a time from the first to
// the last that any of its rows sees (one tile at least, so that every row is
// somebody's to write).
struct Unit {
  int sequence, head, first, rows;       // rows of queries [first, first + rows)
  int tile, tiles;
};

// Keys [from, to) that the row at a place sees.
__device__ __forceinline__ int keys_to(const AttentionArgs& a, const Sequence& s, int place) {
  if (!a.causal) return place < 0 ? 0 : s.keys;
  return place + 1 < 0 ? 0 : (place + 1 < s.keys ? place + 1 : s.keys);
}
__device__ __forceinline__ int keys_from(const AttentionArgs& a, int place) {
  return a.window && place >= a.window ? place - a.window + 1 : 0;
}

template <int R, int TILE>
__device__ __forceinline__ void unit_tiles(const AttentionArgs& a, const Sequence& s, int j, int* tile, int* tiles) {
  const int rows = s.rows * a.group, last = (j + 1) * R < rows ? (j + 1) * R : rows;
  const int from = keys_from(a, s.place + j * R / a.group) / TILE;
  const int to = (keys_to(a, s, s.place + (last - 1) / a.group) + TILE - 1) / TILE;
  *tile = from;
  *tiles = to > from ? to - from : 1;
}
// The unit that is walked j-th of `units`: first, last, second, last but one and
// so on.  In a prompt the first units see few keys and the last many, and each
// costs its rows' loads and stores besides its tiles: so all blocks have about
// as many.
__device__ __forceinline__ int unit_at(int j, int units) { return j & 1 ? units - 1 - (j >> 1) : j >> 1; }
template <int R>
__device__ __forceinline__ int units_of(const AttentionArgs& a, const Sequence& s) {
  return (s.rows * a.group + R - 1) / R;
}
// Tiles of all units of a sequence and one head, for each lane's own sequence
// (rows 0: none); of a whole warp, whose lanes share the units where there are
// many.
template <int R, int TILE>
__device__ __forceinline__ int64_t sequence_tiles(const AttentionArgs& a, const Sequence& s, int lane) {
  const int units = units_of<R>(a, s);
  int64_t n = 0;
  const bool many = units > 4;
  if (!many)
    for (int j = 0; j < units; ++j) {
      int tile, tiles;
      unit_tiles<R, TILE>(a, s, j, &tile, &tiles);
      n += tiles;
    }
  for (uint32_t left = __ballot_sync(kFull, many); left; left &= left - 1) {
    const int owner = __ffs(left) - 1;
    Sequence of = s;
    of.rows = __shfl_sync(kFull, s.rows, owner);
    of.keys = __shfl_sync(kFull, s.keys, owner);
    of.place = __shfl_sync(kFull, s.place, owner);
    int64_t sum = 0;
    for (int j = lane; j < units_of<R>(a, of); j += 32) {
      int tile, tiles;
      unit_tiles<R, TILE>(a, of, j, &tile, &tiles);
      sum += tiles;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    if (lane == owner) n = sum;
  }
  return n;
}

// A block's range of the tiles of all units, which are ordered by sequence,
// head, and rows: block c of n has tiles [c T / n, (c + 1) T / n) of T (n no
// more than T), so that its first and its last unit may be shared with others.
struct Range {
  int64_t total, begin, end;             // tiles
  int blocks;                            // that have any
  int sequence;                          // that has `begin`
  int64_t before;                        // tiles of the sequences before it
  int64_t each;                          // tiles of a head of that sequence
  Sequence s;                            // that sequence
};
__device__ __forceinline__ int64_t range_begin(int64_t total, int block, int blocks) { return divided(total * block, blocks); }
// The block whose range has a tile (the last that begins at or before it).
__device__ __forceinline__ int block_of(int64_t total, int64_t tile, int blocks) {
  return (int)divided((tile + 1) * blocks - 1, total);
}

// Of a whole block of THREADS threads.  LEAST: tiles that a block has at least
// where there are few.  `shared`: THREADS / 16 + 3 words of 8 bytes.
//
// Starts that fall and rise again may give several sequences the same rows.  Where
// these are more in sum than there are tokens, nothing is computed or counted: a
// large batch's could keep the kernel busy for hours.
template <int R, int TILE, int THREADS, int LEAST>
__device__ __forceinline__ Range block_range(const AttentionArgs& a, int64_t* shared, int* bad) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.batch.sequences;
  Range r;
  r.s = {0, 0, 0, 0, 0};
  auto divide = [&](int64_t rows) {
    if (rows > a.batch.tokens) {
      *bad |= kBadRows;
      r.total = 0;
    }
    r.blocks = r.total < (int64_t)gridDim.x * LEAST ? (int)((r.total + LEAST - 1) / LEAST) : (int)gridDim.x;
    const int c = (int)blockIdx.x < r.blocks ? blockIdx.x : r.blocks;
    r.begin = r.blocks ? range_begin(r.total, c, r.blocks) : 0;
    r.end = c < r.blocks ? range_begin(r.total, c + 1, r.blocks) : r.begin;
    r.sequence = 0;
    r.before = 0;
    r.each = 1;
  };
  if (n <= 32) {                         // each warp for itself, a lane a sequence
    if (lane < n) r.s = sequence_of(a.batch, a.cache.page_shift, lane, bad);
    const int64_t rows = __reduce_add_sync(kFull, (uint32_t)r.s.rows);     // 32 times 2^20 at the most
    const int64_t each = rows > a.batch.tokens ? 0 : sequence_tiles<R, TILE>(a, r.s, lane), mine = each * a.cache.heads;
    int64_t prefix = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t other = __shfl_up_sync(kFull, prefix, off);
      if (lane >= off) prefix += other;
    }
    r.total = __shfl_sync(kFull, prefix, 31);
    divide(rows);
    if (r.begin == r.end) return r;
    const int owner = __ffs(__ballot_sync(kFull, prefix > r.begin)) - 1;
    r.sequence = owner;
    r.before = __shfl_sync(kFull, prefix - mine, owner);
    r.each = __shfl_sync(kFull, each, owner);
    r.s.row = __shfl_sync(kFull, r.s.row, owner);
    r.s.rows = __shfl_sync(kFull, r.s.rows, owner);
    r.s.length = __shfl_sync(kFull, r.s.length, owner);
    r.s.keys = __shfl_sync(kFull, r.s.keys, owner);
    r.s.place = __shfl_sync(kFull, r.s.place, owner);
    return r;
  }
  int64_t mine = 0, sum = 0, rows = 0;   // tiles of the last sequence looked at; tiles, and rows, of all that this thread has
  auto tiles_of = [&](int i, int* report, int64_t* rows) {
    Sequence s = {0, 0, 0, 0, 0};
    if (i < n) s = sequence_of(a.batch, a.cache.page_shift, i, report);
    *rows += s.rows;
    if (__any_sync(kFull, *rows > a.batch.tokens)) return (int64_t)0;
    return sequence_tiles<R, TILE>(a, s, lane) * a.cache.heads;
  };
  for (int i0 = 0; i0 < n; i0 += THREADS) {
    mine = tiles_of(i0 + tid, bad, &rows);
    sum += mine;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, off);
    rows += __shfl_xor_sync(kFull, rows, off);
  }
  if (lane == 0) {
    shared[warp] = sum;
    shared[kWarps + 3 + warp] = rows;
  }
  __syncthreads();
  r.total = 0;
  int64_t all_rows = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    r.total += shared[w];
    all_rows += shared[kWarps + 3 + w];
  }
  divide(all_rows);
  if (r.begin == r.end) return r;        // the whole block
  // The sequence that has `begin`: prefix sums of THREADS sequences at a time.
  int64_t before = 0;
  for (int i0 = 0; i0 < n; i0 += THREADS) {
    const int i = i0 + tid;
    int ignored = 0;
    int64_t these = 0;
    if (n > THREADS) mine = tiles_of(i, &ignored, &these);
    int64_t prefix = mine;               // inclusive, of the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t other = __shfl_up_sync(kFull, prefix, off);
      if (lane >= off) prefix += other;
    }
    __syncthreads();
    if (lane == 31) shared[warp] = prefix;
    __syncthreads();
    int64_t block = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) prefix += shared[w];
      block += shared[w];
    }
    if (before + prefix > r.begin && before + prefix - mine <= r.begin) {
      shared[kWarps] = i;
      shared[kWarps + 1] = before + prefix - mine;
      shared[kWarps + 2] = mine / a.cache.heads;
    }
    before += block;
    if (before > r.begin) break;
  }
  __syncthreads();
  r.sequence = (int)shared[kWarps];
  r.before = shared[kWarps + 1];
  r.each = shared[kWarps + 2];
  int ignored = 0;
  r.s = sequence_of(a.batch, a.cache.page_shift, r.sequence, &ignored);
  __syncthreads();
  return r;
}

// Walks the units of a block's range: `unit` is the one at hand, the block has
// `take` of its tiles from its tile `in` on.  Every thread walks for itself, its
// warp together.
template <int R, int TILE>
struct Walk {
  int64_t at, end;
  Sequence s;
  Unit unit;
  int j, in, take;                       // units of the head before, tiles of the unit before, tiles of it that are the block's

  __device__ __forceinline__ void start(const AttentionArgs& a, const Range& r) {
    at = r.begin;
    end = r.end;
    if (at >= end) return;
    unit.sequence = r.sequence;
    s = r.s;
    unit.head = (int)divided(at - r.before, r.each);
    int64_t left = at - r.before - unit.head * r.each;
    // The unit that has this tile: a warp's lanes look at 32 at a time.
    const int lane = threadIdx.x & 31, units = units_of<R>(a, s);
    for (j = 0;; j += 32) {
      int tile = 0, tiles = 0;
      if (j + lane < units) unit_tiles<R, TILE>(a, s, unit_at(j + lane, units), &tile, &tiles);
      int64_t prefix = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t other = __shfl_up_sync(kFull, prefix, off);
        if (lane >= off) prefix += other;
      }
      const uint32_t past = __ballot_sync(kFull, prefix > left);
      if (past == 0 && j + 32 < units) {
        left -= __shfl_sync(kFull, prefix, 31);
        continue;
      }
      const int k = past ? __ffs(past) - 1 : 0;
      left -= __shfl_sync(kFull, prefix - tiles, k);
      j += k;
      break;
    }
    in = (int)left;
    enter(a);
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ bool whole() const { return in == 0 && take == unit.tiles; }
  __device__ __forceinline__ void next(const AttentionArgs& a, int* bad) {
    at += take;
    if (at >= end) return;               // else the unit has been walked to its end
    in = 0;
    if (++j == units_of<R>(a, s)) {
      j = 0;
      if (++unit.head == a.cache.heads) {
        unit.head = 0;
        do s = sequence_of(a.batch, a.cache.page_shift, ++unit.sequence, bad);
        while (s.rows == 0);
      }
    }
    enter(a);
  }

 private:
  __device__ __forceinline__ void enter(const AttentionArgs& a) {
    const int u = unit_at(j, units_of<R>(a, s));
    unit_tiles<R, TILE>(a, s, u, &unit.tile, &unit.tiles);
    unit.first = u * R;
    unit.rows = s.rows * a.group - unit.first < R ? s.rows * a.group - unit.first : R;
    take = unit.tiles - in < end - at ? unit.tiles - in : (int)(end - at);
  }
};

// Workspace: two slots a block, for the parts of its first and its last unit
// (R rows of maximum, sum and D sums of values, fp32), and what to join.
struct Join {
  int blocks;                            // that share the unit: this one and the ones behind it; 0: none
  int slot;                              // of this block's part
  int row, head, first, rows;            // first token row of the sequence; the unit
};
__host__ __device__ inline int64_t slot_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }
__host__ __device__ inline int64_t join_bytes(int blocks) { return ((int64_t)blocks * sizeof(Join) + 255) / 256 * 256; }
inline int64_t workspace_bytes(int blocks, int rows, int dim) {
  return join_bytes(blocks) + 2 * (int64_t)blocks * slot_floats(rows, dim) * 4;
}
__device__ __forceinline__ Join* joins(const AttentionArgs& a) { return reinterpret_cast<Join*>(a.partial); }
__device__ __forceinline__ float* slot_at(const AttentionArgs& a, int blocks, int slot, int rows, int dim) {
  return reinterpret_cast<float*>(reinterpret_cast<char*>(a.partial) + join_bytes(blocks)) + slot * slot_floats(rows, dim);
}

// Block c's part of the unit at hand: in slot 2 c if the unit has the block's
// first tile, else in slot 2 c + 1.
template <int R, int TILE>
__device__ __forceinline__ int slot_of(const Walk<R, TILE>& w, const Range& r) {
  return 2 * (int)blockIdx.x + (w.at - w.in > r.begin ? 1 : 0);
}
// The first part's block names the others that have parts of the unit.
template <int R, int TILE>
__device__ __forceinline__ void name_parts(const AttentionArgs& a, const Walk<R, TILE>& w, const Range& r) {
  const int last = block_of(r.total, w.at + w.unit.tiles - 1, r.blocks);
  joins(a)[blockIdx.x] = {last - (int)blockIdx.x + 1, slot_of(w, r), w.s.row, w.unit.head, w.unit.first, w.unit.rows};
}

__device__ __forceinline__ float exp2_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float log2_of(float v) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// What a weight is in f16.  A value's step s is f times a power of two S (value_scale)
// with f from 1 to 2, or less or more than that where s is outside 2^-14 .. 2^6.  The
// matrix instructions take P = w f 2^-m and V = (c - z) S, both in f16, and add
// their products in fp32: (c - z) S is exact, P has 11 bits, and the sum of weights
// takes P / f in fp32.  (With all of s in P a key of a large step and weight pushes
// the other keys' weights below f16's least: a row of zeros has a step of 1 by
// definition.)
//
// A row's m is raised when a score passes it by kMostWeight, so weights are 2^15 at
// the most, and then to AHEAD above the score less kMostWeight.  So the weight that
// raises it is a power of two, 2^(15 - AHEAD), and exact: where one key has most of a
// row, nothing is lost of it.  11 bits are left to weights down to 2^-14, those below
// have a step of 2^-24: with AHEAD 4 and 8, 2^-25 and 2^-21, and 2^-35 and 2^-31, of
// the largest.
constexpr float kMostWeight = 15.0f;
template <int AHEAD>
__device__ __forceinline__ float raised(float m, float top) { return fmaxf(m, top - (kMostWeight - AHEAD)); }

// A value's step.  A place that was never written may have a step of 0 and codes
// of 0: its value adds nothing, but its weight counts.  With a step far below fp16's
// least the weight's part of the sum is exact and its product with the value rounds
// to nothing.  NaN stays NaN.
__device__ __forceinline__ float value_step(uint32_t meta) { return max_nan(meta_step(meta), 0x1p-60f); }
// S as f16 bits, the step's power of two within 2^-14 .. 2^5: with it both 1024 + z
// and a single code are f16 numbers that are no subnormals, which matrix
// instructions would align like 2^-14.
__device__ __forceinline__ uint32_t value_scale(uint32_t meta) { return min(max(meta & 0x7C00u, 0x0400u), 0x5000u); }
// f = s / S, exactly.
__device__ __forceinline__ float value_factor(uint32_t meta) {
  return __fmul_rn(value_step(meta), __uint_as_float(((127u + 15u) << 23) - (value_scale(meta) << 13)));
}

// Query rows as f16, scaled by a power of two that takes the row's largest
// element to [2^14, 2^15): bf16 values stay exact down to 2^-31 of it (f16's
// subnormals begin 2^-29 below and hold 2^-39 of it).
__device__ __forceinline__ float row_factor(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);                  // biased
  if (e == 255) return 1.0f;
  return __uint_as_float((uint32_t)(127 + 14 + 127 - (e < 27 ? 27 : e)) << 23);
}

// One value of a result row in out's type.
__device__ __forceinline__ void store_value(const AttentionArgs& a, int64_t at, float v) {
  if (a.dtype == ECHO_BF16) static_cast<__nv_bfloat16*>(a.out.data)[at] = from_float<__nv_bfloat16>(v);
  else static_cast<__half*>(a.out.data)[at] = from_float<__half>(v);
}
__device__ __forceinline__ void store_values4(const AttentionArgs& a, int64_t at, const float (&v)[4], bool vector) {
  if (!vector) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_value(a, at + i, v[i]);
  } else if (a.dtype == ECHO_BF16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out.data) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    const __half2 lo = __floats2half2_rn(v[0], v[1]), hi = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<__half*>(a.out.data) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}
// Whether rows of out take 8-byte stores.
inline bool vector_rows(const HeadsArgs& h) { return on_boundary(h.data, 8) && h.ld % 4 == 0 && h.head_stride % 4 == 0; }

// Blocks that can have a tile, of `most`: a small batch is not waited for by
// blocks that only find out that they have nothing to do.
inline int useful_blocks(const AttentionArgs& a, int rows, int tile, int most) {
  const int64_t units = a.cache.heads * (((int64_t)a.batch.tokens * a.group + rows - 1) / rows + a.batch.sequences);
  const int64_t keys = (int64_t)a.batch.table_pages << a.cache.page_shift, tiles = keys / tile + 1;
  if (units >= most || tiles >= most) return most;
  return (int)(units * tiles < most ? units * tiles : most);
}

// Joins the parts of units that several blocks of a kernel before have had.
cudaError_t launch_join(const AttentionArgs& a, int blocks, int rows, cudaStream_t s);
// attn_many.cu; attn_few.cu has the rest.
cudaError_t launch_attention_many(const AttentionArgs& a, int sms, cudaStream_t s);
int64_t attention_many_bytes(int head_dim, int sms);

}  // namespace echo
