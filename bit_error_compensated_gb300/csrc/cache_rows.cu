// cache_rows.cu -- echo_cache_append and echo_cache_read (include/echo.h).
//
// A head's row of a token is one group: head_dim / 16 lanes hold it, 16 values
// each, so that a warp takes 8, 4 or 2 rows with 16-byte accesses and its
// lanes' shuffles find a row's range.  A warp's rows belong to one token, whose
// sequence its 32 lanes look for together.  A row of 128 in 16 bits is 256 bytes
// in and 68 out (4 bits).  8192 tokens of 8 heads of 128, bf16: written in 15.2 us
// (2.7 TB/s, bound by instructions: range, step, rounding; 18.9 where every lane
// finds its group's step), read in 10.6 to 11.4 (3.7 TB/s); 64 tokens in 3.1 and 2.4.
#include "serve_common.h"

namespace echo {
namespace {

ECHO_STATUS_WORD

constexpr int kWarps = 4;
constexpr int64_t kManySteps = 4 * 152 * 16;      // of the machine's warps, see launch

// Values [8 NL h + 8 q, + 8) of a row, h = 0, 1, as lane q of the row's NL.
template <typename T, int NL>
__device__ __forceinline__ void load_row(const T* row, int q, bool aligned, Pack<T, 8> (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const T* p = row + 8 * NL * h + 8 * q;
    if (aligned) {
      v[h] = load_pack<T, 8>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h].v[i] = p[i];
    }
  }
}

// Which rows of which token a lane works on: warps take G steps of 32 / NL rows
// of a token's 2 * heads.
struct Place {
  int token, row;                // the first; row: head, or heads + head of the values
};
template <int NL, int G>
__device__ __forceinline__ Place place_of(int heads, int lane) {
  constexpr int kRows = 32 / NL * G;
  const int each = (2 * heads + kRows - 1) / kRows;      // warps a token
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  Place p;
  p.token = (int)divided(w, each);
  p.row = (int)(w - (int64_t)p.token * each) * kRows + lane / NL;
  return p;
}

// What only a look at all starts shows.
__device__ __forceinline__ void check_starts(const BatchArgs& b) {
  if (blockIdx.x != 0) return;
  bool bad = false;
  for (int i = threadIdx.x; i < b.sequences; i += 32 * kWarps)
    bad |= b.starts[i] < 0 || b.starts[i + 1] < b.starts[i] || b.starts[i + 1] > b.tokens;
  if (bad) report(kBadRows);
}

// The place of a token in its sequence, or -1, and whether it is a batch's at all.
__device__ __forceinline__ bool token_place(const BatchArgs& b, int page_shift, int t, int lane, int* sequence,
                                            int* place) {
  const int i = sequence_at(b, t, lane);
  if (i < 0 || i >= b.sequences) return false;
  int bad = 0;
  const Sequence s = sequence_of(b, page_shift, i, &bad);
  if (t < s.row || t >= s.row + s.rows) return false;
  *sequence = i;
  *place = s.place + (t - s.row);
  return true;
}

template <typename T, int NL, int G>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const RowsArgs a, const int aligned) {
  constexpr int kStep = 32 / NL;
  pdl_wait();
  pdl_trigger();
  check_starts(a.batch);
  const int lane = threadIdx.x & 31, q = lane % NL, heads = a.cache.heads;
  const Place p = place_of<NL, G>(heads, lane);
  if (p.token >= a.batch.tokens) return;                 // the whole warp
  Pack<T, 8> v[G][2];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int row = p.row + i * kStep;
    if (row >= 2 * heads) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[i][k / 8].v[k % 8] = from_float<T>(0.0f);
      continue;
    }
    const HeadsArgs& from = row >= heads ? a.v : a.k;
    load_row<T, NL>(static_cast<const T*>(from.data) + p.token * from.ld + (row >= heads ? row - heads : row) * from.head_stride,
                    q, aligned, v[i]);
  }
  __syncwarp();
  int sequence, place;
  if (!token_place(a.batch, a.cache.page_shift, p.token, lane, &sequence, &place) || place < 0) return;
  const int page = page_of(a.batch, a.cache, sequence, place);
  if (page < 0) {
    if (lane == 0) report(kBadPage);
    return;
  }
  const float L = a.cache.bits == 4 ? 15.0f : 255.0f;
  float lo[G], hi[G];
#pragma unroll
  for (int i = 0; i < G; ++i) range_of<T>(v[i], lo[i], hi[i]);
  const GroupStep mine = shared_step<NL, G>(lo, hi, q, L);
  // (the values' groups of a page follow its keys')
  if (q < G && p.row + q * kStep < 2 * heads) {
    a.cache.meta[group_index(a.cache, page, p.row + q * kStep, place)] = mine.meta;
    if (!mine.finite) report(kNaNGroup);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int row = p.row + i * kStep;
    if (p.row - lane / NL + i * kStep >= 2 * heads) break;               // the whole warp
    const GroupStep g = step_at<NL, G>(mine, i);
    if (row >= 2 * heads) continue;
    const int64_t at = group_index(a.cache, page, row, place);
    uint8_t* codes = a.cache.codes + at * (2 * NL * a.cache.bits);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = 8 * NL * h + 8 * q;
      float eight[8];
      to_floats<T, 8>(v[i][h], eight);
      uint32_t low, high;
      if (a.cache.bits == 4) {
        group_codes8<4>(eight, g, low, high);
        *reinterpret_cast<uint32_t*>(codes + first / 2) = low | high << 16;
      } else {
        group_codes8<8>(eight, g, low, high);
        *reinterpret_cast<uint2*>(codes + first) = make_uint2(low, high);
      }
    }
    __syncwarp();
  }
}

template <typename T, int NL, int G>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(const RowsArgs a, const int aligned) {
  constexpr int kStep = 32 / NL;
  pdl_wait();
  pdl_trigger();
  check_starts(a.batch);
  const int lane = threadIdx.x & 31, q = lane % NL, heads = a.cache.heads;
  const Place p = place_of<NL, G>(heads, lane);
  if (p.token >= a.batch.tokens) return;                 // the whole warp
  int sequence, place;
  if (!token_place(a.batch, a.cache.page_shift, p.token, lane, &sequence, &place)) return;
  const int page = place < 0 ? -1 : page_of(a.batch, a.cache, sequence, place);
  if (page < 0 && place >= 0 && lane == 0) report(kBadPage);
  uint32_t word[G][4] = {}, meta[G] = {};
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int row = p.row + i * kStep;
    if (row >= 2 * heads || page < 0) continue;
    const int64_t at = group_index(a.cache, page, row, place);
    meta[i] = a.cache.meta[at];
    const uint8_t* codes = a.cache.codes + at * (2 * NL * a.cache.bits);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = 8 * NL * h + 8 * q;
      if (a.cache.bits == 4) {
        word[i][2 * h] = *reinterpret_cast<const uint32_t*>(codes + first / 2);
      } else {
        const uint2 two = *reinterpret_cast<const uint2*>(codes + first);
        word[i][2 * h] = two.x;
        word[i][2 * h + 1] = two.y;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int row = p.row + i * kStep;
    if (row >= 2 * heads) break;
    const HeadsArgs& into = row >= heads ? a.v : a.k;
    if (into.data == nullptr) continue;
    const float s = meta_step(meta[i]), z = meta_zero(meta[i]);
    T* to_row = static_cast<T*>(into.data) + p.token * into.ld + (row >= heads ? row - heads : row) * into.head_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t c = a.cache.bits == 4 ? (word[i][2 * h] >> (4 * k)) & 15u : (word[i][2 * h + k / 4] >> (8 * (k % 4))) & 255u;
        v[k] = __fmul_rn(s, __fsub_rn((float)c, z));     // exact: 11 and 9 bits
      }
      T* to = to_row + 8 * NL * h + 8 * q;
      if (aligned) {
        store_floats<T, 8>(to, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) to[k] = from_float<T>(v[k]);
      }
    }
  }
}

template <typename T, int NL, int G, bool APPEND>
cudaError_t launch(const RowsArgs& a, cudaStream_t s) {
  constexpr int kRows = 32 / NL * G;
  const int64_t each = (2 * a.cache.heads + kRows - 1) / kRows;
  bool aligned = true;
  for (const HeadsArgs* h : {&a.k, &a.v})
    aligned = aligned && on_boundary(h->data, 16) && h->ld % (16 / sizeof(T)) == 0 && h->head_stride % (16 / sizeof(T)) == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((each * a.batch.tokens + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  if constexpr (APPEND) return cudaLaunchKernelEx(&cfg, append_kernel<T, NL, G>, a, (int)aligned);
  else return cudaLaunchKernelEx(&cfg, read_kernel<T, NL, G>, a, (int)aligned);
}
// Where a step a warp would fill the machine several times over, a warp takes
// two (if a token has as many): its place is looked for once for them (three loads
// that wait for each other), their loads are in flight together, and lanes share
// the finding of steps (four: 15.7 us for 8192 tokens, two 15.2).
template <typename T, int NL>
cudaError_t launch(const RowsArgs& a, bool append, cudaStream_t s) {
  const int each = (2 * a.cache.heads + 32 / NL - 1) / (32 / NL);        // steps a token
  const bool many = (int64_t)a.batch.tokens * each > kManySteps;
  if (!append) return many && each > 1 ? launch<T, NL, 2, false>(a, s) : launch<T, NL, 1, false>(a, s);
  return many && each > 1 ? launch<T, NL, 2, true>(a, s) : launch<T, NL, 1, true>(a, s);
}
template <typename T>
cudaError_t launch(const RowsArgs& a, bool append, cudaStream_t s) {
  if (a.cache.head_dim == 64) return launch<T, 4>(a, append, s);
  if (a.cache.head_dim == 128) return launch<T, 8>(a, append, s);
  return launch<T, 16>(a, append, s);
}
cudaError_t launch(const RowsArgs& a, int dtype, bool append, cudaStream_t s) {
  if (dtype == ECHO_F32) return launch<float>(a, append, s);
  if (dtype == ECHO_BF16) return launch<__nv_bfloat16>(a, append, s);
  return launch<__half>(a, append, s);
}

}  // namespace

cudaError_t launch_append(const RowsArgs& a, int dtype, cudaStream_t s) { return launch(a, dtype, true, s); }
cudaError_t launch_read(const RowsArgs& a, int dtype, cudaStream_t s) { return launch(a, dtype, false, s); }
StatusWord rows_status() { return {read_status, clear_status_bits}; }

}  // namespace echo
