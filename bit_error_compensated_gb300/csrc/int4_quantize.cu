// int4_quantize.cu -- echo_quantize_weights (include/echo.h): weights to 4-bit
// codes in groups along their depth.
//
// group / 16 lanes hold a group, 16 values each, as in the all-reduce's push;
// a warp takes up to twice 8, 4 or 2 groups of a row that follow each other.
// 14336 x 4096 bf16 take 41 us (3.6 TB/s), bound by instructions; with a step
// that every lane of a group finds by itself, 55 us (437 instructions for 16
// values a lane).
#include "serve_common.h"

namespace echo {
namespace {

ECHO_STATUS_WORD

constexpr int kWarps = 8;
constexpr int64_t kManySteps = 4 * 152 * 16;      // of the machine's warps, see launch

// G: steps of 32 / NL groups, one after the other in a row, that a warp takes
// (their loads are in flight together).
template <typename T, int NL, int G>
__global__ void __launch_bounds__(32 * kWarps) quantize_weights_kernel(const WeightsArgs a, const int aligned) {
  constexpr int kGroups = 32 / NL, kGroup = 16 * NL;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, q = lane % NL;
  const int groups = (int)((a.depth + kGroup - 1) / kGroup), each = (groups + kGroups * G - 1) / (kGroups * G);   // warps a row
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t row = divided(w, each);
  if (row >= a.ranks * a.channels) return;               // the whole warp
  const int64_t rank = divided(row, a.channels), channel = row - rank * a.channels;
  const int64_t group0 = (w - row * each) * kGroups * G + lane / NL;
  const T* from = static_cast<const T*>(a.w) + rank * a.rank_w + channel * a.ld_w;
  Pack<T, 8> v[G][2];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int64_t k0 = (group0 + i * kGroups) * kGroup, here = a.depth - k0;             // values of this group, if fewer than all
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = 8 * NL * h + 8 * q;
      if (aligned && first + 8 <= here) {
        v[i][h] = load_pack<T, 8>(from + k0 + first);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][h].v[k] = first + k < here ? from[k0 + first + k] : from_float<T>(0.0f);
      }
    }
  }
  __syncwarp();
  float lo[G], hi[G];
#pragma unroll
  for (int i = 0; i < G; ++i) range_of<T>(v[i], lo[i], hi[i]);
  const GroupStep mine = shared_step<NL, G>(lo, hi, q, 15.0f);
  if (q < G && group0 + q * kGroups < groups) {
    a.meta[rank * a.rank_meta + channel * a.ld_meta + group0 + q * kGroups] = mine.meta;
    if (!mine.finite) report(kNaNGroup);
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int64_t k0 = (group0 + i * kGroups) * kGroup, here = a.depth - k0;
    const GroupStep g = step_at<NL, G>(mine, i);
    if (here > 0) {
      uint8_t* to = a.codes + rank * a.rank_codes + channel * a.ld_codes + k0 / 2;
      const bool words = ((uintptr_t)to & 3) == 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int first = 8 * NL * h + 8 * q;
        float eight[8];
        to_floats<T, 8>(v[i][h], eight);
        uint32_t low, high;
        group_codes8<4>(eight, g, low, high);
        uint32_t codes = low | high << 16;
        if (here - first < 8) codes &= here > first ? (1u << (4 * (here - first))) - 1 : 0;     // behind the row's end: 0
        if (words && first + 8 <= here) {
          *reinterpret_cast<uint32_t*>(to + first / 2) = codes;
        } else {
#pragma unroll
          for (int k = 0; k < 8; k += 2)
            if (first + k < here) to[(first + k) / 2] = (uint8_t)(codes >> (4 * k));
        }
      }
    }
    __syncwarp();
  }
}

template <typename T, int NL, int G>
cudaError_t launch(const WeightsArgs& a, cudaStream_t s) {
  constexpr int kGroups = 32 / NL, kGroup = 16 * NL;
  const int64_t groups = (a.depth + kGroup - 1) / kGroup;
  const int64_t warps = (groups + kGroups * G - 1) / (kGroups * G) * a.ranks * a.channels;
  const int64_t in16 = 16 / (int64_t)sizeof(T);
  const bool aligned = on_boundary(a.w, 16) && (a.channels == 1 || a.ld_w % in16 == 0) && (a.ranks == 1 || a.rank_w % in16 == 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, quantize_weights_kernel<T, NL, G>, a, (int)aligned);
}
// Two steps a warp where one each would fill the machine several times over (four:
// 43 us for 14336 x 4096, two 41, one 55).
template <typename T, int NL>
cudaError_t launch(const WeightsArgs& a, cudaStream_t s) {
  constexpr int kSpan = 16 * 32;
  const int64_t steps = (a.depth + kSpan - 1) / kSpan * a.ranks * a.channels;
  return steps > kManySteps ? launch<T, NL, 2>(a, s) : launch<T, NL, 1>(a, s);
}
template <typename T>
cudaError_t launch(const WeightsArgs& a, cudaStream_t s) {
  if (a.group == 64) return launch<T, 4>(a, s);
  if (a.group == 128) return launch<T, 8>(a, s);
  return launch<T, 16>(a, s);
}

}  // namespace

cudaError_t launch_quantize_weights(const WeightsArgs& a, int dtype, cudaStream_t s) {
  if (dtype == ECHO_F32) return launch<float>(a, s);
  if (dtype == ECHO_BF16) return launch<__nv_bfloat16>(a, s);
  return launch<__half>(a, s);
}
StatusWord weights_status() { return {read_status, clear_status_bits}; }

}  // namespace echo
