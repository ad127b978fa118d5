// norm_fwd.cu -- echo_norm: the reduced block output joins the residual stream
// and the next block's input is normalised (include/echo.h).
//
//     n = norm(y) w_post + b_post,  r = x + scale gate n,  h = norm(r) w_pre + b_pre
//
// A row's elements stay in its threads' registers from the loads of x and y to
// the stores of r and h, so each is read or written once; the statistics are
// sums over the row's threads, the variance in a second pass over the
// registers (no cancellation).  It is bound by those bytes.
#include "norm_common.h"

namespace echo {
namespace {

constexpr int kMaxWarps = 32;

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxBits {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return a > b ? a : b;
  }
};

// Sums and maxima over the threads of a row (a whole number of warps of the
// block).  Each uses one of two sets of slots in turn, so one barrier is
// enough: a set is written again only after the next sum's barrier, which its
// readers have passed.  Slots past a row's warps stay 0, neutral to both.
struct RowReduce {
  uint32_t (*slots)[kMaxWarps];      // [2][kMaxWarps]
  int first, count, warp, lane;      // the row's slots, this thread's place in them
  int which;
  template <typename V, typename Op>
  __device__ __forceinline__ V all(V v, Op op) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    if (count == 1) return v;
    V* s = reinterpret_cast<V*>(&slots[which][first]);
    which ^= 1;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < count; ++i) v = op(v, s[i]);
    return v;
  }
};

template <typename T, int VEC, int NV>
constexpr int norm_max_threads() {
  return VEC == 1 ? (NV == 4 ? 256 : 1024) : NV == 1 ? 256 : NV == 2 ? 512 : VEC == 4 ? 1024 : 512;
}

template <typename T, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(norm_max_threads<T, VEC, NV>())
norm_kernel(const NormArgs a) {
  __shared__ uint32_t slots[2][kMaxWarps];
  constexpr int E = VEC * NV;
  const int tid = threadIdx.x, threads = blockDim.x;
  for (int i = threadIdx.y * threads + tid; i < 2 * kMaxWarps; i += threads * blockDim.y)
    slots[i / kMaxWarps][i % kMaxWarps] = 0;
  __syncthreads();
  RowReduce red{slots, (int)threadIdx.y * (threads / 32), threads / 32, tid >> 5, tid & 31, 0};
  const float inv_width = 1.0f / (float)a.width;
  pdl_wait();
  pdl_trigger();

  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < a.rows;
       base += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = base + threadIdx.y;
    const bool active = row < a.rows;
    bool on[NV];
    Pack<T, VEC> px[NV], py[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * threads + tid) * VEC;
      on[j] = active && col < a.width;
      if (on[j]) {
        if (a.y) py[j] = load_pack<T, VEC>(static_cast<const T*>(a.y) + row * a.ld_y + col);
        px[j] = load_pack<T, VEC>(static_cast<const T*>(a.x) + row * a.ld_x + col);
      }
    }
    float v[E];            // y, then n, then r, then h; 0 outside the row
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;

    // Centres v (layer norm) and returns 1 / sqrt(var + eps).
    auto centre = [&](float& mean) {
      float s = 0.f;
      if (LAYER) {
#pragma unroll
        for (int i = 0; i < E; ++i) s += v[i];
        mean = red.all(s, Add()) * inv_width;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = on[i / VEC] ? v[i] - mean : 0.f;
        s = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s += v[i] * v[i];
      return rsqrtf(red.all(s, Add()) * inv_width + a.eps);
    };

#pragma unroll
    for (int i = 0; i < E; ++i)
      v[i] = a.y && on[i / VEC] ? to_float(py[i / VEC].v[i % VEC]) : 0.f;
    if (a.post) rstd1 = centre(mean1);
    const int64_t gate_row = a.gate ? row / a.gate_span : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * threads + tid) * VEC;
      if (on[j]) {
        float w[VEC], b[VEC];
        if (a.post) {
          load_param<T, VEC>(a.w_post, a.params_f32, col, 1.f, w);
          load_param<T, VEC>(a.b_post, a.params_f32, col, 0.f, b);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[j * VEC + i] = v[j * VEC + i] * rstd1 * w[i] + b[i];
        }
        if (a.gate && !a.gate_scalar) {
          load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + col, 1.f, w);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[j * VEC + i] *= w[i];
        } else if (a.gate) {
          float g[1];
          load_param<T, 1>(a.gate, a.params_f32, gate_row, 1.f, g);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[j * VEC + i] *= g[0];
        }
        Pack<T, VEC> out;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float& r = v[j * VEC + i];
          r = a.y ? to_float(px[j].v[i]) + a.scale * r : to_float(px[j].v[i]);
          out.v[i] = from_float<T>(r);
        }
        if (a.r) store_pack<T, VEC>(static_cast<T*>(a.r) + row * a.ld_r + col, out);
      }
    }
    if (a.h || a.codes || a.stats) rstd2 = centre(mean2);
    uint32_t amax = __float_as_uint(kTinyAmax);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * threads + tid) * VEC;
      if (on[j] && (a.h || a.codes)) {
        float w[VEC], b[VEC], h[VEC];
        load_param<T, VEC>(a.w_pre, a.params_f32, col, 1.f, w);
        load_param<T, VEC>(a.b_pre, a.params_f32, col, 0.f, b);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          h[i] = v[j * VEC + i] * rstd2 * w[i] + b[i];
          v[j * VEC + i] = h[i];
          amax = max(amax, abs_bits(h[i]));
        }
        if (a.h) store_floats<T, VEC>(static_cast<T*>(a.h) + row * a.ld_h + col, h);
      }
    }
    if (a.codes) {
      const float top = __uint_as_float(red.all(amax, MaxBits()));
      const float inv = __fdiv_rn(127.f, top);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * threads + tid) * VEC;
        if (on[j]) {
          Pack<int8_t, VEC> q;
#pragma unroll
          for (int i = 0; i < VEC; ++i) q.v[i] = (int8_t)quantize_code(v[j * VEC + i], inv);
          int8_t* to = a.codes + row * a.ld_codes + col;
          if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(&q);
          } else if constexpr (VEC == 4) {
            *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(&q);
          } else {
            *to = q.v[0];
          }
        }
      }
      if (tid == 0 && active) a.scales[row] = __fdiv_rn(top, 127.f);
    }
    if (a.stats && tid == 0 && active)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(mean1, rstd1, mean2, rstd2);
  }
}

template <typename T, int VEC, int NV>
cudaError_t launch(const NormArgs& a, int layer, int sms, cudaStream_t s) {
  const int threads = ((a.width + VEC * NV - 1) / (VEC * NV) + 31) / 32 * 32;
  const int rows = threads < 128 ? 128 / threads : 1;
  const int64_t blocks = (a.rows + rows - 1) / rows, most = (int64_t)sms * 64;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
  cfg.blockDim = dim3(threads, rows);
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return layer ? cudaLaunchKernelEx(&cfg, norm_kernel<T, VEC, NV, true>, a)
               : cudaLaunchKernelEx(&cfg, norm_kernel<T, VEC, NV, false>, a);
}

}  // namespace

template <>
cudaError_t launch_norm<ECHO_ELEM>(const NormArgs& a, int layer, bool vec, int sms, cudaStream_t s) {
  using T = ECHO_ELEM;
  constexpr int V = 16 / sizeof(T);
  if (!vec) return a.width <= 1024 ? launch<T, 1, 4>(a, layer, sms, s) : launch<T, 1, 16>(a, layer, sms, s);
  if (a.width <= 256 * V) return launch<T, V, 1>(a, layer, sms, s);
  if (a.width <= 1024 * V) return launch<T, V, 2>(a, layer, sms, s);
  return launch<T, V, 4>(a, layer, sms, s);
}

}  // namespace echo
