// norm_bwd.cu -- echo_norm_backward: gradients of the residual join
// (include/echo.h).  With a = norm(y) before its weight, b = norm(r) before
// its weight, and m(.) the mean over the row:
//
//     g = dh w_pre,    D = dr + rstd2 (g - [m(g)] - b m(g b)),        dx = D
//     dgate = scale D n,  dn = scale gate D,  f = dn w_post,
//     dy = rstd1 (f - [m(f)] - a m(f a))     (dn without the post norm)
//     dw_pre = sum dh b, db_pre = sum dh, dw_post = sum dn a, db_post = sum dn
//
// ([.] for layer norms only).  A worker (a row's worth of threads) takes a
// contiguous range of rows, keeps each row in registers from its four loads
// to its two stores, and keeps the column sums of the parameters' gradients
// in registers over all its rows; a second, small kernel adds the workers'
// sums in a fixed order.  Rows wider than one block's registers are split by
// columns over a cluster, whose blocks exchange the row sums through
// distributed shared memory.
#include "norm_common.h"

namespace echo {
namespace {

constexpr int kThreads = 256;          // of a block at most
constexpr int kBlocksPerSm = 2;        // of a call's grid
constexpr int kMaxCluster = 4;         // ECHO_NORM_MAX_WIDTH / (16 * kThreads)
constexpr int kSlots = kThreads / 32 * kMaxCluster;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// Sums over a row's threads: those of its warps of this block and, in a
// cluster, of the other blocks'.  A warp writes its sum to the slot that
// belongs to it in every block; then one barrier (of the cluster, or of the
// block) and everyone adds the slots in the same order.  Two sets of slots in
// turn, as a set is written again only behind the next sum's barrier.
template <int N>
struct RowSums {
  float (*slots)[kSlots][N];           // [2]
  int first, count, warp, lane;        // the row's slots; this warp's among them
  int blocks;                          // of the cluster
  int which;
  __device__ __forceinline__ void all(float (&v)[N]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], d);
    if (count == 1) return;
    float(*s)[N] = slots[which];
    which ^= 1;
    if (blocks > 1) {
      if (lane < blocks) {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at) : "r"(smem_u32(&s[first + warp][0])), "r"(lane));
#pragma unroll
        for (int k = 0; k < N; ++k)
          asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at + 4 * k), "f"(v[k]) : "memory");
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                   "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) s[first + warp][k] = v[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = s[first][k];
    for (int i = 1; i < count; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += s[first + i][k];
  }
};

template <typename T, int VEC, int NV, bool LAYER, bool GATE>
__global__ void __launch_bounds__(kThreads)
norm_grad_kernel(const NormGradArgs a, int blocks, int block_cols) {
  constexpr int E = VEC * NV;
  __shared__ float slots[2][kSlots][3];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int part = (int)blockIdx.x % blocks;             // of the row's columns
  const int64_t worker = (int64_t)(blockIdx.x / blocks) * blockDim.y + threadIdx.y;
  const int col0 = part * block_cols;
  const int warps = threads / 32;
  RowSums<3> sums{slots, (int)threadIdx.y * warps, warps * blocks, part * warps + (tid >> 5),
                  tid & 31, blocks, 0};
  const float inv_width = 1.0f / (float)a.width;
  if (blocks > 1)                      // every block's slots exist before the first is written
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();

  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * threads + tid) * VEC;
    in[j] = c < block_cols && col0 + c < a.width;
  }
  auto col_of = [&](int j) { return col0 + (j * threads + tid) * VEC; };

  float sum_wpost[E], sum_bpost[LAYER ? E : 1], sum_wpre[E], sum_bpre[LAYER ? E : 1];
  float sum_gate[GATE ? E : 1];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    sum_wpost[i] = sum_wpre[i] = 0.f;
    if (LAYER) sum_bpost[i] = sum_bpre[i] = 0.f;
    if (GATE) sum_gate[i] = 0.f;
  }
  float sum_scalar = 0.f;

  const int64_t row0 = worker * a.span;
  const int64_t row1 = row0 + a.span < a.rows ? row0 + a.span : a.rows;
  int64_t gate_row = a.gate ? row0 / a.gate_span : 0;
  int64_t gate_left = a.gate ? a.gate_span - (row0 - gate_row * a.gate_span) : 0;
  bool gate_whole = a.gate && gate_left == a.gate_span;   // its first row is this worker's

  for (int64_t step = 0; step < a.span; ++step) {
    const int64_t row = row0 + step;
    const bool active = row < row1;
    bool on[NV];
    float hat1[E], hat2[E], g[E], d[E];
    float4 st = make_float4(0.f, 1.f, 0.f, 1.f);
    if (active && a.stats) st = __ldg(reinterpret_cast<const float4*>(a.stats) + row);
    float s[3] = {0.f, 0.f, 0.f};
    float gate_value = 1.f;
    if (a.gate && a.gate_scalar && active) {
      float one[1];
      load_param<T, 1>(a.gate, a.params_f32, gate_row, 1.f, one);
      gate_value = one[0];
    }
    // n and gate of vector j, from a
    auto n_of = [&](int j, float (&n)[VEC], float (&gate)[VEC]) {
      float w[VEC], b[VEC];
      if (a.post) {
        load_param<T, VEC>(a.w_post, a.params_f32, col_of(j), 1.f, w);
        load_param<T, VEC>(a.b_post, a.params_f32, col_of(j), 0.f, b);
      }
      if (GATE) load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + col_of(j), 1.f, gate);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        n[i] = a.post ? hat1[j * VEC + i] * w[i] + b[i] : hat1[j * VEC + i];
        if (!GATE) gate[i] = gate_value;
      }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      on[j] = active && in[j];
      Pack<T, VEC> px, py, pr, ph;
      if (on[j]) {
        px = load_pack<T, VEC>(static_cast<const T*>(a.x) + row * a.ld_x + col_of(j));
        if (a.y) py = load_pack<T, VEC>(static_cast<const T*>(a.y) + row * a.ld_y + col_of(j));
        if (a.dr) pr = load_pack<T, VEC>(static_cast<const T*>(a.dr) + row * a.ld_dr + col_of(j));
        if (a.dh) ph = load_pack<T, VEC>(static_cast<const T*>(a.dh) + row * a.ld_dh + col_of(j));
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float y = a.y ? to_float(py.v[i]) : 0.f;
          hat1[j * VEC + i] = a.post ? (y - st.x) * st.y : y;
        }
        float n[VEC], gate[VEC], w[VEC];
        n_of(j, n, gate);
        load_param<T, VEC>(a.w_pre, a.params_f32, col_of(j), 1.f, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int k = j * VEC + i;
          const float r = a.y ? to_float(px.v[i]) + a.scale * (gate[i] * n[i]) : to_float(px.v[i]);
          hat2[k] = (r - st.z) * st.w;
          const float dh = a.dh ? to_float(ph.v[i]) : 0.f;
          sum_wpre[k] += dh * hat2[k];
          if (LAYER) sum_bpre[k] += dh;
          g[k] = dh * w[i];
          d[k] = a.dr ? to_float(pr.v[i]) : 0.f;
          s[0] += g[k] * hat2[k];
          if (LAYER) s[1] += g[k];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          hat1[j * VEC + i] = hat2[j * VEC + i] = g[j * VEC + i] = d[j * VEC + i] = 0.f;
      }
    }
    if (a.dh) {
      sums.all(s);
      s[0] *= inv_width;
      s[1] *= inv_width;
    }
    float t[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
      if (a.dh) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int k = j * VEC + i;
          d[k] += st.w * (g[k] - (LAYER ? s[1] : 0.f) - hat2[k] * s[0]);
        }
      }
      float dx[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) dx[i] = d[j * VEC + i];
      if (a.dx) store_floats<T, VEC>(static_cast<T*>(a.dx) + row * a.ld_dx + col_of(j), dx);
      if (!a.y) continue;
      float n[VEC], gate[VEC], w[VEC];
      n_of(j, n, gate);
      if (a.post) load_param<T, VEC>(a.w_post, a.params_f32, col_of(j), 1.f, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int k = j * VEC + i;
        const float sd = a.scale * d[k];
        if (GATE) sum_gate[k] += sd * n[i];
        else t[2] += sd * n[i];
        float dn = sd * gate[i];
        if (a.post) {
          sum_wpost[k] += dn * hat1[k];
          if (LAYER) sum_bpost[k] += dn;
          dn *= w[i];
          t[0] += dn * hat1[k];
          if (LAYER) t[1] += dn;
        }
        g[k] = dn;
      }
    }
    if (a.post || a.gate_scalar) {
      sums.all(t);
      t[0] *= inv_width;
      t[1] *= inv_width;
    }
    if (a.y && a.dy) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        float dy[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int k = j * VEC + i;
          dy[i] = a.post ? st.y * (g[k] - (LAYER ? t[1] : 0.f) - hat1[k] * t[0]) : g[k];
        }
        store_floats<T, VEC>(static_cast<T*>(a.dy) + row * a.ld_dy + col_of(j), dy);
      }
    }
    // The gate's gradient: a gate row whose rows are all this worker's is
    // written; one that began before its range goes to the worker's first
    // slot, one that goes on behind it to the second, for norm_grad_finish.
    if (a.gate && active) --gate_left;
    if (a.dgate && active) {
      sum_scalar += t[2];
      if (gate_left == 0 || row + 1 == row1) {
        const bool direct = gate_whole && gate_left == 0;
        const int64_t cols = GATE ? a.width : 1;
        float* slot = a.gate_partial + (2 * worker + (gate_whole ? 1 : 0)) * cols;
        if (GATE) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (!in[j]) continue;
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              v[i] = sum_gate[j * VEC + i];
              sum_gate[j * VEC + i] = 0.f;
            }
            const int64_t at = gate_row * a.width + col_of(j);
            if (!direct) store_floats<float, VEC>(slot + col_of(j), v);
            else if (a.params_f32) store_floats<float, VEC>(static_cast<float*>(a.dgate) + at, v);
            else store_floats<T, VEC>(static_cast<T*>(a.dgate) + at, v);
          }
        } else {
          if (tid == 0 && part == 0) {
            if (!direct) slot[0] = sum_scalar;
            else if (a.params_f32) static_cast<float*>(a.dgate)[gate_row] = sum_scalar;
            else static_cast<T*>(a.dgate)[gate_row] = from_float<T>(sum_scalar);
          }
          sum_scalar = 0.f;
        }
      }
    }
    if (a.gate && active && gate_left == 0) {
      ++gate_row;
      gate_left = a.gate_span;
      gate_whole = true;
    }
  }

  if (worker < a.workers) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      const int64_t at = worker * a.width + col_of(j);
      auto put = [&](float* to, const float* from) {
        if (!to) return;
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = from[j * VEC + i];
        store_floats<float, VEC>(to + at, v);
      };
      put(a.partial[0], sum_wpost);
      if (LAYER) put(a.partial[1], sum_bpost);
      put(a.partial[2], sum_wpre);
      if (LAYER) put(a.partial[3], sum_bpre);
    }
  }
  // No block of a cluster may end while another can still write to its slots.
  if (blocks > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Adds the workers' column sums: blockIdx.y 0..3 a parameter each, 4 the gate
// rows that more than one worker shares.
constexpr int kFinishRows = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kFinishRows)
norm_grad_finish(const NormGradArgs a) {
  __shared__ float part[kFinishRows][33];
  pdl_wait();
  pdl_trigger();
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  const int which = blockIdx.y;
  auto put = [&](void* to, int64_t at, float v) {
    if (a.params_f32) static_cast<float*>(to)[at] = v;
    else static_cast<T*>(to)[at] = from_float<T>(v);
  };
  if (which < 4) {
    if (!a.dparam[which]) return;
    float s = 0.f;
    if (col < a.width)
      for (int64_t w = threadIdx.y; w < a.workers; w += kFinishRows)
        s += a.partial[which][w * a.width + col];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < a.width) {
      s = part[0][threadIdx.x];
      for (int i = 1; i < kFinishRows; ++i) s += part[i][threadIdx.x];
      put(a.dparam[which], col, s);
    }
    return;
  }
  const int64_t cols = a.gate_scalar ? 1 : a.width;
  if (!a.dgate || col >= cols) return;
  // Worker b's range begins inside a gate row that began in worker b - 1's:
  // that one's second slot and the first slots of all that follow are its sum.
  for (int64_t b = 1 + threadIdx.y; b < a.workers; b += kFinishRows) {
    const int64_t g = b * a.span / a.gate_span, begin = g * a.gate_span, end = begin + a.gate_span;
    if (begin == b * a.span || begin < (b - 1) * a.span) continue;
    float s = a.gate_partial[(2 * (b - 1) + 1) * cols + col];
    for (int64_t w = b; w < a.workers && w * a.span < end; ++w)
      s += a.gate_partial[2 * w * cols + col];
    put(a.dgate, g * cols + col, s);
  }
}

template <typename T, int VEC, int NV, bool LAYER, bool GATE>
cudaError_t launch(NormGradArgs a, int sms, cudaStream_t s) {
  const int blocks = (a.width + VEC * NV * kThreads - 1) / (VEC * NV * kThreads);
  const int block_cols = ((a.width + blocks - 1) / blocks + VEC - 1) / VEC * VEC;
  const int threads = ((block_cols + VEC * NV - 1) / (VEC * NV) + 31) / 32 * 32;
  const int rows = threads < 128 ? 128 / threads : 1;
  const int64_t most = (int64_t)(kBlocksPerSm * sms / blocks) * rows;
  a.span = (a.rows + most - 1) / most;
  a.workers = (a.rows + a.span - 1) / a.span;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.workers + rows - 1) / rows * blocks));
  cfg.blockDim = dim3(threads, rows);
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {overlapped_launch()};
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = blocks;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, norm_grad_kernel<T, VEC, NV, LAYER, GATE>, a, blocks, block_cols);
  bool any = a.dgate && a.workers > 1;
  for (int k = 0; k < 4; ++k) any = any || a.dparam[k];
  if (e != cudaSuccess || !any) return e;
  cudaLaunchConfig_t fin = {};
  fin.gridDim = dim3((unsigned)((a.width + 31) / 32), 5);
  fin.blockDim = dim3(32, kFinishRows);
  fin.stream = s;
  fin.attrs = at;
  fin.numAttrs = 1;
  return cudaLaunchKernelEx(&fin, norm_grad_finish<T>, a);
}

template <typename T, int VEC, int NV>
cudaError_t pick(const NormGradArgs& a, int layer, int sms, cudaStream_t s) {
  const bool gate = a.gate && !a.gate_scalar;
  if (layer) return gate ? launch<T, VEC, NV, true, true>(a, sms, s) : launch<T, VEC, NV, true, false>(a, sms, s);
  return gate ? launch<T, VEC, NV, false, true>(a, sms, s) : launch<T, VEC, NV, false, false>(a, sms, s);
}

}  // namespace

template <>
cudaError_t launch_norm_grad<ECHO_ELEM>(NormGradArgs a, int layer, bool vec, int sms, cudaStream_t s) {
  using T = ECHO_ELEM;
  constexpr int V = 16 / sizeof(T);
  const bool narrow = a.width <= 8 * kThreads;
  if (!vec) return narrow ? pick<T, 1, 8>(a, layer, sms, s) : pick<T, 1, 16>(a, layer, sms, s);
  return narrow ? pick<T, V, 8 / V>(a, layer, sms, s) : pick<T, V, 16 / V>(a, layer, sms, s);
}

}  // namespace echo
