// norm_fwd.cu -- echo_norm: the reduced block output joins the residual stream
// and the next block's input is normalised (include/echo.h).
//
//     n = norm(y) w_post + b_post,  r = x + scale gate n,  h = norm(r) w_pre + b_pre
//
// A row's elements stay in its threads' registers from the loads of x and y to
// the stores of r and h, so each is read or written once; the statistics are
// sums over the row's threads, the variance in a second pass over the
// registers (no cancellation).  It is bound by those bytes.
//
// norm_stream_kernel takes rows up to 8192 elements.  At the memory's rate a
// row of 4096 16-bit elements (32 KB moved) leaves an SM 1400 cycles, so what
// can be done once is: a thread keeps its columns' parameters in registers
// over all its rows, the scale, a shared gate and the post norm's
// weight multiplied into one factor.  Rows come through a ring of asynchronous
// copies, several ahead (16-bit rows that are not made of 16-byte pieces, which
// such copies do not take, element by element through registers, one ahead).
// norm_kernel takes longer rows: 1024 threads an SM at 64 registers hold x, the
// next x and y and the row, of which 170 to 300 bytes a thread are spilled.
//
// One GB300, 8192 x 4096 bf16, RMS: 47 us, 5.7 TB/s, 0.84 of the copy rate;
// what is left are the two sums' round trips through shuffles and barriers
// (short scoreboard 1.7 of 6 cycles an instruction, issue 60%).  fp32, same
// rows: 94 us, 5.7 TB/s.  One row: 2.7 us, a launch and one trip to memory.
// Layer norms (four sums, eight elements a thread): 96 us, fp32 108.  Longer
// rows: 8192 x 12288 bf16 369 us, layer norms 397, 2.2 and 2.0 TB/s (spills, and
// no ring); 4096 x 16384 239 and 259.
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
// readers have passed.  Slots past a row's warps stay 0, neutral to both, so
// that four are read at a time.
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
    struct __align__(16) Four { V v[4]; };
    const Four* f = reinterpret_cast<const Four*>(s);
    v = op(op(f[0].v[0], f[0].v[1]), op(f[0].v[2], f[0].v[3]));
#pragma unroll
    for (int i = 1; i < kMaxWarps / 4; ++i)
      if (4 * i < count) v = op(v, op(op(f[i].v[0], f[i].v[1]), op(f[i].v[2], f[i].v[3])));
    return v;
  }
};

// v[i] op= parameters i of the vector at `p` (nothing where there is none).
template <typename T, int VEC>
__device__ __forceinline__ void scale_by(const void* p, int f32, int64_t col, float (&v)[VEC]) {
  if (p == nullptr) return;
  float w[VEC];
  load_param<T, VEC>(p, f32, col, w);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] *= w[i];
}
template <typename T, int VEC>
__device__ __forceinline__ void shift_by(const void* p, int f32, int64_t col, float (&v)[VEC]) {
  if (p == nullptr) return;
  float b[VEC];
  load_param<T, VEC>(p, f32, col, b);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] += b[i];
}

template <typename T, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(1024)
norm_kernel(const NormArgs a) {
  __shared__ __align__(16) uint32_t slots[2][kMaxWarps];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  for (int i = threadIdx.y * threads + tid; i < 2 * kMaxWarps; i += threads * blockDim.y)
    slots[i / kMaxWarps][i % kMaxWarps] = 0;
  __syncthreads();
  RowReduce red{slots, (int)threadIdx.y * 4, threads / 32, tid >> 5, tid & 31, 0};
  const float inv_width = 1.0f / (float)a.width;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = (j * threads + tid) * VEC < a.width;
  auto col = [&](int j) { return (j * threads + tid) * VEC; };
  pdl_wait();
  pdl_trigger();

  Pack<T, VEC> next_x[NV], next_y[NV];
  auto load_row = [&](int64_t at) {
    if (at >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + at * a.ld_x;
    const T* y = static_cast<const T*>(a.y) + at * a.ld_y;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in[j]) {
        if (a.y) next_y[j] = load_pack<T, VEC>(y + col(j));
        next_x[j] = load_pack<T, VEC>(x + col(j));
      }
  };
  load_row(row);
  // The gate row of a row, kept up as the rows advance by `step`.
  int64_t gate_row = 0, gate_pos = 0, gate_step = 0, gate_rest = 0;
  if (a.gate && a.gate_span < a.rows) {
    gate_row = row / a.gate_span;
    gate_pos = row - gate_row * a.gate_span;
    gate_step = step / a.gate_span;
    gate_rest = step - gate_step * a.gate_span;
  }
  // All rows of a block take the same number of turns, as its sums' barriers need.
  for (int64_t base = row - threadIdx.y; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    Pack<T, VEC> px[NV];
    float v[NV][VEC];      // y, then n, then r, then h; 0 outside the row
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      px[j] = next_x[j];
      if (a.y && active && in[j]) {
        to_floats<T, VEC>(next_y[j], v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
      }
    }
    load_row(row + step);
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
    // Centres v (layer norm) and returns 1 / sqrt(var + eps).
    auto centre = [&](float& mean) {
      float s = 0.f;
      if (LAYER) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s += v[j][i];
        mean = red.all(s, Add()) * inv_width;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (active && in[j])
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] -= mean;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += v[j][i] * v[j][i];
      return rsqrtf(red.all(s, Add()) * inv_width + a.eps);
    };

    if (a.post) rstd1 = centre(mean1);
    // A layer norm's bias is added to the scaled row as it is: divided by rstd
    // first, it would be lost where the variance overflows and rstd is 0.
    float factor = LAYER ? a.scale : a.scale * rstd1;
    if (a.gate && a.gate_scalar && active) {
      float g[1];
      load_param<T, 1>(a.gate, a.params_f32, gate_row, g);
      factor *= g[0];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!active || !in[j]) continue;
      if (a.y) {
        if (a.post) {
          if (LAYER)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] *= rstd1;
          scale_by<T, VEC>(a.w_post, a.params_f32, col(j), v[j]);
          if (LAYER) shift_by<T, VEC>(a.b_post, a.params_f32, col(j), v[j]);
        }
        if (a.gate && !a.gate_scalar)
          scale_by<T, VEC>(a.gate, a.params_f32, gate_row * a.width + col(j), v[j]);
      }
      float x[VEC];
      to_floats<T, VEC>(px[j], x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = a.y ? fmaf(factor, v[j][i], x[i]) : x[i];
      if (a.r) store_floats<T, VEC>(static_cast<T*>(a.r) + row * a.ld_r + col(j), v[j]);
    }
    if (a.h || a.codes || a.stats) rstd2 = centre(mean2);
    if (a.h || a.codes) {
      uint32_t amax = __float_as_uint(kTinyAmax);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!active || !in[j]) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] *= rstd2;
        scale_by<T, VEC>(a.w_pre, a.params_f32, col(j), v[j]);
        if (LAYER) shift_by<T, VEC>(a.b_pre, a.params_f32, col(j), v[j]);
        if (a.h) store_floats<T, VEC>(static_cast<T*>(a.h) + row * a.ld_h + col(j), v[j]);
        if (a.codes)
#pragma unroll
          for (int i = 0; i < VEC; ++i) amax = max(amax, abs_bits(v[j][i]));
      }
      if (a.codes) {
        const float top = __uint_as_float(red.all(amax, MaxBits()));
        const float inv = __fdiv_rn(127.f, top);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!active || !in[j]) continue;
          Pack<int8_t, VEC> q;
#pragma unroll
          for (int i = 0; i < VEC; ++i) q.v[i] = (int8_t)quantize_code(v[j][i], inv);
          int8_t* to = a.codes + row * a.ld_codes + col(j);
          if constexpr (VEC == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(&q);
          else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(&q);
          else *to = q.v[0];
        }
        if (tid == 0 && active) a.scales[row] = __fdiv_rn(top, 127.f);
      }
    }
    gate_row += gate_step;
    gate_pos += gate_rest;
    if (gate_pos >= a.gate_span) {
      gate_pos -= a.gate_span;
      ++gate_row;
    }
    if (a.stats && tid == 0 && active)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(mean1, rstd1, mean2, rstd2);
  }
}

// Rows ahead in the ring of asynchronous copies.
template <typename T, int E> constexpr int rows_ahead() { return sizeof(T) == 2 ? 4 : 3; }
// Asynchronous copies take 16 bytes, or an fp32 element.
template <typename T, int VEC> constexpr bool has_ring() { return VEC * sizeof(T) >= 4; }

// GATE: 0 none, or one row for all (multiplied into `mul` and `add`); 1 a row
// of gates, 2 a gate, for each row or several.
// E: elements a thread; MOST: threads of a block, at most, which sets the
// registers a thread may use.  FULL: y, r and h are there, codes are not.
template <typename T, int E, int VEC, bool LAYER, bool POST, int GATE, int MOST, bool FULL>
__global__ void __launch_bounds__(MOST)
norm_stream_kernel(const NormArgs a) {
  constexpr bool RING = has_ring<T, VEC>();
  constexpr int NV = E / VEC, kAhead = RING ? rows_ahead<T, E>() : 1;
  constexpr uint32_t kBytes = VEC * sizeof(T);          // of a piece in the ring
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) uint32_t slots[2][kMaxWarps];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  for (int i = threadIdx.y * threads + tid; i < 2 * kMaxWarps; i += threads * blockDim.y)
    slots[i / kMaxWarps][i % kMaxWarps] = 0;
  __syncthreads();
  RowReduce red{slots, (int)threadIdx.y * 4, threads / 32, tid >> 5, tid & 31, 0};
  const float inv_width = 1.0f / (float)a.width;
  const bool has_y = FULL || a.y, has_r = FULL || a.r, has_h = FULL || a.h, has_codes = !FULL && a.codes;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = (j * threads + tid) * VEC < a.width;
  // This thread's pieces of the ring: x and y of piece j of slot s.
  const uint32_t piece = kBytes * threads * blockDim.y, slot_bytes = 2 * NV * piece;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + kBytes * (threadIdx.y * threads + tid);
  pdl_wait();
  pdl_trigger();

  const char* from[2] = {static_cast<const char*>(a.x) + row * a.ld_x * sizeof(T) + kBytes * tid,
                         static_cast<const char*>(a.y) + row * a.ld_y * sizeof(T) + kBytes * tid};
  const int64_t far[2] = {step * a.ld_x * (int64_t)sizeof(T), step * a.ld_y * (int64_t)sizeof(T)};
  T held[RING ? 1 : 2][RING ? 1 : NV];
  int64_t fetch = row;
  auto fetch_array = [&](int k, uint32_t slot) {
    if (fetch < a.rows && (k == 0 || has_y)) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (in[j]) {
          const char* at = from[k] + j * threads * (int)kBytes;
          const uint32_t to = mine + slot * slot_bytes + (2 * j + k) * piece;
          if constexpr (!RING) held[k][j] = *reinterpret_cast<const T*>(at);
          else if constexpr (VEC == 1) copy4_async(to, at);
          else copy16_async(to, at);
        }
    }
    from[k] += far[k];
  };
  auto take = [&](int k, int j, uint32_t slot, float (&v)[VEC]) {
    const uint32_t at = mine + slot * slot_bytes + (2 * j + k) * piece;
    if constexpr (!RING) v[0] = to_float(held[k][j]);
    else if constexpr (VEC == 1) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
    else to_floats<T, VEC>(load_shared16<T, VEC>(at), v);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
    fetch_array(0, s);
    fetch_array(1, s);
    if (RING) copies_commit();
    fetch += step;
  }

  // The columns' parameters: n = hat1 * mul + add (times the row's gate), h = hat2 * w + b.
  float mul[NV][VEC], add[LAYER ? NV : 1][VEC], w[NV][VEC], b[LAYER ? NV : 1][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * threads + tid) * VEC;
    float g[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      g[i] = a.scale;
      mul[j][i] = w[j][i] = 1.f;
      if (LAYER) add[j][i] = b[j][i] = 0.f;
    }
    if (!in[j]) continue;
    if (GATE == 0) scale_by<T, VEC>(a.gate, a.params_f32, col, g);
    load_param<T, VEC>(a.w_pre, a.params_f32, col, 1.f, w[j]);
    if (POST) load_param<T, VEC>(a.w_post, a.params_f32, col, 1.f, mul[j]);
    if (LAYER) {
      load_param<T, VEC>(a.b_pre, a.params_f32, col, 0.f, b[j]);
      if (POST) load_param<T, VEC>(a.b_post, a.params_f32, col, 0.f, add[j]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      mul[j][i] *= g[i];
      if (LAYER) add[j][i] *= g[i];
    }
  }
  // The gate row of a row, kept up as the rows advance by `step`.
  int64_t gate_row = 0, gate_pos = 0, gate_step = 0, gate_rest = 0;
  if (GATE != 0) {
    gate_row = row / a.gate_span;
    gate_pos = row - gate_row * a.gate_span;
    gate_step = step / a.gate_span;
    gate_rest = step - gate_step * a.gate_span;
  }
  char* to_r = static_cast<char*>(a.r) + row * a.ld_r * sizeof(T) + kBytes * tid;
  char* to_h = static_cast<char*>(a.h) + row * a.ld_h * sizeof(T) + kBytes * tid;
  const int64_t far_r = step * a.ld_r * sizeof(T), far_h = step * a.ld_h * sizeof(T);
  uint32_t slot = 0;

  // All rows of a block take the same number of turns, as its sums' barriers need.
  for (int64_t base = row - threadIdx.y; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    if (RING) copies_wait<kAhead - 1>();
    float v[NV][VEC];      // y, then r, then h; 0 outside the row
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
    auto centre = [&](float& mean) {
      float s = 0.f;
      if (LAYER) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s += v[j][i];
        mean = red.all(s, Add()) * inv_width;
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (active && in[j])
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] -= mean;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = fmaf(v[j][i], v[j][i], s);
      return rsqrtf(red.all(s, Add()) * inv_width + a.eps);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (has_y && active && in[j]) {
        take(1, j, slot, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
      }
    }
    if (!RING) fetch_array(1, 0);       // what has been read makes room for the next row's
    if (POST) rstd1 = centre(mean1);
    float factor = rstd1, gate = 1.f;
    if (GATE == 2 && active) {
      float one[1];
      load_param<T, 1>(a.gate, a.params_f32, gate_row, one);
      gate = one[0];
      factor *= gate;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!active || !in[j]) continue;
      float x[VEC];
      take(0, j, slot, x);
      if (has_y) {
        float g[VEC];
        if (GATE == 1) load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + (j * threads + tid) * VEC, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float n = POST ? v[j][i] * factor : GATE == 2 ? v[j][i] * gate : v[j][i];
          if (LAYER && GATE == 2) n = fmaf(n, mul[j][i], add[j][i] * gate);
          else if (LAYER) n = fmaf(n, mul[j][i], add[j][i]);
          if (GATE == 1) v[j][i] = LAYER ? fmaf(n, g[i], x[i]) : fmaf(n * mul[j][i], g[i], x[i]);
          else v[j][i] = LAYER ? n + x[i] : fmaf(n, mul[j][i], x[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = x[i];
      }
      if (has_r) store_floats<T, VEC>(reinterpret_cast<T*>(to_r) + j * threads * VEC, v[j]);
    }
    fetch_array(0, slot);               // this thread has read its pieces of the slot
    if (RING) {
      fetch_array(1, slot);
      copies_commit();
      slot = slot == kAhead - 1 ? 0 : slot + 1;
    }
    fetch += step;
    if (has_h || has_codes || a.stats) rstd2 = centre(mean2);
    if (has_h || has_codes) {
      uint32_t amax = __float_as_uint(kTinyAmax);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!active || !in[j]) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          v[j][i] = LAYER ? fmaf(v[j][i] * rstd2, w[j][i], b[j][i]) : v[j][i] * rstd2 * w[j][i];
        if (has_h) store_floats<T, VEC>(reinterpret_cast<T*>(to_h) + j * threads * VEC, v[j]);
        if (has_codes)
#pragma unroll
          for (int i = 0; i < VEC; ++i) amax = max(amax, abs_bits(v[j][i]));
      }
      if (has_codes) {
        const float top = __uint_as_float(red.all(amax, MaxBits()));
        const float inv = __fdiv_rn(127.f, top);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!active || !in[j]) continue;
          Pack<int8_t, VEC> q;
#pragma unroll
          for (int i = 0; i < VEC; ++i) q.v[i] = (int8_t)quantize_code(v[j][i], inv);
          int8_t* to = a.codes + row * a.ld_codes + (j * threads + tid) * VEC;
          if constexpr (VEC == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(&q);
          else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(&q);
          else *to = q.v[0];
        }
        if (tid == 0 && active) a.scales[row] = __fdiv_rn(top, 127.f);
      }
    }
    if (a.stats && tid == 0 && active)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(mean1, rstd1, mean2, rstd2);
    to_r += far_r;
    to_h += far_h;
    if (GATE != 0) {
      gate_row += gate_step;
      gate_pos += gate_rest;
      if (gate_pos >= a.gate_span) {
        gate_pos -= a.gate_span;
        ++gate_row;
      }
    }
  }
  if (RING) copies_wait<0>();
}

template <typename T, int VEC, int NV>
cudaError_t launch(const NormArgs& a, int layer, int sms, cudaStream_t s) {
  const int threads = ((a.width + VEC * NV - 1) / (VEC * NV) + 31) / 32 * 32;
  const int rows = threads < 128 ? 128 / threads : 1;
  // As many blocks as 64 registers a thread let run at once.
  const int64_t blocks = (a.rows + rows - 1) / rows, most = (int64_t)sms * (1024 / (threads * rows));
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

template <typename T, int E, int VEC, bool LAYER, bool POST, int GATE, int MOST, bool FULL>
cudaError_t launch_most(const NormArgs& a, int sms, cudaStream_t s) {
  constexpr int kRing = has_ring<T, VEC>() ? rows_ahead<T, E>() * 2 * E * (int)sizeof(T) : 0;   // bytes a thread
  const int threads = ((a.width + E - 1) / E + 31) / 32 * 32;
  const int rows = threads < 128 ? 128 / threads : 1;
  const int smem = kRing * threads * rows;
  static OncePerDevice prepared;
  cudaError_t e = prepared.run([] {
    return cudaFuncSetAttribute(norm_stream_kernel<T, E, VEC, LAYER, POST, GATE, MOST, FULL>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * MOST);
  });
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.rows + rows - 1) / rows;
  int at_once = MOST / (threads * rows);               // by registers; and by shared memory
  if constexpr (kRing > 0)
    if (at_once > 200 * 1024 / smem) at_once = 200 * 1024 / smem;
  if (at_once < 1) at_once = 1;
  const int64_t most = (int64_t)sms * at_once;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
  cfg.blockDim = dim3(threads, rows);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  cfg.attrs = &overlapped;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_stream_kernel<T, E, VEC, LAYER, POST, GATE, MOST, FULL>, a);
}

// Elements and registers a thread.  RMS norms of 16-byte pieces: 16 elements
// at 128 registers, which halve what a row costs a warp besides its elements
// (8192 x 4096 bf16: 52 us, with 8 at 64 registers 54; a gate a token 54, 65),
// but 8 where there are no more rows than blocks, and one row's latency is
// the time (1 x 4096: 2.7 us, 3.5 with 16).  Layer norms keep two more
// parameters a column, single elements more addresses: 8 elements, at 128
// registers as far as blocks of 512 threads reach (1001 x 1537 fp32, layer
// norms: 12 us, at 64 registers 15).
template <typename T, int VEC, bool LAYER, bool POST, int GATE>
cudaError_t launch_stream(const NormArgs& a, int sms, cudaStream_t s) {
  if constexpr (LAYER || VEC == 1) {
    if (a.width <= 4096) return launch_most<T, 8, VEC, LAYER, POST, GATE, 512, false>(a, sms, s);
    return launch_most<T, 8, VEC, LAYER, POST, GATE, 1024, false>(a, sms, s);
  } else {
    if (a.rows <= 2 * sms) return launch_most<T, 8, VEC, LAYER, POST, GATE, 1024, false>(a, sms, s);
    return a.y && a.r && a.h && !a.codes ? launch_most<T, 16, VEC, LAYER, POST, GATE, 512, true>(a, sms, s)
                                         : launch_most<T, 16, VEC, LAYER, POST, GATE, 512, false>(a, sms, s);
  }
}

template <typename T, int VEC, bool LAYER, bool POST>
cudaError_t pick_gate(const NormArgs& a, int sms, cudaStream_t s) {
  if (!a.gate || (!a.gate_scalar && a.gate_span >= a.rows)) return launch_stream<T, VEC, LAYER, POST, 0>(a, sms, s);
  return a.gate_scalar ? launch_stream<T, VEC, LAYER, POST, 2>(a, sms, s)
                       : launch_stream<T, VEC, LAYER, POST, 1>(a, sms, s);
}

template <typename T, int VEC>
cudaError_t pick_norm(const NormArgs& a, int layer, int sms, cudaStream_t s) {
  if (layer) return a.post ? pick_gate<T, VEC, true, true>(a, sms, s) : pick_gate<T, VEC, true, false>(a, sms, s);
  return a.post ? pick_gate<T, VEC, false, true>(a, sms, s) : pick_gate<T, VEC, false, false>(a, sms, s);
}

}  // namespace

template <>
cudaError_t launch_norm<ECHO_ELEM>(const NormArgs& a, int layer, bool vec, int sms, cudaStream_t s) {
  using T = ECHO_ELEM;
  constexpr int V = 16 / sizeof(T);
  if (a.width > 8192) return vec ? launch<T, V, 16 / V>(a, layer, sms, s) : launch<T, 1, 16>(a, layer, sms, s);
  return vec ? pick_norm<T, V>(a, layer, sms, s) : pick_norm<T, 1>(a, layer, sms, s);
}

}  // namespace echo
