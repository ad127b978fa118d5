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
// contiguous range of rows and keeps the column sums of the parameters'
// gradients in registers over all of them; a second, small kernel adds the
// workers' sums in a fixed order.  Rows wider than one block's threads are
// split by columns over a cluster, whose blocks exchange the row sums through
// distributed shared memory.
//
// The bytes (12 a 16-bit element) leave an SM 2090 cycles a row of 4096, so
// instructions count: rows of 16-byte pieces come through a ring of
// asynchronous copies (others element by element, a row ahead in registers);
// scale, gate and weight are multiplied once (one gate row for all) or once a
// row; and with one gate row for all, or while a gate row lasts, only
// A = sum D a (and sum D) are kept, of which dw_post is scale gate A and dgate
// is scale (w_post A + b_post sum D).
//
// One GB300, bf16, RMS: 8192 x 4096 in 71 us, 5.7 TB/s, 0.84 of the copy rate,
// both kernels; 32768 x 4096 with a gate a token 343 us (a third row sum).
// Layer norms 109 us (twice the sums, eight elements a thread); 8192 x 12288 391
// us, layer norms 694 (clusters of two, spills).  Bound by instructions (scalar
// arithmetic: 679 a warp and row of 16 elements a thread, issue slots 59% busy)
// and the row sums' latency at 16 warps an SM.
#include "norm_common.h"

namespace echo {
namespace {

constexpr int kMaxCluster = 4;         // ECHO_NORM_MAX_WIDTH / (8 * kStreamThreads)

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// Sums of N values over a row's threads: those of its warps of this block and,
// in a cluster, of the other blocks'.  A warp writes its sum to the slot that
// belongs to it in every block; then one barrier (of the cluster, or of the
// block) and everyone adds the slots in the same order, four at a time (those
// past a row's warps stay 0).  Two sets of slots in turn, as a set is written
// again only behind the next sum's barrier.
constexpr int kStreamThreads = kNormGradThreads;
constexpr int kStreamSlots = kStreamThreads / 32 * kMaxCluster;

struct StreamSums {
  float (*slots)[3][kStreamSlots];     // [2]
  int first, count, warp, lane, blocks;
  int which;
  template <int N>
  __device__ __forceinline__ void all(float (&v)[N]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], d);
    if (count == 1) return;
    float(*s)[kStreamSlots] = slots[which];
    which ^= 1;
    if (blocks > 1) {
      if (lane < blocks) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          uint32_t at;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(at) : "r"(smem_u32(&s[k][first + warp])), "r"(lane));
          asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(at), "f"(v[k]) : "memory");
        }
      }
      cluster_barrier();
    } else {
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k][first + warp] = v[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float4* f = reinterpret_cast<const float4*>(&s[k][first]);
      v[k] = (f[0].x + f[0].y) + (f[0].z + f[0].w);
    }
    for (int i = 1; 4 * i < count; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float4 f = reinterpret_cast<const float4*>(&s[k][first])[i];
        v[k] += (f.x + f.y) + (f.z + f.w);
      }
  }
};

// A running sum that keeps what each addition rounds off (Kahan): a scalar
// gate's gradient adds width times rows terms, which often nearly cancel.
// Without it 40000 exact terms were 4e-6 off; 32768 x 4096 with a gate a token
// pays 4 of 343 us for it.
struct CarefulSum {
  float sum = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float y = __fsub_rn(v, lost), t = __fadd_rn(sum, y);
    lost = __fsub_rn(__fsub_rn(t, sum), y);
    sum = t;
  }
};

// Rows ahead in the ring of asynchronous copies: 128 KB for a full block.  E:
// elements of a row a thread has, 8 or 16.
template <typename T, int E> constexpr int rows_ahead() { return 64 / (E * (int)sizeof(T)); }
// Asynchronous copies take 16 bytes, or an fp32 element.
template <typename T, int VEC> constexpr bool has_ring() { return VEC * sizeof(T) >= 4; }
// 16-byte pieces of shared memory a thread has: the ring's (x, y, dr, dh) and
// its columns' fp32 parameters (mul, w, and for layer norms add).
template <typename T, int E, int VEC, bool LAYER>
constexpr int grad_pieces() {
  return (has_ring<T, VEC>() ? rows_ahead<T, E>() * 4 * (E * (int)sizeof(T) / 16) : 0) + (LAYER ? 3 : 2) * (E / 4);
}

// GATE: 0 none, or one row for all; 1 a row of gates, 2 a gate, for each row
// or several.
// FULL: x, y, dr, dh, dx and dy are all there (8192 x 4096 bf16: 74 us, with
// the branches 80).
template <typename T, int E, int VEC, bool LAYER, bool POST, int GATE, bool FULL>
__global__ void __launch_bounds__(kStreamThreads, 1)
norm_grad_kernel(const NormGradArgs a, int blocks, int block_cols) {
  constexpr int NV = E / VEC, kAhead = has_ring<T, VEC>() ? rows_ahead<T, E>() : 1;
  constexpr bool RING = has_ring<T, VEC>();
  constexpr bool SUM0 = LAYER && POST;                  // sum D is needed (db_post, dgate)
  extern __shared__ __align__(16) uint8_t room[];
  __shared__ __align__(16) float slots[2][3][kStreamSlots];
  const int tid = threadIdx.x, threads = blockDim.x, all_threads = threads * blockDim.y;
  const int me = threadIdx.y * threads + tid;
  const int part = (int)blockIdx.x % blocks;            // of the row's columns
  const int64_t worker = (int64_t)(blockIdx.x / blocks) * blockDim.y + threadIdx.y;
  const int col0 = part * block_cols, warps = threads / 32;
  StreamSums sums{slots, blockDim.y > 1 ? (int)threadIdx.y * 4 : 0, warps * blocks, part * warps + (tid >> 5),
                  tid & 31, blocks, 0};
  for (int i = me; i < 6 * kStreamSlots; i += all_threads) (&slots[0][0][0])[i] = 0.f;
  __syncthreads();
  if (blocks > 1) cluster_barrier();   // every block's slots are ready before the first is written
  const float inv_width = 1.0f / (float)a.width;
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) in[j] = (j * threads + tid) * VEC < block_cols && col0 + (j * threads + tid) * VEC < a.width;
  const int my_col = col0 + tid * VEC;                  // of piece j: + j * threads * VEC
  pdl_wait();
  pdl_trigger();

  const int64_t row0 = worker * a.span;
  const int64_t row1 = row0 + a.span < a.rows ? row0 + a.span : a.rows;
  constexpr uint32_t kBytes = VEC * sizeof(T);          // of a piece in the ring
  const uint32_t piece = 16u * all_threads, ring_piece = kBytes * all_threads, slot_bytes = 4 * NV * ring_piece;
  const uint32_t mine = smem_u32(room) + kBytes * me;
  const uint32_t params = smem_u32(room) + (RING ? kAhead * slot_bytes : 0u) + (VEC == 1 ? 4u : 16u) * me;
  auto start = [&](const void* p, int64_t ld) {
    return static_cast<const char*>(p) + (row0 * ld + my_col) * (int64_t)sizeof(T);
  };
  const char* from[4] = {start(a.x, a.ld_x), start(a.y, a.ld_y), start(a.dr, a.ld_dr), start(a.dh, a.ld_dh)};
  const bool has_y = FULL || a.y, has_dr = FULL || a.dr, has_dh = FULL || a.dh, has_dx = FULL || a.dx,
             has_dy = FULL || a.dy;
  const bool there[4] = {true, has_y, has_dr, has_dh};
  const int64_t far[4] = {a.ld_x * (int64_t)sizeof(T), a.ld_y * (int64_t)sizeof(T), a.ld_dr * (int64_t)sizeof(T),
                          a.ld_dh * (int64_t)sizeof(T)};
  // Whole pieces wait in the ring; single elements, which asynchronous copies
  // do not take, in registers.
  T held[RING ? 1 : 4][RING ? 1 : NV];
  int64_t fetch = row0;
  auto fetch_array = [&](int k, uint32_t slot) {
    if (fetch < row1 && there[k]) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (in[j]) {
          const char* at = from[k] + j * threads * (int)kBytes;
          const uint32_t to = mine + slot * slot_bytes + (4 * j + k) * ring_piece;
          if constexpr (!RING) held[k][j] = *reinterpret_cast<const T*>(at);
          else if constexpr (VEC == 1) copy4_async(to, at);
          else copy16_async(to, at);
        }
    }
    from[k] += far[k];
  };
  auto take = [&](int k, int j, uint32_t slot, float (&v)[VEC]) {
    const uint32_t at = mine + slot * slot_bytes + (4 * j + k) * ring_piece;
    if constexpr (!RING) v[0] = to_float(held[k][j]);
    else if constexpr (VEC == 1) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
    else to_floats<T, VEC>(load_shared16<T, VEC>(at), v);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
#pragma unroll
    for (int k = 0; k < 4; ++k) fetch_array(k, s);
    if (RING) copies_commit();
    ++fetch;
  }

  // The columns' parameters, as fp32 in this thread's shared memory: mul and
  // add of n * scale (times the gate, if it is one row) = hat1 * mul + add,
  // and w of the norm of r.
  auto put = [&](int at, int j, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      asm volatile("st.shared.f32 [%0], %1;" :: "r"(params + (uint32_t)(at * E + j) * (piece / 4)), "f"(v[0]) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                     :: "r"(params + (uint32_t)(at * (E / 4) + j * (VEC / 4) + i / 4) * piece), "f"(v[i]), "f"(v[i + 1]),
                        "f"(v[i + 2]), "f"(v[i + 3]) : "memory");
    }
  };
  auto get = [&](int at, int j, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(params + (uint32_t)(at * E + j) * (piece / 4)) : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                     : "r"(params + (uint32_t)(at * (E / 4) + j * (VEC / 4) + i / 4) * piece) : "memory");
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = my_col + j * threads * VEC;
    float g[VEC], m[VEC], w[VEC], b[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      g[i] = a.scale;
      m[i] = w[i] = 1.f;
      b[i] = 0.f;
    }
    if (in[j]) {
      if (GATE == 0 && a.gate) {
        load_param<T, VEC>(a.gate, a.params_f32, col, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] *= a.scale;
      }
      load_param<T, VEC>(a.w_pre, a.params_f32, col, 1.f, w);
      if (POST) load_param<T, VEC>(a.w_post, a.params_f32, col, 1.f, m);
      if (SUM0) load_param<T, VEC>(a.b_post, a.params_f32, col, 0.f, b);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      m[i] *= g[i];
      b[i] *= g[i];
    }
    put(0, j, m);
    put(1, j, w);
    if (LAYER) put(2, j, b);
  }

  float sum_a[NV][VEC], sum_d[SUM0 ? NV : 1][VEC];      // of D a, D: all rows, or the gate row's
  float sum_wpost[GATE == 1 ? NV : 1][VEC], sum_bpost[GATE == 1 && SUM0 ? NV : 1][VEC];
  float sum_wpre[NV][VEC], sum_bpre[LAYER ? NV : 1][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sum_a[j][i] = sum_wpre[j][i] = 0.f;
      if (SUM0) sum_d[j][i] = 0.f;
      if (GATE == 1) sum_wpost[j][i] = 0.f;
      if (GATE == 1 && SUM0) sum_bpost[j][i] = 0.f;
      if (LAYER) sum_bpre[j][i] = 0.f;
    }
  CarefulSum sum_scalar;
  int64_t gate_row = 0, gate_left = 0;
  bool gate_whole = false;             // the gate row's first row is this worker's
  if (GATE != 0) {
    gate_row = row0 / a.gate_span;
    gate_left = a.gate_span - (row0 - gate_row * a.gate_span);
    gate_whole = gate_left == a.gate_span;
  }
  char* to_dx = static_cast<char*>(a.dx) + (row0 * a.ld_dx + my_col) * (int64_t)sizeof(T);
  char* to_dy = static_cast<char*>(a.dy) + (row0 * a.ld_dy + my_col) * (int64_t)sizeof(T);
  const float4 no_stats = make_float4(0.f, 1.f, 0.f, 1.f);
  const float4* stats = pinned(reinterpret_cast<const float4*>(a.stats) + row0);
  auto load_stats = [&]() {
    const uint4 v = load_free16(stats);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  };
  float4 next_stats = a.stats && row0 < row1 ? load_stats() : no_stats;
  uint32_t slot = 0;

  for (int64_t step = 0; step < a.span; ++step) {
    const int64_t row = row0 + step;
    const bool active = row < row1;
    const float4 st = next_stats;
    ++stats;
    // The next row's are read here; with layer norms, of which a thread keeps
    // more, once this row's have been used (8192 x 4096 bf16: 109 us, here 112;
    // RMS norms 71 here and 86 there).
    if (!LAYER && a.stats && row + 1 < row1) next_stats = load_stats();
    float gate = 1.f;
    if (GATE == 2 && active) {
      float one[1];
      load_param<T, 1>(a.gate, a.params_f32, gate_row, one);
      gate = one[0];
    }
    if (RING) copies_wait<kAhead - 1>();
    float hat1[NV][VEC], hat2[NV][VEC], g[NV][VEC];     // g: dh w, then f
    float s[LAYER ? 2 : 1] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!active || !in[j]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) hat1[j][i] = hat2[j][i] = g[j][i] = 0.f;
        continue;
      }
      float x[VEC], m[VEC];
      take(0, j, slot, x);
      if (has_y) {
        take(1, j, slot, hat1[j]);
        if (POST)
#pragma unroll
          for (int i = 0; i < VEC; ++i) hat1[j][i] = LAYER ? (hat1[j][i] - st.x) * st.y : hat1[j][i] * st.y;
        get(0, j, m);
        if (GATE == 1) {
          float q[VEC];
          load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + my_col + j * threads * VEC, q);
#pragma unroll
          for (int i = 0; i < VEC; ++i) m[i] *= q[i];
          if (SUM0) {
            float b[VEC];
            get(2, j, b);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = fmaf(b[i], q[i], x[i]);
          }
        } else if (SUM0) {
          float b[VEC];
          get(2, j, b);
#pragma unroll
          for (int i = 0; i < VEC; ++i) x[i] = GATE == 2 ? fmaf(b[i], gate, x[i]) : x[i] + b[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = fmaf(hat1[j][i], GATE == 2 ? m[i] * gate : m[i], x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) hat1[j][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) hat2[j][i] = LAYER ? (x[i] - st.z) * st.w : x[i] * st.w;
      if (has_dh) {
        float w[VEC];
        take(3, j, slot, g[j]);
        get(1, j, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sum_wpre[j][i] = fmaf(g[j][i], hat2[j][i], sum_wpre[j][i]);
          if (LAYER) sum_bpre[j][i] += g[j][i];
          g[j][i] *= w[i];
          s[0] = fmaf(g[j][i], hat2[j][i], s[0]);
          if (LAYER) s[1] += g[j][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[j][i] = 0.f;
      }
    }
    if (!RING) {                        // what has been read makes room for the next row's
      fetch_array(0, 0);
      fetch_array(1, 0);
      fetch_array(3, 0);
    }
    if (LAYER && a.stats && row + 1 < row1) next_stats = load_stats();
    if (has_dh) {
      sums.all(s);
#pragma unroll
      for (float& v : s) v *= inv_width;
    }
    float t[(LAYER ? 2 : 1) + (GATE == 2 ? 1 : 0)] = {};
    constexpr int kScalar = LAYER ? 2 : 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!active || !in[j]) continue;
      float d[VEC];
      if (has_dr) {
        take(2, j, slot, d);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float back = fmaf(-s[0], hat2[j][i], LAYER ? g[j][i] - s[LAYER ? 1 : 0] : g[j][i]);
        d[i] = fmaf(st.w, back, d[i]);
      }
      if (has_dx) store_floats<T, VEC>(reinterpret_cast<T*>(to_dx) + j * threads * VEC, d);
      if (!has_y) continue;
      float m[VEC];
      get(0, j, m);
      if (GATE == 1) {
        float q[VEC];
        load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + my_col + j * threads * VEC, q);
#pragma unroll
        for (int i = 0; i < VEC; ++i) m[i] *= q[i];
      }
      if (GATE == 2) {
        const float k = a.scale * gate;
        float b[VEC];
        if (SUM0) get(2, j, b);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float n = SUM0 ? fmaf(hat1[j][i], m[i], b[i]) : hat1[j][i] * m[i];
          t[kScalar < (int)(sizeof(t) / sizeof(float)) ? kScalar : 0] += d[i] * n;
          m[i] *= gate;
          sum_a[j][i] = fmaf(d[i] * k, hat1[j][i], sum_a[j][i]);
          if (SUM0) sum_d[j][i] = fmaf(d[i], k, sum_d[j][i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sum_a[j][i] = fmaf(d[i], hat1[j][i], sum_a[j][i]);
          if (SUM0) sum_d[j][i] += d[i];
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        g[j][i] = d[i] * m[i];
        if (POST) {
          t[0] = fmaf(g[j][i], hat1[j][i], t[0]);
          if (LAYER) t[LAYER ? 1 : 0] += g[j][i];
        }
      }
    }
    if (!RING) {
      fetch_array(2, 0);
    } else {                            // this thread has read its pieces of the slot
#pragma unroll
      for (int k = 0; k < 4; ++k) fetch_array(k, slot);
      copies_commit();
      slot = slot == kAhead - 1 ? 0 : slot + 1;
    }
    ++fetch;
    if (POST || GATE == 2) {
      sums.all(t);
      t[0] *= inv_width;
      if (LAYER) t[LAYER ? 1 : 0] *= inv_width;
    }
    if (has_dy) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!active || !in[j]) continue;
        if (POST)
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            g[j][i] = st.y * fmaf(-t[0], hat1[j][i], LAYER ? g[j][i] - t[LAYER ? 1 : 0] : g[j][i]);
        store_floats<T, VEC>(reinterpret_cast<T*>(to_dy) + j * threads * VEC, g[j]);
      }
    }
    to_dx += a.ld_dx * sizeof(T);
    to_dy += a.ld_dy * sizeof(T);
    // A gate row ends, or this worker's part of it: a gate row whose rows are
    // all this worker's is written; of the others, the part of one that began
    // before its range goes to the worker's first slot, of one that goes on
    // behind it to the second, for norm_grad_finish.
    if (GATE != 0 && active) {
      if (GATE == 2) sum_scalar.add(t[kScalar < (int)(sizeof(t) / sizeof(float)) ? kScalar : 0]);
      if (--gate_left == 0 || row + 1 == row1) {
        const bool direct = gate_whole && gate_left == 0;
        const int64_t cols = GATE == 1 ? a.width : 1;
        float* part_of = a.gate_partial + (2 * worker + (gate_whole ? 1 : 0)) * cols;
        if (GATE == 1) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (!in[j]) continue;
            const int col = my_col + j * threads * VEC;
            float m[VEC], q[VEC];
            get(0, j, m);
            load_param<T, VEC>(a.gate, a.params_f32, gate_row * a.width + col, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              m[i] *= sum_a[j][i];
              sum_wpost[j][i] = fmaf(a.scale * q[i], sum_a[j][i], sum_wpost[j][i]);
              sum_a[j][i] = 0.f;
            }
            if (SUM0) {
              float b[VEC];
              get(2, j, b);
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                m[i] = fmaf(b[i], sum_d[j][i], m[i]);
                sum_bpost[j][i] = fmaf(a.scale * q[i], sum_d[j][i], sum_bpost[j][i]);
                sum_d[j][i] = 0.f;
              }
            }
            if (!a.dgate) continue;
            const int64_t at = gate_row * a.width + col;
            if (!direct) store_floats<float, VEC>(part_of + col, m);
            else if (a.params_f32) store_floats<float, VEC>(static_cast<float*>(a.dgate) + at, m);
            else store_floats<T, VEC>(static_cast<T*>(a.dgate) + at, m);
          }
        } else {
          if (a.dgate && tid == 0 && part == 0) {
            if (!direct) part_of[0] = sum_scalar.sum;
            else if (a.params_f32) static_cast<float*>(a.dgate)[gate_row] = sum_scalar.sum;
            else static_cast<T*>(a.dgate)[gate_row] = from_float<T>(sum_scalar.sum);
          }
          sum_scalar = CarefulSum();
        }
        if (gate_left == 0) {
          ++gate_row;
          gate_left = a.gate_span;
          gate_whole = true;
        }
      }
    }
  }
  if (RING) copies_wait<0>();

  if (worker < a.workers) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      const int64_t at = worker * a.width + my_col + j * threads * VEC;
      if (a.partial[0]) store_floats<float, VEC>(a.partial[0] + at, GATE == 1 ? sum_wpost[GATE == 1 ? j : 0] : sum_a[j]);
      if (SUM0 && a.partial[1])
        store_floats<float, VEC>(a.partial[1] + at, GATE == 1 ? sum_bpost[GATE == 1 && SUM0 ? j : 0] : sum_d[SUM0 ? j : 0]);
      if (a.partial[2]) store_floats<float, VEC>(a.partial[2] + at, sum_wpre[j]);
      if (LAYER && a.partial[3]) store_floats<float, VEC>(a.partial[3] + at, sum_bpre[LAYER ? j : 0]);
    }
  }
  // No block of a cluster may end while another can still write to its slots.
  if (blocks > 1) cluster_barrier();
}

// Adds the workers' column sums: blockIdx.y 0..3 a parameter each (with folded
// sums, 0 the gate too), from 4 on the gate rows that more than one worker
// shares, spread over the workers whose ranges begin inside one.
constexpr int kFinishRows = 32, kMaxGateBlocks = 32;

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
  auto parameter = [&](const void* p, float missing) {
    if (!p) return missing;
    return a.params_f32 ? static_cast<const float*>(p)[col] : to_float(static_cast<const T*>(p)[col]);
  };
  // The sum of one of the partials' columns (the block's, threads y = 0).
  auto total = [&](const float* partial) {
    float s = 0.f;
    if (col < a.width && partial) {
#pragma unroll 8
      for (int64_t w = threadIdx.y; w < a.workers; w += kFinishRows) s += partial[w * a.width + col];
    }
    __syncthreads();
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
      s = part[0][threadIdx.x];
      for (int i = 1; i < kFinishRows; ++i) s += part[i][threadIdx.x];
    }
    return s;
  };
  if (which == 0 && a.folded) {        // one gate row: dgate = scale (w_post sum D a + b_post sum D)
    if (!a.dparam[0] && !a.dgate) return;
    const bool bias = a.dgate && a.post && a.b_post;
    const float da = total(a.partial[0]), d = bias ? total(a.partial[1]) : 0.f;
    if (threadIdx.y == 0 && col < a.width) {
      if (a.dparam[0]) put(a.dparam[0], col, da * (a.scale * parameter(a.gate, 1.f)));
      if (a.dgate)
        put(a.dgate, col, a.scale * fmaf(a.post ? parameter(a.w_post, 1.f) : 1.f, da, bias ? parameter(a.b_post, 0.f) * d : 0.f));
    }
    return;
  }
  if (which < 4) {
    if (!a.dparam[which]) return;
    float s = total(a.partial[which]);
    if (threadIdx.y == 0 && col < a.width) {
      if (a.folded && which == 1) s *= a.scale * parameter(a.gate, 1.f);
      put(a.dparam[which], col, s);
    }
    return;
  }
  const int64_t cols = a.gate_scalar ? 1 : a.width;
  if (!a.dgate || col >= cols) return;
  // Worker b's range begins inside a gate row that began in worker b - 1's:
  // that one's second slot and the first slots of all that follow are its sum.
  for (int64_t b = 1 + threadIdx.y + (int64_t)kFinishRows * (which - 4); b < a.workers;
       b += (int64_t)kFinishRows * (gridDim.y - 4)) {
    const int64_t g = b * a.span / a.gate_span, begin = g * a.gate_span, end = begin + a.gate_span;
    if (begin == b * a.span || begin < (b - 1) * a.span) continue;
    const int64_t last = (end + a.span - 1) / a.span < a.workers ? (end + a.span - 1) / a.span : a.workers;
    const float first = a.gate_partial[(2 * (b - 1) + 1) * cols + col];
    if (a.gate_scalar) {
      CarefulSum s;
      s.add(first);
#pragma unroll 8
      for (int64_t w = b; w < last; ++w) s.add(a.gate_partial[2 * w]);
      put(a.dgate, g, s.sum);
    } else {
      float s = first;
#pragma unroll 8
      for (int64_t w = b; w < last; ++w) s += a.gate_partial[2 * w * cols + col];
      put(a.dgate, g * cols + col, s);
    }
  }
}

template <typename T>
cudaError_t launch_finish(const NormGradArgs& a, cudaStream_t s) {
  bool any = a.dgate && (a.folded || a.workers > 1);
  for (int k = 0; k < 4; ++k) any = any || a.dparam[k];
  if (!any) return cudaSuccess;
  cudaLaunchConfig_t fin = {};
  const int64_t gate_blocks = (a.workers + kFinishRows - 1) / kFinishRows;
  fin.gridDim = dim3((unsigned)((a.width + 31) / 32),
                     4 + (a.folded || !a.dgate ? 0 : (unsigned)(gate_blocks < kMaxGateBlocks ? gate_blocks : kMaxGateBlocks)));
  fin.blockDim = dim3(32, kFinishRows);
  fin.stream = s;
  cudaLaunchAttribute overlapped = overlapped_launch();
  fin.attrs = &overlapped;
  fin.numAttrs = 1;
  return cudaLaunchKernelEx(&fin, norm_grad_finish<T>, a);
}

template <typename T, int E, int VEC, bool LAYER, bool POST, int GATE, bool FULL>
cudaError_t launch_stream(NormGradArgs a, int sms, cudaStream_t s) {
  const NormGradShape shape(a.width, E);
  const int blocks = shape.blocks, block_cols = shape.block_cols, threads = shape.threads, rows = shape.rows;
  const int smem = grad_pieces<T, E, VEC, LAYER>() * 16 * threads * rows;
  static OncePerDevice prepared;
  cudaError_t e = prepared.run([] {
    return cudaFuncSetAttribute(norm_grad_kernel<T, E, VEC, LAYER, POST, GATE, FULL>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                grad_pieces<T, E, VEC, LAYER>() * 16 * kStreamThreads);
  });
  if (e != cudaSuccess) return e;
  const int64_t most = shape.workers(sms, 216 * 1024 / smem);
  a.span = (a.rows + most - 1) / most;
  a.workers = (a.rows + a.span - 1) / a.span;
  a.folded = GATE == 0;
  if (!(LAYER && POST)) a.partial[1] = nullptr;        // no b_post, no sum of D
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.workers + rows - 1) / rows * blocks));
  cfg.blockDim = dim3(threads, rows);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {overlapped_launch()};
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = blocks;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, norm_grad_kernel<T, E, VEC, LAYER, POST, GATE, FULL>, a, blocks, block_cols);
  return e != cudaSuccess ? e : launch_finish<T>(a, s);
}

// Elements a thread: 16 halve what a row costs a warp besides its elements,
// and fit 128 registers where a thread keeps two sums a column (8192 x 4096
// bf16, RMS: 80 us, with 8: 92); with three or more (layer norms, a row of
// gates) they spill (RMS, 128 gate rows: 185 us, with 8: 114), as does a row
// of single elements.  Past 4096 columns 8 need a cluster, whose barrier waits
// for the copies and stores in flight, so that 16 can be the lesser evil in
// spite of their spills.  In us with 16, with 8:
//   4096 x 8192, no gate or a scalar, RMS (no spills): bf16 76, 176
//   4096 x 8192, layer norms: bf16 195, 204; fp32 275, 229
//   4096 x 8192, layer norms, a row of gates: bf16 257, 235; fp32 302, 289
//   4096 x 8192, RMS, a row of gates: bf16 180, 206; fp32 239, 249
//     and without the norm after the block: bf16 152, 128; fp32 197, 166
//   4096 x 8200 (two blocks, three), layer norms: bf16 268, 495; fp32 385, 555
//   2048 x 12288, layer norms, a row of gates: bf16 257, 361; fp32 306, 427
// So 8 up to 8192 columns, the most that two blocks hold, for fp32 layer norms
// and for a row of gates where there are layer norms or no norm after the block.
template <typename T, int VEC, bool LAYER, bool POST, int GATE>
cudaError_t pick_elements(const NormGradArgs& a, int sms, cudaStream_t s) {
  if constexpr (VEC > 1 && !LAYER && GATE != 1) {
    return a.y && a.dr && a.dh && a.dx && a.dy ? launch_stream<T, 16, VEC, LAYER, POST, GATE, true>(a, sms, s)
                                               : launch_stream<T, 16, VEC, LAYER, POST, GATE, false>(a, sms, s);
  } else {
    constexpr bool kPair = (LAYER && sizeof(T) == 4) || (GATE == 1 && (LAYER || !POST));
    if constexpr (VEC > 1)
      if (a.width > (kPair ? 16 : 8) * kStreamThreads) return launch_stream<T, 16, VEC, LAYER, POST, GATE, false>(a, sms, s);
    return launch_stream<T, 8, VEC, LAYER, POST, GATE, false>(a, sms, s);
  }
}

template <typename T, int VEC, bool LAYER, bool POST>
cudaError_t pick_gate(const NormGradArgs& a, int sms, cudaStream_t s) {
  if (!a.gate || (!a.gate_scalar && a.gate_span >= a.rows)) return pick_elements<T, VEC, LAYER, POST, 0>(a, sms, s);
  return a.gate_scalar ? pick_elements<T, VEC, LAYER, POST, 2>(a, sms, s)
                       : pick_elements<T, VEC, LAYER, POST, 1>(a, sms, s);
}

template <typename T, int VEC>
cudaError_t pick_norm(const NormGradArgs& a, int layer, int sms, cudaStream_t s) {
  if (layer) return a.post ? pick_gate<T, VEC, true, true>(a, sms, s) : pick_gate<T, VEC, true, false>(a, sms, s);
  return a.post ? pick_gate<T, VEC, false, true>(a, sms, s) : pick_gate<T, VEC, false, false>(a, sms, s);
}

}  // namespace

template <>
cudaError_t launch_norm_grad<ECHO_ELEM>(NormGradArgs a, int layer, bool vec, int sms, cudaStream_t s) {
  using T = ECHO_ELEM;
  return vec ? pick_norm<T, 16 / sizeof(T)>(a, layer, sms, s) : pick_norm<T, 1>(a, layer, sms, s);
}

}  // namespace echo
