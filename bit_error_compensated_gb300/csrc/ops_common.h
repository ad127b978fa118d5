// ops_common.h -- shared by the operators around the all-reduce (norm_*.cu,
// int8_*.cu): element types, vector accesses, block sums, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/echo.h"

namespace echo {

int note_cuda_error(cudaError_t e);    // echo_api.cu

#define ECHO_OPS_CUDA(call)                                    \
  do {                                                         \
    cudaError_t e_ = (call);                                   \
    if (e_ != cudaSuccess) {                                   \
      cudaGetLastError();   /* the caller's next check is not this call's */ \
      return echo::note_cuda_error(e_);                        \
    }                                                          \
  } while (0)

// ------------------------------------------------------------------ device
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}

// N contiguous elements as they lie in memory, moved in 16-byte pieces (N * size a
// multiple of 16, 16-byte aligned) or, for N == 1, as one element.
template <typename T, int N>
struct __align__(sizeof(T) * N >= 16 ? 16 : sizeof(T) * N) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  Pack<T, N> out;
  if constexpr (N * sizeof(T) >= 16) {
    const uint4* src = reinterpret_cast<const uint4*>(p);
    uint4* dst = reinterpret_cast<uint4*>(&out);
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) dst[i] = src[i];
  } else {
    static_assert(N == 1, "packs are 16-byte pieces or single elements");
    out.v[0] = p[0];
  }
  return out;
}

template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& in) {
  if constexpr (N * sizeof(T) >= 16) {
    const uint4* src = reinterpret_cast<const uint4*>(&in);
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = src[i];
  } else {
    p[0] = in.v[0];
  }
}

// The elements of a pack as floats, and back, two at a time.
template <typename T, int N>
__device__ __forceinline__ void to_floats(const Pack<T, N>& in, float (&v)[N]) {
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t two = reinterpret_cast<const uint32_t*>(&in)[i / 2];
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        v[i] = __uint_as_float(two << 16);
        v[i + 1] = __uint_as_float(two & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
        v[i] = f.x;
        v[i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_float(in.v[i]);
  }
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> from_floats(const float (&v)[N]) {
  Pack<T, N> out;
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(v[i], v[i + 1]);
        reinterpret_cast<uint32_t*>(&out)[i / 2] = *reinterpret_cast<const uint32_t*>(&two);
      } else {
        const __half2 two = __floats2half2_rn(v[i], v[i + 1]);
        reinterpret_cast<uint32_t*>(&out)[i / 2] = *reinterpret_cast<const uint32_t*>(&two);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out.v[i] = from_float<T>(v[i]);
  }
  return out;
}

template <typename T, int N>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[N]) {
  store_pack<T, N>(p, from_floats<T, N>(v));
}

// 32 bytes, a whole sector, in one store (32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Copies of 16 bytes into shared memory that a thread reads back itself (no
// barrier between): in flight while it works, without registers.
__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4_async(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(PENDING) : "memory");
}
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_shared16(uint32_t at) {
  static_assert(sizeof(T) * N == 16, "one 16-byte piece");
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return *reinterpret_cast<const Pack<T, N>*>(&v);
}

// A barrier of all threads of a cluster.  Its instructions are .aligned: the
// lanes of a warp, which may have taken different branches on their way here,
// have to be together.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// See overlapped_launch below.  What a kernel reads of the one before, it reads
// behind the wait by ordinary loads: the read-only path (__ldg) is for memory
// that nothing writes while the kernel's blocks exist.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Ordinary loads of what nothing writes once the kernel is past its wait: the
// compiler may place them anywhere behind the point where their pointer was
// pinned, across other memory operations, as registers allow.
template <typename T>
__device__ __forceinline__ const T* pinned(const T* p) {
  asm volatile("" : "+l"(p) :: "memory");
  return p;
}
__device__ __forceinline__ uint4 load_free16(const void* p) {
  uint4 v;
  asm("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Zeros where the 16 bytes are not `there`, without a branch.
__device__ __forceinline__ uint4 load_free16(const void* p, bool there) {
  uint4 v;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((uint32_t)there));
  return v;
}
__device__ __forceinline__ uint32_t load_free4(const void* p) {
  uint32_t v;
  asm("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// The smallest amax a quantized row is scaled by.
constexpr float kTinyAmax = 7.703719777548943e-34f;   // 2^-110
// The largest |v| of a row as the bits of a float: unlike fmaxf this keeps
// NaNs (their bits are above infinity's).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// rint(v * inv) for |v| * inv <= 127 (with inv = 127 / amax, rounded); 0 for NaN.
__device__ __forceinline__ int quantize_code(float v, float inv) {
  return __float2int_rn(__fmul_rn(v, inv));
}

// -------------------------------------------------------------------- host
inline int elem_size(int dtype) { return dtype == ECHO_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) {
  return dtype == ECHO_F32 || dtype == ECHO_BF16 || dtype == ECHO_F16;
}
inline bool on_boundary(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Work done once per device by the first call that needs it (a kernel's
// attributes); calls that race do the same work twice.
struct OncePerDevice {
  std::atomic<uint64_t> done{0};
  template <typename F>
  cudaError_t run(F&& work) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = work();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// SMs of the current device.
inline cudaError_t device_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *sms = known[dev & 63].load(std::memory_order_relaxed);
  if (*sms) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) known[dev & 63].store(*sms, std::memory_order_relaxed);
  return e;
}

// Programmatic dependent launch: the kernel's blocks may be placed while the
// one before it in the stream still runs; each of these kernels waits
// (pdl_wait) before it touches memory, and lets the next one's blocks be
// placed (pdl_trigger) once it runs itself.
inline cudaLaunchAttribute overlapped_launch() {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}

// A strided matrix in memory: `rows` rows of `bytes` bytes, `pitch` bytes apart.
struct Region {
  uintptr_t at = 0;
  int64_t rows = 0, bytes = 0, pitch = 0;
};
inline Region region(const void* p, int64_t rows, int64_t cols, int64_t ld, int size) {
  Region r;
  if (p == nullptr || rows <= 0 || cols <= 0) return r;
  r.at = (uintptr_t)p;
  r.rows = rows;
  r.bytes = cols * size;
  r.pitch = ld * size;
  return r;
}
// Whether two matrices may share a byte.  Columns of one matrix, or rows of
// different tensors that alternate, do not: exact where the pitches are equal,
// by the whole ranges otherwise.
inline bool overlaps(const Region& a, const Region& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  const uintptr_t ea = a.at + (uintptr_t)((a.rows - 1) * a.pitch + a.bytes);
  const uintptr_t eb = b.at + (uintptr_t)((b.rows - 1) * b.pitch + b.bytes);
  if (ea <= b.at || eb <= a.at) return false;
  if (a.pitch == b.pitch && a.pitch > 0) {
    const bool first = a.at <= b.at;
    const int64_t d = (int64_t)((first ? b.at - a.at : a.at - b.at) % (uintptr_t)a.pitch);
    const int64_t low = first ? a.bytes : b.bytes, high = first ? b.bytes : a.bytes;
    if (d >= low && a.pitch - d >= high) return false;
  }
  return true;
}
inline bool same(const Region& a, const Region& b) {
  return a.at == b.at && a.rows == b.rows && a.bytes == b.bytes && (a.pitch == b.pitch || a.rows == 1);
}

}  // namespace echo
