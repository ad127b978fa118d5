// int8_load.h -- 16 codes of a row at a time, their conversion to f16, and the
// layout of the tokens' f16 codes in the workspace of a product.
#pragma once

#include "int8_common.h"

namespace echo {

// Codes k..k+15 of a row of `depth` codes, zeros behind its end (k a multiple
// of 16).  ALIGNED: rows start on 16-byte boundaries, so all but a ragged last
// piece is one load.  Otherwise a piece inside the row is put together from
// the aligned words around it, all of them inside the row too, and only a
// row's ends go byte by byte.  `row` is pinned behind the wait if the kernel
// before may write the codes.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_codes(const int8_t* row, int64_t k, int64_t depth) {
  const int8_t* p = row + k;
  if (ALIGNED && k + 16 <= depth) return load_free16(p);
  if (!ALIGNED && k >= 3 && k + 19 <= depth) {
    uint4 v;
    const uint32_t shift = (uint32_t)((uintptr_t)p & 3) * 8;
    const uint32_t* w = reinterpret_cast<const uint32_t*>((uintptr_t)p & ~(uintptr_t)3);
    const uint32_t a = load_free4(w), b = load_free4(w + 1), c = load_free4(w + 2), d = load_free4(w + 3);
    const uint32_t e = shift ? load_free4(w + 4) : 0;
    v.x = __funnelshift_r(a, b, shift);
    v.y = __funnelshift_r(b, c, shift);
    v.z = __funnelshift_r(c, d, shift);
    v.w = __funnelshift_r(d, e, shift);
    return v;
  }
  uint64_t low = 0, high = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    if (k + i < depth) low |= (uint64_t)(uint8_t)p[i] << (8 * i);
    if (k + i + 8 < depth) high |= (uint64_t)(uint8_t)p[i + 8] << (8 * i);
  }
  return make_uint4((uint32_t)low, (uint32_t)(low >> 32), (uint32_t)high, (uint32_t)(high >> 32));
}

// Four codes as two pairs of f16, exactly: with the sign bit turned a code is
// 128 more than it was, and behind the byte 0x64 it is the significand of
// 1024 + (code + 128); 1152 is then taken off.
__device__ __forceinline__ void codes_to_f16(uint32_t four, uint32_t& low, uint32_t& high) {
  const uint32_t u = four ^ 0x80808080u;
  const __half2 bias = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
  const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), bias);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), bias);
  low = *reinterpret_cast<const uint32_t*>(&a);
  high = *reinterpret_cast<const uint32_t*>(&b);
}

// The workspace of a product of many tokens holds their codes as f16 in the
// blocks that a copy takes to shared memory whole: 128 tokens x 128 codes, two
// halves of 64 codes, each row's 128 bytes in eight 16-byte pieces that are
// swizzled (piece ^ row % 8), as the matrix instruction reads them.
constexpr int kBlockTokens = 128, kBlockCodes = 128;
constexpr int kBlockBytes = kBlockTokens * kBlockCodes * 2;

__host__ __device__ inline int64_t wide_blocks(int64_t extent) { return (extent + 127) / 128; }

// Where code k (a multiple of 8) of token t of a rank lies: its byte offset.
__device__ __forceinline__ int64_t wide_offset(int64_t rank, int64_t t, int64_t k, int64_t tokens, int64_t depth) {
  const int64_t block = (rank * wide_blocks(tokens) + (t >> 7)) * wide_blocks(depth) + (k >> 7);
  const uint32_t r = (uint32_t)t & 127u, c = (uint32_t)k & 127u;
  return block * kBlockBytes + (c >> 6) * (kBlockBytes / 2) + r * 128 + ((((c & 63u) >> 3) ^ (r & 7u)) << 4);
}

}  // namespace echo
