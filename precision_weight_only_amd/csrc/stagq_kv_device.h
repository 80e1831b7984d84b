// Device helpers shared by the kernels of the key/value cache in 4 bits.
#pragma once
#include <hip/hip_runtime.h>

#include "stagq.h"
#include "stagq_kv_layout.h"

namespace stagq {
namespace kv {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// A lane's chunk of N code dwords (12-byte ones are 4-byte aligned).
template <int N>
struct Chunk;
template <> struct Chunk<2> { typedef u2_t type; };
template <> struct Chunk<3> { struct type { uint32_t v[3]; __device__ uint32_t operator[](int i) const { return v[i]; } }; };
template <> struct Chunk<4> { typedef u4_t type; };

// One strided tensor [batch, tokens, heads, head_dim].
struct Tensor {
  uint8_t* data;
  int dtype, tokens, heads;
  int64_t sb, st, sh;  // elements
};

// The cache and the sequences of one call.
struct Cache {
  uint8_t* buf;
  const int* table;
  const int* lengths;
  int64_t table_stride;
  uint64_t page_bytes;
  uint32_t head_bytes;
  int pages, width, shift;  // page_tokens = 1 << shift
  int heads, batch;
};

__device__ __forceinline__ float half_bits(uint32_t h) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ uint32_t bits_half(_Float16 h) { return __builtin_bit_cast(uint16_t, h); }

// Start of the head's part of the page that holds a slot; null where there is
// no page (slot outside the table, entry outside the pages).
__device__ __forceinline__ uint8_t* page_head(const Cache& c, int b, int head, int64_t slot) {
  const int64_t e = slot >> c.shift;
  if (slot < 0 || e >= c.width) return nullptr;
  const int page = c.table[int64_t(b) * c.table_stride + e];
  if (page < 0 || page >= c.pages) return nullptr;
  return c.buf + uint64_t(page) * c.page_bytes + uint64_t(head) * c.head_bytes;
}
// Start of the 32-token block that holds a slot.
template <int D, int G>
__device__ __forceinline__ uint8_t* block_at(const Cache& c, int b, int head, int64_t slot) {
  uint8_t* h = page_head(c, b, head, slot);
  if (!h) return nullptr;
  return h + uint32_t((slot & ((int64_t(1) << c.shift) - 1)) / kBlock) * block_bytes(D, G);
}

// The eight codes of a dword as fp16 pairs (2i, 2i + 1) of value u * 2^-20: the
// codes go to mantissa bits 4..7 of fp16 subnormals, which the matrix
// instruction takes as they are.  Bits 0..3 would save two of the shifts, but
// there the instruction's alignment of the products drops low bits (measured:
// errors up to 2^-17.4 of the largest product instead of 2^-22.9).
constexpr float kCodeUnit = 1048576.0f;  // 2^20
__device__ __forceinline__ h8_t codes8(uint32_t x) {
  const uint32_t m = 0x00f000f0u;
  u4_t r;
  r[0] = (x << 4) & m;
  r[1] = x & m;
  r[2] = (x >> 4) & m;
  r[3] = (x >> 8) & m;
  return __builtin_bit_cast(h8_t, r);
}
// The same codes as fp16 integers: 1024 + u by the exponent's bits, minus 1024.
__device__ __forceinline__ h2_t code_pair(uint32_t x, int i) {
  const uint32_t w = ((x >> (4 * i)) & 0x000f000fu) | 0x64006400u;
  const h2_t k = {(_Float16)1024.0f, (_Float16)1024.0f};
  return __builtin_bit_cast(h2_t, w) - k;
}

// And divided by 256 (exact).
__device__ __forceinline__ h2_t code_pair_256th(uint32_t x, int i) {
  const uint32_t w = ((x >> (4 * i)) & 0x000f000fu) | 0x64006400u;
  const h2_t m = {(_Float16)0.00390625f, (_Float16)0.00390625f}, k = {(_Float16)-4.0f, (_Float16)-4.0f};
  return __builtin_elementwise_fma(__builtin_bit_cast(h2_t, w), m, k);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Reductions over the four lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ float max_sets(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_sets(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Reductions over the sixteen lanes of one residue modulo 4.
__device__ __forceinline__ float max_quads(float v) {
#pragma unroll
  for (int d = 4; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float sum_quads(float v) {
#pragma unroll
  for (int d = 4; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ void unpack8(const uint8_t* p, int dtype, float* f) {
  if (dtype == STAGQ_F32) {
    const f4_t a = *reinterpret_cast<const f4_t*>(p), b = *reinterpret_cast<const f4_t*>(p + 16);
    for (int i = 0; i < 4; i++) { f[i] = a[i]; f[4 + i] = b[i]; }
  } else {
    const u4_t v = *reinterpret_cast<const u4_t*>(p);
    if (dtype == STAGQ_F16) {
      const h8_t h = __builtin_bit_cast(h8_t, v);
      for (int i = 0; i < 8; i++) f[i] = (float)h[i];
    } else {
      for (int i = 0; i < 4; i++) {
        f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
        f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
      }
    }
  }
}
// Element e of eight bf16 values.
__device__ __forceinline__ float bf16_of(u4_t v, int e) {
  const uint32_t w = v[e / 2];
  return __builtin_bit_cast(float, (e & 1) ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ h4_t low4(h8_t v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3); }
__device__ __forceinline__ h4_t high4(h8_t v) { return __builtin_shufflevector(v, v, 4, 5, 6, 7); }
__device__ __forceinline__ uint16_t to_16(float v, int dtype) {  // one rounding, nearest even
  if (dtype == STAGQ_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// 2^e with e chosen so that the largest magnitude of a bf16 row lands in
// [2^14, 2^15): the row times 2^e in fp16 is exact but for elements some 2^24
// below the largest.  1 for a row of zeros and one with an infinity or NaN
// (which stay what they are).
__device__ __forceinline__ float row_scale(float amax) {
  const uint32_t e = (__builtin_bit_cast(uint32_t, amax) >> 23) & 255u;
  if (e == 0u || e == 255u) return 1.0f;
  int f = 127 + 14 + 127 - int(e);
  f = f > 254 ? 254 : f;
  return __builtin_bit_cast(float, uint32_t(f) << 23);
}

}  // namespace kv
}  // namespace stagq
