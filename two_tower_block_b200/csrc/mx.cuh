// The microscaled element format of the quantised context cache: e4m3 values (4 exponent bits,
// bias 7, 3 mantissa bits, largest 448) with one scale per 32 elements along the head dimension,
// a power of two 2^e held as the byte e + 127 (0..254).
//
// An e4m3 value times a power of two has 4 significant bits, so it is exact in bf16 (8 bits) down
// to bf16's subnormals: attention over the cache is attention over exactly representable bf16
// operands, and the tensor cores' bf16 form takes them without a further rounding.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace tt {

constexpr int kMxBlock = 32;   // elements per scale

// Multipliers (each a bf16 pair of equal values) whose product is 2^(120 + e), e = byte - 127:
// two factors, because 2^(120 + e) itself is beyond bf16 for e > 7.
struct MxScale {
  uint32_t a, b;
};
__device__ __forceinline__ MxScale mx_scale(uint32_t byte) {
  const int e = (int)byte - 127;
  const int h = e >> 1;
  MxScale s;
  s.a = (uint32_t)(60 + 127 + h) * 0x00800080u;        // exponent field at bit 7 of both halves
  s.b = (uint32_t)(60 + 127 + e - h) * 0x00800080u;
  return s;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Four e4m3 bytes -> four bf16 (two pairs, memory order), scaled.  The seven magnitude bits of a
// byte moved under bf16's exponent field read as the value times 2^-120 (exact for e4m3's
// subnormals too: they land on bf16 subnormals).
__device__ __forceinline__ uint2 mx_to_bf16x4(uint32_t w, MxScale s) {
  const uint32_t lo = __byte_perm(w, 0u, 0x1404), hi = __byte_perm(w, 0u, 0x3424);
  const uint32_t x = (lo & 0x80008000u) | ((lo >> 4) & 0x07F007F0u);
  const uint32_t y = (hi & 0x80008000u) | ((hi >> 4) & 0x07F007F0u);
  return make_uint2(mul_bf16x2(mul_bf16x2(x, s.a), s.b), mul_bf16x2(mul_bf16x2(y, s.a), s.b));
}

}  // namespace tt
