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

// A scale byte as multipliers of values that read 2^120 too small (mx_to_bf16x4): 2^(120 + e) as a
// bf16 pair of equal values, and for e > 7, where that leaves bf16, the rest as a second one.
constexpr uint32_t kMxOneFactor = 134;   // largest byte (e = 7) that one factor holds
__device__ __forceinline__ uint32_t mx_factor(uint32_t byte) { return min(byte + 120u, 254u) * 0x00800080u; }
__device__ __forceinline__ uint32_t mx_rest(uint32_t byte) {
  return (127u + (byte > kMxOneFactor ? byte - kMxOneFactor : 0u)) * 0x00800080u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Four e4m3 bytes -> four bf16 (two pairs, memory order) times `factor`.  Each byte is widened to 16
// bits with its sign (the permute's sign mode) and moved up by four: its seven magnitude bits then lie
// at the bottom of bf16's exponent and the top of its mantissa, which reads as the value times 2^-120
// (exact for e4m3's subnormals too: they land on bf16 subnormals).
__device__ __forceinline__ uint2 mx_to_bf16x4(uint32_t w, uint32_t factor) {
  uint32_t x, y;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(x) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(y) : "r"(w));
  return make_uint2(mul_bf16x2((x << 4) & 0x87F087F0u, factor), mul_bf16x2((y << 4) & 0x87F087F0u, factor));
}
// e4m3's NaN (all seven magnitude bits set) among four bytes: adding one to every byte carries into bit 7 of
// such a byte, and of no other unless a NaN lies below it.  Non-zero in the bits kMxNan: there is one.
constexpr uint32_t kMxNan = 0x80808080u;
__device__ __forceinline__ uint32_t mx_nan_bits(uint32_t w) { return (w + 0x01010101u) ^ w; }
// The NaNs of a word over the four bf16 that mx_to_bf16x4 makes of it (480 times the scale).
__device__ __forceinline__ uint2 mx_keep_nan(uint2 v, uint32_t w) {
  const uint32_t n = (w & 0x7F7F7F7Fu) + 0x01010101u;   // bit 7 of a byte; to bit 0 of its half, times a NaN's bits
  return make_uint2(v.x | (((n >> 7) & 1u) | ((n << 1) & 0x10000u)) * 0x7FC0u,
                    v.y | (((n >> 23) & 1u) | ((n >> 15) & 0x10000u)) * 0x7FC0u);
}
// Eight bytes of one scale block -> eight bf16, NaN where they are e4m3's.
__device__ __forceinline__ uint4 mx_to_bf16x8(uint2 w, uint32_t byte) {
  const uint32_t f = mx_factor(byte);
  const uint2 a = mx_to_bf16x4(w.x, f), b = mx_to_bf16x4(w.y, f);
  uint4 r = make_uint4(a.x, a.y, b.x, b.y);
  if (byte > kMxOneFactor) {
    const uint32_t g = mx_rest(byte);
    r = make_uint4(mul_bf16x2(r.x, g), mul_bf16x2(r.y, g), mul_bf16x2(r.z, g), mul_bf16x2(r.w, g));
  }
  if ((mx_nan_bits(w.x) | mx_nan_bits(w.y)) & kMxNan) {
    const uint2 x = mx_keep_nan(make_uint2(r.x, r.y), w.x), y = mx_keep_nan(make_uint2(r.z, r.w), w.y);
    r = make_uint4(x.x, x.y, y.x, y.y);
  }
  return r;
}

}  // namespace tt
