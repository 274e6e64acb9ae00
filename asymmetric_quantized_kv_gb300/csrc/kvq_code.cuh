// Exact conversions that the tensor-core kernels over PER_BLOCK caches share: 8-bit
// codes to f16, and bf16 values to f16 after scaling by a power of two.
#pragma once

#include "kvq_internal.cuh"
#include "kvq_ptx.cuh"

namespace kvq {

constexpr int kI8 = 0, kE4 = 1, kE5 = 2;  // formats as template arguments
constexpr int fmt_index(int fmt) { return fmt == KVQ_INT8 ? kI8 : fmt == KVQ_FP8_E4M3 ? kE4 : kE5; }

constexpr int kMinExp = -100;  // smallest value-scale exponent that rides in a softmax's (2^100 x 2^27 tokens stays finite)
// Exponent of values that are all zero: far below that of any others, whose weights would lose bits to theirs.
constexpr int kZeroExp = -32;

// The four 8-bit codes of a word as two f16x2 (bytes 0, 1 and 2, 3).
template <int F>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (F == kI8) {
    const uint32_t x = w ^ 0x80808080u;  // code + 128, into the mantissa of 1024
    lo = ptx::hsub2(ptx::prmt(x, 0x64646464u, 0x4140u), 0x64806480u);
    hi = ptx::hsub2(ptx::prmt(x, 0x64646464u, 0x4342u), 0x64806480u);
  } else if constexpr (F == kE4) {
    lo = ptx::e4m3x2_to_f16x2(ptx::lo16(w));
    hi = ptx::e4m3x2_to_f16x2(ptx::hi16(w));
  } else {  // E5M2 is the upper byte of an f16
    lo = ptx::prmt(w, 0u, 0x1404u);
    hi = ptx::prmt(w, 0u, 0x3424u);
  }
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// Exponent of |x| (x finite, not 0; subnormals count as 2^-126).
__device__ __forceinline__ int exponent_of(float x) { return max(1, (__float_as_int(x) >> 23) & 255) - 127; }

// A bf16 pair times a power of two, as f16x2.
__device__ __forceinline__ uint32_t bf16x2_scaled(uint32_t u, float s) {
  return ptx::pack_f16x2(__uint_as_float(u << 16) * s, __uint_as_float(u & 0xffff0000u) * s);
}
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t m, uint32_t u) {  // of magnitudes, as bits
  const uint32_t a = u & 0x7fff7fffu;
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(m), "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {  // of magnitudes, as bits
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The same of finite magnitudes, as bits + 0x80: infinities and NaN wrap to the bottom (a token that a row does not see
// then leaves the scaling of those it sees alone).
__device__ __forceinline__ uint32_t bf16x2_finite_max(uint32_t m, uint32_t u) {
  return bf16x2_absmax(m, (u & 0x7fff7fffu) + 0x00800080u);
}
__device__ __forceinline__ uint32_t finite_top(uint32_t m) {  // the larger of the two
  return max(max(m & 0xffffu, m >> 16), 0x80u) - 0x80u;
}
__device__ __forceinline__ uint32_t chunk_top(const uint4& x) {  // largest finite magnitude of 8 values
  return finite_top(bf16x2_finite_max(bf16x2_finite_max(bf16x2_finite_max(bf16x2_finite_max(0u, x.x), x.y), x.z), x.w));
}
// Numbers that are not finite have all exponent bits set (E4M3: and all of the mantissa's): one more in the lowest of
// these carries into the sign's place.
struct FiniteTest {
  uint32_t bits, one, sign;
  __device__ __forceinline__ uint32_t carry(uint32_t w) const { return (w & bits) + one; }  // or'ed over words, then:
  __device__ __forceinline__ bool fails(uint32_t carries) const { return (carries & sign) != 0u; }
};
constexpr FiniteTest kFiniteE4{0x7f7f7f7fu, 0x01010101u, 0x80808080u}, kFiniteE5{0x7c7c7c7cu, 0x04040404u, 0x80808080u};
constexpr FiniteTest kFiniteBf16x2{0x7f807f80u, 0x00800080u, 0x80008000u}, kFiniteF16x2{0x7c007c00u, 0x04000400u, 0x80008000u};
// Exponent k such that 2^-k brings values of largest magnitude `top` (bf16 bits) into [2^8, 2^9).
__device__ __forceinline__ int norm_exponent(uint32_t top) {
  const int k = exponent_of(__uint_as_float(top << 16)) - 8;
  return top == 0 ? 0 : max(-126, min(k, 119));
}
// The same for values, whose exponent rides in the softmax's.
__device__ __forceinline__ int value_exponent(uint32_t top) { return top == 0 ? kZeroExp : max(kMinExp, norm_exponent(top)); }
__device__ __forceinline__ void norm_factors(uint32_t top, float& down, float& up) {
  const int k = norm_exponent(top);
  down = pow2i(-k);
  up = pow2i(k);
}

}  // namespace kvq
