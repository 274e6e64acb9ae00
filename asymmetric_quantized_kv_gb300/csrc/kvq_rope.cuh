// The position rotation of kvq_rope_append, in the exact rounding of include/kvq.h:
// a pair (x, y) of channels becomes (x*c - y*s, x*s + y*c), every product and sum one
// fp32 operation, then one rounding to the source dtype.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

__device__ __forceinline__ float rope_first(float x, float y, float c, float s) {
  return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}
__device__ __forceinline__ float rope_second(float x, float y, float c, float s) {
  return __fadd_rn(__fmul_rn(x, s), __fmul_rn(y, c));
}

// The other channel of rotated channel c's pair.
__device__ __forceinline__ int rope_partner(const RopeView& r, int c) {
  return r.halves ? (c < r.rot / 2 ? c + r.rot / 2 : c - r.rot / 2) : c ^ 1;
}

// Channel c < rot of the token at position pos: x its value, y its partner's.  The result is
// rounded to the source dtype.
__device__ __forceinline__ float rope_channel(const RopeView& r, int pos, int c, float x, float y, int bf16) {
  const int half = r.rot / 2;
  const bool first = r.halves ? c < half : (c & 1) == 0;
  const int i = r.halves ? (first ? c : c - half) : c >> 1;
  const float* row = r.cs + (long long)pos * r.rot;
  const float z = first ? rope_first(x, y, row[i], row[half + i]) : rope_second(y, x, row[i], row[half + i]);
  return bf16 ? __bfloat162float(__float2bfloat16_rn(z)) : z;
}

}  // namespace kvq
