// Device helpers of the state pool kernels: slot checks and page codes.
#pragma once
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

__device__ __forceinline__ void pool_error(const PoolRef& p) {
  __hip_atomic_fetch_or(p.err, kErrPoolSlot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether entry `n` may write slot `dst`: no other entry j that does
// something (in[j] >= lo and out[j] >= 0) may read it (in[j]) or write it
// (out[j]). Every wave that writes a part of the page asks this, with the
// same answer in each, so an index given twice leaves the page as it was
// instead of a mixture of two results. All 64 lanes call it together; each
// takes four entries per step (the arrays are 16-byte aligned).
__device__ __forceinline__ bool pool_claimed(const int32_t* in, const int32_t* out, int count, int n,
                                             int dst, int lo) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  bool hit = false;
  for (int j0 = 4 * (int)__lane_id(); j0 < count; j0 += 4 * WAVE) {
    if (j0 + 4 <= count) {
      const i32x4 a = *reinterpret_cast<const i32x4*>(in + j0);
      const i32x4 b = in == out ? a : *reinterpret_cast<const i32x4*>(out + j0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        hit |= j0 + e != n && a[e] >= lo && b[e] >= 0 && (a[e] == dst || b[e] == dst);
    } else {
      for (int j = j0; j < count; ++j) {
        const int a = in[j], b = out[j];
        hit |= j != n && a >= lo && b >= 0 && (a == dst || b == dst);
      }
    }
  }
  return __ballot(hit) != 0;
}

// Four codes of one word as floats (unscaled).
template <int FMT>
__device__ __forceinline__ void codes4(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == 1) {
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    const f32x2v lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f32x2v hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    x[0] = lo[0];
    x[1] = lo[1];
    x[2] = hi[0];
    x[3] = hi[1];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = static_cast<float>(static_cast<int8_t>((w >> (8 * e)) & 0xFFu));
  }
}

// Four values of a tile to codes c = RNE(fl(x r)) and their word, r = fl(1/d)
// from the tile's own amax, so no clamp is needed (see quant4 in
// gdn_device.h). The integer format rounds by adding 1.5 * 2^23: the sum's
// low byte is the integer in two's complement and the difference the value
// (|x r| <= 127 (1 + 2^-21) < 2^22), one add each instead of a rounding, a
// conversion and a mask.
template <int FMT>
__device__ __forceinline__ uint32_t quant_word(float (&x)[4], float r) {
  if constexpr (FMT == 1) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r, x[1] * r, 0, false);
    const uint32_t w = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r, x[3] * r, lo, true));
    codes4<1>(w, x);
    return w;
  } else {
    // the product rounds before the sum (no fused multiply-add)
#pragma clang fp contract(off)
    constexpr float kMagic = 12582912.f;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p = x[e] * r;
      const float y = p + kMagic;
      b[e] = __builtin_bit_cast(uint32_t, y);
      x[e] = y - kMagic;
    }
    // bytes (b0, b1) and (b2, b3) into halves, then into one word
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
    return lo | (hi << 16);
  }
}

}  // namespace gdn
