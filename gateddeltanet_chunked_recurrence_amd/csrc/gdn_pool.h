// Device helpers of the state pool kernels: slot checks and page codes.
#pragma once
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

__device__ __forceinline__ void pool_error(const PoolRef& p) {
  __hip_atomic_fetch_or(p.err, kErrPoolSlot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether another entry than `n` reads (in[j]) or writes (out[j]) slot `dst`,
// so that entry `n` may not write it. Every wave that writes a part of the page
// asks this, with the same answer in each, so an index given twice leaves the
// page as it was instead of a mixture of two results. Entries that touch no
// page do not count: those refused for a slot outside the pool, and those with
// nothing to do. COPY: an entry reads in[j] (-1: none, the page is cleared) and
// writes out[j] >= 0, unless the two are one. Otherwise it reads in[j] >= 0 and
// writes out[j] (-1: not kept), unless it has no token (lens, of T at most) and
// no other page to copy to. All 64 lanes call this together; each takes four
// entries per load (the arrays are 16-byte aligned), and four loads are in
// flight at once: 1,024 entries cost one round trip to L2. The last vector is
// read again by lanes past it (asking twice changes nothing). lens is read only
// where an entry names the slot.
template <bool COPY>
__device__ __forceinline__ bool pool_claimed(const PoolRef& p, const int32_t* in, const int32_t* out, int count,
                                             int n, int dst, int T = 1, const int32_t* lens = nullptr) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  const int lane = __lane_id(), nv = count >> 2;
  bool hit = false;
  const uint32_t slots = (uint32_t)p.slots;
  auto test = [&](int j, int a, int b) {
    bool names = (j != n) & ((a == dst) | (b == dst));
    if constexpr (COPY) names &= ((uint32_t)a + 1u <= slots) & ((uint32_t)b < slots) & (a != b);
    else names &= ((uint32_t)a < slots) & ((uint32_t)b + 1u <= slots);
    hit |= names;
  };
  for (int v0 = 0; v0 < nv; v0 += 4 * WAVE) {
    i32x4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v0 + u * WAVE < nv) a[u] = reinterpret_cast<const i32x4*>(in)[min(v0 + u * WAVE + lane, nv - 1)];
    if (in != out) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v0 + u * WAVE < nv) b[u] = reinterpret_cast<const i32x4*>(out)[min(v0 + u * WAVE + lane, nv - 1)];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v0 + u * WAVE < nv)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          test(4 * min(v0 + u * WAVE + lane, nv - 1) + e, a[u][e], in != out ? b[u][e] : a[u][e]);
  }
  const int last = 4 * nv + lane;
  if (last < count) test(last, in[last], out[last]);
  if (__ballot(hit) == 0) return false;
  if (!COPY && (T == 0 || lens)) {               // seldom: the entries that name the slot, by their tokens
    hit = false;
    for (int j = lane; j < count; j += WAVE) {
      const int a = in[j], b = out[j];
      if (j == n || (a != dst && b != dst) || (uint32_t)a >= slots || (uint32_t)b + 1u > slots) continue;
      hit |= (T > 0 && (!lens || lens[j] > 0)) || (b != a && b != -1);
    }
    return __ballot(hit) != 0;
  }
  return true;
}

// An E4M3 code can be NaN, an integer one cannot: an INT8 tile with a value that
// is not finite takes the scale NaN, so that every later read and step of it is
// NaN instead of what the codes happen to be. So its amax keeps a NaN
// (v_maximum3_f32: as many instructions as a maximum that leaves NaN out).
template <int FMT>
__device__ __forceinline__ float larger(float m, float x) {
  if constexpr (FMT == 2) return __builtin_elementwise_maximum(m, fabsf(x));
  else return fmaxf(m, fabsf(x));
}
template <int FMT>
__device__ __forceinline__ float wave_largest(float m) {  // as wave_max
  m = larger<FMT>(m, dpp_f<0xB1>(m));
  m = larger<FMT>(m, dpp_f<0x4E>(m));
  m = larger<FMT>(m, dpp_f<0x141>(m));
  m = larger<FMT>(m, dpp_f<0x140>(m));
  return larger<FMT>(larger<FMT>(read_lane(m, 0), read_lane(m, 16)), larger<FMT>(read_lane(m, 32), read_lane(m, 48)));
}

// The tile scale under the pool's rule: amax / q_max as gdn_qdq_state, or amax
// times the FP32-rounded 1 / q_max as PyTorch divides a tensor by a number.
// INT8: plus 0, or NaN where amax is not finite.
template <int FMT>
__device__ __forceinline__ float pool_scale(const PoolRef& p, float amax) {
  constexpr float kRecip = 1.0f / QdqFmt<FMT>::qmax;
  const float d = p.recip ? fmaxf(amax * kRecip, 1.17549435e-38f) : qdq_scale<FMT>(amax);
  return FMT == 2 ? d + (amax - amax) : d;
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

// Eight codes (two words) as the bf16 values they are (exact: E4M3 has four
// significant bits, the integers at most seven).
template <int FMT>
__device__ __forceinline__ bf16x8 codes8_bf16(uint32_t w0, uint32_t w1) {
  bf16x8 b;
  if constexpr (FMT == 1) {
    typedef bf16 bf16x2v __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int w = static_cast<int>(h < 2 ? w0 : w1);
      const bf16x2v x = (h & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
      b[2 * h] = x[0];
      b[2 * h + 1] = x[1];
    }
  } else {
    float x[8];
    codes4<FMT>(w0, *reinterpret_cast<float(*)[4]>(&x[0]));
    codes4<FMT>(w1, *reinterpret_cast<float(*)[4]>(&x[4]));
#pragma unroll
    for (int c = 0; c < 8; ++c) b[c] = to_bf16(x[c]);
  }
  return b;
}

// Four values of a tile to the word of their codes c = RNE(fl(x r)), r = fl(1/d)
// from the tile's own amax, so no clamp is needed (see quant4 in
// gdn_device.h). The integer format rounds by adding 1.5 * 2^23: the sum's
// low byte is the integer in two's complement (|x r| <= 127 (1 + 2^-21) < 2^22),
// one add instead of a rounding, a conversion and a mask.
template <int FMT>
__device__ __forceinline__ uint32_t quant_word(const float (&x)[4], float r) {
  if constexpr (FMT == 1) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r, x[1] * r, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r, x[3] * r, lo, true));
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
    }
    // bytes (b0, b1) and (b2, b3) into halves, then into one word
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
    return lo | (hi << 16);
  }
}

}  // namespace gdn
