// Rules on logits before a choice: penalties of repeated tokens, biases, grammar
// masks. Per row (beam w of request b) and token t, with n_t the times that t was
// generated and "said" meaning that it occurs in the prompt or the generation:
//   x <- said(t) ? (x > 0 ? x / rho : x rho) : x
//   x <- x - freq n_t - pres [n_t > 0]
//   x <- x + bias_t
//   x <- -inf where the row's mask has bit t 0
// in FP32, rounded once. Tokens that no rule names keep their bits.
//
// Bound: the logits, read and written once; the rules are sparse but for the mask.
// A workgroup takes one tile of a row's vocabulary with a word of LDS per token.
// First the history and the biases mark the words of their tokens in the tile (a
// count, a flag, the bias's place: integer atomics, so their order does not
// matter). Then they are walked again: the first to set a token's bit owns it, gathers
// its logit, and leaves the result in its word. The dense pass is a copy that looks
// the words up: no division and no branch in it.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

// A word of the tile: 0, or while marked: flag "said" (31), the bias's place plus
// one (20..30), times generated (0..19); then the result, never 0.
constexpr uint32_t kSaid = 0x80000000u;
constexpr int kPlaceShift = 20;
constexpr uint32_t kTimes = (1u << kPlaceShift) - 1, kPlace = 0x7FFu;

template <bool F32> struct Io;
template <> struct Io<false> {
  using T = uint16_t;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float wide(T x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
  static __device__ __forceinline__ uint32_t result(float x) {
    const bf16 b = to_bf16(x);
    return 0x10000u | __builtin_bit_cast(uint16_t, b);
  }
  static __device__ __forceinline__ T take(uint32_t w) { return (T)w; }
  static constexpr T LOWEST = 0xFF80u, NANV = 0x7FC0u;
};
template <> struct Io<true> {
  using T = uint32_t;
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float wide(T x) { return __builtin_bit_cast(float, x); }
  // a NaN is made the canonical one, so that no result is 0
  static __device__ __forceinline__ uint32_t result(float x) {
    return (x != x ? 0x7FC00000u : __builtin_bit_cast(uint32_t, x)) ^ 0x7FFFFFFFu;
  }
  static __device__ __forceinline__ T take(uint32_t w) { return w ^ 0x7FFFFFFFu; }
  static constexpr T LOWEST = 0xFF800000u, NANV = 0x7FC00000u;
};

template <bool F32, int THREADS>
__global__ void __launch_bounds__(THREADS) rules_kernel(RulesArgs a) {
  using I = Io<F32>;
  using T = typename I::T;
  constexpr int VEC = I::VEC, ES = sizeof(T);
  typedef T Vec __attribute__((ext_vector_type(VEC)));
  extern __shared__ __attribute__((aligned(16))) uint32_t word[];   // [tile], [tile / 32] owned, bias ids and values
  const int row = blockIdx.x / a.tiles, tile = blockIdx.x - row * a.tiles, b = row / a.W, tid = threadIdx.x;
  const T* in = static_cast<const T*>(a.logits) + (int64_t)row * a.in_stride;
  T* out = static_cast<T*>(a.out) + (int64_t)row * a.out_stride;
  // a tile is whole vectors of the output: the first one starts before the row where
  // that is not aligned
  const int skew = (int)((reinterpret_cast<uintptr_t>(out) / ES) % VEC);
  const int v0 = tile * a.tile - skew, lo = max(v0, 0), hi = min(v0 + a.tile, a.V);
  if (lo >= hi) return;
  const int mrow = a.mask ? (a.mask_rows ? a.mask_rows[row] : row) : -1;
  if (mrow < -1 || mrow >= a.masks) {                     // no such mask: the row says so
    if (tid == 0 && a.mask) __hip_atomic_fetch_or(a.err, kErrRuleRow, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (a.mask) {
      for (int v = lo + tid; v < hi; v += THREADS) out[v] = I::NANV;
      return;
    }
  }
  const uint32_t low = lo - v0, high = hi - v0;
  const bool marks = a.tokens || a.nb > 0;
  if (marks) {
    uint32_t* const owned = word + a.tile;
    int32_t* const ids = reinterpret_cast<int32_t*>(owned + a.tile / 32);
    float* const add = reinterpret_cast<float*>(ids + a.nb);
    for (int i = 4 * tid; i < a.tile + a.tile / 32; i += 4 * THREADS)
      *reinterpret_cast<u32x4*>(word + i) = u32x4{0, 0, 0, 0};
    for (int i = tid; i < a.nb; i += THREADS) {
      ids[i] = a.bias_ids[(int64_t)b * a.nb + i];
      add[i] = a.bias_vals[(int64_t)b * a.nb + i];
    }
    __syncthreads();
    // the tile's tokens of the history, eight loads at a time
    const int len = a.tokens ? min(max(a.lens ? a.lens[row] : a.L, 0), a.L) : 0;
    const int prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
    const int32_t* tok = a.tokens + (int64_t)row * a.tok_stride;
    auto history = [&](auto&& f) {
      constexpr int AHEAD = 8;
      for (int i0 = tid; i0 < len; i0 += AHEAD * THREADS) {
        int t[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) t[u] = i0 + u * THREADS < len ? tok[i0 + u * THREADS] : -1;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const uint32_t at = (uint32_t)t[u] - (uint32_t)v0;
          if (t[u] >= 0 && at >= low && at < high) f(i0 + u * THREADS, at);
        }
      }
    };
    history([&](int i, uint32_t at) {
      if (i < prompt) atomicOr(&word[at], kSaid);
      else atomicAdd(&word[at], 1u);
    });
    // an id's first entry takes the sum of all that name it, in their order
    constexpr int MINE = kRulesMaxBias / THREADS;
    float sum[MINE];
    uint32_t first[MINE];
#pragma unroll
    for (int u = 0; u < MINE; ++u) {
      const int i = tid + u * THREADS, id = i < a.nb ? ids[i] : -1;
      const uint32_t at = (uint32_t)id - (uint32_t)v0;
      sum[u] = 0.f;
      first[u] = id >= 0 && at >= low && at < high;
      if (first[u]) {
        for (int j = 0; j < a.nb; ++j)
          if (ids[j] == id) {
            if (j < i) first[u] = 0;
            sum[u] += add[j];
          }
        if (first[u]) atomicAdd(&word[at], (uint32_t)(i + 1) << kPlaceShift);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MINE; ++u)
      if (first[u]) add[tid + u * THREADS] = sum[u];
    __syncthreads();
    const float rho = a.repetition ? a.repetition[b] : 1.f, pres = a.presence ? a.presence[b] : 0.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    auto settle = [&](uint32_t at) {
      const uint32_t bit = 1u << (at & 31);
      if (atomicOr(&owned[at >> 5], bit) & bit) return;   // another's
      const uint32_t w = word[at], times = w & kTimes, place = (w >> kPlaceShift) & kPlace;
      float x = I::wide(in[(int)at + v0]);
      if ((w & kSaid) || times) x = x > 0.f ? x / rho : x * rho;
      if (times) x = (x - freq * (float)times) - pres;
      if (place) {
        const float y = add[place - 1];
        x = y == -__builtin_inff() ? y : x + y;           // a ban is one, whatever the logit
      }
      word[at] = I::result(x);
    };
    history([&](int, uint32_t at) { settle(at); });
#pragma unroll
    for (int u = 0; u < MINE; ++u)
      if (first[u]) settle((uint32_t)ids[tid + u * THREADS] - (uint32_t)v0);
    __syncthreads();
  }
  // ---- the dense pass
  const uint32_t* bits = mrow >= 0 ? a.mask + (int64_t)mrow * a.words : nullptr;
  auto one = [&](int v) {
    T x = in[v];
    if (marks) {
      const uint32_t w = word[v - v0];
      x = w ? I::take(w) : x;
    }
    if (bits && !((bits[v >> 5] >> (v & 31)) & 1)) x = I::LOWEST;
    out[v] = x;
  };
  constexpr int AHEAD = 4;
  for (int p0 = tid * VEC; p0 < a.tile; p0 += AHEAD * THREADS * VEC) {
    Vec x[AHEAD];
    uint32_t m[AHEAD];
    bool whole[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int p = p0 + u * THREADS * VEC, v = v0 + p;
      whole[u] = p < a.tile && v >= 0 && v + VEC <= a.V;
      m[u] = ~0u;
      if (whole[u]) {
        __builtin_memcpy(&x[u], in + v, sizeof(Vec));     // aligned to an element only
        if (bits) {
          const int at = v & 31;
          const uint32_t w0 = bits[v >> 5], w1 = at + VEC > 32 ? bits[(v >> 5) + 1] : 0u;
          m[u] = __builtin_amdgcn_alignbit(w1, w0, at);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int p = p0 + u * THREADS * VEC, v = v0 + p;
      if (whole[u]) {
        if (marks) {
#pragma unroll
          for (int h = 0; h < VEC / 4; ++h) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(word + p + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][4 * h + e] = w[e] ? I::take(w[e]) : x[u][4 * h + e];
          }
        }
        if (bits) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[u][e] = (m[u] >> e) & 1 ? x[u][e] : I::LOWEST;
        }
        *reinterpret_cast<Vec*>(out + v) = x[u];
      } else if (p < a.tile) {
        for (int e = max(v, lo); e < min(v + VEC, hi); ++e) one(e);
      }
    }
  }
}

template <bool F32, int THREADS>
void launch(const RulesArgs& a, hipStream_t s) {
  const size_t lds = a.tokens || a.nb > 0 ? (size_t)a.tile * 4 + a.tile / 8 + (size_t)a.nb * 8 : 0;
  rules_kernel<F32, THREADS><<<dim3((unsigned)(a.B * a.W * a.tiles)), THREADS, lds, s>>>(a);
}

}  // namespace

// Tiles of 1,024 to 16,384 tokens (a row's history is read once per tile, so few
// are better; but two workgroups per CU have to be there).
void rules_plan(RulesArgs& a) {
  const int64_t rows = (int64_t)a.B * a.W;
  a.tile = 16384;
  while (a.tile > 1024 && rows * ((a.V + a.tile - 1) / a.tile) < 512) a.tile /= 2;
  a.tiles = (a.V + 7 + a.tile - 1) / a.tile;              // the skew may take another
}

hipError_t launch_rules(const RulesArgs& a, hipStream_t s) {
  if (a.tile >= 8192) a.f32 ? launch<true, 512>(a, s) : launch<false, 512>(a, s);
  else a.f32 ? launch<true, 256>(a, s) : launch<false, 256>(a, s);
  return hipGetLastError();
}

}  // namespace gdn
