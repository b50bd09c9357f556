// Beam search's selection over beams and vocabulary: log-softmax of every
// beam's logits, added to the beam's score, and the K best (beam, token) pairs
// of each request, in one pass over the logits.
//
//   total[w, t] = score[w] + (x[w, t] - m_w) - log sum_t exp(x[w, t] - m_w)
//
// Within a beam the order of the totals is the order of the logits, so the
// first kernel needs no log-sum: one workgroup per (row, split of the
// vocabulary) keeps its part of the row in registers (1 to 8 16-byte loads per
// lane, all in flight at once) and leaves the part's maximum, its sum of
// exponentials and its K largest logits with their tokens. The second kernel,
// one workgroup per request, joins the parts: log-sums per beam, totals of
// the candidates, the K best. Bound: reading the logits once from HBM.
//
// The K largest of a part: the K-th largest of the workgroup's 256 lane maxima
// is a bound that at least K elements reach, found by bisection over the upper
// 16 bits of an order-preserving integer (16 rounds of four ballots; a bound too
// low by less than one such step only lets a few more elements through).
// Elements that reach it (little more than K) go to a list in LDS, where each
// finds its rank by counting. Only a list that overflows (many equal logits)
// takes the slow way, K passes that each find the next element in order.
// Elements are distinct by (value, token), so the result does not depend on
// the order in which the list was filled.
//
// Sums: FP32 within a part (at most 64 terms per lane, then a tree), FP64
// across parts and for the totals. An exponent is exp2((x - m) log2(e)) with
// the difference taken first, so its error is relative to x - m.
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / WAVE;
constexpr int kList = 512;                       // candidates of one part kept in LDS
constexpr float kInf = __builtin_huge_valf();
constexpr float kMaxF = 3.4028234663852886e38f;

// Order-preserving map of floats (no NaN) to unsigned integers and back; both
// zeros map to one integer (-0 + 0 = +0).
__device__ __forceinline__ uint32_t ord32(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Larger first, equal values by the lower token.
__device__ __forceinline__ uint64_t pick_key(float x, int token) {
  return (uint64_t)ord32(x) << 32 | (uint32_t)~token;
}

// The largest t of BITS upper bits such that at least `want` of the N keys per
// lane are >= t << (32 - BITS) (keys: ord32 of values).
template <int BITS, int N>
__device__ __forceinline__ uint32_t kth_bound(const uint32_t (&key)[N], int want) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t c = t | (1u << b);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __builtin_popcountll(__ballot(key[i] >= c));
    if (n >= want) t = c;
  }
  return t;
}

// The sum over the 64 lanes, in every lane: DPP within rows of 16, then the
// four row sums through scalar registers.
__device__ __forceinline__ float wave_total(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  x += dpp_f<0x140>(x);
  return (read_lane(x, 0) + read_lane(x, 16)) + (read_lane(x, 32) + read_lane(x, 48));
}

// Workspace of one call: per (row, split) the maximum and the sum, and the K
// best as keys (0 where there are fewer).
struct Ws {
  float2* ms;
  uint64_t* key;
};
__host__ __device__ inline int64_t up16(int64_t x) { return (x + 15) & ~int64_t(15); }
__host__ __device__ inline Ws ws_of(const BeamArgs& a) {
  const int64_t parts = (int64_t)a.B * a.W * a.splits;
  char* p = static_cast<char*>(a.ws);
  Ws w;
  w.ms = reinterpret_cast<float2*>(p);
  w.key = reinterpret_cast<uint64_t*>(p + up16(parts * 8));
  return w;
}

template <bool F32>
__device__ __forceinline__ float elem(const u32x4& v, int e) {
  const uint32_t u = F32 ? v[e] : e & 1 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16;
  return __builtin_bit_cast(float, u);
}

template <bool F32, int E>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(BeamArgs a) {
  constexpr int ES = F32 ? 4 : 2, VE = 16 / ES;
  __shared__ float sm[kWaves], ss[kWaves];
  __shared__ __attribute__((aligned(16))) uint32_t tops[kThreads];
  __shared__ uint64_t list[kList], best;
  __shared__ int count;
  const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits, tid = threadIdx.x;
  const int wave = tid >> 6, lane = tid & 63;
  if (a.finished && a.finished[row]) return;
  const char* base = static_cast<const char*>(a.logits) + (int64_t)row * a.row_stride * ES;
  // vectors on 16-byte boundaries: the row starts `off` elements into the first
  const int off = (int)((reinterpret_cast<uintptr_t>(base) & 15) / ES);
  const char* vec0 = base - (int64_t)off * ES;
  const int first = split * (E * kThreads) + tid;
  if (tid == 0) count = 0;
  auto token0 = [&](int j) { return (first + j * kThreads) * VE - off; };   // of vector j's first element
  auto load = [&](int j) {
    const uint32_t ninf = F32 ? 0xFF800000u : 0xFF80FF80u;
    const int lo = token0(j);
    u32x4 raw{ninf, ninf, ninf, ninf};
    if (lo >= 0 && lo + VE <= a.V) {
      raw = *reinterpret_cast<const u32x4*>(vec0 + (int64_t)(first + j * kThreads) * 16);
    } else if (lo + VE > 0 && lo < a.V) {
      // the row's ends: single elements
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (lo + e >= 0 && lo + e < a.V) {
          if constexpr (F32) {
            raw[e] = reinterpret_cast<const uint32_t*>(base)[lo + e];
          } else {
            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[lo + e];
            raw[e / 2] = e & 1 ? (raw[e / 2] & 0xFFFFu) | h << 16 : (raw[e / 2] & 0xFFFF0000u) | h;
          }
        }
    }
    return raw;
  };
  // NaN counts as masked, +inf as the largest finite value
  auto plain = [](float v) { return v != v ? -kInf : fminf(v, kMaxF); };

  u32x4 raw[E];
#pragma unroll
  for (int j = 0; j < E; ++j) raw[j] = load(j);
  float x[E * VE], top = -kInf, vtop[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    vtop[j] = -kInf;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      x[j * VE + e] = elem<F32>(raw[j], e);
      vtop[j] = fmaxf(vtop[j], x[j * VE + e]);
    }
    top = fmaxf(top, vtop[j]);
  }
  constexpr float kLog2e = 1.4426950408889634f;
  // m: finite even where everything is masked, so that -inf - m is -inf
  float m = fmaxf(wave_max(top), -kMaxF), s = 0.f;
#pragma unroll
  for (int i = 0; i < E * VE; ++i) s += fexp2((x[i] - m) * kLog2e);
  // A NaN, or +inf (whose difference with itself is NaN), shows in the sum
  if (__ballot(!(s <= kMaxF)) != 0) {
    top = -kInf;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      vtop[j] = -kInf;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        x[j * VE + e] = plain(x[j * VE + e]);
        vtop[j] = fmaxf(vtop[j], x[j * VE + e]);
      }
      top = fmaxf(top, vtop[j]);
    }
    m = fmaxf(wave_max(top), -kMaxF);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < E * VE; ++i) s += fexp2((x[i] - m) * kLog2e);
  }
  tops[tid] = ord32(top);
  s = wave_total(s);
  if (lane == 0) {
    sm[wave] = m;
    ss[wave] = s;
  }
  __syncthreads();
  const u32x4 t4 = *reinterpret_cast<const u32x4*>(tops + 4 * lane);
  const uint32_t tk[4] = {t4[0], t4[1], t4[2], t4[3]};
  const uint32_t bound = kth_bound<16>(tk, a.K);
  // at least the smallest value above -inf (its upper 16 bits alone would let -inf through)
  const float reach = fmaxf(unord32(max(bound, ord32(-kInf))), -kMaxF);
  const int64_t part = (int64_t)row * a.splits + split;
  const Ws w = ws_of(a);
  if (tid == 0) {
    float M = sm[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) M = fmaxf(M, sm[i]);
    float S = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) S += ss[i] * fexp2((sm[i] - M) * kLog2e);
    w.ms[part] = make_float2(M, S);
  }
  if (__ballot(top >= reach) != 0) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (__ballot(vtop[j] >= reach) == 0) continue;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (x[j * VE + e] >= reach) {
          const int p = atomicAdd(&count, 1);
          if (p < kList) list[p] = pick_key(x[j * VE + e], token0(j) + e);
        }
    }
  }
  __syncthreads();
  const int n = count;
  uint64_t* out = w.key + part * a.K;
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t mine = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += list[j] > mine;
      if (rank < a.K) out[rank] = mine;
    }
    for (int i = n + tid; i < a.K; i += kThreads) out[i] = 0;
    return;
  }
  // more ties than the list holds: the next element in order, K times, read
  // again (the registers of the elements are given up by now)
  uint64_t prev = ~0ull;
  for (int found = 0; found < a.K; ++found) {
    uint64_t mine = 0;
#pragma unroll 1
    for (int j = 0; j < E; ++j) {
      asm volatile("" ::: "memory");             // not hoisted out of the passes, which would take the registers
      const u32x4 v = load(j);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = plain(elem<F32>(v, e));
        const uint64_t k = pick_key(y, token0(j) + e);
        if (y >= reach && k < prev && k > mine) mine = k;
      }
    }
    __syncthreads();
    if (tid == 0) best = 0;
    __syncthreads();
    if (mine) atomicMax(reinterpret_cast<unsigned long long*>(&best), (unsigned long long)mine);
    __syncthreads();
    prev = best;
    if (tid == 0) out[found] = prev;
    if (prev == 0) prev = 1;                     // none left: the rest is 0 too
  }
}

// One candidate of the join: order by total, then beam, then token.
struct Cand {
  double total;
  int beam, token;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  if (a.total != b.total) return a.total > b.total;
  return a.beam != b.beam ? a.beam < b.beam : a.token < b.token;
}

// ONE: all candidates of a request fit kHeld per thread, and stay in registers.
constexpr int kHeld = 12;
template <bool ONE>
__global__ void __launch_bounds__(kThreads) beam_join_kernel(BeamArgs a) {
  constexpr float kLog2e = 1.4426950408889634f;
  // total = (x - top) + shift, with the beam's largest logit and score - log
  // sum exp(x - top); shift -inf: no candidates
  __shared__ double topx[kBeamMaxW], shift[kBeamMaxW];
  __shared__ Cand list[kList], best[kWaves];
  __shared__ __attribute__((aligned(16))) uint32_t tops[kThreads];
  __shared__ int count;
  const int b = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const Ws w = ws_of(a);
  const int per = a.splits * a.K, cand = a.W * per;
  const uint64_t* keys = w.key + (int64_t)b * cand;
  uint64_t held[ONE ? kHeld : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held[u] = tid + u * kThreads < cand ? keys[tid + u * kThreads] : 0;
  }
  if (tid == 0) count = 0;
  for (int beam = wave; beam < a.W; beam += kWaves) {
    const int row = b * a.W + beam;
    const float score = a.scores[row];
    double sh = -(double)kInf, tx = 0.0;
    if (a.finished && a.finished[row]) {
      sh = score;
    } else {
      const float2* ms = w.ms + (int64_t)row * a.splits;
      float M = -kMaxF;
      float2 f{-kMaxF, 0.f};
      if (lane < a.splits) f = ms[lane];
      for (int i = lane + WAVE; i < a.splits; i += WAVE) M = fmaxf(M, ms[i].x);
      M = wave_max(fmaxf(M, f.x));
      // each part's share relative to the largest: its FP32 error is that of
      // an exponential of a difference, as within a part
      double S = (double)(f.y * fexp2((f.x - M) * kLog2e));
      for (int i = lane + WAVE; i < a.splits; i += WAVE) S += (double)(ms[i].y * fexp2((ms[i].x - M) * kLog2e));
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) S += __shfl_xor(S, o, WAVE);
      tx = M;
      if (S > 0.0) sh = (double)score - log(S);
    }
    if (lane == 0) {
      topx[beam] = tx;
      shift[beam] = sh > -(double)kInf ? sh : -(double)kInf;
    }
  }
  for (int i = tid; i < a.K; i += kThreads) {
    a.out_scores[(int64_t)b * a.K + i] = -kInf;
    a.parents[(int64_t)b * a.K + i] = -1;
    a.tokens[(int64_t)b * a.K + i] = -1;
  }
  __syncthreads();
  auto get = [&](int i, uint64_t key, Cand& c) -> bool {
    c.beam = i / per;
    const double sh = shift[c.beam];
    if (!(sh > -(double)kInf)) return false;
    if (a.finished && a.finished[b * a.W + c.beam]) {
      c.total = sh;
      c.token = a.pad_token;
      return i == c.beam * per;
    }
    if (key == 0) return false;
    c.total = ((double)unord32((uint32_t)(key >> 32)) - topx[c.beam]) + sh;
    c.token = ~(uint32_t)key;
    return true;
  };
  // a bound that at least K candidates reach (all of them where there are fewer)
  uint32_t top = 0, ck[ONE ? kHeld : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      Cand c;
      ck[u] = 0;
      if (tid + u * kThreads < cand && get(tid + u * kThreads, held[u], c)) ck[u] = ord32((float)c.total);
      top = max(top, ck[u]);
    }
  } else {
    for (int i = tid; i < cand; i += kThreads) {
      Cand c;
      if (get(i, keys[i], c)) top = max(top, ord32((float)c.total));
    }
  }
  tops[tid] = top;
  __syncthreads();
  const u32x4 t4 = *reinterpret_cast<const u32x4*>(tops + 4 * lane);
  const uint32_t tk[4] = {t4[0], t4[1], t4[2], t4[3]};
  const uint32_t bound = max(kth_bound<20>(tk, a.K), 1u);
  auto keep = [&](int i, uint64_t key) {
    Cand c;
    if (get(i, key, c) && ord32((float)c.total) >= bound) {
      const int p = atomicAdd(&count, 1);
      if (p < kList) list[p] = c;
    }
  };
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (ck[u] >= bound) keep(tid + u * kThreads, held[u]);
  } else {
    for (int i = tid; i < cand; i += kThreads) keep(i, keys[i]);
  }
  __syncthreads();
  const int n = count;
  auto put = [&](int rank, const Cand& c) {
    a.out_scores[(int64_t)b * a.K + rank] = (float)c.total;
    a.parents[(int64_t)b * a.K + rank] = c.beam;
    a.tokens[(int64_t)b * a.K + rank] = c.token;
  };
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const Cand mine = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(list[j], mine);
      if (rank < a.K) put(rank, mine);
    }
    return;
  }
  // more equal totals than the list holds: the next candidate in order, K times
  Cand prev{(double)kInf, -1, -1};
  for (int found = 0; found < a.K; ++found) {
    Cand mine{-(double)kInf, 0, 0};
    for (int i = tid; i < cand; i += kThreads) {
      Cand c;
      if (get(i, keys[i], c) && before(prev, c) && before(c, mine)) mine = c;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const Cand other{__shfl_xor(mine.total, o, WAVE), __shfl_xor(mine.beam, o, WAVE),
                       __shfl_xor(mine.token, o, WAVE)};
      if (before(other, mine)) mine = other;
    }
    __syncthreads();                             // the last round's reads of `best` are done
    if (lane == 0) best[wave] = mine;
    __syncthreads();
    prev = best[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i)
      if (before(best[i], prev)) prev = best[i];
    if (!(prev.total > -(double)kInf)) break;
    if (tid == 0) put(found, prev);
  }
}

}  // namespace

void beam_plan(BeamArgs& a) {
  const int ve = a.f32 ? 4 : 8;
  const int64_t rows = (int64_t)a.B * a.W;
  // one more vector than V / ve where a row starts off a 16-byte boundary
  const int64_t nv = (a.V + ve - 2) / ve + 1;
  int e = 8;
  while (e > 1 && rows * ((nv + e * kThreads - 1) / (e * kThreads)) < 1024) e /= 2;
  a.vecs = e;
  a.splits = (int)((nv + e * kThreads - 1) / (e * kThreads));
}

int64_t beam_workspace_bytes(const BeamArgs& a) {
  const int64_t parts = (int64_t)a.B * a.W * a.splits;
  return up16(parts * 8) + parts * a.K * 8;
}

namespace {
template <bool F32>
void launch_parts(const BeamArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * a.W * a.splits));
  switch (a.vecs) {
    case 1: beam_part_kernel<F32, 1><<<grid, kThreads, 0, s>>>(a); break;
    case 2: beam_part_kernel<F32, 2><<<grid, kThreads, 0, s>>>(a); break;
    case 4: beam_part_kernel<F32, 4><<<grid, kThreads, 0, s>>>(a); break;
    default: beam_part_kernel<F32, 8><<<grid, kThreads, 0, s>>>(a); break;
  }
}
}  // namespace

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
  if (a.f32) launch_parts<true>(a, s);
  else launch_parts<false>(a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)a.B);
  if ((int64_t)a.W * a.splits * a.K <= kHeld * kThreads) beam_join_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else beam_join_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gdn
