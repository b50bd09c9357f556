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
// The K largest of a part: the K-th largest of a wave's 64 lane maxima is a
// bound that at least K elements reach, found by bisection over the upper 16
// bits of an order-preserving integer (16 ballots; a bound too low by less
// than one such step only lets a few more elements through). The largest of
// the four waves' bounds holds for the part; elements that reach it (about 2 K)
// go to a list in LDS, where each finds its rank by counting. Only a list that
// overflows (many equal logits) takes the slow way, K passes that each find
// the next element in order. Elements are distinct by (value, token), so the
// result does not depend on the order in which the list was filled.
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

// The largest t of `bits` upper bits such that at least `want` lanes have
// key >= t << (32 - bits) (key: ord32 of each lane's value).
template <int BITS>
__device__ __forceinline__ uint32_t kth_bound(uint32_t key, int want) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t c = t | (1u << b);
    if (__builtin_popcountll(__ballot(key >= c)) >= want) t = c;
  }
  return t;
}

// Workspace of one call: per (row, split) the maximum and the sum, the count
// and the K best as keys.
struct Ws {
  float* m;
  float* s;
  int32_t* cnt;
  uint64_t* key;
};
__host__ __device__ inline int64_t up16(int64_t x) { return (x + 15) & ~int64_t(15); }
__host__ __device__ inline Ws ws_of(const BeamArgs& a) {
  const int64_t parts = (int64_t)a.B * a.W * a.splits;
  char* p = static_cast<char*>(a.ws);
  Ws w;
  w.m = reinterpret_cast<float*>(p);
  w.s = reinterpret_cast<float*>(p + up16(parts * 4));
  w.cnt = reinterpret_cast<int32_t*>(p + 2 * up16(parts * 4));
  w.key = reinterpret_cast<uint64_t*>(p + 3 * up16(parts * 4));
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
  __shared__ uint32_t sb[kWaves];
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

  u32x4 raw[E];
  const uint32_t ninf = F32 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int lo = (first + j * kThreads) * VE - off;      // token of the vector's first element
    raw[j] = u32x4{ninf, ninf, ninf, ninf};
    if (lo >= 0 && lo + VE <= a.V) {
      raw[j] = *reinterpret_cast<const u32x4*>(vec0 + (int64_t)(first + j * kThreads) * 16);
    } else if (lo + VE > 0 && lo < a.V) {
      // the row's ends: single elements
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (lo + e >= 0 && lo + e < a.V) {
          if constexpr (F32) {
            raw[j][e] = reinterpret_cast<const uint32_t*>(base)[lo + e];
          } else {
            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[lo + e];
            raw[j][e / 2] = e & 1 ? (raw[j][e / 2] & 0xFFFFu) | h << 16 : (raw[j][e / 2] & 0xFFFF0000u) | h;
          }
        }
    }
  }
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
  // A NaN, or +inf (whose difference with itself is NaN), shows in the sum:
  // count NaN as masked, +inf as the largest finite value, and sum again.
  if (__ballot(!(s <= kMaxF)) != 0) {
    top = -kInf;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      vtop[j] = -kInf;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float& v = x[j * VE + e];
        v = v != v ? -kInf : fminf(v, kMaxF);
        vtop[j] = fmaxf(vtop[j], v);
      }
      top = fmaxf(top, vtop[j]);
    }
    m = fmaxf(wave_max(top), -kMaxF);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < E * VE; ++i) s += fexp2((x[i] - m) * kLog2e);
  }
  s = wave_sum(s);
  const uint32_t bound_w = kth_bound<16>(ord32(top), min(a.K, WAVE));
  if (lane == 0) {
    sm[wave] = m;
    ss[wave] = s;
    sb[wave] = bound_w;
  }
  __syncthreads();
  uint32_t bound = sb[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) bound = max(bound, sb[w]);
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
    w.m[part] = M;
    w.s[part] = S;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (__ballot(vtop[j] >= reach) == 0) continue;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (x[j * VE + e] >= reach) {
        const int p = atomicAdd(&count, 1);
        if (p < kList) list[p] = pick_key(x[j * VE + e], (first + j * kThreads) * VE - off + e);
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
    if (tid == 0) w.cnt[part] = min(n, a.K);
    return;
  }
  // more ties than the list holds: the next element in order, K times
  uint64_t prev = ~0ull;
  int found = 0;
  for (; found < a.K; ++found) {
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < E * VE; ++i) {
      const uint64_t k = pick_key(x[i], (first + (i / VE) * kThreads) * VE - off + i % VE);
      if (x[i] >= reach && k < prev && k > mine) mine = k;
    }
    __syncthreads();
    if (tid == 0) best = 0;
    __syncthreads();
    if (mine) atomicMax(reinterpret_cast<unsigned long long*>(&best), (unsigned long long)mine);
    __syncthreads();
    prev = best;
    if (prev == 0) break;
    if (tid == 0) out[found] = prev;
  }
  if (tid == 0) w.cnt[part] = found;
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

__global__ void __launch_bounds__(kThreads) beam_join_kernel(BeamArgs a) {
  // total = (x - top) + shift, with the beam's largest logit and score - log
  // sum exp(x - top); shift -inf: no candidates
  __shared__ double topx[kBeamMaxW], shift[kBeamMaxW];
  __shared__ double ctot[kList];
  __shared__ int cbeam[kList], ctok[kList];
  __shared__ uint32_t sb[kWaves];
  __shared__ Cand best[kWaves];
  __shared__ int count;
  const int b = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const Ws w = ws_of(a);
  const int per = a.splits * a.K, cand = a.W * per;
  if (tid == 0) count = 0;
  for (int beam = wave; beam < a.W; beam += kWaves) {
    const int row = b * a.W + beam;
    const float score = a.scores[row];
    double sh = -(double)kInf, tx = 0.0;
    if (a.finished && a.finished[row]) {
      sh = score;
    } else {
      float M = -kMaxF;
      for (int i = lane; i < a.splits; i += WAVE) M = fmaxf(M, w.m[(int64_t)row * a.splits + i]);
      M = wave_max(M);
      double S = 0.0;
      for (int i = lane; i < a.splits; i += WAVE) {
        const int64_t p = (int64_t)row * a.splits + i;
        S += (double)w.s[p] * exp((double)w.m[p] - (double)M);
      }
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
  auto get = [&](int i, Cand& c) -> bool {
    c.beam = i / per;
    const int r = i - c.beam * per, split = r / a.K, k = r - split * a.K, row = b * a.W + c.beam;
    const double sh = shift[c.beam];
    if (!(sh > -(double)kInf)) return false;
    if (a.finished && a.finished[row]) {
      c.total = sh;
      c.token = a.pad_token;
      return r == 0;
    }
    const int64_t part = (int64_t)row * a.splits + split;
    if (k >= w.cnt[part]) return false;
    const uint64_t key = w.key[part * a.K + k];
    c.total = ((double)unord32((uint32_t)(key >> 32)) - topx[c.beam]) + sh;
    c.token = ~(uint32_t)key;
    return true;
  };
  // a bound that at least K candidates reach (all of them where a wave has fewer)
  uint32_t top = 0;
  for (int i = tid; i < cand; i += kThreads) {
    Cand c;
    if (get(i, c)) top = max(top, ord32((float)c.total));
  }
  const uint32_t bw = kth_bound<20>(top, min(a.K, WAVE));
  if (lane == 0) sb[wave] = bw;
  __syncthreads();
  uint32_t bound = sb[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) bound = max(bound, sb[i]);
  for (int i = tid; i < cand; i += kThreads) {
    Cand c;
    if (get(i, c) && ord32((float)c.total) >= bound) {
      const int p = atomicAdd(&count, 1);
      if (p < kList) {
        ctot[p] = c.total;
        cbeam[p] = c.beam;
        ctok[p] = c.token;
      }
    }
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
      const Cand mine{ctot[i], cbeam[i], ctok[i]};
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(Cand{ctot[j], cbeam[j], ctok[j]}, mine);
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
      if (get(i, c) && before(prev, c) && before(c, mine)) mine = c;
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
  return 3 * up16(parts * 4) + parts * a.K * 8;
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
  beam_join_kernel<<<dim3((unsigned)a.B), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gdn
