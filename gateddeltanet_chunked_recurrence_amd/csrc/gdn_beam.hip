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
// the candidates, the K best. Bound: reading the logits once from HBM. 512 rows
// of 100,003 bf16 logits (102 MB): 40 us, of which the parts 32.0 and the join 8.4
// (FP32, 205 MB: 44 to 50). 100,003 logits are 6.1 parts of eight vectors per lane, so a
// row's seventh part is a tenth full and costs what the others do. Reading alone takes 19 and the vector ALUs are busy for 16.5 (630 instructions per
// wave of 4,096 elements: five per element for maximum and sum, the rest for the
// choice); the two overlap little, as a workgroup waits for its loads first and
// three times for its slowest wave later. Elements kept packed (74 VGPRs instead of
// 100, more workgroups per CU) give the same time, workgroups that walk over
// parts and load the next one early 44 (153 VGPRs). 4 rows of 131,072: 12 us (5.9 and
// 6.5), two launches and their dependent loads. The 512 rows with all but 50 tokens
// masked: 46 us with -inf, 100 with the type's lowest value (636 when equal logits
// were taken one by one).
//
// The K largest of a part: a bound that at least K elements reach, from the
// 256 lane maxima: the K-th largest of one wave's 64 is one (the best of the four
// is taken), and the least of the four waves' ceil(K / 4)-th largest another,
// closer one where the large elements are spread out. Each is found by
// bisection over the upper bits (12 and 16) of an order-preserving integer, a
// ballot per bit; a bound too low by less than one step only lets a few more
// elements through.
// Elements that reach it (little more than K) go to a list in LDS, where each
// finds its rank by counting. Where a list overflows (a row's ragged end, or many
// equal logits), the bound is bisected over all elements of the part; among those
// equal to the K-th largest value, counts in token order give the places.
// Elements are distinct by (value, token), so the result does not depend on
// the order in which the list was filled.
//
// Sums: FP32 within a part (at most 64 terms per lane, then a tree), FP64
// across parts and for the totals. An exponential is 2^(x L - C) with L =
// fl(log2 e) and C = fl(m L), one FMA, rounded relative to the small difference;
// that C and L are rounded themselves is taken back in FP64 at the end (see
// log_sum); from |m| = 2^20 on the difference is taken first.
#include "gdn_device.h"
#include "gdn_launch.h"

namespace gdn {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / WAVE;
constexpr int kList = 128;                       // candidates that one wave keeps in LDS
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

// The largest t of BITS upper bits such that at least `want` of the keys are
// >= t << (32 - BITS) (keys: ord32 of values; one per lane, or N per lane).
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

constexpr float kLog2e = 1.4426950408889634f;    // L; L / log2(e) - 1 = kLDelta
constexpr double kLDelta = (double)kLog2e / 1.4426950408889634074 - 1.0;
constexpr float kBig = 0x1p20f;
// The exponent base of maximum m, and 2^(x L - base). The base is rounded, so
// the share of x = m itself is 2^(m L - fl(m L)): taken back at the end, but
// beyond 2^32 it overflows or vanishes. From 2^20 on (rows masked throughout
// with a large finite number, or +inf) the difference is taken first, and the
// base is m L as it is.
__device__ __forceinline__ float base_of(float m) { return fabsf(m) < kBig ? m * kLog2e : m; }
__device__ __forceinline__ float share_of(float x, float m, float base) {
  return fabsf(m) < kBig ? fexp2(fmaf(x, kLog2e, -base)) : fexp2((x - m) * kLog2e);
}
// The factor that brings a sum from maximum m to maximum M >= m: 2 to the
// difference of their bases, (m - M) L and what each base was rounded by. Not
// one fused multiply-add over m L and M L: that leaves out one of the roundings
// (6e-5 of a log-sum at logits near 1,000).
__device__ __forceinline__ float base_error(float m) {
  return fabsf(m) < kBig ? fmaf(m, kLog2e, -(m * kLog2e)) : 0.f;
}
__device__ __forceinline__ float rescale(float m, float M) {
#pragma clang fp contract(off)
  return fexp2((m - M) * kLog2e + (base_error(M) - base_error(m)));
}
// log sum exp(x) - M of a sum s of shares of maximum M: ln 2 log2(s) plus what
// the base was rounded by, fl(M L) / log2(e) - M, minus what the rounding of L adds, which
// is kLDelta times the mean of x: M, but for kLDelta times their distance (1e-7).
__device__ __forceinline__ double log_sum(double s, float M) {
  if (!(fabsf(M) < kBig)) return log(s);
  const double ln2 = 0.69314718055994530942;
  return log(s) + ((double)(M * kLog2e) * ln2 - (double)M) - kLDelta * (double)M;
}

// A double moved between lanes by a DPP pattern (see dpp_f).
template <int CTRL>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The set lanes of a mask below this one.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
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

// Workspace of one call: per (row, split) the maximum and the sum, and per
// request the K best of its W * splits parts as keys (0 where there are fewer), all
// parts' first, then all second and so on. The pitch of a rank is odd, so that
// the join's threads, which take every 256th, meet all ranks of all parts.
struct Ws {
  float2* ms;
  uint64_t* key;
  int pitch;
};
__host__ __device__ inline int64_t up16(int64_t x) { return (x + 15) & ~int64_t(15); }
__host__ __device__ inline Ws ws_of(const BeamArgs& a) {
  const int64_t parts = (int64_t)a.B * a.W * a.splits;
  char* p = static_cast<char*>(a.ws);
  Ws w;
  w.ms = reinterpret_cast<float2*>(p);
  w.key = reinterpret_cast<uint64_t*>(p + up16(parts * 8));
  w.pitch = (a.W * a.splits) | 1;
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
  __shared__ uint32_t sb[kWaves][2];
  __shared__ uint64_t list[kWaves][kList];
  __shared__ int counts[kWaves], tally[2][kWaves], equals[E][kWaves];
  const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits, tid = threadIdx.x;
  const int wave = tid >> 6, lane = tid & 63;
  if (a.finished && a.finished[row]) return;
  const char* base = static_cast<const char*>(a.logits) + (int64_t)row * a.row_stride * ES;
  // vectors on 16-byte boundaries: the row starts `off` elements into the first
  const int off = (int)((reinterpret_cast<uintptr_t>(base) & 15) / ES);
  const char* vec0 = base - (int64_t)off * ES;
  const int first = split * (E * kThreads) + tid;
  auto token0 = [&](int j) { return (first + j * kThreads) * VE - off; };   // of vector j's first element
  // The part's vectors, -inf outside the row. Only the row's first and last parts
  // have vectors that are not whole: code for ends in every load took 80 KB,
  // more than the instruction cache holds.
  auto load_part = [&](u32x4 (&raw)[E]) {
    const char* at = vec0 + (int64_t)first * 16;
    const int whole = split * (E * kThreads) * VE - off;
    if (whole >= 0 && whole + E * kThreads * VE <= a.V) {
#pragma unroll
      for (int j = 0; j < E; ++j) raw[j] = *reinterpret_cast<const u32x4*>(at + j * (kThreads * 16));
      return;
    }
    const uint32_t ninf = F32 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      raw[j] = u32x4{ninf, ninf, ninf, ninf};
      if (token0(j) >= 0 && token0(j) + VE <= a.V) raw[j] = *reinterpret_cast<const u32x4*>(at + j * (kThreads * 16));
    }
    // the row's two ends, element by element
    const int last = (a.V + off - 1) / VE;
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
      const int v = end == 0 ? 0 : last, lo = v * VE - off;
      const bool ragged = lo < 0 || lo + VE > a.V;
      if (!ragged || v < first || v >= first + E * kThreads || (v - first) % kThreads != 0) continue;
      u32x4 x{ninf, ninf, ninf, ninf};
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (lo + e >= 0 && lo + e < a.V) {
          if constexpr (F32) {
            x[e] = reinterpret_cast<const uint32_t*>(base)[lo + e];
          } else {
            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[lo + e];
            x[e / 2] = e & 1 ? (x[e / 2] & 0xFFFFu) | h << 16 : (x[e / 2] & 0xFFFF0000u) | h;
          }
        }
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (v == first + j * kThreads) raw[j] = x;
    }
  };
  // NaN counts as masked, +inf as the largest finite value
  auto plain = [](float v) { return v != v ? -kInf : fminf(v, kMaxF); };

  u32x4 raw[E];
  load_part(raw);
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
  // m: finite even where everything is masked, so that -inf - m is -inf
  float m = fmaxf(wave_max(top), -kMaxF), s = 0.f;
  const float base0 = m * kLog2e;
#pragma unroll
  for (int i = 0; i < E * VE; ++i) s += fexp2(fmaf(x[i], kLog2e, -base0));
  // Seldom: a NaN or +inf (both make the sum NaN), or a maximum beyond kBig
  if (__ballot(!(s <= kMaxF) || !(fabsf(m) < kBig)) != 0) {
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
    const float base = base_of(m);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < E * VE; ++i) s += share_of(x[i], m, base);
  }
  s = wave_total(s);
  const uint32_t tk[1] = {ord32(top)};
  const uint32_t b0 = kth_bound<12>(tk, min(a.K, WAVE)), b1 = kth_bound<16>(tk, (a.K + kWaves - 1) / kWaves);
  if (lane == 0) {
    sm[wave] = m;
    ss[wave] = s;
    sb[wave][0] = b0;
    sb[wave][1] = b1;
  }
  __syncthreads();
  uint32_t most = sb[0][0], least = sb[0][1];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    most = max(most, sb[i][0]);
    least = min(least, sb[i][1]);
  }
  // at least the smallest value above -inf
  const uint32_t bound = max(max(most, least), ord32(-kMaxF));
  float M = sm[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) M = fmaxf(M, sm[i]);
  const Ws w = ws_of(a);
  if (tid == 0) {
    float S = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) S += ss[i] * rescale(sm[i], M);
    w.ms[(int64_t)row * a.splits + split] = make_float2(M, S);
  }
  const int request = row / a.W, part = (row - request * a.W) * a.splits + split;
  uint64_t* out = w.key + (int64_t)request * a.K * w.pitch + part;
  auto put = [&](int rank, uint64_t key) { out[(int64_t)rank * w.pitch] = key; };
  // each wave's list: places by counting the lanes below, no atomics
  int mine_n = 0;
  if (__ballot(top >= unord32(bound)) != 0) {
    const float reach = unord32(bound);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (__ballot(vtop[j] >= reach) == 0) continue;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint64_t hit = __ballot(x[j * VE + e] >= reach);
        if (hit == 0) continue;
        const int at = mine_n + lanes_below(hit);
        if (x[j * VE + e] >= reach && at < kList) list[wave][at] = pick_key(x[j * VE + e], token0(j) + e);
        mine_n += __builtin_popcountll(hit);
      }
    }
  }
  int n = 0, longest = 0;
  auto count = [&]() {
    if (lane == 0) counts[wave] = mine_n;
    __syncthreads();
    n = longest = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      n += counts[i];
      longest = max(longest, counts[i]);
    }
  };
  count();
  int first_free = a.K;                          // places from here on hold no candidate of the lists
  if (longest > kList) {
    // Seldom: the bound is too low for the lists. Raise it by bisection, all
    // elements counted, until one list could hold those that reach it or it is
    // the K-th largest value itself. The elements are read again and stay
    // packed, so that this part takes no registers from the usual case.
    asm volatile("" ::: "memory");
    load_part(raw);
    auto repack = [&]() {                        // not unpacked once for all the passes
#pragma unroll
      for (int j = 0; j < E; ++j) asm volatile("" : "+v"(raw[j]));
    };
    auto value = [&](int j, int e) { return plain(elem<F32>(raw[j], e)); };
    uint32_t lo = bound, hi = ord32(M) + 1;      // n >= K elements reach lo, `above` < K reach hi
    uint32_t c = hi - 1;                         // the maximum first: a masked part is all equal
    int above = 0, turn = 0;
    while (n > kList && hi - lo > 1) {
      const float y = unord32(c);
      repack();
      // counts in lanes: with a ballot per element the scalar registers spill,
      // in the usual case too (512 rows of 100,003: 36 us instead of 33)
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) mine += value(j, e) >= y ? 1.f : 0.f;
      mine = wave_total(mine);
      if (lane == 0) tally[turn][wave] = (int)mine;
      __syncthreads();                           // the buffers alternate
      int have = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) have += tally[turn][i];
      turn ^= 1;
      if (have >= a.K) {
        lo = c;
        n = have;
      } else {
        hi = c;
        above = have;
      }
      c = lo + (hi - lo) / 2;
    }
    repack();
    if (n > kList) {
      // more elements of the K-th largest value than a list holds: the places
      // behind the larger ones go to the first of them by token
      const float y = unord32(lo);
      lo = hi;
      first_free = above;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float mine = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) mine += value(j, e) == y ? 1.f : 0.f;
        mine = wave_total(mine);
        if (lane == 0) equals[j][wave] = (int)mine;
      }
      __syncthreads();
      int from = above;                          // vectors of all waves in turn: the order of the tokens
#pragma unroll
      for (int j = 0; j < E; ++j)
#pragma unroll 1
        for (int o = 0; o < kWaves; ++o) {
          if (o == wave && from < a.K && equals[j][o] != 0) {
            int at = from;
#pragma unroll
            for (int e = 0; e < VE; ++e) at += lanes_below(__ballot(value(j, e) == y));
#pragma unroll
            for (int e = 0; e < VE; ++e)
              if (value(j, e) == y) {
                if (at < a.K) put(at, pick_key(y, token0(j) + e));
                ++at;
              }
          }
          from += equals[j][o];
        }
    }
    repack();
    const float reach = unord32(lo);
    mine_n = 0;
#pragma unroll
    for (int j = 0; j < E; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = value(j, e);
        const uint64_t hit = __ballot(y >= reach);
        if (hit == 0) continue;
        if (y >= reach) list[wave][mine_n + lanes_below(hit)] = pick_key(y, token0(j) + e);
        mine_n += __builtin_popcountll(hit);
      }
    count();
  }
  if (n <= WAVE) {
    // the usual case: one wave, an element per lane, ranks by broadcasts
    if (wave != 0) return;
    int seg = 0, at = lane;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i)
      if (seg == i && at >= counts[i]) {
        at -= counts[i];
        ++seg;
      }
    const uint64_t mine = lane < n ? list[seg][at] : 0;
    const int lo = (int)(uint32_t)mine, hi = (int)(uint32_t)(mine >> 32);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t other = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, j) << 32 |
                             (uint32_t)__builtin_amdgcn_readlane(lo, j);
      rank += other > mine;
    }
    if (lane < n) {
      if (rank < a.K) put(rank, mine);
    } else if (lane < first_free) {
      put(lane, 0);
    }
    return;
  }
  // n > 64 >= K: every place is written
  for (int i = lane; i < mine_n; i += WAVE) {
    const uint64_t mine = list[wave][i];
    int rank = 0;
    for (int o = 0; o < kWaves; ++o) {
      const int c = counts[o];
      for (int j = 0; j < c; ++j) rank += list[o][j] > mine;
    }
    if (rank < a.K) put(rank, mine);
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
constexpr int kHeld = 12, kParts = 1024;         // kParts: parts of a request kept in LDS
template <bool ONE>
__global__ void __launch_bounds__(kThreads) beam_join_kernel(BeamArgs a) {
  // total = (x - top) + shift, with the beam's largest logit and score - log
  // sum exp(x - top); shift -inf: no candidates
  __shared__ double topx[kBeamMaxW], shift[kBeamMaxW];
  __shared__ Cand list[kWaves][kList], best[kWaves];
  __shared__ __attribute__((aligned(16))) uint32_t tops[kThreads];
  __shared__ int counts[kWaves];
  __shared__ float2 pms[kParts];
  __shared__ float score_of[kBeamMaxW];
  __shared__ uint8_t done_of[kBeamMaxW];
  const int b = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const Ws w = ws_of(a);
  const int parts = a.W * a.splits, cand = a.K * w.pitch;
  const uint64_t* keys = w.key + (int64_t)b * cand;
  uint64_t held[ONE ? kHeld : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held[u] = tid + u * kThreads < cand ? keys[tid + u * kThreads] : 0;
  }
  // every part's maximum and sum, the scores and the flags, in one round trip
  const float2* ms = w.ms + (int64_t)b * parts;
  for (int i = tid; i < parts && i < kParts; i += kThreads) pms[i] = ms[i];
  if (tid < a.W) {
    score_of[tid] = a.scores[b * a.W + tid];
    done_of[tid] = a.finished ? a.finished[b * a.W + tid] : 0;
  }
  __syncthreads();
  auto part_of = [&](int i) { return i < kParts ? pms[i] : ms[i]; };
  // the log-sums: eight lanes per beam, all beams at once
  static_assert(8 * kBeamMaxW <= kThreads, "eight lanes per beam");
  if ((tid & ~63) < 8 * a.W) {
    const int beam = min(tid >> 3, a.W - 1), sub = tid & 7;
    float M = -kMaxF;
    for (int i = sub; i < a.splits; i += 8) M = fmaxf(M, part_of(beam * a.splits + i).x);
    M = fmaxf(M, dpp_f<0xB1>(M));
    M = fmaxf(M, dpp_f<0x4E>(M));
    M = fmaxf(M, dpp_f<0x141>(M));
    // each part's share relative to the largest: its FP32 error is that of
    // an exponential of a difference, as within a part
    double S = 0.0;
    for (int i = sub; i < a.splits; i += 8) {
      const float2 f = part_of(beam * a.splits + i);
      S += (double)(f.y * rescale(f.x, M));
    }
    S += dpp_d<0xB1>(S);
    S += dpp_d<0x4E>(S);
    S += dpp_d<0x141>(S);
    const double score = (double)score_of[beam], sh = done_of[beam] ? score : S > 0.0 ? score - log_sum(S, M) : -(double)kInf;
    if (sub == 0 && tid >> 3 < a.W) {
      topx[beam] = done_of[beam] ? 0.0 : (double)M;
      shift[beam] = sh > -(double)kInf ? sh : -(double)kInf;
    }
  }
  for (int i = tid; i < a.K; i += kThreads) {
    a.out_scores[(int64_t)b * a.K + i] = -kInf;
    a.parents[(int64_t)b * a.K + i] = -1;
    a.tokens[(int64_t)b * a.K + i] = -1;
  }
  __syncthreads();
  // i / d: exact for d > 1 and i d < 2^32, as i < kHeld kThreads
  const uint32_t by_pitch = 0xFFFFFFFFu / (uint32_t)w.pitch + 1, by_splits = 0xFFFFFFFFu / (uint32_t)a.splits + 1;
  auto over = [&](int i, int d, uint32_t magic) { return ONE && d > 1 ? (int)__umulhi((uint32_t)i, magic) : i / d; };
  auto get = [&](int i, uint64_t key, Cand& c) -> bool {
    const int rank = over(i, w.pitch, by_pitch), part = i - rank * w.pitch;
    if (part >= parts) return false;             // the pitch's last column
    c.beam = over(part, a.splits, by_splits);
    const double sh = shift[c.beam];
    if (!(sh > -(double)kInf)) return false;
    if (done_of[c.beam]) {
      c.total = sh;
      c.token = a.pad_token;
      return rank == 0 && part == c.beam * a.splits;
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
  int mine_n = 0;
  auto keep = [&](int i, uint64_t key, bool likely) {
    Cand c{};
    const bool hit = likely && get(i, key, c) && ord32((float)c.total) >= bound;
    const uint64_t lanes = __ballot(hit);
    const int at = mine_n + lanes_below(lanes);
    if (hit && at < kList) list[wave][at] = c;
    mine_n += __builtin_popcountll(lanes);
  };
  if constexpr (ONE) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (__ballot(ck[u] >= bound) != 0) keep(tid + u * kThreads, held[u], ck[u] >= bound);
  } else {
    for (int i0 = 0; i0 < cand; i0 += kThreads) keep(i0 + tid, i0 + tid < cand ? keys[i0 + tid] : 0, i0 + tid < cand);
  }
  if (lane == 0) counts[wave] = mine_n;
  __syncthreads();
  int longest = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) longest = max(longest, counts[i]);
  auto put = [&](int rank, const Cand& c) {
    a.out_scores[(int64_t)b * a.K + rank] = (float)c.total;
    a.parents[(int64_t)b * a.K + rank] = c.beam;
    a.tokens[(int64_t)b * a.K + rank] = c.token;
  };
  int n = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) n += counts[i];
  if (n <= WAVE) {
    // the usual case: one wave, a candidate per lane, ranks by broadcasts
    if (wave != 0) return;
    int seg = 0, at = lane;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i)
      if (seg == i && at >= counts[i]) {
        at -= counts[i];
        ++seg;
      }
    if (lane >= n) return;
    const Cand mine = list[seg][at];
    const uint64_t bits = __builtin_bit_cast(uint64_t, mine.total);
    const int lo = (int)(uint32_t)bits, hi = (int)(uint32_t)(bits >> 32);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      Cand c;
      c.total = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, j) << 32 |
                                               (uint32_t)__builtin_amdgcn_readlane(lo, j));
      c.beam = __builtin_amdgcn_readlane(mine.beam, j);
      c.token = __builtin_amdgcn_readlane(mine.token, j);
      rank += before(c, mine);
    }
    if (rank < a.K) put(rank, mine);
    return;
  }
  if (longest <= kList) {
    for (int i = lane; i < mine_n; i += WAVE) {
      const Cand mine = list[wave][i];
      int rank = 0;
      for (int o = 0; o < kWaves; ++o) {
        const int c = counts[o];
        for (int j = 0; j < c; ++j) rank += before(list[o][j], mine);
      }
      if (rank < a.K) put(rank, mine);
    }
    return;
  }
  // more equal totals than a list holds: the next candidate in order, K times
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
  // As much per workgroup as leaves 64 of them: 4 rows of 131,072 bf16 logits take
  // 12.6 us at one vector per lane (260 parts, whose candidates the second kernel
  // reads), 11.7 at four (68) or eight (36); 512 rows of 100,003 take 90, 41 and 42.
  int e = 8;
  while (e > 1 && rows * ((nv + e * kThreads - 1) / (e * kThreads)) < 64) e /= 2;
  a.vecs = e;
  a.splits = (int)((nv + e * kThreads - 1) / (e * kThreads));
}

int64_t beam_workspace_bytes(const BeamArgs& a) {
  const int64_t parts = (int64_t)a.B * a.W * a.splits;
  return up16(parts * 8) + (int64_t)a.B * a.K * ((a.W * a.splits) | 1) * 8;
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
  if (((int64_t)a.W * a.splits | 1) * a.K <= kHeld * kThreads) beam_join_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else beam_join_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gdn
