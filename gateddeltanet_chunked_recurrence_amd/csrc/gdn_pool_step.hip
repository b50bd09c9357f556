// Recurrent step of the gated delta rule on the pages of a state pool: the
// serving form of the decode steps in gdn_decode.hip, with the states really
// held in one byte per element. Per sequence n, value head h and token t, with
// S = d c the state of slot slots[n] (c codes, d one scale per block_v value
// rows):
//   alpha = exp(g_t);  u = beta_t (v_t - alpha S^T k_t)
//   S' = alpha S + k_t u^T;  o_before = scale S'^T q_t
//   S <- QDQ(S')  (amax of the tile -> d', c' = RNE(S' fl(1/d')))
//   o_after = scale S^T q_t
// and the last S goes to slot slots_out[n] (or back). As executed, with
// a = alpha d:  p = c^T k, w = c^T q;  u = beta (v - a p);
//   o_before = scale (a w + (k . q) u);  S' = a c + k u^T
// so both products read the codes as they are and the output needs no pass
// over S'.
//
// Bound: a token moves Dk Dv bytes in and out per head for 6 Dk Dv FLOP, so
// at many sequences this is a copy (bound by HBM). The page is value-major
// ([Dv, Dk], Dk contiguous), so a scale tile is one contiguous block and the
// sums over Dk run along a row.
//
// Pages of codes: the products on the matrix cores, as an integer or E4M3 code
// is exact in bf16. With 16 state rows as the columns of B (32 keys deep),
// v_mfma_f32_16x16x32_bf16 forms
//   - p and w: A has k and q as rows, repeated every four rows, so that each
//     lane finds both sums of its own state row in its accumulator;
//   - S' in units of a, c + k (u / a): A picks 16 of the 32 keys (a permuted
//     identity), then adds k times u / a, both as sums of bf16 parts (three parts are
//     exact for 24 bits). The keys of a 16x16 result tile are those of one dword
//     of codes per lane, so its four values are quantized into that dword.
// The vector ALUs keep half an instruction per element to decode, two to
// quantize and half for the amax. With S' and the sums on them (FP32 FMAs)
// they took 6.9 instructions per element and, at 1,024 sequences of 32 heads
// (Dv 256, 1.8 GB in and out), bound the step: 460 us.
// Pages of FP32 states move four times the bytes; their sums stay on the
// vector ALUs.
//
// Measured, E4M3 with bf16 inputs, read from one page and written to another: 1,024
// sequences of 32 heads (128 x 256) 436 us; a plain copy of the same pages
// at random places takes 360 to 400, this loop without its stores 303, with nothing but
// loads and stores 445. Counters: 1,096 MB read and 1,094 written, 5.0 TB/s, where
// the distinct parents and the inputs are 713 MB: each child of a parent reads it
// from beyond L2 again. 192 sequences of 16 heads (128 x 128) 25.6 us, 3.2 TB/s:
// about two tiles per wave, so loads and stores of the ends stand alone.
// One sequence 5.5 us: a launch and one trip to HBM after the slots. Dropped: two
// tiles ahead at two waves per SIMD 508 us (it spills at three), tiles unquantized
// twice instead of held at four waves 457, non-temporal stores 474, one wave per tile
// without the loop 530 to 555. What is kept fills the 168 registers of three waves
// too: with 128 keys and two row tiles most E4M3 variants keep up to 60 bytes a lane in
// scratch (the 192 sequences 28, 5 MB written; the 1,024 none). Inputs in FP32 take 27 to 30 us where bf16 takes 25: the parts of k and q are
// made once per head, in LDS (53 us when every tile split them again). INT8 at 192
// sequences: 35 us. Two things bind it: the conversions to bf16 by way of floats
// (a shift, an extraction and a conversion per element), and that the compiler
// carries the next tile's codes as bytes, whose shifts stand right behind their
// loads and wait for them before this tile's products.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_pool.h"

namespace gdn {

namespace {

// The sum over the eight neighbouring lanes that hold one row.
__device__ __forceinline__ float sum_row(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  return x;
}

// Four consecutive bf16 or FP32 elements.
template <bool F32>
__device__ __forceinline__ f32x4 load4(const void* p) {
  if constexpr (F32) return *reinterpret_cast<const f32x4*>(p);
  const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
  return f32x4{from_bf16(v[0]), from_bf16(v[1]), from_bf16(v[2]), from_bf16(v[3])};
}
template <bool F32>
__device__ __forceinline__ void store4(void* p, f32x4 x) {
  if constexpr (F32) *reinterpret_cast<f32x4*>(p) = x;
  else *reinterpret_cast<bf16x4*>(p) = bf16x4{to_bf16(x[0]), to_bf16(x[1]), to_bf16(x[2]), to_bf16(x[3])};
}

// What every wave of a call does first: its sequence, head and rows, whether
// it may run, and where its state goes.
struct StepUnit {
  int n, h, row;              // sequence, value head, first row of the wave
  int T, slot, to;
  bool idle;                  // no sequence, or nothing to do
};
__device__ __forceinline__ StepUnit step_unit(const PoolStepArgs& a, int unit, int rpw) {
  const int per = a.pool.Dv / rpw, ph = per * a.pool.Hv;
  StepUnit w;
  w.n = unit / ph;
  const int rem = unit - w.n * ph;
  w.h = rem / per;
  w.row = (rem - w.h * per) * rpw;
  w.T = a.lens ? min(max(a.lens[w.n], 0), a.T) : a.T;
  w.slot = a.slots[w.n];
  w.to = a.slots_out ? a.slots_out[w.n] : w.slot;
  w.idle = w.slot == -1 || (w.T == 0 && w.to == w.slot);
  return w;
}
__device__ __forceinline__ bool step_in_ok(const PoolStepArgs& a, const StepUnit& w) {
  return w.slot >= 0 && w.slot < a.pool.slots;
}
__device__ __forceinline__ bool step_refused(const PoolStepArgs& a, const StepUnit& w) {
  if (!step_in_ok(a, w) || w.to < -1 || w.to >= a.pool.slots) return true;
  return w.to >= 0 && pool_claimed<false>(a.pool, a.slots, a.slots_out ? a.slots_out : a.slots, a.B, w.n, w.to, a.T, a.lens);
}

// ------------------------------------------------------------ pages of codes
// Part m of a float: three bf16 values whose sum is the float (to 2^-24), then 0.
__device__ __forceinline__ bf16 split_part(float x, int m) {
  const bf16 h = to_bf16(x);
  const float r1 = x - from_bf16(h);
  const bf16 mid = to_bf16(r1);
  const bf16 low = to_bf16(r1 - from_bf16(mid));
  return m == 0 ? h : m == 1 ? mid : m == 2 ? low : to_bf16(0.f);
}

// A wave's LDS: k and q (FP32: also their bf16 parts), zeros, and k laid out for the update:
// for result tile x = 4 s + c and row m, the A row of key 64 s + 16 (m >> 2) + 4 c
// + (m & 3): bf16 (k, k, k, 0...), FP32 the parts (k1, k1, k1, k2, k2, k3, 0, 0).
template <int DK, bool F32>
struct HeadLds {
  static constexpr int ES = F32 ? 4 : 2, HB = 2 * DK * ES, LB = HB / WAVE;
  static constexpr int ZERO = HB, PARTS = HB + DK * ES, ROWS = PARTS + (F32 ? 6 * DK * 2 : 0), BYTES = ROWS + 16 * DK;
};

// Writes a head's LDS from the lanes' shares of k and q (LB bytes each).
template <int DK, bool F32>
__device__ __forceinline__ void head_to_lds(char* hb, const uint32_t* share) {
  using H = HeadLds<DK, F32>;
  const int lane = __lane_id();
  if constexpr (H::LB == 16) *reinterpret_cast<u32x4*>(hb + lane * 16) = u32x4{share[0], share[1], share[2], share[3]};
  else if constexpr (H::LB == 8) *reinterpret_cast<uint2*>(hb + lane * 8) = make_uint2(share[0], share[1]);
  else *reinterpret_cast<uint32_t*>(hb + lane * 4) = share[0];
  if constexpr (F32) {
    // a lane holds DK / 32 keys of k (lanes below 32) or q: their three parts, [which][part][key]
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {
      const float x = __builtin_bit_cast(float, share[i]);
      bf16* p = reinterpret_cast<bf16*>(hb + H::PARTS) + (lane >> 5) * 3 * DK + (lane & 31) * (DK / 32) + i;
#pragma unroll
      for (int m = 0; m < 3; ++m) p[m * DK] = split_part(x, m);
    }
  }
  // a lane below 32 holds DK / 32 keys of k
  if (lane < 32) {
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {
      const int key = lane * (DK / 32) + i, s = key >> 6, y = key & 63;
      const int x = 4 * s + ((y >> 2) & 3), m = 4 * (y >> 4) + (y & 3);
      bf16x8 row{};
      if constexpr (F32) {
        const float k = __builtin_bit_cast(float, share[i]);
        const bf16 k1 = split_part(k, 0), k2 = split_part(k, 1);
        row[0] = row[1] = row[2] = k1;
        row[3] = row[4] = k2;
        row[5] = split_part(k, 2);
      } else {
        const uint32_t w = share[i / 2];
        const bf16 k = __builtin_bit_cast(bf16, static_cast<uint16_t>(i & 1 ? w >> 16 : w & 0xFFFFu));
        row[0] = row[1] = row[2] = k;
      }
      *reinterpret_cast<bf16x8*>(hb + H::ROWS + (16 * x + m) * 16) = row;
    }
  }
  // the wave's own buffer: LDS operations of a wave stay in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
template <int DK, bool F32>
__device__ __forceinline__ void head_zeros(char* hb) {
  using H = HeadLds<DK, F32>;
  for (int i = 4 * __lane_id(); i < DK * H::ES; i += 4 * WAVE) *reinterpret_cast<uint32_t*>(hb + H::ZERO + i) = 0;
}

// The lane's row of A for the row sums over keys 64 s + 16 g + 8 i .. + 7. bf16
// inputs: k (r % 4 == 0), q (1) or zeros. FP32: part r % 4 of k (which = 0) or q (1).
template <int DK, bool F32>
__device__ __forceinline__ bf16x8 sum_row_of(const char* hb, int r, int g, int s, int i, int which) {
  using H = HeadLds<DK, F32>;
  int row;
  if constexpr (F32) row = (r & 3) == 3 ? H::ZERO : H::PARTS + (which * 3 + (r & 3)) * DK * 2;
  else row = (r & 2) ? H::ZERO : (r & 1) * (H::HB / 2);
  return *reinterpret_cast<const bf16x8*>(hb + row + (64 * s + 16 * g + 8 * i) * 2);
}

// k . q, in every lane.
template <int DK, bool F32>
__device__ __forceinline__ float head_kq(const char* hb, int r, int g) {
  using H = HeadLds<DK, F32>;
  if constexpr (F32) {
    float kq = 0.f;
    const float *k = reinterpret_cast<const float*>(hb), *q = reinterpret_cast<const float*>(hb + H::HB / 2);
#pragma unroll
    for (int i = 0; i < DK / WAVE; ++i) kq = fmaf(k[WAVE * i + 16 * g + r], q[WAVE * i + 16 * g + r], kq);
    return wave_sum(kq);
  } else {
    f32x4 acc = zero4();
#pragma unroll
    for (int s = 0; s < DK / 64; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc = mfma(sum_row_of<DK, F32>(hb, r, g, s, i, 0),
                   *reinterpret_cast<const bf16x8*>(hb + (64 * s + 16 * g + 8 * i) * 2), acc);
    return acc[1];
  }
}

// One token on the rows of a wave: 16 NT rows of one scale tile, lane (r = lane
// & 15, g = lane >> 4) holding, of each 16-row tile, row r and the keys 64 s + 16 g
// .. + 15 (one 16-byte piece per s). In: codes `raw`, a = exp(g) d. Out: the new
// codes in `raw`, the tile's scale d and the outputs o. `join` makes the
// tile's amax of a wave's; `decoded` is called when the codes are in bf16.
template <int DK, int FMT, bool F32, int NT, typename Decoded, typename Join>
__device__ __forceinline__ void step_tile(const PoolRef& P, const char* hb, u32x4 (&raw)[NT][DK / 64],
                                          float alpha, float beta, float kq, float scale,
                                          const float (&v)[NT], float (&o)[NT], float& d, bool after,
                                          Decoded decoded, Join join) {
  using H = HeadLds<DK, F32>;
  constexpr int NS = DK / 64;
  const int lane = __lane_id(), r = lane & 15, g = lane >> 4;
  // the codes as B operands
  bf16x8 b[NT][NS][2];
  auto decode = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          b[j][s][i] = codes8_bf16<FMT>(raw[j][s][2 * i], raw[j][s][2 * i + 1]);
          // integers go through floats: eight at a time, not all at once
          if constexpr (FMT == 2) __builtin_amdgcn_sched_barrier(0);
        }
  };
  float p[NT], q[NT];
  auto row_sums = [&]() {
    f32x4 ak[NT], aq[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) ak[j] = aq[j] = zero4();
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 rk = sum_row_of<DK, F32>(hb, r, g, s, i, 0);
        bf16x8 rq = rk;
        if constexpr (F32) rq = sum_row_of<DK, F32>(hb, r, g, s, i, 1);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          ak[j] = mfma(rk, b[j][s][i], ak[j]);
          if constexpr (F32) aq[j] = mfma(rq, b[j][s][i], aq[j]);
        }
      }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      p[j] = F32 ? ak[j][0] + (ak[j][1] + ak[j][2]) : ak[j][0];
      q[j] = F32 ? aq[j][0] + (aq[j][1] + aq[j][2]) : ak[j][1];
    }
  };
  decode();
  decoded();
  row_sums();
  // The update in units of a, or of 2^-64 where a is smaller (a state forgotten
  // within a token, or the zero page with its scale 2^-126), so that u / unit
  // cannot overflow for |u| < 2^63; the codes then count a / unit < 1 each,
  // rounded to bf16: that rounds values below 2^-55 only. From a = 2 on the codes
  // count a's power of two (exact in bf16) and the unit is the rest, so that unit / d
  // below stays finite down to the smallest d, 2^-126 (a tile that becomes zero).
  const uint32_t abits = __builtin_bit_cast(uint32_t, alpha);
  const float unit = fmaxf(alpha >= 2.f ? __builtin_bit_cast(float, (abits & 0x007FFFFFu) | 0x3F800000u) : alpha, 0x1p-64f);
  const float ru = 1.0f / unit;
  const uint32_t half = alpha >= 2.f         ? (abits >> 16) & 0x7F80u
                        : alpha >= 0x1p-64f ? 0x3F80u
                                             : __builtin_bit_cast(uint16_t, to_bf16(alpha * ru));
  const uint32_t one = half | half << 16;
  // A of tiles with even and odd c: row m picks, for lanes g == m >> 2, element 4 (c & 1) + (m & 3)
  bf16x8 pick[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    u32x4 w{0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[2 * c + h] = (g == r >> 2 && (r & 2) == 2 * h) ? one & (r & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
    pick[c] = __builtin_bit_cast(bf16x8, w);
  }
  const char* krow = hb + (g == 0 ? H::ROWS + 16 * r : (int)H::ZERO);
  f32x4 S[NT][4 * NS];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const float u = beta * fmaf(-alpha, p[j], v[j]);
    o[j] = scale * fmaf(kq, u, alpha * q[j]);
    const float uu = u * ru;
    bf16x8 ub{};
    const bf16 u1 = to_bf16(uu);
    const float r1 = uu - from_bf16(u1);
    const bf16 u2 = to_bf16(r1), u3 = to_bf16(r1 - from_bf16(u2));
    ub[0] = u1;
    ub[1] = u2;
    ub[2] = u3;
    if constexpr (F32) {
      ub[3] = u1;
      ub[4] = u2;
      ub[5] = u1;
    }
#pragma unroll
    for (int x = 0; x < 4 * NS; ++x) {
      const bf16x8 kr = *reinterpret_cast<const bf16x8*>(krow + (g == 0 ? 256 * x : 0));
      f32x4 acc = mfma(pick[x & 1], b[j][x >> 2][(x >> 1) & 1], zero4());
      acc = mfma(kr, ub, acc);
      S[j][x] = acc;
      m = larger<FMT>(larger<FMT>(m, acc[0]), acc[1]);
      m = larger<FMT>(larger<FMT>(m, acc[2]), acc[3]);
    }
  }
  d = pool_scale<FMT>(P, join(wave_largest<FMT>(m)) * unit);
  const float rd = (1.0f / d) * unit;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int x = 0; x < 4 * NS; ++x) {
      const float y[4] = {S[j][x][0], S[j][x][1], S[j][x][2], S[j][x][3]};
      raw[j][x >> 2][x & 3] = quant_word<FMT>(y, rd);
      if constexpr (FMT == 2) __builtin_amdgcn_sched_barrier(0);
    }
  if (after) {
    decode();
    row_sums();
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j] = scale * (d * q[j]);
  }
}

// A lane's share of k and q of one token and head (LB bytes of [k | q]).
template <int DK, bool F32>
__device__ __forceinline__ void load_share(const PoolStepArgs& a, int64_t token, int hk, uint32_t* share) {
  using H = HeadLds<DK, F32>;
  const int at = __lane_id() * H::LB, off = at % (H::HB / 2);
  const char* kp = static_cast<const char*>(a.k) + (token * a.ks + hk * DK) * H::ES;
  const char* qp = static_cast<const char*>(a.q) + (token * a.qs + hk * DK) * H::ES;
  const char* p = (at < H::HB / 2 ? kp : qp) + off;
  if constexpr (H::LB == 16) {
    const u32x4 y = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) share[i] = y[i];
  } else if constexpr (H::LB == 8) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    share[0] = y.x;
    share[1] = y.y;
  } else {
    share[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Several tokens, or lengths: one wave per 16 NT rows, the state stays in
// registers as codes between tokens.
template <int DK, int FMT, bool F32, int NT, int WPT>
__global__ void __launch_bounds__((WPT == 1 ? 4 : WPT) * WAVE)
pool_step_many_kernel(PoolStepArgs a, int waves) {
  using H = HeadLds<DK, F32>;
  constexpr int NW = WPT == 1 ? 4 : WPT, NS = DK / 64, ES = H::ES, RPW = 16 * NT;
  __shared__ __attribute__((aligned(16))) char hbuf[NW][H::BYTES];
  __shared__ float xm[2][NW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const int wunit = blockIdx.x * NW + wave;
  if (wunit >= waves) return;                   // only where the waves are independent
  const PoolRef& P = a.pool;
  const int r = lane & 15, g = lane >> 4;
  const StepUnit w = step_unit(a, wunit, RPW);
  if (w.idle) {                                 // uniform over a tile's waves
    if (w.slot != -1 && !step_in_ok(a, w) && lane == 0) pool_error(P);
    return;
  }
  const int Hv = P.Hv, Dv = P.Dv, hk = w.h / (Hv / a.Hqk);
  const int64_t tok0 = (int64_t)w.n * a.T, o_tok = (int64_t)Hv * Dv;
  u32x4 raw[NT][NS];
  const int64_t head = (int64_t)w.h * Dv * DK + (int64_t)(w.row + r) * DK + 16 * g;
  const int tile = w.h * (Dv / P.block_v) + w.row / P.block_v;
  float d = 1.f;
  if (step_in_ok(a, w)) {
    const uint8_t* src = P.data + (a.layer_page + w.slot) * P.page + head;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int s = 0; s < NS; ++s) raw[j][s] = *reinterpret_cast<const u32x4*>(src + 16 * j * DK + 64 * s);
    d = P.scales[(a.layer_page + w.slot) * P.tiles + tile];
  }
  uint32_t share[H::LB / 4];
  float v[NT], o[NT], gate = 0.f, beta = 0.f;
  auto load_token = [&](int t) {
    load_share<DK, F32>(a, tok0 + t, hk, share);
    const char* vp = static_cast<const char*>(a.v) + ((tok0 + t) * a.vs + (int64_t)w.h * Dv + w.row + r) * ES;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      v[j] = F32 ? reinterpret_cast<const float*>(vp)[16 * j] : from_bf16(reinterpret_cast<const bf16*>(vp)[16 * j]);
    gate = a.g[(tok0 + t) * Hv + w.h];
    beta = a.beta[(tok0 + t) * Hv + w.h];
  };
  if (w.T > 0) load_token(0);
  char* op = static_cast<char*>(a.o) + (tok0 * o_tok + (int64_t)w.h * Dv + w.row + r) * ES;
  auto put_o = [&](int t) {
    if (g == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (F32) reinterpret_cast<float*>(op + t * o_tok * ES)[16 * j] = o[j];
        else reinterpret_cast<bf16*>(op + t * o_tok * ES)[16 * j] = to_bf16(o[j]);
      }
    }
  };
  if (step_refused(a, w)) {
    // the outputs say so, the pages stay as they are
    if (lane == 0) pool_error(P);
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j] = __builtin_nanf("");
    for (int t = 0; t < w.T; ++t) put_o(t);
    return;
  }
  char* hb = hbuf[wave];
  head_zeros<DK, F32>(hb);
  for (int t = 0; t < w.T; ++t) {
    head_to_lds<DK, F32>(hb, share);
    const float kq = head_kq<DK, F32>(hb, r, g), alpha = expf(gate) * d, bt = beta;
    float vt[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) vt[j] = v[j];
    step_tile<DK, FMT, F32, NT>(
        P, hb, raw, alpha, bt, kq, a.scale, vt, o, d, a.readout != 0,
        [&]() {
          if (t + 1 < w.T) load_token(t + 1);
        },
        [&](float m) {
          if constexpr (WPT > 1) {
            // the buffers alternate, so one barrier per token is enough: a wave
            // that writes xm[t & 1] again has passed the barrier of token t + 1,
            // which every wave reaches after reading xm[t & 1]
            if (lane == 0) xm[t & 1][wave] = m;
            lds_barrier();
#pragma unroll
            for (int i = 0; i < NW; ++i) m = larger<FMT>(m, xm[t & 1][i]);
          }
          return m;
        });
    put_o(t);
  }
  if (w.to < 0) return;                         // the state is not kept
  uint8_t* dst = P.data + (a.layer_page + w.to) * P.page + head;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int s = 0; s < NS; ++s) *reinterpret_cast<u32x4*>(dst + 16 * j * DK + 64 * s) = raw[j][s];
  if (lane == 0 && w.row % P.block_v == 0) P.scales[(a.layer_page + w.to) * P.tiles + tile] = d;
}

// One token per sequence, the usual call: persistent groups of waves, WPT
// waves to a scale tile, that run over their elements (sequence, head, `span`
// tiles of it) and load the next tile's codes and the next head's inputs
// before they compute the current ones. A wave that is launched per tile
// waits for its slot, then for its codes, with nothing else in flight.
template <int DK, int FMT, bool F32, int NT, int WPT, bool AFTER>
__global__ void __launch_bounds__((WPT == 1 ? 4 : WPT) * WAVE, 3)
pool_step_one_kernel(PoolStepArgs a, int lspan, int lparts, int elems, int chunk) {
  using H = HeadLds<DK, F32>;
  constexpr int NW = WPT == 1 ? 4 : WPT, NS = DK / 64, ES = H::ES, RPW = 16 * NT, BV = WPT * RPW;
  __shared__ __attribute__((aligned(16))) char hbuf[NW][H::BYTES];
  __shared__ float xm[2][NW];
  const PoolRef& P = a.pool;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const int sub = wave % WPT, r = lane & 15, g = lane >> 4;
  const int Hv = P.Hv, hp = Hv << lparts, span = 1 << lspan;
  const int tph = 1 << (lspan + lparts);               // tiles per head
  int e = (blockIdx.x * (NW / WPT) + wave / WPT) * chunk;
  const int end = min(e + chunk, elems);
  if (e >= end) return;
  char* hb = hbuf[wave];
  head_zeros<DK, F32>(hb);
  const int row_in = sub * RPW + r, loff = row_in * DK + 16 * g;
  // an element's place: first tile, inputs, page read (uniform)
  struct Place {
    const uint8_t* src;
    const float* scale;
    const char* v;
    int n, h, tile, slot, to;
  };
  int seq, ph;
  auto place = [&](int slot, int to) {
    Place x;
    x.n = seq;
    x.h = ph >> lparts;
    x.tile = (ph & ((1 << lparts) - 1)) << lspan;
    x.slot = slot;
    x.to = to;
    const int64_t page = a.layer_page + slot, tile = x.h * tph + x.tile;
    x.src = P.data + page * P.page + tile * (BV * DK);
    x.scale = P.scales + page * P.tiles + tile;
    x.v = static_cast<const char*>(a.v) + ((int64_t)seq * a.vs + tile * BV) * ES;
    return x;
  };
  uint32_t share[H::LB / 4];
  float gn = 0.f, bn = 0.f;
  auto load_head = [&](const Place& x) {
    load_share<DK, F32>(a, x.n, x.h / (Hv / a.Hqk), share);
    gn = a.g[(int64_t)x.n * Hv + x.h];
    bn = a.beta[(int64_t)x.n * Hv + x.h];
  };
  u32x4 rawn[NT][NS];
  float dn = 1.f;
  uint32_t vn[NT];
  auto load_tile = [&](const Place& x, int t) {
    const uint8_t* src = x.src + t * (BV * DK);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int s = 0; s < NS; ++s)
        rawn[j][s] = *reinterpret_cast<const u32x4*>(src + (loff + 16 * j * DK + 64 * s));
    dn = x.scale[t];
    const char* vp = x.v + t * (BV * ES);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      vn[j] = F32 ? reinterpret_cast<const uint32_t*>(vp)[row_in + 16 * j]
                  : reinterpret_cast<const uint16_t*>(vp)[row_in + 16 * j];
  };
  seq = __builtin_amdgcn_readfirstlane(e / hp);
  ph = e - seq * hp;
  const int slot0 = a.slots[seq];
  Place nxt = place(slot0, a.slots_out ? a.slots_out[seq] : slot0);
  if (nxt.slot >= 0 && nxt.slot < P.slots) {
    load_head(nxt);
    load_tile(nxt, 0);
  }
  int checked = -1, turn = 0;
  bool refused = false;
  for (; e < end; ++e) {
    const Place cur = nxt;
    // the element after this one
    const bool more = e + 1 < end;
    if (more) {
      int slot = cur.slot, to = cur.to;
      if (++ph == hp) {
        ph = 0;
        ++seq;
        slot = a.slots[seq];
        to = a.slots_out ? a.slots_out[seq] : slot;
      }
      nxt = place(slot, to);
    }
    const bool fetch = more && nxt.slot >= 0 && nxt.slot < P.slots;
    if (checked != cur.n) {
      checked = cur.n;
      refused = cur.slot < 0 || cur.slot >= P.slots || cur.to < -1 || cur.to >= P.slots ||
                (cur.to >= 0 &&
                 pool_claimed<false>(P, a.slots, a.slots_out ? a.slots_out : a.slots, a.B, cur.n, cur.to));
      if (refused && cur.slot != -1 && lane == 0) pool_error(P);
    }
    char* op = static_cast<char*>(a.o) + ((int64_t)cur.n * Hv * tph + cur.h * tph + cur.tile) * (BV * ES);
    auto put_o = [&](int t, const float (&o)[NT]) {
      if (g == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (F32) reinterpret_cast<float*>(op + t * (BV * ES))[row_in + 16 * j] = o[j];
          else reinterpret_cast<bf16*>(op + t * (BV * ES))[row_in + 16 * j] = to_bf16(o[j]);
        }
      }
    };
    if (refused) {                                     // or no sequence here
      if (cur.slot != -1) {
        float nan[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) nan[j] = __builtin_nanf("");
        for (int t = 0; t < span; ++t) put_o(t, nan);
      }
      if (fetch) {
        load_head(nxt);
        load_tile(nxt, 0);
      }
      continue;
    }
    head_to_lds<DK, F32>(hb, share);
    const float decay = expf(gn), beta = bn, kq = AFTER ? 0.f : head_kq<DK, F32>(hb, r, g);
    if (fetch) load_head(nxt);
    const int64_t topage = a.layer_page + cur.to, ctile = cur.h * tph + cur.tile;
    uint8_t* dst = P.data + topage * P.page + ctile * (BV * DK);
    float* dscale = P.scales + topage * P.tiles + ctile;
    for (int t = 0; t < span; ++t) {
      u32x4 raw[NT][NS];
      float v[NT], o[NT], d;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        v[j] = __builtin_bit_cast(float, F32 ? vn[j] : vn[j] << 16);   // not at the load: that would wait for it
#pragma unroll
        for (int s = 0; s < NS; ++s) raw[j][s] = rawn[j][s];
      }
      const float alpha = decay * dn;
      step_tile<DK, FMT, F32, NT>(
          P, hb, raw, alpha, beta, kq, a.scale, v, o, d, AFTER,
          [&]() {
            if (t + 1 < span) load_tile(cur, t + 1);
            else if (fetch) load_tile(nxt, 0);
          },
          [&](float m) {
            if constexpr (WPT > 1) {
              // the buffers alternate, so one barrier per tile is enough
              if (lane == 0) xm[turn][wave] = m;
              lds_barrier();
#pragma unroll
              for (int i = 0; i < NW; ++i) m = larger<FMT>(m, xm[turn][i]);
              turn ^= 1;
            }
            return m;
          });
      // the next tile's loads, and the last tile's stores, before this tile's
      // stores: a later wait for the loads would wait for these stores too
      vm_drain();
      put_o(t, o);
      if (cur.to >= 0) {
        uint8_t* dt = dst + t * (BV * DK);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int s = 0; s < NS; ++s)
            *reinterpret_cast<u32x4*>(dt + (loff + 16 * j * DK + 64 * s)) = raw[j][s];
        if (lane == 0 && sub == 0) dscale[t] = d;
      }
    }
  }
}

// ------------------------------------------------------ pages of FP32 states
// Eight lanes per row, four keys of every 32 each, so that they touch whole
// 128-byte lines in each load; a row sum is DK / 8 FMAs and three DPP adds. One
// wave holds kRows32 rows, four per eight lanes; waves are independent. 90
// sequences of up to 5 tokens, 6 heads of 64 x 64 (9 MB in, 9 out): 7.5 us, 8.2
// without the next token's loads ahead; bound by latency (four waves per CU).
constexpr int kRows32 = 32;
template <int DK, bool F32>
__global__ void __launch_bounds__(4 * WAVE) pool_step_f32_kernel(PoolStepArgs a, int waves) {
  constexpr int NV = DK / 32, ES = F32 ? 4 : 2, NR = kRows32 / 8;
  static_assert(NR == 4, "one vector of v and o per lane");
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= waves) return;
  const PoolRef& P = a.pool;
  const int lane = __lane_id(), c = lane & 7;
  const StepUnit w = step_unit(a, unit, kRows32);
  if (w.idle) {
    if (w.slot != -1 && !step_in_ok(a, w) && lane == 0) pool_error(P);
    return;
  }
  const int Hv = P.Hv, Dv = P.Dv, hk = w.h / (Hv / a.Hqk), row0 = w.row + (lane >> 3) * NR;
  const int64_t tok0 = (int64_t)w.n * a.T, o_tok = (int64_t)Hv * Dv;
  const int64_t head = ((int64_t)w.h * Dv + row0) * DK + 4 * c;
  f32x4 S[NR][NV];
  if (step_in_ok(a, w)) {
    const float* src = reinterpret_cast<const float*>(P.data + (a.layer_page + w.slot) * P.page) + head;
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int i = 0; i < NV; ++i) S[j][i] = *reinterpret_cast<const f32x4*>(src + j * DK + 32 * i);
  }
  f32x4 k[NV], q[NV], v, o;
  float gate = 0.f, beta = 0.f;
  auto load_token = [&](int t) {
    const char* kp = static_cast<const char*>(a.k) + ((tok0 + t) * a.ks + (int64_t)hk * DK + 4 * c) * ES;
    const char* qp = static_cast<const char*>(a.q) + ((tok0 + t) * a.qs + (int64_t)hk * DK + 4 * c) * ES;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      k[i] = load4<F32>(kp + 32 * i * ES);
      q[i] = load4<F32>(qp + 32 * i * ES);
    }
    v = load4<F32>(static_cast<const char*>(a.v) + ((tok0 + t) * a.vs + (int64_t)w.h * Dv + row0) * ES);
    gate = a.g[(tok0 + t) * Hv + w.h];
    beta = a.beta[(tok0 + t) * Hv + w.h];
  };
  if (w.T > 0) load_token(0);
  char* op = static_cast<char*>(a.o) + (tok0 * o_tok + (int64_t)w.h * Dv + row0) * ES;
  if (step_refused(a, w)) {
    if (lane == 0) pool_error(P);
    const float nan = __builtin_nanf("");
    if (c == 0)
      for (int t = 0; t < w.T; ++t) store4<F32>(op + t * o_tok * ES, f32x4{nan, nan, nan, nan});
    return;
  }
  for (int t = 0; t < w.T; ++t) {
    const float alpha = expf(gate), bt = beta;
    f32x4 kt[NV], qt[NV], vt = v;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      kt[i] = k[i];
      qt[i] = q[i];
    }
    if (t + 1 < w.T) load_token(t + 1);          // while this token is computed
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) kq = fmaf(kt[i][e], qt[i][e], kq);
    kq = sum_row(kq);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      float p = 0.f, x = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p = fmaf(S[j][i][e], kt[i][e], p);
          x = fmaf(S[j][i][e], qt[i][e], x);
        }
      p = sum_row(p);
      x = sum_row(x);
      const float u = bt * fmaf(-alpha, p, vt[j]);
      o[j] = a.scale * fmaf(kq, u, alpha * x);       // both readouts: nothing is rounded on the way
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][i][e] = fmaf(kt[i][e], u, alpha * S[j][i][e]);
    }
    if (c == 0) store4<F32>(op + t * o_tok * ES, o);
  }
  if (w.to < 0) return;
  float* dst = reinterpret_cast<float*>(P.data + (a.layer_page + w.to) * P.page) + head;
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int i = 0; i < NV; ++i) *reinterpret_cast<f32x4*>(dst + j * DK + 32 * i) = S[j][i];
}

inline int ilog2(int x) {
  int l = 0;
  while (x > 1) {
    x >>= 1;
    ++l;
  }
  return l;
}

template <int DK, int FMT, bool F32, int NT, int WPT>
void launch_codes_wpt(const PoolStepArgs& a, hipStream_t s) {
  constexpr int NW = WPT == 1 ? 4 : WPT;
  if (a.T == 1 && !a.lens) {
    // Groups that fit the device at three waves per SIMD. With at least as many
    // heads, an element is a whole head, and at most two per group: one
    // group for its share of all elements was slower at 1,024 sequences of 32
    // heads (467 us against 439 with two and 442 with one, of one build).
    const int tph = a.pool.Dv / a.pool.block_v, gpb = NW / WPT, heads = a.B * a.pool.Hv;
    const int room = device_cus() * std::max(1, 12 / NW) * gpb, span = heads >= room ? tph : 1;
    const int elems = heads * (tph / span), chunk = std::min(2, (elems + room - 1) / room);
    const int blocks = ((elems + chunk - 1) / chunk + gpb - 1) / gpb;
    if (a.readout)
      pool_step_one_kernel<DK, FMT, F32, NT, WPT, true><<<dim3(blocks), NW * WAVE, 0, s>>>(
          a, ilog2(span), ilog2(tph / span), elems, chunk);
    else
      pool_step_one_kernel<DK, FMT, F32, NT, WPT, false><<<dim3(blocks), NW * WAVE, 0, s>>>(
          a, ilog2(span), ilog2(tph / span), elems, chunk);
  } else {
    const int waves = a.B * a.pool.Hv * (a.pool.Dv / (16 * NT));
    pool_step_many_kernel<DK, FMT, F32, NT, WPT><<<dim3((waves + NW - 1) / NW), NW * WAVE, 0, s>>>(a, waves);
  }
}

// 16-row tiles per wave: two, or one where the integer format's conversions
// would spill at 128 keys (192 sequences of 16 heads; tiles of 32, 64 and 128 at Dv
// 128, of 256 at Dv 256: 31, 35, 53 and 111 us with one, 74, 77, 85 and 186 with two;
// E4M3 27.5, 28, 34 and 71 with one, 25.4, 25.4, 30 and 65.5 with two). A tile of 16
// is one. INT8 tiles of 256 at 128 keys are 16 waves, which caps them at 128
// registers: they spill 25 to 51.
template <int DK, int FMT, bool F32>
void launch_codes(const PoolStepArgs& a, hipStream_t s) {
  constexpr int NT = FMT == 2 && DK == 128 ? 1 : 2;
  switch (a.pool.block_v) {
    case 16: return launch_codes_wpt<DK, FMT, F32, 1, 1>(a, s);
    case 32: return launch_codes_wpt<DK, FMT, F32, NT, 2 / NT>(a, s);
    case 64: return launch_codes_wpt<DK, FMT, F32, NT, 4 / NT>(a, s);
    case 128: return launch_codes_wpt<DK, FMT, F32, NT, 8 / NT>(a, s);
    default: return launch_codes_wpt<DK, FMT, F32, NT, 16 / NT>(a, s);
  }
}

template <int DK, bool F32>
void launch_dk(const PoolStepArgs& a, hipStream_t s) {
  if (a.pool.fmt == 1) return launch_codes<DK, 1, F32>(a, s);
  if (a.pool.fmt == 2) return launch_codes<DK, 2, F32>(a, s);
  const int waves = a.B * a.pool.Hv * (a.pool.Dv / kRows32);
  pool_step_f32_kernel<DK, F32><<<dim3((unsigned)((waves + 3) / 4)), 4 * WAVE, 0, s>>>(a, waves);
}

}  // namespace

hipError_t launch_pool_step(const PoolStepArgs& a, hipStream_t s) {
  if (a.pool.Dk == 128) a.f32_io ? launch_dk<128, true>(a, s) : launch_dk<128, false>(a, s);
  else a.f32_io ? launch_dk<64, true>(a, s) : launch_dk<64, false>(a, s);
  return hipGetLastError();
}

}  // namespace gdn
