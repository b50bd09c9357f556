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
// so the state is decoded once, both products read the codes as they are
// (exact in FP32) and the output needs no pass over S'. All arithmetic is FP32.
//
// Bound: a token moves Dk Dv bytes in and out per head for 6 Dk Dv FLOP, so
// at many sequences this is a copy (bound by HBM). The page is value-major
// ([Dv, Dk], Dk contiguous): a scale tile is one contiguous block, and the
// sums over Dk run along a row, mostly inside a lane: 8 lanes (Dk 128; 4 at
// Dk 64) hold a row as 16 codes each, so a sum is 16 FMAs and 3 (2) DPP adds.
// With key-major pages every row sum would instead cross 16 lanes for each of
// 16 columns. One wave holds RPW consecutive rows of one tile (16-byte loads,
// NLD per lane, all issued at once); a tile of several waves exchanges its
// amax through LDS. The vector ALUs do the products: at most 7 instructions
// per element, and matrix cores would need the codes converted to bf16 and
// leave 14 of 16 columns empty.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_pool.h"

namespace gdn {

namespace {

// The sum over the LPR lanes that hold one row (4 or 8 neighbours).
template <int LPR>
__device__ __forceinline__ float sum_row(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  if constexpr (LPR == 8) x += dpp_f<0x141>(x);
  return x;
}

// N consecutive bf16 or FP32 elements at p (aligned to their size, at most 16
// bytes per access).
template <int N, bool F32>
__device__ __forceinline__ void ld_run(const void* p, float (&x)[N]) {
  if constexpr (F32) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const f32x4 v = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = reinterpret_cast<const float*>(p)[i];
    }
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const bf16x8 v = reinterpret_cast<const bf16x8*>(p)[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * i + e] = from_bf16(v[e]);
    }
  } else if constexpr (N == 4) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = from_bf16(v[e]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = from_bf16(reinterpret_cast<const bf16*>(p)[i]);
  }
}

template <int N, bool F32>
__device__ __forceinline__ void st_run(void* p, const float (&x)[N]) {
  if constexpr (F32) {
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<f32x4*>(p)[i] = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<float*>(p)[i] = x[i];
    }
  } else if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      bf16x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = to_bf16(x[8 * i + e]);
      reinterpret_cast<bf16x8*>(p)[i] = v;
    }
  } else if constexpr (N == 4) {
    *reinterpret_cast<bf16x4*>(p) = bf16x4{to_bf16(x[0]), to_bf16(x[1]), to_bf16(x[2]), to_bf16(x[3])};
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<bf16*>(p)[i] = to_bf16(x[i]);
  }
}

// How a wave covers its rows. With codes a lane holds 16 consecutive keys of
// a row; FP32 states are read as four keys every 32, so that the eight lanes
// of a row together touch whole 128-byte lines in each load.
template <int DK, int FMT>
struct StepMap {
  static constexpr int LPR = FMT != 0 ? DK / 16 : 8;    // lanes per row
  static constexpr int EPL = DK / LPR;                  // keys per lane
  static constexpr int GR = WAVE / LPR;                 // rows side by side
};

// NW waves per workgroup. A tile of WPT waves (block_v / RPW) is one
// workgroup (NW = WPT); with WPT = 1 the waves are independent.
template <int DK, int FMT, bool F32, int NLD, int NW>
__global__ void __launch_bounds__(NW * WAVE) pool_step_kernel(PoolStepArgs a, int wpt, int waves) {
  using M = StepMap<DK, FMT>;
  constexpr int LPR = M::LPR, EPL = M::EPL, RPW = M::GR * NLD, ES = F32 ? 4 : 2;
  __shared__ float xm[2][NW];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const int gw = blockIdx.x * NW + wave;
  if (gw >= waves) return;                      // only where the waves are independent
  const PoolRef& P = a.pool;
  const int Hv = P.Hv, Dv = P.Dv, per = Dv / RPW;
  const int n = gw / (per * Hv), rem = gw - n * per * Hv, h = rem / per, row_w = (rem - h * per) * RPW;
  const int grp = lane / LPR, c = lane % LPR, row0 = row_w + grp * NLD;   // the lane's first row
  int T = a.T;
  if (a.lens) T = min(max(a.lens[n], 0), T);
  const int slot = a.slots[n];
  if (slot == -1) return;                       // no sequence here (uniform over a tile)
  const int32_t* outs = a.slots_out ? a.slots_out : a.slots;
  const int to = outs[n];
  const bool in_ok = slot >= 0 && slot < P.slots, out_ok = to >= -1 && to < P.slots;

  u32x4 raw[NLD * (FMT != 0 ? 1 : EPL / 4)];
  const int64_t head = (int64_t)h * Dv * DK * (FMT != 0 ? 1 : 4);
  // byte offset of the lane's piece j within a page
  auto piece = [&](int j) -> int64_t {
    if constexpr (FMT != 0) return head + (int64_t)(row0 + j) * DK + 16 * c;
    else return head + ((int64_t)(row0 + j / (EPL / 4)) * DK + 32 * (j % (EPL / 4)) + 4 * c) * 4;
  };
  if (in_ok) {
    const uint8_t* src = P.data + (a.layer_page + slot) * P.page;
#pragma unroll
    for (int j = 0; j < (int)(sizeof(raw) / sizeof(raw[0])); ++j)
      raw[j] = *reinterpret_cast<const u32x4*>(src + piece(j));
  }
  const int tile = FMT != 0 ? h * (Dv / P.block_v) + row_w / P.block_v : 0;
  float d = 1.f;
  if (FMT != 0 && in_ok) d = P.scales[(a.layer_page + slot) * P.tiles + tile];
  const bool claimed = to >= 0 && pool_claimed(a.slots, outs, a.B, n, to, 0);
  const int hk = h / (Hv / a.Hqk);
  const int64_t o_tok = (int64_t)Hv * Dv;
  const int64_t o_off = (int64_t)n * a.T * o_tok + (int64_t)h * Dv + row0;
  if (!in_ok || !out_ok || claimed) {
    // refused: the outputs say so, the pages stay as they are
    if (lane == 0) pool_error(P);
    float nan[NLD];
#pragma unroll
    for (int j = 0; j < NLD; ++j) nan[j] = __builtin_nanf("");
    if (c == 0)
      for (int t = 0; t < T; ++t)
        st_run<NLD, F32>(static_cast<char*>(a.o) + (o_off + t * o_tok) * ES, nan);
    return;
  }
  if (T == 0 && to == slot) return;

  float S[NLD][EPL];
#pragma unroll
  for (int j = 0; j < NLD; ++j) {
    if constexpr (FMT != 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) codes4<FMT>(raw[j][i], *reinterpret_cast<float(*)[4]>(&S[j][4 * i]));
    } else {
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i) {
        const f32x4 x = __builtin_bit_cast(f32x4, raw[j * (EPL / 4) + i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][4 * i + e] = x[e];
      }
    }
  }
  const char* qp = static_cast<const char*>(a.q) + ((int64_t)n * a.T * a.qs + (int64_t)hk * DK) * ES;
  const char* kp = static_cast<const char*>(a.k) + ((int64_t)n * a.T * a.ks + (int64_t)hk * DK) * ES;
  const char* vp = static_cast<const char*>(a.v) + ((int64_t)n * a.T * a.vs + (int64_t)h * Dv + row0) * ES;
  auto ld_keys = [&](const char* p, float (&x)[EPL]) {
    if constexpr (FMT != 0) {
      ld_run<EPL, F32>(p + 16 * c * ES, x);
    } else {
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i)
        ld_run<4, F32>(p + (32 * i + 4 * c) * ES, *reinterpret_cast<float(*)[4]>(&x[4 * i]));
    }
  };
  for (int t = 0; t < T; ++t) {
    float k[EPL], q[EPL], v[NLD], o[NLD];
    ld_keys(kp + (int64_t)t * a.ks * ES, k);
    ld_keys(qp + (int64_t)t * a.qs * ES, q);
    ld_run<NLD, F32>(vp + (int64_t)t * a.vs * ES, v);
    const int64_t gi = ((int64_t)n * a.T + t) * Hv + h;
    const float alpha = expf(a.g[gi]) * d, beta = a.beta[gi];
    float kq = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) kq = fmaf(k[e], q[e], kq);
    kq = sum_row<LPR>(kq);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NLD; ++j) {
      float p = 0.f, w = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        p = fmaf(S[j][e], k[e], p);
        w = fmaf(S[j][e], q[e], w);
      }
      p = sum_row<LPR>(p);
      w = sum_row<LPR>(w);
      const float u = beta * fmaf(-alpha, p, v[j]);
      o[j] = a.scale * fmaf(kq, u, alpha * w);
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        S[j][e] = fmaf(k[e], u, alpha * S[j][e]);
        m = fmaxf(m, fabsf(S[j][e]));
      }
    }
    if constexpr (FMT != 0) {
      m = wave_max(m);
      if (wpt > 1) {
        // the buffers alternate, so one barrier per token is enough: a wave
        // that writes xm[t & 1] again has passed the barrier of token t + 1,
        // which every wave reaches after reading xm[t & 1]
        if (lane == 0) xm[t & 1][wave] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) m = fmaxf(m, xm[t & 1][i]);
      }
      d = qdq_scale<FMT>(m);
      const float r = 1.0f / d;
#pragma unroll
      for (int j = 0; j < NLD; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          raw[j][i] = quant_word<FMT>(*reinterpret_cast<float(*)[4]>(&S[j][4 * i]), r);
    }
    if (a.readout != 0) {
#pragma unroll
      for (int j = 0; j < NLD; ++j) {
        float w = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) w = fmaf(S[j][e], q[e], w);
        o[j] = a.scale * (d * sum_row<LPR>(w));
      }
    }
    if (c == 0) st_run<NLD, F32>(static_cast<char*>(a.o) + (o_off + t * o_tok) * ES, o);
  }
  if (to < 0) return;                           // the state is not kept
  uint8_t* dst = P.data + (a.layer_page + to) * P.page;
  if constexpr (FMT == 0) {
#pragma unroll
    for (int j = 0; j < NLD; ++j)
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i)
        raw[j * (EPL / 4) + i] = __builtin_bit_cast(
            u32x4, f32x4{S[j][4 * i], S[j][4 * i + 1], S[j][4 * i + 2], S[j][4 * i + 3]});
  }
#pragma unroll
  for (int j = 0; j < (int)(sizeof(raw) / sizeof(raw[0])); ++j)
    *reinterpret_cast<u32x4*>(dst + piece(j)) = raw[j];
  if (FMT != 0 && lane == 0 && row_w % P.block_v == 0)
    P.scales[(a.layer_page + to) * P.tiles + tile] = d;
}

template <int DK, int FMT, bool F32, int RPW>
hipError_t launch_rows(const PoolStepArgs& a, hipStream_t s) {
  constexpr int NLD = RPW / StepMap<DK, FMT>::GR;
  const int wpt = FMT != 0 ? a.pool.block_v / RPW : 1;
  const int64_t waves = (int64_t)a.B * a.pool.Hv * (a.pool.Dv / RPW);
  if (wpt <= 4) {
    // tiles of one, two or four waves: workgroups of four, or of the tile
    if (wpt == 2)
      pool_step_kernel<DK, FMT, F32, NLD, 2><<<dim3((unsigned)(waves / 2)), 2 * WAVE, 0, s>>>(a, wpt, (int)waves);
    else
      pool_step_kernel<DK, FMT, F32, NLD, 4><<<dim3((unsigned)((waves + 3) / 4)), 4 * WAVE, 0, s>>>(a, wpt, (int)waves);
  } else if (wpt == 8) {
    pool_step_kernel<DK, FMT, F32, NLD, 8><<<dim3((unsigned)(waves / 8)), 8 * WAVE, 0, s>>>(a, wpt, (int)waves);
  } else {
    pool_step_kernel<DK, FMT, F32, NLD, 16><<<dim3((unsigned)(waves / 16)), 16 * WAVE, 0, s>>>(a, wpt, (int)waves);
  }
  return hipGetLastError();
}

template <int DK, int FMT, bool F32>
hipError_t launch_dk(const PoolStepArgs& a, hipStream_t s) {
  if (FMT != 0 && a.pool.block_v == 16) return launch_rows<DK, FMT, F32, 16>(a, s);
  return launch_rows<DK, FMT, F32, 32>(a, s);
}

template <int DK, int FMT>
hipError_t launch_fmt(const PoolStepArgs& a, hipStream_t s) {
  return a.f32_io ? launch_dk<DK, FMT, true>(a, s) : launch_dk<DK, FMT, false>(a, s);
}

template <int DK>
hipError_t launch_pool_step_dk(const PoolStepArgs& a, hipStream_t s) {
  if (a.pool.fmt == 0) return launch_fmt<DK, 0>(a, s);
  return a.pool.fmt == 1 ? launch_fmt<DK, 1>(a, s) : launch_fmt<DK, 2>(a, s);
}

}  // namespace

hipError_t launch_pool_step(const PoolStepArgs& a, hipStream_t s) {
  return a.pool.Dk == 128 ? launch_pool_step_dk<128>(a, s) : launch_pool_step_dk<64>(a, s);
}

}  // namespace gdn
