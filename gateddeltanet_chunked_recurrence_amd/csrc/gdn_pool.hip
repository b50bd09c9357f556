// State pool pages: FP32 states in and out, page copies, and the reordering
// of beams. All of it is data movement, bound by HBM; the recurrent step on
// the pages is in gdn_pool_step.hip.
//
// A page holds Hv states value-major: codes [Hv, Dv, Dk] with one scale per
// block_v value rows (the [Dk, block_v] tile of the chunk and decode paths, a
// contiguous block here), or FP32 states [Hv, Dv, Dk] with the format off.
#include "gdn_device.h"
#include "gdn_launch.h"
#include "gdn_pool.h"

namespace gdn {

namespace {

constexpr float kTinyScale = 1.17549435e-38f;   // 2^-126, the scale of a zero tile

// ------------------------------------------------- FP32 states <-> codes
// One workgroup per (state, group of whole tiles of at least 64 value
// columns), one wave per 64 columns x 64 keys. Lane (cq = lane & 15,
// kg = lane >> 4) holds columns 4 cq .. + 3 of keys 16 kg .. + 15: 16-byte FP32
// accesses, 256 contiguous bytes per key, and 16-byte code accesses, 64
// contiguous bytes per value row; the transposition between the key-major
// states and the value-major pages is then only the choice of registers. 64
// sequences of 16 heads of 128 x 128 (67 MB of FP32, 17 MB of codes): 17.2 us to
// pages, 14.8 from them, 4.9 and 5.7 TB/s.
template <int DK>
struct XchgPos {
  int n, h, col, key;
};
template <int DK>
__device__ __forceinline__ XchgPos<DK> xchg_pos(const PoolRef& P, int cols, int wave) {
  const int per = P.Dv / cols;
  const int b = blockIdx.x, n = b / (per * P.Hv), rem = b - n * per * P.Hv, h = rem / per;
  constexpr int KW = DK / 64;
  return {n, h, (rem - h * per) * cols + 64 * (wave / KW), 64 * (wave % KW)};
}

template <int DK, int FMT>
__global__ void __launch_bounds__(512) pool_write_kernel(PoolRef P, int64_t layer_page,
                                                         const int32_t* slots, int count,
                                                         const float* states, int cols) {
  __shared__ float xm[8][4];                     // amax per wave and 16 columns
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const XchgPos<DK> w = xchg_pos<DK>(P, cols, wave);
  const int slot = slots[w.n];
  if (slot == -1) return;
  const int cq = lane & 15, kg = lane >> 4, col = w.col + 4 * cq, key = w.key + 16 * kg;
  const float* src = states + ((int64_t)w.n * P.Hv + w.h) * DK * P.Dv + col;
  f32x4 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = *reinterpret_cast<const f32x4*>(src + (int64_t)(key + i) * P.Dv);
  if (slot < 0 || slot >= P.slots || pool_claimed<false>(P, slots, slots, count, w.n, slot)) {
    if (lane == 0) pool_error(P);
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = larger<FMT>(m, x[i][e]);
  // over the 16 columns of four lanes and the wave's 64 keys
  m = larger<FMT>(m, dpp_f<0xB1>(m));
  m = larger<FMT>(m, dpp_f<0x4E>(m));
  m = larger<FMT>(m, __shfl_xor(m, 16, WAVE));
  m = larger<FMT>(m, __shfl_xor(m, 32, WAVE));
  if (lane < 16 && (lane & 3) == 0) xm[wave][lane >> 2] = m;
  __syncthreads();
  // the tile's waves: its keys (KW of them) and, above 64 columns, its column blocks
  constexpr int KW = DK / 64;
  const int bv = P.block_v, nb = bv > 64 ? bv / 64 : 1, w0 = (wave / (KW * nb)) * KW * nb;
  const int q0 = bv >= 64 ? 0 : (cq >> 2) & ~(bv / 16 - 1), nq = bv >= 64 ? 4 : bv / 16;
  float amax = 0.f;
  for (int i = 0; i < KW * nb; ++i)
    for (int q = 0; q < nq; ++q) amax = larger<FMT>(amax, xm[w0 + i][q0 + q]);
  const float d = pool_scale<FMT>(P, amax), r = 1.0f / d;
  uint8_t* dst = P.data + (layer_page + slot) * P.page + (int64_t)w.h * P.Dv * DK;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[4] = {x[4 * i][e], x[4 * i + 1][e], x[4 * i + 2][e], x[4 * i + 3][e]};
      o[i] = quant_word<FMT>(y, r);
    }
    *reinterpret_cast<u32x4*>(dst + (int64_t)(col + e) * DK + key) = o;
  }
  if (w.key == 0 && kg == 0 && col % bv == 0)
    P.scales[(layer_page + slot) * P.tiles + w.h * (P.Dv / bv) + col / bv] = d;
}

template <int DK, int FMT>
__global__ void __launch_bounds__(512) pool_read_kernel(PoolRef P, int64_t layer_page,
                                                        const int32_t* slots, float* states,
                                                        int cols) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const XchgPos<DK> w = xchg_pos<DK>(P, cols, wave);
  const int slot = slots[w.n];
  const int cq = lane & 15, kg = lane >> 4, col = w.col + 4 * cq, key = w.key + 16 * kg;
  float* dst = states + ((int64_t)w.n * P.Hv + w.h) * DK * P.Dv + col;
  if (slot < 0 || slot >= P.slots) {             // -1: a fresh sequence, the zero state
    if (slot != -1 && lane == 0) pool_error(P);
    const float z = slot == -1 ? 0.f : __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < 16; ++i)
      *reinterpret_cast<f32x4*>(dst + (int64_t)(key + i) * P.Dv) = f32x4{z, z, z, z};
    return;
  }
  const uint8_t* src = P.data + (layer_page + slot) * P.page + (int64_t)w.h * P.Dv * DK;
  u32x4 c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = *reinterpret_cast<const u32x4*>(src + (int64_t)(col + e) * DK + key);
  // four columns never straddle a tile (block_v >= 16)
  const float d = P.scales[(layer_page + slot) * P.tiles + w.h * (P.Dv / P.block_v) + col / P.block_v];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) codes4<FMT>(c[e][i], x[e]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<f32x4*>(dst + (int64_t)(key + 4 * i + k) * P.Dv) =
          f32x4{x[0][k] * d, x[1][k] * d, x[2][k] * d, x[3][k] * d};
  }
}

// FP32 pages: the transposition of FP32 states. One wave per 32 columns x 64
// keys; lane (cq = lane & 7, kq = lane >> 3) moves 4 x 4 blocks at columns
// 4 cq and keys 4 kq (+ 32 for the second block), whole 128-byte lines on both
// sides: eight lanes along the columns in a load, eight along the keys in a
// store. 64 sequences of 16 heads of 128 x 128, out and in (268 MB): 60 us, 4.5 TB/s.
template <bool WRITE>
__global__ void __launch_bounds__(256) pool_f32_kernel(PoolRef P, int64_t layer_page,
                                                       const int32_t* slots, int count,
                                                       float* states, int units) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = __lane_id();
  const int u = blockIdx.x * 4 + wave;
  if (u >= units) return;
  const int kw = P.Dk / 64, per = P.Dv / 32 * kw;
  const int n = u / (per * P.Hv), rem = u - n * per * P.Hv, h = rem / per, b = rem - h * per;
  const int slot = slots[n];
  if (WRITE && slot == -1) return;
  bool ok = slot >= 0 && slot < P.slots;
  if (WRITE && ok) ok = !pool_claimed<false>(P, slots, slots, count, n, slot);
  if (!ok && slot != -1 && lane == 0) pool_error(P);
  if (WRITE && !ok) return;
  const int64_t page_off = ok ? (layer_page + slot) * P.page : 0;
  float* page = reinterpret_cast<float*>(P.data + page_off) + (int64_t)h * P.Dv * P.Dk;
  float* st = states + ((int64_t)n * P.Hv + h) * P.Dk * P.Dv;
  const int c0 = 32 * (b / kw), k0 = 64 * (b % kw), l8 = lane & 7, g8 = lane >> 3;
  f32x4 x[2][4];
  if (WRITE) {
    const int col = c0 + 4 * l8;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[s][i] = *reinterpret_cast<const f32x4*>(st + (int64_t)(k0 + 32 * s + 4 * g8 + i) * P.Dv + col);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(page + (int64_t)(col + e) * P.Dk + k0 + 32 * s + 4 * g8) =
            f32x4{x[s][0][e], x[s][1][e], x[s][2][e], x[s][3][e]};
  } else {
    // lanes along the keys in the load: the roles of l8 and g8 change
    const int col = c0 + 4 * g8;
    const float z = slot == -1 ? 0.f : __builtin_nanf("");
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[s][e] = ok ? *reinterpret_cast<const f32x4*>(page + (int64_t)(col + e) * P.Dk + k0 + 32 * s + 4 * l8)
                     : f32x4{z, z, z, z};
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(st + (int64_t)(k0 + 32 * s + 4 * l8 + i) * P.Dv + col) =
            f32x4{x[s][0][i], x[s][1][i], x[s][2][i], x[s][3][i]};
  }
}

// ------------------------------------------------------------ page copies
// One workgroup per (part of a page, move, layer); 16 bytes per lane and
// access, U accesses each. The last part is the page's scales. The loads go
// out before the slots are checked for being named twice, the stores after.
// Stores are non-temporal, loads are not: 60 forks of 12 layers (208 MB read
// once and written, pages of 256 KB) take 39 us so (5.3 TB/s; a large linear
// copy reaches 5.6 to 6.6 on this card), 45 with plain stores, 58 with
// non-temporal loads too (a parent is read several times) or with the check
// before the loads; 49 with one access per lane, 39.5 with eight.
constexpr int kMoveThreads = 256;

template <int U>
__global__ void __launch_bounds__(kMoveThreads) pool_copy_kernel(PoolRef P, const int32_t* src,
                                                                 const int32_t* dst, int count,
                                                                 int parts) {
  const int part = blockIdx.x, m = blockIdx.y, layer = blockIdx.z, lane = __lane_id();
  const int from = src[m], to = dst[m];
  const bool ok = from >= -1 && from < P.slots && to >= 0 && to < P.slots;
  if (to == -1 || (from == to && ok)) return;
  const int64_t base = (int64_t)layer * P.slots;
  u32x4 x[U];
  const int64_t off = (int64_t)part * (U * kMoveThreads * 16) + threadIdx.x * 16;
  if (part < parts) {
    const uint8_t* s = P.data + (base + from) * P.page + off;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = u32x4{0, 0, 0, 0};
      if (ok && from >= 0 && off + (int64_t)i * (kMoveThreads * 16) < P.page)
        x[i] = *reinterpret_cast<const u32x4*>(s + i * (kMoveThreads * 16));
    }
  }
  if (!ok || pool_claimed<true>(P, src, dst, count, m, to)) {
    if (lane == 0) pool_error(P);
    return;
  }
  if (part == parts) {
    float* d = P.scales + (base + to) * P.tiles;
    for (int i = threadIdx.x; i < P.tiles; i += kMoveThreads)
      d[i] = from < 0 ? kTinyScale : P.scales[(base + from) * P.tiles + i];
    return;
  }
  uint8_t* d = P.data + (base + to) * P.page + off;
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (off + (int64_t)i * (kMoveThreads * 16) < P.page)
      __builtin_nontemporal_store(x[i], reinterpret_cast<u32x4*>(d + i * (kMoveThreads * 16)));
}

// ------------------------------------------------------------- reordering
// Beam w of a group takes the page of beam parents[w], all at once and in
// place: a lane holds its 16 bytes of every beam's parent (W registers of 16
// bytes), so no page is read after it was written and no staging copy is
// needed; each page that changes is written once and each parent read once
// from HBM (a second beam of the same parent hits a cache). Beams that keep
// their own page move nothing. 16 groups of 4 beams, 12 layers (268 MB): 47 us
// (5.7 TB/s; 44 to 49 by what the caches still hold); with plain stores 64, with one
// part per lane 55. 4 groups of 16 (314 MB) take 57 us, 2 of 32 (321 MB) 56, though
// the widest bucket holds 167 registers and spills scalars.
template <int W, int U>
__global__ void __launch_bounds__(kMoveThreads)
pool_reorder_kernel(PoolRef P, const int32_t* slots, const int32_t* parents, int width, int parts) {
  const int part = blockIdx.x, grp = blockIdx.y, layer = blockIdx.z, lane = __lane_id();
  const int total = gridDim.y * width;
  // the beams' slots and parents, one lane each
  int slot = -1, par = -1;
  if (lane < width) {
    slot = slots[grp * width + lane];
    par = parents[grp * width + lane];
  }
  // a beam moves when it has a page, a parent and they differ; a slot outside
  // the pool is an error also where nothing moves
  const bool wants = slot != -1 && par != -1 && par != lane;
  const int from = __shfl(slot, par >= 0 && par < width ? par : 0, WAVE);
  bool bad = slot < -1 || slot >= P.slots || (wants && (par < 0 || par >= width || from < 0 || from >= P.slots));
  const uint64_t loads = __ballot(wants && !bad);
  const int64_t base = (int64_t)layer * P.slots;
  const int64_t off = (int64_t)part * (U * kMoveThreads * 16) + threadIdx.x * 16;
  u32x4 x[W][U];
  if (part < parts) {
#pragma unroll
    for (int w = 0; w < W; ++w)
      if ((loads >> w) & 1) {
        const uint8_t* s = P.data + (base + __builtin_amdgcn_readlane(from, w)) * P.page + off;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (off + (int64_t)i * (kMoveThreads * 16) < P.page)
            x[w][i] = *reinterpret_cast<const u32x4*>(s + i * (kMoveThreads * 16));
      }
  }
  // slots named twice: the lanes scan all entries, for every moving beam at once
  uint32_t hits = 0;
  for (int j = lane; j < total; j += WAVE) {
    const int other = slots[j];
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (((loads >> w) & 1) && other == __builtin_amdgcn_readlane(slot, w) && j != grp * width + w) hits |= 1u << w;
  }
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (((loads >> w) & 1) && __ballot((hits >> w) & 1) && lane == w) bad = true;
  if (bad) pool_error(P);
  const uint64_t any = __ballot(wants && !bad);
  if (part == parts) {
    for (int i = threadIdx.x; i < P.tiles; i += kMoveThreads) {
      float y[W];
#pragma unroll
      for (int w = 0; w < W; ++w)
        if ((any >> w) & 1) y[w] = P.scales[(base + __builtin_amdgcn_readlane(from, w)) * P.tiles + i];
#pragma unroll
      for (int w = 0; w < W; ++w)
        if ((any >> w) & 1) P.scales[(base + __builtin_amdgcn_readlane(slot, w)) * P.tiles + i] = y[w];
    }
    return;
  }
#pragma unroll
  for (int w = 0; w < W; ++w)
    if ((any >> w) & 1) {
      uint8_t* d = P.data + (base + __builtin_amdgcn_readlane(slot, w)) * P.page + off;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (off + (int64_t)i * (kMoveThreads * 16) < P.page)
          __builtin_nontemporal_store(x[w][i], reinterpret_cast<u32x4*>(d + i * (kMoveThreads * 16)));
    }
}

template <int W, int U>
hipError_t reorder_launch(const PoolRef& p, const int32_t* slots, const int32_t* parents, int groups,
                          int width, hipStream_t s) {
  const int parts = (int)((p.page + U * kMoveThreads * 16 - 1) / (U * kMoveThreads * 16));
  pool_reorder_kernel<W, U><<<dim3(parts + (p.tiles > 0), groups, p.layers), kMoveThreads, 0, s>>>(
      p, slots, parents, width, parts);
  return hipGetLastError();
}

template <int DK, int FMT>
hipError_t write_launch(const PoolRef& p, int64_t lp, const int32_t* slots, int n, const float* states,
                        hipStream_t s) {
  const int cols = p.block_v > 64 ? p.block_v : 64;
  pool_write_kernel<DK, FMT><<<dim3((unsigned)(n * p.Hv * (p.Dv / cols))), cols / 64 * (DK / 64) * WAVE, 0,
                               s>>>(p, lp, slots, n, states, cols);
  return hipGetLastError();
}
template <int DK, int FMT>
hipError_t read_launch(const PoolRef& p, int64_t lp, const int32_t* slots, int n, float* states,
                       hipStream_t s) {
  pool_read_kernel<DK, FMT><<<dim3((unsigned)(n * p.Hv * (p.Dv / 64))), DK / 64 * WAVE, 0, s>>>(
      p, lp, slots, states, 64);
  return hipGetLastError();
}

template <bool WRITE>
hipError_t f32_launch(const PoolRef& p, int64_t lp, const int32_t* slots, int n, float* states,
                      hipStream_t s) {
  const int units = n * p.Hv * (p.Dv / 32) * (p.Dk / 64);
  pool_f32_kernel<WRITE><<<dim3((unsigned)((units + 3) / 4)), 4 * WAVE, 0, s>>>(p, lp, slots, n, states, units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pool_write(const PoolRef& p, int layer, const int32_t* slots, int n,
                             const float* states, hipStream_t s) {
  const int64_t lp = (int64_t)layer * p.slots;
  if (p.fmt == 0) return f32_launch<true>(p, lp, slots, n, const_cast<float*>(states), s);
  if (p.Dk == 128)
    return p.fmt == 1 ? write_launch<128, 1>(p, lp, slots, n, states, s)
                      : write_launch<128, 2>(p, lp, slots, n, states, s);
  return p.fmt == 1 ? write_launch<64, 1>(p, lp, slots, n, states, s)
                    : write_launch<64, 2>(p, lp, slots, n, states, s);
}

hipError_t launch_pool_read(const PoolRef& p, int layer, const int32_t* slots, int n, float* states,
                            hipStream_t s) {
  const int64_t lp = (int64_t)layer * p.slots;
  if (p.fmt == 0) return f32_launch<false>(p, lp, slots, n, states, s);
  if (p.Dk == 128)
    return p.fmt == 1 ? read_launch<128, 1>(p, lp, slots, n, states, s)
                      : read_launch<128, 2>(p, lp, slots, n, states, s);
  return p.fmt == 1 ? read_launch<64, 1>(p, lp, slots, n, states, s)
                    : read_launch<64, 2>(p, lp, slots, n, states, s);
}

hipError_t launch_pool_copy(const PoolRef& p, const int32_t* src, const int32_t* dst, int n,
                            hipStream_t s) {
  constexpr int U = 4;
  const int parts = (int)((p.page + U * kMoveThreads * 16 - 1) / (U * kMoveThreads * 16));
  pool_copy_kernel<U><<<dim3(parts + (p.tiles > 0), n, p.layers), kMoveThreads, 0, s>>>(p, src, dst, n, parts);
  return hipGetLastError();
}

// The bucket of the width; narrow groups take several parts per lane.
hipError_t launch_pool_reorder(const PoolRef& p, const int32_t* slots, const int32_t* parents,
                               int groups, int width, hipStream_t s) {
  if (width <= 4) return reorder_launch<4, 4>(p, slots, parents, groups, width, s);
  if (width <= 8) return reorder_launch<8, 2>(p, slots, parents, groups, width, s);
  if (width <= 16) return reorder_launch<16, 1>(p, slots, parents, groups, width, s);
  return reorder_launch<32, 1>(p, slots, parents, groups, width, s);
}

}  // namespace gdn
