// Residual add + RMSNorm with 8-bit outputs, and its backward:
//
//   h = x + res;  r = 1 / sqrt(mean(h^2) + eps);  y = gamma * h * r
//   forward   h in bf16 and y as e4m3, with the scales the 8-bit GEMMs take
//             (one power of two per 32 columns, or one per tensor)
//   backward  g = dy * gamma;  dx = r g - r (r mean(g h)) (r h) + d_h;
//             dgamma = sum_i dy (r h)
//
// Each element is read once and each output written once; both are bound by
// HBM (7 and 8 bytes an element).  A row lives in the registers of one block or
// warp from its load to its store: sums, r and y are fp32, h and dx are rounded
// to bf16 once.
#pragma once

#include "coda_embed.cuh"

namespace coda {

// Sum over the row's threads, a warp or the block (of two warps or more); every
// one gets it.  `red` holds 32 floats; the caller synchronises before its next use.
template <bool WARP>
__device__ __forceinline__ float norm8_sum(float s, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (WARP) return s;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = red[threadIdx.x & 31];  // entries past the block's warps are zero
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One block per row, or (WARP) a warp; its thread t holds the 8-column vectors
// t and t + threads.  MX: four neighbouring threads hold a 32-column block,
// sixteen the four blocks whose scale bytes make one word of the A layout; rows
// from M up to a whole 128-row block only write their scale bytes (127).
// !MX: codes of y / s_y; amax = max |y| by atomic max on its bits (the order of
// a maximum does not matter), or a plain store where one block is all.
constexpr int kNorm8Vpt = 2;

template <bool MX, bool WARP, int MAXT, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) add_rmsnorm_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ res,
    const __nv_bfloat16* __restrict__ gamma, float eps, const float* __restrict__ s_y,
    __nv_bfloat16* __restrict__ h_out, uint8_t* __restrict__ q, uint8_t* __restrict__ sf, unsigned* amax,
    float* __restrict__ r_out, int64_t M, int N, int nrb) {
  constexpr int VPT = kNorm8Vpt;
  __shared__ float red[32];
  __shared__ unsigned mred[32];
  pdl_begin();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (MX && row >= M) {
    for (int j = tid; j < N / 128; j += nt)
      *reinterpret_cast<uint32_t*>(sf + mx_sf_offset_a(static_cast<int>(row), 4 * j, nrb)) = 0x7f7f7f7fu;
    return;
  }
  if (!WARP && tid < 32) red[tid] = 0.f;
  const int cols = row < M ? N : 0;  // (past the last row a warp only takes part in the maximum)
  const size_t ro = static_cast<size_t>(row) * N;
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (tid + k * nt) * 8;
    xv[k] = rv[k] = make_uint4(0, 0, 0, 0);
    if (c < cols) {
      xv[k] = __ldcs(reinterpret_cast<const uint4*>(x + ro + c));
      if (res != nullptr) rv[k] = __ldcs(reinterpret_cast<const uint4*>(res + ro + c));
    }
  }
  uint4 gv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (tid + k * nt) * 8;
    gv[k] = c < cols ? __ldg(reinterpret_cast<const uint4*>(gamma + c)) : make_uint4(0, 0, 0, 0);
  }
  if (!WARP) __syncthreads();  // `red` is cleared
  float h[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const uint32_t xw[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w};
    const uint32_t rw[4] = {rv[k].x, rv[k].y, rv[k].z, rv[k].w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf16lo(xw[e]) + bf16lo(rw[e]), b = bf16hi(xw[e]) + bf16hi(rw[e]);
      h[k][2 * e] = a;
      h[k][2 * e + 1] = b;
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
      o[e] = pack_bf16x2(a, b);
    }
    const int c = (tid + k * nt) * 8;
    if (h_out != nullptr && c < cols) *reinterpret_cast<uint4*>(h_out + ro + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  const float r = rsqrtf(norm8_sum<WARP>(ss, red) / static_cast<float>(N) + eps);
  if (tid == 0 && cols > 0 && r_out != nullptr) r_out[row] = r;
  const float inv = MX ? 0.f : 1.0f / __ldg(s_y);
  float am = 0.f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (tid + k * nt) * 8;
    const uint32_t gw[4] = {gv[k].x, gv[k].y, gv[k].z, gv[k].w};
    float y[8];
    float bm = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = bf16lo(gw[e]) * h[k][2 * e] * r;
      y[2 * e + 1] = bf16hi(gw[e]) * h[k][2 * e + 1] * r;
      bm = fmaxf(bm, fmaxf(fabsf(y[2 * e]), fabsf(y[2 * e + 1])));
    }
    float f = inv;
    if (MX) {
      bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
      bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
      const int e = mx_e4m3_exponent(bm);
      f = exp2_neg(e);
      uint32_t word = static_cast<uint32_t>(e + 127) << (8 * ((threadIdx.x >> 2) & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if ((threadIdx.x & 15) == 0 && c < cols)
        *reinterpret_cast<uint32_t*>(sf + mx_sf_offset_a(static_cast<int>(row), c >> 5, nrb)) = word;
    } else {
      am = fmaxf(am, bm);
    }
    const uint32_t q0 = pack_e4m3x2(y[0] * f, y[1] * f) | (pack_e4m3x2(y[2] * f, y[3] * f) << 16);
    const uint32_t q1 = pack_e4m3x2(y[4] * f, y[5] * f) | (pack_e4m3x2(y[6] * f, y[7] * f) << 16);
    if (c < cols) *reinterpret_cast<uint2*>(q + ro + c) = make_uint2(q0, q1);
  }
  if (!MX) {
    unsigned u = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
    if (blockDim.x > 32) {
      if ((threadIdx.x & 31) == 0) mred[threadIdx.x >> 5] = u;
      __syncthreads();
      if (threadIdx.x >= 32) return;
      u = __reduce_max_sync(0xffffffffu, threadIdx.x < blockDim.x / 32 ? mred[threadIdx.x] : 0u);
    }
    if (threadIdx.x == 0) {
      if (gridDim.x == 1)
        *amax = u;
      else if (u != 0u)
        atomicMax(amax, u);
    }
  }
}

// A block (WARP: a warp) walks rows blockIdx, + gridDim, ...  dgamma's terms stay
// in registers over the block's rows; the blocks' sums part[block][N] are added up
// by norm8_dgamma_kernel in a fixed order.  What bounds it is how much is in
// flight.  Up to 128 threads (2048 columns) the next row's vectors are requested
// before this row's sum is reduced, in as many blocks (BLOCKS of MAXT threads on
// an SM) as have registers for both rows: 8192 x 2048 with 4 or 5 blocks 24.7 us,
// 6 31.9, without the next row and 8 blocks 28.1; 8192 x 1536 with 4 21.3, with 5
// 20.4.  Wider rows are better off with twice the blocks and one row each (8192 x
// 4096: 50.3 us against 59.0, 4096 x 4104 32.0 against 50.5, 4096 x 8192 51.1
// against 66.3).  Times are of the whole call, this launch and
// norm8_dgamma_kernel, back to back with its outputs given.
template <bool WARP, int MAXT, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) add_rmsnorm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, const __nv_bfloat16* __restrict__ h, const float* __restrict__ r,
    const __nv_bfloat16* __restrict__ gamma, const __nv_bfloat16* __restrict__ d_h, __nv_bfloat16* __restrict__ dx,
    float* __restrict__ part, int64_t M, int N) {
  constexpr int VPT = kNorm8Vpt;
  constexpr bool kAhead = MAXT <= 128;
  __shared__ float red[2][32];
  pdl_begin();
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
  const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * (MAXT / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * (MAXT / 32) : gridDim.x;
  if (!WARP && tid < 32) red[0][tid] = red[1][tid] = 0.f;
  uint4 yv[VPT], hv[VPT], sv[VPT];
  float dg[VPT][8];
  const auto load = [&](int64_t row) {
    const size_t ro = static_cast<size_t>(row) * N;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (tid + k * nt) * 8;
      yv[k] = hv[k] = sv[k] = make_uint4(0, 0, 0, 0);
      if (c < N && row < M) {
        yv[k] = __ldcs(reinterpret_cast<const uint4*>(dy + ro + c));
        hv[k] = __ldcs(reinterpret_cast<const uint4*>(h + ro + c));
        if (d_h != nullptr) sv[k] = __ldcs(reinterpret_cast<const uint4*>(d_h + ro + c));
      }
    }
  };
  const auto gamma_of = [&](int k) {  // (from L1: registers hold the rows in flight)
    const int c = (tid + k * nt) * 8;
    return c < N ? __ldg(reinterpret_cast<const uint4*>(gamma + c)) : make_uint4(0, 0, 0, 0);
  };
  if (kAhead) load(first);
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[k][e] = 0.f;
  if (!WARP) __syncthreads();
  int it = 0;
  for (int64_t row = first; row < M; row += step, it ^= 1) {
    if (!kAhead) load(row);
    uint4 y0[VPT], h0[VPT], s0[VPT];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      y0[k] = yv[k];
      h0[k] = hv[k];
      s0[k] = sv[k];
      const uint4 g = gamma_of(k);
      const uint32_t yw[4] = {y0[k].x, y0[k].y, y0[k].z, y0[k].w}, hw[4] = {h0[k].x, h0[k].y, h0[k].z, h0[k].w};
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(bf16lo(yw[e]) * bf16lo(gw[e]), bf16lo(hw[e]), s);
        s = fmaf(bf16hi(yw[e]) * bf16hi(gw[e]), bf16hi(hw[e]), s);
      }
    }
    const float ri = __ldg(r + row);
    if (kAhead) load(row + step);
    // (r^3 would leave fp32 for rows 1e13 away from one: r meets the sum and h first)
    const float coef = -ri * norm8_sum<WARP>(s, red[it]) / static_cast<float>(N) * ri;
    const size_t ro = static_cast<size_t>(row) * N;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int c = (tid + k * nt) * 8;
      const uint4 g = gamma_of(k);
      const uint32_t yw[4] = {y0[k].x, y0[k].y, y0[k].z, y0[k].w}, hw[4] = {h0[k].x, h0[k].y, h0[k].z, h0[k].w};
      const uint32_t sw[4] = {s0[k].x, s0[k].y, s0[k].z, s0[k].w}, gw[4] = {g.x, g.y, g.z, g.w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ya = bf16lo(yw[e]), yb = bf16hi(yw[e]);
        const float ha = bf16lo(hw[e]) * ri, hb = bf16hi(hw[e]) * ri;
        dg[k][2 * e] = fmaf(ya, ha, dg[k][2 * e]);
        dg[k][2 * e + 1] = fmaf(yb, hb, dg[k][2 * e + 1]);
        o[e] = pack_bf16x2(fmaf(ya * ri, bf16lo(gw[e]), fmaf(coef, ha, bf16lo(sw[e]))),
                           fmaf(yb * ri, bf16hi(gw[e]), fmaf(coef, hb, bf16hi(sw[e]))));
      }
      if (c < N) *reinterpret_cast<uint4*>(dx + ro + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (WARP) {
    // the warps' terms, added in order by the first
    __shared__ float terms[MAXT / 32 - 1][8 * kNorm8Vpt][32];
    const int warp = threadIdx.x >> 5;
    if (warp > 0) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) terms[warp - 1][k * 8 + e][tid] = dg[k][e];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < MAXT / 32 - 1; ++w)
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[k][e] += terms[w][k * 8 + e][tid];
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (tid + k * nt) * 8;
    if (c < N) {
      float* o = part + static_cast<size_t>(blockIdx.x) * N + c;
      *reinterpret_cast<float4*>(o) = make_float4(dg[k][0], dg[k][1], dg[k][2], dg[k][3]);
      *reinterpret_cast<float4*>(o + 4) = make_float4(dg[k][4], dg[k][5], dg[k][6], dg[k][7]);
    }
  }
}

// dgamma_j = sum over blocks of part[block][j]: a block takes 32 columns, warp w
// the blocks w, w + 32, ..., whose sums are added in order.
__global__ void __launch_bounds__(1024) norm8_dgamma_kernel(const float* __restrict__ part, int nblk, int N,
                                                           float* __restrict__ dgamma) {
  __shared__ float red[32][33];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (j < N) {
#pragma unroll 8
    for (int b = warp; b < nblk; b += 32) s += part[static_cast<size_t>(b) * N + j];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < N) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += red[w][lane];
    dgamma[j] = t;
  }
}

}  // namespace coda
