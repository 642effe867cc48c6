// Token embedding and its gradient: the input end of the model, before the
// first norm of the GEMM-epilogue chain.
//
//   forward   h_i = s E[t_i];  hg_i = gamma * h_i;  partial[t, i] = sum over the
//             128-column slot t of h_i^2 -- the three tensors the row-scaled
//             GEMMs take, so the first norm needs no pass of its own
//   backward  dE[v] = s sum_{i: t_i = v} dh_i   (fp32, rows in increasing i)
//
// A token outside [0, V) (padding) gives a zero row and no gradient.
// Both are bound by HBM.
#pragma once

#include "../coda_device.cuh"

namespace coda {

__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ forward

// A warp takes 256 columns (8 per lane) of kEmbRows rows: the rows' tokens are
// read first, then all of their table rows are requested before one is used.
// A 128-column slot is half a warp.
constexpr int kEmbRows = 4;
constexpr int kEmbWarps = 8;

__global__ void __launch_bounds__(32 * kEmbWarps) embed_kernel(
    const int64_t* __restrict__ tokens, const __nv_bfloat16* __restrict__ E, float scale,
    const __nv_bfloat16* __restrict__ gamma, __nv_bfloat16* __restrict__ h_out, __nv_bfloat16* __restrict__ hg_out,
    float* __restrict__ partial, int64_t M, int D, int64_t V, int nspan) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kEmbWarps + (threadIdx.x >> 5);
  const int64_t r0 = item / nspan * kEmbRows;
  if (r0 >= M) return;
  const int c0 = static_cast<int>(item % nspan) * 256 + lane * 8;
  const bool in = c0 < D;
  uint4 v[kEmbRows];
  int64_t tok[kEmbRows];
#pragma unroll
  for (int u = 0; u < kEmbRows; ++u) tok[u] = r0 + u < M ? __ldg(tokens + r0 + u) : -1;
#pragma unroll
  for (int u = 0; u < kEmbRows; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    if (in && tok[u] >= 0 && tok[u] < V) v[u] = __ldg(reinterpret_cast<const uint4*>(E + tok[u] * D + c0));
  }
  uint4 g4 = make_uint4(0, 0, 0, 0);
  if (in && hg_out != nullptr) g4 = __ldg(reinterpret_cast<const uint4*>(gamma + c0));
  const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
  for (int u = 0; u < kEmbRows; ++u) {
    if (r0 + u >= M) break;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t oh[4], og[4];
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf16lo(w[e]) * scale, b = bf16hi(w[e]) * scale;
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
      oh[e] = pack_bf16x2(a, b);
      og[e] = pack_bf16x2(a * bf16lo(gw[e]), b * bf16hi(gw[e]));
    }
    if (in) {
      const size_t o = static_cast<size_t>(r0 + u) * D + c0;
      if (h_out != nullptr) *reinterpret_cast<uint4*>(h_out + o) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
      if (hg_out != nullptr) *reinterpret_cast<uint4*>(hg_out + o) = make_uint4(og[0], og[1], og[2], og[3]);
    }
    if (partial != nullptr) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if ((lane & 15) == 0 && in) partial[static_cast<size_t>(c0 >> 7) * M + r0 + u] = ss;
    }
  }
}

// ----------------------------------------------------------------- backward
//
// 1. embed_sort_kernel: the (token, row) pairs in order of token, rows of one
//    token in increasing order (a least-significant-digit radix sort, which is
//    stable), by one cluster of eight CTAs, and a bitmap of the tokens that
//    occur.  The other clusters meanwhile fill the first rows of dE with zeros.
// 2. embed_bwd_kernel: each block takes `chunk` consecutive pairs, whatever
//    their tokens, so a token that fills half of the batch costs no more than
//    distinct ones.  A token's run inside one chunk is summed and written; the
//    sums of a run that crosses a chunk's border go to the workspace.  Other
//    blocks write zeros to dE's remaining rows whose tokens do not occur: they
//    are most of the traffic, and overlap the sums.
// 3. embed_bwd_join_kernel: adds a crossing run's parts in order.
// Every sum has one order, given by the tokens alone: no atomics on values.

constexpr int kSortBits = 9;  // 2 passes for up to 262143 tokens; 512 counters for each of 32 warps: 64 KB
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;
constexpr int kSortSmem = (kSortThreads / 32 * kSortBins + 3 * kSortBins) * 4;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Writes `len` zero bytes (a multiple of 16) to dst as bulk copies of at most
// kZeroPiece from a zeroed shared buffer, by one thread; the copies are left in
// flight (bulk_wait_all before the block ends).
constexpr int kZeroPiece = 16384;

__device__ __forceinline__ void zero_run(uint8_t* dst, size_t len, const void* zeros) {
  for (size_t o = 0; o < len; o += kZeroPiece) {
    const uint32_t n = static_cast<uint32_t>(len - o < kZeroPiece ? len - o : kZeroPiece);
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + o), "r"(smem_u32(zeros)),
                 "r"(n)
                 : "memory");
    bulk_commit();
    bulk_wait_read<8>();
  }
}

__device__ __forceinline__ void zero_buffer(void* buf) {
  for (int i = threadIdx.x; i < kZeroPiece / 16; i += blockDim.x)
    reinterpret_cast<uint4*>(buf)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  __syncthreads();
}

// One launch of clusters of eight.  Cluster 0 sorts into pairs (passes of
// kSortBits bits, ping-pong between buf0 and buf1, the last pass ending in
// `pairs`), clears and fills the bitmap (null: none wanted) and clears the
// count of crossing runs; the others zero the first zero_bytes of dE.  Each warp
// owns a
// contiguous part of the pairs: it counts its digits, the counts are scanned
// over warps, CTAs (through distributed shared memory) and bins, and it places
// its pairs, 32 at a time in order, ranked among equal digits by a match.
__global__ void __cluster_dims__(kSortCluster, 1, 1) __launch_bounds__(kSortThreads)
    embed_sort_kernel(const int64_t* __restrict__ tokens, int M, int64_t V, int passes, int2* buf0, int2* buf1,
                      uint8_t* dE, size_t zero_bytes,
                      uint32_t* bitmap, size_t words, int* crossing) {
  extern __shared__ __align__(16) uint32_t sm[];
  pdl_begin();
  if (blockIdx.x >= kSortCluster) {
    zero_buffer(sm);
    if (threadIdx.x == 0) {
      constexpr size_t kTake = 8 * kZeroPiece;
      for (size_t o = (blockIdx.x - kSortCluster) * kTake; o < zero_bytes; o += (gridDim.x - kSortCluster) * kTake)
        zero_run(dE + o, zero_bytes - o < kTake ? zero_bytes - o : kTake, sm);
      bulk_wait_all<0>();
    }
    return;
  }
  uint32_t* hist = sm;                                      // [32 warps][bins]
  uint32_t* total = sm + kSortThreads / 32 * kSortBins;     // this CTA's count of each bin
  uint32_t* base = total + kSortBins;                       // first place of this CTA's pairs of each bin
  uint32_t* scan = base + kSortBins;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = static_cast<int>(blockIdx.x);
  constexpr int kWarps = kSortThreads / 32 * kSortCluster;
  // 32 pairs, or a multiple, per warp
  const int per = ((M + kWarps - 1) / kWarps + 31) & ~31;
  const int64_t lo64 = static_cast<int64_t>(cta * (kSortThreads / 32) + warp) * per;
  const int lo = static_cast<int>(lo64 < M ? lo64 : M);
  const int hi = static_cast<int>(lo64 + per < M ? lo64 + per : M);
  uint32_t* mine = hist + warp * kSortBins;
  if (cta == 0 && threadIdx.x == 0) *crossing = 0;
  if (bitmap != nullptr) {
    for (size_t i = static_cast<size_t>(cta) * kSortThreads + threadIdx.x; i < words; i += kSortThreads * kSortCluster)
      bitmap[i] = 0;
    cluster_sync_all();
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int2* src = pass & 1 ? buf1 : buf0;
    int2* dst = pass & 1 ? buf0 : buf1;
    const int shift = pass * kSortBits;
    auto get = [&](int i) {
      if (pass > 0) return __ldcg(src + i);
      const int64_t t = __ldg(tokens + i);
      return make_int2(t >= 0 && t < V ? static_cast<int>(t) : static_cast<int>(V), i);  // padding sorts last
    };
    for (int b = lane; b < kSortBins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const bool on = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, on);
      if (on) {
        const int tok = get(i0 + lane).x;
        if (pass == 0 && bitmap != nullptr && tok < V) atomicOr(&bitmap[tok >> 5], 1u << (tok & 31));
        const uint32_t d = (static_cast<uint32_t>(tok) >> shift) & (kSortBins - 1);
        const unsigned same = __match_any_sync(act, d);
        if ((same & ((1u << lane) - 1u)) == 0) mine[d] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    // over the CTA's warps
    if (threadIdx.x < kSortBins) {
      uint32_t s = 0;
      for (int k = 0; k < kSortThreads / 32; ++k) {
        const uint32_t c = hist[k * kSortBins + threadIdx.x];
        hist[k * kSortBins + threadIdx.x] = s;
        s += c;
      }
      total[threadIdx.x] = s;
    }
    cluster_sync_all();
    // over the cluster's CTAs
    uint32_t before = 0, all = 0;
    if (threadIdx.x < kSortBins) {
      const uint32_t a = smem_u32(total + threadIdx.x);
      for (int k = 0; k < kSortCluster; ++k) {
        const uint32_t c = ld_cluster_u32(mapa_shared(a, k));
        before += k < cta ? c : 0u;
        all += c;
      }
      scan[threadIdx.x] = all;
    }
    __syncthreads();
    // over the bins (512: one warp, 16 bins per lane)
    if (warp == 0) {
      uint32_t s = 0, v[kSortBins / 32];
#pragma unroll
      for (int k = 0; k < kSortBins / 32; ++k) {
        v[k] = s;
        s += scan[lane * (kSortBins / 32) + k];
      }
      uint32_t x = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
#pragma unroll
      for (int k = 0; k < kSortBins / 32; ++k) scan[lane * (kSortBins / 32) + k] = v[k] + x - s;
    }
    __syncthreads();
    if (threadIdx.x < kSortBins) base[threadIdx.x] = scan[threadIdx.x] + before;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const bool on = i0 + lane < hi;
      const unsigned act = __ballot_sync(0xffffffffu, on);
      if (on) {
        const int2 e = get(i0 + lane);
        const uint32_t d = (static_cast<uint32_t>(e.x) >> shift) & (kSortBins - 1);
        const unsigned same = __match_any_sync(act, d);
        const uint32_t at = mine[d];
        __syncwarp(act);
        if ((same & ((1u << lane) - 1u)) == 0) mine[d] = at + __popc(same);
        dst[base[d] + at + __popc(same & ((1u << lane) - 1u))] = e;
      }
      __syncwarp();
    }
    cluster_sync_all();  // the pairs are visible to the cluster; `total` may be overwritten
  }
}

// Eight columns of dE[tok]: stored, or added to what is there (x, y); the
// product is rounded by itself, so that what is added is what would be stored.
__device__ __forceinline__ void embed_put(float4* o, const float (&a)[8], float scale, bool add, float4 x, float4 y) {
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = __fmul_rn(scale, a[e]);
  if (add) {
    s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
    s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
  }
  o[0] = make_float4(s[0], s[1], s[2], s[3]);
  o[1] = make_float4(s[4], s[5], s[6], s[7]);
}

constexpr int kEmbBwdThreads = 256;  // 2048 columns, eight per thread
constexpr int kEmbBwdMaxChunk = 1024;
constexpr int kEmbBwdUnroll = 8;  // rows requested together

// Blocks [0, items * spans) sum: chunk block / spans, columns from 2048 * (block
// % spans).  part: [items][2][D] -- a chunk's sum of the run that began before
// it, and of the run that begins in it and goes on after it; the chunks with the
// latter are listed in `list` (in any order).  ACC: the sums are added to dE.
// The other blocks each zero those of 2^unit rows (from zero_row on) that the
// bitmap lacks.
template <bool ACC>
__global__ void __launch_bounds__(kEmbBwdThreads) embed_bwd_kernel(
    const int2* __restrict__ pairs, const __nv_bfloat16* __restrict__ dh, float scale, float* __restrict__ dE,
    float* __restrict__ part, int* __restrict__ list, int* __restrict__ crossing, int M, int64_t V, int D, int chunk,
    int items, int spans, const uint32_t* __restrict__ bitmap, int64_t zero_row, int unit) {
  __shared__ int2 sp[kEmbBwdMaxChunk + 1];
  __shared__ int before;
  pdl_begin();
  if (!ACC && blockIdx.x >= static_cast<unsigned>(items) * spans) {
    const int64_t first = zero_row + (static_cast<int64_t>(blockIdx.x - items * spans) << unit);
    const int rows = static_cast<int>(min(static_cast<int64_t>(1 << unit), V - first));  // all in one word
    uint32_t free = ~(__ldg(bitmap + (first >> 5)) >> (first & 31)) & (rows == 32 ? ~0u : (1u << rows) - 1u);
    while (free != 0) {
      const int r0 = __ffs(free) - 1;
      const uint32_t rest = ~(free >> r0);
      const int n = rest == 0 ? 32 : __ffs(rest) - 1;  // free rows from r0 on
      float4* o = reinterpret_cast<float4*>(dE + (first + r0) * D);
      const size_t len = static_cast<size_t>(n) * D / 4;
#pragma unroll 8
      for (size_t i = threadIdx.x; i < len; i += blockDim.x) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      free = r0 + n >= 32 ? 0u : free & (~0u << (r0 + n));
    }
    return;
  }
  const int item = static_cast<int>(blockIdx.x) / spans, span = static_cast<int>(blockIdx.x) % spans;
  const int64_t p0 = static_cast<int64_t>(item) * chunk;
  const int n = static_cast<int>(M - p0 < chunk ? M - p0 : chunk);
  // (sp[n]: the pair after the chunk)
  for (int i = threadIdx.x; i <= n; i += blockDim.x) sp[i] = p0 + i < M ? pairs[p0 + i] : make_int2(-1, 0);
  if (threadIdx.x == 0) before = p0 > 0 ? pairs[p0 - 1].x : -1;
  __syncthreads();
  if (span == 0 && threadIdx.x == 0 && sp[n].x == sp[n - 1].x && sp[n].x < V && !(before == sp[n].x))
    list[atomicAdd(crossing, 1)] = item;
  const int c0 = (span * kEmbBwdThreads + threadIdx.x) * 8;
  if (c0 >= D) return;
  float a[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = 0.f;
  bool from_before = before == sp[0].x;
  for (int i0 = 0; i0 < n; i0 += kEmbBwdUnroll) {
    uint4 v[kEmbBwdUnroll];
    float4 x[kEmbBwdUnroll], y[kEmbBwdUnroll];  // ACC: dE's row where a run ends
#pragma unroll
    for (int u = 0; u < kEmbBwdUnroll; ++u) {
      const int i = i0 + u;
      if (i >= n || sp[i].x >= V) continue;
      v[u] = __ldcs(reinterpret_cast<const uint4*>(dh + static_cast<size_t>(sp[i].y) * D + c0));
      if (ACC && sp[i + 1].x != sp[i].x) {
        const float4* o = reinterpret_cast<const float4*>(dE + static_cast<size_t>(sp[i].x) * D + c0);
        x[u] = __ldcs(o);
        y[u] = __ldcs(o + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kEmbBwdUnroll; ++u) {
      const int i = i0 + u;
      if (i >= n || sp[i].x >= V) return;  // padding comes last
      const int tok = sp[i].x;
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[2 * e] += bf16lo(w[e]);
        a[2 * e + 1] += bf16hi(w[e]);
      }
      const bool ends = sp[i + 1].x != tok;
      if (!ends && i + 1 < n) continue;
      if (from_before || !ends) {
        float* o = part + (static_cast<size_t>(item) * 2 + (from_before ? 0 : 1)) * D + c0;
        *reinterpret_cast<float4*>(o) = make_float4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(a[4], a[5], a[6], a[7]);
      } else {
        embed_put(reinterpret_cast<float4*>(dE + static_cast<size_t>(tok) * D + c0), a, scale, ACC, x[u], y[u]);
      }
      from_before = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = 0.f;
    }
  }
}

// The runs that cross a chunk's border: the listed chunk i and the parts of the
// run that begins there and goes on after it.  A block takes 256 columns of one
// run at a time.  Eight groups of 32 threads each add a contiguous share of the
// parts, in order; the groups' sums are added in order.
constexpr int kJoinGroups = 8;

__global__ void __launch_bounds__(32 * kJoinGroups) embed_bwd_join_kernel(
    const int2* __restrict__ pairs, const float* __restrict__ part, const int* __restrict__ list,
    const int* __restrict__ crossing, float scale, float* __restrict__ dE, int D, int chunk, int items,
    int accumulate) {
  __shared__ float red[kJoinGroups][32][9];
  pdl_begin();
  const int spans = (D + 255) / 256;
  const int64_t work = static_cast<int64_t>(__ldg(crossing)) * spans;
  const int grp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t t = blockIdx.x; t < work; t += gridDim.x) {
    const int i = __ldg(list + t / spans);
    const int c0 = (static_cast<int>(t % spans) * 32 + lane) * 8;
    const int tok = __ldg(&pairs[static_cast<int64_t>(i + 1) * chunk].x);
    // its other parts are the first of chunks i + 1 .. lo - 1
    int lo = i + 1, hi = items;  // first chunk in (i, items] whose first pair has another token
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(&pairs[static_cast<int64_t>(mid) * chunk].x) == tok)
        lo = mid + 1;
      else
        hi = mid;
    }
    const int n = lo - i;  // parts: chunk i's second, then those
    const int k0 = static_cast<int>(static_cast<int64_t>(n) * grp / kJoinGroups);
    const int k1 = static_cast<int>(static_cast<int64_t>(n) * (grp + 1) / kJoinGroups);
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = 0.f;
    if (c0 < D) {
#pragma unroll 4
      for (int k = k0; k < k1; ++k) {
        const float* s = part + (static_cast<size_t>(i + k) * 2 + (k == 0 ? 1 : 0)) * D + c0;
        const float4 x = *reinterpret_cast<const float4*>(s), y = *reinterpret_cast<const float4*>(s + 4);
        a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
        a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[grp][lane][e] = a[e];
    __syncthreads();
    if (grp == 0 && c0 < D) {
#pragma unroll
      for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += red[g][lane][e];
      float4* o = reinterpret_cast<float4*>(dE + static_cast<size_t>(tok) * D + c0);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (accumulate) x = o[0], y = o[1];
      embed_put(o, a, scale, accumulate != 0, x, y);
    }
    __syncthreads();
  }
}

}  // namespace coda
