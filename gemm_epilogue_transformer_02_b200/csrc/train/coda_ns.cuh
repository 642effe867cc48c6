// Newton-Schulz orthogonalisation of a weight's update, as the Muon optimiser
// does it.  For a matrix G (a gradient or a momentum):
//
//   X_0 = G / (|G|_F + eps)
//   A = X X^T;  B = b A + c A^2;  X <- a X + B X        (steps times)
//
// X keeps G's singular vectors and every step maps a singular value s to
// a s + b s^3 + c s^5, which drives them all towards one.  The Gram matrix is
// taken on the smaller side (a G with more rows than columns uses X^T X and
// X <- a X + X B).
//
// Each step is three tensor-core GEMMs with fused epilogues:
//   gram    acc = X X^T           A = acc, symmetric
//   square  acc = A A             B = b A + c acc, symmetric
//   update  acc = B X (or X B)    X' = a X + acc
//
// Symmetry.  Only the tiles on and below the diagonal of A and B are computed
// and stored (half of the work of those two GEMMs).  A GEMM that needs a block
// above the diagonal loads its mirror image and tells the tensor core that the
// operand is transposed: the K-major and the MN-major form of a 64-wide
// k-block take the same shared memory, so the choice is one tensor map and two
// descriptor fields per k-block.
//
// Precision.  Operands are fp16, not bf16: with |X|_F = 1 every value is
// bounded, so scaled by powers of two they use fp16's 11 bits where bf16 would
// keep 8 (same tensor-core rate).  Sums are fp32.  Two corrections keep the
// roundings off the result where they would grow:
//   - near the end A and B are close to multiples of the identity, and most of
//     their norm is on the diagonal.  What fp16 drops there is kept in fp32
//     (dA, dB: one value per row) and applied by the epilogues:
//     (A + D)^2 = A^2 + D A + A D + D^2, and (B + E) X = B X + E X;
//   - a small singular value grows by up to `a` in every step, and so does what
//     rounding X put there.  X is therefore kept as a high and a low fp16 part;
//     the GEMMs read the high part and the term a X both.  The last step drops
//     the low part: nothing grows after it.
// Against 64 bits this gives 0.5e-3 to 1.4e-3 (relative to |X|_F) for
// Gaussian, correlated and nearly low-rank matrices, where plain bf16 products
// give 0.9e-2 to 3e-1 and fp16 without the two corrections up to 4e-2; the
// bf16 rounding of the output alone is 1.7e-3.
#pragma once

#include <cuda_fp16.h>

#include "../coda_device.cuh"

namespace coda {

// Powers of two the fp16 values are stored with.  Singular values stay below
// 1.3 with the Muon coefficients, so X fits with a factor of 12 to spare and A
// and B with a factor of 37 and 16.
constexpr float kNsScaleX = 4096.f;
constexpr float kNsScaleA = 1024.f;
constexpr float kNsScaleB = 1024.f;

constexpr int kNsThreads = 192;  // TMA producer, MMA issuer, four epilogue warps
constexpr int kNsEpiWarps = 4;
constexpr int kNsStages = 6;
constexpr int kNsOpBytes = 128 * 64 * 2;  // one operand's 128 rows of a 64-wide k-block
constexpr int kNsStageBytes = 2 * kNsOpBytes;
constexpr int kNsEpiBytes = 8192;  // staging per epilogue warp: two 32 x 64 fp16 boxes
constexpr int kNsBars = 2 * kNsStages + 2 + 2 + 1;
constexpr int kNsSmemBytes = 1024 + kNsStages * kNsStageBytes + kNsEpiWarps * kNsEpiBytes + kNsBars * 8 + 16;
static_assert(kNsSmemBytes <= 232448, "shared memory");

enum NsKind : int { kNsGram = 0, kNsSquare, kNsUpdate };

// How an operand's 128 rows (of the output's rows or columns) by 64 k of a
// k-block are found: stored [row, k], stored [k, row], or in a symmetric matrix
// of which the blocks (of `sym_block`) on and below the diagonal are stored.
enum NsMajor : int { kNsK = 0, kNsMN, kNsSym };

struct NsOperand {
  CUtensorMap k;   // [batch, row, k], box 128 rows x 64 k
  CUtensorMap mn;  // [batch, k, row], box 64 k x 64 rows
  int major;
};

struct NsParams {
  NsOperand P, Q;          // acc[i, j] = sum_k P[i, k] Q[j, k]
  CUtensorMap out0, out1;  // stores, box 32 rows x 64 columns: result (high part), low part
  const __half* in0;       // epilogue input of the output's shape: A (square), X high (update)
  const __half* in1;       // X low (update), or null
  const float* d_in;       // dA [batch, rows] (square), dB (update)
  float* d_out;            // dA (gram), dB (square): what fp16 drops of the diagonal
  int rows, cols, K, batch;
  int n_rt, n_ct, tiles;   // row tiles, column tiles, tiles of one matrix
  int sym_block;
  int tall;                // update: X B (dB goes with the columns)
  int last;                // update: the result is the bf16 output
  int has_low;             // update: the result's low part is stored
  float a, b, c;           // coefficients
  uint64_t wait_ns;
};

// 3-D tiled copies (x, y, batch).
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* m, uint32_t bar_cluster_addr,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* smem_src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Instruction descriptor of kind::f16 with fp16 A and B (format code 0) and
// fp32 D; fields as in idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Whether the k-block at k0 of an operand's rows at row0 is loaded [k, row].
__device__ __forceinline__ bool ns_is_mn(int major, int row0, int k0, int sym_block) {
  return major == kNsMN || (major == kNsSym && k0 / sym_block > row0 / sym_block);
}

// Unit u -> matrix, row tile, column tile.  A symmetric result takes the tiles
// on and below the diagonal, row by row: row i starts at tile i (i + 1) / 2.
template <bool SYM>
__device__ __forceinline__ void ns_map(const NsParams& p, int u, int& bz, int& rt, int& ct) {
  bz = u / p.tiles;
  const int t = u - bz * p.tiles;
  if (SYM) {
    int i = static_cast<int>((sqrtf(8.f * static_cast<float>(t) + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    rt = i;
    ct = t - i * (i + 1) / 2;
  } else if (p.n_rt <= p.n_ct) {  // the tiles that share the longer side's operand follow each other
    ct = t / p.n_rt;
    rt = t - ct * p.n_rt;
  } else {
    rt = t / p.n_ct;
    ct = t - rt * p.n_ct;
  }
}

// PAIR: a cluster of two CTAs per 256 x 256 tile (cta_group::2, rank r owns
// accumulator rows [128 r, 128 r + 128) and loads those rows of P and its half
// of Q's); otherwise one CTA per 128 x 128 tile.
template <int KIND, bool PAIR>
__global__ void __launch_bounds__(kNsThreads, 1) ns_gemm_kernel(const __grid_constant__ NsParams p) {
  constexpr int kTile = PAIR ? 256 : 128;
  constexpr bool kSymOut = KIND != kNsUpdate;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sEpi = smem + kNsStages * kNsStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + kNsEpiWarps * kNsEpiBytes);
  uint64_t* empty = full + kNsStages;
  uint64_t* tfull = empty + kNsStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int step = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  const int first = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int nunits = p.tiles * p.batch;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 2 * kNsEpiWarps : kNsEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_holder, 2 * kTile);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 2 * kTile);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const WaitCtx w{abort_flag, p.wait_ns};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nkb = (p.K + 63) / 64;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full), 0) : 0u;
      for (int u = first; ok && u < nunits; u += step) {
        int bz, rt, ct;
        ns_map<kSymOut>(p, u, bz, rt, ct);
        const int row0 = rt * kTile + rank * 128;
        const int col0 = ct * kTile + rank * 128;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, w)) {
            ok = false;
            break;
          }
          if (!PAIR || rank == 0) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * kNsStageBytes);
          uint8_t* dst = smem + stage * kNsStageBytes;
          const uint32_t fb = full0 + stage * 8;
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const NsOperand& op = o == 0 ? p.P : p.Q;
            const int r0 = o == 0 ? row0 : col0;
            uint8_t* d = dst + o * kNsOpBytes;
            if (!ns_is_mn(op.major, r0, kb * 64, p.sym_block)) {
              if (PAIR)
                tma_load_3d_pair(d, &op.k, fb, kb * 64, r0, bz);
              else
                tma_load_3d(d, &op.k, &full[stage], kb * 64, r0, bz);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (PAIR)
                  tma_load_3d_pair(d + j * 8192, &op.mn, fb, r0 + j * 64, kb * 64, bz);
                else
                  tma_load_3d(d + j * 8192, &op.mn, &full[stage], r0 + j * 64, kb * 64, bz);
              }
            }
          }
          ++issued;
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy must have landed before shared memory goes away: the MMA's
      // release of a stage follows its copies.
      const long n = issued < kNsStages ? issued : kNsStages;
      for (long i = 0; i < n; ++i) {
        if (stage == 0) {
          stage = kNsStages - 1;
          phase ^= 1u;
        } else {
          --stage;
        }
        int no_abort = 0;
        (void)mbar_wait(PAIR ? &empty[stage] : &full[stage], phase, WaitCtx{&no_abort, p.wait_ns});
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int u = first; ok && u < nunits; u += step, ++it) {
        int bz, rt, ct;
        ns_map<kSymOut>(p, u, bz, rt, ct);
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, w)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kTile;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool pm = ns_is_mn(p.P.major, rt * kTile, kb * 64, p.sym_block);
          const bool qm = ns_is_mn(p.Q.major, ct * kTile, kb * 64, p.sym_block);
          const uint32_t idesc = idesc_f16_f32(kTile, kTile, pm, qm);
          const uint32_t a0 = smem_u32(smem + stage * kNsStageBytes);
          const uint32_t b0 = a0 + kNsOpBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = pm ? sdesc_sw128(a0 + kk * 2048, 8192, 1024) : sdesc_sw128(a0 + kk * 32, 16, 1024);
            const uint64_t bd = qm ? sdesc_sw128(b0 + kk * 2048, 8192, 1024) : sdesc_sw128(b0 + kk * 32, 16, 1024);
            const uint32_t accum = (kb | kk) ? 1u : 0u;
            // (the kind::f16 instruction; the descriptor says fp16 operands)
            if (PAIR)
              tc_mma_bf16_pair(d, ad, bd, idesc, accum);
            else
              tc_mma_bf16(d, ad, bd, idesc, accum);
          }
          if (PAIR)
            tc_commit_pair_mc(&empty[stage], 0x3);
          else
            tc_commit(&empty[stage]);
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (PAIR)
          tc_commit_pair_mc(&tfull[acc], 0x3);
        else
          tc_commit(&tfull[acc]);
      }
      if (PAIR)
        tc_commit_pair(drain);
      else
        tc_commit(drain);
      int no_abort = 0;
      (void)mbar_wait(drain, 0, WaitCtx{&no_abort, p.wait_ns});
    }
  } else {
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    uint8_t* stg = sEpi + (warp - 2) * kNsEpiBytes;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    uint32_t cnt = 0;
    int it = 0;
    for (int u = first; u < nunits; u += step, ++it) {
      int bz, rt, ct;
      ns_map<kSymOut>(p, u, bz, rt, ct);
      const int acc = it & 1;
      const int row0 = rt * kTile + rank * 128 + q * 32;
      const int row = row0 + lane;
      const int col0 = ct * kTile;
      const bool live = row < p.rows;
      const size_t base = (static_cast<size_t>(bz) * p.rows + (live ? row : 0)) * p.cols;
      const float* dv = KIND == kNsGram ? nullptr : p.d_in + static_cast<size_t>(bz) * (KIND == kNsUpdate && p.tall ? p.cols : p.rows);
      const bool by_col = KIND == kNsSquare || (KIND == kNsUpdate && p.tall);
      float di = 0.f;
      if (KIND == kNsSquare || (KIND == kNsUpdate && !p.tall)) di = live ? __ldg(dv + row) : 0.f;
      int nch = (p.cols - col0 + 63) / 64;
      if (nch > kTile / 64) nch = kTile / 64;
      if (row0 >= p.rows) nch = 0;  // (uniform over the warp)
      uint4 x0[4], x1[4];
      auto fetch = [&](int col) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x0[j] = make_uint4(0, 0, 0, 0);
          x1[j] = make_uint4(0, 0, 0, 0);
          if (KIND != kNsGram && live && col + j * 8 < p.cols) {
            x0[j] = *reinterpret_cast<const uint4*>(p.in0 + base + col + j * 8);
            if (KIND == kNsUpdate && p.in1 != nullptr)
              x1[j] = *reinterpret_cast<const uint4*>(p.in1 + base + col + j * 8);
          }
        }
      };
      if (nch > 0) fetch(col0);
      // Warp-uniform outcome: tcgen05.ld below is a warp-collective instruction.
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (it >> 1) & 1, w))) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kTile;
      for (int ch = 0; ch < nch; ++ch) {
        const int cc = col0 + ch * 64;
        uint8_t* S0 = KIND == kNsUpdate ? stg : stg + (cnt & 1) * 4096;
        uint8_t* S1 = stg + 4096;
        if (lane == 0) {
          if (KIND == kNsUpdate)
            bulk_wait_read<0>();
          else
            bulk_wait_read<1>();
        }
        __syncwarp();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int c32 = cc + hh * 32;
          uint4 y0[4], y1[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y0[j] = x0[j];
            y1[j] = x1[j];
          }
          if (hh == 0 || ch + 1 < nch) fetch(c32 + 32);
          uint32_t v[32];
          tmem_ld32(taddr + ch * 64 + hh * 32, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w0[4] = {y0[j].x, y0[j].y, y0[j].z, y0[j].w};
            const uint32_t w1[4] = {y1[j].x, y1[j].y, y1[j].z, y1[j].w};
            float dj[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (by_col && c32 + j * 8 < p.cols) {
              const float4 lo = __ldg(reinterpret_cast<const float4*>(dv + c32 + j * 8));
              const float4 hi = __ldg(reinterpret_cast<const float4*>(dv + c32 + j * 8 + 4));
              dj[0] = lo.x, dj[1] = lo.y, dj[2] = lo.z, dj[3] = lo.w;
              dj[4] = hi.x, dj[5] = hi.y, dj[6] = hi.z, dj[7] = hi.w;
            }
            uint32_t o0[4], o1[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float r[2];
              const float2 in = unpack_f16x2(w0[e]);
              const float2 inl = unpack_f16x2(w1[e]);
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int col = c32 + j * 8 + 2 * e + t;
                const float ac = __uint_as_float(v[j * 8 + 2 * e + t]);
                const float i0 = t ? in.y : in.x;
                const float d = dj[2 * e + t];
                if (KIND == kNsGram) {
                  r[t] = ac * (kNsScaleA / (kNsScaleX * kNsScaleX));
                } else if (KIND == kNsSquare) {
                  // true values: A_ij = i0 / S_A, (A^2)_ij = ac / S_A^2 + (d_i + d_j) A_ij
                  float sq = fmaf(di + d, i0 * (1.f / kNsScaleA), ac * (1.f / (kNsScaleA * kNsScaleA)));
                  float lin = i0 * (1.f / kNsScaleA);
                  if (rt == ct && col == row) {
                    sq = fmaf(d, d, sq);
                    lin += d;
                  }
                  r[t] = fmaf(p.c, sq, p.b * lin) * kNsScaleB;
                } else {
                  const float x = i0 + (t ? inl.y : inl.x);
                  r[t] = fmaf(p.a, x, fmaf(p.tall ? d : di, x, ac * (1.f / kNsScaleB)));
                }
                if (KIND != kNsUpdate && rt == ct && col == row && live)
                  p.d_out[static_cast<size_t>(bz) * p.rows + row] =
                      (r[t] - __half2float(__float2half_rn(r[t]))) *
                      (KIND == kNsGram ? 1.f / kNsScaleA : 1.f / kNsScaleB);
              }
              if (KIND == kNsUpdate && p.last) {
                o0[e] = pack_bf16x2(r[0] * (1.f / kNsScaleX), r[1] * (1.f / kNsScaleX));
                o1[e] = 0;
              } else {
                o0[e] = pack_f16x2(r[0], r[1]);
                const float2 h = unpack_f16x2(o0[e]);
                o1[e] = KIND == kNsUpdate ? pack_f16x2(r[0] - h.x, r[1] - h.y) : 0u;
              }
            }
            st_shared_v4(S0 + sw128_off(lane, hh * 4 + j), make_uint4(o0[0], o0[1], o0[2], o0[3]));
            if (KIND == kNsUpdate && p.has_low)
              st_shared_v4(S1 + sw128_off(lane, hh * 4 + j), make_uint4(o1[0], o1[1], o1[2], o1[3]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&p.out0, S0, cc, row0, bz);
          if (KIND == kNsUpdate && p.has_low) tma_store_3d(&p.out1, S1, cc, row0, bz);
          bulk_commit();
        }
        ++cnt;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_cluster(tempty0 + acc * 8);
        else
          mbar_arrive(&tempty[acc]);
      }
    }
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, 2 * kTile);
    else
      tmem_dealloc(tmem_base, 2 * kTile);
  }
}

// ------------------------------------------------------------ |G|_F and X_0

// Sums of squares of a matrix's parts in 64 bits (an fp32 sum would overflow
// or vanish for entries beyond 1e19 or below 1e-22): block (i, bz) takes
// 8-element groups i * 256 + thread, + 256 * nblk, ... of matrix bz.
constexpr int kNsNormThreads = 256;

__device__ __forceinline__ double ns_block_sum(double s, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int i = 0; i < kNsNormThreads / 32; ++i) s += red[i];
  return s;
}

__global__ void __launch_bounds__(kNsNormThreads) ns_sumsq_kernel(const float* __restrict__ G, size_t n8, int nblk,
                                                                 double* __restrict__ part) {
  __shared__ double red[kNsNormThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float4* g = reinterpret_cast<const float4*>(G) + static_cast<size_t>(blockIdx.y) * n8 * 2;
  double s = 0.0;
  for (size_t i = blockIdx.x * static_cast<size_t>(kNsNormThreads) + threadIdx.x; i < n8;
       i += static_cast<size_t>(nblk) * kNsNormThreads) {
    const float4 a = __ldg(g + 2 * i), b = __ldg(g + 2 * i + 1);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), s);
  }
  s = ns_block_sum(s, red);
  if (threadIdx.x == 0) part[static_cast<size_t>(blockIdx.y) * nblk + blockIdx.x] = s;
}

// X_0 = G / (|G|_F + eps), times the stored scale, as high and low fp16 parts.
// The factor goes on in two steps so that it may pass fp32's range (a G of
// 1e-30 with eps 0).
__global__ void __launch_bounds__(kNsNormThreads) ns_scale_kernel(const float* __restrict__ G, size_t n8, int nblk,
                                                                 const double* __restrict__ part, double eps,
                                                                 __half* __restrict__ hi, __half* __restrict__ lo) {
  __shared__ double red[kNsNormThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s = 0.0;
  for (int i = threadIdx.x; i < nblk; i += kNsNormThreads) s += part[static_cast<size_t>(blockIdx.y) * nblk + i];
  s = ns_block_sum(s, red);
  const double f = static_cast<double>(kNsScaleX) / (sqrt(s) + eps);
  const float f1 = f > 1e20 ? 1.8446744073709552e19f : (f < 1e-20 ? 5.421010862427522e-20f : 1.f);  // 2^64, 2^-64
  const float f2 = static_cast<float>(f / static_cast<double>(f1));
  const size_t off = static_cast<size_t>(blockIdx.y) * n8;
  const float4* g = reinterpret_cast<const float4*>(G) + off * 2;
  for (size_t i = blockIdx.x * static_cast<size_t>(kNsNormThreads) + threadIdx.x; i < n8;
       i += static_cast<size_t>(gridDim.x) * kNsNormThreads) {
    const float4 a = __ldg(g + 2 * i), b = __ldg(g + 2 * i + 1);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = v[2 * e] * f1 * f2, x1 = v[2 * e + 1] * f1 * f2;
      h[e] = pack_f16x2(x0, x1);
      const float2 hf = unpack_f16x2(h[e]);
      l[e] = pack_f16x2(x0 - hf.x, x1 - hf.y);
    }
    reinterpret_cast<uint4*>(hi)[off + i] = make_uint4(h[0], h[1], h[2], h[3]);
    if (lo != nullptr) reinterpret_cast<uint4*>(lo)[off + i] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

}  // namespace coda
