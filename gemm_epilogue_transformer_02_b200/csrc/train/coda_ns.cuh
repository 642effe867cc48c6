// Newton-Schulz orthogonalisation of a weight's update, as the Muon optimiser
// does it.  For a matrix G (a gradient or a momentum):
//
//   X_0 = G / (|G|_F + eps)
//   A = X X^T;  P = a I + b A + c A^2;  X <- P X        (steps times)
//
// X keeps G's singular vectors and every step maps a singular value s to
// a s + b s^3 + c s^5, which drives them all towards one.  The Gram matrix is
// taken on the smaller side (a G with more rows than columns uses X^T X and
// X <- X P).  Everything is a tensor-core GEMM with a fused epilogue:
//   gram    A = X X^T                      symmetric
//   square  P = a I + b A + c (A A)        symmetric
//   update  X' = P X (or X P)
//
// Symmetry.  Only the tiles on and below the diagonal of a symmetric result are
// computed and stored (half of the work).  A GEMM that needs a block above the
// diagonal loads its mirror image and tells the tensor core that the operand is
// transposed: the K-major and the MN-major form of a 64-wide k-block take the
// same shared memory, so the choice is one tensor map and two descriptor fields
// per k-block.
//
// Every step forms A from X anew.  Several steps on the small side alone (A' =
// P A P, X' = P' P X: all of them are polynomials of the first A) would save
// s^2 l operations each, but A's rounding, relative to its large entries, then
// stands for the small directions' share of the next steps: with one direction
// in G and noise of 3e-4 beside it five steps as 3 + 2 ended 5e-2 of |X|_F off
// (512 x 1024), 2 + 2 + 1 1e-2, a pair of steps at the end alone 4e-3, and
// single ones 0.9e-3.
//
// Precision.  Operands are fp16, not bf16: with |X|_F = 1 every value is
// bounded, so scaled by powers of two they use fp16's 11 bits where bf16 would
// keep 8 (same tensor-core rate).  Sums are fp32.  Two corrections keep the
// roundings off the result where they would grow:
//   - near the end A and P are close to multiples of the identity, and most of
//     their norm is on the diagonal.  What fp16 drops there (d) is kept in fp32
//     beside the rounded diagonal (f) and applied by the epilogues: a product's
//     diagonal gets d1 f2 + f1 d2 + d1 d2 (off the diagonal that is as small as
//     the rounding of the other entries), and X' = P X + d X;
//   - a small singular value grows by up to `a` in every step, and so does what
//     rounding X put there.  X is therefore kept as a high and a low fp16 part;
//     the GEMMs read the high part, and the diagonal of P (all of P where X is
//     small) multiplies the low part too.  The last update drops it.
// Against 64 bits this gives 0.2e-3 to 1.1e-3 of |X|_F for Gaussian and
// correlated matrices after five steps (sides of 64 and more).  Where a few
// directions hold the norm the others lie in the low part, which sees only P's
// diagonal, and the entries of P beside it, of 2.7 / s for one direction, are
// what is left out: with the smaller side s up to 1.5e-3 + 0.65 / s.  Plain bf16
// products give 0.9e-2 and 3e-1.  The bf16 rounding of the output alone is
// 1.7e-3.
#pragma once

#include <cuda_fp16.h>

#include "../coda_device.cuh"

namespace coda {

// Powers of two the fp16 values are stored with.  With the Muon coefficients
// singular values stay below 1.3 and P below 3.5, so X fits with a factor of 12
// to spare, A with 37, P with 73.
constexpr float kNsScaleX = 4096.f;
constexpr float kNsScaleA = 1024.f;
constexpr float kNsScaleP = 256.f;

constexpr int kNsEpiWarps = 8;                     // two per TMEM lane quarter, each half of a tile's columns
// Warps: loads of the left operand, MMA issue, epilogue, loads of the right
// operand.  One thread takes 140 to 220 cycles to issue a copy, and with both
// operands' 350 and its loop as long as a k-block's MMAs.
constexpr int kNsThreads = 96 + 32 * kNsEpiWarps;
constexpr int kNsRightWarp = 2 + kNsEpiWarps;
// The loads of a unit are at most this many units ahead of its epilogue (eight
// stages of one k-block each, and two accumulators).
constexpr int kNsAhead = 16;
constexpr int kNsBoxBytes = 32 * 32 * 2;  // a 32 x 32 box of an epilogue
constexpr uint64_t kNsDrainNs = 10000000;  // 10 ms: copies land within microseconds

// A tile's shape and what a CTA keeps for it in shared memory.  N = 256: a
// cluster of two CTAs per 256 x 256 tile (cta_group::2; rank r owns accumulator
// rows [128 r, 128 r + 128) and loads those rows of the left operand and its
// half of the right one's).  N = 128, 64: one CTA per 128 x N tile.  A 128 x 64
// tile gives each epilogue warp one block, and eight stages hold a K of 512 at
// once; it is for matrices whose tiles would leave most SMs idle.
template <int N>
struct NsTile {
  static constexpr bool kPair = N == 256;
  static constexpr int kM = kPair ? 256 : 128;
  static constexpr int kN = N;
  static constexpr int kStages = N == 64 ? 8 : 5;
  static constexpr int kRight = kPair ? 128 : N;                       // rows of the right operand a CTA loads
  static constexpr int kLeftBytes = 128 * 64 * 2;                      // of a 64-wide k-block
  static constexpr int kStageBytes = kLeftBytes + kRight * 64 * 2;
  static constexpr int kHalf = N / 2;                                  // columns of an epilogue warp
  static constexpr int kBlks = kHalf / 32;                             // blocks of 32 columns
  static constexpr int kBufs = kBlks > 1 ? 2 : 1;                      // its staging buffers: a high and a low box
  static constexpr int kEpiBytes = kBufs * 2 * kNsBoxBytes;
  static constexpr int kWarps = (kPair ? 2 : 1) * kNsEpiWarps;         // epilogue warps of a tile
  static constexpr int kBars = 2 * kStages + 2 + 2 + 1 + kNsAhead + 2 * kNsEpiWarps;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kNsEpiWarps * kEpiBytes + kBars * 8 + kNsAhead * 4 + 32;
  static_assert(kSmem <= 232448, "shared memory");
};

// The three phases of a step.
enum NsKind : int { kNsGram = 0, kNsSquare, kNsUpdate, kNsKinds };

// One GEMM's tiles, acc[i, j] = sum_k P[i, k] Q[j, k], over the batch.
struct NsGeo {
  int rows, cols, nkb;    // output size of one matrix, 64-wide k-blocks
  int n_rt, n_ct, tiles;  // row tiles, column tiles, tiles of one matrix (half of them for a symmetric result)
  int whole;              // the first `whole` tiles are one unit each,
  int rest;               // the other `rest` tiles
  int splits;             // are `splits` units each, over equal shares of the k-blocks
  int arrivals;           // at each matrix's counter in one such phase
};

// The symmetric matrices.
enum NsBuf : int { kBufA = 0, kBufP, kBufs };

// The loads of one matrix [batch, y, x], with 64-wide k-blocks.  A K-major
// operand's 128 rows come as one copy: a single thread issues them, and at the
// start of a GEMM the first MMAs wait for that (as two copies 5 to 7 % more time;
// an MN-major operand's 128 rows as one 4-D copy took longer than as two).
struct NsMaps {
  CUtensorMap k128;  // K-major: 128 rows (y) x 64 k (x)
  CUtensorMap b64;   // 64 x 64, of either form
};

struct NsParams {
  NsMaps X[2];  // X's high part, by the step's parity
  NsMaps S[kBufs];
  // the epilogues' boxes of 32 x 32 (64-byte swizzle): X's high and low parts, the symmetric matrices, the output
  CUtensorMap Hbox[2], Lbox[2], Sbox[kBufs], Obox;
  float2* diag[kBufs];  // [batch, s]: (d, f): what fp16 drops of the diagonal, and the rounded diagonal
  float* part;          // partial accumulators of the split tiles
  int* counters;        // [batch]: arrivals of finished units: of each matrix (if few), or of all at the first;
                        // then for each kind of phase those of the split tiles' parts
  NsGeo geo[kNsKinds];
  int batch, steps, tall;
  int few;              // a unit waits for its own matrix (else for all of them)
  float a, b, c;
  uint64_t wait_ns;
};

// Walks the phases; every role of every CTA takes the same ones.  A matrix's
// phase begins when its last one is complete.
struct NsSeq {
  int kind = -1;
  int step = 0;       // X of this step is in buffer step & 1
  unsigned done = 0;  // arrivals of a matrix's units in the phases before this one
  __device__ __forceinline__ bool next(const NsParams& p) {
    if (kind >= 0) done += static_cast<unsigned>(p.geo[kind].arrivals);
    if (++kind == kNsKinds) {
      kind = 0;
      ++step;
    }
    return step < p.steps;
  }
  __device__ __forceinline__ bool first() const { return step == 0 && kind == 0; }
};

// 3-D tiled copies (x, y, batch).  PAIR: the barrier may be the other CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const CUtensorMap* m, uint32_t bar, int c0, int c1,
                                            int c2) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
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

// Two fp32 values in a 64-bit register pair: one instruction for both.
__device__ __forceinline__ uint64_t f2_bits(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t f2_set(float x, float y) { return f2_bits(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ float2 f2_get(uint64_t v) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ uint64_t f2_half(uint32_t h) {  // two fp16 values
  const float2 f = unpack_f16x2(h);
  return f2_set(f.x, f.y);
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) { return f2_fma(b, f2_set(-1.f, -1.f), a); }

// Wait (bounded) until *addr has reached target (both count modulo 2^32), polling without a pause: few threads
// wait, and each poll takes a trip to L2.
__device__ __noinline__ bool ns_count_wait(const int* addr, unsigned target, const WaitCtx& w) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (static_cast<int>(static_cast<unsigned>(ld_acquire(addr)) - target) >= 0) return true;
    if ((i & 63u) == 0) {
      if (*w.abort_flag) return false;
      if (globaltimer_ns() - t0 > w.limit_ns) {
        *w.abort_flag = 1;
        atomicCAS(&g_coda_status, 0, kDevTimeout);
        return false;
      }
    }
  }
}

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Adds to a counter in shared memory and returns its old value; orders this
// thread's accesses with those of the CTA's other threads that add to it.
__device__ __forceinline__ int add_acq_rel_cta(int* addr, int v) {
  int old;
  asm volatile("atom.acq_rel.cta.shared::cta.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(addr)), "r"(v) : "memory");
  return old;
}

// A unit of work: a tile (matrix, row tile, column tile) and its k-blocks.
struct NsUnit {
  int bz, rt, ct;
  int kb0, kb1;
  int part;   // which of a split tile's parts (-1: a whole tile)
  int split;  // the split tile's number
  int weight;  // of its arrival: those of one tile make `splits`
};

// A symmetric result takes the square blocks on and below the diagonal, row by
// row (row i starts at block i (i + 1) / 2), each of kM / kN tiles.  Otherwise the tiles that share the longer
// side's operand follow each other.
template <bool SYM, class T>
__device__ __forceinline__ NsUnit ns_unit_of(const NsGeo& g, int u) {
  NsUnit n;
  int t = u;
  n.part = -1;
  n.split = 0;
  n.weight = g.splits;
  n.kb0 = 0;
  n.kb1 = g.nkb;
  if (u >= g.whole) {
    n.split = (u - g.whole) / g.splits;
    const int k = (u - g.whole) - n.split * g.splits;
    t = g.whole + n.split;
    if (g.splits > 1) {
      n.part = k;
      n.weight = 1;
      n.kb0 = g.nkb * k / g.splits;
      n.kb1 = g.nkb * (k + 1) / g.splits;
    }
  }
  n.bz = t / g.tiles;
  t -= n.bz * g.tiles;
  if (SYM) {
    constexpr int kParts = T::kM / T::kN;
    const int part = t % kParts;
    t /= kParts;
    int i = static_cast<int>((sqrtf(8.f * static_cast<float>(t) + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    n.rt = i;
    n.ct = (t - i * (i + 1) / 2) * kParts + part;
  } else if (g.n_rt <= g.n_ct) {
    n.ct = t / g.n_rt;
    n.rt = t - n.ct * g.n_rt;
  } else {
    n.rt = t / g.n_ct;
    n.ct = t - n.rt * g.n_ct;
  }
  return n;
}

template <class T>
__device__ __forceinline__ NsUnit ns_unit(const NsParams& p, const NsSeq& s, int u) {
  const NsGeo& g = p.geo[s.kind];
  return s.kind == kNsUpdate ? ns_unit_of<false, T>(g, u) : ns_unit_of<true, T>(g, u);
}

__device__ __forceinline__ int ns_units(const NsParams& p, const NsSeq& s) {
  const NsGeo& g = p.geo[s.kind];
  return g.whole + g.rest * g.splits;
}

// What unit n has to wait for that the CTA's last one of the phase (waited: -1 for
// the first) did not: a matrix, all of them (p.batch), or nothing (-1).
__device__ __forceinline__ int ns_need(const NsParams& p, const NsSeq& s, const NsUnit& n, int& waited) {
  const int need = p.few && n.part < 0 ? n.bz : p.batch;
  if (s.first() || need == waited || waited == p.batch) return -1;
  waited = need;
  return need;
}

// An operand of one GEMM.  Of a symmetric matrix the blocks of M x M on and below
// the diagonal are stored: of a tile's rows (the first is `row`) the k-blocks
// from first_mn on lie above it and are loaded [k, row] (MN-major).
enum NsMajor : int { kNsK = 0, kNsMN, kNsSym };
struct NsOperand {
  const NsMaps* maps;
  int major;
  template <int M>
  __device__ __forceinline__ int first_mn(int row) const {
    return major == kNsMN ? 0 : (major == kNsK ? 1 << 30 : (row / M + 1) * (M / 64));
  }
};

__device__ __forceinline__ void ns_operands(const NsParams& p, const NsSeq& s, NsOperand& P, NsOperand& Q) {
  const NsMaps* x = &p.X[s.step & 1];
  if (s.kind == kNsGram) {
    P = Q = NsOperand{x, p.tall ? kNsMN : kNsK};
  } else if (s.kind == kNsSquare) {
    P = Q = NsOperand{&p.S[kBufA], kNsSym};
  } else {
    const NsOperand sp{&p.S[kBufP], kNsSym};
    P = p.tall ? NsOperand{x, kNsK} : sp;
    Q = p.tall ? sp : NsOperand{x, kNsMN};
  }
}

// An operand's `ROWS` rows at r0 of one k-block, to shared memory (addresses as
// the instruction takes them: the loop that issues these is as long as a
// k-block's MMAs on small tiles).
template <int ROWS, bool PAIR>
__device__ __forceinline__ void ns_load(uint32_t dst, const NsMaps* maps, bool mn, int r0, int k0, int bz,
                                        uint32_t bar) {
  if (!mn) {
    tma_load_3d<PAIR>(dst, ROWS == 128 ? &maps->k128 : &maps->b64, bar, k0, r0, bz);
  } else {
#pragma unroll
    for (int j = 0; j < ROWS / 64; ++j) tma_load_3d<PAIR>(dst + j * 8192, &maps->b64, bar, r0 + j * 64, k0, bz);
  }
}

// Byte offset of 16-byte chunk `chunk` (0..3) of row `row` in a box of 64-byte
// rows with the 64-byte swizzle (base aligned to 512 bytes).
__device__ __forceinline__ uint32_t sw64_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

constexpr int kNsSplitCounters = 37 * 16;  // of one GEMM: split tiles (at most half of the slots) x warps

// What an epilogue warp keeps.
struct NsEpi {
  uint8_t* stg;       // its two buffers
  uint64_t* bars;     // a barrier for each, for the loads
  uint32_t taddr;     // TMEM address of its lanes, first accumulator
  int rank, q, half;  // CTA of the pair, lane quarter, half of the columns
  int lane;
  uint32_t cnt;       // blocks done: block i uses buffer i & 1
  uint32_t loads;     // bit i: parity of buffer i's next load
  uint32_t flying;    // bit i: buffer i's load has not been waited for
};

// v[4 j ..] += o
__device__ __forceinline__ void ns_add4(uint32_t (&v)[32], int j, const float4& o) {
  v[4 * j] = __float_as_uint(__uint_as_float(v[4 * j]) + o.x);
  v[4 * j + 1] = __float_as_uint(__uint_as_float(v[4 * j + 1]) + o.y);
  v[4 * j + 2] = __float_as_uint(__uint_as_float(v[4 * j + 2]) + o.z);
  v[4 * j + 3] = __float_as_uint(__uint_as_float(v[4 * j + 3]) + o.w);
}

// One unit's epilogue for one warp: 32 rows x half of the tile's columns, in
// blocks of 32 columns (a thread has one row).  A block's inputs come by TMA
// into a staging buffer, one block ahead (the first one's during the main
// loop); the thread replaces its row by the results, which leave by TMA from the
// same buffer.  (Direct loads of a row per thread touch 32 lines an instruction
// and bound the update at 20 us a tile.)  Sixteen warps with a quarter of the
// columns each, or tensor-memory loads of 8 columns in a small loop, were
// slower.  Returns false if a wait gave up.
template <int KIND, class T>
__device__ __forceinline__ bool ns_epilogue(const NsParams& p, int step, const NsUnit& n, int acc, uint32_t parity,
                                            uint64_t* tfull, NsEpi& e, const WaitCtx& w) {
  constexpr int kHalf = T::kHalf;
  constexpr int kBlks = T::kBlks;
  const NsGeo& g = p.geo[KIND];
  constexpr int kOut = KIND == kNsGram ? kBufA : kBufP;  // (of a symmetric result)
  const int par = step & 1;
  const bool last = step == p.steps - 1;
  const bool in_low = KIND == kNsUpdate && (!last || step == 0);  // X has a low part
  const bool has_low = KIND == kNsUpdate && step < p.steps - 2;   // the next step reads one
  const CUtensorMap* in0 = KIND == kNsSquare ? &p.Sbox[kBufA] : &p.Hbox[par];
  const CUtensorMap* in1 = &p.Lbox[par];
  const int lane = e.lane;
  const int row0 = n.rt * T::kM + e.rank * 128 + e.q * 32;
  const int row = row0 + lane;
  const int col0 = n.ct * T::kN + e.half * kHalf;
  const bool live = row < g.rows;
  // The diagonal of P: of the row of P X, of the column of X P.  Written by
  // other CTAs of this launch: read through L2.
  const bool by_col = KIND == kNsUpdate && p.tall;
  const float2* dv = p.diag[kBufP] + static_cast<size_t>(n.bz) * (by_col ? g.cols : g.rows);
  float2 di = make_float2(0.f, 0.f);  // (d, f + d) of the row
  if (KIND == kNsUpdate && !by_col && live) {
    di = __ldcg(dv + row);
    di.y += di.x;
  }
  int nblk = (g.cols - col0 + 31) / 32;
  if (nblk > kBlks) nblk = kBlks;
  if (row0 >= g.rows || nblk < 0) nblk = 0;  // (uniform over the warp)
  // the blocks this warp finishes: all, or of a split tile this part's share
  int b0 = 0, b1 = nblk;
  if (kBlks > 1 && n.part >= 0) {
    b0 = n.part * (kBlks / g.splits);
    b1 = min(nblk, b0 + kBlks / g.splits);
  }
  float2 dc = make_float2(0.f, 0.f);  // (d, f + d) of the block's column number `lane`
  auto fetch = [&](int b, uint32_t cnt) {
    if (KIND == kNsGram) return;
    const int c = col0 + b * 32;
    e.flying |= 1u << (cnt & (T::kBufs - 1));
    if (lane == 0) {
      bulk_wait_read<0>();  // the buffer's last store has left it
      uint8_t* d = e.stg + (cnt & (T::kBufs - 1)) * (2 * kNsBoxBytes);
      mbar_arrive_expect_tx(&e.bars[cnt & (T::kBufs - 1)], in_low ? 2 * kNsBoxBytes : kNsBoxBytes);
      tma_load_3d<false>(smem_u32(d), in0, smem_u32(&e.bars[cnt & (T::kBufs - 1)]), c, row0, n.bz);
      if (in_low)
        tma_load_3d<false>(smem_u32(d + kNsBoxBytes), in1, smem_u32(&e.bars[cnt & (T::kBufs - 1)]), c, row0, n.bz);
    }
    if (by_col && c + lane < g.cols) {
      dc = __ldcg(dv + c + lane);
      dc.y += dc.x;
    }
  };
  if (b0 < b1) fetch(b0, e.cnt);
  // Warp-uniform outcomes: tcgen05.ld below is a warp-collective instruction.
  if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], parity, w))) return false;
  tc_fence_after();
  const uint32_t taddr = e.taddr + acc * T::kN + e.half * kHalf;
  // A split tile: each part hands the others' blocks of its accumulator over
  // through memory, waits for theirs and adds up the parts of its own blocks in
  // an order that does not depend on whose they are.  The parts run at the same
  // time (they are the last units of their CTAs in this GEMM).  A lane's float4
  // lie 512 bytes apart, so a warp's access is contiguous.
  constexpr size_t kPart = static_cast<size_t>(T::kWarps) * 32 * kHalf / 4;  // float4 of a tile's part
  float4* part = nullptr;
  if (kBlks > 1 && n.part >= 0 && nblk > 0) {
    const int region = (e.rank * 4 + e.q) * 2 + e.half;
    part = reinterpret_cast<float4*>(p.part) + static_cast<size_t>(n.split) * g.splits * kPart +
           region * (32 * kHalf / 4) + lane;
#pragma unroll 1
    for (int b = 0; b < nblk; ++b) {
      if (b >= b0 && b < b1) continue;
      uint32_t v[32];
      tmem_ld32(taddr + b * 32, v);
      tmem_ld_wait(v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        __stcg(part + n.part * kPart + (b * 8 + j) * 32,
               make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                           __uint_as_float(v[4 * j + 3])));
    }
    __syncwarp();
    int ok = 1;
    if (lane == 0) {
      int* c = p.counters + p.batch + KIND * kNsSplitCounters + n.split * T::kWarps + region;
      red_release_add(c, 1);
      if (b0 < b1) ok = ns_count_wait(c, g.splits * (step + 1), w) ? 1 : 0;
    }
    __syncwarp();
    if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
  }
  // the result's scale, and the accumulator's share of it
  constexpr float so = KIND == kNsGram ? kNsScaleA : kNsScaleP;
  const float sc = KIND == kNsSquare ? p.c * (kNsScaleP / (kNsScaleA * kNsScaleA))
                                     : (KIND == kNsGram ? kNsScaleA / (kNsScaleX * kNsScaleX) : 1.f / kNsScaleP);
#pragma unroll 1
  for (int b = b0; b < b1; ++b, ++e.cnt) {
    const int c32 = col0 + b * 32;
    const int buf = e.cnt & (T::kBufs - 1);
    uint8_t* S0 = e.stg + buf * (2 * kNsBoxBytes);
    uint8_t* S1 = S0 + kNsBoxBytes;
    const float2 dcb = dc;
    if (KIND == kNsGram) {
      if (lane == 0) bulk_wait_read<T::kBufs - 1>();
      __syncwarp();
    } else {
      if (b + 1 < b1) fetch(b + 1, e.cnt + 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&e.bars[buf], (e.loads >> buf) & 1, w))) return false;
      e.loads ^= 1u << buf;
      e.flying &= ~(1u << buf);
    }
    uint4 x0[4], x1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (KIND != kNsGram) x0[j] = ld_shared_v4(S0 + sw64_off(lane, j));
      if (in_low) x1[j] = ld_shared_v4(S1 + sw64_off(lane, j));
    }
    uint32_t v[32];
    tmem_ld32(taddr + b * 32, v);
    tmem_ld_wait(v);
    if (kBlks > 1 && part != nullptr) {
      // (p0 + p1), or (p0 + p1) + (p2 + p3): own and partner first, then the other pair
      const float4* f = part + b * 256;
      float4 o[8], q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __ldcg(f + (n.part ^ 1) * kPart + j * 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) ns_add4(v, j, o[j]);
      if (g.splits == 4) {
        f += ((n.part ^ 2) & 2) * kPart;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = __ldcg(f + j * 32);
          q[j] = __ldcg(f + kPart + j * 32);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          ns_add4(v, j, make_float4(o[j].x + q[j].x, o[j].y + q[j].y, o[j].z + q[j].z, o[j].w + q[j].w));
      }
    }
    uint64_t r[16];  // the results, two to a register pair
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = f2_mul(f2_bits(v[2 * i], v[2 * i + 1]), f2_set(sc, sc));
    if (KIND != kNsGram) {
      uint64_t in[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0[4] = {x0[j].x, x0[j].y, x0[j].z, x0[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) in[4 * j + i] = f2_half(w0[i]);
      }
      if (KIND == kNsSquare) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          r[i] = f2_fma(in[i], f2_set(p.b * (kNsScaleP / kNsScaleA), p.b * (kNsScaleP / kNsScaleA)), r[i]);
      } else {  // d X + (f + d) (X's low part)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint64_t d = f2_set(di.x, di.x);
          if (by_col)
            d = f2_set(__shfl_sync(0xffffffffu, dcb.x, 2 * i), __shfl_sync(0xffffffffu, dcb.x, 2 * i + 1));
          r[i] = f2_fma(in[i], d, r[i]);
        }
        if (in_low) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w1[4] = {x1[j].x, x1[j].y, x1[j].z, x1[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = 4 * j + i;
              uint64_t q = f2_set(di.y, di.y);
              if (by_col)
                q = f2_set(__shfl_sync(0xffffffffu, dcb.y, 2 * at), __shfl_sync(0xffffffffu, dcb.y, 2 * at + 1));
              r[at] = f2_fma(f2_half(w1[i]), q, r[at]);
            }
          }
        }
      }
    }
    if (KIND != kNsUpdate && c32 == row0) {
      // the block of this row's diagonal entry, column `lane`
      float corr = 0.f, dval = 0.f;
      const size_t at = static_cast<size_t>(n.bz) * g.rows + (live ? row : 0);
      if (KIND == kNsSquare) {
        const float2 q = __ldcg(p.diag[kBufA] + at);
        corr = fmaf(q.x, q.y, fmaf(q.y, q.x, q.x * q.x)) * so;
        corr = fmaf(p.c, corr, fmaf(p.b, q.x, p.a) * so);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float2 x = f2_get(r[i]);
        x.x += lane == 2 * i ? corr : 0.f;
        x.y += lane == 2 * i + 1 ? corr : 0.f;
        dval = lane == 2 * i ? x.x : (lane == 2 * i + 1 ? x.y : dval);
        r[i] = f2_set(x.x, x.y);
      }
      const float f = __half2float(__float2half_rn(dval));
      if (live) p.diag[kOut][at] = make_float2((dval - f) / so, f / so);
    }
    uint32_t o[16];
    if (KIND == kNsUpdate && last) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = f2_get(f2_mul(r[i], f2_set(1.f / kNsScaleX, 1.f / kNsScaleX)));
        o[i] = pack_bf16x2(x.x, x.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = f2_get(r[i]);
        o[i] = pack_f16x2(x.x, x.y);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(S0 + sw64_off(lane, j), make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
    if (has_low) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = f2_get(f2_sub(r[i], f2_half(o[i])));
        o[i] = pack_f16x2(x.x, x.y);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        st_shared_v4(S1 + sw64_off(lane, j), make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      const CUtensorMap* m = KIND != kNsUpdate ? &p.Sbox[kOut] : (last ? &p.Obox : &p.Hbox[par ^ 1]);
      tma_store_3d(m, S0, c32, row0, n.bz);
      if (has_low) tma_store_3d(&p.Lbox[par ^ 1], S1, c32, row0, n.bz);
      bulk_commit();
    }
  }
  return true;
}

// All steps in one persistent launch.  The CTAs (or CTA pairs) take the units of
// a phase in turn, and go from phase to phase.  A unit loads what other CTAs
// wrote in the phase before: a CTA arrives at a counter in global memory when
// its epilogue warps' stores have completed, and the thread that issues a unit's
// left loads polls until the last phase is complete, and lets the other loads and
// the epilogue warps go on through an mbarrier.  One counter for all matrices
// makes that a barrier between GEMMs, and the CTAs arrive once for a phase.  With
// a few units for each CTA (`few`) each matrix has its own, and the last units of
// one phase run beside the first of the next: 586 against 626 us for four of 2048
// x 2048, 237 against 270 for eight of 1024 x 1024, 125 against 153 for sixteen of
// 512 x 512.  With many units the phases' ends matter less than an arrival for
// each: 706 against 674 for 128 of 512 x 512, 990 against 735 for 3000 of 64 x 64
// (equal within 5 % at seven units for each CTA).  Every buffer is written one
// phase or more after the phases that read it, of the same matrix.  The split
// tiles' exchange buffers are no matrix's: their units wait for all matrices.  A
// unit only waits for units before it in the order that all CTAs follow, and all
// CTAs are resident at once, by a cooperative launch.
//
// Times here and at the tile rule: calls back to back with normal entries in G.
// Where a gradient's products keep the clock lower they are longer (690 us for
// four of 2048 x 2048).
template <class T>
__global__ void __launch_bounds__(kNsThreads, 1) ns_kernel(const __grid_constant__ NsParams p) {
  constexpr bool PAIR = T::kPair;
  constexpr int kStages = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sEpi = smem + kStages * T::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + kNsEpiWarps * T::kEpiBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* go = drain + 1;         // the i-th wait of this CTA is over: barrier i mod kNsAhead
  uint64_t* ebars = go + kNsAhead;  // two for each epilogue warp
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ebars + 2 * kNsEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* warps_done = reinterpret_cast<int*>(tmem_holder + 2);  // [kNsAhead]: epilogue warps done with unit i

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // (uniform for the compiler too)
  const int lane = threadIdx.x & 31;
  const int rank = PAIR ? __shfl_sync(0xffffffffu, static_cast<int>(cluster_ctarank()), 0) : 0;
  const int step = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
  const int first = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 2 * kNsEpiWarps : kNsEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kNsAhead; ++i) {
      mbar_init(&go[i], 1);
      warps_done[i] = 0;
    }
    for (int i = 0; i < 2 * kNsEpiWarps; ++i) mbar_init(&ebars[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_holder, 2 * T::kN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 2 * T::kN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const WaitCtx w{abort_flag, p.wait_ns};
  // Copies and MMAs in flight are waited for at the end, after a wait that gave up
  // too, however short the caller's limit is.
  const uint64_t drain_ns = p.wait_ns > kNsDrainNs ? p.wait_ns : kNsDrainNs;

  // The issuing warps run as whole warps, with one elected thread issuing: the
  // instructions take their operands from uniform registers, and in code of a
  // single thread every operand is moved there one by one (an MMA loop of 590
  // cycles a k-block, against 512 of a pair's MMAs).
  if (warp == 0 || warp == kNsRightWarp) {
    const bool left = warp == 0;
    const bool leader = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    int it = 0;  // waits so far
    bool ok = true;
    const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
    const uint32_t smem0 = smem_u32(smem) + (left ? 0 : T::kLeftBytes);
    for (NsSeq s; ok && s.next(p);) {
      const int nunits = ns_units(p, s);
      int waited = -1;
      for (int u = first; ok && u < nunits; u += step) {
        const NsUnit n = ns_unit<T>(p, s, u);
        NsOperand P, Q;
        ns_operands(p, s, P, Q);
        NsOperand op = left ? P : Q;
        const int row = left ? n.rt * T::kM : n.ct * T::kN;
        int mn = op.template first_mn<T::kM>(row), r0 = row + rank * 128;
        asm volatile("" : "+l"(op.maps), "+r"(mn), "+r"(r0));  // worked out before the wait, not after it
        const int need = ns_need(p, s, n, waited);
        if (need >= 0) {
          bool passed = true;
          if (left) {
            const int b0 = need < p.batch ? need : 0, b1 = need < p.batch ? need + 1 : (p.few ? p.batch : 1);
            const unsigned target = p.few ? s.done : s.done * static_cast<unsigned>(p.batch);
            for (int b = b0 + lane; b < b1; b += 32) passed = passed && ns_count_wait(p.counters + b, target, w);
            if (b1 - b0 > 1) {
              // each lane has acquired its counters: the arrival of lane 0 hands on all of them
              __syncwarp();
              passed = __all_sync(0xffffffffu, passed);
            }
            if (lane == 0 && passed) mbar_arrive(&go[it & (kNsAhead - 1)]);
          } else {
            passed = mbar_wait(&go[it & (kNsAhead - 1)], (it / kNsAhead) & 1, w);
          }
          if (!__all_sync(0xffffffffu, passed)) {
            ok = false;
            break;
          }
          __syncwarp();
          fence_proxy_async_global();  // the loads below see what other CTAs' copies wrote
          ++it;
        }
        for (int kb = n.kb0; kb < n.kb1; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, w))) {
            ok = false;
            break;
          }
          const uint32_t dst = smem0 + stage * T::kStageBytes, bar = full0 + stage * 8;
          if (leader) {
            if (left) {
              if (!PAIR || rank == 0) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * T::kStageBytes);
              ns_load<128, PAIR>(dst, op.maps, kb >= mn, r0, kb * 64, n.bz, bar);
            } else {
              ns_load<T::kRight, PAIR>(dst, op.maps, kb >= mn, r0, kb * 64, n.bz, bar);
            }
          }
          if (issued < kStages) ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    // Every copy must have landed before shared memory goes away: the MMA's
    // release of a stage follows its copies.
    for (int i = 0; i < issued; ++i) {
      if (stage == 0) {
        stage = kStages - 1;
        phase ^= 1u;
      } else {
        --stage;
      }
      int no_abort = 0;
      (void)mbar_wait(PAIR ? &empty[stage] : &full[stage], phase, WaitCtx{&no_abort, drain_ns});
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const bool leader = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      const uint32_t smem0 = smem_u32(smem);
      constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024, version 1, 128-byte swizzle
      for (NsSeq s; ok && s.next(p);) {
        const int nunits = ns_units(p, s);
        for (int u = first; ok && u < nunits; u += step, ++it) {
          const NsUnit n = ns_unit<T>(p, s, u);
          NsOperand P, Q;
          ns_operands(p, s, P, Q);
          const int acc = it & 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, w))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * T::kN;
          const int mnp = P.template first_mn<T::kM>(n.rt * T::kM), mnq = Q.template first_mn<T::kM>(n.ct * T::kN);
          for (int kb = n.kb0; kb < n.kb1; ++kb) {
            // between two GEMMs this waits as long as the slowest CTA works
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, w))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const bool pm = kb >= mnp, qm = kb >= mnq;
            const uint32_t idesc = idesc_f16_f32(T::kM, T::kN, false, false) | (pm ? 1u << 15 : 0u) | (qm ? 1u << 16 : 0u);
            // The descriptors' low words: address and leading offset (sdesc_sw128)
            // in units of 16 bytes.  A step is 32 bytes of a K-major row, 16 rows of
            // 128 bytes of an MN-major block.
            const uint32_t a0 = (smem0 + stage * T::kStageBytes) >> 4;
            const uint32_t la = a0 | (pm ? 512u << 16 : 1u << 16);
            const uint32_t lb = (a0 + (T::kLeftBytes >> 4)) | (qm ? 512u << 16 : 1u << 16);
            const uint32_t sa = pm ? 128u : 2u, sb = qm ? 128u : 2u;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t accum = (kb != n.kb0 || kk != 0) ? 1u : 0u;
                const uint64_t ad = f2_bits(la + kk * sa, kDescHigh), bd = f2_bits(lb + kk * sb, kDescHigh);
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
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (leader) {
            if (PAIR)
              tc_commit_pair_mc(&tfull[acc], 0x3);
            else
              tc_commit(&tfull[acc]);
          }
        }
      }
      if (leader) {
        if (PAIR)
          tc_commit_pair(drain);
        else
          tc_commit(drain);
      }
      int no_abort = 0;
      (void)mbar_wait(drain, 0, WaitCtx{&no_abort, drain_ns});
      __syncwarp();
    }
  } else {
    NsEpi e;
    e.stg = sEpi + (warp - 2) * T::kEpiBytes;
    e.q = warp & 3;  // the TMEM lane quarter this warp may access
    e.half = (warp - 2) >> 2;
    e.rank = rank;
    e.lane = lane;
    e.bars = ebars + 2 * (warp - 2);
    e.cnt = 0;
    e.loads = 0;
    e.flying = 0;
    e.taddr = tmem_base + (static_cast<uint32_t>(e.q * 32) << 16);
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    int it = 0;
    bool ok = true;
    int waits = 0;
    for (NsSeq s; ok && s.next(p);) {
      const int nunits = ns_units(p, s);
      int waited = -1, arrive = 0;
      for (int u = first; ok && u < nunits; u += step, ++it) {
        const NsUnit n = ns_unit<T>(p, s, u);
        if (ns_need(p, s, n, waited) >= 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(&go[waits & (kNsAhead - 1)], (waits / kNsAhead) & 1, w))) {
            ok = false;
            break;
          }
          if (lane == 0) fence_proxy_async_global();
          ++waits;
        }
        const int acc = it & 1;
        const uint32_t par = (it >> 1) & 1;
        if (s.kind == kNsSquare)
          ok = ns_epilogue<kNsSquare, T>(p, s.step, n, acc, par, tfull, e, w);
        else if (s.kind == kNsUpdate)
          ok = ns_epilogue<kNsUpdate, T>(p, s.step, n, acc, par, tfull, e, w);
        else
          ok = ns_epilogue<kNsGram, T>(p, s.step, n, acc, par, tfull, e, w);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_cluster(tempty0 + acc * 8);
          else
            mbar_arrive(&tempty[acc]);
        }
        if (!ok) break;
        arrive += n.weight;
        if (!p.few && u + step < nunits) continue;
        // this warp's results of the unit (or of all its units of the phase) are in memory: arrive
        if (lane == 0) {
          bulk_wait_all<0>();
          fence_proxy_async_global();
        }
        __syncwarp();
        // the CTA's last warp arrives for all of them: its release covers what the
        // others' lanes wrote before the warp barrier and their arrivals here
        int* done = &warps_done[it & (kNsAhead - 1)];
        if (lane == 0 && add_acq_rel_cta(done, 1) == kNsEpiWarps - 1) {
          *done = 0;
          red_release_add(p.counters + (p.few ? n.bz : 0), arrive);
        }
        arrive = 0;
      }
    }
    // (a wait that gave up leaves loads behind)
    for (int i = 0; i < T::kBufs; ++i) {
      int no_abort = 0;
      if ((e.flying >> i) & 1) (void)mbar_wait(&e.bars[i], (e.loads >> i) & 1, WaitCtx{&no_abort, drain_ns});
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
      tmem_dealloc_pair(tmem_base, 2 * T::kN);
    else
      tmem_dealloc(tmem_base, 2 * T::kN);
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

// X_0 = G / (|G|_F + eps), times the stored scale, as high and low fp16 parts
// (and the counters of ns_kernel, which runs next, set to zero).
// The factor goes on in two steps so that it may pass fp32's range (a G of
// 1e-30 with eps 0).
__global__ void __launch_bounds__(kNsNormThreads) ns_scale_kernel(const float* __restrict__ G, size_t n8, int nblk,
                                                                 const double* __restrict__ part, double eps,
                                                                 __half* __restrict__ hi, __half* __restrict__ lo,
                                                                 int* __restrict__ counters, int ncounters) {
  __shared__ double red[kNsNormThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < ncounters; i += kNsNormThreads) counters[i] = 0;
  double s = 0.0;
  for (int i = threadIdx.x; i < nblk; i += kNsNormThreads) s += part[static_cast<size_t>(blockIdx.y) * nblk + i];
  s = ns_block_sum(s, red);
  const double f = static_cast<double>(kNsScaleX) / (sqrt(s) + eps);
  const float f1 = f > 1e20 ? 1.8446744073709552e19f : (f < 1e-20 ? 5.421010862427522e-20f : 1.f);  // 2^64, 2^-64
  const float f2 = static_cast<float>(f / static_cast<double>(f1));
  const size_t off = static_cast<size_t>(blockIdx.y) * n8;
  const float4* g = reinterpret_cast<const float4*>(G) + off * 2;
  // from the end, which the sums have read last and left in L2
  for (size_t r = blockIdx.x * static_cast<size_t>(kNsNormThreads) + threadIdx.x; r < n8;
       r += static_cast<size_t>(gridDim.x) * kNsNormThreads) {
    const size_t i = n8 - 1 - r;
    const float4 a = __ldcs(g + 2 * i), b = __ldcs(g + 2 * i + 1);
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
    reinterpret_cast<uint4*>(lo)[off + i] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

}  // namespace coda
