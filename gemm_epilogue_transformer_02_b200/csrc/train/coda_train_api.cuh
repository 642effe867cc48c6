// Host side of the training-step calls around the GEMM chain: token embedding,
// residual add + RMSNorm with 8-bit outputs, Newton-Schulz orthogonalisation.
// Included by coda.cu (it uses its validation, device and tensor-map helpers);
// contracts in include/coda.h.
#pragma once

#include "coda_embed.cuh"
#include "coda_norm8.cuh"
#include "coda_ns.cuh"

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;

// A launch with programmatic stream serialisation (the kernel waits for the
// previous one itself), as the GEMMs'.
template <class... KArgs, class... Args>
coda_status_t launch_pdl(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, KArgs(args)...) == cudaSuccess ? CODA_OK : CODA_ERR_LAUNCH;
}

// ---------------------------------------------------------------- embedding

// Pairs per block of the embedding backward: 16, so that a batch of some
// thousand tokens gives some hundred blocks; more once that would make over 2048
// blocks, which bounds the parts a run over many chunks is joined from (up to
// 2^21 rows: from there on a block takes 1024 pairs).
inline int embed_chunk(int64_t M) {
  int64_t c = 16;
  while (c < coda::kEmbBwdMaxChunk && M > 2048 * c) c *= 2;
  return static_cast<int>(c);
}

// The sort counts rows in ints, up to 1023 past the last.
constexpr int64_t kEmbBwdMaxRows = kMaxInt - 1023;

struct EmbedWs {
  size_t buf0, buf1, part, list, crossing, bitmap, words, bytes;
  int chunk, items;
};

inline EmbedWs embed_ws(int64_t M, int64_t D, int64_t V) {
  EmbedWs w;
  w.chunk = embed_chunk(M);
  w.items = static_cast<int>((M + w.chunk - 1) / w.chunk);
  w.words = static_cast<size_t>((V + 31) / 32);
  w.buf0 = 0;
  w.buf1 = align256(static_cast<size_t>(M) * 8);
  w.part = 2 * w.buf1;
  w.list = w.part + align256(static_cast<size_t>(w.items) * 2 * D * 4);
  w.crossing = w.list + align256(static_cast<size_t>(w.items) * 4);
  w.bitmap = w.crossing + 256;
  w.bytes = w.bitmap + align256(w.words * 4);
  return w;
}

// Spans of columns of the summing blocks, and 2^unit rows of a zeroing one: about
// 64 KB, so that the blocks that run together write a compact range.
inline int embed_bwd_spans(int64_t D) {
  return static_cast<int>((D + 8 * coda::kEmbBwdThreads - 1) / (8 * coda::kEmbBwdThreads));
}
inline int embed_bwd_unit(int64_t D) {
  int unit = 0;
  while (unit < 5 && ((D * 4) << (unit + 1)) <= 65536) ++unit;
  return unit;
}

// (blocks are counted in ints)
inline bool embed_bwd_shape_ok(int64_t M, int64_t D, int64_t V) {
  return M >= 0 && M <= kEmbBwdMaxRows && dim_ok(D) && V > 0 && V < kMaxInt &&
         (M + embed_chunk(M) - 1) / embed_chunk(M) * embed_bwd_spans(D) < kMaxInt / 2 &&
         (V >> embed_bwd_unit(D)) < kMaxInt / 2;
}

// Bytes of dE that the sorting launch zeroes: as many as HBM takes while one
// cluster sorts (14 us for 8192 tokens).
inline size_t embed_zero_first(int64_t M) { return (size_t(48) << 20) + static_cast<size_t>(M) * 4096; }

// --------------------------------------------------------------------- norm

// Two 8-column vectors a thread, so a row of up to 16384 columns stays in one
// block's registers.  Narrow rows have a warp each, four to a block: as blocks of
// 64 threads they were bound by the rate at which blocks start and by their
// barriers (MXFP8, 32768 x 128 34.2 us against 14.1, 16384 x 512 17.7 against
// 11.6; but 1024 columns, four vectors a lane, 12.8 against 11.8 as blocks).
constexpr int64_t kNorm8MaxN = 16384;
constexpr int64_t kNorm8WarpN = 512;
constexpr int kNorm8WarpThreads = 128;
inline int norm8_threads(int64_t N) { return static_cast<int>(((N / 8 + 1) / 2 + 31) & ~int64_t(31)); }

template <bool MX>
coda_status_t launch_norm8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps, const float* s_y,
                           uint16_t* h_out, uint8_t* q, uint8_t* sf, unsigned* amax, float* r_out, int64_t M,
                           int64_t N, cudaStream_t s) {
  const int64_t nrb = (M + 127) / 128, rows = MX ? nrb * 128 : M;
  const bool warp = N <= kNorm8WarpN;
  const int threads = warp ? static_cast<int>(std::min<int64_t>(kNorm8WarpThreads, 32 * rows)) : norm8_threads(N);
  const int64_t blocks = warp ? (rows + threads / 32 - 1) / (threads / 32) : rows;
  if (!MX && blocks > 1 && cudaMemsetAsync(amax, 0, sizeof(float), s) != cudaSuccess) return CODA_ERR_LAUNCH;
  // (registers for as many blocks as hide each other's reductions: 4096 x 8192
  // 41.3 us against 47.5 with two of 512 threads, 2048 x 16384 45.1 against 55.0)
  auto kern = warp             ? add_rmsnorm_kernel<MX, true, kNorm8WarpThreads, 1>
              : threads <= 256 ? add_rmsnorm_kernel<MX, false, 256, 5>
              : threads <= 512 ? add_rmsnorm_kernel<MX, false, 512, 4>
                               : add_rmsnorm_kernel<MX, false, 1024, 2>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), threads, 0, s,
                    reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(res),
                    reinterpret_cast<const __nv_bfloat16*>(gamma), eps, s_y, reinterpret_cast<__nv_bfloat16*>(h_out),
                    q, sf, amax, r_out, M, static_cast<int>(N), static_cast<int>(nrb));
}

// Blocks of the norm's backward: as many as 148 SMs hold at once, so that every
// block has as many rows (narrow rows, a warp each: 16384 x 512 16.7 us, five
// blocks 17.7, a block for each row's warp 20.5).
inline int norm8_bwd_blocks(int64_t M, int64_t N) {
  if (N <= kNorm8WarpN) return static_cast<int>(std::min<int64_t>((M + 3) / 4, 148 * 4));
  const int t = norm8_threads(N);
  return static_cast<int>(std::min<int64_t>(M, 148 * (t <= 128 ? 640 / t : t <= 512 ? 1024 / t : 1)));
}

// ------------------------------------------------------------ Newton-Schulz

constexpr int kNsMaxNormBlocks = 1184;  // eight for each of 148 SMs

// With up to this many units for each CTA (or pair) in the longest phase each unit
// waits for its own matrix (ns_kernel has the figures).
constexpr int kNsFew = 4;

inline int ns_counters(int64_t batch) { return static_cast<int>(batch) + kNsKinds * kNsSplitCounters; }

// The longest side, which a Gram matrix sums over: its one tile of a narrow matrix,
// in two parts, takes 0.25 us for each of their 64-wide k-blocks (0.65 s for five
// steps at 8 x 2^26), and the other CTAs' waits for a part end after a second.
constexpr int64_t kNsMaxSide = int64_t(1) << 28;

// (byte strides of the tensor maps; tiles are counted in ints)
inline bool ns_shape_ok(int64_t batch, int64_t m, int64_t n) {
  return batch >= 0 && batch <= 65535 && dim_ok(m) && dim_ok(n) && std::max(m, n) <= kNsMaxSide &&
         m * n <= int64_t(1) << 38 &&
         2 * batch * ((m + 127) / 128) * ((n + 63) / 64) <= kMaxInt;
}

struct NsPlan {
  int64_t batch, m, n, s;  // s: the smaller side
  bool tall;
  int tile;                // 256: 256 x 256 tiles on CTA pairs; 128, 64: 128 x tile
  int norm_blocks;
  size_t hi[2], lo[2], sym[kBufs], diag[kBufs], sums, counters, part, bytes;
};

inline NsPlan ns_plan(int64_t batch, int64_t m, int64_t n) {
  NsPlan p;
  p.batch = batch;
  p.m = m;
  p.n = n;
  p.tall = m > n;
  p.s = p.tall ? n : m;
  // CTA pairs (half of the operand traffic) where their 256 x 256 tiles fill more
  // than one round of the 74 pairs, in us against the 128 x 128 tiles: with a
  // long K those of X (319 against 381 for two of 2048 x 2048, 582 against 795 for
  // four, 1030 against 1490 at 4096 x 4096), with a shorter one those of the square
  // matrices too, whose phases are most of a step (310 against 409 for twelve of
  // 1024 x 1024, 442 against 506 for sixteen), or, of a long side, several rounds
  // of X's (691 against 854 at 1024 x 32768, 428 against 463 at 1024 x 16384, 469
  // against 538 at 512 x 32768; for five of 1024 x 4096 500 against 541, but for
  // four 418 against 393: a batch's square phases have more tiles).  With fewer
  // the four times as many small ones end sooner: 193 against 203 at 1024 x 4096,
  // 303 against 325 at 1152 x 8192; eight of 1024 x 1024 (255) are equal.  The
  // smallest where all of them run at once: 94 against 113 us at 512 x 512, 73
  // against 91 at 256 x 256.
  const int64_t t256 = batch * ((m + 255) / 256) * ((n + 255) / 256);
  const int64_t s256 = (p.s + 255) / 256, square = batch * s256 * s256;
  const bool pairs = p.s >= 1536 ? t256 >= 100
                                 : (p.s >= 1024 && square >= 150) ||
                                       (p.s >= 512 && std::max(m, n) >= 2 * p.s && t256 >= (batch == 1 ? 180 : 300));
  p.tile = pairs ? 256 : batch * ((m + 127) / 128) * ((n + 63) / 64) <= 148 ? 64 : 128;
  const int64_t n8 = m * n / 8;
  p.norm_blocks = static_cast<int>(std::min<int64_t>(kNsMaxNormBlocks, (n8 + 2047) / 2048));
  size_t o = 0;
  const auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    p.hi[i] = take(static_cast<size_t>(batch) * m * n * 2);
    p.lo[i] = take(static_cast<size_t>(batch) * m * n * 2);
  }
  for (int i = 0; i < kBufs; ++i) {
    p.sym[i] = take(static_cast<size_t>(batch) * p.s * p.s * 2);
    p.diag[i] = take(static_cast<size_t>(batch) * p.s * 8);
  }
  p.sums = take(static_cast<size_t>(batch) * p.norm_blocks * 8);
  p.counters = take(static_cast<size_t>(ns_counters(batch)) * 4);
  // at most one split unit per CTA (pair) of the grid
  p.part = take(p.tile == 64 ? 0 : static_cast<size_t>(148) * 128 * p.tile * 4);
  p.bytes = o;
  return p;
}

// [batch, rows, cols] of 2-byte elements, box box_rows x 64 with the 128-byte
// swizzle, or box_rows x 32 with the 64-byte one; out-of-range elements read as
// zero and are not written.
bool tmap3d(CUtensorMap* m, const void* base, bool bf16, uint64_t cols, uint64_t rows, uint64_t batch,
            uint32_t box_rows, uint32_t box_cols = 64) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {cols, rows, batch};
  cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool ns_maps(NsMaps* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch) {
  return tmap3d(&m->k128, base, false, cols, rows, batch, 128) && tmap3d(&m->b64, base, false, cols, rows, batch, 64);
}

// A GEMM's tiles over `slots` CTAs (or pairs).  Whole rounds of tiles are one
// unit each.  A last round that fills at most half of the slots is split by
// k-blocks, into two parts or, on pairs, four, if they fit and are at least
// eight k-blocks long: the parts exchange accumulators through memory (about 4
// us), which costs less than the k-blocks it saves only then.
NsGeo ns_geo(int64_t batch, int64_t rows, int64_t cols, int64_t K, bool sym, int tile, int slots) {
  const int tm = tile == 256 ? 256 : 128;
  NsGeo g;
  g.rows = static_cast<int>(rows);
  g.cols = static_cast<int>(cols);
  g.nkb = static_cast<int>((K + 63) / 64);
  g.n_rt = static_cast<int>((rows + tm - 1) / tm);
  g.n_ct = static_cast<int>((cols + tile - 1) / tile);
  g.tiles = sym ? g.n_rt * (g.n_rt + 1) / 2 * (tm / tile) : g.n_rt * g.n_ct;
  const int all = static_cast<int>(batch) * g.tiles;
  g.rest = all % slots;
  g.whole = all - g.rest;
  g.splits = 1;
  while (g.rest > 0 && 2 * g.splits <= tile / 64 && 2 * g.splits * g.rest <= slots &&
         g.nkb / (2 * g.splits) >= 8)
    g.splits *= 2;
  // of each CTA at each of a matrix's tiles, a whole one as often as a split one
  g.arrivals = g.tiles * g.splits * (tile == 256 ? 2 : 1);
  return g;
}

template <int N>
coda_status_t ns_launch(int dev, DevInfo* info, NsParams& p, const NsPlan& pl, cudaStream_t stream) {
  static bool done[64];
  static int slots[64];  // CTAs (or pairs) resident at once
  auto kern = ns_kernel<NsTile<N>>;
  constexpr bool PAIR = NsTile<N>::kPair;
  constexpr int kSmem = NsTile<N>::kSmem;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kNsThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return CODA_ERR_LAUNCH;
      int n = info->sms;
      if (PAIR) {
        cfg.gridDim = dim3(2 * (info->sms / 2), 1, 1);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return CODA_ERR_LAUNCH;
      }
      slots[dev] = std::min(n, PAIR ? 74 : 148);  // (the workspace has room for that many)
      done[dev] = true;
    }
  }
  const int64_t s = pl.s, l = pl.tall ? pl.m : pl.n;
  p.geo[kNsGram] = ns_geo(pl.batch, s, s, l, true, N, slots[dev]);
  p.geo[kNsSquare] = ns_geo(pl.batch, s, s, s, true, N, slots[dev]);
  p.geo[kNsUpdate] = ns_geo(pl.batch, pl.m, pl.n, s, false, N, slots[dev]);
  int n = 0, units = 0;
  for (const NsGeo& g : p.geo) {
    n = std::max(n, g.whole > 0 ? slots[dev] : g.rest * g.splits);
    units = std::max(units, g.whole + g.rest * g.splits);
  }
  p.few = pl.batch > 1 && units <= kNsFew * slots[dev];
  p.wait_ns = static_cast<uint64_t>(g_wait_ns);
  cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * n : n), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? CODA_OK : CODA_ERR_LAUNCH;
}

}  // namespace

extern "C" {

coda_status_t coda_embed(const int64_t* tokens, const uint16_t* E, float scale, const uint16_t* gamma, uint16_t* h_out,
                         uint16_t* hg_out, float* partial, int64_t M, int64_t D, int64_t V, void* stream) {
  CODA_CHECK(M >= 0 && M <= kMaxInt && dim_ok(D) && V > 0 && V < kMaxInt, CODA_ERR_SHAPE);
  const int64_t nspan = (D + 255) / 256;
  const int64_t items = (M + kEmbRows - 1) / kEmbRows * nspan;
  const int64_t blocks = (items + kEmbWarps - 1) / kEmbWarps;
  CODA_CHECK(blocks <= kMaxInt, CODA_ERR_SHAPE);
  if (M == 0) return CODA_OK;  // (an empty tensor has no address)
  CODA_CHECK(tokens && E && (h_out || hg_out || partial) && (!hg_out || gamma), CODA_ERR_NULL);
  CODA_CHECK(al16(tokens) && al16(E) && al16(gamma) && al16(h_out) && al16(hg_out) && al16(partial), CODA_ERR_ALIGN);
  int dev;
  DevInfo* info;
  const coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  return launch_pdl(embed_kernel, dim3(static_cast<unsigned>(blocks)), 32 * kEmbWarps, 0,
                    static_cast<cudaStream_t>(stream), tokens, reinterpret_cast<const __nv_bfloat16*>(E), scale,
                    reinterpret_cast<const __nv_bfloat16*>(gamma), reinterpret_cast<__nv_bfloat16*>(h_out),
                    reinterpret_cast<__nv_bfloat16*>(hg_out), partial, M, static_cast<int>(D), V,
                    static_cast<int>(nspan));
}

size_t coda_embed_bwd_workspace_size(int64_t M, int64_t D, int64_t V) {
  if (M <= 0 || !embed_bwd_shape_ok(M, D, V)) return 0;
  return embed_ws(M, D, V).bytes;
}

coda_status_t coda_embed_bwd(const int64_t* tokens, const uint16_t* dh, float scale, float* dE, int accumulate, void* ws,
                             size_t ws_bytes, int64_t M, int64_t D, int64_t V, void* stream) {
  CODA_CHECK(embed_bwd_shape_ok(M, D, V), CODA_ERR_SHAPE);
  CODA_CHECK(dE && (M == 0 || (tokens && dh)), CODA_ERR_NULL);
  CODA_CHECK(al16(tokens) && al16(dh) && al16(dE) && al16(ws), CODA_ERR_ALIGN);
  CODA_CHECK(M == 0 || (ws && ws_bytes >= embed_ws(M, D, V).bytes), CODA_ERR_WORKSPACE);
  if (M == 0 && accumulate) return CODA_OK;
  int dev;
  DevInfo* info;
  coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0)
    return cudaMemsetAsync(dE, 0, static_cast<size_t>(V) * D * 4, s) == cudaSuccess ? CODA_OK : CODA_ERR_LAUNCH;
  static bool done[64];
  static int clusters[64];
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[dev]) {
      if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem) !=
          cudaSuccess)
        return CODA_ERR_LAUNCH;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(kSortCluster * 64));
      cfg.blockDim = dim3(kSortThreads);
      cfg.dynamicSmemBytes = kSortSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = kSortCluster;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&clusters[dev], embed_sort_kernel, &cfg) != cudaSuccess || clusters[dev] < 2) {
        cudaGetLastError();
        clusters[dev] = 2;
      }
      done[dev] = true;
    }
  }
  const EmbedWs w = embed_ws(M, D, V);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int2* b0 = reinterpret_cast<int2*>(base + w.buf0);
  int2* b1 = reinterpret_cast<int2*>(base + w.buf1);
  float* part = reinterpret_cast<float*>(base + w.part);
  int bits = 1;
  while ((V >> bits) > 0) ++bits;  // keys 0 .. V
  const int passes = (bits + kSortBits - 1) / kSortBits;
  // pass 0 reads the tokens and writes b1, pass 1 writes b0, ...
  const int2* pairs = passes & 1 ? b1 : b0;
  int* list = reinterpret_cast<int*>(base + w.list);
  int* crossing = reinterpret_cast<int*>(base + w.crossing);
  uint32_t* bitmap = accumulate ? nullptr : reinterpret_cast<uint32_t*>(base + w.bitmap);
  const size_t row = static_cast<size_t>(D) * 4;
  // whole words of the bitmap (32 rows) go to the sorting launch
  const int64_t zero_row =
      accumulate ? 0 : std::min<int64_t>(V, static_cast<int64_t>(embed_zero_first(M) / (32 * row)) * 32);
  // a cluster for every eight takes of eight pieces, at most as many as run at
  // once beside the sorting one (a second wave of them took 120 us more)
  const size_t take = size_t(64) * kZeroPiece;
  const int64_t zc = std::min<int64_t>(clusters[dev] - 1, static_cast<int64_t>((zero_row * row + take - 1) / take));
  st = launch_pdl(embed_sort_kernel, dim3(static_cast<unsigned>(kSortCluster * (1 + zc))), kSortThreads, kSortSmem,
                  s, tokens, static_cast<int>(M), V, passes, b0, b1, reinterpret_cast<uint8_t*>(dE), zero_row * row,
                  bitmap, w.words, crossing);
  if (st != CODA_OK) return st;
  const int threads = static_cast<int>(std::min<int64_t>(kEmbBwdThreads, (D / 8 + 31) & ~int64_t(31)));
  const int spans = embed_bwd_spans(D), unit = embed_bwd_unit(D);
  const int64_t zb = accumulate ? 0 : (V - zero_row + (1 << unit) - 1) >> unit;
  auto sum = accumulate ? embed_bwd_kernel<true> : embed_bwd_kernel<false>;
  st = launch_pdl(sum, dim3(static_cast<unsigned>(w.items * spans + zb)), threads, 0, s, pairs,
                  reinterpret_cast<const __nv_bfloat16*>(dh), scale, dE, part, list, crossing, static_cast<int>(M), V,
                  static_cast<int>(D), w.chunk, w.items, spans, static_cast<const uint32_t*>(bitmap), zero_row, unit);
  if (st != CODA_OK || w.items == 1) return st;
  const int64_t jb = std::min<int64_t>(2 * info->sms, (w.items - 1) * ((D + 255) / 256));
  return launch_pdl(embed_bwd_join_kernel, dim3(static_cast<unsigned>(jb)), 32 * kJoinGroups, 0, s, pairs,
                    static_cast<const float*>(part), static_cast<const int*>(list), static_cast<const int*>(crossing),
                    scale, dE, static_cast<int>(D), w.chunk, w.items, accumulate ? 1 : 0);
}

coda_status_t coda_add_rmsnorm_mx(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                                  uint16_t* h_out, uint8_t* yq_out, uint8_t* ysf_out, float* r_out, int64_t M,
                                  int64_t N, void* stream) {
  CODA_CHECK(M >= 0 && M <= kMaxInt - 127 && dim_ok(N) && N % 128 == 0 && N <= kNorm8MaxN && eps >= 0.f,
             CODA_ERR_SHAPE);
  if (M == 0) return CODA_OK;
  CODA_CHECK(x && gamma && yq_out && ysf_out, CODA_ERR_NULL);
  CODA_CHECK(al16(x) && al16(res) && al16(gamma) && al16(h_out) && al16(yq_out) && al16(ysf_out) && al16(r_out),
             CODA_ERR_ALIGN);
  int dev;
  DevInfo* info;
  const coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  return launch_norm8<true>(x, res, gamma, eps, nullptr, h_out, yq_out, ysf_out, nullptr, r_out, M, N,
                            static_cast<cudaStream_t>(stream));
}

coda_status_t coda_add_rmsnorm_fp8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                                   const float* s_y, uint16_t* h_out, uint8_t* y8_out, float* amax_out, float* r_out,
                                   int64_t M, int64_t N, void* stream) {
  CODA_CHECK(M >= 0 && M <= kMaxInt && dim_ok(N) && N % 16 == 0 && N <= kNorm8MaxN && eps >= 0.f, CODA_ERR_SHAPE);
  if (M == 0) return CODA_OK;
  CODA_CHECK(x && gamma && s_y && y8_out && amax_out, CODA_ERR_NULL);
  CODA_CHECK(al16(x) && al16(res) && al16(gamma) && al16(s_y) && al16(h_out) && al16(y8_out) && al16(amax_out) &&
                 al16(r_out),
             CODA_ERR_ALIGN);
  int dev;
  DevInfo* info;
  const coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_norm8<false>(x, res, gamma, eps, s_y, h_out, y8_out, nullptr, reinterpret_cast<unsigned*>(amax_out),
                             r_out, M, N, s);
}

size_t coda_add_rmsnorm_bwd_workspace_size(int64_t M, int64_t N) {
  if (M <= 0 || !dim_ok(N) || N > kNorm8MaxN) return 0;
  return static_cast<size_t>(norm8_bwd_blocks(M, N)) * N * 4;
}

coda_status_t coda_add_rmsnorm_bwd(const uint16_t* dy, const uint16_t* h, const float* r, const uint16_t* gamma,
                                   const uint16_t* d_h, uint16_t* dx_out, float* dgamma_out, void* ws,
                                   size_t ws_bytes, int64_t M, int64_t N, void* stream) {
  CODA_CHECK(M >= 0 && M <= kMaxInt && dim_ok(N) && N <= kNorm8MaxN, CODA_ERR_SHAPE);
  CODA_CHECK(dgamma_out && (M == 0 || (dy && h && r && gamma && dx_out)), CODA_ERR_NULL);
  CODA_CHECK(al16(dy) && al16(h) && al16(r) && al16(gamma) && al16(d_h) && al16(dx_out) && al16(dgamma_out) &&
                 al16(ws),
             CODA_ERR_ALIGN);
  CODA_CHECK(M == 0 || (ws && ws_bytes >= coda_add_rmsnorm_bwd_workspace_size(M, N)), CODA_ERR_WORKSPACE);
  int dev;
  DevInfo* info;
  coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0)
    return cudaMemsetAsync(dgamma_out, 0, static_cast<size_t>(N) * 4, s) == cudaSuccess ? CODA_OK : CODA_ERR_LAUNCH;
  const int blocks = norm8_bwd_blocks(M, N);
  const int threads = N <= kNorm8WarpN ? kNorm8WarpThreads : norm8_threads(N);
  auto kern = N <= kNorm8WarpN ? add_rmsnorm_bwd_kernel<true, kNorm8WarpThreads, 4>
                               : (threads <= 128   ? add_rmsnorm_bwd_kernel<false, 128, 5>
                                  : threads <= 256 ? add_rmsnorm_bwd_kernel<false, 256, 4>
                                  : threads <= 512 ? add_rmsnorm_bwd_kernel<false, 512, 2>
                                                   : add_rmsnorm_bwd_kernel<false, 1024, 1>);
  st = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), threads, 0, s,
                  reinterpret_cast<const __nv_bfloat16*>(dy), reinterpret_cast<const __nv_bfloat16*>(h), r,
                  reinterpret_cast<const __nv_bfloat16*>(gamma), reinterpret_cast<const __nv_bfloat16*>(d_h),
                  reinterpret_cast<__nv_bfloat16*>(dx_out), static_cast<float*>(ws), M, static_cast<int>(N));
  if (st != CODA_OK) return st;
  return launch_pdl(norm8_dgamma_kernel, dim3(static_cast<unsigned>((N + 31) / 32)), 1024, 0, s,
                    static_cast<const float*>(ws), blocks, static_cast<int>(N), dgamma_out);
}

size_t coda_newton_schulz_workspace_size(int64_t batch, int64_t m, int64_t n) {
  if (batch <= 0 || !ns_shape_ok(batch, m, n)) return 0;
  return ns_plan(batch, m, n).bytes;
}

coda_status_t coda_newton_schulz(const float* G, uint16_t* out, int64_t batch, int64_t m, int64_t n, int steps, float a,
                                 float b, float c, float eps, void* ws, size_t ws_bytes, void* stream) {
  CODA_CHECK(ns_shape_ok(batch, m, n) && steps >= 1 && steps <= 100 && eps >= 0.f, CODA_ERR_SHAPE);
  if (batch == 0) return CODA_OK;
  CODA_CHECK(G && out, CODA_ERR_NULL);
  CODA_CHECK(al16(G) && al16(out) && al16(ws), CODA_ERR_ALIGN);
  const NsPlan pl = ns_plan(batch, m, n);
  CODA_CHECK(ws && ws_bytes >= pl.bytes, CODA_ERR_WORKSPACE);
  int dev;
  DevInfo* info;
  coda_status_t st = current_device(&dev, &info);
  if (st != CODA_OK) return st;
  cudaStream_t stm = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  double* sums = reinterpret_cast<double*>(w + pl.sums);
  NsParams p{};
  __half* hi[2] = {reinterpret_cast<__half*>(w + pl.hi[0]), reinterpret_cast<__half*>(w + pl.hi[1])};
  __half* lo[2] = {reinterpret_cast<__half*>(w + pl.lo[0]), reinterpret_cast<__half*>(w + pl.lo[1])};
  for (int i = 0; i < kBufs; ++i) p.diag[i] = reinterpret_cast<float2*>(w + pl.diag[i]);
  p.part = reinterpret_cast<float*>(w + pl.part);
  p.counters = reinterpret_cast<int*>(w + pl.counters);
  p.batch = static_cast<int>(batch);
  p.steps = steps;
  p.tall = pl.tall ? 1 : 0;
  p.a = a;
  p.b = b;
  p.c = c;
  const int64_t s = pl.s;
  bool ok = true;
  for (int i = 0; i < 2; ++i)
    ok = ok && ns_maps(&p.X[i], hi[i], n, m, batch) && tmap3d(&p.Hbox[i], hi[i], false, n, m, batch, 32, 32) &&
         tmap3d(&p.Lbox[i], lo[i], false, n, m, batch, 32, 32);
  for (int i = 0; i < kBufs; ++i) {
    const void* b = w + pl.sym[i];
    ok = ok && ns_maps(&p.S[i], b, s, s, batch) && tmap3d(&p.Sbox[i], b, false, s, s, batch, 32, 32);
  }
  ok = ok && tmap3d(&p.Obox, out, true, n, m, batch, 32, 32);
  if (!ok) return CODA_ERR_INTERNAL;
  const size_t n8 = static_cast<size_t>(m) * n / 8;
  st = launch_pdl(ns_sumsq_kernel, dim3(static_cast<unsigned>(pl.norm_blocks), static_cast<unsigned>(batch)),
                  kNsNormThreads, 0, stm, G, n8, pl.norm_blocks, sums);
  if (st != CODA_OK) return st;
  st = launch_pdl(ns_scale_kernel, dim3(static_cast<unsigned>(pl.norm_blocks), static_cast<unsigned>(batch)),
                  kNsNormThreads, 0, stm, G, n8, pl.norm_blocks, static_cast<const double*>(sums),
                  static_cast<double>(eps), hi[0], lo[0], p.counters,
                  ns_counters(batch));
  if (st != CODA_OK) return st;
  if (pl.tile == 256) return ns_launch<256>(dev, info, p, pl, stm);
  return pl.tile == 128 ? ns_launch<128>(dev, info, p, pl, stm) : ns_launch<64>(dev, info, p, pl, stm);
}

}  // extern "C"
