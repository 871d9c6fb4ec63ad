// Grouped matmul by expert over ragged rows, bf16 on the tensor cores:
//   forward          y[r]  = x[r] W_e^T     W_e [n, k], rows offsets[e] .. offsets[e+1]
//   input gradient   dx[r] = dy[r] W_e
//   weight gradient  dW_e  = sum over the expert's rows of dy[r]^T x[r]
//
// All three read x, dy, W in the layout the caller holds: the tensor cores
// take an operand with its contraction index innermost (x and W forward, dy in
// the input gradient) or outermost (W in the input gradient, dy and x in the
// weight gradient), so no transposed copy of weights or rows exists.
//
// Two SMs (a CTA pair, tcgen05 cta_group::2) compute one 256 x N tile.  Per
// 64-wide K block each CTA stages its 128 of the tile's 256 M rows and half of
// its N rows, 32 KB for 2 x 128 x 256 x 64 products: a third less traffic from
// L2 and into shared memory than a 128 x 256 tile per CTA.
//   forward, input gradient   M = 256 columns of the output (rows of W_e),
//                             N = up to 256 of the expert's rows
//   weight gradient           M = 256 rows of dW_e, N = 256 columns
// The rows as N: an expert's rows are split into equal tiles of at most 256,
// rounded up to 32, so a tile of few rows runs short MMAs and loads few rows
// (an expert of 270 rows costs 320, as M it would cost 384).  The accumulator
// then holds the output transposed (a TMEM lane is an output column); the
// epilogue turns 32 x 32 blocks through shared memory.
//
// Forward and input gradient are fed from L2: a pair's K block of 256 x 256
// moves 64 KB for 512 cycles of MMA, near what L2 gives 148 SMs at once, and a
// tile of 144 rows moves 50 KB for 288.  So with enough units two row tiles of
// an expert share one unit: each W block is staged once for both, and both
// accumulators (256 TMEM columns each) are filled.  Where the last round would
// leave most pairs idle its experts' units are cut in two again (ragged_schedule;
// called back to back, forward of 32 x 512 rows, 2048 x 4096: 245 us, uncut 249;
// of 64 x about 400 rows, 1536 x 2048: 179 and 183).
//
// Measured, bf16, in a burst and after a second of it (the 1000 W cap): 8192 x
// 4096 x 7168 dense forward 311 us (1.55 PFLOP/s) and 367, level with the
// library's product of that shape; 65536 rows of 256 experts, 2048 x 7168: 1.70
// and 2.0 to 2.25 ms; input gradient of 24576 rows of 64 experts, 1408 x 2048: 127
// and 155 us; weight gradients of 32 experts, 16384 skewed rows, 4096 x 7168: 1.01
// and 1.11 ms, bound by stores where experts are small (a pure fill of memory runs
// at 3.9 TB/s).  The loops of the issuing warps are walked by the whole warp with
// one elected lane issuing: from one lane of a diverged branch the same kernel was
// 12-18% slower.
//
// Units are ordered expert-major, then in blocks of N tiles (raster below): pairs
// running side by side share weights and rows through L2, and each expert's weights stream
// from HBM once.  Rows of the next expert inside a load only reach output rows
// that are not stored.  The weight gradient contracts over the rows: in an
// expert's last K block the rows past its end are overwritten with zeros in
// shared memory (in both operands, as 0 * NaN is NaN) before the MMA reads them.
//
// Roles per CTA: warp 0 TMA producer; warp 1 TMEM owner, in the pair's leader
// MMA issuer, in its peer forwarding accumulator releases; warps 2-9 drain the
// accumulators (fp32, rounded once to bf16): with one tile a unit one of them,
// while the next tile accumulates in the other; with two tiles a unit both, and
// the next unit's products wait for that.  Warp 10 (weight gradient) clears the
// rows past an expert's end.
// Waits are bounded and set the status word when they give up.
#include <cuda.h>
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "internal.h"
#include "matmul_util.cuh"
#include "pair_launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int GM = 256, GN = 256, GBK = 64;
constexpr int kHalf = 128;                        // M rows (and at most N rows) of one CTA
constexpr int kChunkBytes = 64 * GBK * 2;         // 64 x 64 operand chunk, contraction outermost
constexpr int kHalfBytes = kHalf * GBK * 2;       // 16 KB
constexpr int kEpiWarps = 8;
constexpr int kStgBytes = 4096;                   // staging per epilogue warp (dw: two of them)
constexpr uint32_t kTmemCols = 2 * GN;

enum GMode { kFwd = 0, kDx = 1, kDw = 2 };

constexpr int pair_threads(int mode) { return 64 + 32 * kEpiWarps + (mode == kDw ? 32 : 0); }
// Operand ring: a stage holds one K block of a CTA's M half and of `share` N
// halves; dw keeps one stage less for a second staging buffer per warp.
__host__ __device__ constexpr int stage_bytes(int share) { return (1 + share) * kHalfBytes; }
__host__ __device__ constexpr int stages(int mode, int share) {
  return share == 2 ? 4 : mode == kDw ? 5 : 6;
}
__host__ __device__ constexpr int staging_bytes(int mode) {
  return kEpiWarps * kStgBytes * (mode == kDw ? 2 : 1);
}
constexpr size_t pair_smem(int mode, int share, int E) {
  return 1024 + (size_t)stages(mode, share) * stage_bytes(share) + staging_bytes(mode) + 256 +
         (mode == kDw ? 0 : (size_t)(E + 1) * 4);
}
static_assert(pair_smem(kFwd, 1, kMatmulMaxGroups) <= 232448, "shared-memory opt-in");
static_assert(pair_smem(kFwd, 2, kMatmulMaxGroups) <= 232448, "shared-memory opt-in");
static_assert(pair_smem(kDw, 1, 0) <= 232448, "shared-memory opt-in");

struct alignas(64) GArgs {
  CUtensorMap tmM;    // fwd: W box {64, 128, 1}; dx: W box {64, 64, 1}; dw: dy box {64, 64}
  CUtensorMap tmN;    // fwd, dx: rows box {64, 128}; dw: x box {64, 64}
  CUtensorMap tmNs[3];  // fwd, dx: rows boxes {64, 16}, {64, 32}, {64, 64}
  CUtensorMap tmOut;  // fwd, dx: out [R, m] box {32, 32}, not swizzled; dw: dW box {64, 32, 1}
  const int32_t* offsets;
  __nv_bfloat16* out;
  uint32_t* status;
  int E, R;
  int m;     // fwd, dx: output columns; dw: n
  int cols;  // dw: k
  int kdim;  // fwd, dx: contraction length
};

// Equal row tiles of an expert: at most 256 rows each, a multiple of 32.
__device__ __forceinline__ int row_tile(int rows, int tiles) {
  return ((rows + tiles - 1) / tiles + 31) & ~31;
}

// Tile (m, n) of an expert's unit `local`: blocks of kBlockN N tiles, within a
// block M tile by M tile.  The pairs at work then share kBlockN tiles of the N
// operand and as many of the M operand as there are pairs to a block row, in
// place of the whole N operand.  (us with no blocks, blocks of 4, 8, 12, 16:
// forward 8192 x 4096 x 7168 385, 367, 361, 365, 362; 16384 x 2048 x 2048 112, 106,
// 107, 108, 108; weight gradients of 8192 rows, 7168 x 7168 694, 669, 650, 656, 652,
// of 32 experts with 16384 skewed rows, 4096 x 7168 1164, 1144, 1135, 1137, 1138.
// Four more shapes differ by less than 3% between blocks of 8 to 16.)
constexpr int kBlockN = 12;
__device__ __forceinline__ void raster(int local, int MT, int NT, int& m, int& n) {
  const int b = local / (MT * kBlockN), rest = local - b * (MT * kBlockN);
  const int wide = min(kBlockN, NT - b * kBlockN);
  m = rest / wide;
  n = b * kBlockN + rest - m * wide;
}

// A CTA's N rows of one K block, `half` of them (a multiple of 16, at most
// 128), in at most two copies: many copies of 16 rows each took 2-3x longer,
// one box of the next size up moves up to 60% more than needed.
struct RowBoxes {
  int first, second;  // index of the box (16 << i rows), -1: none
  __device__ __forceinline__ explicit RowBoxes(int half) {
    first = half > 96 ? 3 : half > 64 || half == 64 ? 2 : half >= 32 ? 1 : 0;
    const int left = half > 96 ? 0 : half - (16 << first);
    second = left <= 0 ? -1 : left > 16 ? 1 : 0;
  }
  __device__ __forceinline__ int rows() const {
    return (16 << first) + (second < 0 ? 0 : 16 << second);
  }
};

// kShare: row tiles per unit (fwd, dx: 1 or 2; dw: 1)
template <int kMode, int kShare>
__global__ void __launch_bounds__(pair_threads(kMode), 1) grouped_matmul_pair_kernel(
    const __grid_constant__ GArgs args) {
  constexpr int kStages = stages(kMode, kShare), kStageBytes = stage_bytes(kShare);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = base + (size_t)kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + staging_bytes(kMode));
  uint64_t* full = bars;             // [kStages] leader: both CTAs' copies have landed
  uint64_t* empty = full + kStages;    // [kStages] each CTA: the MMAs have read the stage
  uint64_t* tfull = empty + kStages;   // [2] each CTA: accumulator complete
  uint64_t* tempty = tfull + 2;      // [2] leader: the peer's epilogue has read it
  uint64_t* edone = tempty + 2;      // [2] each CTA: its epilogue warps have read it
  uint64_t* drain = edone + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  // dw: [kStages] each CTA: its last-block copies have landed; leader: cleared
  uint64_t* tland = reinterpret_cast<uint64_t*>(tmem_holder) + 1;
  uint64_t* tclear = tland + kStages;
  int* start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);
  int* single = start - 1;  // fwd, dx: from this expert on a unit is one row tile

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int MT = (args.m + GM - 1) / GM;
  const int NT = (args.cols + GN - 1) / GN;  // dw

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      if constexpr (kMode == kDw) {
        mbar_init(&tland[s], 1);
        mbar_init(&tclear[s], 2);
      }
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 1);
      mbar_init(&edone[a], kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_2sm(tmem_holder, kTmemCols);
    tmem_relinquish_2sm();
  }
  if constexpr (kMode != kDw) {
    if (warp == 0) {
      const int from = ragged_schedule(args.offsets, args.E, args.R, kShare * GN, MT, start,
                                       args.status, kShare == 2 ? npairs : 0);
      if (lane == 0) *single = from;
    }
  }
  tc_fence_before();
  __syncthreads();
  mm_cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = kMode == kDw ? args.E * MT * NT : start[args.E];

  struct Unit {
    int g, first, rows;  // expert, its first row, its rows
    int m0;              // first M index of the tile
    int n0;              // first N index
    int tiles;           // N tiles (accumulators): 1, or 2 (fwd, dx)
    int width[2];        // N of each, a multiple of 32
    int kb;              // K blocks
  };
  auto decode = [&](int u) {
    Unit t;
    bool bad = false;
    t.tiles = 1;
    t.width[1] = 0;
    if constexpr (kMode == kDw) {
      t.g = u / (MT * NT);
      int m, n;
      raster(u - t.g * (MT * NT), MT, NT, m, n);
      t.m0 = m * GM;
      t.n0 = n * GN;
      t.width[0] = min(GN, (args.cols - t.n0 + 31) & ~31);
      t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
      t.kb = (t.rows + GBK - 1) / GBK;
      if (bad && m == 0 && n == 0 && tid == 0) atomicOr(args.status, kErrBadIndex);
    } else {
      t.g = ragged_group(start, args.E, u);
      t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
      const int tiles = (t.rows + GN - 1) / GN, local = u - start[t.g];
      const int each = kShare == 2 && t.g < *single ? 2 : 1;  // row tiles per unit
      const int runs = (tiles + each - 1) / each;  // units per M tile
      int m, n;
      raster(local, MT, runs, m, n);
      const int w = row_tile(t.rows, tiles), t0 = n * each;
      t.m0 = m * GM;
      t.n0 = t0 * w;
      t.width[0] = min(w, (t.rows - t.n0 + 31) & ~31);
      if (each == 2 && t0 + 1 < tiles) {
        t.tiles = 2;
        t.width[1] = min(w, (t.rows - t.n0 - w + 31) & ~31);
      }
      t.kb = (args.kdim + GBK - 1) / GBK;
    }
    return t;
  };
  // dw: the unit's last K block holds rows past the expert's end in its last
  // 16-row step, which warp 10 clears
  auto ragged_end = [&](const Unit& t) { return kMode == kDw && (t.rows & 15) != 0; };

  if (warp == 0) {
    // ---- TMA producer: like the MMA issuer, the warp walks the loop together
    // and one lane issues ----
    if (elect_one()) {
      tma_prefetch_desc(&args.tmM);
      tma_prefetch_desc(&args.tmN);
    }
    __syncwarp();
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    uint32_t tissued = 0, tphase = 0;  // last blocks: per stage, parity of the next use
    bool ok = true;
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);  // the leader's barriers
    Unit t{};
    if (pair < total) t = decode(pair);
    for (int u = pair; u < total && ok; u += npairs) {
      const int mrow = t.m0 + (int)rank * kHalf;
      Unit next = t;
      if (t.kb == 0 && u + npairs < total) next = decode(u + npairs);
      // dw: 64-wide chunks of this CTA's columns; fwd, dx: its rows of each tile
      const int half = t.width[0] / 2, nrow = t.n0 + (int)rank * half;
      const int nchunks = (half + 63) / 64;
      const RowBoxes box0(half), box1(t.tiles == 2 ? t.width[1] / 2 : 16);
      const int row0 = t.first + nrow;
      const int row1 = t.first + t.n0 + t.width[0] + (int)rank * (t.width[1] / 2);
      const uint32_t bytes =
          kHalfBytes +
          (uint32_t)(kMode == kDw
                         ? nchunks * kChunkBytes
                         : (box0.rows() + (t.tiles == 2 ? box1.rows() : 0)) * (GBK * 2));
      for (int kb = 0; kb < t.kb; ++kb) {
        ok = mm_wait(&empty[stage], phase ^ 1u, args.status);
        if (!ok) break;
        uint8_t* sm = base + (size_t)stage * kStageBytes;
        uint8_t* sn = sm + kHalfBytes;
        const uint32_t fbar = full0 + 8u * (uint32_t)stage;
        const bool last = kb + 1 == t.kb && ragged_end(t);
        if (elect_one()) {
          if constexpr (kMode == kDw) {
            const int r = t.first + kb * GBK;
            if (last) {
              // lands on this CTA's own barrier; `full` only advances
              mbar_arrive_expect_tx(&tland[stage], bytes);
              for (int c = 0; c < 2; ++c)
                tma_load_2d(sm + c * kChunkBytes, &args.tmM, mrow + 64 * c, r, &tland[stage]);
              for (int c = 0; c < nchunks; ++c)
                tma_load_2d(sn + c * kChunkBytes, &args.tmN, nrow + 64 * c, r, &tland[stage]);
              if (leader) mbar_arrive(&full[stage]);
            } else {
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
              for (int c = 0; c < 2; ++c)
                tma_load_2d_2sm(sm + c * kChunkBytes, &args.tmM, mrow + 64 * c, r, fbar);
              for (int c = 0; c < nchunks; ++c)
                tma_load_2d_2sm(sn + c * kChunkBytes, &args.tmN, nrow + 64 * c, r, fbar);
            }
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
            if constexpr (kMode == kFwd) {
              tma_load_3d_2sm(sm, &args.tmM, kb * GBK, mrow, t.g, fbar);
            } else {
              tma_load_3d_2sm(sm, &args.tmM, mrow, kb * GBK, t.g, fbar);
              tma_load_3d_2sm(sm + kChunkBytes, &args.tmM, mrow + 64, kb * GBK, t.g, fbar);
            }
            auto rows_in = [&](uint8_t* dst, const RowBoxes& box, int row) {
              tma_load_2d_2sm(dst, box.first == 3 ? &args.tmN : &args.tmNs[box.first], kb * GBK,
                              row, fbar);
              if (box.second >= 0)
                tma_load_2d_2sm(dst + (16 << box.first) * (GBK * 2), &args.tmNs[box.second],
                                kb * GBK, row + (16 << box.first), fbar);
            };
            rows_in(sn, box0, row0);
            if (kShare == 2 && t.tiles == 2) rows_in(sn + kHalfBytes, box1, row1);
          }
        }
        __syncwarp();
        if (last) {
          tissued |= 1u << stage;
          tphase ^= 1u << stage;
        }
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (kb == 0 && u + npairs < total) next = decode(u + npairs);
      }
      t = next;
    }
    // every copy has landed before the CTA exits, also where the warp that reads
    // them gave up; the leader's barriers count the peer's copies too
    for (int s = 0; s < kStages; ++s) {
      if (leader && ((issued >> s) & 1u)) mm_drain(&full[s], (parity >> s) & 1u, args.status);
      if (kMode == kDw && ((tissued >> s) & 1u))
        mm_drain(&tland[s], ((tphase >> s) & 1u) ^ 1u, args.status);
    }
    mm_settle(args.status);
  } else if (warp == 1) {
    if (leader) {
      // ---- MMA issuer: the warp walks the loop together, so that addresses stay
      // warp-uniform, and one lane issues ----
      constexpr uint32_t kMajor = (kMode == kDx ? kIdescAMn : 0u) |
                                  (kMode == kDw ? kIdescAMn | kIdescBMn : 0u);
      constexpr bool kAInner = kMode == kFwd, kBInner = kMode != kDw;
      const uint32_t ring = smem_u32(base);
      const uint64_t ad0 = kAInner ? smem_desc_sw128(ring) : smem_desc_mn_sw128(ring, kChunkBytes);
      const uint64_t bd0 = kBInner ? smem_desc_sw128(ring + kHalfBytes)
                                   : smem_desc_mn_sw128(ring + kHalfBytes, kChunkBytes);
      const uint32_t a_hi = desc_hi(ad0), b_hi = desc_hi(bd0);
      constexpr uint32_t kAStep = (kAInner ? 32 : 2048) / 16, kBStep = (kBInner ? 32 : 2048) / 16;
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      int use = 0;  // accumulator uses so far
      bool ok = true;
      Unit t{};
      if (pair < total) t = decode(pair);
      for (int u = pair; u < total && ok; u += npairs) {
        for (int j = 0; j < t.tiles && ok; ++j) {
          const uint32_t ap = (((use + j) >> 1) & 1) ^ 1u;
          ok = mm_wait(&edone[(use + j) & 1], ap, args.status) &&
               mm_wait(&tempty[(use + j) & 1], ap, args.status);
        }
        if (!ok) break;
        tc_fence_after();
        Unit next = t;
        if (t.kb == 0 && u + npairs < total) next = decode(u + npairs);
        for (int kb = 0; kb < t.kb && ok; ++kb) {
          int steps = GBK / 16;
          if constexpr (kMode == kDw) {
            if (kb + 1 == t.kb) {
              steps = (t.rows - kb * GBK + 15) / 16;
              if (ragged_end(t)) {
                ok = mm_wait<true>(&tclear[stage], (tphase >> stage) & 1u, args.status);
                if (!ok) break;
                tphase ^= 1u << stage;
              }
            }
          }
          ok = mm_wait(&full[stage], phase, args.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t off = (uint32_t)stage * (kStageBytes / 16);
          const uint32_t a_lo = desc_lo(ad0) + off, b_lo = desc_lo(bd0) + off;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < kShare; ++j) {
              if (j >= t.tiles) break;
              const uint32_t idesc = idesc_bf16_f32(GM, t.width[j]) | kMajor;
              const uint32_t d_tmem = tmem_base + ((use + j) & 1) * GN;
#pragma unroll
              for (int k = 0; k < GBK / 16; ++k)
                if (kMode != kDw || k < steps)
                  mma_bf16_2sm_parts(d_tmem, a_lo + k * kAStep, a_hi,
                                     b_lo + j * (kHalfBytes / 16) + k * kBStep, b_hi, idesc,
                                     k == 0 ? (uint32_t)(kb != 0) : 1u);
            }
            mma_commit_2sm_mc(&empty[stage], 0x3);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          // the next unit is looked up while this one's products run
          if (kb == 0 && u + npairs < total) next = decode(u + npairs);
        }
        if (!ok) break;
        if (elect_one()) {
          for (int j = 0; j < t.tiles; ++j)  // without K blocks: arrives at once
            mma_commit_2sm_mc(&tfull[(use + j) & 1], 0x3);
        }
        __syncwarp();
        use += t.tiles;
        t = next;
      }
      if (elect_one()) mma_commit_2sm(drain);
      __syncwarp();
      mm_drain(drain, 0, args.status);
    } else if (!leader && lane == 0) {
      // forward each accumulator release of this CTA's epilogue to the leader
      const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
      int use = 0;
      bool ok = true;
      for (int u = pair; u < total && ok; u += npairs) {
        const Unit t = decode(u);
        for (int j = 0; j < t.tiles && ok; ++j, ++use) {
          ok = mm_wait_thread(&edone[use & 1], (use >> 1) & 1, args.status, contraction_ms(t.kb));
          if (ok) mbar_arrive_peer(tempty0 + 8u * (uint32_t)(use & 1));
        }
      }
    }
  } else if (kMode == kDw && warp == 2 + kEpiWarps) {
    // ---- rows past an expert's end, in its last 16-row step: one 128-byte line
    // per row and 64-wide chunk ----
    int kbs = 0;    // K blocks of the units so far
    int since = 0;  // of those after the last wait
    uint32_t tphase = 0;
    const uint32_t tclear0 = mapa_shared(smem_u32(&tclear[0]), 0);
    for (int u = pair; u < total; u += npairs) {
      const Unit t = decode(u);
      kbs += t.kb;
      since += t.kb;
      if (!ragged_end(t)) continue;
      const int stage = (kbs - 1) % kStages;
      if (!mm_wait(&tland[stage], (tphase >> stage) & 1u, args.status, contraction_ms(since)))
        break;
      since = 0;
      tphase ^= 1u << stage;
      uint8_t* sm = base + (size_t)stage * kStageBytes;
      const int valid = t.rows - (t.kb - 1) * GBK, lines = ((valid + 15) & ~15) - valid;
      for (int i = lane; i < lines * (kStageBytes / kChunkBytes) * 8; i += 32) {
        const int piece = i & 7, line = (i >> 3) % lines, c = (i >> 3) / lines;
        *reinterpret_cast<uint4*>(sm + c * kChunkBytes + (valid + line) * 128 + piece * 16) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tclear0 + 8u * (uint32_t)stage);
    }
  } else {
    // ---- epilogue ----
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quadrant; two warps each
    uint8_t* stg = staging + (size_t)(warp - 2) * (staging_bytes(kMode) / kEpiWarps);
    int use = 0, buf = 0;
    bool ok = true;
    for (int u = pair; u < total && ok; u += npairs) {
      const Unit t = decode(u);
      const int m = t.m0 + (int)rank * kHalf + q * 32;  // this warp's first M index
      for (int j = 0; j < t.tiles; ++j, ++use) {
        const int acc = use & 1;
        ok = mm_wait(&tfull[acc], (use >> 1) & 1, args.status, contraction_ms(t.kb));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * GN;
        if (kMode == kDw && m < args.m) {
          // 32 rows of dW_e, 64 columns at a time
#pragma unroll 1
          for (int c = half * 128; c < half * 128 + 128; c += 64, buf ^= 1) {
            if (t.n0 + c >= args.cols) break;
            uint32_t p[32];
            if (t.kb == 0) {  // an expert without rows: a zero gradient
#pragma unroll
              for (int i = 0; i < 32; ++i) p[i] = 0u;
            } else {
              uint32_t v0[32], v1[32];
              __syncwarp();  // lane 0 has stored the piece before
              tmem_ld32(taddr + c, v0);
              tmem_ld32(taddr + c + 32, v1);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                p[i] = bf16x2_bits(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]));
                p[16 + i] =
                    bf16x2_bits(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]));
              }
            }
            uint8_t* tile = stg + buf * kStgBytes;
            if (lane == 0) bulk_wait_read_but_one();  // this buffer's last store has read it
            __syncwarp();
            uint8_t* my = tile + lane * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(my + ((i ^ (lane & 7)) << 4)) =
                  make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&args.tmOut, tile, t.n0 + c, m, t.g);
              bulk_commit_group();
            }
          }
        }
        if (kMode != kDw && m < args.m) {
          // lane = output column m + lane, register = row: blocks of 32 rows,
          // alternately by the two warps of a quadrant, turned in the staging
          // buffer (row i at 64 i, column at 2 lane)
          const int n0 = t.n0 + (j == 0 ? 0 : t.width[0]);
          const int width = t.width[j];
#pragma unroll 1
          for (int b = half * 32; b < width; b += 64, buf ^= 1) {
            const int left = t.rows - n0 - b;
            if (left <= 0) break;
            uint32_t v[32];
            __syncwarp();  // lane 0 has stored the block before
            tmem_ld32(taddr + b, v);
            tmem_wait_ld();
            uint8_t* tile = stg + buf * 2048;
            if (lane == 0) bulk_wait_read_but_one();  // this buffer's last store has read it
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              *reinterpret_cast<__nv_bfloat16*>(tile + i * 64 + lane * 2) =
                  __float2bfloat16_rn(__uint_as_float(v[i]));
            const int r = t.first + n0 + b;
            if (left >= 32) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&args.tmOut, tile, m, r);
                bulk_commit_group();
              }
            } else {
              // the expert's last rows: 16 bytes a lane, 8 rows at a time.  Their
              // piece is an empty group: the buffers' turns are counted in groups
              if (lane == 0) bulk_commit_group();
              __syncwarp();
              const int c = (lane & 3) * 8;
              for (int i = lane >> 2; i < left; i += 8)
                if (m + c < args.m)
                  *reinterpret_cast<uint4*>(args.out + (size_t)(r + i) * (size_t)args.m + m + c) =
                      *reinterpret_cast<const uint4*>(tile + i * 64 + c * 2);
              __syncwarp();
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&edone[acc]);
      }
    }
    if (lane == 0) bulk_wait_all();  // the staging buffers outlive the stores that read them
  }

  tc_fence_before();
  __syncthreads();
  mm_cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem_base, kTmemCols);
  }
}

template <int kMode, int kShare>
cudaError_t launch_pair(const GArgs& a, long long units, cudaStream_t st) {
  return launch_pairs(grouped_matmul_pair_kernel<kMode, kShare>, a, pair_smem(kMode, kShare, a.E),
                      pair_smem(kMode, kShare, kMode == kDw ? 0 : kMatmulMaxGroups),
                      pair_threads(kMode), units, "grouped matmul", st);
}

}  // namespace

int launch_grouped_matmul_bf16(int mode, const void* rows, int R, const int32_t* offsets, int E,
                               const void* w, int n, int k, void* out, void* ws,
                               cudaStream_t st) {
  if (matmul_is_narrow(R, E, mode == kDx ? k : n))
    return launch_matmul_narrow(mode == kDx, rows, 0, nullptr, 0, R, offsets, E, w, nullptr, n, k,
                                out, ws, st);
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GArgs a{};
  a.offsets = offsets;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<uint32_t*>(ws);
  a.E = E;
  a.R = R;
  a.m = mode == kDx ? k : n;
  a.kdim = mode == kDx ? n : k;
  const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)k * 2, (uint64_t)k * n * 2};
  const uint32_t box[3] = {64, mode == kDx ? 64u : 128u, 1};
  if (!make_map_nd(&a.tmM, w, BF, 3, dims, strides, box) ||
      !make_map(&a.tmN, rows, BF, 2, a.kdim, R, 64, 128) ||
      !make_map(&a.tmNs[0], rows, BF, 2, a.kdim, R, 64, 16) ||
      !make_map(&a.tmNs[1], rows, BF, 2, a.kdim, R, 64, 32) ||
      !make_map(&a.tmNs[2], rows, BF, 2, a.kdim, R, 64, 64) ||
      !make_map_swizzled(&a.tmOut, out, BF, 2, a.m, R, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE)) {
    note_text("grouped matmul: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const long long tiles = R / GN + (R < E ? R : E);  // no more row tiles than this
  const long long units = tiles * ((a.m + GM - 1) / GM);
  const bool share = units >= 8 * (num_sms() / 2);
  const cudaError_t e =
      mode == kFwd
          ? (share ? launch_pair<kFwd, 2>(a, units, st) : launch_pair<kFwd, 1>(a, units, st))
          : (share ? launch_pair<kDx, 2>(a, units, st) : launch_pair<kDx, 1>(a, units, st));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_grouped_matmul_dw_bf16(const void* dy, const void* x, int R, const int32_t* offsets,
                                  int E, int n, int k, void* dw, void* ws, cudaStream_t st) {
  if (matmul_dw_splits(R, E, n, k) > 1)
    return launch_matmul_dw_small(dy, x, R, offsets, E, n, k, dw, ws, st);
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GArgs a{};
  a.offsets = offsets;
  a.out = static_cast<__nv_bfloat16*>(dw);
  a.status = static_cast<uint32_t*>(ws);
  a.E = E;
  a.R = R;
  a.m = n;
  a.cols = k;
  const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)k * 2, (uint64_t)k * n * 2};
  const uint32_t box[3] = {64, 32, 1};
  if (!make_map(&a.tmM, dy, BF, 2, n, R, 64, 64) || !make_map(&a.tmN, x, BF, 2, k, R, 64, 64) ||
      !make_map_nd(&a.tmOut, dw, BF, 3, dims, strides, box)) {
    note_text("grouped matmul weight gradient: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const long long units = (long long)E * ((n + GM - 1) / GM) * ((k + GN - 1) / GN);
  return launch_pair<kDw, 1>(a, units, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
