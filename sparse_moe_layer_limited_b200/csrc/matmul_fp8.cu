// Block-scaled FP8 matmul, dense or by expert over ragged rows:
//   forward         y[r, j]  = sum_b sa[r, b] sw[e, j/128, b] sum_{i in b} qa[r, i] qw[e, j, i]
//   input gradient  dx[r, i] = sum_b sa[r, b] sw[e, b, i/128] sum_{j in b} qa[r, j] qw[e, j, i]
// b runs over the 128-wide blocks of the contraction index.  Rows carry one
// fp32 scale per 1x128 tile (E4M3 or E5M2 codes), the weight one per 128x128
// block (E4M3).  The input gradient reads the same codes and scales as the
// forward: its weight operand has the contraction index outermost.
//
// Each 128-wide slice of a 128 x 256 output tile is one product on the tensor
// cores (fp32) into one of two 256-column TMEM buffers; eight epilogue warps
// multiply it by the two scales and add it to fp32 registers, 128 running sums
// a thread, while the next slice fills the other buffer.  The scales are read
// from global memory two slices ahead.  The result is rounded once to bf16.
//
// 8192 x 4096 x 7168: 238 us in a burst (2.02 PFLOP/s), 280 us under sustained
// power; 16411 skewed rows of 64 experts, 2048 x 7168: input gradient 365 and 427
// to 440 us, forward 336 and 398.  Of a slice's 1100 cycles 512 are MMA; without
// the promotion's reads of TMEM the first took 197 us (when the kernel took 245),
// with half the operand traffic as well 170 us, without the multiply-adds no less
// than with them.  The next unit and its first scales are looked up before a unit
// is stored, in 32-column pieces through two buffers.  Measured and not taken: CTA
// pairs (a third less operand traffic: 240 us dense, but 256-row tiles cost ragged
// experts 25%).
//
// Also here: the quantisers that make the codes, per 1x128 tile of a row and
// per 128x128 block (tile_scale below).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "epilogue.cuh"
#include "fp8_util.cuh"
#include "internal.h"
#include "matmul_util.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int PBM = 128, PBN = 256, PBK = 128;
constexpr int PStages = 4;
constexpr int PABytes = PBM * PBK;
constexpr int PStageBytes = PABytes + PBN * PBK;
constexpr int PEpiWarps = 8;
constexpr int PThreads = 128 + 32 * PEpiWarps;  // a warpgroup of control warps, two of epilogue
constexpr int PStg = 4096;      // per epilogue warp: two pieces of 32 rows x 32 bf16
constexpr int PCols = PBN / 2;  // columns per epilogue warp
constexpr int kAhead = 2;       // slices whose scales are loaded together

constexpr size_t fp8_mm_smem(int E) {
  return 1024 + (size_t)PStages * PStageBytes + PEpiWarps * PStg + 256 + (size_t)(E + 1) * 4;
}
static_assert(fp8_mm_smem(kMatmulMaxGroups) <= 232448, "shared-memory opt-in");

struct alignas(64) PArgs {
  CUtensorMap tmA;    // row codes [R, K], box {128, 128}
  CUtensorMap tmA32;  // the same, box {128, 32}
  CUtensorMap tmB;    // weight codes [E, n, k]: fwd box {128, 256, 1}, dx box {128, 128, 1}
  CUtensorMap tmB64;  // fwd: box {128, 64, 1}, for a narrow last column tile
  CUtensorMap tmOut;  // out [R, cols] bf16, box {32, 32} (cols % 8 == 0)
  const int32_t* offsets;
  const float* sa;  // [KB, sa_ld]
  const float* sw;  // [E, ceil(n/128), ceil(k/128)]
  __nv_bfloat16* out;
  uint32_t* status;
  long long sa_ld;
  int E, R;
  int cols, kdim;
  int nb, kb;     // blocks along n and k
  uint32_t a_fmt;
};

__device__ __forceinline__ void fma2(float& a0, float& a1, float x0, float x1, float s) {
  asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
      "mov.b64 rc, {%0, %1};\n\tfma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1), "f"(s));
}

template <bool kDx>
__global__ void __launch_bounds__(PThreads, 1) matmul_fp8_kernel(
    const __grid_constant__ PArgs args) {
  constexpr int kChunkCols = kDx ? 128 : 64;           // weight columns per TMA box
  constexpr int kChunk = kChunkCols * PBK;             // its bytes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = base + (size_t)PStages * PStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + PEpiWarps * PStg);
  uint64_t* full = bars;
  uint64_t* empty = full + PStages;
  uint64_t* sfull = empty + PStages;  // [2] slice buffer written
  uint64_t* sempty = sfull + 2;       // [2] slice buffer read
  uint64_t* drain = sempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  int* start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int NT = (args.cols + PBN - 1) / PBN;
  const int KB = (args.kdim + PBK - 1) / PBK;

  if (tid == 0) {
    for (int s = 0; s < PStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sfull[a], 1);
      mbar_init(&sempty[a], PEpiWarps);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 0) ragged_schedule(args.offsets, args.E, args.R, PBM, NT, start, args.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = start[args.E];

  struct Unit {
    int g, first, rows, m, n;
  };
  auto decode = [&](int u) {
    Unit t;
    bool bad = false;
    t.g = ragged_group(start, args.E, u);
    t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
    const int mt = (t.rows + PBM - 1) / PBM;
    const int local = u - start[t.g];
    t.n = local / mt;
    t.m = local - t.n * mt;
    return t;
  };

  // 384 threads launch with 168 registers each; the control warps hand 112 of
  // theirs to the epilogue: 128 * 56 + 256 * 224 = 384 * 168
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---- TMA producer: the warp walks the loop together, so that addresses stay
      // warp-uniform, and one lane issues ----
      if (elect_one()) {
        tma_prefetch_desc(&args.tmA);
        tma_prefetch_desc(&args.tmB);
      }
      __syncwarp();
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      Unit t{};
      if (blockIdx.x < total) t = decode(blockIdx.x);
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        Unit next = t;
        const int nc = min(PBN / kChunkCols, (args.cols - t.n * PBN + kChunkCols - 1) / kChunkCols);
        const int na = min(4, (t.rows - t.m * PBM + 31) / 32);
        const int r = t.first + t.m * PBM;
        const uint32_t bytes = (uint32_t)(nc * kChunk + na * 32 * PBK);
        for (int kb = 0; kb < KB; ++kb) {
          ok = mm_wait(&empty[stage], phase ^ 1u, args.status);
          if (!ok) break;
          uint8_t* sa = base + (size_t)stage * PStageBytes;
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[stage], bytes);
            if (na == 4) {
              tma_load_2d(sa, &args.tmA, kb * PBK, r, &full[stage]);
            } else {
              for (int c = 0; c < na; ++c)
                tma_load_2d(sa + c * (32 * PBK), &args.tmA32, kb * PBK, r + 32 * c, &full[stage]);
            }
            if (nc == PBN / kChunkCols && kDx == 0) {
              tma_load_3d(sa + PABytes, &args.tmB, kb * PBK, t.n * PBN, t.g, &full[stage]);
            } else {
              for (int c = 0; c < nc; ++c) {
                const int col = t.n * PBN + kChunkCols * c;
                if constexpr (kDx)
                  tma_load_3d(sa + PABytes + c * kChunk, &args.tmB, col, kb * PBK, t.g,
                              &full[stage]);
                else
                  tma_load_3d(sa + PABytes + c * kChunk, &args.tmB64, kb * PBK, col, t.g,
                              &full[stage]);
              }
            }
          }
          __syncwarp();
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == PStages) {
            stage = 0;
            phase ^= 1u;
          }
          // the next unit is looked up while this one's copies are in flight
          if (kb == 0 && u + (int)gridDim.x < total) next = decode(u + gridDim.x);
        }
        t = next;
      }
      // every copy has landed before the CTA exits, also where the MMA warp gave up
      for (int s = 0; s < PStages; ++s)
        if ((issued >> s) & 1u) mm_drain(&full[s], (parity >> s) & 1u, args.status);
    } else if (warp == 1) {
      // ---- MMA issuer, one TMEM buffer per slice ----
      const uint32_t ring = smem_u32(base);
      const uint64_t ad0 = smem_desc_sw128(ring);
      const uint64_t bd0 = kDx ? smem_desc_mn_sw128(ring + PABytes, kChunk)
                               : smem_desc_sw128(ring + PABytes);
      const uint32_t a_hi = desc_hi(ad0), b_hi = desc_hi(bd0);
      constexpr uint32_t kBStep = (kDx ? 4096 : 32) / 16;
      int stage = 0;
      uint32_t phase = 0, slice = 0;
      bool ok = true;
      Unit t{};
      if (blockIdx.x < total) t = decode(blockIdx.x);
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        Unit next = t;
        const int width = min(PBN, args.cols - t.n * PBN);
        const uint32_t idesc = idesc_f8_f32(PBM, (width + 15) / 16 * 16, args.a_fmt, kF8E4M3) |
                               (kDx ? kIdescBMn : 0u);
        for (int kb = 0; kb < KB; ++kb, ++slice) {
          const uint32_t sb = slice & 1u;
          ok = mm_wait(&sempty[sb], ((slice >> 1) & 1u) ^ 1u, args.status) &&
               mm_wait(&full[stage], phase, args.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t off = (uint32_t)stage * (PStageBytes / 16);
          const uint32_t a_lo = desc_lo(ad0) + off, b_lo = desc_lo(bd0) + off;
          if (elect_one()) {
  #pragma unroll
            for (int k = 0; k < PBK / 32; ++k)
              mma_f8_parts(tmem_base + sb * PBN, a_lo + k * 2, a_hi, b_lo + k * kBStep, b_hi, idesc,
                           k != 0);
            mma_commit(&empty[stage]);
            mma_commit(&sfull[sb]);
          }
          __syncwarp();
          if (++stage == PStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (kb == 0 && u + (int)gridDim.x < total) next = decode(u + gridDim.x);
        }
        t = next;
      }
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mm_drain(drain, 0, args.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- promotion and epilogue: two warps per lane quadrant, 128 columns each ----
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stg = staging + (size_t)(warp - 4) * PStg;
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + half * PCols;
    const bool tma_out = (args.cols & 7) == 0;
    uint32_t slice = 0;
    int buf = 0;
    bool ok = true;
    // the unit at hand, as this warp sees it
    struct View {
      int r0, left, col0;  // its first row of the expert, the rows from there, its first column
      bool live;           // it has rows and columns (the same for the whole warp)
      const float *sa, *sw;
    };
    const int sw_step = kDx ? args.kb : 1;
    auto view = [&](const Unit& t) {
      View v;
      v.r0 = t.m * PBM + q * 32;
      v.left = t.rows - v.r0;
      v.col0 = t.n * PBN + half * PCols;
      v.live = v.left > 0 && v.col0 < args.cols;
      // scales: sa[kb][row], and the weight block of this warp's columns
      v.sa = args.sa + min(t.first + v.r0 + lane, args.R - 1);
      v.sw = args.sw + (size_t)t.g * args.nb * args.kb +
             (kDx ? (size_t)(v.col0 / 128) : (size_t)(v.col0 / 128) * args.kb);
      return v;
    };
    // loaded kAhead slices ahead (a unit's first ones before the unit before it
    // is stored), multiplied when used
    float row_sc[kAhead], w_sc[kAhead], row_nx[kAhead], w_nx[kAhead];
    auto scales = [&](const View& v, int kb) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        row_nx[j] = w_nx[j] = 0.f;
        if (v.live && kb + j < KB) {
          row_nx[j] = __ldg(v.sa + (size_t)(kb + j) * args.sa_ld);
          w_nx[j] = __ldg(v.sw + (size_t)(kb + j) * sw_step);
        }
      }
    };
    Unit t{};
    if (blockIdx.x < total) t = decode(blockIdx.x);
    View v{};
    if (blockIdx.x < total) {
      v = view(t);
      scales(v, 0);
    }
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
      float acc[PCols];
#pragma unroll
      for (int i = 0; i < PCols; ++i) acc[i] = 0.f;
      for (int kb = 0; kb < KB && ok; kb += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          row_sc[j] = row_nx[j];
          w_sc[j] = w_nx[j];
        }
        if (kb + kAhead < KB) scales(v, kb + kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (kb + j >= KB) break;
          const float sc = row_sc[j] * w_sc[j];
          const uint32_t sb = slice & 1u;
          if (!mm_wait(&sfull[sb], (slice >> 1) & 1u, args.status)) {
            ok = false;
            break;
          }
          ++slice;
          tc_fence_after();
          if (v.live) {
#pragma unroll
            for (int c = 0; c < PCols; c += 64) {
              uint32_t p[4][16];
#pragma unroll
              for (int l = 0; l < 4; ++l) tmem_ld16(tbase + sb * PBN + c + 16 * l, p[l]);
              tmem_wait_ld();
              if (c + 64 == PCols) {  // the slice is in registers: hand the buffer back
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[sb]);
              }
#pragma unroll
              for (int l = 0; l < 4; ++l)
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                  fma2(acc[c + 16 * l + i], acc[c + 16 * l + i + 1], __uint_as_float(p[l][i]),
                       __uint_as_float(p[l][i + 1]), sc);
            }
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[sb]);
          }
        }
      }
      if (!ok) break;
      const Unit done = t;
      const View d = v;
      if (u + (int)gridDim.x < total) {
        t = decode(u + gridDim.x);
        v = view(t);
        scales(v, 0);
      }
      if (!d.live) continue;
      // 32 columns at a time through two staging buffers (64-byte rows, their
      // 16-byte chunks swizzled as the store reads them)
#pragma unroll
      for (int c = 0; c < PCols; c += 32, buf ^= 1) {
        const int col = d.col0 + c;
        if (col >= args.cols) break;
        uint8_t* tile = stg + buf * (PStg / 2);
        if (lane == 0) bulk_wait_read_but_one();  // this buffer's last store has read it
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* a = acc + c + 8 * j;
          *reinterpret_cast<uint4*>(tile + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(bf16x2_bits(a[0], a[1]), bf16x2_bits(a[2], a[3]),
                         bf16x2_bits(a[4], a[5]), bf16x2_bits(a[6], a[7]));
        }
        if (tma_out && d.left >= 32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&args.tmOut, tile, col, done.first + d.r0);
            bulk_commit_group();
          }
          continue;
        }
        if (lane == 0) bulk_commit_group();  // the buffers' turns are counted in groups
        __syncwarp();
        const int rows = min(32, d.left);
        __nv_bfloat16* dst = args.out + (size_t)(done.first + d.r0) * (size_t)args.cols + col;
        if (tma_out) {
          // the expert's last rows: 16 bytes a lane, 8 rows at a time
          const int j = lane & 3;
          for (int i = lane >> 2; i < rows; i += 8)
            if (col + 8 * j < args.cols)
              *reinterpret_cast<uint4*>(dst + (size_t)i * args.cols + 8 * j) =
                  *reinterpret_cast<const uint4*>(tile + i * 64 + ((j ^ ((i >> 1) & 3)) << 4));
        } else if (col + lane < args.cols) {
          // rows that do not start on 16 bytes: a column a lane, row by row
          for (int i = 0; i < rows; ++i)
            dst[(size_t)i * args.cols + lane] = *reinterpret_cast<const __nv_bfloat16*>(
                tile + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
        }
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---- quantisers -------------------------------------------------------------------
// top: the largest finite code (448 E4M3, 57344 E5M2).  scale = amax / top and
// inverse = top * (1 / amax), each operation rounded to fp32; all zeros give
// scale 1.  A max-abs below 2^-100 counts as 2^-100: its inverse would pass
// the fp32 range and turn the tile's zeros into NaN.
struct TileScale {
  float scale, inverse;
};
__device__ __forceinline__ TileScale tile_scale(float amax, float top) {
  if (amax == 0.f) return {1.f, 0.f};
  amax = fmaxf(amax, 0x1p-100f);
  return {__fdiv_rn(amax, top), __fmul_rn(top, __frcp_rn(amax))};
}
// 8 values -> 8 codes: round to nearest even with saturation; NaN stays NaN.
template <bool kE5M2>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inverse) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(v[2 * p], inverse), __fmul_rn(v[2 * p + 1], inverse)),
        __NV_SATFINITE, kE5M2 ? __NV_E5M2 : __NV_E4M3);
    w[p >> 1] |= (uint32_t)c2 << (16 * (p & 1));
  }
  return make_uint2(w[0], w[1]);
}

// Rows [rows, cols], cols a multiple of 16: a half-warp takes a 1x128 tile, 8
// values per lane (lanes past the last column hold zeros), four tiles at a time:
// four loads a lane are in flight, and lane j of the half computes tile j's
// scale for all.  The max-abs is taken on packed bf16 pairs (exact).  The
// tile's row and block advance by constants; one division at the start.  Four
// resident CTAs an SM and only the stores predicated: 8192 x 7168 36 us (4.95
// TB/s; eight CTAs in two waves, with branches around the code making, 42).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {  // of a (>= 0) and |b|
  b &= 0x7fff7fffu;
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
constexpr int kQuantCtas = 4;
template <bool kE5M2>
__global__ void __launch_bounds__(256, kQuantCtas) quantize_rows_kernel(
    const __nv_bfloat16* __restrict__ x, long long rows, int cols, uint8_t* __restrict__ q,
    float* __restrict__ sc, long long sc_ld) {
  constexpr int kUnroll = 4;
  const int per_row = (cols + QB - 1) / QB;
  const int l16 = threadIdx.x & 15;
  const long long hw = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  const long long stride = ((long long)gridDim.x * blockDim.x) >> 4;
  const int step_b = (int)(stride % per_row);
  const long long step_r = stride / per_row;
  long long r = hw / per_row;
  int b = (int)(hw - r * per_row);
  // every half-warp of a warp walks the same number of tiles: the shuffles stay
  // converged (tiles past the end are not live)
  const long long tiles = rows * per_row;
  for (long long t0 = (hw & ~1ll); t0 < tiles; t0 += kUnroll * stride) {
    uint4 raw[kUnroll];
    long long at[kUnroll];   // this lane's 8 values of tile j: element offset, -1 none
    long long my_sc = -1;    // lane j < 4: where tile j's scale goes
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      raw[j] = make_uint4(0u, 0u, 0u, 0u);
      const int c = b * QB + 8 * l16;
      at[j] = r < rows && c < cols ? r * cols + c : -1;
      if (at[j] >= 0) raw[j] = __ldg(reinterpret_cast<const uint4*>(x + at[j]));
      if (l16 == j && r < rows) my_sc = (long long)b * sc_ld + r;
      r += step_r;
      b += step_b;
      if (b >= per_row) {
        b -= per_row;
        ++r;
      }
    }
    float amax = 0.f;  // lane j < 4: of tile j
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      uint32_t m = max_abs2(max_abs2(max_abs2(max_abs2(0u, raw[j].x), raw[j].y), raw[j].z),
                            raw[j].w);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_abs2(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (l16 == j)
        amax = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    const TileScale s = tile_scale(amax, kE5M2 ? 57344.f : 448.f);
    if (my_sc >= 0) sc[my_sc] = s.scale;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const float inverse = __shfl_sync(0xffffffffu, s.inverse, j, 16);
      float v[8];
      bf16x8_to_f32(raw[j], v);
      const uint2 codes = codes8<kE5M2>(v, inverse);
      if (at[j] >= 0) *reinterpret_cast<uint2*>(q + at[j]) = codes;
    }
  }
}

// One 128x128 block of one matrix per CTA of 128 threads: sixteen lanes cover a
// row's 128 columns with 16-byte loads, kept in registers for the second pass.
// 32 x 2048 x 7168: 225 us (6.3 TB/s of the 3 bytes a weight that it cannot do
// without), one 4096 x 7168 14.4 us.
__global__ void __launch_bounds__(128) quantize_blocks_kernel(const __nv_bfloat16* __restrict__ w,
                                                              int n, int k, int nb, int kb,
                                                              uint8_t* __restrict__ q,
                                                              float* __restrict__ sc) {
  __shared__ float red[4];
  const long long blk = blockIdx.x;
  const int bc = (int)(blk % kb);
  const long long eb = blk / kb;
  const int br = (int)(eb % nb);
  const long long e = eb / nb;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int col = bc * QB + 8 * (lane & 15);
  const int row0 = br * QB + warp * 32 + (lane >> 4);
  const size_t at0 = ((size_t)e * n + row0) * (size_t)k + col;
  uint4 raw[16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row0 + 2 * i < n && col < k)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(w + at0 + (size_t)(2 * i) * k));
    float f[8];
    bf16x8_to_f32(raw[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const TileScale ts = tile_scale(amax, 448.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (row0 + 2 * i >= n || col >= k) continue;
    float f[8];
    bf16x8_to_f32(raw[i], f);
    *reinterpret_cast<uint2*>(q + at0 + (size_t)(2 * i) * k) = codes8<false>(f, ts.inverse);
  }
  if (t == 0) sc[blk] = ts.scale;
}

template <bool kDx>
cudaError_t launch(const PArgs& a, cudaStream_t st) {
  const size_t smem = fp8_mm_smem(a.E);
  cudaError_t e = note_cuda(cudaFuncSetAttribute(matmul_fp8_kernel<kDx>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)fp8_mm_smem(kMatmulMaxGroups)),
                            "fp8 matmul: set shared-memory size");
  if (e != cudaSuccess) return e;
  const long long mt = a.R / PBM + (a.R < a.E ? a.R : a.E);  // no more row tiles than this
  const long long units = mt * ((a.cols + PBN - 1) / PBN);
  const int grid = (int)(units < num_sms() ? units : num_sms());
  matmul_fp8_kernel<kDx><<<grid, PThreads, smem, st>>>(a);
  return note_cuda(cudaGetLastError(), "fp8 matmul launch");
}

}  // namespace

// dx == 0: a [R, k], out [R, n]; dx == 1: a [R, n], out [R, k].  e5m2: a's format.
int launch_matmul_fp8(int dx, int e5m2, const void* a_codes, const float* a_scales, long long sa_ld,
                      int R, const int32_t* offsets, int E, const void* w, const float* w_scales,
                      int n, int k, void* out, void* ws, cudaStream_t st) {
  if (matmul_is_narrow(R, E, dx ? k : n))
    return launch_matmul_narrow(dx, a_codes, e5m2, a_scales, sa_ld, R, offsets, E, w, w_scales, n,
                                k, out, ws, st);
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  PArgs a{};
  a.offsets = offsets;
  a.sa = a_scales;
  a.sa_ld = sa_ld;
  a.sw = w_scales;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<uint32_t*>(ws);
  a.E = E;
  a.R = R;
  a.cols = dx ? k : n;
  a.kdim = dx ? n : k;
  a.nb = (n + QB - 1) / QB;
  a.kb = (k + QB - 1) / QB;
  a.a_fmt = e5m2 ? kF8E5M2 : kF8E4M3;
  const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)k, (uint64_t)k * n};
  const uint32_t box[3] = {128, dx ? 128u : 256u, 1}, box64[3] = {128, 64, 1};
  if (!make_map(&a.tmA, a_codes, U8, 1, a.kdim, R, PBK, 128) ||
      !make_map(&a.tmA32, a_codes, U8, 1, a.kdim, R, PBK, 32) ||
      !make_map_nd(&a.tmB, w, U8, 3, dims, strides, box) ||
      (!dx && !make_map_nd(&a.tmB64, w, U8, 3, dims, strides, box64)) ||
      (a.cols % 8 == 0 && !make_map_swizzled(&a.tmOut, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                                             a.cols, R, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))) {
    note_text("fp8 matmul: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const cudaError_t e = dx ? launch<true>(a, st) : launch<false>(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

cudaError_t launch_quantize_rows_fp8(const void* x, long long rows, int cols, int e5m2,
                                     uint8_t* codes, float* scales, long long sc_ld,
                                     cudaStream_t st) {
  const long long tiles = rows * ((cols + QB - 1) / QB);
  long long blocks = (tiles * 16 + 255) / 256;
  const long long most = num_sms() * kQuantCtas;
  if (blocks > most) blocks = most;
  auto kernel = e5m2 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>;
  kernel<<<(int)blocks, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x), rows, cols, codes,
                                      scales, sc_ld);
  return note_cuda(cudaGetLastError(), "row quantisation launch");
}

cudaError_t launch_quantize_blocks_fp8(const void* w, int E, int n, int k, uint8_t* codes,
                                       float* scales, cudaStream_t st) {
  const int nb = (n + QB - 1) / QB, kb = (k + QB - 1) / QB;
  const long long blocks = (long long)E * nb * kb;
  quantize_blocks_kernel<<<(unsigned)blocks, 128, 0, st>>>(static_cast<const __nv_bfloat16*>(w), n,
                                                           k, nb, kb, codes, scales);
  return note_cuda(cudaGetLastError(), "block quantisation launch");
}

}  // namespace moe
