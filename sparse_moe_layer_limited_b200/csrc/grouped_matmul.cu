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
// Work unit: a 128 x kBN output tile.  Forward and input gradient order the
// units expert-major, then column tile, then row tile: CTAs running side by
// side share a weight tile through L2 and each expert's weights stream from
// HBM once.  The last column tile runs MMAs of its own width (rounded up to
// 16) and loads only the 64-wide chunks it has; a row tile loads 32-row boxes
// it has rows for, so a decode step's 1-row experts read 4 KB of rows per 32
// KB of weights.  Rows of the next expert inside a box only reach output rows
// that are not stored.  The weight gradient contracts over the rows: in an
// expert's last K block the rows past its end are overwritten with zeros in
// shared memory (in both operands, as 0 * NaN is NaN) before the MMA reads them.
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer and TMEM owner, then
// the epilogue warps, which drain one accumulator (fp32, rounded once to bf16)
// while the next tile accumulates in the other.  Full 32-row groups leave by
// TMA stores of 64 columns, an expert's ragged last rows by row stores.
// Waits are bounded and set the status word when they give up.
#include <cuda.h>
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "internal.h"
#include "matmul_util.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int GBM = 128, GBK = 64;
constexpr int kChunkBytes = 64 * 64 * 2;  // 64 x 64 bf16 operand chunk
constexpr int GABytes = GBM * GBK * 2;
constexpr int GStg = 32 * 128;            // per epilogue warp: 32 rows x 64 bf16

enum GMode { kFwd = 0, kDx = 1, kDw = 2 };

template <int kBN>
struct GCfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStages = kBN == 256 ? 4 : 6;
  static constexpr int kStageBytes = GABytes + kBN * GBK * 2;
  static constexpr size_t smem(int E) {
    return 1024 + (size_t)kStages * kStageBytes + kEpiWarps * GStg + 256 + (size_t)(E + 1) * 4;
  }
};
static_assert(GCfg<256>::smem(kMatmulMaxGroups) <= 232448, "shared-memory opt-in");
static_assert(GCfg<128>::smem(kMatmulMaxGroups) <= 232448, "shared-memory opt-in");

struct alignas(64) GArgs {
  CUtensorMap tmA;    // fwd / dx: rows [R, K], box {64, 128}; dw: dy [R, n], box {64, 64}
  CUtensorMap tmA32;  // fwd / dx: the same with box {64, 32}
  CUtensorMap tmB;    // fwd / dx: W [E, n, k], box {64, 64, 1}; dw: x [R, k], box {64, 64}
  CUtensorMap tmOut;  // fwd / dx: out [R, cols], box {64, 32}; dw: dW [E, n, k], box {64, 32, 1}
  const int32_t* offsets;
  __nv_bfloat16* out;
  uint32_t* status;
  int E, R;
  int m;     // dw: n (rows of dW_e); else unused
  int cols;  // output columns
  int kdim;  // fwd / dx: contraction length
};

template <int kMode, int kBN>
__global__ void __launch_bounds__(GCfg<kBN>::kThreads, 1) grouped_matmul_kernel(
    const __grid_constant__ GArgs args) {
  using C = GCfg<kBN>;
  constexpr int kStages = C::kStages, kStageBytes = C::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = base + (size_t)kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + C::kEpiWarps * GStg);
  uint64_t* full = bars;
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // [2]
  uint64_t* tempty = tfull + 2;       // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  int* start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NT = (args.cols + kBN - 1) / kBN;
  const int MT = (args.m + GBM - 1) / GBM;  // dw

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], C::kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 2 * kBN);
    tmem_relinquish();
  }
  if constexpr (kMode != kDw) {
    if (warp == 0) ragged_schedule(args.offsets, args.E, args.R, GBM, NT, start, args.status);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = kMode == kDw ? args.E * MT * NT : start[args.E];

  // unit -> expert g, its first row and row count, row tile m, column tile n
  struct Unit {
    int g, first, rows, m, n, kb;
  };
  auto decode = [&](int u) {
    Unit t;
    bool bad = false;
    if constexpr (kMode == kDw) {
      t.g = u / (MT * NT);
      const int local = u - t.g * (MT * NT);
      t.m = local / NT;
      t.n = local - t.m * NT;
      t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
      t.kb = (t.rows + GBK - 1) / GBK;
      if (bad && t.m == 0 && t.n == 0) atomicOr(args.status, kErrBadIndex);
    } else {
      t.g = ragged_group(start, args.E, u);
      t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
      const int mt = (t.rows + GBM - 1) / GBM;
      const int local = u - start[t.g];
      t.n = local / mt;
      t.m = local - t.n * mt;
      t.kb = (args.kdim + GBK - 1) / GBK;
    }
    return t;
  };

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      tma_prefetch_desc(&args.tmA);
      tma_prefetch_desc(&args.tmB);
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const Unit t = decode(u);
        const int nc = min(kBN / 64, (args.cols - t.n * kBN + 63) / 64);  // column chunks
        const int rows = kMode == kDw ? args.m : t.rows;
        const int left = rows - t.m * GBM;
        // A: 64-wide chunks (dw) or 32-row boxes that hold rows of the tile
        const int na = kMode == kDw ? (left > 64 ? 2 : 1) : min(4, (left + 31) / 32);
        const uint32_t bytes =
            (uint32_t)nc * kChunkBytes + (uint32_t)na * (kMode == kDw ? kChunkBytes : 32 * 128);
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!mm_wait(&empty[stage], phase ^ 1u, args.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = base + (size_t)stage * kStageBytes;
          uint8_t* sb = sa + GABytes;
          mbar_arrive_expect_tx(&full[stage], bytes);
          if constexpr (kMode == kDw) {
            const int r = t.first + kb * GBK;
            for (int c = 0; c < na; ++c)
              tma_load_2d(sa + c * kChunkBytes, &args.tmA, t.m * GBM + 64 * c, r, &full[stage]);
            for (int c = 0; c < nc; ++c)
              tma_load_2d(sb + c * kChunkBytes, &args.tmB, t.n * kBN + 64 * c, r, &full[stage]);
          } else {
            const int r = t.first + t.m * GBM;
            if (na == 4) {
              tma_load_2d(sa, &args.tmA, kb * GBK, r, &full[stage]);
            } else {
              for (int c = 0; c < na; ++c)
                tma_load_2d(sa + c * (32 * 128), &args.tmA32, kb * GBK, r + 32 * c, &full[stage]);
            }
            for (int c = 0; c < nc; ++c) {
              const int col = t.n * kBN + 64 * c;
              if constexpr (kMode == kFwd)
                tma_load_3d(sb + c * kChunkBytes, &args.tmB, kb * GBK, col, t.g, &full[stage]);
              else
                tma_load_3d(sb + c * kChunkBytes, &args.tmB, col, kb * GBK, t.g, &full[stage]);
            }
          }
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // let the copies already issued land before the CTA exits
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1u)
            mm_wait(&full[s], (parity >> s) & 1u, args.status, kMatmulTimeoutNs / 8);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer (the whole warp walks the loop; lane 0 issues) ----
    constexpr uint32_t kMajor = (kMode == kDw ? kIdescAMn | kIdescBMn : 0u) |
                                (kMode == kDx ? kIdescBMn : 0u);
    int stage = 0;
    uint32_t phase = 0;
    int local = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++local) {
      const Unit t = decode(u);
      const int width = min(kBN, args.cols - t.n * kBN);
      const uint32_t idesc = idesc_bf16_f32(GBM, (width + 15) / 16 * 16) | kMajor;
      const int acc = local & 1;
      if (!mm_wait(&tempty[acc], ((local >> 1) & 1) ^ 1u, args.status)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * kBN;
      for (int kb = 0; kb < t.kb; ++kb) {
        if (!mm_wait(&full[stage], phase, args.status)) {
          ok = false;
          break;
        }
        uint8_t* sa = base + (size_t)stage * kStageBytes;
        int steps = GBK / 16;
        if constexpr (kMode == kDw) {
          // rows of this K block that belong to the expert; the rest of the
          // last 16-row step is zeroed: one 128-byte line per row and chunk
          const int valid = t.rows - kb * GBK;
          if (valid < GBK) {
            steps = (valid + 15) / 16;
            const int lines = steps * 16 - valid;
            const int chunks = (GABytes + kBN * GBK * 2) / kChunkBytes;
            for (int i = lane; i < lines * chunks * 8; i += 32) {
              const int piece = i & 7, line = (i >> 3) % lines, c = (i >> 3) / lines;
              *reinterpret_cast<uint4*>(sa + c * kChunkBytes + (valid + line) * 128 + piece * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (lane == 0) {
          tc_fence_after();
          const uint32_t a0 = smem_u32(sa), b0 = a0 + GABytes;
#pragma unroll
          for (int k = 0; k < GBK / 16; ++k) {
            if (k < steps) {
              const uint64_t ad = kMode == kDw ? smem_desc_mn_sw128(a0 + k * 2048, kChunkBytes)
                                               : smem_desc_sw128(a0 + k * 32);
              const uint64_t bd = kMode == kFwd ? smem_desc_sw128(b0 + k * 32)
                                                : smem_desc_mn_sw128(b0 + k * 2048, kChunkBytes);
              mma_bf16(d_tmem, ad, bd, idesc, (kb | k) != 0);
            }
          }
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && lane == 0) mma_commit(&tfull[acc]);  // without K blocks: arrives at once
      __syncwarp();
    }
    if (lane == 0) {
      mma_commit(drain);
      mm_wait(drain, 0, args.status, kMatmulTimeoutNs / 8);
    }
    __syncwarp();
  } else {
    // ---- epilogue: two warps per TMEM lane quadrant, kBN / 2 columns each ----
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = staging + (size_t)(warp - 2) * GStg;
    int local = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++local) {
      const Unit t = decode(u);
      const int acc = local & 1;
      if (!mm_wait(&tfull[acc], (local >> 1) & 1, args.status)) break;
      tc_fence_after();
      const int r0 = t.m * GBM + q * 32;  // this warp's first row of the group (of dW_e)
      const int left = (kMode == kDw ? args.m : t.rows) - r0;
      const bool by_tma = kMode == kDw || left >= 32;
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * kBN;
#pragma unroll 1
      for (int c = half * (kBN / 2); c < (half + 1) * (kBN / 2); c += 64) {
        const int col = t.n * kBN + c;
        if (left <= 0 || col >= args.cols) break;  // warp-uniform
        uint32_t p[32];
        if (kMode == kDw && t.kb == 0) {  // an expert without rows: a zero gradient
#pragma unroll
          for (int i = 0; i < 32; ++i) p[i] = 0u;
        } else {
          uint32_t v0[32], v1[32];
          tmem_ld32(taddr + c, v0);
          tmem_ld32(taddr + c + 32, v1);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = bf16x2_bits(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]));
            p[16 + i] = bf16x2_bits(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]));
          }
        }
        if (by_tma) {
          if (lane == 0) bulk_wait_read_all();  // the previous piece has left the buffer
          __syncwarp();
          uint8_t* my = stg + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(my + ((j ^ (lane & 7)) << 4)) =
                make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kMode == kDw)
              tma_store_3d(&args.tmOut, stg, col, r0, t.g);
            else
              tma_store_2d(&args.tmOut, stg, col, t.first + r0);
            bulk_commit_group();
          }
        } else if (lane < left) {
          __nv_bfloat16* dst =
              args.out + (size_t)(t.first + r0 + lane) * (size_t)args.cols + col;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + 8 * j < args.cols)
              reinterpret_cast<uint4*>(dst)[j] =
                  make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
    if (lane == 0) bulk_wait_all();  // the staging buffer outlives the stores that read it
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kBN);
  }
}

template <int kMode, int kBN>
cudaError_t launch(const GArgs& a, long long units, cudaStream_t st) {
  const size_t smem = GCfg<kBN>::smem(a.E);
  auto kernel = grouped_matmul_kernel<kMode, kBN>;
  cudaError_t e =
      note_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem),
                "grouped matmul: set shared-memory size");
  if (e != cudaSuccess) return e;
  const int grid = (int)(units < num_sms() ? units : num_sms());
  kernel<<<grid, GCfg<kBN>::kThreads, smem, st>>>(a);
  return note_cuda(cudaGetLastError(), "grouped matmul launch");
}

}  // namespace

// mode 0: rows = x [R, k], out = y [R, n]; 1: rows = dy [R, n], out = dx [R, k];
// w [E, n, k], bf16, n and k multiples of 8.
int launch_grouped_matmul_bf16(int mode, const void* rows, int R, const int32_t* offsets, int E,
                               const void* w, int n, int k, void* out, void* ws,
                               cudaStream_t st) {
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GArgs a{};
  a.offsets = offsets;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<uint32_t*>(ws);
  a.E = E;
  a.R = R;
  a.cols = mode == kDx ? k : n;
  a.kdim = mode == kDx ? n : k;
  const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)k * 2, (uint64_t)k * n * 2};
  const uint32_t box[3] = {64, 64, 1};
  if (!make_map(&a.tmA, rows, BF, 2, a.kdim, R, 64, 128) ||
      !make_map(&a.tmA32, rows, BF, 2, a.kdim, R, 64, 32) ||
      !make_map_nd(&a.tmB, w, BF, 3, dims, strides, box) ||
      !make_map_swizzled(&a.tmOut, out, BF, 2, a.cols, R, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B)) {
    note_text("grouped matmul: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const long long mt = R / GBM + (R < E ? R : E);  // no more row tiles than this
  const long long units = mt * ((a.cols + 255) / 256);
  const cudaError_t e =
      mode == kFwd ? launch<kFwd, 256>(a, units, st) : launch<kDx, 256>(a, units, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// dw [E, n, k] from dy [R, n] and x [R, k], bf16, n and k multiples of 8.
int launch_grouped_matmul_dw_bf16(const void* dy, const void* x, int R, const int32_t* offsets,
                                  int E, int n, int k, void* dw, void* ws, cudaStream_t st) {
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
  if (!make_map(&a.tmA, dy, BF, 2, n, R, 64, 64) || !make_map(&a.tmB, x, BF, 2, k, R, 64, 64) ||
      !make_map_nd(&a.tmOut, dw, BF, 3, dims, strides, box)) {
    note_text("grouped matmul weight gradient: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const long long units = (long long)E * ((n + GBM - 1) / GBM) * ((k + 255) / 256);
  return launch<kDw, 256>(a, units, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
