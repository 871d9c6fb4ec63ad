// Matmuls with few rows (decode steps, small batches): the forward and input
// gradient of grouped_matmul.cu (bf16) and matmul_fp8.cu (FP8 with block
// scales) where their 256-wide tiles would leave most SMs without work.
//
// Such a call streams the weights once; its time is how many SMs pull them and
// how much each keeps in flight.  A unit is 128 output columns (the M index of
// the MMA: the weight is the A operand) by at most 64 rows (N), so the copies
// are almost only weight bytes.  Where even these units are too few, a cluster
// of up to 8 CTAs splits the unit's contraction; each CTA leaves its fp32
// partial tile in its shared memory and the cluster adds them, rank by rank, in
// order (every CTA takes its share of the rows), through distributed shared
// memory.  No workspace, no atomics.
//
// Measured: one row of 2048 x 7168 bf16 16.4 us (27 on the pair kernel), 8 rows on
// 8 experts of 2048 x 7168 45 us (5.2 TB/s of weights), FP8 7 rows of 7168 x 2048
// 9.7 us (14.8), 64 rows of 4096 x 7168 16.4 us (31); 6-7 us of each are start and
// end (tensor memory, barriers, first copies, the cluster's two barriers).
//
// FP8: every 128-wide slice is one product into its own TMEM buffer (eight of
// 64 columns in flight), multiplied by sa[row] * sw and added to fp32 registers.
// All 128 output columns of a unit lie in one weight block, so the factor
// depends on the row alone; it is formed once per 64 slices in shared memory.
//
// Waits are bounded and set the status word when they give up; after that a
// CTA still takes part in every cluster barrier.
#include <cuda.h>
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "fp8_util.cuh"
#include "internal.h"
#include "matmul_util.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int NM = 128, NN = 64;      // output columns and rows of a unit
constexpr int NRowBytes = 128;        // contraction bytes per stage: 64 bf16 or 128 codes
constexpr int NABytes = NM * NRowBytes, NBBytes = NN * NRowBytes;
constexpr int NStageBytes = NABytes + NBBytes;
constexpr int NStages = 6;
constexpr int NThreads = 192;         // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr int NPartBytes = NN * NM * 4;
constexpr int NScaleSlices = 64;
constexpr int NScaleBytes = NScaleSlices * NN * 4;
constexpr int NBufs = 8;              // FP8 slice buffers; bf16 uses two of them as accumulators
constexpr int kMaxSplit = 8;

constexpr size_t narrow_smem(int E) {
  return 1024 + (size_t)NStages * NStageBytes + NPartBytes + NScaleBytes + 256 +
         (size_t)(E + 1) * 4;
}
static_assert(narrow_smem(kMatmulMaxGroups) <= 232448, "shared-memory opt-in");

struct alignas(64) NArgs {
  CUtensorMap tmW;      // weight [E, n, k]: forward box {128 bytes, 128, 1}; input gradient
                        // bf16 {64, 64, 1}, FP8 {128, 128, 1}
  CUtensorMap tmX[3];   // rows, boxes of 16, 32, 64 rows
  const int32_t* offsets;
  __nv_bfloat16* out;   // [R, m]
  uint32_t* status;
  const float* sa;      // FP8: [KB, sa_ld]
  const float* sw;      // FP8: [E, nb, kb]
  long long sa_ld;
  int E, R;
  int m, kdim;          // output columns, contraction length
  int nb, kb;           // FP8: blocks along n and k
  int splits;           // CTAs of a cluster
  uint32_t a_fmt;       // FP8: format of the rows
};

__device__ __forceinline__ void fma2v(float& a0, float& a1, float x0, float x1, float s0,
                                      float s1) {
  asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%0, %1};\n\tfma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1), "f"(s0), "f"(s1));
}
__device__ __forceinline__ float peer_f32(uint32_t local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(local, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void epilogue_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

template <bool kFp8, bool kDx>
__global__ void __launch_bounds__(NThreads, 1) matmul_narrow_kernel(
    const __grid_constant__ NArgs args) {
  constexpr int kElem = kFp8 ? 1 : 2;
  constexpr int kBK = NRowBytes / kElem;            // contraction indexes per stage
  constexpr int kStepK = 32 / kElem;                // per MMA
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(base + (size_t)NStages * NStageBytes);  // [row][column]
  float* factor = part + NN * NM;                                                // [slice][row]
  uint64_t* bars = reinterpret_cast<uint64_t*>(factor + NScaleSlices * NN);
  uint64_t* full = bars;
  uint64_t* empty = full + NStages;
  uint64_t* tfull = empty + NStages;   // [NBufs]
  uint64_t* tempty = tfull + NBufs;    // [NBufs]
  uint64_t* drain = tempty + NBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  int* start = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int S = args.splits;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int first_unit = blockIdx.x / S, step = gridDim.x / S;
  const int MT = (args.m + NM - 1) / NM;
  const int KB = (args.kdim + kBK - 1) / kBK;
  const int per = (KB + S - 1) / S;
  const int kb0 = min(KB, rank * per), kcnt = min(KB, kb0 + per) - kb0;  // this CTA's K blocks

  if (tid == 0) {
    for (int s = 0; s < NStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < NBufs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 0) ragged_schedule(args.offsets, args.E, args.R, NN, MT, start, args.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = start[args.E];

  struct Unit {
    int g, first, rows;  // expert, its first row, its rows
    int m0, n0, width;   // output column, row of the expert, N (a multiple of 16)
  };
  auto decode = [&](int u) {
    Unit t;
    bool bad = false;
    t.g = ragged_group(start, args.E, u);
    t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
    const int tiles = (t.rows + NN - 1) / NN, local = u - start[t.g];
    const int w = ((t.rows + tiles - 1) / tiles + 15) & ~15;
    t.m0 = local / tiles * NM;
    t.n0 = local % tiles * w;
    t.width = min(w, (t.rows - t.n0 + 15) & ~15);
    return t;
  };

  if (warp == 0) {
    // ---- TMA producer ----
    if (elect_one()) tma_prefetch_desc(&args.tmW);
    __syncwarp();
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      const int box = t.width <= 16 ? 0 : t.width <= 32 ? 1 : 2;
      const uint32_t bytes = NABytes + (uint32_t)(16 << box) * NRowBytes;
      for (int i = 0; i < kcnt && ok; ++i) {
        ok = mm_wait(&empty[stage], phase ^ 1u, args.status);
        if (!ok) break;
        uint8_t* sa = base + (size_t)stage * NStageBytes;
        const int k = (kb0 + i) * kBK;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], bytes);
          if constexpr (!kDx) {
            tma_load_3d(sa, &args.tmW, k, t.m0, t.g, &full[stage]);
          } else if constexpr (kFp8) {
            tma_load_3d(sa, &args.tmW, t.m0, k, t.g, &full[stage]);
          } else {
            tma_load_3d(sa, &args.tmW, t.m0, k, t.g, &full[stage]);
            tma_load_3d(sa + NABytes / 2, &args.tmW, t.m0 + 64, k, t.g, &full[stage]);
          }
          tma_load_2d(sa + NABytes, &args.tmX[box], k, t.first + t.n0, &full[stage]);
        }
        __syncwarp();
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == NStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (u + step >= total) {
        // every copy has landed before the CTA exits, also where the MMA warp gave up
        // (before the last barriers: here the wait is under the products')
        for (int s = 0; s < NStages; ++s)
          if ((issued >> s) & 1u) mm_drain(&full[s], (parity >> s) & 1u, args.status);
      }
      if (S > 1) {
        mm_cluster_sync();
        mm_cluster_sync();
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    const uint32_t ring = smem_u32(base);
    constexpr uint32_t kChunk = kFp8 ? NABytes : NABytes / 2;  // contraction outermost
    const uint64_t ad0 = kDx ? smem_desc_mn_sw128(ring, kChunk) : smem_desc_sw128(ring);
    const uint64_t bd0 = smem_desc_sw128(ring + NABytes);
    const uint32_t a_hi = desc_hi(ad0), b_hi = desc_hi(bd0);
    constexpr uint32_t kAStep = (kDx ? kStepK * 128 : 32) / 16;
    int stage = 0;
    uint32_t phase = 0, use = 0;  // buffers used so far
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      // A is the weight (E4M3), B the rows
      const uint32_t idesc = (kFp8 ? idesc_f8_f32(NM, t.width, kF8E4M3, args.a_fmt)
                                   : idesc_bf16_f32(NM, t.width)) |
                             (kDx ? kIdescAMn : 0u);
      for (int i = 0; i < kcnt && ok; ++i) {
        const uint32_t buf = use % NBufs, use_parity = ((use / NBufs) & 1u) ^ 1u;
        if (kFp8 || i == 0) ok = mm_wait(&tempty[buf], use_parity, args.status);
        ok = ok && mm_wait(&full[stage], phase, args.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t off = (uint32_t)stage * (NStageBytes / 16);
        const uint32_t a_lo = desc_lo(ad0) + off, b_lo = desc_lo(bd0) + off;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < NRowBytes / 32; ++k) {
            if constexpr (kFp8)
              mma_f8_parts(tmem_base + buf * NN, a_lo + k * kAStep, a_hi, b_lo + k * 2, b_hi,
                           idesc, k != 0);
            else
              mma_bf16_parts(tmem_base + buf * NN, a_lo + k * kAStep, a_hi, b_lo + k * 2, b_hi,
                             idesc, (uint32_t)((i | k) != 0));
          }
          mma_commit(&empty[stage]);
          if (kFp8 || i + 1 == kcnt) mma_commit(&tfull[buf]);
        }
        __syncwarp();
        if (kFp8 || i + 1 == kcnt) ++use;
        if (++stage == NStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (S > 1) {
        mm_cluster_sync();
        mm_cluster_sync();
      }
    }
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mm_drain(drain, 0, args.status);
  } else {
    // ---- epilogue: lane = output column, register = row ----
    const int q = warp & 3;
    const int col = q * 32 + lane, et = tid - 64;  // column of the unit; epilogue thread
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t use = 0;
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      const bool wide = t.width > 32;
      float acc[NN];
#pragma unroll
      for (int i = 0; i < NN; ++i) acc[i] = 0.f;
      if constexpr (kFp8) {
        const float* sw = args.sw + (size_t)t.g * args.nb * args.kb +
                          (kDx ? (size_t)(t.m0 / QB) : (size_t)(t.m0 / QB) * args.kb);
        const int sw_step = kDx ? args.kb : 1;
        for (int i = 0; i < kcnt; ++i, ++use) {  // (after a time-out the barriers go on)
          if (i % NScaleSlices == 0) {
            // the next slices' factors: row et % 64, every second slice
            epilogue_sync();
            const int row = min(t.first + t.n0 + (et & 63), args.R - 1);
            const int n = min(NScaleSlices, kcnt - i);
            for (int j = et >> 6; j < n; j += 2)
              factor[j * NN + (et & 63)] =
                  __ldg(args.sa + (size_t)(kb0 + i + j) * args.sa_ld + row) *
                  __ldg(sw + (size_t)(kb0 + i + j) * sw_step);
            epilogue_sync();
          }
          const uint32_t buf = use % NBufs;
          ok = ok && mm_wait(&tfull[buf], (use / NBufs) & 1u, args.status);
          if (!ok) continue;
          tc_fence_after();
          const float4* f = reinterpret_cast<const float4*>(factor + (i % NScaleSlices) * NN);
          uint32_t p[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 0 || wide) {
              tmem_ld32(tbase + buf * NN + 32 * h, p);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 s = f[8 * h + e / 4];
                fma2v(acc[32 * h + e], acc[32 * h + e + 1], __uint_as_float(p[e]),
                      __uint_as_float(p[e + 1]), s.x, s.y);
                fma2v(acc[32 * h + e + 2], acc[32 * h + e + 3], __uint_as_float(p[e + 2]),
                      __uint_as_float(p[e + 3]), s.z, s.w);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
      } else if (kcnt > 0 && ok) {
        const uint32_t buf = use % NBufs;
        ok = mm_wait(&tfull[buf], (use / NBufs) & 1u, args.status, contraction_ms(kcnt));
        if (ok) {
          tc_fence_after();
          uint32_t p[32];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (h == 0 || wide) {
              tmem_ld32(tbase + buf * NN + 32 * h, p);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) acc[32 * h + e] = __uint_as_float(p[e]);
            }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
          ++use;
        }
      }
      const int rows = min(t.width, t.rows - t.n0);
      __nv_bfloat16* dst = args.out + (size_t)(t.first + t.n0) * (size_t)args.m + t.m0 + col;
      const bool in = t.m0 + col < args.m;
      if (S == 1) {
        if (in && ok) {
#pragma unroll
          for (int i = 0; i < NN; ++i)
            if (i < rows) dst[(size_t)i * args.m] = __float2bfloat16_rn(acc[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NN; ++i)
          if (i < rows) part[i * NM + col] = acc[i];
        mm_cluster_sync();
        const uint32_t mine = smem_u32(part) + (uint32_t)col * 4;
        for (int i = rank; i < rows; i += S) {
          float sum = 0.f;
          for (int j = 0; j < S; ++j) sum += peer_f32(mine + (uint32_t)i * (NM * 4), (uint32_t)j);
          if (in && ok) dst[(size_t)i * args.m] = __float2bfloat16_rn(sum);
        }
        mm_cluster_sync();  // everyone has read this CTA's partial tile
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <bool kFp8, bool kDx>
cudaError_t launch(const NArgs& a, long long units, cudaStream_t st) {
  auto kernel = matmul_narrow_kernel<kFp8, kDx>;
  cudaError_t e =
      note_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)narrow_smem(kMatmulMaxGroups)),
                "narrow matmul: set shared-memory size");
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NThreads, 1, 1);
  cfg.dynamicSmemBytes = narrow_smem(a.E);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long most = num_sms() / a.splits;
  cfg.gridDim = dim3((unsigned)((units < most ? units : most) * a.splits), 1, 1);
  return note_cuda(cudaLaunchKernelEx(&cfg, kernel, a), "narrow matmul launch");
}

// No more units than this: row tiles of at most 64 times column tiles of 128.
long long narrow_units(int R, int E, int cols) {
  const long long tiles = E == 1 ? (R + NN - 1) / NN : (long long)R / NN + (R < E ? R : E);
  return tiles * ((cols + NM - 1) / NM);
}

}  // namespace

// The narrow kernel takes a call whose units all fit on the SMs at once (so
// none waits for a second round, which the kernels for many rows overlap better).
// us here and there, 2048 x 7168, called back to back:
//   units                                  32       64       128      144      160
//   bf16 forward, one expert             21 / 35  30 / 41  35 / 41  35 / 33  63 / 37
//   bf16 forward, a row for each expert     -     25 / 31  45 / 45  49 / 49  75 / 71
//   FP8 forward, one expert              18 / 49  27 / 34  31 / 33  31 / 33  54 / 33
//   FP8 forward, a row for each expert      -     16 / 32  33 / 34  33 / 35  50 / 35
// The input gradients run as the forwards do.
bool matmul_is_narrow(int R, int E, int cols) { return narrow_units(R, E, cols) <= num_sms(); }

// Argument meanings as at launch_grouped_matmul_bf16 and launch_matmul_fp8;
// a_scales == nullptr: bf16.
int launch_matmul_narrow(int dx, const void* rows, int e5m2, const float* a_scales,
                         long long sa_ld, int R, const int32_t* offsets, int E, const void* w,
                         const float* w_scales, int n, int k, void* out, void* ws,
                         cudaStream_t st) {
  const bool fp8 = a_scales != nullptr;
  const auto dt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const size_t elem = fp8 ? 1 : 2;
  const uint32_t inner = NRowBytes / (uint32_t)elem;
  NArgs a{};
  a.offsets = offsets;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<uint32_t*>(ws);
  a.sa = a_scales;
  a.sw = w_scales;
  a.sa_ld = sa_ld;
  a.E = E;
  a.R = R;
  a.m = dx ? k : n;
  a.kdim = dx ? n : k;
  a.nb = (n + QB - 1) / QB;
  a.kb = (k + QB - 1) / QB;
  a.a_fmt = e5m2 ? kF8E5M2 : kF8E4M3;
  const long long units = narrow_units(R, E, a.m);
  // split the contraction while the SMs are not filled and a CTA keeps at
  // least four K blocks
  const int blocks = (a.kdim + (int)inner - 1) / (int)inner;
  a.splits = 1;
  while (a.splits < kMaxSplit && units * a.splits * 2 <= num_sms() &&
         blocks >= 8 * a.splits)
    a.splits *= 2;
  const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)k * elem, (uint64_t)k * n * elem};
  const uint32_t box[3] = {inner, dx ? inner : (uint32_t)NM, 1};
  bool ok = make_map_nd(&a.tmW, w, dt, 3, dims, strides, box);
  for (int i = 0; i < 3; ++i)
    ok = ok && make_map(&a.tmX[i], rows, dt, elem, a.kdim, R, inner, 16u << i);
  if (!ok) {
    note_text("narrow matmul: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  const cudaError_t e = fp8 ? (dx ? launch<true, true>(a, units, st) : launch<true, false>(a, units, st))
                            : (dx ? launch<false, true>(a, units, st) : launch<false, false>(a, units, st));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
