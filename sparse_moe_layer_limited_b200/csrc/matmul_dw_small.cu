// Weight gradients with few output tiles (a narrow or single matrix, a low-rank
// factor): dW_e = sum over the expert's rows of dy[r]^T x[r], bf16, where the
// 256 x 256 tiles of grouped_matmul.cu would leave most SMs without work.
//
// A unit is a 128 x 128 tile of dW_e, and a cluster of 2 to 8 CTAs splits the
// expert's rows.  Each CTA leaves its fp32 partial tile in its shared memory, and
// the cluster adds them, rank by rank, in order (every CTA takes its share of the
// tile), through distributed shared memory.  No workspace, no atomics.
//
// Measured (in brackets the pair kernel): 24415 rows of 3296 x 40 43 us (105),
// 16384 of 1024 x 1024 45 us (79), 100000 of 64 x 64 50 us (248): bound by what an
// SM pulls, 32 KB of operands for 256 cycles of MMA, and by how many take part.
// Not split, on 75 to 148 units, it is level with the pair kernel (16384 rows of
// 256 x 7168 85 us against 81), which therefore keeps those calls.
//
// Both operands have the contraction (the rows) outermost, as in
// grouped_matmul.cu, and the rows past an expert's end in its last 16-row step
// are overwritten with zeros in shared memory before the MMA reads them.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer (it also clears those rows),
// warps 2-5 epilogue.  Waits are bounded and set the status word when they give
// up; after that a CTA still takes part in every cluster barrier.
#include <cuda.h>
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "internal.h"
#include "matmul_util.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int DT = 128;                      // tile rows (n) and columns (k)
constexpr int DBK = 64;                      // expert rows per stage
constexpr int DChunk = 64 * DBK * 2;         // 64 columns of an operand
constexpr int DOperand = 2 * DChunk;
constexpr int DStageBytes = 2 * DOperand;
constexpr int DStages = 4;
constexpr int DThreads = 192;
constexpr int DPartBytes = DT * DT * 4;
constexpr int DSmem = 1024 + DStages * DStageBytes + DPartBytes + 256;
constexpr int kMaxSplit = 8;
static_assert(DSmem <= 232448, "shared-memory opt-in");

struct alignas(64) DArgs {
  CUtensorMap tmA;  // dy [R, n], box {64, 64}
  CUtensorMap tmB;  // x [R, k], box {64, 64}
  const int32_t* offsets;
  __nv_bfloat16* out;  // [E, n, k]
  uint32_t* status;
  int E, R, n, k;
  int splits;  // CTAs of a cluster
};

// Partial tile: row r's 16-byte piece p lies at piece p ^ (r & 31), so that lanes
// with a row each do not meet in a bank.
__device__ __forceinline__ int part_at(int r, int piece) {
  return (r * (DT / 4) + (piece ^ (r & 31))) * 4;
}

__global__ void __launch_bounds__(DThreads, 1) matmul_dw_small_kernel(
    const __grid_constant__ DArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(base + (size_t)DStages * DStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(part + DT * DT);
  uint64_t* empty = full + DStages;
  uint64_t* tfull = empty + DStages;  // [2]
  uint64_t* tempty = tfull + 2;       // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int S = args.splits;
  const int rank = (int)cluster_ctarank();
  const int MT = (args.n + DT - 1) / DT, NT = (args.k + DT - 1) / DT;
  const int total = args.E * MT * NT, step = gridDim.x / S;
  const int first_unit = blockIdx.x / S;

  if (tid == 0) {
    for (int s = 0; s < DStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 2 * DT);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  struct Unit {
    int g, first, rows;  // expert, its first row, its rows
    int m0, n0, width;   // row and column of dW_e, columns (a multiple of 16)
    int kb0, kcnt;       // this CTA's K blocks
  };
  auto decode = [&](int u) {
    Unit t;
    bool bad = false;
    t.g = u / (MT * NT);
    const int local = u - t.g * (MT * NT), m = local / NT;
    t.m0 = m * DT;
    t.n0 = (local - m * NT) * DT;
    t.width = min(DT, (args.k - t.n0 + 15) & ~15);
    t.rows = group_rows(args.offsets, t.g, args.R, &t.first, &bad);
    if (bad && tid == 0) atomicOr(args.status, kErrBadIndex);
    const int blocks = (t.rows + DBK - 1) / DBK, per = (blocks + S - 1) / S;
    t.kb0 = min(blocks, rank * per);
    t.kcnt = min(blocks, t.kb0 + per) - t.kb0;
    return t;
  };

  if (warp == 0) {
    // ---- TMA producer ----
    if (elect_one()) {
      tma_prefetch_desc(&args.tmA);
      tma_prefetch_desc(&args.tmB);
    }
    __syncwarp();
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      const int chunks = (t.width + 63) / 64;
      for (int i = 0; i < t.kcnt && ok; ++i) {
        ok = mm_wait(&empty[stage], phase ^ 1u, args.status);
        if (!ok) break;
        uint8_t* sa = base + (size_t)stage * DStageBytes;
        const int r = t.first + (t.kb0 + i) * DBK;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], (uint32_t)(DOperand + chunks * DChunk));
          for (int c = 0; c < 2; ++c)
            tma_load_2d(sa + c * DChunk, &args.tmA, t.m0 + 64 * c, r, &full[stage]);
          for (int c = 0; c < chunks; ++c)
            tma_load_2d(sa + DOperand + c * DChunk, &args.tmB, t.n0 + 64 * c, r, &full[stage]);
        }
        __syncwarp();
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == DStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (u + step >= total) {
        // every copy has landed before the CTA exits, also where the MMA warp gave up
        // (before the last barriers: here the wait is under the products')
        for (int s = 0; s < DStages; ++s)
          if ((issued >> s) & 1u) mm_drain(&full[s], (parity >> s) & 1u, args.status);
      }
      mm_cluster_sync();
      mm_cluster_sync();
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    const uint32_t ring = smem_u32(base);
    const uint64_t ad0 = smem_desc_mn_sw128(ring, DChunk);
    const uint64_t bd0 = smem_desc_mn_sw128(ring + DOperand, DChunk);
    const uint32_t a_hi = desc_hi(ad0), b_hi = desc_hi(bd0);
    constexpr uint32_t kStep = 16 * 128 / 16;  // 16 rows of a chunk
    int stage = 0;
    uint32_t phase = 0, use = 0;  // accumulators used so far
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      const uint32_t idesc = idesc_bf16_f32(DT, t.width) | kIdescAMn | kIdescBMn;
      const uint32_t buf = use & 1u;
      if (t.kcnt > 0) ok = ok && mm_wait(&tempty[buf], ((use >> 1) & 1u) ^ 1u, args.status);
      for (int i = 0; i < t.kcnt && ok; ++i) {
        ok = mm_wait(&full[stage], phase, args.status);
        if (!ok) break;
        const int valid = min(DBK, t.rows - (t.kb0 + i) * DBK), steps = (valid + 15) / 16;
        const int lines = steps * 16 - valid;  // to clear, in each chunk
        if (lines > 0) {
          uint8_t* sa = base + (size_t)stage * DStageBytes;
          for (int j = lane; j < lines * 4 * 8; j += 32) {
            const int piece = j & 7, line = (j >> 3) % lines, c = (j >> 3) / lines;
            *reinterpret_cast<uint4*>(sa + c * DChunk + (valid + line) * 128 + piece * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        const uint32_t off = (uint32_t)stage * (DStageBytes / 16);
        const uint32_t a_lo = desc_lo(ad0) + off, b_lo = desc_lo(bd0) + off;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < DBK / 16; ++k)
            if (k < steps)
              mma_bf16_parts(tmem_base + buf * DT, a_lo + k * kStep, a_hi, b_lo + k * kStep, b_hi,
                             idesc, (uint32_t)((i | k) != 0));
          mma_commit(&empty[stage]);
          if (i + 1 == t.kcnt) mma_commit(&tfull[buf]);
        }
        __syncwarp();
        if (i + 1 == t.kcnt) ++use;
        if (++stage == DStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      mm_cluster_sync();
      mm_cluster_sync();
    }
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mm_drain(drain, 0, args.status);
  } else {
    // ---- epilogue: a TMEM lane is a row of the tile ----
    const int q = warp & 3, row = q * 32 + lane, et = tid - 64;
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t use = 0;
    bool ok = true;
    for (int u = first_unit; u < total; u += step) {
      const Unit t = decode(u);
      const uint32_t buf = use & 1u;
      if (t.kcnt > 0 && ok) {
        ok = mm_wait(&tfull[buf], (use >> 1) & 1u, args.status, contraction_ms(t.kcnt));
        ++use;
      }
      if (ok) {
        tc_fence_after();
        for (int c = 0; c < t.width; c += 32) {
          uint32_t p[32];
          if (t.kcnt > 0) {
            tmem_ld32(tbase + buf * DT + c, p);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = 0u;  // no rows: zeros
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + part_at(row, (c + e) / 4)) =
                make_uint4(p[e], p[e + 1], p[e + 2], p[e + 3]);
        }
        tc_fence_before();
        __syncwarp();
        if (t.kcnt > 0 && lane == 0) mbar_arrive(&tempty[buf]);
      }
      mm_cluster_sync();
      // 8 columns a thread, sixteen threads a row
      for (int i = rank * 128 + et; i < DT * (DT / 8); i += S * 128) {
        const int r = i >> 4, c = (i & 15) * 8;
        if (t.m0 + r >= args.n || t.n0 + c >= args.k) continue;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const uint32_t lo = smem_u32(part + part_at(r, c / 4));
        const uint32_t hi = smem_u32(part + part_at(r, c / 4 + 1));
        for (int j = 0; j < S; ++j) {
          float f[8];
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                       : "r"(mapa_shared(lo, (uint32_t)j))
                       : "memory");
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                       : "r"(mapa_shared(hi, (uint32_t)j))
                       : "memory");
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += f[e];
        }
        if (ok)
          *reinterpret_cast<uint4*>(args.out + ((size_t)t.g * args.n + t.m0 + r) * args.k + t.n0 +
                                    c) =
              make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                         bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
      }
      mm_cluster_sync();  // everyone has read this CTA's partial tile
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * DT);
  }
}

long long dw_units(int E, int n, int k) {
  return (long long)E * ((n + DT - 1) / DT) * ((k + DT - 1) / DT);
}

}  // namespace

// CTAs that share a unit: more while the SMs are not filled and a CTA keeps at
// least four K blocks of an average expert.  1: not a case for this kernel.
int matmul_dw_splits(int R, int E, int n, int k) {
  const long long units = dw_units(E, n, k);
  int s = 1;
  while (s < kMaxSplit && units * s * 2 <= num_sms() && R / E >= 8 * DBK * s) s *= 2;
  return s;
}

int launch_matmul_dw_small(const void* dy, const void* x, int R, const int32_t* offsets, int E,
                           int n, int k, void* dw, void* ws, cudaStream_t st) {
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  DArgs a{};
  a.offsets = offsets;
  a.out = static_cast<__nv_bfloat16*>(dw);
  a.status = static_cast<uint32_t*>(ws);
  a.E = E;
  a.R = R;
  a.n = n;
  a.k = k;
  if (!make_map(&a.tmA, dy, BF, 2, n, R, 64, 64) || !make_map(&a.tmB, x, BF, 2, k, R, 64, 64)) {
    note_text("small weight gradient: tensor-map encoding failed");
    return MOE_ERR_CUDA;
  }
  a.splits = matmul_dw_splits(R, E, n, k);
  cudaError_t e = note_cuda(cudaFuncSetAttribute(matmul_dw_small_kernel,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, DSmem),
                            "small weight gradient: set shared-memory size");
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(DThreads, 1, 1);
  cfg.dynamicSmemBytes = DSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long units = dw_units(E, n, k), most = num_sms() / a.splits;
  cfg.gridDim = dim3((unsigned)((units < most ? units : most) * a.splits), 1, 1);
  e = note_cuda(cudaLaunchKernelEx(&cfg, matmul_dw_small_kernel, a), "small weight gradient launch");
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
