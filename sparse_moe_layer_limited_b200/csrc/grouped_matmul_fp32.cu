// Grouped matmul by expert over ragged rows in fp32 on the CUDA cores (the
// tensor cores have no fp32 operands): the three products of
// grouped_matmul.cu, any n and k.
//
// A CTA of 256 threads owns a BM x BN output tile; each thread keeps TM x TN
// running sums in registers and adds one contraction index at a time, so a
// sum is a plain fp32 chain (two columns to a packed multiply-add).  Slices of 16
// contraction indexes go through two shared-memory buffers in turn; the next
// slice's loads are issued before the current one is multiplied.  Tiles by size:
// 128 x 128 (two CTAs an SM) where they fill the SMs, 64 x 64 below that, 16 x 128
// for experts of few rows.  Small problems split the contraction over a cluster of
// up to 8 CTAs, whose partial tiles are added rank by rank, in order, through
// distributed shared memory.
//
// Measured (in brackets without splits and the smaller tile): 8 experts x 1024
// rows, 1024 x 1024: 396 us (43 TFLOP/s; the fp32 library product by expert takes
// 377), 64 rows of 2000 x 2000 25 us (37), 16 rows of two 4096 x 4096 78 us (181).
// 8 x 8 sums a thread issue 4 shared loads and 32 packed multiply-adds per
// contraction index; the multiply-add pipe bounds it.
#include <cuda_runtime.h>

#include "internal.h"
#include "f32x2.cuh"
#include "matmul_util.cuh"

namespace moe {
namespace {

constexpr int SBK = 16, SThreads = 256;

struct SArgs {
  const float* a;  // fwd: x; dx, dw: dy
  const float* b;  // fwd, dx: w; dw: x
  float* out;
  const int32_t* offsets;
  uint32_t* status;
  int E, R, n, k;
  int splits;  // CTAs of a cluster
};

// One operand's share of a slice: 16 contraction indexes by B rows (or columns)
// of the tile, four values per thread and round.  kInner: the contraction index
// is the contiguous one.  kVec: rows start on 16-byte boundaries, and the four
// values are consecutive; else they lie SThreads apart, so that a warp's loads
// are contiguous.
template <int B, bool kInner, bool kVec>
struct Operand {
  static constexpr int kRounds = (B * SBK / 4 + SThreads - 1) / SThreads;
  static constexpr bool kAll = B * SBK / 4 >= SThreads;  // every thread has work
  float v[kRounds][4];
  __device__ __forceinline__ static int lin(int q, int e) {
    return kVec ? ((q * SThreads + (int)threadIdx.x) * 4 + e)
                : (q * 4 + e) * SThreads + (int)threadIdx.x;
  }
  // value e of round q: contraction index kk of the slice, row (column) i
  __device__ __forceinline__ static int kk(int l) { return kInner ? l % SBK : l / B; }
  __device__ __forceinline__ static int i(int l) { return kInner ? l / SBK : l % B; }
  // src: element (row or contraction index r, c) at src[r * ld + c]; i0 + i is
  // valid below ilim, k0 + kk below klim
  __device__ __forceinline__ void fetch(const float* src, size_t ld, int i0, int ilim, int k0,
                                        int klim) {
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      if constexpr (kVec) {
        const int l = lin(q, 0), ii = i0 + i(l), k = k0 + kk(l);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if ((kAll || i(l) < B) && (kAll || kk(l) < SBK) && ii < ilim && k < klim)
          f = __ldg(reinterpret_cast<const float4*>(kInner ? src + (size_t)ii * ld + k
                                                           : src + (size_t)k * ld + ii));
        v[q][0] = f.x;
        v[q][1] = f.y;
        v[q][2] = f.z;
        v[q][3] = f.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int l = lin(q, e), ii = i0 + i(l), k = k0 + kk(l);
          v[q][e] = 0.f;
          if ((kAll || i(l) < B) && (kAll || kk(l) < SBK) && ii < ilim && k < klim)
            v[q][e] = __ldg(kInner ? src + (size_t)ii * ld + k : src + (size_t)k * ld + ii);
        }
      }
    }
  }
  // into dst [SBK][B + pad]
  __device__ __forceinline__ void stage(float* dst, int pitch) const {
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      if constexpr (kVec && !kInner) {
        const int l = lin(q, 0);
        if (kAll || kk(l) < SBK)
          *reinterpret_cast<float4*>(dst + kk(l) * pitch + i(l)) =
              make_float4(v[q][0], v[q][1], v[q][2], v[q][3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int l = lin(q, e);
          if ((kAll || i(l) < B) && (kAll || kk(l) < SBK)) dst[kk(l) * pitch + i(l)] = v[q][e];
        }
      }
    }
  }
};

// kMode as in grouped_matmul.cu: 0 forward, 1 input gradient, 2 weight gradient
template <int kMode, int BM, int BN, int TM, int TN, bool kVec>
__global__ void __launch_bounds__(SThreads, BM == 16 ? 4 : 2) grouped_matmul_fp32_kernel(const SArgs args) {
  static_assert((BM / TM) * (BN / TN) == SThreads, "one micro-tile per thread");
  constexpr bool kAInner = kMode != 2;  // A's contraction index is the contiguous one
  constexpr bool kBInner = kMode == 0;
  constexpr int kPad = 4;
  // a thread's rows come in groups of RV consecutive ones, its columns of CV
  constexpr int RV = TM < 4 ? TM : 4, CV = TN < 4 ? TN : 4;
  // two slice buffers; the partial tile of a split contraction takes their place
  constexpr int kSlice = SBK * (BM + kPad) + SBK * (BN + kPad);
  extern __shared__ float4 shared4[];
  float* shared = reinterpret_cast<float*>(shared4);
  __shared__ int start[kMatmulMaxGroups + 1];
  const int tid = threadIdx.x;
  const int rows_out = kMode == 2 ? args.n : 0;
  const int cols = kMode == 0 ? args.n : args.k;
  const int NT = (cols + BN - 1) / BN, MT = (rows_out + BM - 1) / BM;
  if constexpr (kMode != 2) {
    if (tid < 32) ragged_schedule(args.offsets, args.E, args.R, BM, NT, start, args.status);
    __syncthreads();
  }
  const long long total = kMode == 2 ? (long long)args.E * MT * NT : start[args.E];
  const int S = args.splits;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  for (long long u = blockIdx.x / S; u < total; u += gridDim.x / S) {
    int g, m, nt, first, rows;
    bool bad = false;
    if constexpr (kMode == 2) {
      g = (int)(u / (MT * NT));
      const int local = (int)(u - (long long)g * (MT * NT));
      m = local / NT;
      nt = local - m * NT;
      rows = group_rows(args.offsets, g, args.R, &first, &bad);
      if (bad && local == 0 && tid == 0) atomicOr(args.status, kErrBadIndex);
    } else {
      g = ragged_group(start, args.E, (int)u);
      rows = group_rows(args.offsets, g, args.R, &first, &bad);
      const int mt = (rows + BM - 1) / BM, local = (int)u - start[g];
      nt = local / mt;
      m = local - nt * mt;
    }
    const int m0 = m * BM, n0 = nt * BN;
    const int kfull = kMode == 0 ? args.k : (kMode == 1 ? args.n : rows);
    // this CTA's contraction range: whole slices
    const int per = ((kfull + S - 1) / S + SBK - 1) / SBK * SBK;
    const int kbeg = min(kfull, rank * per), kdim = min(kfull, kbeg + per);
    const int mlim = kMode == 2 ? args.n : rows;
    // A [row][k] (fwd x, dx dy) or [k][row] (dw dy); B [col][k] (fwd W) or
    // [k][col] (dx W, dw x)
    const float* A = args.a + (size_t)first * (kMode == 0 ? args.k : args.n);
    const float* B = kMode == 2 ? args.b + (size_t)first * args.k
                                : args.b + (size_t)g * args.n * args.k;
    Operand<BM, kAInner, kVec> oa;
    Operand<BN, kBInner, kVec> ob;
    auto fetch = [&](int k0) {
      oa.fetch(A, kMode == 0 ? args.k : args.n, m0, mlim, k0, kdim);
      ob.fetch(B, args.k, n0, cols, k0, kdim);
    };
    auto stage = [&](int buf) {
      oa.stage(shared + buf * kSlice, BM + kPad);
      ob.stage(shared + buf * kSlice + SBK * (BM + kPad), BN + kPad);
    };
    // thread (ty, tx): rows RV ty + RV (BM / TM) h + .., columns likewise
    const int tx = tid % (BN / TN), ty = tid / (BN / TN);
    // 8 x 8 sums a thread: pairs of columns in packed multiply-adds; on the
    // smaller ones their operand copies cost more than they save
    constexpr bool kPairs = TN == 8;
    float acc[TM][TN];
    f32x2 acc2[kPairs ? TM : 1][TN / 2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        acc[i][j] = 0.f;
        if constexpr (kPairs) acc2[i][j / 2] = 0ull;
      }
    int buf = 0;
    if (kbeg < kdim) {
      fetch(kbeg);
      stage(0);
    }
    __syncthreads();
    for (int k0 = kbeg; k0 < kdim; k0 += SBK, buf ^= 1) {
      const bool more = k0 + SBK < kdim;
      if (more) fetch(k0 + SBK);
      const float* As = shared + buf * kSlice;
      const float* Bs = As + SBK * (BM + kPad);
#pragma unroll
      for (int kk = 0; kk < SBK; ++kk) {
        float fa[TM];
        alignas(16) float fb[TN];
#pragma unroll
        for (int h = 0; h < TM / RV; ++h) {
          const float* p = As + kk * (BM + kPad) + h * (BM / TM) * RV + ty * RV;
          if constexpr (RV == 4)
            *reinterpret_cast<float4*>(fa + 4 * h) = *reinterpret_cast<const float4*>(p);
          else
            *reinterpret_cast<float2*>(fa + 2 * h) = *reinterpret_cast<const float2*>(p);
        }
#pragma unroll
        for (int h = 0; h < TN / CV; ++h)
          *reinterpret_cast<float4*>(fb + 4 * h) = *reinterpret_cast<const float4*>(
              Bs + kk * (BN + kPad) + h * (BN / TN) * CV + tx * CV);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if constexpr (kPairs) {
            const f32x2 a2 = pair2(fa[i], fa[i]);
#pragma unroll
            for (int j = 0; j < TN / 2; ++j)
              acc2[i][j] = fma2(a2, pair2(fb[2 * j], fb[2 * j + 1]), acc2[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(fa[i], fb[j], acc[i][j]);
          }
        }
      }
      if (more) stage(buf ^ 1);
      __syncthreads();
    }
    if constexpr (kPairs) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
          const float2 f = split2(acc2[i][j]);
          acc[i][2 * j] = f.x;
          acc[i][2 * j + 1] = f.y;
        }
    }
    auto row_of = [&](int i) { return (i / RV) * (BM / TM) * RV + ty * RV + i % RV; };
    auto store = [&](int r, int c, const float* v) {  // CV sums of output row r of the tile
      if (m0 + r >= mlim) return;
      float* dst = kMode == 2 ? args.out + ((size_t)g * args.n + m0 + r) * args.k
                              : args.out + (size_t)(first + m0 + r) * cols;
      c += n0;
      if constexpr (kVec) {
        if (c < cols) *reinterpret_cast<float4*>(dst + c) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < cols) dst[c + j] = v[j];
      }
    };
    if (S == 1) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < TN / CV; ++h)
          store(row_of(i), h * (BN / TN) * CV + tx * CV, &acc[i][CV * h]);
    } else {
      // the slices' buffers are free (the loop ends with a barrier)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < TN / CV; ++h)
          *reinterpret_cast<float4*>(shared + row_of(i) * BN + h * (BN / TN) * CV + tx * CV) =
              make_float4(acc[i][CV * h], acc[i][CV * h + 1], acc[i][CV * h + 2],
                          acc[i][CV * h + 3]);
      mm_cluster_sync();
      for (int q = rank * SThreads + tid; q < BM * BN / 4; q += S * SThreads) {
        const uint32_t at = smem_u32(shared + 4 * q);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < S; ++p) {
          float4 f;
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                       : "r"(mapa_shared(at, (uint32_t)p))
                       : "memory");
          v[0] += f.x;
          v[1] += f.y;
          v[2] += f.z;
          v[3] += f.w;
        }
        store(4 * q / BN, 4 * q % BN, v);
      }
      mm_cluster_sync();  // everyone has read this CTA's partial tile
    }
  }
}

// Shared memory of a tile: two slices, or the partial tile.
constexpr int tile_bytes(int BM, int BN) {
  const int two = 2 * SBK * (BM + 4 + BN + 4), part = BM * BN;
  return (two > part ? two : part) * 4;
}

template <int kMode, int BM, int BN, int TM, int TN>
cudaError_t launch(SArgs a, long long units, int kdim, cudaStream_t st) {
  // split while the SMs are not filled (twice; the few-row tile, whose CTAs are
  // small and wait for memory, four times) and a CTA keeps at least 4 slices
  constexpr int kFill = BM == 16 ? 4 : 2;
  a.splits = 1;
  while (a.splits < 8 && units * a.splits * 2 <= kFill * num_sms() &&
         kdim >= 8 * SBK * a.splits)
    a.splits *= 2;
  // rows on 16-byte boundaries
  auto kernel = a.n % 4 == 0 && a.k % 4 == 0 ? grouped_matmul_fp32_kernel<kMode, BM, BN, TM, TN, true>
                                             : grouped_matmul_fp32_kernel<kMode, BM, BN, TM, TN, false>;
  constexpr int smem = tile_bytes(BM, BN);
  cudaError_t e = cudaSuccess;
  if constexpr (smem > 48 * 1024)
    e = note_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                  "fp32 grouped matmul: set shared-memory size");
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(SThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long most = num_sms() * 32 / a.splits;
  cfg.gridDim = dim3((unsigned)((units < most ? units : most) * a.splits), 1, 1);
  return note_cuda(cudaLaunchKernelEx(&cfg, kernel, a), "fp32 grouped matmul launch");
}

template <int kMode>
cudaError_t launch_mode(const SArgs& a, cudaStream_t st) {
  const int cols = kMode == 0 ? a.n : a.k;
  // contraction length: of the average expert for the weight gradient
  const int kdim = kMode == 0 ? a.k : kMode == 1 ? a.n : a.R / a.E;
  auto units = [&](int bm, int bn) {
    const long long mt = kMode == 2 ? (long long)a.E * ((a.n + bm - 1) / bm)
                         : a.E == 1 ? (a.R + bm - 1) / bm
                                    : a.R / bm + (a.R < a.E ? a.R : a.E);
    return mt * ((cols + bn - 1) / bn);
  };
  if constexpr (kMode != 2) {
    // experts of 16 rows or fewer on average: most of a taller tile would be empty
    if (a.R <= 16LL * a.E) return launch<kMode, 16, 128, 2, 4>(a, units(16, 128), kdim, st);
  }
  if (units(128, 128) >= 2 * num_sms())
    return launch<kMode, 128, 128, 8, 8>(a, units(128, 128), kdim, st);
  return launch<kMode, 64, 64, 4, 4>(a, units(64, 64), kdim, st);
}

}  // namespace

int launch_grouped_matmul_fp32(int mode, const float* a, const float* b, int R,
                               const int32_t* offsets, int E, int n, int k, float* out, void* ws,
                               cudaStream_t st) {
  const SArgs s{a, b, out, offsets, static_cast<uint32_t*>(ws), E, R, n, k, 1};
  const cudaError_t e = mode == 0   ? launch_mode<0>(s, st)
                        : mode == 1 ? launch_mode<1>(s, st)
                                    : launch_mode<2>(s, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
