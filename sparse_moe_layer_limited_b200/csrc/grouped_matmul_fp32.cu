// Grouped matmul by expert over ragged rows in fp32 on the CUDA cores (the
// tensor cores have no fp32 operands): the three products of
// grouped_matmul.cu, any n and k.
//
// A CTA of 256 threads owns a BM x BN output tile; each thread keeps TM x TN
// running sums in registers and adds one contraction index at a time, so a
// sum is a plain fp32 chain.  Slices of 16 contraction indexes go through
// shared memory; the next slice's loads are issued before the current one is
// multiplied.  A 128 x 128 tile reads 16 bytes of shared memory per 16
// multiply-adds of a thread, which is what bounds it; the 64 x 64 tile is for
// problems with too few large tiles to fill the SMs.
#include <cuda_runtime.h>

#include "internal.h"
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
};

// 4 consecutive floats of a row of `len` at column c (zeros past the end, or
// when the row itself is absent)
template <bool kVec>
__device__ __forceinline__ float4 load4(const float* row, bool live, int c, int len) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!live) return v;
  if constexpr (kVec) {
    if (c < len) v = __ldg(reinterpret_cast<const float4*>(row + c));
  } else {
    if (c < len) v.x = __ldg(row + c);
    if (c + 1 < len) v.y = __ldg(row + c + 1);
    if (c + 2 < len) v.z = __ldg(row + c + 2);
    if (c + 3 < len) v.w = __ldg(row + c + 3);
  }
  return v;
}

// kMode as in grouped_matmul.cu: 0 forward, 1 input gradient, 2 weight gradient
template <int kMode, int BM, int BN, int TM, int TN, bool kVec>
__global__ void __launch_bounds__(SThreads) grouped_matmul_fp32_kernel(const SArgs args) {
  static_assert((BM / TM) * (BN / TN) == SThreads, "one micro-tile per thread");
  constexpr bool kAInner = kMode != 2;  // A's contraction index is the contiguous one
  constexpr bool kBInner = kMode == 0;
  constexpr int kPad = 4;
  __shared__ alignas(16) float As[SBK][BM + kPad];
  __shared__ alignas(16) float Bs[SBK][BN + kPad];
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
  for (long long u = blockIdx.x; u < total; u += gridDim.x) {
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
    const int kdim = kMode == 0 ? args.k : (kMode == 1 ? args.n : rows);
    const int mlim = kMode == 2 ? args.n : rows;
    const float* W = args.b + (kMode == 2 ? 0 : (size_t)g * args.n * args.k);
    constexpr int QA = BM * SBK / 4 / SThreads, QB4 = BN * SBK / 4 / SThreads;
    float4 ra[QA], rb[QB4];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int q = 0; q < QA; ++q) {
        const int it = tid + q * SThreads;
        if constexpr (kAInner) {
          const int i = it >> 2, kk = k0 + (it & 3) * 4;
          const int lda = kMode == 0 ? args.k : args.n;
          ra[q] = load4<kVec>(args.a + (size_t)(first + m0 + i) * lda, m0 + i < mlim, kk, kdim);
        } else {
          const int kk = k0 + it / (BM / 4), i = m0 + it % (BM / 4) * 4;
          ra[q] = load4<kVec>(args.a + (size_t)(first + kk) * args.n, kk < kdim, i, args.n);
        }
      }
#pragma unroll
      for (int q = 0; q < QB4; ++q) {
        const int it = tid + q * SThreads;
        if constexpr (kBInner) {
          const int j = it >> 2, kk = k0 + (it & 3) * 4;
          rb[q] = load4<kVec>(W + (size_t)(n0 + j) * args.k, n0 + j < cols, kk, kdim);
        } else {
          const int kk = k0 + it / (BN / 4), j = n0 + it % (BN / 4) * 4;
          const float* row = kMode == 1 ? W + (size_t)kk * args.k
                                        : args.b + (size_t)(first + kk) * args.k;
          rb[q] = load4<kVec>(row, kk < kdim, j, args.k);
        }
      }
    };
    auto stage = [&]() {
#pragma unroll
      for (int q = 0; q < QA; ++q) {
        const int it = tid + q * SThreads;
        if constexpr (kAInner) {
          const int i = it >> 2, kk = (it & 3) * 4;
          As[kk][i] = ra[q].x;
          As[kk + 1][i] = ra[q].y;
          As[kk + 2][i] = ra[q].z;
          As[kk + 3][i] = ra[q].w;
        } else {
          *reinterpret_cast<float4*>(&As[it / (BM / 4)][it % (BM / 4) * 4]) = ra[q];
        }
      }
#pragma unroll
      for (int q = 0; q < QB4; ++q) {
        const int it = tid + q * SThreads;
        if constexpr (kBInner) {
          const int j = it >> 2, kk = (it & 3) * 4;
          Bs[kk][j] = rb[q].x;
          Bs[kk + 1][j] = rb[q].y;
          Bs[kk + 2][j] = rb[q].z;
          Bs[kk + 3][j] = rb[q].w;
        } else {
          *reinterpret_cast<float4*>(&Bs[it / (BN / 4)][it % (BN / 4) * 4]) = rb[q];
        }
      }
    };
    // thread (ty, tx): rows 4 ty + 4 (BM / TM) * half .., columns likewise
    const int tx = tid % (BN / TN), ty = tid / (BN / TN);
    float acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
    if (kdim > 0) fetch(0);
    for (int k0 = 0; k0 < kdim; k0 += SBK) {
      __syncthreads();
      stage();
      __syncthreads();
      if (k0 + SBK < kdim) fetch(k0 + SBK);
#pragma unroll
      for (int kk = 0; kk < SBK; ++kk) {
        float fa[TM], fb[TN];
#pragma unroll
        for (int h = 0; h < TM / 4; ++h)
          *reinterpret_cast<float4*>(fa + 4 * h) =
              *reinterpret_cast<const float4*>(&As[kk][h * (BM / TM) * 4 + ty * 4]);
#pragma unroll
        for (int h = 0; h < TN / 4; ++h)
          *reinterpret_cast<float4*>(fb + 4 * h) =
              *reinterpret_cast<const float4*>(&Bs[kk][h * (BN / TN) * 4 + tx * 4]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(fa[i], fb[j], acc[i][j]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = m0 + (i / 4) * (BM / TM) * 4 + ty * 4 + (i & 3);
      if (r >= mlim) continue;
      float* dst = kMode == 2 ? args.out + ((size_t)g * args.n + r) * args.k
                              : args.out + (size_t)(first + r) * cols;
#pragma unroll
      for (int h = 0; h < TN / 4; ++h) {
        const int c = n0 + h * (BN / TN) * 4 + tx * 4;
        if constexpr (kVec) {
          if (c < cols)
            *reinterpret_cast<float4*>(dst + c) = make_float4(
                acc[i][4 * h], acc[i][4 * h + 1], acc[i][4 * h + 2], acc[i][4 * h + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < cols) dst[c + j] = acc[i][4 * h + j];
        }
      }
    }
  }
}

template <int kMode, int BM, int BN, int TM, int TN>
cudaError_t launch(const SArgs& a, long long units, cudaStream_t st) {
  const int grid = (int)(units < 148 * 32 ? units : 148 * 32);
  if (a.n % 4 == 0 && a.k % 4 == 0)  // rows on 16-byte boundaries
    grouped_matmul_fp32_kernel<kMode, BM, BN, TM, TN, true><<<grid, SThreads, 0, st>>>(a);
  else
    grouped_matmul_fp32_kernel<kMode, BM, BN, TM, TN, false><<<grid, SThreads, 0, st>>>(a);
  return note_cuda(cudaGetLastError(), "fp32 grouped matmul launch");
}

template <int kMode>
cudaError_t launch_mode(const SArgs& a, cudaStream_t st) {
  const int cols = kMode == 0 ? a.n : a.k;
  auto units = [&](int bm, int bn) {
    const long long mt = kMode == 2 ? (long long)a.E * ((a.n + bm - 1) / bm)
                                    : a.R / bm + (a.R < a.E ? a.R : a.E);
    return mt * ((cols + bn - 1) / bn);
  };
  if (units(128, 128) >= 2 * num_sms()) return launch<kMode, 128, 128, 8, 8>(a, units(128, 128), st);
  return launch<kMode, 64, 64, 4, 4>(a, units(64, 64), st);
}

}  // namespace

int launch_grouped_matmul_fp32(int mode, const float* a, const float* b, int R,
                               const int32_t* offsets, int E, int n, int k, float* out, void* ws,
                               cudaStream_t st) {
  const SArgs s{a, b, out, offsets, static_cast<uint32_t*>(ws), E, R, n, k};
  const cudaError_t e = mode == 0   ? launch_mode<0>(s, st)
                        : mode == 1 ? launch_mode<1>(s, st)
                                    : launch_mode<2>(s, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
