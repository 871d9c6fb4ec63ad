// Layer norm of the rows in front of the layer, and its backward pass:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
//   y    = (x - mean) rstd w + b
//   h    = dy w,  z = (x - mean) rstd
//   dx   = rstd (h - mean(h) - z mean(h z)),  dw = sum_rows dy z,  db = sum_rows dy
//
// Both passes are bound by HBM: a row is read once into registers, reduced,
// and written.  kT threads share a row (a warp up to 1024 columns, then 128,
// 256 or 512 threads); each holds up to 32 of its elements, in 16-byte pieces
// when the rows are 16-byte aligned, else one by one.  The next row's loads are
// issued before the current row is reduced.
//
// Statistics: each thread takes the mean and the centred square sum of its own
// elements, and pairs (count, mean, M2) are merged by Chan's update, so one
// block-wide exchange suffices and a large common offset does not cancel.
//
// dw and db: every CTA keeps the column sums of its rows in registers (its
// thread groups added in order at the end) and writes one fp32 partial row;
// a second kernel adds the partial rows in order.  No atomics: repeated calls
// give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxD = 16384;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// A row as kT threads hold it: piece p of thread t is elements
// (p * kT + t) * VEC .. + VEC - 1, present when its first element is below d
// (d is a multiple of VEC).
template <typename T, int VEC, int PIECES, int kT>
struct RowRegs {
  struct alignas(sizeof(T) * VEC) Piece {
    T v[VEC];
  };
  Piece p[PIECES];
  __device__ __forceinline__ void load(const T* row, int t, int d) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (i * kT + t) * VEC;
      if (c < d) p[i] = *reinterpret_cast<const Piece*>(row + c);
    }
  }
};

template <int VEC>
struct alignas(VEC >= 4 ? 16 : 4 * VEC) F32Piece {
  float v[VEC];
};

struct Stat {
  float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float f = __fdividef(b.n, n), d = b.mean - a.mean;
  return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Stat shfl(const Stat& s, int o) {
  return {__shfl_xor_sync(0xffffffffu, s.n, o), __shfl_xor_sync(0xffffffffu, s.mean, o),
          __shfl_xor_sync(0xffffffffu, s.m2, o)};
}
// The merge in lane order from either side gives both lanes the same bits.
__device__ __forceinline__ Stat warp_merge(Stat s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Stat t = shfl(s, o);
    s = (lane & o) ? merge(t, s) : merge(s, t);
  }
  return s;
}

template <typename T, int VEC, int PIECES, int kT>
__global__ void __launch_bounds__(kT < 128 ? 128 : kT) layer_norm_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, float eps,
    int R, int d, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kWarps = kT / 32;
  constexpr int kGroups = (kT < 128 ? 128 : kT) / kT;  // rows a CTA works on at once
  __shared__ Stat part[2][kWarps];
  const int t = threadIdx.x % kT, group = threadIdx.x / kT;
  const int warp = t >> 5, lane = t & 31;
  const int step = gridDim.x * kGroups;
  int r = blockIdx.x * kGroups + group;
  RowRegs<T, VEC, PIECES, kT> cur, next;
  if (r < R) cur.load(x + (size_t)r * d, t, d);
  // with several warps a row, every warp of the CTA sees the same r
  for (int it = 0; r < R; r += step, ++it) {
    if (r + step < R && r + step > r) next.load(x + (size_t)(r + step) * d, t, d);
    Stat s{0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if ((i * kT + t) * VEC < d) {
        s.n += VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.mean += to_f32(cur.p[i].v[e]);
      }
    if (s.n > 0.f) s.mean = __fdividef(s.mean, s.n);
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if ((i * kT + t) * VEC < d) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float c = to_f32(cur.p[i].v[e]) - s.mean;
          s.m2 = fmaf(c, c, s.m2);
        }
      }
    s = warp_merge(s);
    if constexpr (kWarps > 1) {
      Stat* buf = part[it & 1];
      if (lane == 0) buf[warp] = s;
      __syncthreads();
      s = buf[0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) s = merge(s, buf[i]);
    }
    const float mu = s.mean, rs = rsqrtf(s.m2 / (float)d + eps);
    if (t == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    T* yrow = y + (size_t)r * d;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (i * kT + t) * VEC;
      if (c < d) {
        using Piece = typename RowRegs<T, VEC, PIECES, kT>::Piece;
        Piece o;
        float wv[VEC], bv[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e += (VEC < 4 ? VEC : 4)) {
          constexpr int S = VEC < 4 ? VEC : 4;
          *reinterpret_cast<F32Piece<S>*>(wv + e) =
              *reinterpret_cast<const F32Piece<S>*>(w + c + e);
          if (b != nullptr)
            *reinterpret_cast<F32Piece<S>*>(bv + e) =
                *reinterpret_cast<const F32Piece<S>*>(b + c + e);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float z = (to_f32(cur.p[i].v[e]) - mu) * rs;
          o.v[e] = from_f32<T>(b != nullptr ? fmaf(z, wv[e], bv[e]) : z * wv[e]);
        }
        *reinterpret_cast<Piece*>(yrow + c) = o;
      }
    }
    cur = next;
    if (r + step < r) break;  // the row index would pass 2^31
  }
}

// One partial row of dw and db per CTA: part [gridDim.x][2][d].
template <typename T, int VEC, int PIECES, int kT>
__global__ void __launch_bounds__(kT < 128 ? 128 : kT) layer_norm_bwd_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, int R, int d,
    T* __restrict__ dx, float* __restrict__ part) {
  constexpr int kWarps = kT / 32;
  constexpr int kGroups = (kT < 128 ? 128 : kT) / kT;
  __shared__ float2 red[2][kWarps];
  extern __shared__ float gsum[];  // kGroups > 1: [2][d]
  const int t = threadIdx.x % kT, group = threadIdx.x / kT;
  const int warp = t >> 5, lane = t & 31;
  const int step = gridDim.x * kGroups;
  int r = blockIdx.x * kGroups + group;
  RowRegs<T, VEC, PIECES, kT> cx, cd, nx, nd;
  float aw[PIECES][VEC], ab[PIECES][VEC];
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) aw[i][e] = ab[i][e] = 0.f;
  if (r < R) {
    cx.load(x + (size_t)r * d, t, d);
    cd.load(dy + (size_t)r * d, t, d);
  }
  const float inv_d = 1.f / (float)d;
  for (int it = 0; r < R; r += step, ++it) {
    const float mu = mean[r], rs = rstd[r];
    if (r + step < R && r + step > r) {
      nx.load(x + (size_t)(r + step) * d, t, d);
      nd.load(dy + (size_t)(r + step) * d, t, d);
    }
    float s1 = 0.f, s2 = 0.f;
    float wv[PIECES][VEC];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (i * kT + t) * VEC;
      if (c < d) {
#pragma unroll
        for (int e = 0; e < VEC; e += (VEC < 4 ? VEC : 4)) {
          constexpr int S = VEC < 4 ? VEC : 4;
          *reinterpret_cast<F32Piece<S>*>(wv[i] + e) =
              *reinterpret_cast<const F32Piece<S>*>(w + c + e);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float g = to_f32(cd.p[i].v[e]);
          const float z = (to_f32(cx.p[i].v[e]) - mu) * rs;
          const float h = g * wv[i][e];
          s1 += h;
          s2 = fmaf(h, z, s2);
          aw[i][e] = fmaf(g, z, aw[i][e]);
          ab[i][e] += g;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if constexpr (kWarps > 1) {
      float2* buf = red[it & 1];
      if (lane == 0) buf[warp] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        s1 += buf[i].x;
        s2 += buf[i].y;
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
    T* drow = dx + (size_t)r * d;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (i * kT + t) * VEC;
      if (c < d) {
        typename RowRegs<T, VEC, PIECES, kT>::Piece o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float z = (to_f32(cx.p[i].v[e]) - mu) * rs;
          o.v[e] = from_f32<T>(rs * (to_f32(cd.p[i].v[e]) * wv[i][e] - s1 - z * s2));
        }
        *reinterpret_cast<typename RowRegs<T, VEC, PIECES, kT>::Piece*>(drow + c) = o;
      }
    }
    cx = nx;
    cd = nd;
    if (r + step < r) break;
  }
  float* prow = part + (size_t)blockIdx.x * 2 * d;
  if constexpr (kGroups > 1) {
    // the groups' sums are added in group order
    for (int g = 0; g < kGroups; ++g) {
      if (group == g) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int c = (i * kT + t) * VEC + e;
            if (c < d) {
              if (g > 0) {
                aw[i][e] += gsum[c];
                ab[i][e] += gsum[d + c];
              }
              gsum[c] = aw[i][e];
              gsum[d + c] = ab[i][e];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) prow[c] = gsum[c];
  } else {
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * kT + t) * VEC + e;
        if (c < d) {
          prow[c] = aw[i][e];
          prow[d + c] = ab[i][e];
        }
      }
  }
}

// out[c] = sum over the P partial rows, in a fixed order: 8 chains of rows
// p, p + 8, .. per column, added in chain order.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* __restrict__ part, int P,
                                                          int d, float* __restrict__ dw,
                                                          float* __restrict__ db) {
  __shared__ float s[8][33];
  const int cx = threadIdx.x & 31, cy = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float v = 0.f;
  if (c < 2 * d)
    for (int p = cy; p < P; p += 8) v += part[(size_t)p * 2 * d + c];
  s[cy][cx] = v;
  __syncthreads();
  if (cy == 0 && c < 2 * d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][cx];
    if (c < d)
      dw[c] = v;
    else if (db != nullptr)
      db[c - d] = v;
  }
}

// CTAs of the backward kernel = partial rows: at most two per SM.
int bwd_ctas(int R, int d) {
  const int groups = d <= 1024 ? 4 : 1;
  const long long want = ((long long)R + groups - 1) / groups;
  return (int)(want < 2 * 148 ? (want < 1 ? 1 : want) : 2 * 148);
}

struct Fwd {
  const void* x;
  const float *w, *b;
  float eps;
  int R, d;
  void* y;
  float *mean, *rstd;
};
struct Bwd {
  const void *dy, *x;
  const float *w, *mean, *rstd;
  int R, d;
  void* dx;
  float* part;
};

template <typename T, int VEC, int PIECES, int kT>
void go(const Fwd& a, cudaStream_t st) {
  constexpr int kBlock = kT < 128 ? 128 : kT;
  const long long want = ((long long)a.R + kBlock / kT - 1) / (kBlock / kT);
  const int cap = 148 * (1024 / kBlock);
  layer_norm_kernel<T, VEC, PIECES, kT><<<(int)(want < cap ? want : cap), kBlock, 0, st>>>(
      static_cast<const T*>(a.x), a.w, a.b, a.eps, a.R, a.d, static_cast<T*>(a.y), a.mean, a.rstd);
}
template <typename T, int VEC, int PIECES, int kT>
void go(const Bwd& a, cudaStream_t st) {
  constexpr int kBlock = kT < 128 ? 128 : kT;
  const size_t smem = kBlock > kT ? (size_t)2 * a.d * 4 : 0;
  layer_norm_bwd_kernel<T, VEC, PIECES, kT><<<bwd_ctas(a.R, a.d), kBlock, smem, st>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.mean, a.rstd, a.R, a.d,
      static_cast<T*>(a.dx), a.part);
}

// Threads per row and elements per thread by width: as few threads as hold the
// row in 32 elements each, fewer elements for short rows.
template <typename T, int VEC, typename Args>
void by_width(const Args& a, cudaStream_t st) {
  if (a.d <= 256) go<T, VEC, 8 / VEC, 32>(a, st);
  else if (a.d <= 512) go<T, VEC, 16 / VEC, 32>(a, st);
  else if (a.d <= 1024) go<T, VEC, 32 / VEC, 32>(a, st);
  else if (a.d <= 2048) go<T, VEC, 16 / VEC, 128>(a, st);
  else if (a.d <= 4096) go<T, VEC, 32 / VEC, 128>(a, st);
  else if (a.d <= 8192) go<T, VEC, 32 / VEC, 256>(a, st);
  else go<T, VEC, 32 / VEC, 512>(a, st);
}
template <typename Args>
void by_type(const Args& a, int dtype, cudaStream_t st) {
  if (dtype == MOE_DTYPE_BF16) {
    if (a.d % 8 == 0) by_width<__nv_bfloat16, 8>(a, st);
    else by_width<__nv_bfloat16, 1>(a, st);
  } else {
    if (a.d % 4 == 0) by_width<float, 4>(a, st);
    else by_width<float, 1>(a, st);
  }
}

}  // namespace

int layer_norm_max_d() { return kMaxD; }

size_t layer_norm_ws_bytes(int R, int d) { return (size_t)bwd_ctas(R, d) * 2 * d * 4; }

cudaError_t launch_layer_norm(int dtype, const void* x, const float* w, const float* b, float eps,
                              int R, int d, void* y, float* mean, float* rstd, cudaStream_t st) {
  by_type(Fwd{x, w, b, eps, R, d, y, mean, rstd}, dtype, st);
  return note_cuda(cudaGetLastError(), "layer norm launch");
}

cudaError_t launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* w,
                                       const float* mean, const float* rstd, int R, int d,
                                       void* dx, float* dw, float* db, void* ws,
                                       cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  by_type(Bwd{dy, x, w, mean, rstd, R, d, dx, part}, dtype, st);
  cudaError_t e = note_cuda(cudaGetLastError(), "layer norm backward launch");
  if (e != cudaSuccess) return e;
  column_sums_kernel<<<(2 * d + 31) / 32, 256, 0, st>>>(part, bwd_ctas(R, d), d, dw, db);
  return note_cuda(cudaGetLastError(), "layer norm column sums launch");
}

}  // namespace moe
