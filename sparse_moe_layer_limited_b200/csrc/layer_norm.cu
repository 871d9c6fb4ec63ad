// Layer norm of the rows in front of the layer, and its backward pass:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
//   y    = (x - mean) rstd w + b
//   h    = dy w,  z = (x - mean) rstd
//   dx   = rstd (h - mean(h) - z mean(h z)),  dw = sum_rows dy z,  db = sum_rows dy
//
// Both passes are bound by HBM: a row is read once, reduced, and written.
//   narrow, or not in whole 16-byte pieces up to 1024 columns: a warp per row,
//                        up to 32 elements a lane in registers, the next row
//                        loaded while the current one is reduced
//   rows in whole 16-byte pieces (row_kernel, row_bwd_kernel): a CTA of
//                        one thread per two pieces works on two rows at a time,
//                        with one block barrier, while bulk copies bring the next
//                        four rows into shared memory (172 KB of ring per SM in
//                        the backward at 7168 columns)
//   the other wide ones  128 to 512 threads a row, elements in registers
//
// Statistics: each thread takes the mean and the centred square sum of its own
// elements, and (count, mean, M2) are merged by Chan's update, so a large
// common offset does not cancel.
//
// dw and db: every CTA keeps the column sums of its rows in registers (its
// thread groups added in order at the end) and writes one fp32 partial row;
// a second kernel adds the partial rows in order.  No atomics: repeated calls
// give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "f32x2.cuh"
#include "internal.h"
#include "ptx.cuh"

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

// ---- rows of 16-byte pieces, one thread per piece -------------------------------------
__device__ __forceinline__ float both(f32x2 v) {
  const float2 f = split2(v);
  return f.x + f.y;
}

// A 16-byte piece of a row as pairs.
__device__ __forceinline__ void bulk_load(const void* smem, const void* gmem, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem)),
      "l"(gmem), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
template <typename T>
struct Pack {
  static constexpr int N = 16 / sizeof(T), P = N / 2;
};
__device__ __forceinline__ void unpack(const uint4& u, f32x2 (&v)[4], __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pair2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4& u, f32x2 (&v)[2], float) {
  v[0] = pair2(__uint_as_float(u.x), __uint_as_float(u.y));
  v[1] = pair2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 pack(const f32x2 (&v)[4], __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = split2(v[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const f32x2 (&v)[2], float) {
  const float2 a = split2(v[0]), b = split2(v[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                    __float_as_uint(b.y));
}
template <int P>
__device__ __forceinline__ void load_f32(const float* p, f32x2 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p + 2 * i));
    v[i] = pair2(f.x, f.y);
    v[i + 1] = pair2(f.z, f.w);
  }
}

// Sums over a warp of N values (1, 2 or 4) at once: every exchange halves the
// values a lane carries, so 4 values take 6 exchanges instead of 20.  Lane l
// ends with the total of value slot(l) = l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n /= 2, o /= 2) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[n / 2 + i] : v[i], give = up ? v[i] : v[n / 2 + i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float r = v[0];
#pragma unroll
  for (; o > 0; o /= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}
// Block-wide sums of N values, given each warp's in buf[value][warp]: value i
// to every lane.  Two warps' values a lane and 32 / N lanes a value.
template <int N>
__device__ __forceinline__ void block_sums(const float (*buf)[32], int warps, float (&out)[N]) {
  constexpr int L = 32 / N;
  const int lane = threadIdx.x & 31, w = lane % L;
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (w + i * L < warps) r += buf[lane / L][w + i * L];
#pragma unroll
  for (int o = L / 2; o > 0; o /= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __shfl_sync(0xffffffffu, r, i * L);
}

// A CTA's rows blockIdx.x, blockIdx.x + gridDim.x, .. on their way through the
// ring, ROWS at a time: one thread orders whole rows as bulk copies, which land
// on a barrier per slot.
// A wait gives up after a second or two: false, and the caller's rows are NaN.
template <typename T, int OPS, int PIECES, int ROWS, int S>
struct Ring {
  const T* src[OPS];
  const uint4* mem;
  uint64_t* bar;           // [S / ROWS]
  size_t row_step;         // elements from one of the CTA's rows to the next
  uint32_t row_bytes, slot_bytes;
  int rows, fetched, put, get;
  uint32_t phase;          // parity of the slot to be read next
  bool in[PIECES];         // this thread's piece i exists
  __device__ __forceinline__ Ring(const uint4* ring, uint64_t* bars, int n, int d) {
    const int kT = blockDim.x, t = threadIdx.x;
    mem = ring;
    bar = bars;
    row_bytes = (uint32_t)d * sizeof(T);
    slot_bytes = OPS * PIECES * (uint32_t)kT * 16;
    row_step = (size_t)gridDim.x * d;
    rows = n;
    fetched = put = get = 0;
    phase = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) in[i] = (i * kT + t) * (int)(16 / sizeof(T)) < d;
    if (t == 0) {
      for (int i = 0; i < S / ROWS; ++i) mbar_init(&bars[i], 1);
      fence_barrier_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ void operand(int op, const T* p, int d) {
    src[op] = p + (size_t)blockIdx.x * d;
  }
  // Thread 0: the next ROWS rows into their slots, which every thread has read.
  __device__ __forceinline__ void fetch() {
    const int n = min(ROWS, rows - fetched);
    if (n > 0) {
      mbar_arrive_expect_tx(&bar[put], (uint32_t)(n * OPS) * row_bytes);
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int op = 0; op < OPS; ++op)
          bulk_load(at(put * ROWS + k, op, 0), src[op] + (size_t)(fetched + k) * row_step,
                    row_bytes, &bar[put]);
      fetched += n;
      put = put + 1 == S / ROWS ? 0 : put + 1;
    }
  }
  __device__ __forceinline__ bool wait() {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(&bar[get], phase)) return true;
      if ((it & 255u) == 0) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > 2000000000ull) return false;
      }
    }
  }
  __device__ __forceinline__ const uint4* at(int slot, int op, int i) const {
    return mem + ((slot * OPS + op) * PIECES + i) * (int)blockDim.x;
  }
  __device__ __forceinline__ uint4 read(int k, int op, int i) const {
    return at(get * ROWS + k, op, i)[threadIdx.x];
  }
  __device__ __forceinline__ void next() {
    if (++get == S / ROWS) {
      get = 0;
      phase ^= 1u;
    }
  }
};

// ROWS rows at a time: their reductions overlap, and a reduction's instructions
// are shared by 16 elements a thread.  8192 x 7168 bf16: forward 54 us (4.4
// TB/s, 0.66 of the measured copy), backward 84 us with the column sums (4.2
// TB/s); what is left is instruction issue and the wait for a row's reduction.
// Measured and not taken: 8 elements a thread and one row at a time, a CTA of
// 896 threads (72 and 116 us); one row at a time in two CTAs an SM (52 and
// 100 us); 16-byte copies by every thread (54 and 96 us).
template <typename T, int PIECES, int ROWS, int S>
__global__ void __launch_bounds__(ROWS == 2 ? 512 : 1024) row_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, float eps,
    int R, int d, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  static_assert(S % ROWS == 0 && S > ROWS, "whole iterations in the ring");
  constexpr int V = Pack<T>::N, P = Pack<T>::P;
  extern __shared__ uint4 ring[];        // [S][PIECES][kT]
  __shared__ float part[2][ROWS][3][32];   // count, mean, M2 of each warp
  const int kT = blockDim.x, t = threadIdx.x, warp = t >> 5, lane = t & 31, warps = kT >> 5;
  const int rows = (R - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // this CTA's
  __shared__ uint64_t bars[S / ROWS];
  Ring<T, 1, PIECES, ROWS, S> in(ring, bars, rows, d);
  in.operand(0, x, d);
  if (t == 0)
    for (int i = 0; i < S; i += ROWS) in.fetch();
  f32x2 wv[PIECES][P], bv[PIECES][P];  // this thread's columns never change
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = (i * kT + t) * V;
#pragma unroll
    for (int e = 0; e < P; ++e) wv[i][e] = bv[i][e] = 0ull;
    if (c < d) {
      load_f32(w + c, wv[i]);
      if (b != nullptr) load_f32(b + c, bv[i]);
    }
  }
  const float inv_d = 1.f / (float)d;
  // all lanes of the warp hold PIECES whole pieces
  const bool whole = ((PIECES - 1) * kT + (warp + 1) * 32) * V <= d;
  int flip = 0;
  size_t row = blockIdx.x;
  for (int done = 0; done < rows; done += ROWS, flip ^= 1) {
    const bool landed = in.wait();
    f32x2 v[ROWS][PIECES][P];
    Stat s[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      s[k] = Stat{0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (in.in[i]) {
          unpack(in.read(k, 0, i), v[k][i], T{});
          f32x2 sum = v[k][i][0];
#pragma unroll
          for (int e = 1; e < P; ++e) sum = add2(sum, v[k][i][e]);
          const float m = both(sum) * (1.f / V);
          const f32x2 m1 = pair2(-m, -m);
          f32x2 sq = 0ull;
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f32x2 c = add2(v[k][i][e], m1);
            sq = fma2(c, c, sq);
          }
          const float m2 = both(sq);
          if (i == 0) {
            s[k] = Stat{(float)V, m, m2};
          } else {  // equal counts so far: i pieces and one more
            const float dm = m - s[k].mean;
            s[k].mean = fmaf(dm, 1.f / (i + 1), s[k].mean);
            s[k].m2 = fmaf(dm * dm, V * (float)i / (i + 1), s[k].m2 + m2);
            s[k].n += V;
          }
        }
    }
    in.next();
    if (whole) {  // equal counts: the merged mean is the middle of the two
      float n = PIECES * V;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1, n *= 2.f)
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
          const float m = __shfl_xor_sync(0xffffffffu, s[k].mean, o);
          const float m2 = __shfl_xor_sync(0xffffffffu, s[k].m2, o);
          const float dm = m - s[k].mean;
          s[k].mean = 0.5f * (s[k].mean + m);
          s[k].m2 = fmaf(dm * dm, 0.5f * n, s[k].m2 + m2);
          s[k].n = 2.f * n;
        }
    } else {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) s[k] = warp_merge(s[k]);
    }
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        part[flip][k][0][warp] = s[k].n;
        part[flip][k][1][warp] = s[k].mean;
        part[flip][k][2][warp] = s[k].m2;
      }
    __syncthreads();
    if (t == 0) in.fetch();  // every thread has read these rows' slots
    // the warps' statistics: mean first, then the squares around it.  Lanes
    // 0-15 take the first row, lanes 16-31 the second (ROWS == 1: all lanes)
    constexpr int L = 32 / ROWS;
    const int k0 = lane / L, w0 = lane % L;
    float cn[ROWS], cm[ROWS], cs[ROWS], a = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int q = w0 + i * L;
      const bool in = q < warps;
      cn[i] = in ? part[flip][k0][0][q] : 0.f;
      cm[i] = in ? part[flip][k0][1][q] : 0.f;
      cs[i] = in ? part[flip][k0][2][q] : 0.f;
      a = fmaf(cn[i], cm[i], a);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const float mk = a * inv_d;
    a = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float dm = cm[i] - mk;
      a += fmaf(cn[i] * dm, dm, cs[i]);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const float rk1 = landed ? rsqrtf(a * inv_d + eps) : __int_as_float(0x7fffffff);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (done + k >= rows) break;
      const float mu = __shfl_sync(0xffffffffu, mk, k * L), rs = __shfl_sync(0xffffffffu, rk1, k * L);
      if (t == 0) {
        mean[row] = mu;
        rstd[row] = rs;
      }
      const f32x2 mu2 = pair2(-mu, -mu), rs2 = pair2(rs, rs);
      T* dst = y + row * d;
      row += gridDim.x;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int c = (i * kT + t) * V;
        if (c < d) {
#pragma unroll
          for (int e = 0; e < P; ++e)
            v[k][i][e] = fma2(mul2(add2(v[k][i][e], mu2), rs2), wv[i][e], bv[i][e]);
          *reinterpret_cast<uint4*>(dst + c) = pack(v[k][i], T{});
        }
      }
    }
  }
}

// One partial row of dw and db per CTA, as below.  kExact: every thread has all
// its pieces (d = 2 kT pieces), so nothing is predicated.
template <typename T, int PIECES, int ROWS, int S, int kThreads, bool kExact>
__global__ void __launch_bounds__(kThreads) row_bwd_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, int R, int d,
    T* __restrict__ dx, float* __restrict__ part) {
  static_assert(S % ROWS == 0 && S > ROWS, "whole iterations in the ring");
  constexpr int V = Pack<T>::N, P = Pack<T>::P;
  extern __shared__ uint4 ring[];  // [S][2][PIECES][kT]
  __shared__ float red[2][2 * ROWS][32];
  __shared__ uint64_t bars[S / ROWS];
  const int kT = blockDim.x, t = threadIdx.x, warp = t >> 5, lane = t & 31, warps = kT >> 5;
  const int rows = (R - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // this CTA's
  Ring<T, 2, PIECES, ROWS, S> in(ring, bars, rows, d);
  in.operand(0, x, d);
  in.operand(1, dy, d);
  if (t == 0)
    for (int i = 0; i < S; i += ROWS) in.fetch();
  f32x2 wv[PIECES][P], aw[PIECES][P], ab[PIECES][P];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = (i * kT + t) * V;
#pragma unroll
    for (int e = 0; e < P; ++e) wv[i][e] = aw[i][e] = ab[i][e] = 0ull;
    if (kExact || c < d) load_f32(w + c, wv[i]);
  }
  const float inv_d = 1.f / (float)d;
  float mu[ROWS], rs[ROWS];
  const float* mp = mean + blockIdx.x;
  const float* rp = rstd + blockIdx.x;
  auto row_stats = [&](int at, float (&m)[ROWS], float (&q)[ROWS]) {  // rows at, at + 1, ..
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      m[k] = q[k] = 0.f;
      if (at + k < rows) {
        m[k] = __ldg(mp);
        q[k] = __ldg(rp);
        mp += gridDim.x;
        rp += gridDim.x;
      }
    }
  };
  row_stats(0, mu, rs);
  char* dst = reinterpret_cast<char*>(dx + (size_t)blockIdx.x * d) + t * 16;
  int flip = 0;
  for (int done = 0; done < rows; done += ROWS, flip ^= 1) {
    float mu1[ROWS], rs1[ROWS];  // the next rows'
    row_stats(done + ROWS, mu1, rs1);
    if (!in.wait())
#pragma unroll
      for (int k = 0; k < ROWS; ++k) mu[k] = __int_as_float(0x7fffffff);
    f32x2 z[ROWS][PIECES][P], h[ROWS][PIECES][P];
    float sums[2 * ROWS];  // h of each row, then h z of each row
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      f32x2 s1 = 0ull, s2 = 0ull;
      if (done + k < rows) {
        const f32x2 mu2 = pair2(-mu[k], -mu[k]), rs2 = pair2(rs[k], rs[k]);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if (kExact || in.in[i]) {
            f32x2 g[P];
            unpack(in.read(k, 0, i), z[k][i], T{});
            unpack(in.read(k, 1, i), g, T{});
#pragma unroll
            for (int e = 0; e < P; ++e) {
              z[k][i][e] = mul2(add2(z[k][i][e], mu2), rs2);
              h[k][i][e] = mul2(g[e], wv[i][e]);
              s1 = add2(s1, h[k][i][e]);
              s2 = fma2(h[k][i][e], z[k][i][e], s2);
              aw[i][e] = fma2(g[e], z[k][i][e], aw[i][e]);
              ab[i][e] = add2(ab[i][e], g[e]);
            }
          }
      }
      sums[k] = both(s1);
      sums[ROWS + k] = both(s2);
    }
    in.next();
    const float mine = warp_sums<2 * ROWS>(sums);
    if (lane % (16 / ROWS) == 0) red[flip][lane / (16 / ROWS)][warp] = mine;
    __syncthreads();
    if (t == 0) in.fetch();  // every thread has read these rows' slots
    block_sums<2 * ROWS>(red[flip], warps, sums);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (done + k >= rows) break;
      // dx = rs h - rs (mean(h) + z mean(h z))
      const float a = -rs[k] * (sums[k] * inv_d), c = -rs[k] * (sums[ROWS + k] * inv_d);
      const f32x2 rs2 = pair2(rs[k], rs[k]), a2 = pair2(a, a), c2 = pair2(c, c);
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (kExact || in.in[i]) {
#pragma unroll
          for (int e = 0; e < P; ++e)
            z[k][i][e] = fma2(h[k][i][e], rs2, fma2(z[k][i][e], c2, a2));
          *reinterpret_cast<uint4*>(dst + i * kT * 16) = pack(z[k][i], T{});
        }
      dst += in.row_step * sizeof(T);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      mu[k] = mu1[k];
      rs[k] = rs1[k];
    }
  }
  float* prow = part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = (i * kT + t) * V;
    if (c < d) {
#pragma unroll
      for (int e = 0; e < P; e += 2) {
        *reinterpret_cast<ulonglong2*>(prow + c + 2 * e) = make_ulonglong2(aw[i][e], aw[i][e + 1]);
        *reinterpret_cast<ulonglong2*>(prow + d + c + 2 * e) =
            make_ulonglong2(ab[i][e], ab[i][e + 1]);
      }
    }
  }
}

// ---- elements in registers --------------------------------------------------------------
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

// out[c] = sum over the P partial rows, in a fixed order: 32 chains of rows p,
// p + 32, .. per column, then the chains.  A thread owns 4 columns (1 where d is
// odd) of its chain.  Launched to overlap the end of the kernel before it.
template <int V>
__global__ void __launch_bounds__(256) column_sums_kernel(const float* __restrict__ part, int P,
                                                          int d, float* __restrict__ dw,
                                                          float* __restrict__ db) {
  __shared__ float s[32][8 * V + 1];
  const int cx = threadIdx.x & 7, cy = threadIdx.x >> 3;
  const int c = (blockIdx.x * 8 + cx) * V;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v[V] = {};
  if (c < 2 * d) {
#pragma unroll 4
    for (int p = cy; p < P; p += 32) {
      const float* src = part + (size_t)p * 2 * d + c;
      if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        v[0] += f.x;
        v[1] += f.y;
        v[2] += f.z;
        v[3] += f.w;
      } else {
        v[0] += *src;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s[cy][cx * V + e] = v[e];
  __syncthreads();
  const int t = threadIdx.x, out = blockIdx.x * 8 * V + t;
  if (t < 8 * V && out < 2 * d) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][t];
    if (out < d)
      dw[out] = sum;
    else if (db != nullptr)
      db[out - d] = sum;
  }
}

// The row kernels take rows of whole 16-byte pieces, two pieces a thread.  Up to
// 16 KB a row: two rows at a time, a ring of six; up to 32 KB: one at a time, a
// ring of three (what fits in shared memory).  Narrower than `from` columns a
// warp per row holds its elements in registers: forward 512 (100000 x 320 bf16
// 60 us against 70, 30000 x 512 21 against 17), backward 257 (100000 x 320 113
// us against 80, 16384 x 1024 38 against 34).
constexpr int kFwdFrom = 512, kBwdFrom = 257;
bool by_rows(int d, int elem, int from) {
  return d >= from && d % (16 / elem) == 0 && d * elem <= 32768;
}
int row_threads(int d, int elem) { return ((d / (16 / elem) + 1) / 2 + 31) / 32 * 32; }
int rows_per_sm(int d, int elem) {  // CTAs of a row kernel on an SM: 512 threads in all
  const int t = row_threads(d, elem);
  return t >= 512 ? 1 : 512 / t;
}
// CTAs of the backward kernel = partial rows.
int bwd_ctas(int R, int d, int elem) {
  const bool rows = by_rows(d, elem, kBwdFrom);
  const int groups = !rows && d <= 1024 ? 4 : 1;
  const long long want = ((long long)R + groups - 1) / groups;
  const long long most = 148LL * (rows ? rows_per_sm(d, elem) : 2);
  return (int)(want < most ? (want < 1 ? 1 : want) : most);
}

struct Fwd {
  static constexpr int kFrom = kFwdFrom;
  const void* x;
  const float *w, *b;
  float eps;
  int R, d;
  void* y;
  float *mean, *rstd;
};
struct Bwd {
  static constexpr int kFrom = kBwdFrom;
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
  layer_norm_bwd_kernel<T, VEC, PIECES, kT><<<bwd_ctas(a.R, a.d, sizeof(T)), kBlock, smem, st>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.mean, a.rstd, a.R, a.d,
      static_cast<T*>(a.dx), a.part);
}

template <typename T, int ROWS, int S>
cudaError_t rows_launch(const Fwd& a, cudaStream_t st) {
  const int kT = row_threads(a.d, sizeof(T));
  const size_t smem = (size_t)S * 2 * kT * 16;
  auto kernel = row_kernel<T, 2, ROWS, S>;
  // the same opt-in for every width: host threads may call at the same time
  constexpr int most_smem = S * 2 * (ROWS == 2 ? 512 : 1024) * 16;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       most_smem);
  if (e != cudaSuccess) return e;
  const int most = 148 * rows_per_sm(a.d, sizeof(T));
  kernel<<<a.R < most ? a.R : most, kT, smem, st>>>(static_cast<const T*>(a.x), a.w, a.b, a.eps,
                                                    a.R, a.d, static_cast<T*>(a.y), a.mean,
                                                    a.rstd);
  return cudaGetLastError();
}
template <typename T, int ROWS, int S, int kThreads, bool kExact>
cudaError_t rows_launch_bwd(const Bwd& a, cudaStream_t st) {
  const int kT = row_threads(a.d, sizeof(T));
  const size_t smem = (size_t)S * 2 * 2 * kT * 16;
  auto kernel = row_bwd_kernel<T, 2, ROWS, S, kThreads, kExact>;
  constexpr int most_smem = S * 2 * 2 * kThreads * 16;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       most_smem);
  if (e != cudaSuccess) return e;
  kernel<<<bwd_ctas(a.R, a.d, sizeof(T)), kT, smem, st>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.mean, a.rstd, a.R, a.d,
      static_cast<T*>(a.dx), a.part);
  return cudaGetLastError();
}
template <typename T, int ROWS, int S>
cudaError_t rows_launch(const Bwd& a, cudaStream_t st) {
  const int kT = row_threads(a.d, sizeof(T));
  const bool exact = a.d == 2 * kT * (16 / (int)sizeof(T));
  if constexpr (ROWS == 2) {
    // up to 448 threads a thread may have 144 registers instead of 128
    if (kT <= 448)
      return exact ? rows_launch_bwd<T, ROWS, S, 448, true>(a, st)
                   : rows_launch_bwd<T, ROWS, S, 448, false>(a, st);
    return rows_launch_bwd<T, ROWS, S, 512, false>(a, st);
  } else {
    return rows_launch_bwd<T, ROWS, S, 1024, false>(a, st);
  }
}
template <typename T, typename Args>
cudaError_t rows(const Args& a, cudaStream_t st) {
  if (a.d * (int)sizeof(T) <= 16384) return rows_launch<T, 2, 6>(a, st);
  return rows_launch<T, 1, 3>(a, st);
}

// Elements in registers: as few threads per row as hold it in 32 elements each,
// fewer elements for short rows.  Aligned rows come here where they are narrow,
// or (fp32) wider than the row kernels take.
template <typename T, int VEC, typename Args>
void by_width(const Args& a, cudaStream_t st) {
  if (a.d <= 256) return go<T, VEC, 8 / VEC, 32>(a, st);
  if constexpr (VEC == 1 || Args::kFrom > 257) {
    if (a.d <= 512) return go<T, VEC, 16 / VEC, 32>(a, st);
  }
  if constexpr (VEC == 1) {
    if (a.d <= 1024) return go<T, VEC, 32, 32>(a, st);
    if (a.d <= 2048) return go<T, VEC, 16, 128>(a, st);
    if (a.d <= 4096) return go<T, VEC, 32, 128>(a, st);
    if (a.d <= 8192) return go<T, VEC, 32, 256>(a, st);
  }
  if constexpr (VEC == 1 || sizeof(T) == 4) go<T, VEC, 32 / VEC, 512>(a, st);
}
template <typename Args>
cudaError_t by_type(const Args& a, int dtype, cudaStream_t st) {
  if (by_rows(a.d, (int)dtype_bytes(dtype), Args::kFrom))
    return dtype == MOE_DTYPE_BF16 ? rows<__nv_bfloat16>(a, st) : rows<float>(a, st);
  if (dtype == MOE_DTYPE_BF16) {
    if (a.d % 8 == 0) by_width<__nv_bfloat16, 8>(a, st);
    else by_width<__nv_bfloat16, 1>(a, st);
  } else {
    if (a.d % 4 == 0) by_width<float, 4>(a, st);
    else by_width<float, 1>(a, st);
  }
  return cudaGetLastError();
}

}  // namespace

int layer_norm_max_d() { return kMaxD; }

size_t layer_norm_ws_bytes(int R, int d) {  // for either type
  const int a = bwd_ctas(R, d, 2), b = bwd_ctas(R, d, 4);
  return (size_t)(a > b ? a : b) * 2 * d * 4;
}

cudaError_t launch_layer_norm(int dtype, const void* x, const float* w, const float* b, float eps,
                              int R, int d, void* y, float* mean, float* rstd, cudaStream_t st) {
  return note_cuda(by_type(Fwd{x, w, b, eps, R, d, y, mean, rstd}, dtype, st),
                   "layer norm launch");
}

cudaError_t launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* w,
                                       const float* mean, const float* rstd, int R, int d,
                                       void* dx, float* dw, float* db, void* ws,
                                       cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  cudaError_t e = note_cuda(by_type(Bwd{dy, x, w, mean, rstd, R, d, dx, part}, dtype, st),
                            "layer norm backward launch");
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int P = bwd_ctas(R, d, (int)dtype_bytes(dtype)), v = d % 4 == 0 ? 4 : 1;
  cfg.gridDim = dim3((unsigned)((2 * d + 8 * v - 1) / (8 * v)), 1, 1);
  return note_cuda(cudaLaunchKernelEx(&cfg, v == 4 ? column_sums_kernel<4> : column_sums_kernel<1>,
                                      (const float*)part, P, d, dw, db),
                   "layer norm column sums launch");
}

}  // namespace moe
