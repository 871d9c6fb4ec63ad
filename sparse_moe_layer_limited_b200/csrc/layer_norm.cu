// Layer norm of the rows in front of the layer, and its backward pass:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
//   y    = (x - mean) rstd w + b
//   h    = dy w,  z = (x - mean) rstd
//   dx   = rstd (h - mean(h) - z mean(h z)),  dw = sum_rows dy z,  db = sum_rows dy
//
// Both passes are bound by HBM: a row is read once, reduced, and written.
//   rows of whole 16-byte pieces up to 32 KB (row_kernel, row_bwd_kernel): a CTA
//                        of one thread per two or four pieces, one block barrier
//                        a reduction, while bulk copies bring the next rows into
//                        shared memory (172 KB of ring per SM at 7168 columns)
//   the others           a warp, or 128 to 1024 threads, per row, up to 32
//                        elements a thread in registers, the next row loaded
//                        while the current one is reduced
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

// Without branches around its pieces, and two to four CTAs an SM: 8192 x 7001
// bf16 93 us, with them 131.
template <typename T, int VEC, int PIECES, int kT>
__global__ void __launch_bounds__(kT < 128 ? 128 : kT,
                                 kT < 128 ? 4 : kT < 512 ? 512 / kT : 1) layer_norm_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, float eps,
    int R, int d, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kWarps = kT / 32;
  constexpr int kGroups = (kT < 128 ? 128 : kT) / kT;  // rows a CTA works on at once
  __shared__ Stat part[2][kWarps];
  const int t = threadIdx.x % kT, group = threadIdx.x / kT;
  const int warp = t >> 5, lane = t & 31;
  const int step = gridDim.x * kGroups;
  int r = blockIdx.x * kGroups + group;
  RowRegs<T, VEC, PIECES, kT> cur{}, next{};  // absent pieces stay zeros
  if (r < R) cur.load(x + (size_t)r * d, t, d);
  // with several warps a row, every warp of the CTA sees the same r
  for (int it = 0; r < R; r += step, ++it) {
    if (r + step < R) next.load(x + (size_t)(r + step) * d, t, d);
    Stat s{0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      s.n += (i * kT + t) * VEC < d ? (float)VEC : 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) s.mean += to_f32(cur.p[i].v[e]);
    }
    if (s.n > 0.f) s.mean = __fdividef(s.mean, s.n);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const bool has = (i * kT + t) * VEC < d;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float c = has ? to_f32(cur.p[i].v[e]) - s.mean : 0.f;
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
      typename RowRegs<T, VEC, PIECES, kT>::Piece o;
      float wv[VEC], bv[VEC];
#pragma unroll
      for (int e = 0; e < VEC; e += (VEC < 4 ? VEC : 4)) {
        constexpr int S = VEC < 4 ? VEC : 4;
        F32Piece<S> p{}, q{};
        if (c < d) p = *reinterpret_cast<const F32Piece<S>*>(w + c + e);
        if (c < d && b != nullptr) q = *reinterpret_cast<const F32Piece<S>*>(b + c + e);
        *reinterpret_cast<F32Piece<S>*>(wv + e) = p;
        *reinterpret_cast<F32Piece<S>*>(bv + e) = q;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o.v[e] = from_f32<T>(fmaf((to_f32(cur.p[i].v[e]) - mu) * rs, wv[e], bv[e]));
      if (c < d) *reinterpret_cast<typename RowRegs<T, VEC, PIECES, kT>::Piece*>(yrow + c) = o;
    }
    cur = next;
  }
}

// ---- rows of 16-byte pieces, two or four to a thread -------------------------------------
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

// ROWS rows at a time.  kExact: every thread has all its pieces (d = PIECES kT
// pieces); otherwise a piece that a thread lacks is zeros that count for
// nothing.  Either way the code between the barriers has no branch but the
// warp's choice of merge: with one around each piece 8192 x 7168 bf16 took 54
// us, now 42 (5.5 TB/s; a plain copy of these bytes takes 39 to 42).
template <typename T, int PIECES, int ROWS, int S, int kThreads, bool kExact>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) row_kernel(
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
    if (kExact || c < d) {
      load_f32(w + c, wv[i]);
      if (b != nullptr) load_f32(b + c, bv[i]);
    }
  }
  const float inv_d = 1.f / (float)d;
  // all lanes of the warp hold PIECES whole pieces
  const bool whole = ((PIECES - 1) * kT + (warp + 1) * 32) * V <= d;
  float warp_n = 0.f;  // this warp's elements
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    warp_n += (float)V * __popc(__ballot_sync(0xffffffffu, in.in[i]));
  const float inv_warp = warp_n > 0.f ? 1.f / warp_n : 0.f;
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
      for (int i = 0; i < PIECES; ++i) {
        uint4 raw = in.read(k, 0, i);
        const bool has = kExact || in.in[i];
        if (!has) raw = make_uint4(0u, 0u, 0u, 0u);
        unpack(raw, v[k][i], T{});
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
          s[k] = Stat{has ? (float)V : 0.f, m, m2};
        } else {  // equal counts so far: i pieces and one more, or none
          const float dm = m - s[k].mean;
          s[k].mean = fmaf(dm, has ? 1.f / (i + 1) : 0.f, s[k].mean);
          s[k].m2 = fmaf(dm * dm, has ? V * (float)i / (i + 1) : 0.f, s[k].m2 + m2);
          s[k].n += has ? (float)V : 0.f;
        }
      }
    }
    in.next();
    if (kExact || whole) {  // equal counts: the merged mean is the middle of the two
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
      for (int k = 0; k < ROWS; ++k) {  // the warp's mean, then the squares around it
        float a = s[k].n * s[k].mean;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        a *= inv_warp;
        const float dm = s[k].mean - a;
        float q = fmaf(s[k].n * dm, dm, s[k].m2);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
        s[k] = Stat{warp_n, a, q};
      }
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
#pragma unroll
        for (int e = 0; e < P; ++e)
          v[k][i][e] = fma2(mul2(add2(v[k][i][e], mu2), rs2), wv[i][e], bv[i][e]);
        const uint4 o = pack(v[k][i], T{});
        if (kExact || in.in[i]) *reinterpret_cast<uint4*>(dst + (i * kT + t) * V) = o;
      }
    }
  }
}

// One partial row of dw and db per CTA, as below.  z and h are kept in registers
// until the row's sums are known, or (kReread) formed again from the ring, which
// leaves room for four pieces a thread and two CTAs an SM: 8192 x 7168 bf16 84
// us kept, 70 reread with the column sums (5.0 TB/s).
template <typename T, int PIECES, int ROWS, int S, int kThreads, bool kExact, bool kReread>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) row_bwd_kernel(
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
    constexpr int KR = kReread ? 1 : ROWS, KP = kReread ? 1 : PIECES;
    f32x2 z[KR][KP][P], h[KR][KP][P];
    float sums[2 * ROWS];  // h of each row, then h z of each row
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      f32x2 s1 = 0ull, s2 = 0ull;
      if (done + k < rows) {
        const f32x2 mu2 = pair2(-mu[k], -mu[k]), rs2 = pair2(rs[k], rs[k]);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          f32x2 g[P];
          f32x2 (&zi)[P] = z[kReread ? 0 : k][kReread ? 0 : i];
          f32x2 (&hi)[P] = h[kReread ? 0 : k][kReread ? 0 : i];
          const uint4 none = make_uint4(0u, 0u, 0u, 0u);
          const uint4 rx = in.read(k, 0, i), rg = in.read(k, 1, i);
          const bool has = kExact || in.in[i];
          unpack(has ? rx : none, zi, T{});
          unpack(has ? rg : none, g, T{});
#pragma unroll
          for (int e = 0; e < P; ++e) {
            zi[e] = mul2(add2(zi[e], mu2), rs2);
            hi[e] = mul2(g[e], wv[i][e]);
            s1 = add2(s1, hi[e]);
            s2 = fma2(hi[e], zi[e], s2);
            aw[i][e] = fma2(g[e], zi[e], aw[i][e]);
            ab[i][e] = add2(ab[i][e], g[e]);
          }
        }
      }
      sums[k] = both(s1);
      sums[ROWS + k] = both(s2);
    }
    if constexpr (!kReread) in.next();
    const float mine = warp_sums<2 * ROWS>(sums);
    if (lane % (16 / ROWS) == 0) red[flip][lane / (16 / ROWS)][warp] = mine;
    __syncthreads();
    // every thread has read these rows' slots (kReread: those of the rows before)
    if (t == 0 && (!kReread || done > 0)) in.fetch();
    block_sums<2 * ROWS>(red[flip], warps, sums);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (done + k >= rows) break;
      // dx = rs h - rs (mean(h) + z mean(h z))
      const float a = -rs[k] * (sums[k] * inv_d), c = -rs[k] * (sums[ROWS + k] * inv_d);
      const f32x2 rs2 = pair2(rs[k], rs[k]), a2 = pair2(a, a), c2 = pair2(c, c);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        f32x2 o[P];
        if constexpr (kReread) {
          f32x2 g[P];
          const f32x2 mu2 = pair2(-mu[k], -mu[k]);
          unpack(in.read(k, 0, i), o, T{});
          unpack(in.read(k, 1, i), g, T{});
#pragma unroll
          for (int e = 0; e < P; ++e) {
            o[e] = mul2(add2(o[e], mu2), rs2);
            o[e] = fma2(mul2(g[e], wv[i][e]), rs2, fma2(o[e], c2, a2));
          }
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) o[e] = fma2(h[k][i][e], rs2, fma2(z[k][i][e], c2, a2));
        }
        const uint4 u = pack(o, T{});
        if (kExact || in.in[i]) *reinterpret_cast<uint4*>(dst + i * kT * 16) = u;
      }
      dst += in.row_step * sizeof(T);
    }
    if constexpr (kReread) in.next();
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
// One partial row of dw and db per CTA: part [gridDim.x][2][d].  Absent pieces
// are zeros (times the first weight) and need no branch, and a thread has 16
// elements at most: 8192 x 7001 bf16 129 us (215 with branches and 32 elements,
// 256 threads a row), 4000 x 15001 382 us (1200).  The 1024-thread forms, above
// 8192 columns, spill some 650 bytes a thread: fp32 4000 x 16384 384 us (the
// forward, 512 threads, 98).
template <typename T, int VEC, int PIECES, int kT>
__global__ void __launch_bounds__(kT < 128 ? 128 : kT,
                                 kT < 128 ? 4 : kT < 512 ? 512 / kT : 1) layer_norm_bwd_kernel(
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
  RowRegs<T, VEC, PIECES, kT> cx{}, cd{}, nx{}, nd{};  // absent pieces stay zeros
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
    if (r + step < R) {
      nx.load(x + (size_t)(r + step) * d, t, d);
      nd.load(dy + (size_t)(r + step) * d, t, d);
    }
    float s1 = 0.f, s2 = 0.f;
    float wv[PIECES][VEC];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (i * kT + t) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; e += (VEC < 4 ? VEC : 4)) {
        constexpr int S = VEC < 4 ? VEC : 4;
        *reinterpret_cast<F32Piece<S>*>(wv[i] + e) =
            *reinterpret_cast<const F32Piece<S>*>(w + (c < d ? c : 0) + e);
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
      typename RowRegs<T, VEC, PIECES, kT>::Piece o;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float z = (to_f32(cx.p[i].v[e]) - mu) * rs;
        o.v[e] = from_f32<T>(rs * (to_f32(cd.p[i].v[e]) * wv[i][e] - s1 - z * s2));
      }
      if (c < d) *reinterpret_cast<typename RowRegs<T, VEC, PIECES, kT>::Piece*>(drow + c) = o;
    }
    cx = nx;
    cd = nd;
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

bool by_rows(int d, int elem) { return d % (16 / elem) == 0 && d * elem <= 32768; }
// Threads of a row kernel's CTA, and the CTAs an SM holds: 512 threads in all.
int row_threads(int d, int elem, int pieces) {
  return ((d / (16 / elem) + pieces - 1) / pieces + 31) / 32 * 32;
}
int rows_per_sm(int d, int elem, int pieces) {
  return 512 / row_threads(d, elem, pieces);
}
// Pieces a thread.  Forward: two and two rows at a time up to 4096 columns, above
// four and one row (29 M elements of bf16 in rows of 4096: 41.5 us against 44.5,
// of 5120: 51.2 against 44.8).  Backward: the same by size, up to 8 KB a row
// (8192 rows of 2048 bf16 38 us against 50; of 7168 79 against 70).
int fwd_pieces(int d) { return d <= 4096 ? 2 : 4; }
int bwd_pieces(int d, int elem) { return d * elem <= 8192 ? 2 : 4; }
// CTAs of the backward kernel = partial rows.
int bwd_ctas(int R, int d, int elem) {
  const bool rows = by_rows(d, elem);
  const int groups = !rows && d <= 512 ? 4 : 1;
  const long long want = ((long long)R + groups - 1) / groups;
  const long long most = num_sms() * (rows        ? rows_per_sm(d, elem, bwd_pieces(d, elem))
                                      : d <= 2048 ? 4
                                      : d <= 4096 ? 2
                                                  : 1);  // 512 threads or more
  return (int)(want < most ? (want < 1 ? 1 : want) : most);
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
  const int cap = num_sms() * (1024 / kBlock);
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

template <typename T, int PIECES, int ROWS, int S, int kThreads, bool kExact>
cudaError_t rows_launch(const Fwd& a, cudaStream_t st) {
  const int kT = row_threads(a.d, sizeof(T), PIECES);
  auto kernel = row_kernel<T, PIECES, ROWS, S, kThreads, kExact>;
  // the same opt-in for every width: host threads may call at the same time
  constexpr int most_smem = S * PIECES * kThreads * 16;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       most_smem);
  if (e != cudaSuccess) return e;
  const int most = num_sms() * rows_per_sm(a.d, sizeof(T), PIECES);
  kernel<<<a.R < most ? a.R : most, kT, S * PIECES * kT * 16, st>>>(
      static_cast<const T*>(a.x), a.w, a.b, a.eps, a.R, a.d, static_cast<T*>(a.y), a.mean, a.rstd);
  return cudaGetLastError();
}
template <typename T, int PIECES, int ROWS, int S, int kThreads, bool kExact>
cudaError_t rows_launch(const Bwd& a, cudaStream_t st) {
  const int kT = row_threads(a.d, sizeof(T), PIECES);
  auto kernel = row_bwd_kernel<T, PIECES, ROWS, S, kThreads, kExact, ROWS == 1>;
  constexpr int most_smem = S * PIECES * 2 * kThreads * 16;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       most_smem);
  if (e != cudaSuccess) return e;
  kernel<<<bwd_ctas(a.R, a.d, sizeof(T)), kT, S * PIECES * 2 * kT * 16, st>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.mean, a.rstd, a.R, a.d,
      static_cast<T*>(a.dx), a.part);
  return cudaGetLastError();
}
template <typename T, int PIECES, int ROWS, int S, int kThreads, typename Args>
cudaError_t rows_full(const Args& a, cudaStream_t st) {
  if (a.d == PIECES * row_threads(a.d, sizeof(T), PIECES) * (16 / (int)sizeof(T)))
    return rows_launch<T, PIECES, ROWS, S, kThreads, true>(a, st);
  return rows_launch<T, PIECES, ROWS, S, kThreads, false>(a, st);
}
template <typename T>
cudaError_t rows(const Fwd& a, cudaStream_t st) {
  if (fwd_pieces(a.d) == 2) return rows_full<T, 2, 2, 6, 128 * sizeof(T)>(a, st);
  if (a.d * (int)sizeof(T) <= 16384) return rows_full<T, 4, 1, 6, 256>(a, st);
  return rows_full<T, 4, 1, 6, 512>(a, st);
}
template <typename T>
cudaError_t rows(const Bwd& a, cudaStream_t st) {
  if (bwd_pieces(a.d, sizeof(T)) == 2) return rows_full<T, 2, 2, 6, 256>(a, st);
  if (a.d * (int)sizeof(T) <= 16384) return rows_full<T, 4, 1, 3, 256>(a, st);
  return rows_full<T, 4, 1, 3, 512>(a, st);
}

// Elements in registers: rows that are not whole 16-byte pieces, and fp32 rows
// wider than the row kernels take.
template <typename T>
void by_width(const Fwd& a, cudaStream_t st) {
  if (a.d <= 256) return go<T, 1, 8, 32>(a, st);
  if (a.d <= 512) return go<T, 1, 16, 32>(a, st);
  if (a.d <= 1024) return go<T, 1, 32, 32>(a, st);
  if (a.d <= 2048) return go<T, 1, 16, 128>(a, st);
  if (a.d <= 4096) return go<T, 1, 32, 128>(a, st);
  if (a.d <= 8192) return go<T, 1, 32, 256>(a, st);
  if constexpr (sizeof(T) == 4) {
    if (a.d % 4 == 0) return go<T, 4, 8, 512>(a, st);
  }
  go<T, 1, 32, 512>(a, st);
}
template <typename T>
void by_width(const Bwd& a, cudaStream_t st) {
  if (a.d <= 256) return go<T, 1, 8, 32>(a, st);
  if (a.d <= 512) return go<T, 1, 16, 32>(a, st);
  if (a.d <= 1024) return go<T, 1, 8, 128>(a, st);
  if (a.d <= 2048) return go<T, 1, 16, 128>(a, st);
  if (a.d <= 4096) return go<T, 1, 16, 256>(a, st);
  if (a.d <= 8192) return go<T, 1, 16, 512>(a, st);
  if constexpr (sizeof(T) == 4) {
    if (a.d % 4 == 0) return go<T, 4, 4, 1024>(a, st);
  }
  go<T, 1, 16, 1024>(a, st);
}
template <typename T, typename Args>
cudaError_t by_type(const Args& a, cudaStream_t st) {
  if (by_rows(a.d, sizeof(T))) return rows<T>(a, st);
  by_width<T>(a, st);
  return cudaGetLastError();
}
template <typename Args>
cudaError_t launch_norm(const Args& a, int dtype, cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16 ? by_type<__nv_bfloat16>(a, st) : by_type<float>(a, st);
}

}  // namespace

int layer_norm_max_d() { return kMaxD; }

size_t layer_norm_ws_bytes(int R, int d) {  // for either type
  const int a = bwd_ctas(R, d, 2), b = bwd_ctas(R, d, 4);
  return (size_t)(a > b ? a : b) * 2 * d * 4;
}

cudaError_t launch_layer_norm(int dtype, const void* x, const float* w, const float* b, float eps,
                              int R, int d, void* y, float* mean, float* rstd, cudaStream_t st) {
  return note_cuda(launch_norm(Fwd{x, w, b, eps, R, d, y, mean, rstd}, dtype, st),
                   "layer norm launch");
}

cudaError_t launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* w,
                                       const float* mean, const float* rstd, int R, int d,
                                       void* dx, float* dw, float* db, void* ws,
                                       cudaStream_t st) {
  float* part = static_cast<float*>(ws);
  cudaError_t e = note_cuda(launch_norm(Bwd{dy, x, w, mean, rstd, R, d, dx, part}, dtype, st),
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
