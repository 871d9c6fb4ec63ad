// Shared by the grouped bf16 matmul (grouped_matmul.cu) and the block-scaled
// FP8 matmul (matmul_fp8.cu): the ragged tile schedule, operand descriptors
// for tiles whose contraction index is the outer one, and a bounded wait.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace moe {

constexpr int kMatmulMaxGroups = 384;  // tile table entries that fit beside the operand ring
// Waits are timed in steps of 2^20 ns (about a millisecond), in 32 bits.
constexpr uint32_t kMatmulTimeoutMs = 2000, kDrainMs = 50;
// A wait for a whole contraction of `blocks` K blocks: 2 us a block beside that
// (they take 0.1 to 0.6), as an expert may own 2^31 rows and these are its blocks.
__device__ __forceinline__ uint32_t contraction_ms(int blocks) {
  return kMatmulTimeoutMs + (uint32_t)blocks / 500u;
}
__device__ __forceinline__ uint32_t clock_ms() { return (uint32_t)(globaltimer_ns() >> 20); }

// One try of a wait.  `cluster`: cluster-scope acquire, for barriers that the
// peer CTA arrives on.
__device__ __forceinline__ bool mm_try(uint64_t* bar, uint32_t parity, bool cluster) {
  uint32_t ok;
  if (cluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return ok != 0;
}
// mbar_wait_bounded for the matmul kernels: only a recorded time-out makes
// other waits give up, so a call that reports bad offsets still completes its
// good groups; and the clock is first read after 64 tries, as reading it on
// every wait that does not succeed at once delays the pipeline.
//
// The whole warp waits and gets one verdict: elect.sync, __syncwarp and aligned
// cluster barriers follow, which lanes that go different ways never leave.  Each
// lane sees the phase for itself (that orders its later reads); a lane that has
// seen it keeps seeing it, so the warp gives up only while no lane has, on the
// word of lane 0.
template <bool kCluster = false>
__device__ __forceinline__ bool mm_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                        uint32_t limit_ms = kMatmulTimeoutMs) {
  uint32_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    const bool ready = mm_try(bar, parity, kCluster);
    if (__all_sync(0xffffffffu, ready)) return true;
    if (it == 64) t0 = clock_ms();
    if ((it & 63u) == 0 && !__any_sync(0xffffffffu, ready)) {
      uint32_t seen = *reinterpret_cast<volatile uint32_t*>(err) & kErrWaitTimeout;
      if (clock_ms() - t0 > limit_ms) {
        atomicOr(err, kErrWaitTimeout);
        seen = 1;
      }
      if (__shfl_sync(0xffffffffu, seen, 0)) return false;
    }
  }
}
// The whole warp waits for its own copies or products in flight before the CTA
// ends, whatever the status word says: a CTA that gives up because another one
// has must not hand its shared memory on while copies still write to it.
__device__ __forceinline__ void mm_drain(uint64_t* bar, uint32_t parity, uint32_t* err) {
  uint32_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mm_try(bar, parity, false))) return;
    if ((it & 63u) == 0) {
      if (it == 64) t0 = clock_ms();
      const bool over = clock_ms() - t0 > kDrainMs;
      if (over) atomicOr(err, kErrWaitTimeout);
      if (__shfl_sync(0xffffffffu, over, 0)) return;
    }
  }
}
// After a recorded time-out: time for copies to land whose barrier may never
// complete (a pair's peer signals the leader's, which may not have armed it).
// A copy lands within microseconds.
__device__ __forceinline__ void mm_settle(const uint32_t* err) {
  if (*reinterpret_cast<const volatile uint32_t*>(err) & kErrWaitTimeout) {
    const uint32_t t0 = clock_ms();
    while (clock_ms() - t0 < 2) __nanosleep(1000);
  }
  __syncwarp();
}
// mm_wait for a single thread.
__device__ __forceinline__ bool mm_wait_thread(uint64_t* bar, uint32_t parity, uint32_t* err,
                                               uint32_t limit_ms = kMatmulTimeoutMs) {
  uint32_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mm_try(bar, parity, false)) return true;
    if ((it & 63u) == 0) {
      if (*reinterpret_cast<volatile uint32_t*>(err) & kErrWaitTimeout) return false;
      if (it == 64) t0 = clock_ms();
      if (clock_ms() - t0 > limit_ms) {
        atomicOr(err, kErrWaitTimeout);
        return false;
      }
    }
  }
}

// The aligned cluster barrier wants the warp's lanes together; code that lets them
// go different ways (stores of a tile's edge, one lane's arrive) comes before it.
__device__ __forceinline__ void mm_cluster_sync() {
  __syncwarp();
  cluster_sync_all();
}

// Arrive on a barrier of the pair's other CTA (shared::cluster address) without
// a cluster-scope release: for hand-overs that order no memory, only TMEM reads
// (which tcgen05.fence orders around the barrier).  With release and acquire at
// cluster scope each such hand-over costs over a thousand cycles.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Rows [first, first + count) of group g; offsets == nullptr is one group of
// all R rows.  A group whose offsets do not satisfy 0 <= o[g] <= o[g+1] <= R
// counts as empty (*bad is set).
__device__ __forceinline__ int group_rows(const int32_t* offsets, int g, int R, int* first,
                                          bool* bad) {
  if (offsets == nullptr) {
    *first = 0;
    return R;
  }
  const int lo = __ldg(offsets + g), hi = __ldg(offsets + g + 1);
  *first = lo;
  if (lo < 0 || hi < lo || hi > R) {
    *first = 0;
    *bad = true;
    return 0;
  }
  return hi - lo;
}

// start[g] = units before group g, start[E] = their total; called by one warp.  A
// group of `rows` rows has ceil(rows / tile_m) runs of `per` units.  `pairs` > 0:
// that many workers take the units in turn, and a unit may be cut in two (runs of
// tile_m / 2 rows).  Where the last round leaves more than half of the workers
// without a unit, the groups that reach into it are cut, if the halves then fit
// into half a round: with `rest` units in the last round, and the first of these
// groups starting s units before it, 2 rest + s halves.  Returns the first group
// that is cut (E: none).
__device__ __forceinline__ int ragged_schedule(const int32_t* offsets, int E, int R, int tile_m,
                                               int per, int* start, uint32_t* status,
                                               int pairs = 0) {
  const int lane = threadIdx.x & 31;
  const int chunk = (E + 31) / 32;
  const int g0 = min(E, lane * chunk), g1 = min(E, g0 + chunk);
  bool bad = false;
  int first, single = E;
  for (int pass = 0; pass < 2; ++pass) {
    int sum = 0;
    for (int g = g0; g < g1; ++g) {
      const int tm = g < single ? tile_m : tile_m / 2;
      const int mt = (group_rows(offsets, g, R, &first, &bad) + tm - 1) / tm;
      start[g] = mt;
      sum += mt;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    int run = inc - sum;
    const int total = __shfl_sync(0xffffffffu, inc, 31) * per;
    const int rest = pairs > 0 ? total % pairs : 0;
    const int round = total - rest;  // units before the last round
    int from = E;
    for (int g = g0; g < g1; ++g) {
      const int before = run * per;
      run += start[g];
      start[g] = before;
      if (rest > 0 && before <= round && run * per > round && 2 * rest + round - before <= pairs)
        from = g;
    }
    if (lane == 31) start[E] = total;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) from = min(from, __shfl_xor_sync(0xffffffffu, from, o));
    if (pass == 1 || from == E) break;
    single = from;
  }
  if (bad) atomicOr(status, kErrBadIndex);
  return single;
}

// The group of unit u: start[g] <= u < start[g + 1].
__device__ __forceinline__ int ragged_group(const int* start, int E, int u) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// Shared-memory matrix descriptor of an operand stored with its contraction
// index outermost: chunks of 128 bytes of the M (or N) index by 8 contraction
// rows are 1024-byte swizzle atoms; the next 8 contraction rows follow at
// 1024 bytes, the next 128 bytes of the M (or N) index at `chunk_bytes`.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t chunk_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(chunk_bytes >> 4) << 16;  // leading byte offset: next chunk along M / N
  d |= (uint64_t)(1024u >> 4) << 32;        // stride byte offset: next 8 contraction rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Instruction-descriptor bits: operand stored contraction-outermost.
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;


// The two 32-bit halves of a descriptor: only the low one changes as a kernel
// walks its ring and the contraction steps (addresses count 16-byte units).
__device__ __forceinline__ uint32_t desc_lo(uint64_t d) { return (uint32_t)d; }
__device__ __forceinline__ uint32_t desc_hi(uint64_t d) { return (uint32_t)(d >> 32); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void mma_bf16_2sm_parts(uint32_t tmem_d, uint32_t a_lo, uint32_t a_hi,
                                                   uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_f8_parts(uint32_t tmem_d, uint32_t a_lo, uint32_t a_hi,
                                                 uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_parts(uint32_t tmem_d, uint32_t a_lo, uint32_t a_hi,
                                                 uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The same, completing on the pair leader's barrier (see tma_load_2d_2sm).
__device__ __forceinline__ void tma_load_3d_2sm(void* smem_dst, const CUtensorMap* map, int32_t x,
                                                int32_t y, int32_t z, uint32_t bar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster_addr)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src,
                                             int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace moe
