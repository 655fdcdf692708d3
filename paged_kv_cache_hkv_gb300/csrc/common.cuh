// Device helpers shared by the paged KV cache kernels (sm_103a).
#pragma once

#include <cuda.h>  // CUtensorMap (type only; the driver is reached at run time)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

constexpr uint32_t kErrSlotRange = 0x1u;
constexpr uint32_t kErrBlockRange = 0x2u;
constexpr uint32_t kErrLengths = 0x4u;
constexpr uint32_t kErrTimeout = 0x8u;
constexpr uint32_t kErrShared = 0x10u;
constexpr uint32_t kErrNoBlocks = 0x20u;
constexpr uint32_t kErrRefCount = 0x40u;

// The attention kernels move keys in chunks of 16 (one decode stage, one
// MMA K step). A cache block holds 8, 16 or 32 tokens, so a chunk is two
// 8-token blocks, one 16-token block or half of a 32-token block.
constexpr int kChunkKeys = 16;
// An on-chip wait that has not completed after this long is treated as lost.
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint64_t kDrainLimitNs = 100000000ull;  // 0.1 s, when cleaning up

// Programmatic dependent launch. Every kernel of the step lets the next one
// launch as soon as it starts (its CTAs then run their prologue while this
// grid finishes), and waits for the previous grid -- its completion and the
// visibility of its memory -- before touching anything that grid wrote. Both
// are no-ops for a kernel launched without the attribute.
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// Make barrier initialisation visible to the async proxy (TMA, tensor core).
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase with the given parity to complete. Gives up after
// `limit_ns` and returns false (the caller records kErrTimeout).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity,
                                          uint64_t limit_ns = kWaitLimitNs) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (global_ns() - t0 > limit_ns) return false;
  }
}

// Order this thread's generic-proxy shared memory accesses before later
// async-proxy (TMA / tensor core) accesses of the same bytes.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Five-dimensional tiled copy (coordinates innermost first).
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
      "r"(smem_u32(bar))
      : "memory");
}

// tma_load_3d with an L2 cache policy (from createpolicy) attached to the read.
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, int c0, int c1,
                                                 int c2, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

// L2 policy for data read once: evict it first.
__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Untiled bulk copy global -> shared; both addresses 16-byte aligned, bytes a
// multiple of 16.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---------------------------------------------------------------- bf16
// Two bf16 packed in a 32-bit word -> two fp32 (a bf16 is the top half of an
// fp32, so this is exact).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// Packed fp32 pair FMA (one instruction for two lanes of work on sm_100+).
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Packed fp32 pair add (sm_100+), flush-to-zero like the rest of the build.
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.ftz.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Packed fp32 pair product (sm_100+).
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.ftz.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Three-input maximum (one instruction on sm_100+); NaN-free inputs.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Largest index i in [0, n) with a[i] <= x, for a non-decreasing a[0..n]
// whose a[0] <= x.
__device__ __forceinline__ int upper_index(const int32_t* a, int n, long long x) {
  int lo = 0, hi = n;  // invariant: a[lo] <= x, answer in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(__ldg(a + mid)) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The same answer as upper_index, found by a whole warp (every lane gets it):
// each round the 32 lanes test 32 evenly spaced candidates, so the search
// takes ceil(log32 n) dependent loads instead of log2 n. The candidates are
// non-decreasing in the lane and a is non-decreasing, so the lanes whose
// candidate is <= x form a prefix; the next interval lies between the last
// of them and the first lane past it.
__device__ __forceinline__ int warp_upper_index(const int32_t* a, int n, long long x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // invariant: a[lo] <= x, answer in [lo, hi)
  while (hi - lo > 1) {
    const int idx = lo + static_cast<int>((static_cast<long long>(lane) * (hi - lo)) >> 5);
    const unsigned le = __ballot_sync(0xffffffffu, static_cast<long long>(__ldg(a + idx)) <= x);
    const int k = 31 - __clz(le);  // lane 0 (candidate lo) is always in
    const int idx_k = __shfl_sync(0xffffffffu, idx, k);
    const int idx_next = __shfl_sync(0xffffffffu, idx, k < 31 ? k + 1 : 31);
    hi = k < 31 ? idx_next : hi;
    lo = idx_k;
  }
  return lo;
}

// ---------------------------------------------------------------- scores
constexpr float kLog2e = 1.4426950408889634f;

// tanh of u for z = 2 log2(e) u. With e = 2^z = exp(2u): tanh u = 1 - 2 / (e + 1),
// whose absolute error of a few 2^-24 is a relative error of the same size
// only away from 0; below |u| = 1/4 the odd series u - u^3/3 + 2u^5/15 -
// 17u^7/315 + 62u^9/2835 (next term below 1e-8 of the value) keeps it relative. A score
// softcap * tanh(u) so carries an error of a few 2^-24 of its own size, whatever the cap.
__device__ __forceinline__ float tanh_log2(float z) {
  const float u = z * 0.34657359027997264f, w = u * u;  // ln(2) / 2
  const float e = exp2f(z);
  const float big = 1.f - __fdividef(2.f, e + 1.f);
  const float small =
      u * (1.f + w * (-1.f / 3 + w * (2.f / 15 + w * (-17.f / 315 + w * (62.f / 2835)))));
  return fabsf(u) < 0.25f ? small : big;
}

// Capped, biased or range-masked scores (pkv_score_options), as the attention
// kernels take them.
struct ScoreParams {
  float softcap;             // 0 = off
  const float* slopes;       // distance bias per q head, or null
  const int32_t* key_begin;  // first key of each query row, or null (0)
  const int32_t* key_end;    // past the last key of each query row, or null (p + 1)
};

// Bias per key of distance of q head h for base-2 scores, 0 without slopes.
// Slopes beyond +-kMaxSlope count as that: times log2(e) and a distance below
// 2^31 the bias stays finite (3e37), where an infinite one times the nearest
// key's distance 0, or minus a row's infinite maximum, would be a NaN.
constexpr float kMaxSlope = 1e28f;
__device__ __forceinline__ float slope_log2(const ScoreParams& s, int h) {
  return s.slopes ? fminf(fmaxf(__ldg(s.slopes + h), -kMaxSlope), kMaxSlope) * kLog2e : 0.f;
}

// Keys [lo, hi) that a row sees; lo == hi == 0 for a row that sees none.
struct KeyRange {
  int lo, hi;
};

// Range of batch row t at position pos of a sequence of L keys, its part from
// key `base` on (the rest is attended elsewhere; 0 = all of it).
__device__ __forceinline__ KeyRange row_keys(const ScoreParams& s, long long t, int pos, int L,
                                             int base) {
  int lo = s.key_begin ? __ldg(s.key_begin + t) : 0;
  int hi = s.key_end ? __ldg(s.key_end + t) : pos + 1;
  lo = max(lo, base);
  hi = min(hi, L);
  return lo < hi ? KeyRange{lo, hi} : KeyRange{0, 0};
}

// 16-key chunks that a decode row streams for its range. A row without keys
// streams one masked chunk, so that its (zero) output is written like any
// other's.
__device__ __forceinline__ int range_chunks(const KeyRange& k) {
  return k.lo < k.hi ? ((k.hi + kChunkKeys - 1) / kChunkKeys) - k.lo / kChunkKeys : 1;
}

}  // namespace pkv
