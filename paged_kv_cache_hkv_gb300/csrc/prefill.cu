// Causal chunked-prefill attention over the paged cache on the 5th-generation
// tensor cores (tcgen05, TMEM accumulators, TMA operands), sm_103a.
//
// What it computes ("vllm v1 源码精读（三）" §4.2; "Inside vLLM" §3.4-3.5):
// request r has c = num_computed tokens already cached and n > 1 new tokens
// (a prompt chunk). Its i-th new token, at absolute position c + i, attends
// keys 0 .. c + i of its own sequence -- the cached prefix and the chunk up to
// itself -- all read through the block table (the chunk's own K/V was written
// into the pool first).
//
// Work item = (request, tile of 128 query rows, kv head). The 128 rows of a
// tile are the G = Hq/Hkv q heads of one kv head for 128/G consecutive
// queries, so every K/V tile feeds all G heads (GQA). Per key tile (128 keys
// = 8 chunks of 16 keys: 8 blocks of 16 tokens, 4 of 32 or 16 of 8):
//   S = Q K^T      tcgen05.mma M=128 N=128, A = Q (smem), B = K (smem)
//   O += P V       tcgen05.mma M=128 N=D, A = P (TMEM), B = V (smem)
// with S in one of three TMEM buffers (tile T of the CTA's stream uses
// buffer T % 3) and one O accumulator. Eight softmax warps share every
// tile: each holds 16 query rows, and each row is split between two threads
// (keys 0..63 and 64..127). A thread reads its half row of S with
// tcgen05.ld, applies the causal mask, keeps a base-2 running max (rescaling
// its half of O in TMEM only when the max grows by more than 2^8) and sum,
// and writes P as bf16 pairs over the S buffer's columns with tcgen05.st.
// A K-copy warp (3-slot ring; the scored instances 2) and a V-copy warp (2-slot
// ring; 3) stream the
// tiles by TMA (128-byte swizzle, one copy per cache block and kv head: the
// fewer and larger the copies, the faster one SM's copy engine goes); one
// thread issues every S and another every PV. The
// CTAs are persistent and take items from a counter; the roles meet only at
// mbarriers, so consecutive items overlap.
//
// Every wait is bounded; on a timeout the kernel records
// PKV_DEVERR_TIMEOUT, drains its copies, frees TMEM and returns.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pkv {

static __device__ uint32_t g_errors_prefill;

namespace tc {

// Shared-memory matrix descriptor (tcgen05), 128-byte swizzle.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) |  // version
         (2ull << 61);                                                         // SWIZZLE_128B
}

// Instruction descriptor, kind::f16: bf16 A and B, fp32 accumulator,
// A K-major, B K-major (b_mn = 0) or MN-major (b_mn = 1).
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Same, with the A operand (M rows x 16 K elements) in tensor memory: lane i
// holds row i, 32-bit column c holds K elements 2c (low half) and 2c + 1.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// tcgen05.wait::ld with the 32 loaded registers as operands, so that no use
// of them can be scheduled before the wait.
__device__ __forceinline__ void wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// The 16-lane x 2 access shape: 16 TMEM lanes from the address's lane,
// threads 0-15 at columns col .. col+31 of lanes 0-15, threads 16-31 at
// columns col+OFF .. col+OFF+31 of the same lanes (asynchronous: the
// registers hold the data only after wait32 on them).
template <int OFF>
__device__ __forceinline__ void ld_half32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(OFF));
}

// Two such loads and the wait for both in one statement: the registers hold
// the data when it ends, so nothing (a spill, a move) can come before.
template <int OFF>
__device__ __forceinline__ void ld_half64(uint32_t t0, uint32_t t1, uint32_t (&a)[32],
                                          uint32_t (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64], %66;\n\t"
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65], %66;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),
        "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]),
        "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]),
        "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
        "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]),
        "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]),
        "=r"(b[14]), "=r"(b[15]), "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]),
        "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]), "=r"(b[24]), "=r"(b[25]),
        "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
      : "r"(t0), "r"(t1), "n"(OFF)
      : "memory");
}

// One such load and its wait.
template <int OFF>
__device__ __forceinline__ void ld_half32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(OFF)
      : "memory");
}

// The same access shape with 8 columns per thread, loaded and waited for.
template <int OFF>
__device__ __forceinline__ void ld_half8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr), "n"(OFF)
      : "memory");
}

template <int OFF>
__device__ __forceinline__ void st_half8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9};" ::"r"(taddr),
      "n"(OFF), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7])
      : "memory");
}

template <int OFF>
__device__ __forceinline__ void st_half16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17};" ::"r"(taddr),
      "n"(OFF), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
      "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int OFF>
__device__ __forceinline__ void st_half32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x32.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33};" ::"r"(
          taddr),
      "n"(OFF), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
      "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
      "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
      "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

}  // namespace tc


constexpr int kTileM = 128;    // query rows (query x head) per tile
constexpr int kTileN = 128;    // keys per tile (8 chunks of 16)
constexpr int kKStages = 3;    // K ring: global tile T uses slot T % 3
constexpr int kVStages = 2;    // V ring: global tile T uses slot T % 2
// The scored kernels split the same memory the other way. S(T) is issued as
// soon as PV(T-3) is done, well before K could run short; V(T) with two slots
// is copied only after PV(T-2), which in items of a few tiles left the softmax
// (it looks at the V rows of partly seen tiles) and the PV waiting for the
// copy's ~1 us.
constexpr int kScoredKStages = 2, kScoredVStages = 3;
static_assert(kScoredKStages + kScoredVStages == kKStages + kVStages, "one ring area");
constexpr int kSBufs = 3;      // S (then P) buffers in TMEM: global tile T uses buffer T % 3
static_assert(kKStages == kSBufs, "K slot T % 3 is freed by the commit of S buffer T % 3");
constexpr uint32_t kTmemS = 128;  // TMEM columns: O at [0, D), S buffer b at [128 + 128b, +128)
constexpr uint32_t kTmemCols = 512;
constexpr int kItemQ = 4;      // claimed work items in flight between the roles
// SCORED: tiles whose chunk masks are kept. The K-copy warp writes the mask of
// T+8 once S(T+6) is done (its ring has two slots), so PV(T+3), so every thread
// has published P(T+3): each has read the mask of T by then.
constexpr int kMaskRing = 8;
constexpr int kMetaReqs = 128;  // prefill requests whose metadata a CTA keeps in shared memory
constexpr float kRescaleLog2 = 8.f;  // lazy rescale threshold (powers of two)
// Scores of a kernel instance: plain, or key ranges with or without a cap
// (ScoreParams::softcap) and a bias (ScoreParams::slopes).
enum : int { kPlain = 0, kRanges = 1, kCap = 2, kBias = 4 };
// Softmax warps of an instance; after them the S-MMA warp, the K-copy warp, the
// V-copy warp and the PV-MMA warp. A capped instance without a bias keeps no
// running maximum, so the threads of a row need nothing of one another in a
// tile: four of them take 32 keys each, and sixteen warps hide one another's
// latencies where eight left the FMA pipe idle half the time. 4 x 2048 rows over
// 8192 keys, D = 128, us with sixteen and with eight warps: softcap 50 (every
// tile by the polynomial) 914 and 990, 15 (one tile in eight exact) 991 and 1163,
// 5 (all exact) 1528 and 1798. At D = 64 half of the sixteen hold no column of O
// and 488 bytes a thread are spilled: 989 and 967, 1072 and 1186, 1531 and 1781,
// and 8191 rows of short documents 122 and 109. Sixteen there too: a cap is for
// scores that reach it. The other instances exchange a row's maximum by a
// shuffle between two threads of one warp.
template <int SC>
__host__ __device__ constexpr int softmax_warps() {
  return SC == (kRanges | kCap) ? 16 : 8;
}
template <int SC>
__host__ __device__ constexpr int prefill_threads() {
  return (softmax_warps<SC>() + 4) * 32;
}
// TMEM column, from the S buffer's, of P for the kk-th 16 keys (eight columns
// each). P overwrites only columns whose scores the writing warp holds: with
// sixteen warps, keys 0..63 and 64..127 are in different ones.
template <int SC>
__host__ __device__ constexpr uint32_t p_column(int kk) {
  return softmax_warps<SC>() == 16 ? (kk >> 2) * 64u + (kk & 3) * 8u : kk * 8u;
}
// Order of an item's key tiles, the kt-th of nkv. With a bias that falls with
// distance the nearest keys weigh most: taken last to first, the running
// maximum is found in the first tile, where the other way round a steep slope
// moves it (and rescales O, after a wait for the last PV) in every tile.
template <int SC>
__device__ __forceinline__ int tile_at(int kt0, int nkv, int kt) {
  return kt0 + ((SC & kBias) ? nkv - 1 - kt : kt);
}

template <int D>
struct PrefillLayout {
  static constexpr int DH = D / 64;                 // 64-element (128-byte) column chunks
  static constexpr uint32_t kChunk = kTileM * 128;  // 128 rows x 128 bytes = 16 KB
  static constexpr uint32_t kQ = 0;
  // K (or V) of one 128-key tile: 16 groups of 8 keys, each DH 128-byte
  // swizzled 8-row atoms (one per 64-element half of d), group-major
  static constexpr uint32_t kGroupBytes = DH * 1024;
  static constexpr uint32_t kTileKV = 16 * kGroupBytes;
  static constexpr uint32_t kK = kQ + DH * kChunk;         // K ring
  static constexpr uint32_t kV = kK + kKStages * kTileKV;  // V ring
  // request metadata: int4 (request, cached, first row, new tokens) [kMetaReqs],
  // then the item prefix int [kMetaReqs + 1]
  static constexpr uint32_t kMeta = kV + kVStages * kTileKV;
  static constexpr uint32_t kBar = kMeta + kMetaReqs * 16 + (kMetaReqs + 1) * 4 + 124;
  static constexpr uint32_t kBad = kBar + 640;  // SCORED: BadKeys of kBadLists items
  static constexpr uint32_t kSums = kBad + 1024;  // 16 softmax warps: row sums [4][2][128]
  static constexpr uint32_t kBytes = kSums + 4096;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // room to align the base
  static_assert(kAlloc <= 232448, "shared memory");
};

// SCORED: keys of an item whose V rows hold an infinity or a NaN and that some
// of its rows may not see. Weight 0 times such a value is a NaN, so their
// elements go into the tensor core as zeros and the rows that do see the key
// get them back in the epilogue.
constexpr int kMaxBadKeys = 48;
constexpr int kBadLists = 5;
struct BadKeys {
  int count;  // above kMaxBadKeys: the list is not complete, every key is looked at
  int k_lo, kv_len;  // of the item, with the first key
  int key[kMaxBadKeys];  // (a key once for each thread that found a part of its row bad)
};
static_assert(kBadLists * sizeof(BadKeys) <= 1024, "bad key area");

struct PrefillParams {
  uint16_t* out;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* qsl;
  const int32_t* num_computed;
  int num_q_heads, num_kv_heads, group, num_blocks;
  int block_shift;  // log2 of the tokens per cache block (3, 4 or 5)
  float scale_log2;
  uint32_t* hdr;
  const int32_t* pf_req;
  const int32_t* pf_prefix;
  // shared-prefix items (see AttnArgs): their partial results go to
  // shared_ml / shared_o instead of the output
  int shared_len, shared_first, shared_num, shared_pieces, shared_tpp;
  float2* shared_ml;
  float* shared_o;
};

// The scored kernels' parameters: capped, biased or range-masked scores.
struct ScoredParams : PrefillParams {
  const uint16_t* pool;
  int num_tokens;
  ScoreParams score;
  float cap_z;      // softcap: 2 log2(e) scale / softcap, S to the argument of tanh_log2
  // softcap by polynomial (see kCapPoly): S^2 up to cap_lim2, -1 = never
  float cap_lim2;
  float cap_a[5];
  bool out32;       // the output is 32-byte aligned
};

// The cap on the tensor core's S without a division or a second exponential:
// for |u| <= 0.8, u = s * scale / softcap,
//   tanh(u) = u (c0 + c1 w + c2 w^2 + c3 w^3 + c4 w^4), w = u^2,
// with the c_i that minimise the largest relative error over that interval
// (1.0e-6: equal-ripple, found by reweighted least squares). The powers of
// scale / softcap and the factor softcap * log2(e) go into the coefficients,
// so a pair of scores takes six packed FMA-pipe instructions. A warp that holds
// a larger |u| takes the exact form for its tile: at softcap 50 and N(0, 3^2)
// scores none does, at 15 one tile in eight, at 5 all do (914, 991 and 1528 us,
// see softmax_warps; key ranges alone take 715: the polynomial's FMA-pipe work is
// most of the difference).
constexpr float kCapLim = 0.8f;
constexpr double kCapPoly[5] = {9.999989943e-01, -3.332537196e-01, 1.323056551e-01,
                                -4.918014086e-02, 1.210013789e-02};
// For scale / softcap in this range (0.125 / 15 to 0.09 / 800 in practice) S^2
// is a normal fp32 number wherever u matters. The coefficients also carry
// softcap * log2(e), and leave fp32 at large caps all the same (softcap 1e5
// under a scale of 1e9): cap_coefficients then says no, and every tile takes
// the exact form.
constexpr float kCapRatioMin = 1e-4f, kCapRatioMax = 1e4f;
// A capped score is at most softcap in size, so 2^score needs no maximum
// taken off it while softcap * log2(e) stays far below fp32's and bf16's
// exponent range. 74 covers softcap = 50 (72.1), and even where every score
// of a row lies at the cap, 2^+-74 leaves 2^53 above for the sum over 2^20
// keys of values up to 2^32, and 2^52 below for values down to 2^-30 with 22
// bits to spare. A wider cap takes the biased instance (without slopes),
// which keeps the maximum.
constexpr float kCapFixedMax = 74.f;


// One work item: (request, 128-row query tile, kv head).
struct PrefillItem {
  int g;       // kv head
  int c;       // cached tokens of the request
  int q0;      // batch row of the request's first query
  int n;       // new tokens of the request
  int i0;      // first query of the tile (within the request)
  int kv_len;  // keys the tile's last query sees (shared items: end of the piece)
  int nkv;     // key tiles
  int kt0;     // first key tile (0, or a shared item's piece start)
  int piece;   // shared items: key piece, else -1
  long long bt_row;  // offset of the request's block table row
  // SCORED items: first key that any row sees; a tile within [full_lo,
  // full_hi) is seen by every row
  int k_lo, full_lo, full_hi;
};

// mbarriers. "commit" ones are arrived on by a tcgen05.commit of an MMA thread
// (S: s_full, q_free, drain[0]; PV: pv_done, o_full, drain[1]). NW softmax warps:
// eight, or sixteen in a capped instance. Rings of KST K and VST V slots: 3 and 2,
// in the scored instances 2 and 3.
struct PrefillShared {
  uint64_t q_full;               // Q tile of the item landed (TMA)
  uint64_t q_free;               // commit: the item's last S read Q
  uint64_t k_full[3];            // K tile landed (TMA); KST used, one per slot of the ring
  uint64_t v_full[3];            // V tile landed (TMA); VST used
  uint64_t s_full[kSBufs];       // commit: S of tile T in TMEM, buffer T % 3, and K slot
                                 // T % KST read; SCORED: and an arrival of the S thread,
                                 // behind which the tile's mask is
  uint64_t pv_done[kSBufs];      // commit: PV of tile T done (P in buffer T % 3 and V slot
                                 // T % VST read, O updated)
  uint64_t p_ready[kSBufs];      // 32 NW arrivals: P of the buffer's tile in TMEM, O
                                 // rescaled, V cleaned (and, for an item's first tile,
                                 // the previous item's O read)
  uint64_t o_full;               // commit: the item's last PV done
  uint64_t drain[2];             // commit: every MMA of the S / PV thread done (teardown)
  uint64_t iq_full[kItemQ];      // item id j published in item_q[j % kItemQ]
  uint64_t iq_free[kItemQ];      // NW + 3 arrivals: every role has read it
  int item_q[kItemQ];
  PrefillItem item_m[kItemQ];    // SCORED: the item described, for every role
  uint32_t masks[kMaskRing];     // SCORED: chunk mask of tile T in masks[T % kMaskRing]
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PrefillShared) <= 640, "barrier area");



// Bounded wait that also gives up once another thread has flagged an abort.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(a, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        atomicOr(&g_errors_prefill, kErrTimeout);
        return false;
      }
    }
  }
}

// The same with its loop out of line, where the code around it has to stay small.
__device__ __noinline__ bool wait_loop(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return wait_or_abort(bar, parity, abort);
}
__device__ __forceinline__ bool wait_small(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(smem_u32(bar), parity) || wait_loop(bar, parity, abort);
}

// Consumers of the item queue (the MMA thread, the V-copy warp, each softmax
// warp): item id number j of this CTA, or -1 after an abort. The calling
// warp's lane 0 releases the slot once every lane has read it.
__device__ __forceinline__ int take_item(PrefillShared& sh, int j, volatile int* abort,
                                         bool whole_warp, PrefillItem* m) {
  const int slot = j % kItemQ;
  if (!wait_or_abort(&sh.iq_full[slot], (j / kItemQ) & 1u, abort)) return -1;
  const int item = *reinterpret_cast<volatile int*>(&sh.item_q[slot]);
  if (m) *m = sh.item_m[slot];
  if (whole_warp) __syncwarp();
  if (!whole_warp || (threadIdx.x & 31) == 0) mbar_arrive(&sh.iq_free[slot]);
  return item;
}

// The same without the release: the caller takes the item later.
__device__ __forceinline__ int peek_item(PrefillShared& sh, int j, volatile int* abort,
                                         PrefillItem* m) {
  const int slot = j % kItemQ;
  if (!wait_or_abort(&sh.iq_full[slot], (j / kItemQ) & 1u, abort)) return -1;
  *m = sh.item_m[slot];
  return *reinterpret_cast<volatile int*>(&sh.item_q[slot]);
}

// Keys of row i of a SCORED item (i < m.n), clipped to what the item attends;
// `ref` is the position its distances count from (see the decode kernel).
// Loaded and evaluated apart, so that the loads can go out early.
struct RowRaw {
  int begin, end, L;
};
struct RowKeys {
  int lo, hi, ref;
};
__device__ __forceinline__ RowRaw load_row(const ScoredParams& p, const PrefillItem& m, int i) {
  RowRaw r{0, 0, 0};
  if (i >= m.n) return r;
  const long long t = static_cast<long long>(m.q0) + i;
  if (t < 0 || t >= p.num_tokens) return r;  // (no row of the batch: it sees no key)
  // (shared-prefix items: row i is the decode of request shared_first + i)
  r.L = m.piece >= 0 ? __ldg(p.seq_lens + p.shared_first + i) : m.c + m.n;
  if (p.score.key_begin) r.begin = __ldg(p.score.key_begin + t);
  if (p.score.key_end) r.end = __ldg(p.score.key_end + t);
  return r;
}
__device__ __forceinline__ RowKeys row_of(const ScoredParams& p, const PrefillItem& m, int i,
                                          const RowRaw& r) {
  if (i >= m.n) return RowKeys{0, 0, 0};
  const int pos = m.piece >= 0 ? r.L - 1 : m.c + i;
  RowKeys k;
  k.lo = max(r.begin, 0);
  k.hi = min(p.score.key_end ? r.end : pos + 1, r.L);
  k.ref = max(min(pos, k.hi - 1), k.lo);
  if (m.piece >= 0) k.hi = min(k.hi, p.shared_len);
  if (k.lo >= k.hi) k.lo = k.hi = 0;
  return k;
}

// The item's keys over all its rows, by a whole warp: {first key that any row
// sees, past the last one, the largest first key, the smallest end}.
__device__ __forceinline__ int4 item_keys(const ScoredParams& p, const PrefillItem& m, int QT) {
  int lo_min = 0x7fffffff, hi_max = 0, lo_max = 0, hi_min = 0x7fffffff;
  const int i1 = min(m.i0 + QT, m.n);
  for (int i = m.i0 + (threadIdx.x & 31); i < i1; i += 32) {
    const RowKeys k = row_of(p, m, i, load_row(p, m, i));
    const bool none = k.lo >= k.hi;
    lo_min = none ? lo_min : min(lo_min, k.lo);
    hi_max = max(hi_max, k.hi);
    lo_max = none ? 0x7fffffff : max(lo_max, k.lo);
    hi_min = min(hi_min, k.hi);
  }
  lo_min = __reduce_min_sync(0xffffffffu, lo_min);
  hi_max = __reduce_max_sync(0xffffffffu, hi_max);
  lo_max = __reduce_max_sync(0xffffffffu, lo_max);
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);
  return make_int4(hi_max > 0 ? lo_min : 0, hi_max, lo_max, hi_min);
}

// Bits lo .. hi-1 of a word (any lo, hi).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << max(hi, 0)) - 1u;
  const uint32_t below_lo = lo >= 32 ? 0xffffffffu : (1u << max(lo, 0)) - 1u;
  return below_hi & ~below_lo;
}

// 32-byte store; the address 32-byte aligned.
__device__ __forceinline__ void st_global_v8(void* dst, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Zero the infinities and NaNs of 8 N bf16 in shared memory; true if there were any.
template <int N>
__device__ __forceinline__ bool zero_nonfinite(uint4* v4) {
  // x * 0 is 0 or, for an infinity or a NaN, a NaN
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 acc = zero;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    uint4 v = v4[x];
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __hfma2(h[e], zero, acc);
  }
  if ((*reinterpret_cast<uint32_t*>(&acc) & 0x7fff7fffu) == 0u) return false;
#pragma unroll 1
  for (int x = 0; x < N; ++x) {
    uint4 v = v4[x];
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
      if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu;
    }
    v4[x] = v;
  }
  return true;
}

// Which of up to 64 elements of some V rows are a NaN, +infinity and -infinity,
// a bit each: their sum with a finite value, whatever the order.
struct Odd {
  unsigned long long nan, pos, neg;
};

__device__ __forceinline__ bool has_nonfinite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    any |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
  return any;
}

// The V row of key j for kv head g, or null if a used entry of its 16-key chunk
// is out of the pool (the chunk is masked).
__device__ __forceinline__ const uint4* v_row_of(const ScoredParams& p, const BadKeys& bad,
                                                 long long bt_row, int g, int D, int j) {
  const int bsh = p.block_shift, own = j >> bsh;
  const int e0 = bsh == 3 ? own & ~1 : own, e1 = bsh == 3 ? own | 1 : own;
  int id = -1;
  for (int e = e0; e <= e1; ++e) {
    if ((e << bsh) >= bad.kv_len || ((e + 1) << bsh) <= bad.k_lo) continue;  // not used
    const int x = __ldg(p.block_table + bt_row + e);
    if (x < 0 || x >= p.num_blocks) return nullptr;
    if (e == own) id = x;
  }
  if (id < 0) return nullptr;
  const long long r = ((static_cast<long long>(id) * 2 + 1) << bsh) + (j & ((1 << bsh) - 1));
  return reinterpret_cast<const uint4*>(p.pool + (r * p.num_kv_heads + g) * D);
}

// Of nd elements (at most 64).
__device__ __forceinline__ Odd odd_of(const uint4* v, int nd) {
  Odd odd{0, 0, 0};
#pragma unroll 4
  for (int x = 0; x < nd / 8; ++x) {
    const uint4 u = __ldg(v + x);
    if (!has_nonfinite(u)) continue;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
      if ((b & 0x7f80u) != 0x7f80u) continue;
      const unsigned long long bit = 1ull << (8 * x + e);
      if (b & 0x7fu)
        odd.nan |= bit;
      else if (b & 0x8000u)
        odd.neg |= bit;
      else
        odd.pos |= bit;
    }
  }
  return odd;
}

// Add the infinities and NaNs of the bad keys that a row sees to the thread's
// part of the row, already stored (bf16, or fp32 partials): V elements d0 ..
// d0+nd-1 of keys lo .. hi-1. By a whole warp, whose lanes 0-15 and 16-31 hold nd
// elements next to each other; `mine`: the thread has a part.
// A lane looks at one key of the list, or, where the list is not complete, at one
// of all the keys that the warp's rows see, and hands what it finds to all: the
// other roles wait meanwhile, and waits are limited. Last keys first: rows full of
// NaN are mostly a step's own, and end the search. (512 rows whose V is all NaN
// over 32768 clean keys take 0.44 ms, clean ones 0.41; by every thread key after
// key it was 93 ms, and over a million keys it would outlast the waits.) Keys of tiles that were not cleaned are found too: adding the same infinity or a NaN
// once more changes nothing.
__device__ __noinline__ void restore_nonfinite(const ScoredParams& p, const BadKeys& bad, int count,
                                               long long bt_row, int g, int D, bool mine, int lo,
                                               int hi, int d0, int nd, uint16_t* out,
                                               float* partial) {
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const bool sees = mine && lo < hi, listed = count <= kMaxBadKeys;
  const int first = __reduce_min_sync(0xffffffffu, sees ? lo : 0x7fffffff);
  const int past = __reduce_max_sync(0xffffffffu, sees ? hi : 0);
  const unsigned long long whole = nd == 64 ? ~0ull : (1ull << nd) - 1ull;
  Odd odd{0, 0, 0};
  for (int left = listed ? count : past - first; left > 0; left -= 32) {
    const int i = left - 1 - lane;
    const int j = i < 0 ? -1 : listed ? bad.key[i] : first + i;
    Odd at[2] = {{0, 0, 0}, {0, 0, 0}};  // what lanes 0-15 and lanes 16-31 hold of key j
    if (j >= first && j < past) {
      const uint4* v = v_row_of(p, bad, bt_row, g, D, j);
      if (v) {
        v += (d0 - half * nd) / 8;
        at[0] = odd_of(v, nd);
        at[1] = odd_of(v + nd / 8, nd);
      }
    }
    const bool any = (at[0].nan | at[0].pos | at[0].neg | at[1].nan | at[1].pos | at[1].neg) != 0;
    for (uint32_t m = __ballot_sync(0xffffffffu, any); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int key = __shfl_sync(0xffffffffu, j, src);
      Odd o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        o[h].nan = __shfl_sync(0xffffffffu, at[h].nan, src);
        o[h].pos = __shfl_sync(0xffffffffu, at[h].pos, src);
        o[h].neg = __shfl_sync(0xffffffffu, at[h].neg, src);
      }
      if (!sees || key < lo || key >= hi) continue;
      odd.nan |= half ? o[1].nan : o[0].nan;
      odd.pos |= half ? o[1].pos : o[0].pos;
      odd.neg |= half ? o[1].neg : o[0].neg;
    }
    // nothing more can change where every element is a NaN
    if (__all_sync(0xffffffffu, !sees || (odd.nan | (odd.pos & odd.neg)) == whole)) break;
  }
  if (!sees) return;
#pragma unroll 1
  for (int x = 0; x < nd; ++x) {
    const unsigned long long bit = 1ull << x;
    if (!((odd.nan | odd.pos | odd.neg) & bit)) continue;
    const bool pos = odd.pos & bit, neg = odd.neg & bit;
    const float f = __uint_as_float((odd.nan & bit) || (pos && neg) ? 0x7fc00000u
                                    : neg                           ? 0xff800000u
                                                                    : 0x7f800000u);
    if (partial)
      partial[x] += f;
    else
      out[x] = static_cast<uint16_t>(
          pack_bf16x2(__uint_as_float(static_cast<uint32_t>(out[x]) << 16) + f, 0.f));
  }
}

// Narrow an item to the key tiles that its rows see (at least one, so that
// rows without keys are written too); a shared-prefix item keeps its piece's tiles.
__device__ __forceinline__ void narrow_item(PrefillItem& m, const int4& keys) {
  m.k_lo = keys.x;
  m.full_lo = keys.z;
  m.full_hi = keys.w;
  if (m.piece >= 0) {
    m.kv_len = min(m.kv_len, keys.y);
  } else {
    m.kv_len = keys.y;
    m.kt0 = keys.x / kTileN;
    m.nkv = max(1, (m.kv_len + kTileN - 1) / kTileN - m.kt0);
  }
}

// Items of the k-th prefill request are numbered tile-major, longest tile
// first: local index l -> kv head l % Hkv, tile ntile - 1 - l / Hkv. The
// request's metadata comes from the CTA's shared-memory copy when it holds
// every prefill request (meta != nullptr), else from global memory.
__device__ __forceinline__ PrefillItem prefill_item(const PrefillParams& p, int n_req, int item,
                                                    int QT, const int4* meta,
                                                    const int* meta_prefix) {
  PrefillItem m;
  int r, local;
  if (meta) {
    int lo = 0, hi = n_req;  // meta_prefix[lo] <= item < meta_prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (meta_prefix[mid] <= item) lo = mid; else hi = mid;
    }
    const int4 v = meta[lo];
    r = v.x;
    m.c = v.y;
    m.q0 = v.z;
    m.n = v.w;
    local = item - meta_prefix[lo];
  } else {
    const int k = upper_index(p.pf_prefix, n_req, item);
    r = __ldg(p.pf_req + k);
    local = item - __ldg(p.pf_prefix + k);
    if (r >= 0) {
      m.c = __ldg(p.num_computed + r);
      m.q0 = __ldg(p.qsl + r);
      m.n = __ldg(p.qsl + r + 1) - m.q0;
    } else {
      m.c = p.shared_len;
      m.q0 = __ldg(p.qsl + p.shared_first);
      m.n = p.shared_num;
    }
  }
  m.g = local % p.num_kv_heads;
  if (r < 0) {
    // shared-prefix item: rows = the run's decode rows (one per request) x
    // the kv head's q heads, keys = one piece of the shared prefix, all of
    // them visible to every row
    const int rest = local / p.num_kv_heads;
    m.piece = rest % p.shared_pieces;
    m.i0 = (rest / p.shared_pieces) * QT;
    const int tiles = (p.shared_len + kTileN - 1) / kTileN;
    m.kt0 = m.piece * p.shared_tpp;
    m.nkv = min(p.shared_tpp, tiles - m.kt0);
    m.kv_len = min((m.kt0 + m.nkv) * kTileN, p.shared_len);
    m.bt_row = static_cast<long long>(p.shared_first) * p.max_blocks;
    return m;
  }
  m.piece = -1;
  m.kt0 = 0;
  const int ntile = (m.n + QT - 1) / QT;
  const int mt = ntile - 1 - local / p.num_kv_heads;
  m.i0 = mt * QT;
  const int i_last = min(m.i0 + QT, m.n) - 1;
  m.kv_len = m.c + i_last + 1;
  m.nkv = (m.kv_len + kTileN - 1) / kTileN;
  m.bt_row = static_cast<long long>(r) * p.max_blocks;
  return m;
}

// Block table entry e of the item's request if it holds keys < kv_len and its
// id is in the pool, else -1.
// SCORED: neither are entries in front of the item's first key.
template <bool SCORED>
__device__ __forceinline__ bool entry_used(const PrefillParams& p, const PrefillItem& m, int e) {
  return (e << p.block_shift) < m.kv_len && (!SCORED || ((e + 1) << p.block_shift) > m.k_lo);
}
template <bool SCORED>
__device__ __forceinline__ int entry_id(const PrefillParams& p, const PrefillItem& m, int e) {
  if (!entry_used<SCORED>(p, m, e)) return -1;
  const int id = __ldg(p.block_table + m.bt_row + e);
  return (id >= 0 && id < p.num_blocks) ? id : -1;
}

// Chunk b (keys 16b .. 16b+15) of tile kt holds keys < kv_len, all of them in
// blocks of the pool.
__device__ __forceinline__ bool chunk_ok(const PrefillParams& p, const PrefillItem& m, int kt, int b) {
  const int k0 = kt * kTileN + b * kChunkKeys;
  if (k0 >= m.kv_len) return false;
  const int bsh = p.block_shift;
  if (bsh == 4) return entry_id<false>(p, m, k0 >> 4) >= 0;
  if (bsh == 5) return entry_id<false>(p, m, k0 >> 5) >= 0;
  return entry_id<false>(p, m, k0 >> 3) >= 0 &&
         (k0 + 8 >= m.kv_len || entry_id<false>(p, m, (k0 >> 3) + 1) >= 0);
}

// cap2 * tanh(u) for z = 2 log2(e) u, cap2 = softcap * log2(e). 1 - 2 / (2^z + 1)
// is off by a few 2^-24 however small u is, so by a few 2^-24 cap2 in the
// exponent of a weight: 2^-15 at most where cap2 <= kCapFixedMax. Wider caps
// need tanh_log2's relative form.
template <bool FIXED>
__device__ __forceinline__ float exact_cap(float z, float cap2) {
  if constexpr (!FIXED) return cap2 * tanh_log2(z);
  return fmaf(-2.f * cap2, __fdividef(1.f, exp2f(z) + 1.f), cap2);
}

// The softmax warps of a SCORED kernel: the roles and lane map of the plain
// ones (see the kernel), with the scores transformed in registers, each row
// masked by its own range, and two things done to keep short items (packed
// documents, windows: a few key tiles each) from waiting on latency one after
// the other. What the next tile or item needs from global memory is loaded a
// tile ahead. And an item's epilogue is left until the next item's first
// tile has been through the softmax, so that the item's last PV runs
// meanwhile; only its reads of O come before that tile's P is published (the
// next PV overwrites O), its stores after.
template <int D, int SC>
__device__ __forceinline__ void scored_softmax(const ScoredParams& p, PrefillShared& sh,
                                               unsigned char* gbase, uint32_t tmem, int n_items) {
  constexpr bool CAP = (SC & kCap) != 0, BIAS = (SC & kBias) != 0;
  constexpr bool FIXED = CAP && !BIAS;  // no running maximum (kCapFixedMax): it stays 0
  using Lay = PrefillLayout<D>;
  constexpr int DH = Lay::DH;
  constexpr int NW = softmax_warps<SC>();
  constexpr int KPT = 512 / NW;  // keys of a tile per thread: 64 or 32
  constexpr int KQ = KPT / 32;
  // O columns per thread in the epilogue; with sixteen warps and D = 64 the
  // first eight hold them all
  constexpr int HC = NW == 16 && D == 128 ? 32 : D / 2;
  constexpr int NQ = HC / 32;
  constexpr uint32_t kRingV = Lay::kK + kScoredKStages * Lay::kTileKV;
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, gsh = 31 - __clz(G);  // G is 1, 2, 4 or 8
  const int ch = lane >> 4;      // of the warp's keys (and O columns), this thread's half
  const int kh = warp >> 3;      // sixteen warps: keys 0..63 or 64..127 of every tile
  const int lane0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
  const int key0 = 64 * kh + KPT * ch;        // this thread's first key of a tile
  const uint32_t scol = 64u * kh;             // the warp's first S (and P) column
  const bool has_o = HC == 32 && D == 64 && NW == 16 ? kh == 0 : true;
  const int ocol = HC * (NW == 16 && D == 128 ? 2 * kh + ch : ch);  // its first O column
  float* sums = reinterpret_cast<float*>(gbase + Lay::kSums);
  const int row = lane0 + (lane & 15);  // query row of this thread (TMEM lane)
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(lane0) << 16);
  BadKeys* bad_lists = reinterpret_cast<BadKeys*>(gbase + Lay::kBad);
  auto valid = [&](int item) { return item >= 0 && item < n_items; };
  const float mul = CAP || BIAS ? 1.f : p.scale_log2;  // scores in registers to base 2
  uint32_t T = 0;  // tiles of earlier items
  bool ok = true;

  // the epilogue of the item before the current one, number it - 1, in two
  // steps around the publication of P (none before the first)
  bool pend = false;
  int pend_i0 = 0, pend_n = 0, pend_q0 = 0, pend_g = 0, pend_piece = -1;
  int pend_lo = 0, pend_hi = 0;
  long long pend_bt = 0;
  float pend_max = 0.f, pend_sum = 0.f;
  auto epilogue_wait = [&](int it, uint32_t Tl) -> bool {
    return wait_small(&sh.o_full, it & 1u, abort_flag) &&
           wait_small(&sh.p_ready[Tl % kSBufs], (Tl / kSBufs) & 1u, abort_flag);
  };
  auto epilogue_load = [&](int it, uint32_t Tl, uint32_t (&o)[NQ][32], int& n_bad) -> bool {
    // the item's bad keys are complete once every thread has published P of
    // its last tile Tl. Five lists: when a thread is here in item it's
    // epilogue, every thread has published all P of item it; others may be
    // storing item it - 1 or filling the lists of the two items after it; no
    // thread uses that of item it - 2 any more, and none fills it again (as
    // item it + 3's) before all have passed here.
    if (!epilogue_wait(it, Tl)) return false;
    n_bad = *reinterpret_cast<volatile int*>(&bad_lists[it % kBadLists].count);
    if (tid == 0) bad_lists[(it + 3) % kBadLists].count = 0;
    tc::fence_after_sync();
    if constexpr (NQ == 2)
      tc::ld_half64<HC>(t_lane, t_lane + 32, o[0], o[NQ - 1]);
    else
      tc::ld_half32_wait<HC>(t_lane + (D == 128 ? scol : 0u), o[0]);
    return true;
  };
  auto epilogue_store = [&](int it, const uint32_t (&o)[NQ][32], int n_bad) {
    float l_tot;
    if constexpr (NW == 16) {
      const float* l = sums + (it & 3) * 256 + row;
      l_tot = l[0] + l[128];
    } else {
      l_tot = pend_sum + __shfl_xor_sync(0xffffffffu, pend_sum, 16);
    }
    const float inv = l_tot == 0.f ? 0.f : 1.f / l_tot;  // no key seen: zeros
    const int qi = pend_i0 + (row >> gsh);
    const bool mine = qi < pend_n && has_o;
    const int head = pend_g * G + (row & (G - 1));
    uint16_t* dst =
        p.out + ((static_cast<long long>(pend_q0) + qi) * p.num_q_heads + head) * D + ocol;
    float* part = nullptr;
    if (pend_piece >= 0) {
      // shared-prefix items keep the row's partial (max, sum, unnormalised O)
      // for the decode of request shared_first + qi: slot of (piece, qi, head)
      const long long pslot =
          (static_cast<long long>(pend_piece) * p.shared_num + qi) * p.num_q_heads + head;
      part = p.shared_o + pslot * D + ocol;
      if (mine) {
        if (ocol == 0) p.shared_ml[pslot] = make_float2(pend_max, l_tot);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float4* d4 = reinterpret_cast<float4*>(part + 32 * q);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            d4[x] = make_float4(__uint_as_float(o[q][4 * x]), __uint_as_float(o[q][4 * x + 1]),
                                __uint_as_float(o[q][4 * x + 2]), __uint_as_float(o[q][4 * x + 3]));
        }
      }
    } else if (mine) {
      // straight from the thread that holds the half row, in whole 32-byte
      // sectors where the output's alignment allows (turning the rows in
      // shared memory first, for stores of whole rows, was slower: 117
      // instead of 107 us on 8191 rows of packed documents)
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        uint4 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t* v = &o[q][8 * x];
          w[x].x = pack_bf16x2(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv);
          w[x].y = pack_bf16x2(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv);
          w[x].z = pack_bf16x2(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv);
          w[x].w = pack_bf16x2(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv);
        }
        if (p.out32) {
          st_global_v8(dst + 32 * q, w[0], w[1]);
          st_global_v8(dst + 32 * q + 16, w[2], w[3]);
        } else {
          uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * q);
#pragma unroll
          for (int x = 0; x < 4; ++x) d4[x] = w[x];
        }
      }
    }
    if (n_bad > 0)
      restore_nonfinite(p, bad_lists[it % kBadLists], n_bad, pend_bt, pend_g, D, mine, pend_lo,
                        pend_hi, ocol, HC, dst, part);
  };

  PrefillItem m{};
  int item = take_item(sh, 0, abort_flag, true, &m);
  RowKeys rk{0, 0, 0};  // the keys of this thread's row
  if (valid(item)) rk = row_of(p, m, m.i0 + (row >> gsh), load_row(p, m, m.i0 + (row >> gsh)));
  int it = 0;
#pragma unroll 1
  for (; valid(item); ++it) {
    const int nkv = m.nkv;
    int item_n = -1;
    RowRaw raw_n{0, 0, 0};
    const bool no_row = m.i0 + (row >> gsh) >= m.n;  // behind the request's rows
    // A row behind the request's holds another request's q, and its threads
    // store nothing. From an infinite maximum on it asks for no rescale, which
    // would move the maxima, and with them the roundings, of its warp's rows.
    float m_run = FIXED ? 0.f : no_row ? INFINITY : -INFINITY, l_run = 0.f;
    // bias per key of distance, base-2 scores
    const float slope2 = BIAS ? slope_log2(p.score, m.g * G + (row & (G - 1))) : 0.f;
#pragma unroll 1
    for (int kt = 0; kt < nkv; ++kt) {
      const uint32_t Tg = T + kt;
      const uint32_t b = Tg % kSBufs;
      const uint32_t t_s = t_lane + kTmemS + kTileN * b;
      if (kt + 1 == nkv) {  // the next item's loads go out
        PrefillItem mn;  // (read again once this item is through: fewer registers)
        item_n = peek_item(sh, it + 1, abort_flag, &mn);
        if (item_n < 0) return;  // aborted
        if (valid(item_n)) raw_n = load_row(p, mn, mn.i0 + (row >> gsh));
      }
      ok = wait_small(&sh.s_full[b], (Tg / kSBufs) & 1u, abort_flag);
      if (!ok) return;
      const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&sh.masks[Tg % kMaskRing]);
      tc::fence_after_sync();
      const int ka = tile_at<SC>(m.kt0, nkv, kt);  // key tile (keys ka*128 ..)
      // `full`: every row of the item sees the whole tile. Masks go by warp,
      // whose 16 rows are a few neighbouring queries: `wfull`.
      const bool full = mask == 0xFFu && ka * kTileN >= m.full_lo &&
                        ka * kTileN + kTileN <= m.full_hi;
      bool wfull = full;
      if (!full) {
        const int k0 = ka * kTileN;
        wfull = mask == 0xFFu &&
                __all_sync(0xffffffffu, no_row || (rk.lo <= k0 && rk.hi >= k0 + kTileN));
      }
      // this thread's keys key0 .. key0+KPT-1 of the tile: sr[0] the first 32
      uint32_t sr[KQ][32];
      auto load_scores = [&]() {
        if constexpr (KQ == 2)
          tc::ld_half64<64>(t_s, t_s + 32, sr[0], sr[KQ - 1]);
        else
          tc::ld_half32_wait<32>(t_s + scol, sr[0]);
      };
      load_scores();
      uint32_t vis[KQ];  // this thread's visible keys, a bit each
#pragma unroll
      for (int q = 0; q < KQ; ++q) vis[q] = 0xffffffffu;
      if (!wfull) {
        const int lo = rk.lo - ka * kTileN - key0, hi = rk.hi - ka * kTileN - key0;
        const uint32_t cm = mask >> (key0 >> 4);
#pragma unroll
        for (int q = 0; q < KQ; ++q)
          vis[q] = bits_between(lo - 32 * q, hi - 32 * q) &
                   (((cm >> (2 * q)) & 1u ? 0xffffu : 0u) |
                    ((cm >> (2 * q + 1)) & 1u ? 0xffff0000u : 0u));
      }
      if constexpr (CAP) {
        // What a masked key holds must not decide which form of the cap is taken.
        if (!wfull) {
#pragma unroll
          for (int q = 0; q < KQ; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(vis[q] & (1u << i))) sr[q][i] = 0u;
        }
        float am[4] = {0.f, 0.f, 0.f, 0.f};  // largest w = S^2
        // the polynomial for all of them, and the vote after it: the maximum
        // and its shuffles then run beside it
        const float2 a0 = make_float2(p.cap_a[0], p.cap_a[0]),
                     a1 = make_float2(p.cap_a[1], p.cap_a[1]),
                     a2 = make_float2(p.cap_a[2], p.cap_a[2]),
                     a3 = make_float2(p.cap_a[3], p.cap_a[3]),
                     a4 = make_float2(p.cap_a[4], p.cap_a[4]);
#pragma unroll
        for (int q = 0; q < KQ; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = make_float2(__uint_as_float(sr[q][i]), __uint_as_float(sr[q][i + 1]));
            const float2 w = fmul2(x, x);
            am[(i >> 1) & 3] = max3f(am[(i >> 1) & 3], w.x, w.y);
            const float2 y = fmul2(x, ffma2(ffma2(ffma2(ffma2(a4, w, a3), w, a2), w, a1), w, a0));
            sr[q][i] = __float_as_uint(y.x);
            sr[q][i + 1] = __float_as_uint(y.y);
          }
        // (nor what lies in q behind the request's rows)
        const float amax = no_row ? 0.f : fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3]));
        if (__any_sync(0xffffffffu, amax > p.cap_lim2)) {
          // exact form, eight scores at a time, S replaced in tensor memory
          // (all in registers, it was 8% faster where every tile needs it and
          // 11% slower where one in eight does: more code in the way of the
          // polynomial)
          const float cap2 = p.score.softcap * kLog2e;
#pragma unroll 1
          for (int c = 0; c < KPT; c += 8) {
            uint32_t x[8];
            tc::ld_half8<KPT>(t_s + scol + c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = __float_as_uint(exact_cap<FIXED>(__uint_as_float(x[i]) * p.cap_z, cap2));
            tc::st_half8<KPT>(t_s + scol + c, x);
          }
          tc::wait_st();
          load_scores();
        }
      }
      if constexpr (BIAS) {
        // score (with a cap already in base 2) - slope2 * |ref - j|
        const float2 k2 = CAP ? make_float2(1.f, 1.f) : make_float2(p.scale_log2, p.scale_log2);
        const int d = ka * kTileN + key0 - rk.ref;  // of this thread's first key
        const float d0 = static_cast<float>(d);
        if (__all_sync(0xffffffffu, d + KPT - 1 <= 0)) {  // every key at or before its row's position
          const float2 base = make_float2(slope2 * d0, slope2 * d0);
          const float2 sl = make_float2(slope2, slope2);
#pragma unroll
          for (int q = 0; q < KQ; ++q)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 bias = ffma2(
                  sl, make_float2(static_cast<float>(q * 32 + i), static_cast<float>(q * 32 + i + 1)),
                  base);
              const float2 y = ffma2(
                  make_float2(__uint_as_float(sr[q][i]), __uint_as_float(sr[q][i + 1])), k2, bias);
              sr[q][i] = __float_as_uint(y.x);
              sr[q][i + 1] = __float_as_uint(y.y);
            }
        } else {
#pragma unroll
          for (int q = 0; q < KQ; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sr[q][i] = __float_as_uint(__uint_as_float(sr[q][i]) * k2.x -
                                         slope2 * fabsf(d0 + static_cast<float>(q * 32 + i)));
        }
      }
      if (!wfull) {  // invisible keys become -inf
#pragma unroll
        for (int q = 0; q < KQ; ++q)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(vis[q] & (1u << i))) sr[q][i] = __float_as_uint(-INFINITY);
      }
      if constexpr (!FIXED) {
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < KQ; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx4[(i >> 1) & 3] =
                max3f(mx4[(i >> 1) & 3], __uint_as_float(sr[q][i]), __uint_as_float(sr[q][i + 1]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        // (scale > 0 keeps the argmax; both threads of the row get the same bits)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * mul;
        if (__any_sync(0xffffffffu, mx > m_run + kRescaleLog2)) {
          const float m_new = fmaxf(m_run, mx);
          const float alpha = (m_new == -INFINITY) ? 1.f : exp2f(m_run - m_new);
          l_run *= alpha;
          m_run = m_new;
          if (kt > 0) {
            // O holds PV of the item's earlier tiles; the last of them is PV(Tg-1)
            const uint32_t Tp = Tg - 1;
            ok = wait_small(&sh.pv_done[Tp % kSBufs], (Tp / kSBufs) & 1u, abort_flag);
            if (!ok) return;
            tc::fence_after_sync();
#pragma unroll 1
            for (int q = 0; q < HC / 32; ++q) {  // this thread's O columns HC*ch + 32q ..
              uint32_t o[32];
              tc::ld_half32<HC>(t_lane + 32 * q, o);
              tc::wait32(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tc::st_half32<HC>(t_lane + 32 * q, o);
            }
          }
        }
      }
      // P = 2^(s * scale - m) as bf16 (-inf -> 0) over the S buffer, a column
      // for two keys (the even one in the low half), in the order of p_column
      float2 ps4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                       make_float2(0.f, 0.f)};
      const float msub = (m_run == -INFINITY) ? 0.f : m_run;
      const float2 sc2 = make_float2(mul, mul), nm2 = make_float2(-msub, -msub);
#pragma unroll
      for (int q = 0; q < KQ; ++q) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float2 e = make_float2(__uint_as_float(sr[q][2 * j]), __uint_as_float(sr[q][2 * j + 1]));
          if constexpr (!FIXED) e = ffma2(e, sc2, nm2);
          const float2 pp = make_float2(exp2f(e.x), exp2f(e.y));
          pk[j] = pack_bf16x2(pp.x, pp.y);
          ps4[j & 3] = fadd2(ps4[j & 3], pp);
        }
        tc::st_half16<KPT / 2>(t_s + scol + 16 * q, pk);
      }
      l_run += ((ps4[0].x + ps4[1].x) + (ps4[2].x + ps4[3].x)) +
               ((ps4[0].y + ps4[1].y) + (ps4[2].y + ps4[3].y));
      // V rows of keys past kv_len or of chunks not loaded must be zero
      // (0 * NaN): for such a tile wait for its V copy first; thread (row,
      // ch) clears 64-element chunk ch of V row `row`
      // in a tile that some row does not see in full, the V rows that
      // stay must be finite
      if (!full) {
        // S(Tg) done implies PV(Tg-3) done, so the slot's barrier is at V(Tg),
        // pending or landed
        const int slot = static_cast<int>(Tg % kScoredVStages);
        ok = wait_small(&sh.v_full[slot], (Tg / kScoredVStages) & 1u, abort_flag);
        if (!ok) return;
        constexpr int VN = 64 / NW;  // 16-byte units of the V row per thread: 8 or 4
        uint4* v4 = reinterpret_cast<uint4*>(gbase + kRingV + slot * Lay::kTileKV +
                                             (row >> 3) * Lay::kGroupBytes + ch * 1024 +
                                             (row & 7) * 128) + VN * kh;
        if (ch < DH && (ka * kTileN + row >= m.kv_len || !(mask >> (row >> 4) & 1u) ||
                        ka * kTileN + row < m.k_lo)) {
#pragma unroll
          for (int x = 0; x < VN; ++x) v4[x] = make_uint4(0, 0, 0, 0);
        } else if (ch < DH && zero_nonfinite<VN>(v4)) {
          BadKeys& bad = reinterpret_cast<BadKeys*>(gbase + Lay::kBad)[it % kBadLists];
          const int i = atomicAdd(&bad.count, 1);
          if (i == 0) {
            bad.k_lo = m.k_lo;
            bad.kv_len = m.kv_len;
          }
          if (i < kMaxBadKeys) bad.key[i] = ka * kTileN + row;
        }
        fence_proxy_async_smem();
      }
      if constexpr (NW == 16) {
        // the item's row sums, in four places by turns: place it & 3 is
        // filled again four items later
        if (kt + 1 == nkv) {
          const float l2 = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
          if (ch == 0) sums[(it & 3) * 256 + kh * 128 + row] = l2;
        }
      }
      tc::wait_st();
      if (!pend) {
        tc::fence_before_sync();
        mbar_arrive(&sh.p_ready[b]);
      } else {
        uint32_t o[NQ][32];
        int n_bad = 0;
        // warps that hold no O wait all the same: what they add to the bad-key
        // lists and the row sums has to come after the other warps' reads and
        // after thread 0's emptying of the list. p_ready, on which every thread
        // has arrived, orders that; o_full, a commit, only the tensor core's work.
        if (has_o ? !epilogue_load(it - 1, T - 1, o, n_bad) : !epilogue_wait(it - 1, T - 1)) return;
        tc::fence_before_sync();
        mbar_arrive(&sh.p_ready[b]);
        if (has_o) epilogue_store(it - 1, o, n_bad);
        pend = false;
      }
    }
    pend = true;
    pend_i0 = m.i0;
    pend_n = m.n;
    pend_q0 = m.q0;
    pend_g = m.g;
    pend_piece = m.piece;
    pend_bt = m.bt_row;
    pend_lo = rk.lo;
    pend_hi = rk.hi;
    pend_max = m_run;
    pend_sum = l_run;
    T += nkv;
    item = take_item(sh, it + 1, abort_flag, true, &m);
    if (valid(item)) rk = row_of(p, m, m.i0 + (row >> gsh), raw_n);
  }
  if (pend) {
    uint32_t o[NQ][32];
    int n_bad = 0;
    if (has_o && epilogue_load(it - 1, T - 1, o, n_bad)) epilogue_store(it - 1, o, n_bad);
  }
}

// Persistent CTAs; each claims its items from a counter (items come longest
// first within a request). Every role walks that list on its own and
// the roles meet only at mbarriers, so the next item's Q/K/V copies and first
// S MMAs overlap the current item's last tiles and epilogue. With NW softmax
// warps (eight; sixteen in a capped instance) and rings of KST K and VST V slots
// (plain 3 and 2, scored 2 and 3):
//   warp NW + 1: Q copy (once the previous item's last S is done) and K tiles
//            (slot T % KST is refilled once S(T) is done);
//   warp NW + 2: V tiles (slot T % VST is refilled once PV(T) is done);
//   warp NW, lane 0: every S, S(T) = Q K^T into S buffer T % 3 once PV(T-3)
//            has read the P that the buffer held;
//   warp NW + 3, lane 0: every PV, O += P V with P read from TMEM, where the
//            softmax warps wrote it over the tile's S (bf16 pairs, one pair
//            per 32-bit column);
//   warps 0..NW-1: the softmax of every tile and the item's epilogue. Of eight,
//            each has 16 query rows and half of each row per thread (each thread
//            normalises and writes half of its row's output columns); of sixteen,
//            two warps share 16 rows.
//
// SCORED (SC other than kPlain): the scores are capped, biased or masked by
// key ranges (ScoreParams). The K-copy warp finds the keys that an item's rows
// see and publishes them with the item, so every role walks only those tiles;
// the softmax warps transform their scores in registers and mask by each
// row's own range. One instance per combination of cap and bias: with all of
// it in one, chosen at run time, the kernel's 130 KB of code missed the
// instruction caches (no_instruction was its largest stall, and 8191 rows of
// packed documents took 180 us instead of 115).
template <int D, int SC>
__global__ void __launch_bounds__(prefill_threads<SC>(), 1)
    prefill_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                   const std::conditional_t<SC == kPlain, PrefillParams, ScoredParams> p) {
  using Lay = PrefillLayout<D>;
  constexpr int DH = Lay::DH;
  constexpr bool SCORED = SC != kPlain;
  constexpr int NW = softmax_warps<SC>();  // warp NW: S, NW + 1: K, NW + 2: V, NW + 3: PV
  constexpr int KST = SCORED ? kScoredKStages : kKStages;
  constexpr int VST = SCORED ? kScoredVStages : kVStages;
  constexpr uint32_t kRingV = Lay::kK + KST * Lay::kTileKV;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  PrefillShared& sh = *reinterpret_cast<PrefillShared*>(gbase + Lay::kBar);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int G = p.group, QT = kTileM / G;

  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_free, 1);
    for (int i = 0; i < KST; ++i) mbar_init(&sh.k_full[i], 1);
    for (int i = 0; i < VST; ++i) mbar_init(&sh.v_full[i], 1);
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&sh.s_full[i], SCORED ? 2 : 1);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.p_ready[i], NW * 32);
    }
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    for (int i = 0; i < kItemQ; ++i) {
      mbar_init(&sh.iq_full[i], 1);
      mbar_init(&sh.iq_free[i], NW + 3);
    }
    sh.abort = 0;
    for (int i = 0; i < kBadLists; ++i) reinterpret_cast<BadKeys*>(gbase + Lay::kBad)[i].count = 0;
    fence_barrier_init();
  }
  if (tid == 32 * (NW + 1)) {
    prefetch_tensormap(&kv_map);
    prefetch_tensormap(&q_map);
  }
  if (warp == NW) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_trigger();
  // barriers, tensor maps and TMEM above do not depend on the plan; its output does
  pdl_wait();
  const int n_items = static_cast<int>(p.hdr[kHdrPrefillItems]);
  const int n_req = static_cast<int>(p.hdr[kHdrPrefillReqs]);
  int4* meta_s = reinterpret_cast<int4*>(gbase + Lay::kMeta);
  int* meta_prefix_s = reinterpret_cast<int*>(gbase + Lay::kMeta + kMetaReqs * 16);
  if (n_req <= kMetaReqs) {
    for (int i = tid; i <= n_req; i += prefill_threads<SC>()) {
      meta_prefix_s[i] = __ldg(p.pf_prefix + i);
      if (i < n_req) {
        const int r = __ldg(p.pf_req + i);
        if (r >= 0) {
          const int q0 = __ldg(p.qsl + r);
          meta_s[i] = make_int4(r, __ldg(p.num_computed + r), q0, __ldg(p.qsl + r + 1) - q0);
        } else {  // the shared-prefix items
          meta_s[i] = make_int4(-1, p.shared_len, __ldg(p.qsl + p.shared_first), p.shared_num);
        }
      }
    }
  }
  // the first work item is claimed while the CTA sets up
  int first_claim = 0;
  if (tid == 32 * (NW + 1)) first_claim = static_cast<int>(atomicAdd(&p.hdr[kHdrPrefillNext], 1u));
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const int4* meta = n_req <= kMetaReqs ? meta_s : nullptr;
  const int* meta_prefix = meta_prefix_s;
  auto valid = [&](int item) { return item >= 0 && item < n_items; };

  if (warp == NW + 1 || warp == NW + 2) {
    // ================= copy warps. Lane (chunk b, d half dh), lanes
    // 0 .. 8*DH-1, issues the copies of that chunk (one of 16 rows, or two of
    // 8 rows for 8-token blocks); the block ids of a 32-entry window of the
    // block table sit in the lanes' registers.
    const int ln = tid & 31;
    const bool is_v = warp == NW + 2;
    const int S = is_v ? VST : KST;
    uint64_t* full = is_v ? sh.v_full : sh.k_full;
    const uint32_t ring = is_v ? kRingV : Lay::kK;
    const int bsh = p.block_shift;
    const int E = kTileN >> bsh;  // table entries per tile
    uint32_t T = 0;               // tiles issued so far (all items)
    bool ok = true;
    int q_loads = 0;
    // SCORED, K: the next item is claimed, and the keys of its rows looked up
    // (two dependent loads), while the current one's last tiles are still in
    // flight, and published for every role at once
    int claimed = n_items;
    PrefillItem claimed_m{};
    auto claim_ahead = [&](int it) {
      const int slot = it % kItemQ;
      int item = n_items;
      if (ln == 0) {
        if (it >= kItemQ)
          ok = wait_or_abort(&sh.iq_free[slot], ((it - kItemQ) / kItemQ) & 1u, abort_flag);
        if (ok) item = it == 0 ? first_claim : static_cast<int>(atomicAdd(&p.hdr[kHdrPrefillNext], 1u));
      }
      claimed = __shfl_sync(0xffffffffu, item, 0);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (valid(claimed)) {
        claimed_m = prefill_item(p, n_req, claimed, QT, meta, meta_prefix);
        if constexpr (SCORED) narrow_item(claimed_m, item_keys(p, claimed_m, QT));
      }
      if (ln == 0) {
        sh.item_q[slot] = claimed;
        sh.item_m[slot] = claimed_m;
        mbar_arrive(&sh.iq_full[slot]);
      }
    };
    for (int it = 0; ok; ++it) {
      int item;
      PrefillItem m;
      if (SCORED && !is_v) {
        claim_ahead(it);
        item = claimed;
        m = claimed_m;
        if (it > 0 && ok && valid(item)) ok = wait_or_abort(&sh.q_free, (it - 1) & 1u, abort_flag);
      } else if (!is_v) {
        // the Q buffer is free once the previous item's last S is done; only
        // then is the next item claimed (work counter), so that items go to
        // the CTAs that are about to be idle
        if (it > 0) ok = wait_or_abort(&sh.q_free, (it - 1) & 1u, abort_flag);
        if (!ok) break;
        item = n_items;
        if (ln == 0) {
          const int slot = it % kItemQ;
          if (it >= kItemQ) ok = wait_or_abort(&sh.iq_free[slot], ((it - kItemQ) / kItemQ) & 1u, abort_flag);
          if (ok) item = it == 0 ? first_claim : static_cast<int>(atomicAdd(&p.hdr[kHdrPrefillNext], 1u));
          sh.item_q[slot] = item;
          mbar_arrive(&sh.iq_full[slot]);
        }
        item = __shfl_sync(0xffffffffu, item, 0);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      } else {
        item = take_item(sh, it, abort_flag, true, SCORED ? &m : nullptr);
        if (item < 0) ok = false;
      }
      if (!ok || !valid(item)) break;
      if constexpr (!SCORED) m = prefill_item(p, n_req, item, QT, meta, meta_prefix);
      if (!is_v) {
        if (ln == 0) {
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&sh.q_full, DH * Lay::kChunk);
#pragma unroll
          for (int dh = 0; dh < DH; ++dh)
            tma_load_3d(gbase + Lay::kQ + dh * Lay::kChunk, &q_map, dh * 64, m.g * G, m.q0 + m.i0,
                        &sh.q_full);
        }
        ++q_loads;
      }
      int win_base = -1000000, win_val = -1;
      for (int kt = 0; kt < m.nkv; ++kt) {
        const int slot = static_cast<int>(T % S);
        if (T >= static_cast<uint32_t>(S)) {
          // the K slot is free once S(T-S) is done, the V slot once PV(T-S) is
          const uint32_t Tp = T - S;
          ok = is_v ? wait_or_abort(&sh.pv_done[Tp % kSBufs], (Tp / kSBufs) & 1u, abort_flag)
                    : wait_or_abort(&sh.s_full[Tp % kSBufs], (Tp / kSBufs) & 1u, abort_flag);
          if (!ok) break;
        }
        const int ka = tile_at<SC>(m.kt0, m.nkv, kt);  // key tile (keys ka*128 ..)
        if (ka * E + E > win_base + 32 || ((SC & kBias) && ka * E < win_base)) {
          // 32 entries from this tile's on (last to first: up to this tile's)
          win_base = (SC & kBias) ? max(0, ka * E + E - 32) : ka * E;
          const int e = win_base + ln;
          win_val = entry_id<SCORED>(p, m, e);
          if (!is_v && entry_used<SCORED>(p, m, e) && win_val < 0)
            atomicOr(&g_errors_prefill, kErrBlockRange);
        }
        // lane j < E copies the K (or V) rows of table entry ka*E + j, kv
        // head g: one box of B rows x D, 8-row groups of pool row
        // (block * 2 + k|v) * B
        const int id = __shfl_sync(0xffffffffu, win_val, (ka * E + (ln & (E - 1)) - win_base) & 31);
        const bool mine = ln < E && id >= 0;
        if constexpr (SCORED) {
          if (!is_v) {
            // the tile's chunks without a used entry out of the pool, a bit
            // each (unused entries lie outside every row's range)
            const uint32_t bad =
                __ballot_sync(0xffffffffu, ln < E && id < 0 && entry_used<true>(p, m, ka * E + ln));
            if (ln == 0) {
              uint32_t ok8 = 0xffu;
              for (uint32_t w = bad; w; w &= w - 1) {
                const int e = __ffs(w) - 1;  // entry: chunk e, 2e and 2e+1, or e/2
                ok8 &= ~(bsh == 5 ? 3u << (2 * e) : bsh == 4 ? 1u << e : 1u << (e >> 1));
              }
              sh.masks[T % kMaskRing] = ok8;  // (seen by way of k_full and the S thread)
            }
          }
        }
        const uint32_t box = static_cast<uint32_t>(Lay::kGroupBytes) << (bsh - 3);
        const uint32_t tx = __reduce_add_sync(0xffffffffu, mine ? box : 0u);
        if (ln == 0) {
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&full[slot], tx);
        }
        __syncwarp();
        if (mine)
          tma_load_5d(gbase + ring + slot * Lay::kTileKV + ln * box, &kv_map, 0, 0, 0, m.g,
                      ((id * 2 + (is_v ? 1 : 0)) << bsh) >> 3, &full[slot]);
        ++T;
      }
    }
    if (!ok) {  // let the copies in flight land before the shared memory goes away
      for (int s = 0; s < S; ++s)
        if (T > static_cast<uint32_t>(s)) {
          const uint32_t last = s + S * ((T - 1 - s) / S);
          mbar_wait(&full[s], (last / S) & 1u, kDrainLimitNs);
        }
      if (!is_v && q_loads > 0) mbar_wait(&sh.q_full, (q_loads - 1) & 1u, kDrainLimitNs);
    }
  } else if (warp == NW || warp == NW + 3) {
    // ================= MMA threads: warp NW issues every S, warp NW + 3 every PV
    if ((tid & 31) == 0) {
      const bool is_s = warp == NW;
      constexpr uint32_t idesc_qk = tc::idesc_bf16(kTileM, kTileN, 0);
      constexpr uint32_t idesc_pv = tc::idesc_bf16(kTileM, D, 1);
      uint32_t T = 0;  // tiles of earlier items
      bool ok = true;
      for (int it = 0; ok; ++it) {
        PrefillItem m;
        const int item = take_item(sh, it, abort_flag, false, SCORED ? &m : nullptr);
        if (item < 0) ok = false;
        if (!ok || !valid(item)) break;
        if constexpr (!SCORED) m = prefill_item(p, n_req, item, QT, meta, meta_prefix);
        const int nkv = m.nkv;
        if (is_s) {
          ok = wait_or_abort(&sh.q_full, it & 1u, abort_flag);
          for (int kt = 0; ok && kt < nkv; ++kt) {
            // S(Tk) = Q K^T into buffer Tk % 3, once PV(Tk-3) has read the
            // P that the buffer holds and K(Tk) has landed
            const uint32_t Tk = T + kt;
            const uint32_t b = Tk % kSBufs;
            if (Tk >= static_cast<uint32_t>(kSBufs))
              ok = wait_or_abort(&sh.pv_done[b], ((Tk - kSBufs) / kSBufs) & 1u, abort_flag);
            const uint32_t ks = SCORED ? Tk % KST : b;
            if (ok) ok = wait_or_abort(&sh.k_full[ks], (Tk / KST) & 1u, abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t sub = (kk & 3) * 32;  // 16 elements within the 64-element half
              const uint64_t a = tc::sw128_desc(base + Lay::kQ + (kk >> 2) * Lay::kChunk + sub, 16, 1024);
              const uint64_t bd = tc::sw128_desc(
                  base + Lay::kK + ks * Lay::kTileKV + (kk >> 2) * 1024 + sub, 16, Lay::kGroupBytes);
              tc::mma_bf16(tmem + kTmemS + kTileN * b, a, bd, idesc_qk, kk > 0);
            }
            tc::commit(&sh.s_full[b]);  // S in TMEM, and the K slot free
            // SCORED: this thread's own arrival, which releases what it has seen
            // of the K-copy warp's writes (the tile's mask) to the softmax warps
            if constexpr (SCORED) mbar_arrive(&sh.s_full[b]);
            if (kt == nkv - 1) tc::commit(&sh.q_free);
          }
        } else {
          for (int kt = 0; ok && kt < nkv; ++kt) {
            // O += P V for tile Tg, P read from its S buffer. The first PV of
            // an item overwrites O: the softmax warps publish P of an item's
            // first tile only after their epilogue of the previous item has
            // read O.
            const uint32_t Tg = T + kt;
            const uint32_t b = Tg % kSBufs;
            const int slot = static_cast<int>(Tg % VST);
            ok = wait_or_abort(&sh.p_ready[b], (Tg / kSBufs) & 1u, abort_flag);
            if (ok) ok = wait_or_abort(&sh.v_full[slot], (Tg / VST) & 1u, abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t vbase = base + kRingV + slot * Lay::kTileKV;
#pragma unroll
            for (int kk = 0; kk < kTileN / 16; ++kk) {
              // keys 16kk .. 16kk+15: two 8-key groups (SBO), d halves 1 KB apart (LBO)
              const uint64_t bd = tc::sw128_desc(vbase + kk * 2 * Lay::kGroupBytes, 1024, Lay::kGroupBytes);
              tc::mma_bf16_ts(tmem, tmem + kTmemS + kTileN * b + p_column<SC>(kk), bd, idesc_pv,
                              (kt > 0 || kk > 0) ? 1u : 0u);
            }
            tc::commit(&sh.pv_done[b]);  // P's buffer and the V slot free
            if (kt == nkv - 1) tc::commit(&sh.o_full);  // the item's O is complete
          }
        }
        T += nkv;
      }
      // every MMA of this thread (and the arrivals of its commits) done
      // before teardown
      tc::commit(&sh.drain[is_s ? 0 : 1]);
      mbar_wait(&sh.drain[is_s ? 0 : 1], 0, ok ? kWaitLimitNs : kDrainLimitNs);
    }
    __syncwarp();
  } else if constexpr (SCORED) {
    scored_softmax<D, SC>(p, sh, gbase, tmem, n_items);
  } else {
    // ================= softmax warps 0..7: every tile of every item. Warp w
    // owns TMEM lanes (query rows) lane0 .. lane0+15 with lane0 = 32*(w%4) +
    // 16*(w/4) (warp w reaches lanes 32*(w%4) .. +31 only). Of each row,
    // thread t < 16 takes keys 0..63 of every tile and thread t + 16 keys
    // 64..127 (the 16x32bx2 TMEM access shape), so a row's max needs one
    // shuffle and no warp waits for another.
    constexpr int HC = D / 2;  // O columns per thread
    const int lane = tid & 31;
    const int ch = lane >> 4;  // key half of this thread
    const int lane0 = 32 * (warp & 3) + 16 * (warp >> 2);
    const int row = lane0 + (lane & 15);  // query row of this thread (TMEM lane)
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lane0) << 16);
    uint32_t T = 0;
    bool ok = true;
    // chunk validity of tile kt of item m (lanes 0..7), read one tile ahead
    auto load_ids = [&](const PrefillItem& mm, int kt) -> int {
      return (lane < 8 && kt < mm.nkv && chunk_ok(p, mm, mm.kt0 + kt, lane)) ? 1 : -1;
    };
    int item = take_item(sh, 0, abort_flag, true, nullptr);
    PrefillItem m{};
    int next_id = -1;
    if (valid(item)) {
      m = prefill_item(p, n_req, item, QT, meta, meta_prefix);
      next_id = load_ids(m, 0);
    }
    for (int it = 0; ok && valid(item); ++it) {
      const int nkv = m.nkv;
      const int qi = m.i0 + row / G;                // query of this row
      const int lim = min(m.c + qi, m.kv_len - 1);  // last key this row may see
      float m_run = -INFINITY, l_run = 0.f;
      for (int kt = 0; kt < nkv; ++kt) {
        const uint32_t Tg = T + kt;
        const uint32_t b = Tg % kSBufs;
        const uint32_t t_s = t_lane + kTmemS + kTileN * b;
        const uint32_t mask = __ballot_sync(0xffffffffu, next_id >= 0) & 0xFFu;
        ok = wait_or_abort(&sh.s_full[b], (Tg / kSBufs) & 1u, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        // a tile every row sees in full needs no mask; otherwise key j of the
        // tile is visible iff j <= lim - 128 ka and its 16-key chunk was
        // loaded (chunk c = keys 16c .. 16c+15)
        const int ka = m.kt0 + kt;  // key tile (keys ka*128 ..)
        const bool full = ka * kTileN + kTileN - 1 <= m.c + m.i0 && mask == 0xFFu;
        // this thread's keys 64ch .. 64ch+63 of the tile: sr[0] the first 32
        uint32_t sr[2][32];
        tc::ld_half32<64>(t_s, sr[0]);
        tc::ld_half32<64>(t_s + 32, sr[1]);
        tc::wait32(sr[0]);
        tc::wait32(sr[1]);
        if (!full) {  // invisible keys become -inf
          const int jlim = lim - ka * kTileN - 64 * ch;
          const uint32_t cm = mask >> (4 * ch);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int j = q * 32 + i;
              if (!(((cm >> (j >> 4)) & 1u) && j <= jlim)) sr[q][i] = __float_as_uint(-INFINITY);
            }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx4[(i >> 1) & 3] =
                max3f(mx4[(i >> 1) & 3], __uint_as_float(sr[q][i]), __uint_as_float(sr[q][i + 1]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        // (scale > 0 keeps the argmax; both threads of the row get the same bits)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * p.scale_log2;
        if (__any_sync(0xffffffffu, mx > m_run + kRescaleLog2)) {
          const float m_new = fmaxf(m_run, mx);
          const float alpha = (m_new == -INFINITY) ? 1.f : exp2f(m_run - m_new);
          l_run *= alpha;
          m_run = m_new;
          if (kt > 0) {
            // O holds PV of the item's earlier tiles; the last of them is PV(Tg-1)
            const uint32_t Tp = Tg - 1;
            ok = wait_or_abort(&sh.pv_done[Tp % kSBufs], (Tp / kSBufs) & 1u, abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int q = 0; q < HC / 32; ++q) {  // this thread's O columns HC*ch + 32q ..
              uint32_t o[32];
              tc::ld_half32<HC>(t_lane + 32 * q, o);
              tc::wait32(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tc::st_half32<HC>(t_lane + 32 * q, o);
            }
          }
        }
        // P = 2^(s * scale - m) as bf16 (-inf -> 0) over the S buffer: column
        // c holds keys 2c (low half) and 2c+1, so this thread's keys land in
        // columns 32ch .. 32ch+31 (pairs of keys in the packed fp32x2 FMA / add)
        float2 ps4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        const float msub = (m_run == -INFINITY) ? 0.f : m_run;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-msub, -msub);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 e = ffma2(
                make_float2(__uint_as_float(sr[q][2 * j]), __uint_as_float(sr[q][2 * j + 1])), sc2, nm2);
            const float2 pp = make_float2(exp2f(e.x), exp2f(e.y));
            pk[j] = pack_bf16x2(pp.x, pp.y);
            ps4[j & 3] = fadd2(ps4[j & 3], pp);
          }
          tc::st_half16<32>(t_s + 16 * q, pk);
        }
        l_run += ((ps4[0].x + ps4[1].x) + (ps4[2].x + ps4[3].x)) +
                 ((ps4[0].y + ps4[1].y) + (ps4[2].y + ps4[3].y));
        // V rows of keys past kv_len or of chunks not loaded must be zero
        // (0 * NaN): for such a tile wait for its V copy first; thread (row,
        // ch) clears 64-element chunk ch of V row `row`
        if (ka * kTileN + kTileN > m.kv_len || mask != 0xFFu) {
          const int slot = static_cast<int>(Tg % kVStages);
          // S(Tg) done only implies PV(Tg-3) done, so the slot's copy
          // barrier may be anywhere from V(Tg-2) pending to V(Tg) landed;
          // once PV(Tg-2) is done (slot released) it is V(Tg) pending or landed
          if (Tg >= static_cast<uint32_t>(kVStages)) {
            const uint32_t Tp = Tg - kVStages;
            ok = wait_or_abort(&sh.pv_done[Tp % kSBufs], (Tp / kSBufs) & 1u, abort_flag);
          }
          if (ok) ok = wait_or_abort(&sh.v_full[slot], (Tg / kVStages) & 1u, abort_flag);
          if (!ok) break;
          if (ch < DH && (ka * kTileN + row >= m.kv_len || !(mask >> (row >> 4) & 1u))) {
            uint4* v4 = reinterpret_cast<uint4*>(gbase + Lay::kV + slot * Lay::kTileKV +
                                                 (row >> 3) * Lay::kGroupBytes + ch * 1024 +
                                                 (row & 7) * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) v4[x] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&sh.p_ready[b]);
        next_id = load_ids(m, kt + 1);  // its latency hides under the next S wait
      }
      if (!ok) break;
      // ---- the next item's id and metadata, while the last PV runs
      const int item_n = take_item(sh, it + 1, abort_flag, true, nullptr);
      if (item_n < 0) {  // aborted
        ok = false;
        break;
      }
      PrefillItem m_next{};
      if (valid(item_n)) {
        m_next = prefill_item(p, n_req, item_n, QT, meta, meta_prefix);
        next_id = load_ids(m_next, 0);
      }
      // ---- epilogue: this thread's O columns HC*ch .. HC*ch + HC - 1 of its row
      ok = wait_or_abort(&sh.o_full, it & 1u, abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const float l_tot = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
      const float inv = 1.f / l_tot;
      const bool store = qi < m.n;
      const int head = m.g * G + row % G;
      // shared-prefix items keep the row's partial (max, sum, unnormalised O)
      // for the decode of request shared_first + qi: slot of (piece, qi, head)
      const bool partial = m.piece >= 0;
      const long long pslot = (static_cast<long long>(m.piece) * p.shared_num + qi) * p.num_q_heads + head;
      if (partial && store && ch == 0) p.shared_ml[pslot] = make_float2(m_run, l_tot);
      uint16_t* dst = p.out + (static_cast<long long>(m.q0 + qi) * p.num_q_heads + head) * D + HC * ch;
#pragma unroll 1
      for (int q = 0; q < HC / 32; ++q) {
        uint32_t o[32];
        tc::ld_half32<HC>(t_lane + 32 * q, o);
        tc::wait32(o);
        if (!store) continue;
        if (partial) {
          float4* d4 = reinterpret_cast<float4*>(p.shared_o + pslot * D + HC * ch + 32 * q);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            d4[x] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * q);
#pragma unroll
          for (int x = 0; x < 4; ++x) d4[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        }
      }
      T += nkv;
      m = m_next;
      item = item_n;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == NW) {
    tc::fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int D, int SC>
static cudaError_t launch_prefill_t(const ScoredParams& p, const CUtensorMap& kv_map,
                                    const CUtensorMap& q_map, int grid, cudaStream_t stream) {
  auto kern = prefill_kernel<D, SC>;
  const int smem = static_cast<int>(PrefillLayout<D>::kAlloc);
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_attr_once(kern, smem, attr_done);
  if (e != cudaSuccess) return e;
  if constexpr (SC == kPlain)
    return launch_pdl(kern, dim3(grid), dim3(prefill_threads<SC>()), static_cast<size_t>(smem), stream, kv_map,
                      q_map, static_cast<const PrefillParams&>(p));
  else
    return launch_pdl(kern, dim3(grid), dim3(prefill_threads<SC>()), static_cast<size_t>(smem), stream, kv_map,
                      q_map, p);
}

// kCapPoly in terms of S = u / ratio and base-2 scores; false (and zeros) where
// that is not to be used: ratio outside its range, or a coefficient that is not
// a normal fp32 number.
static bool cap_coefficients(float softcap, float ratio, float (&out)[5]) {
  bool ok = ratio >= kCapRatioMin && ratio <= kCapRatioMax;
  double f = static_cast<double>(softcap) * kLog2e * ratio;
  for (int i = 0; i < 5; ++i, f *= static_cast<double>(ratio) * ratio) {
    const double c = kCapPoly[i] * f, size = c < 0 ? -c : c;
    ok = ok && size >= FLT_MIN && size <= FLT_MAX;
    out[i] = ok ? static_cast<float>(c) : 0.f;
  }
  if (!ok)
    for (float& c : out) c = 0.f;
  return ok;
}

cudaError_t launch_prefill(const AttnArgs& a, const AttnWorkspace& ws, const CUtensorMap& kv_map,
                           const CUtensorMap& q_map, int num_sms, cudaStream_t stream) {
  ScoredParams p;
  p.out = a.out;
  p.pool = static_cast<const uint16_t*>(a.kv_cache);
  p.num_tokens = a.num_tokens;
  p.block_table = a.block_table;
  p.max_blocks = a.max_blocks;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.num_computed = a.num_computed;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.block_shift = a.block_shift;
  p.scale_log2 = a.scale * kLog2e;
  p.score = a.score;
  p.cap_z = a.score.softcap > 0.f ? 2.f * kLog2e * (a.scale / a.score.softcap) : 0.f;
  p.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
  const float ratio = a.score.softcap > 0.f ? a.scale / a.score.softcap : 0.f;
  const bool poly = cap_coefficients(a.score.softcap, ratio, p.cap_a);
  p.cap_lim2 = poly ? (kCapLim / ratio) * (kCapLim / ratio) : -1.f;
  const bool wide_cap = a.score.softcap * kLog2e > kCapFixedMax;
  p.hdr = ws.hdr;
  p.pf_req = ws.pf_req;
  p.pf_prefix = ws.pf_prefix;
  p.shared_len = a.shared_len;
  p.shared_first = a.shared_first;
  p.shared_num = a.shared_num;
  p.shared_pieces = a.shared_pieces;
  p.shared_tpp = a.shared_tpp;
  p.shared_ml = ws.casc_ml;
  p.shared_o = ws.casc_o;
  // upper bound of work items from the host hints: every row can be in a
  // tile (only rows of requests with more than one new token are, when the
  // call has no shared prefix), plus the shared-prefix items
  const long long tile_q = kTileM / p.group;
  long long max_items = a.max_query_len > 1
      ? ((static_cast<long long>(a.num_tokens) + tile_q - 1) / tile_q + a.num_reqs) *
            a.num_kv_heads
      : 0;
  if (a.shared_num > 0)
    max_items += (a.shared_num + tile_q - 1) / tile_q * a.shared_pieces * a.num_kv_heads;
  const int grid = static_cast<int>(max_items < num_sms ? max_items : num_sms);
  if (grid <= 0) return cudaSuccess;
  const int sc = !a.scored ? kPlain
                           : kRanges | (a.score.softcap > 0.f ? kCap : 0) |
                                 (a.score.slopes || wide_cap ? kBias : 0);
#define PKV_PREFILL_CASE(D_, SC_) \
  if (a.head_dim == D_ && sc == (SC_)) \
    return launch_prefill_t<D_, (SC_)>(p, kv_map, q_map, grid, stream);
#define PKV_PREFILL_D(D_)                                                    \
  PKV_PREFILL_CASE(D_, kPlain) PKV_PREFILL_CASE(D_, kRanges)                 \
  PKV_PREFILL_CASE(D_, kRanges | kCap) PKV_PREFILL_CASE(D_, kRanges | kBias) \
  PKV_PREFILL_CASE(D_, kRanges | kCap | kBias)
  PKV_PREFILL_D(128) PKV_PREFILL_D(64)
#undef PKV_PREFILL_D
#undef PKV_PREFILL_CASE
  return cudaErrorInvalidValue;
}

cudaError_t read_errors_prefill(uint32_t* out, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_errors_prefill, sizeof(v));
  if (e != cudaSuccess) return e;
  *out |= v;
  if (clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_errors_prefill, &z, sizeof(z));
  }
  return e;
}

}  // namespace pkv
