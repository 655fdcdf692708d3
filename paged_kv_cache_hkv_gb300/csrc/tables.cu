// The step's block tables, slot map and lengths built on the device from the
// requests' lengths, and the blocks of finished requests given back
// (sm_103a).
//
// Both calls move integers: a few words per request, one table entry per new
// block, one slot per new token. What they cost is latency -- the launches,
// the dependent loads from a request's lengths to its blocks, and the
// barriers between phases -- and, where thousands of requests are released,
// the rate at which an SM issues scattered atomics.
//
// Every CTA scans the lengths of all requests for itself (thread i takes the
// run of requests [i * per, (i + 1) * per)), which costs a few loads per
// thread and needs no exchange; the prefix sums of the 1024 runs stay in
// shared memory. Work is then spread over the grid by flat indexes (new tokens
// of long requests, released entries): whoever gets a place of one finds its
// request by a binary search of the runs and a walk through one run. One very
// long prompt is so spread as evenly as thousands of decodes. What is not even:
// the build's warps take 128 tokens of long requests in a row and find the first
// one's request only, so a warp whose tokens end one long request and begin the
// next walks over every request that stands between the two in the batch. With
// 4000 decodes there a step takes 597 us that takes 9.7 with the prompts in front.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace pkv {

static __device__ uint32_t g_errors_tables;

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;

// Exclusive prefix sums of N counters over the block's threads: start[c][i] =
// sum of counter c before thread i, start[c][kTableThreads] = total.
template <typename T, int N>
struct RunStarts {
  T start[N][kTableThreads + 1];
  T warp_sum[N][32];
};

template <typename T, int N>
__device__ __forceinline__ void scan_runs(RunStarts<T, N>& s, const T (&v)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc[N];
#pragma unroll
  for (int c = 0; c < N; ++c) inc[c] = v[c];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const T u = __shfl_up_sync(0xffffffffu, inc[c], off);
      if (lane >= off) inc[c] += u;
    }
  if (lane == 31)
#pragma unroll
    for (int c = 0; c < N; ++c) s.warp_sum[c][warp] = inc[c];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const T w = s.warp_sum[c][lane];
      T j = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, j, off);
        if (lane >= off) j += u;
      }
      s.warp_sum[c][lane] = j - w;
      if (lane == 31) s.start[c][kTableThreads] = j;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < N; ++c) s.start[c][threadIdx.x] = s.warp_sum[c][warp] + inc[c] - v[c];
  __syncthreads();
}

// The last run that starts at or before x.
template <typename T>
__device__ __forceinline__ int run_of(const T* start, T x) {
  int lo = 0;
#pragma unroll
  for (int step = kTableThreads / 2; step >= 1; step >>= 1)
    if (start[lo + step] <= x) lo += step;
  return lo;
}

// ------------------------------------------------------------------ build
struct BuildArgs {
  int32_t* block_table;
  int max_blocks;
  int32_t* qsl;
  int32_t* seq_lens;
  int64_t* slots;  // may be null
  const int32_t* num_computed;
  const int32_t* query_lens;
  int num_reqs, num_tokens;
  const int32_t* queue;
  const int32_t* state;
  int32_t* state_out;
  int32_t* ref_cnt;
  int num_blocks, shift;
};

// What a request asks for: batch rows, blocks held, new blocks.
struct Ask {
  int rows, c, have, need;
  bool bad;  // inconsistent lengths: keeps its rows, gets nothing
};

__device__ __forceinline__ Ask ask_of(const BuildArgs& a, int r) {
  const int n = __ldg(a.query_lens + r), c = __ldg(a.num_computed + r);
  const long long B = 1ll << a.shift;
  Ask k{max(n, 0), c, 0, 0, false};
  const long long end = static_cast<long long>(c) + n;
  k.bad = n < 0 || c < 0 || end > 0x7fffffffll ||
          end > (static_cast<long long>(a.max_blocks) << a.shift);
  if (!k.bad) {
    k.have = static_cast<int>((c + B - 1) >> a.shift);
    k.need = static_cast<int>((static_cast<long long>(c) + n + B - 1) >> a.shift) - k.have;
  }
  return k;
}

// Requests of more new tokens than this are spread over warps, token by
// token; the others are done by one thread each (a decode is one token). 512
// requests of 8 tokens take 5.8 us so and 10.3 spread (limit 2); 512 of 32 take 7.9
// spread and 15.3 by one thread each (limit 32). kChunkRows: 4096 requests with
// 102,000 new tokens take 9.7 us with 128, 17.3 with 512 and 7.5 with 32.
constexpr int kShortRows = 8;
constexpr int kChunkRows = 128;  // consecutive tokens of long requests per warp and turn

// The state of the queue after the step: what leaves it is the largest sum of
// asks that it covers. One thread, with the sums before each run of requests.
__device__ __forceinline__ void write_state(const BuildArgs& a, const long long* need_start, int per,
                                            int head, int count, bool state_ok) {
  int h = head, c = count;
  if (state_ok) {
    const long long n = count;
    const int run = run_of(need_start, n);
    long long taken = need_start[run];
    for (int r = run * per; r < min(a.num_reqs, (run + 1) * per); ++r) {
      const long long through = taken + ask_of(a, r).need;
      if (through > n) break;
      taken = through;
    }
    h = static_cast<int>((head + taken) % a.num_blocks);
    c = static_cast<int>(n - taken);
  }
  a.state_out[0] = h;
  a.state_out[1] = c;
}

__device__ __forceinline__ bool state_valid(int head, int count, int num_blocks) {
  return head >= 0 && head < num_blocks && count >= 0 && count <= num_blocks;
}

__global__ void __launch_bounds__(kTableThreads) build_tables_kernel(const BuildArgs a,
                                                                     const bool state_here) {
  __shared__ RunStarts<long long, 3> s;  // batch rows, new blocks, rows of long requests
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int R = a.num_reqs;
  const int head_in = a.state[0], count_in = a.state[1];
  const bool state_ok = state_valid(head_in, count_in, a.num_blocks);
  const int head = state_ok ? head_in : 0, count = state_ok ? count_in : 0;  // bad: nothing to hand out
  uint32_t err = state_ok ? 0u : kErrLengths;

  // rows of a request in the flat index of long requests. Lengths out of
  // range can be anything: no more than the batch's rows are looked at.
  auto long_rows = [&](const Ask& k) -> int {
    return k.rows <= kShortRows ? 0 : k.bad ? min(k.rows, a.num_tokens) : k.rows;
  };

  // ---- every CTA: the sums before each run of requests
  const int per = (R + kTableThreads - 1) / kTableThreads;
  {
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long sum[3] = {0, 0, 0};
    for (int r = r0; r < r1; ++r) {
      const Ask k = ask_of(a, r);
      sum[0] += k.rows;
      sum[1] += k.need;
      sum[2] += long_rows(k);
    }
    scan_runs(s, sum);
  }
  const long long total_rows = s.start[0][kTableThreads], total_long = s.start[2][kTableThreads];
  if (total_rows > a.num_tokens) err |= kErrLengths;

  // place x of the queue, counted from its head, if it is a block of the pool
  auto popped = [&](long long x) -> int {
    long long i = head + x;
    if (i >= a.num_blocks) i -= a.num_blocks;
    const int id = __ldg(a.queue + i);
    if (id >= 0 && id < a.num_blocks) return id;
    err |= kErrBlockRange;
    return -1;
  };
  // The i-th new token of request r (its first row `at`, `before` new blocks
  // asked for by earlier requests): its slot, and, where it is the first
  // token of a new block, the block's table entry and count. First come,
  // first served: a request is granted its blocks if all that is asked for up
  // to and including it is there.
  auto token = [&](int r, const Ask& k, long long at, long long before, int i) {
    const bool granted = k.need == 0 || before + k.need <= count;
    long long slot = -1;
    if (!k.bad) {
      const int pos = k.c + i, lb = pos >> a.shift, off = pos & ((1 << a.shift) - 1);
      int32_t* entry = a.block_table + static_cast<long long>(r) * a.max_blocks + lb;
      int id = -1;
      if (lb < k.have)
        id = granted ? *entry : -1;
      else if (granted)
        id = popped(before + lb - k.have);
      if (lb >= k.have && off == 0) {
        *entry = id;
        if (id >= 0 && a.ref_cnt) a.ref_cnt[id] = 1;
      }
      if (id >= 0 && id < a.num_blocks)
        slot = (static_cast<long long>(id) << a.shift) + off;
      else if (granted)
        err |= kErrBlockRange;
    }
    if (a.slots && at + i < a.num_tokens) a.slots[at + i] = slot;
  };

  const long long first = static_cast<long long>(blockIdx.x) * kTableThreads + tid;
  const long long stride = static_cast<long long>(gridDim.x) * kTableThreads;

  // ---- a thread per request: start, length, and a short request's tokens
  for (long long x = first; x < R; x += stride) {
    const int r = static_cast<int>(x), run = r / per;
    long long at = s.start[0][run], before = s.start[1][run];
    for (int j = run * per; j < r; ++j) {
      const Ask k = ask_of(a, j);
      at += k.rows;
      before += k.need;
    }
    const Ask k = ask_of(a, r);
    const bool granted = k.need == 0 || before + k.need <= count;
    a.qsl[r] = static_cast<int32_t>(at < 0x7fffffffll ? at : 0x7fffffffll);
    a.seq_lens[r] = k.bad || !granted ? 0 : k.c + k.rows;
    if (k.bad) err |= kErrLengths;
    if (!granted) err |= kErrNoBlocks;
    if (k.rows <= kShortRows)
      for (int i = 0; i < k.rows; ++i) token(r, k, at, before, i);
  }

  // ---- long requests: a warp takes kChunkRows tokens in a row. Its lanes
  // start from the request of the first of them and walk on.
  const long long warps = stride / 32;
  for (long long x0 = first / 32 * kChunkRows; x0 < total_long; x0 += warps * kChunkRows) {
    const int run = run_of(s.start[2], x0);
    int r = run * per;
    long long at = s.start[0][run], before = s.start[1][run], flat = s.start[2][run];
    Ask k = ask_of(a, r);
    for (int i = lane; i < kChunkRows && x0 + i < total_long; i += 32) {
      // (lengths that change under the call must not lead past the last request)
      while (flat + long_rows(k) <= x0 + i && r + 1 < R) {
        at += k.rows;
        before += k.need;
        flat += long_rows(k);
        k = ask_of(a, ++r);
      }
      const long long in = x0 + i - flat;
      if (in < k.rows) token(r, k, at, before, static_cast<int>(in));
    }
  }

  // ---- rows behind the last request
  if (a.slots)
    for (long long t = total_rows + first; t < a.num_tokens; t += stride) a.slots[t] = -1;
  if (err) atomicOr(&g_errors_tables, err);

  if (blockIdx.x == 0 && tid == 0) {
    a.qsl[R] = static_cast<int32_t>(total_rows < 0x7fffffffll ? total_rows : 0x7fffffffll);
    if (state_here) write_state(a, s.start[1], per, head_in, count_in, state_ok);
  }
}

// The queue's state replaced in place, after every CTA of the build has read it.
__global__ void __launch_bounds__(kTableThreads) commit_state_kernel(const BuildArgs a) {
  __shared__ RunStarts<long long, 1> s;
  pdl_trigger();
  pdl_wait();
  const int per = (a.num_reqs + kTableThreads - 1) / kTableThreads;
  const int r0 = min(a.num_reqs, static_cast<int>(threadIdx.x) * per), r1 = min(a.num_reqs, r0 + per);
  long long need[1] = {0};
  for (int r = r0; r < r1; ++r) need[0] += ask_of(a, r).need;
  scan_runs(s, need);
  if (threadIdx.x == 0) {
    const int head = a.state[0], count = a.state[1];
    write_state(a, s.start[0], per, head, count, state_valid(head, count, a.num_blocks));
  }
}

// ------------------------------------------------------------------ release
struct ReleaseArgs {
  const int32_t* block_table;
  int max_blocks, num_reqs;
  const int32_t* rows;
  const int32_t* tokens;
  int num_released;
  int32_t* queue;
  const int32_t* state;
  int32_t* state_out;
  int32_t* ref_cnt;
  int num_blocks, shift;
  // large releases: which flat entries free a block (a bit each), how many do
  // in each tile of kTableThreads, and the queue's state before the call
  uint32_t* bits;
  int32_t* tile_freed;
  int32_t* state_copy;
};

// Reference counts double as the scratch that finds each freed block's place.
// While the call runs, a block whose count has reached zero holds kFreed plus
// 1 + the largest flat index at which it was released (its last holder).
// Counts of blocks in use are positive and never come near.
constexpr int kFreed = -(1 << 30);
constexpr int kFreedTop = -(1 << 29);  // flat indexes stay below 2^29

// Entries of the i-th released row, 0 if the row or its length is out of range.
__device__ __forceinline__ int entries_of(const ReleaseArgs& a, int i, int* row, uint32_t* err) {
  const int r = __ldg(a.rows + i);
  *row = r;
  if (r < 0 || r >= a.num_reqs) {
    *err |= kErrLengths;
    return 0;
  }
  const long long n = __ldg(a.tokens + r);
  const long long e = (n + (1 << a.shift) - 1) >> a.shift;
  if (n < 0 || e > a.max_blocks) {
    *err |= kErrLengths;
    return 0;
  }
  return static_cast<int>(e);
}

// The released entries as a flat index, the sums before each run of rows in
// shared memory.
struct ReleaseRuns {
  RunStarts<int, 1> s;
  int row[kTableThreads], entries[kTableThreads];  // of runs of one row
};

__device__ __forceinline__ int release_per(const ReleaseArgs& a) {
  return (a.num_released + kTableThreads - 1) / kTableThreads;
}

// Fills the runs; returns the number of entries (0 under a bad state).
__device__ __forceinline__ int scan_runs_released(const ReleaseArgs& a, ReleaseRuns& v,
                                                  uint32_t* err, bool state_ok) {
  const int per = release_per(a), tid = threadIdx.x;
  const int i0 = min(a.num_released, tid * per), i1 = min(a.num_released, i0 + per);
  int sum[1] = {0}, row = 0, e = 0;
  for (int i = i0; i < i1; ++i) {
    e = entries_of(a, i, &row, err);
    sum[0] += e;
  }
  v.row[tid] = row;
  v.entries[tid] = e;
  scan_runs(v.s, sum);
  if (state_ok) return v.s.start[0][kTableThreads];
  *err |= kErrLengths;
  return 0;
}
__device__ __forceinline__ int scan_released(const ReleaseArgs& a, ReleaseRuns& v, uint32_t* err) {
  return scan_runs_released(a, v, err, state_valid(a.state[0], a.state[1], a.num_blocks));
}

// Block of flat entry x (rows in the order given, each from its last entry),
// -1 if it is out of the pool.
__device__ __forceinline__ int block_of(const ReleaseArgs& a, const ReleaseRuns& v, int x) {
  const int* start = v.s.start[0];
  const int run = run_of(start, x), per = release_per(a);
  int at = start[run], r = v.row[run], e = v.entries[run];
  if (per > 1) {
    int i = run * per;
    uint32_t ignore = 0;
    e = entries_of(a, i, &r, &ignore);
    while (at + e <= x && i + 1 < a.num_released) {
      at += e;
      e = entries_of(a, ++i, &r, &ignore);
    }
  }
  // (lengths that change under the call must not lead outside the table)
  if (x - at >= e) return -1;
  const int b = __ldg(a.block_table + static_cast<long long>(r) * a.max_blocks + (e - 1 - (x - at)));
  return b >= 0 && b < a.num_blocks ? b : -1;
}

// Count block b down; the release that reaches zero marks it. One too many is
// undone and flagged (sums commute, so the marks do not depend on the order
// of the releases).
__device__ __forceinline__ void count_down(const ReleaseArgs& a, int b, uint32_t* err) {
  const int old = atomicSub(a.ref_cnt + b, 1);
  if (old == 1) {
    atomicAdd(a.ref_cnt + b, kFreed);
  } else if (old <= 0) {
    atomicAdd(a.ref_cnt + b, 1);
    *err |= kErrRefCount;
  }
}

// A freed block's place is its last release's.
__device__ __forceinline__ void claim_place(const ReleaseArgs& a, int b, int x) {
  if (__ldcg(a.ref_cnt + b) < kFreedTop) atomicMax(a.ref_cnt + b, kFreed + 1 + x);
}

// Block b to its place, counted from the queue's head.
__device__ __forceinline__ void append_block(const ReleaseArgs& a, int b, int head, long long place,
                                             uint32_t* err) {
  if (b < 0) return;
  a.ref_cnt[b] = 0;
  if (place >= a.num_blocks) {
    *err |= kErrRefCount;  // more blocks than the pool has: the state was wrong
    return;
  }
  long long q = head + place;
  if (q >= a.num_blocks) q -= a.num_blocks;
  a.queue[q] = b;
}

// Large releases run over the whole device, a launch per phase: what bounds
// them is the rate of scattered accesses per SM (1024 rows of 160 blocks took
// 54 us with the last phase, and 90 with all of them, in one cluster of 8).
__global__ void __launch_bounds__(kTableThreads) release_count_kernel(const ReleaseArgs a) {
  __shared__ ReleaseRuns v;
  pdl_trigger();
  pdl_wait();
  uint32_t err = 0;
  const int total = scan_released(a, v, &err);
  for (long long x = static_cast<long long>(blockIdx.x) * kTableThreads + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * kTableThreads) {
    const int b = block_of(a, v, static_cast<int>(x));
    if (b >= 0)
      count_down(a, b, &err);
    else
      err |= kErrBlockRange;
  }
  if (err) atomicOr(&g_errors_tables, err);
}

__global__ void __launch_bounds__(kTableThreads) release_claim_kernel(const ReleaseArgs a) {
  __shared__ ReleaseRuns v;
  pdl_trigger();
  pdl_wait();
  uint32_t err = 0;
  const int total = scan_released(a, v, &err);
  for (long long x = static_cast<long long>(blockIdx.x) * kTableThreads + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * kTableThreads) {
    const int b = block_of(a, v, static_cast<int>(x));
    if (b >= 0) claim_place(a, b, static_cast<int>(x));
  }
}

// Which entries free a block: every claim is in.
__global__ void __launch_bounds__(kTableThreads) release_flag_kernel(const ReleaseArgs a) {
  __shared__ ReleaseRuns v;
  pdl_trigger();
  pdl_wait();
  uint32_t err = 0;
  const int total = scan_released(a, v, &err);
  if (blockIdx.x == 0 && threadIdx.x < 2) a.state_copy[threadIdx.x] = a.state[threadIdx.x];
  const int tiles = (total + kTableThreads - 1) / kTableThreads;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int x = t * kTableThreads + threadIdx.x;
    const int b = x < total ? block_of(a, v, x) : -1;
    const bool own = b >= 0 && __ldcg(a.ref_cnt + b) == kFreed + 1 + x;
    const uint32_t m = __ballot_sync(0xffffffffu, own);
    if ((threadIdx.x & 31) == 0) a.bits[x >> 5] = m;
    const int n = __syncthreads_count(own);
    if (threadIdx.x == 0) a.tile_freed[t] = n;
  }
}

// Freed blocks to their places behind the queue's tail, counts back to zero.
__global__ void __launch_bounds__(kTableThreads) release_append_kernel(const ReleaseArgs a) {
  __shared__ ReleaseRuns v;
  __shared__ int warp_n[32], before_s, all_s;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t err = 0;
  const int head = a.state_copy[0], count = a.state_copy[1];
  const bool state_ok = state_valid(head, count, a.num_blocks);
  // (the state itself may be replaced by now: only the copy counts)
  const int total = scan_runs_released(a, v, &err, state_ok);
  const int tiles = (total + kTableThreads - 1) / kTableThreads;
  // this CTA's tiles in a row; freed blocks before them, and in all
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * blockIdx.x / gridDim.x);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (blockIdx.x + 1) / gridDim.x);
  if (tid == 0) before_s = all_s = 0;
  __syncthreads();
  int sum = 0, upto = 0;
  for (int t = tid; t < tiles; t += kTableThreads) {
    const int n = __ldcg(a.tile_freed + t);
    sum += n;
    if (t < t0) upto += n;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  upto = __reduce_add_sync(0xffffffffu, upto);
  if (lane == 0 && sum) atomicAdd(&all_s, sum);
  if (lane == 0 && upto) atomicAdd(&before_s, upto);
  __syncthreads();
  long long place0 = static_cast<long long>(count) + before_s;
  for (int t = t0; t < t1; ++t) {
    const int x = t * kTableThreads + tid;
    const uint32_t m = __ldcg(a.bits + (x >> 5));
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    const int c = warp_n[lane];
    const int below = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
    const int tile = __reduce_add_sync(0xffffffffu, c);
    if (m >> lane & 1u) {
      append_block(a, block_of(a, v, x), head, place0 + below + __popc(m & ((1u << lane) - 1u)), &err);
    }
    place0 += tile;
    __syncthreads();
  }
  if (err) atomicOr(&g_errors_tables, err);
  if (blockIdx.x == 0 && tid == 0) {
    a.state_out[0] = head;
    a.state_out[1] = state_ok ? min(count + all_s, a.num_blocks) : count;
  }
}

// Small releases in one launch of one cluster, its barrier between the
// phases: up to kSmallEntries entries, kPerThread per thread of the largest
// portable cluster. Their block ids stay in shared memory from the first phase
// on. 8 rows of some 245 entries take 11.1 us so (2.4 of it the measurement's
// copy of the counts) and 14.9 in four launches; at 64 rows of 250 the two are
// even (15.4 us), and a third entry per thread would gain nothing (64 rows of
// 260: 15.7 in one launch, 15.5 in four).
constexpr int kMaxCtas = 8;
constexpr int kPerThread = 2;
constexpr int kShare = kPerThread * kTableThreads;
constexpr int kSmallEntries = kMaxCtas * kShare;

__global__ void __launch_bounds__(kTableThreads) release_small_kernel(const ReleaseArgs a) {
  __shared__ int32_t stash[kShare];
  __shared__ ReleaseRuns v;
  __shared__ int tile_scan[32];
  __shared__ int cta_freed;  // freed blocks of this CTA's share
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int nctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head_in = a.state[0], count_in = a.state[1];
  const bool state_ok = state_valid(head_in, count_in, a.num_blocks);
  uint32_t err = 0;
  const int total = scan_runs_released(a, v, &err, state_ok);

  // this CTA's share of the flat entries, in whole tiles of the block (at most
  // kPerThread: total <= kSmallEntries, and less than a full cluster is launched
  // only for one tile per CTA); entry x0 + n is thread n % kTableThreads's
  const int tiles = (total + kTableThreads - 1) / kTableThreads;
  const int x0 = static_cast<int>(static_cast<long long>(tiles) * rank / nctas) * kTableThreads;
  const int x1 = min(total, static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / nctas) *
                                kTableThreads);
  const int share = max(0, x1 - x0);

  int ids[kPerThread];  // the loads of a thread's entries go out together
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const int n = tid + u * kTableThreads;
    ids[u] = -1;
    if (n < share) {
      ids[u] = block_of(a, v, x0 + n);
      if (ids[u] < 0) err |= kErrBlockRange;
      stash[n] = ids[u];
    }
  }
#pragma unroll
  for (int u = 0; u < kPerThread; ++u)
    if (ids[u] >= 0) count_down(a, ids[u], &err);
  cluster.sync();
  for (int n = tid; n < share; n += kTableThreads)
    if (stash[n] >= 0) claim_place(a, stash[n], x0 + n);
  cluster.sync();
  // ---- how many places this share fills; the stash keeps only their blocks
  int mine = 0;
  for (int n = tid; n < share; n += kTableThreads) {
    const int b = stash[n];
    const bool own = b >= 0 && __ldcg(a.ref_cnt + b) == kFreed + 1 + x0 + n;
    mine += own;
    if (!own) stash[n] = -1;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) tile_scan[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int n = __reduce_add_sync(0xffffffffu, tile_scan[lane]);
    if (lane == 0) cta_freed = n;
  }
  cluster.sync();
  int before = 0, all = 0;
  for (int k = 0; k < nctas; ++k) {
    const int n = *cluster.map_shared_rank(&cta_freed, k);
    if (k < rank) before += n;
    all += n;
  }
  // ---- append in order, a tile at a time
  long long place0 = static_cast<long long>(count_in) + before;
  for (int n0 = 0; n0 < share; n0 += kTableThreads) {
    const int n = n0 + tid;
    const int b = n < share ? stash[n] : -1;
    const unsigned m = __ballot_sync(0xffffffffu, b >= 0);
    __syncthreads();
    if (lane == 0) tile_scan[warp] = __popc(m);
    __syncthreads();
    const int c = tile_scan[lane];
    const int below = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
    const int tile = __reduce_add_sync(0xffffffffu, c);
    if (b >= 0) append_block(a, b, head_in, place0 + below + __popc(m & ((1u << lane) - 1u)), &err);
    place0 += tile;
  }
  if (err) atomicOr(&g_errors_tables, err);
  // no CTA leaves while another reads its count; all have read the state
  cluster.sync();
  if (rank == 0 && tid == 0) {
    a.state_out[0] = head_in;
    a.state_out[1] = state_ok ? min(count_in + all, a.num_blocks) : count_in;
  }
}

// ------------------------------------------------------------------ host
// CTAs of the cluster: a power of two, one for each kTableThreads flat entries
// (one CTA needs no barrier between CTAs) up to kMaxCtas.
static int cluster_ctas(long long entries) {
  int n = 1;
  while (n < kMaxCtas && entries > static_cast<long long>(n) * kTableThreads) n *= 2;
  return n;
}

template <typename Args>
static cudaError_t launch_cluster(void (*kern)(Args), int ctas, cudaStream_t stream,
                                  const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTableThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args);
}

cudaError_t launch_build_tables(int32_t* block_table, int max_blocks, int32_t* qsl,
                                int32_t* seq_lens, int64_t* slots, const int32_t* num_computed,
                                const int32_t* query_lens, int num_reqs, int num_tokens,
                                const int32_t* queue, const int32_t* state, int32_t* state_out,
                                int32_t* ref_cnt, int num_blocks, int block_size, int num_sms,
                                cudaStream_t stream) {
  const BuildArgs a{block_table, max_blocks, qsl,   seq_lens,  slots,   num_computed,
                    query_lens,  num_reqs,   num_tokens, queue, state, state_out,
                    ref_cnt,     num_blocks,
                    static_cast<int>(__builtin_ctz(static_cast<unsigned>(block_size)))};
  // a CTA per 1024 requests or tokens, at most one per SM. The state is
  // replaced by the build itself unless that would be in place with other
  // CTAs still to read it.
  const long long work = num_tokens > num_reqs ? num_tokens : num_reqs;
  const long long want = (work + kTableThreads - 1) / kTableThreads;
  const int grid = static_cast<int>(want < 1 ? 1 : want < num_sms ? want : num_sms);
  const bool apart = state_out + 2 <= state || state + 2 <= state_out;
  const bool state_here = grid == 1 || apart;
  cudaError_t e = launch_pdl(build_tables_kernel, dim3(grid), dim3(kTableThreads), 0, stream, a,
                             state_here);
  if (e != cudaSuccess || state_here) return e;
  return launch_pdl(commit_state_kernel, dim3(1), dim3(kTableThreads), 0, stream, a);
}

cudaError_t launch_release_blocks(const int32_t* block_table, int max_blocks, int num_reqs,
                                  const int32_t* rows, const int32_t* tokens, int num_released,
                                  int32_t* queue, const int32_t* state, int32_t* state_out,
                                  int32_t* ref_cnt, int num_blocks, int block_size,
                                  void* workspace, int num_sms, cudaStream_t stream) {
  ReleaseArgs a{block_table, max_blocks, num_reqs,  rows,    tokens,     num_released,
                queue,       state,      state_out, ref_cnt, num_blocks,
                static_cast<int>(__builtin_ctz(static_cast<unsigned>(block_size))),
                nullptr,     nullptr,    nullptr};
  const long long bound = static_cast<long long>(num_released) * max_blocks;
  // (rows x table width, an upper bound: the lengths are on the device)
  if (bound <= kSmallEntries)
    return launch_cluster(release_small_kernel, cluster_ctas(bound), stream, a);
  char* ws = static_cast<char*>(workspace);
  const long long tiles = (bound + kTableThreads - 1) / kTableThreads;
  a.state_copy = reinterpret_cast<int32_t*>(ws);
  a.tile_freed = reinterpret_cast<int32_t*>(ws + 256);
  a.bits = reinterpret_cast<uint32_t*>(ws + 256 + (tiles * 4 + 255) / 256 * 256);
  const dim3 grid(static_cast<unsigned>(tiles < num_sms ? tiles : num_sms)), block(kTableThreads);
  cudaError_t e = launch_pdl(release_count_kernel, grid, block, 0, stream, a);
  if (e == cudaSuccess) e = launch_pdl(release_claim_kernel, grid, block, 0, stream, a);
  if (e == cudaSuccess) e = launch_pdl(release_flag_kernel, grid, block, 0, stream, a);
  if (e == cudaSuccess) e = launch_pdl(release_append_kernel, grid, block, 0, stream, a);
  return e;
}

size_t release_workspace_bytes(int num_released, int max_blocks) {
  const long long bound = static_cast<long long>(num_released) * max_blocks;
  if (bound <= kSmallEntries) return 0;
  const long long tiles = (bound + kTableThreads - 1) / kTableThreads;
  return static_cast<size_t>(256 + (tiles * 4 + 255) / 256 * 256 + tiles * (kTableThreads / 8));
}

cudaError_t read_errors_tables(uint32_t* out, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_errors_tables, sizeof(v));
  if (e != cudaSuccess) return e;
  *out |= v;
  if (clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_errors_tables, &z, sizeof(z));
  }
  return e;
}

}  // namespace pkv
