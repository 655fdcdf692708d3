// The step's block tables, slot map and lengths built on the device from the
// requests' lengths, and the blocks of finished requests given back
// (sm_103a).
//
// Both calls move integers: a few words per request, one table entry per new
// block, one slot per new token. What they cost is latency -- the launch,
// the dependent loads from a request's lengths to its blocks, and the
// barriers between phases -- so each is a single launch of one thread-block
// cluster: its hardware barrier orders the phases, and the free queue's state
// can be read by every CTA before one of them replaces it in place.
//
// Every CTA scans the lengths of all requests for itself (thread i takes the
// run of requests [i * per, (i + 1) * per)), which costs a few loads per
// thread and needs no exchange; the prefix sums of the 1024 runs stay in
// shared memory. Flat indexes (new tokens, new blocks, released entries) are
// then spread evenly over the cluster's threads, each of which finds its
// request by a binary search of the runs and a walk through one run, so that
// one very long prompt is as evenly spread as thousands of decodes.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace pkv {

static __device__ uint32_t g_errors_tables;

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;

// Prefix sums of two counters over the runs of all threads (start[i] = sum
// before run i, start[kTableThreads] = total).
struct RunStarts {
  long long a[kTableThreads + 1], b[kTableThreads + 1];
};

__device__ __forceinline__ void scan_runs(RunStarts& s, long long a, long long b) {
  __shared__ long long warp_a[32], warp_b[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, ia, off);
    const long long ub = __shfl_up_sync(0xffffffffu, ib, off);
    if (lane >= off) {
      ia += ua;
      ib += ub;
    }
  }
  if (lane == 31) {
    warp_a[warp] = ia;
    warp_b[warp] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    const long long wa = warp_a[lane], wb = warp_b[lane];
    long long ja = wa, jb = wb;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long ua = __shfl_up_sync(0xffffffffu, ja, off);
      const long long ub = __shfl_up_sync(0xffffffffu, jb, off);
      if (lane >= off) {
        ja += ua;
        jb += ub;
      }
    }
    warp_a[lane] = ja - wa;
    warp_b[lane] = jb - wb;
    if (lane == 31) {
      s.a[kTableThreads] = ja;
      s.b[kTableThreads] = jb;
    }
  }
  __syncthreads();
  s.a[threadIdx.x] = warp_a[warp] + ia - a;
  s.b[threadIdx.x] = warp_b[warp] + ib - b;
  __syncthreads();
}

// The run that holds flat index x < start[kTableThreads].
__device__ __forceinline__ int run_of(const long long* start, long long x) {
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

__global__ void __launch_bounds__(kTableThreads) build_tables_kernel(const BuildArgs a) {
  __shared__ RunStarts s;
  __shared__ long long taken_s;
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int nctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x;
  const int R = a.num_reqs;
  int head = a.state[0], count = a.state[1];
  const bool state_ok = head >= 0 && head < a.num_blocks && count >= 0 && count <= a.num_blocks;
  const int head_in = head, count_in = count;
  if (!state_ok) head = count = 0;  // nothing to hand out
  uint32_t err = state_ok ? 0u : kErrLengths;

  // ---- every CTA: batch rows and new blocks before each run of requests
  const int per = (R + kTableThreads - 1) / kTableThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  long long rows = 0, need = 0;
  for (int r = r0; r < r1; ++r) {
    const Ask k = ask_of(a, r);
    rows += k.rows;
    need += k.need;
  }
  if (tid == 0) taken_s = 0;
  scan_runs(s, rows, need);
  const long long total_rows = s.a[kTableThreads], total_need = s.b[kTableThreads];
  if (total_rows > a.num_tokens) err |= kErrLengths;

  // ---- requests: starts and lengths, first come, first served. A request is
  // granted its blocks if all that is asked for up to and including it is
  // there; the largest such sum is what leaves the queue.
  {
    long long at = s.a[tid], through = s.b[tid], taken = 0;
    const bool mine = tid % nctas == rank;
    for (int r = r0; r < r1; ++r) {
      const Ask k = ask_of(a, r);
      through += k.need;
      const bool granted = k.need == 0 || through <= count;
      if (through <= count) taken = through;
      if (mine) {
        a.qsl[r] = static_cast<int32_t>(at < 0x7fffffffll ? at : 0x7fffffffll);
        a.seq_lens[r] = k.bad || !granted ? 0 : k.c + k.rows;
        if (k.bad) err |= kErrLengths;
        if (!granted) err |= kErrNoBlocks;
      }
      at += k.rows;
    }
    if (rank == 0) {
      if (tid == 0)
        a.qsl[R] = static_cast<int32_t>(total_rows < 0x7fffffffll ? total_rows : 0x7fffffffll);
      if (taken > 0) atomicMax(&taken_s, taken);
    }
  }

  const long long stride = static_cast<long long>(nctas) * kTableThreads;
  const long long first = static_cast<long long>(rank) * kTableThreads + tid;
  // place x of the queue, counted from its head
  auto popped = [&](long long x) -> int {
    long long i = head + x;
    if (i >= a.num_blocks) i -= a.num_blocks;
    return __ldg(a.queue + i);
  };

  // ---- new blocks: table entries and reference counts
  for (long long x = first; x < total_need; x += stride) {
    const int run = run_of(s.b, x);
    int r = run * per;
    long long before = s.b[run];
    Ask k = ask_of(a, r);
    while (before + k.need <= x && r + 1 < R) {
      before += k.need;
      k = ask_of(a, ++r);
    }
    // (lengths that change under the call must not lead outside the table)
    const long long entry = k.have + (x - before);
    if (entry >= a.max_blocks) continue;
    int id = -1;
    if (before + k.need <= count) {
      id = popped(x);
      if (id < 0 || id >= a.num_blocks) {
        err |= kErrBlockRange;
        id = -1;
      } else if (a.ref_cnt) {
        a.ref_cnt[id] = 1;
      }
    }
    a.block_table[static_cast<long long>(r) * a.max_blocks + entry] = id;
  }

  // ---- new tokens: slots
  if (a.slots) {
    for (long long t = first; t < a.num_tokens; t += stride) {
      long long slot = -1;
      if (t < total_rows) {
        const int run = run_of(s.a, t);
        int r = run * per;
        long long at = s.a[run], before = s.b[run];
        Ask k = ask_of(a, r);
        while (at + k.rows <= t && r + 1 < R) {
          at += k.rows;
          before += k.need;
          k = ask_of(a, ++r);
        }
        if (!k.bad && t - at < k.rows && (k.need == 0 || before + k.need <= count)) {
          const int pos = k.c + static_cast<int>(t - at);
          const int lb = pos >> a.shift;
          const int id = lb < k.have
                             ? a.block_table[static_cast<long long>(r) * a.max_blocks + lb]
                             : popped(before + lb - k.have);
          if (id >= 0 && id < a.num_blocks)
            slot = (static_cast<long long>(id) << a.shift) + (pos & ((1 << a.shift) - 1));
          else
            err |= kErrBlockRange;
        }
      }
      a.slots[t] = slot;
    }
  }
  if (err) atomicOr(&g_errors_tables, err);

  // every CTA has read the state (it may be replaced in place)
  cluster.sync();
  if (rank == 0 && tid == 0) {
    int h = head_in, c = count_in;
    if (state_ok) {
      h = static_cast<int>((head + taken_s) % a.num_blocks);
      c = static_cast<int>(count - taken_s);
    }
    a.state_out[0] = h;
    a.state_out[1] = c;
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

__global__ void __launch_bounds__(kTableThreads) release_blocks_kernel(const ReleaseArgs a) {
  __shared__ RunStarts s;
  __shared__ int counts[32];   // owners per warp
  __shared__ int cta_owners;   // freed blocks of this CTA's segment
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int nctas = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head_in = a.state[0], count_in = a.state[1];
  const bool state_ok =
      head_in >= 0 && head_in < a.num_blocks && count_in >= 0 && count_in <= a.num_blocks;
  uint32_t err = state_ok ? 0u : kErrLengths;

  const int per = (a.num_released + kTableThreads - 1) / kTableThreads;
  const int i0 = min(a.num_released, tid * per), i1 = min(a.num_released, i0 + per);
  long long sum = 0;
  int row;
  for (int i = i0; i < i1; ++i) sum += entries_of(a, i, &row, &err);
  scan_runs(s, sum, 0);
  // a bad state releases nothing
  const int total = state_ok ? static_cast<int>(s.a[kTableThreads]) : 0;

  // this CTA's segment of the flat entries, in whole tiles of the block
  const int tiles = (total + kTableThreads - 1) / kTableThreads;
  const int x0 = static_cast<int>(static_cast<long long>(tiles) * rank / nctas) * kTableThreads;
  const int x1 = min(total, static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / nctas) *
                                kTableThreads);
  // block of flat entry x: rows in the order given, each from its last entry
  auto block_of = [&](int x) -> int {
    const int run = run_of(s.a, x);
    int i = run * per, r;
    uint32_t ignore = 0;
    long long at = s.a[run];
    int e = entries_of(a, i, &r, &ignore);
    while (at + e <= x && i + 1 < a.num_released) {
      at += e;
      e = entries_of(a, ++i, &r, &ignore);
    }
    // (lengths that change under the call must not lead outside the table)
    if (x - at >= e) return -1;
    return __ldg(a.block_table + static_cast<long long>(r) * a.max_blocks +
                 (e - 1 - static_cast<int>(x - at)));
  };
  auto in_pool = [&](int b) { return b >= 0 && b < a.num_blocks; };

  // ---- count down; the release that reaches zero marks the block. One too
  // many is undone and flagged (sums commute, so the marks do not depend on
  // the order of the releases).
  for (int x = x0 + tid; x < x1; x += kTableThreads) {
    const int b = block_of(x);
    if (!in_pool(b)) {
      err |= kErrBlockRange;
      continue;
    }
    const int old = atomicSub(a.ref_cnt + b, 1);
    if (old == 1) {
      atomicAdd(a.ref_cnt + b, kFreed);
    } else if (old <= 0) {
      atomicAdd(a.ref_cnt + b, 1);
      err |= kErrRefCount;
    }
  }
  cluster.sync();
  // ---- a freed block's place is its last release's
  for (int x = x0 + tid; x < x1; x += kTableThreads) {
    const int b = block_of(x);
    if (in_pool(b) && __ldcg(a.ref_cnt + b) < kFreedTop) atomicMax(a.ref_cnt + b, kFreed + 1 + x);
  }
  cluster.sync();
  auto owner = [&](int x, int* b) -> bool {
    if (x >= x1) return false;
    *b = block_of(x);
    return in_pool(*b) && __ldcg(a.ref_cnt + *b) == kFreed + 1 + x;
  };
  // ---- freed blocks of the segment, then of the segments before it
  int mine = 0, b = 0;
  for (int x = x0; x < x1; x += kTableThreads) mine += owner(x + tid, &b);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) counts[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int n = __reduce_add_sync(0xffffffffu, counts[lane]);
    if (lane == 0) cta_owners = n;
  }
  cluster.sync();
  int before = 0, all = 0;
  for (int k = 0; k < nctas; ++k) {
    const int n = *cluster.map_shared_rank(&cta_owners, k);
    if (k < rank) before += n;
    all += n;
  }
  // ---- append in order
  for (int x = x0; x < x1; x += kTableThreads) {
    const bool own = owner(x + tid, &b);
    const unsigned m = __ballot_sync(0xffffffffu, own);
    __syncthreads();
    if (lane == 0) counts[warp] = __popc(m);
    __syncthreads();
    int upto = 0, tile = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) upto += counts[w];
      tile += counts[w];
    }
    if (own) {
      const long long place = static_cast<long long>(count_in) + before + upto +
                              __popc(m & ((1u << lane) - 1u));
      a.ref_cnt[b] = 0;
      if (place < a.num_blocks) {
        long long q = head_in + place;
        if (q >= a.num_blocks) q -= a.num_blocks;
        a.queue[q] = b;
      } else {
        err |= kErrRefCount;  // more blocks than the pool has: the state was wrong
      }
    }
    before += tile;
  }
  if (err) atomicOr(&g_errors_tables, err);
  // no CTA leaves while another reads its count
  cluster.sync();
  if (rank == 0 && tid == 0) {
    a.state_out[0] = head_in;
    a.state_out[1] = state_ok ? min(count_in + all, a.num_blocks) : count_in;
  }
}

// ------------------------------------------------------------------ host
// CTAs of the cluster: one per kEntriesPerCta flat entries (one CTA needs no
// cluster barrier), at most the portable size.
constexpr long long kEntriesPerCta = 2048;

static int cluster_ctas(long long entries) {
  int n = 1;
  while (n < 8 && entries > n * kEntriesPerCta) n *= 2;
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
                                int32_t* ref_cnt, int num_blocks, int block_size,
                                cudaStream_t stream) {
  const BuildArgs a{block_table, max_blocks, qsl,   seq_lens,  slots,   num_computed,
                    query_lens,  num_reqs,   num_tokens, queue, state, state_out,
                    ref_cnt,     num_blocks,
                    static_cast<int>(__builtin_ctz(static_cast<unsigned>(block_size)))};
  return launch_cluster(build_tables_kernel,
                        cluster_ctas(num_tokens > num_reqs ? num_tokens : num_reqs), stream, a);
}

cudaError_t launch_release_blocks(const int32_t* block_table, int max_blocks, int num_reqs,
                                  const int32_t* rows, const int32_t* tokens, int num_released,
                                  int32_t* queue, const int32_t* state, int32_t* state_out,
                                  int32_t* ref_cnt, int num_blocks, int block_size,
                                  cudaStream_t stream) {
  const ReleaseArgs a{block_table, max_blocks, num_reqs, rows,    tokens,     num_released,
                      queue,       state,      state_out, ref_cnt, num_blocks,
                      static_cast<int>(__builtin_ctz(static_cast<unsigned>(block_size)))};
  return launch_cluster(release_blocks_kernel,
                        cluster_ctas(static_cast<long long>(num_released) * max_blocks), stream, a);
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
