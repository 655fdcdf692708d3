// Split-KV decode over the 8-bit pool (sm_103a): requests of one new token, and
// of a few (guessed tokens that are checked at once), over e4m3 codes with a
// power-of-two scale per row (quant.cuh).
//
// The work split is the bf16 decode's (decode.cu): the step's decode stream of
// (request, 16-key chunk) positions is cut into C equal ranges, a CTA streams its
// range's chunks through a ring of shared-memory stages that a producer warp
// fills by TMA, and what a range boundary cuts leaves partials for the combine
// kernel.
//
// The math is on the tensor cores, for half the bytes a key leaves half the time:
// the bf16 decode's FMAs take 40% of the issue slots at 7 TB/s, and twice the keys
// a second plus their conversion would be over all of them. A consumer warp holds
// MT tiles of 8 units (query row x q head) of one kv head, all in mma.m16n8k16
// with f16 operands:
//   S^T [16 keys x 8 units] = K Q^T: codes become f16 by one conversion per two
//     (exact); a thread's four bytes of a key are its two pairs of a K step, so the
//     dims need no reordering but q's, which is loaded that way. q 2^-e, e as for
//     a row of the pool, is an f16 but for what lies below 2^-32 of the row's
//     largest. The scores are S 2^e times the key's scale.
//   O^T [16 dims x 8 units] += V^T P^T: ldmatrix.trans hands a thread two keys'
//     bytes of two neighbouring dims, the even and odd rows of a V^T tile. P^T is
//     S^T's registers through movmatrix.
// V's scales 2^v go into the exponent of P: weight 2^(s + v - M), M the running
// maximum of s + v, in f16 (11 bits; below 2^-14 of the largest weight 2^-25 of
// it: seen in dims that a V row far larger than the others leaves small). The sum
// of weights keeps a running maximum of s of its own, so that rows of tiny or huge
// V change nothing in it, and O is scaled to it at the end.
// (mma.m16n8k32 on the codes themselves is no shortcut: by the counters each becomes
// conversions of both operands and f16 products, 427 instructions a chunk and warp
// instead of 332, and 244 us instead of 207 on 8 decodes of 32767-131071 keys,
// 32 q and 8 kv heads, D = 128, which the copies alone take 200 for.)
// K, V and the scales of a chunk are a copy or two each: a 4-D box lands them as
// [K|V][kv head][16 keys][D], swizzled, so that ldmatrix finds no bank conflict.
#include <cfloat>
#include <mutex>
#include <vector>

#include "decode.cuh"
#include "quant.cuh"

namespace pkv {

static __device__ uint32_t g_errors_quant_decode;

constexpr int kQuantWarps = 8;  // consumer warps of a CTA at most

// Warps of a CTA of nw consumers with mt unit tiles each. One tile: the consumers
// and the producer. Several: three groups of four warps, of which the last holds the
// producer and hands registers to the others: 4 x 32 x 56 + 8 x 32 x 224 are the
// launch's 12 x 32 x 168. (Nine warps have 168 each, three of them sharing one of the SM's
// four register files: with three tiles 107 us instead of 78 for 64 requests of five
// tokens over 511-4095 keys, 32 q and 8 kv heads, D = 128.)
__host__ __device__ constexpr int quant_threads(int nw, int mt) {
  return mt == 1 ? (nw + 1) * 32 : 12 * 32;
}
__host__ __device__ constexpr int quant_producer(int nw, int mt) {
  return mt == 1 ? nw : kQuantWarps;
}
constexpr int kProducerRegs = 56, kConsumerRegs = 224, kLaunchRegs = 168;
static_assert(4 * kProducerRegs + 8 * kConsumerRegs <= 12 * kLaunchRegs, "registers of the launch");

struct QuantDecodeParams : DecodeParams {
  const uint8_t* scales;
  int num_kv_heads, group_shift;
  int slab_heads;      // kv heads of a CTA
  int warps_per_head;  // consumer warp w: head w / warps_per_head of the slab, its unit
                       // tiles from (w % warps_per_head) * MT on
};

// Shared memory of a CTA (bytes from a 1024-aligned base): S stages of the
// chunk's codes and scales, two words of metadata a stage, the barriers; with two
// or more unit tiles a warp the warps' q, [tile][K step][lane] of 8 bytes.
struct QuantLayout {
  uint32_t kv_bytes, scale_bytes, stage_bytes, meta_off, bar_off, q_off, q_bytes, total;
  __host__ __device__ QuantLayout(int head_dim, int kh, int num_kv_heads, int nw, int mt, int S) {
    kv_bytes = 32u * static_cast<uint32_t>(kh) * head_dim;
    scale_bytes = 32u * static_cast<uint32_t>(num_kv_heads);
    stage_bytes = (kv_bytes + scale_bytes + 1023u) & ~1023u;
    meta_off = S * stage_bytes;
    bar_off = meta_off + S * 32u;
    q_off = (bar_off + 2u * S * 8u + 255u) & ~255u;
    q_bytes = mt > 1 ? static_cast<uint32_t>(mt) * (head_dim / 16) * 256u : 0u;
    total = q_off + nw * q_bytes;
  }
};

__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, int c0, int c1,
                                                 int c2, int c3, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit values, as ldmatrix hands it out, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Four codes as two pairs of f16: the bytes 0, 1 and 2, 3.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int SH, int MT, bool SCORED>
__global__ void __launch_bounds__(quant_threads(kQuantWarps, MT), MT == 1 ? 2 : 1)
    quant_decode_kernel(const __grid_constant__ CUtensorMap kv_map, const QuantDecodeParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int KH = p.slab_heads, WPH = p.warps_per_head, NW = KH * WPH, HKV = p.num_kv_heads;
  const uint32_t S = static_cast<uint32_t>(p.stages);
  const QuantLayout lay(D, KH, HKV, NW, MT, p.stages);
  // of a stage: (flags, first key, out_base, keys of the 16 in front of the end of what
  // the request sees), and with kFirst (batch row, rows, keys, shared keys)
  int4* meta = reinterpret_cast<int4*>(base + lay.meta_off);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + lay.bar_off);
  uint64_t* empty = full + S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int producer = quant_producer(NW, MT);
  if (warp == producer && lane == 0) prefetch_tensormap(&kv_map);
  pdl_wait();

  const long long Cn = p.splits, c = blockIdx.x;
  const int slab = blockIdx.y;
  const long long N = p.hdr[kHdrDecodeBlocks];
  const int r_start = __ldg(p.bound + c);  // -1 when the step has no decode chunk
  const long long x0 = c * N / Cn, x1 = (c + 1) * N / Cn;
  if (x0 >= x1) return;
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    fence_barrier_init();
  }
  __syncthreads();

  // keys of request r before its first streamed one (its shared prefix)
  auto key_base = [&](int r) -> int {
    const int i = r - p.shared_first;
    return (p.shared_num > 0 && i >= 0 && i < p.shared_num && __ldg(p.shared_use + i))
               ? p.shared_chunks * kChunkKeys
               : 0;
  };

  if (warp >= producer) {
    if constexpr (MT > 1) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
      if (warp > producer) return;
    }
    // ================= producer warp
    const uint64_t l2_policy = l2_evict_first_policy();
    // A request, the whole warp alike: its batch rows and keys, the keys [lo, hi)
    // that its rows see between them, and 32 entries of its block table row.
    struct Request {
      int t, n, L, lo, hi, skip, win_base, win;
    };
    auto entry_of = [&](int a) -> int { return SH == 4 ? a : (SH == 5 ? a >> 1 : 2 * a); };
    auto window = [&](int rr, Request& q, int e0) {
      q.win_base = e0;
      const int nent = (q.hi + (1 << SH) - 1) >> SH, j = e0 + lane;
      q.win =
          j < nent ? __ldg(p.block_table + static_cast<long long>(rr) * p.max_blocks + j) : -1;
    };
    auto fetch = [&](int rr, int b) -> Request {  // its chunk b is next
      Request q;
      q.t = __ldg(p.qsl + rr);
      q.n = __ldg(p.qsl + rr + 1) - q.t;
      q.L = __ldg(p.seq_lens + rr);
      q.lo = key_base(rr);
      q.hi = q.L;
      if constexpr (SCORED) {
        const int kb = q.lo;
        int a = 0x7fffffff, z = 0;
        for (int i = lane; i < q.n; i += 32) {
          const KeyRange k =
              row_keys(p.score, static_cast<long long>(q.t) + i, q.L - q.n + i, q.L, kb);
          if (k.lo < k.hi) {
            a = min(a, k.lo);
            z = max(z, k.hi);
          }
        }
        q.hi = __reduce_max_sync(0xffffffffu, z);
        a = __reduce_min_sync(0xffffffffu, a);
        q.lo = q.hi > 0 ? a : 0;
      }
      q.skip = q.lo / kChunkKeys;
      window(rr, q, entry_of(b + q.skip));
      return q;
    };
    int r = r_start;
    int pr = __ldg(p.dec_prefix + r);  // stream position of the request's first chunk
    int nblk = __ldg(p.dec_prefix + r + 1) - pr;
    int blk = static_cast<int>(x0 - pr);
    Request q = fetch(r, blk);
    // The next request is fetched one ahead, so that a boundary waits on no
    // load; only one with chunks (the rows of another may lie behind the batch's).
    int nx_pn = -1;
    Request nx{};
    auto fetch_next = [&]() {
      nx_pn = r + 1 < p.num_reqs ? __ldg(p.dec_prefix + r + 2) : -1;
      if (nx_pn - (pr + nblk) > 0) nx = fetch(r + 1, 0);
    };
    fetch_next();
    int out_base = -1;
    bool new_piece = true, ok = true;
    long long x = x0;
    uint32_t issued = 0, s = 0, eph = 0;
    for (;; ++issued) {
      if (issued >= S && !mbar_wait(&empty[s], eph)) {
        if (lane == 0) atomicOr(&g_errors_quant_decode, kErrTimeout);
        ok = false;
        break;
      }
      if (x >= x1) {
        if (lane == 0) {
          meta[2 * s] = make_int4(kEnd, 0, 0, 0);
          mbar_arrive(&full[s]);
        }
        ++issued;
        break;
      }
      if (new_piece) {
        // a request split over several CTAs, or one whose shared prefix is
        // attended elsewhere, leaves a partial for the combine kernel
        const long long cf = owner_cta(pr, N, Cn), cl = owner_cta(pr + nblk - 1, N, Cn);
        out_base = cf == cl && key_base(r) == 0 ? -1
                   : q.n == 1 ? static_cast<int>((r + c) * p.virt_heads)
                              : static_cast<int>(2 * c + (pr >= x0 ? 1 : 0));
      }
      const int ab = blk + q.skip;  // the chunk's place in the request
      const int e0 = entry_of(ab), e_hi = SH == 3 ? e0 + 1 : e0;
      if (e0 < q.win_base || e_hi >= q.win_base + 32) window(r, q, e0);
      const int phys = __shfl_sync(0xffffffffu, q.win, e0 - q.win_base);
      const int k0 = ab * kChunkKeys;
      const bool none = q.lo >= q.hi;  // no row sees a key
      bool valid = phys >= 0 && phys < p.num_blocks;
      bool first = true, second = false;  // 8-token blocks: keys 0..7 and 8..15 are wanted
      int phys1 = -1;
      if constexpr (SH == 3) {
        phys1 = __shfl_sync(0xffffffffu, q.win, e_hi - q.win_base);
        second = q.hi - k0 > 8;
        first = !SCORED || q.lo - k0 < 8;
        valid = valid || !first;
        if (second) valid = valid && phys1 >= 0 && phys1 < p.num_blocks;
      }
      if (none) valid = false;
      if (lane == 0) {
        const bool last = blk == nblk - 1 || x == x1 - 1;
        meta[2 * s] = make_int4((new_piece ? kFirst : 0) | (last ? kLast : 0) | (valid ? 0 : kInvalid),
                                k0, out_base,
                                min(kChunkKeys, q.hi - k0));
        if (new_piece) meta[2 * s + 1] = make_int4(q.t, q.n, q.L, key_base(r));
        unsigned char* stage = base + s * lay.stage_bytes;
        unsigned char* sc = stage + lay.kv_bytes;
        if (!valid && !none) atomicOr(&g_errors_quant_decode, kErrBlockRange);
        if (valid) {
          const bool half = SH == 3 && !(first && second);
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&full[s], (lay.kv_bytes + lay.scale_bytes) >> (half ? 1 : 0));
          const int hk0 = slab * KH;
          const uint32_t sb = 32u * HKV;  // scale bytes of 16 rows of K and V
          if constexpr (SH == 4) {
            tma_load_4d_hint(stage, &kv_map, 0, 0, hk0, phys * 2, &full[s], l2_policy);
            bulk_load(sc, p.scales + static_cast<long long>(phys) * sb, sb, &full[s]);
          } else if constexpr (SH == 5) {  // rows 0..15 or 16..31 of the block's K and V
            const int row = (ab & 1) * 16;
            tma_load_4d_hint(stage, &kv_map, 0, row, hk0, phys * 2, &full[s], l2_policy);
            const uint8_t* src = p.scales + (static_cast<long long>(phys) * 64 + row) * HKV;
            bulk_load(sc, src, sb / 2, &full[s]);
            bulk_load(sc + sb / 2, src + 32 * HKV, sb / 2, &full[s]);
          } else {  // two blocks of 8
            if (first) {
              tma_load_4d_hint(stage, &kv_map, 0, 0, hk0, phys * 2, &full[s], l2_policy);
              bulk_load(sc, p.scales + static_cast<long long>(phys) * (sb / 2), sb / 2, &full[s]);
            }
            if (second) {
              tma_load_4d_hint(stage + lay.kv_bytes / 2, &kv_map, 0, 0, hk0, phys1 * 2, &full[s],
                               l2_policy);
              bulk_load(sc + sb / 2, p.scales + static_cast<long long>(phys1) * (sb / 2), sb / 2,
                        &full[s]);
            }
          }
        } else {
          mbar_arrive(&full[s]);
        }
      }
      if (++s == S) {  // ring wraps; from the second wrap on, the empty parity flips
        s = 0;
        if (issued + 1 > S) eph ^= 1u;
      }
      ++x;
      ++blk;
      new_piece = false;
      if (blk == nblk) {
        blk = 0;
        new_piece = true;
        if (x < x1) {
          pr += nblk;  // empty requests in between add no chunks
          if (nx_pn - pr > 0) {
            ++r;
            nblk = nx_pn - pr;
            q = nx;
          } else {
            do {
              ++r;
              nblk = __ldg(p.dec_prefix + r + 1) - pr;
            } while (nblk == 0);
            q = fetch(r, 0);
          }
          fetch_next();
        }
      }
    }
    if (!ok && lane == 0) {
      // let every copy in flight land before the shared memory goes away
      for (uint32_t k = (issued > S ? issued - S : 0); k < issued; ++k)
        mbar_wait(&full[k % S], (k / S) & 1u, kDrainLimitNs);
    }
    return;
  }

  if constexpr (MT > 1) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    if (warp >= NW) return;
  }
  // ================= consumer warp: unit tiles tile0 .. tile0+MT-1 of kv head hk
  const int hl = warp / WPH, hk = slab * KH + hl;
  const int tile0 = (warp - hl * WPH) * MT;
  const int g = lane >> 2, t4 = lane & 3;
  const int gsh = p.group_shift, G = 1 << gsh;
  // This lane holds S and P of keys g and g + 8, and O of dims 16 i + 2 g and
  // 16 i + 2 g + 1, for the units 8 (tile0 + mt) + 2 t4 + j, j = 0, 1.
  // q: in registers with one tile, in shared memory with more (a lane's own values)
  uint32_t qb[MT == 1 ? D / 16 : 1][2];
  uint2* qs = reinterpret_cast<uint2*>(base + lay.q_off + warp * lay.q_bytes) + lane;
  float o[MT][D / 16][4];
  float fq[MT][2], m_s[MT][2], m_w[MT][2], l_run[MT][2];
  // SCORED: the unit's keys, and where its distances count from
  int lim_lo[MT][2], lim_hi[MT][2], ref[MT][2];
  float slope2[MT][2];
  const float cap2 = SCORED ? p.score.softcap * kLog2e : 0.f;
  int t = 0, n = 0, my_tiles = 0, hi_all = 0;
  // This lane's ldmatrix address within K: row lane % 8 of an 8-key group, lanes
  // 8-15 and 24-31 of the second group, 16-byte unit lane / 16 swizzled by the row.
  const int row8 = lane & 7, swz = D == 128 ? row8 : row8 >> 1;
  const uint32_t group_step = SH == 3 ? 16u * KH * D : 8u * D;  // bytes between key groups
  const uint32_t kv_step = (SH == 3 ? 8u : 16u) * KH * D;       // K to V
  const uint32_t k_off = (SH == 3 ? 8u : 16u) * hl * D + row8 * D +
                         ((lane >> 3) & 1 ? group_step : 0u) + (((lane >> 4) ^ swz) << 4);

  for (uint32_t s = 0, fph = 0;;) {  // ring slot, parity of its full barrier
    if (!mbar_wait(&full[s], fph)) {
      atomicOr(&g_errors_quant_decode, kErrTimeout);
      break;
    }
    const int4 m = meta[2 * s];
    if (m.x & kEnd) break;
    const int flags = m.x, k0 = m.y, out_base = m.z;
    const unsigned char* stage = base + s * lay.stage_bytes;

    if (flags & kFirst) {
      const int4 f = meta[2 * s + 1];
      t = f.x;
      n = f.y;
      const int L = f.z;
      my_tiles = min(MT, max(0, ((n << gsh) + 7) / 8 - tile0));
      hi_all = L - n + 1;  // keys below it are seen by every row (plain scores)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // q's row of unit 8 (tile0 + mt) + g: dims 16 x + 4 t4 .. + 3
        const int u = 8 * (tile0 + mt) + g, i = u >> gsh, h = u & (G - 1);
        uint2 w[D / 16];
        const uint16_t* src =
            p.q + (static_cast<long long>(t) + i) * p.q_stride + (hk * G + h) * D + 4 * t4;
        uint32_t amax = 0;
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          w[x] = i < n ? __ldg(reinterpret_cast<const uint2*>(src + 16 * x)) : make_uint2(0, 0);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) amax = max(amax, amax8(make_uint4(w[x].x, w[x].y, 0, 0)));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const uint32_t sb = scale_byte(amax);
        const float inv = __uint_as_float((254u - min(sb, 254u)) << 23);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint2 v = make_uint2(pack_f16x2(bf16_lo(w[x].x) * inv, bf16_hi(w[x].x) * inv),
                                     pack_f16x2(bf16_lo(w[x].y) * inv, bf16_hi(w[x].y) * inv));
          if constexpr (MT == 1) {
            qb[x][0] = v.x;
            qb[x][1] = v.y;
          } else {
            qs[(mt * (D / 16) + x) * 32] = v;
          }
        }
        // A row with an infinity or a NaN makes all its scores NaN. So does a place
        // without a row: its zeros would score 0 for keys that no row sees, under whatever
        // V scale lies there, and a rescale that these ask for would move the bits
        // of the tile's rows. (A NaN asks for none and stays in its own place.)
        const float f_mine = i < n ? p.scale_log2 * scale_value(sb) : __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          fq[mt][j] = __shfl_sync(0xffffffffu, f_mine, 8 * t4 + 4 * j);
          const int uj = 8 * (tile0 + mt) + 2 * t4 + j, ij = uj >> gsh;
          m_s[mt][j] = m_w[mt][j] = -FLT_MAX;  // (finite: no difference of infinities)
          l_run[mt][j] = 0.f;
          if constexpr (SCORED) {
            lim_lo[mt][j] = ref[mt][j] = 0;
            lim_hi[mt][j] = 0x7fffffff;  // (a place without a row masks nothing)
            slope2[mt][j] = 0.f;
            if (ij < n) {
              const int pos = L - n + ij;
              const long long row = static_cast<long long>(t) + ij;
              const KeyRange k = row_keys(p.score, row, pos, L, f.w);
              const KeyRange all = row_keys(p.score, row, pos, L, 0);
              lim_lo[mt][j] = k.lo;
              lim_hi[mt][j] = k.hi;
              ref[mt][j] = max(min(pos, all.hi - 1), all.lo);
              slope2[mt][j] = slope_log2(p.score, hk * G + (uj & (G - 1)));
            }
          }
        }
#pragma unroll
        for (int i2 = 0; i2 < D / 16; ++i2)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][i2][e] = 0.f;
      }
    }

    if (!(flags & kInvalid) && my_tiles > 0) {
      const uint32_t k_addr = smem_u32(stage) + k_off, v_addr = k_addr + kv_step;
      // ---- S^T
      float acc[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        uint32_t w[4], a[2][4];
        ldsm4(k_addr ^ (kk << 5), w);
#pragma unroll
        for (int x = 0; x < 4; ++x) codes_f16(w[x], a[x >> 1][x & 1], a[x >> 1][2 + (x & 1)]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (MT == 1) {
              mma_f16(acc[mt], a[h], qb[2 * kk + h][0], qb[2 * kk + h][1]);
            } else {
              const uint2 v = qs[(mt * (D / 16) + 2 * kk + h) * 32];
              mma_f16(acc[mt], a[h], v.x, v.y);
            }
          }
      }
      // ---- scales of keys g and g + 8: K's as a factor, V's as an exponent
      float ks[2], ve[2];
      const unsigned char* sc = stage + lay.kv_bytes + hk;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int kr = SH == 3 ? g + 16 * x : g + 8 * x;
        ks[x] = scale_value(sc[kr * HKV]);
        ve[x] = scale_exponent(sc[(kr + (SH == 3 ? 8 : 16)) * HKV]);
      }
      bool whole = true;  // every unit sees the whole chunk
      if constexpr (SCORED) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            whole = whole && lim_lo[mt][j] <= k0 && lim_hi[mt][j] >= k0 + kChunkKeys;
        whole = __all_sync(0xffffffffu, whole);
      } else {
        whole = hi_all >= k0 + kChunkKeys;
      }
      // ---- softmax: element e is key g + 8 (e / 2), unit j = e % 2
      float sv[MT][4];
      bool high = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e & 1, x = e >> 1;
          float v = acc[mt][e] * (fq[mt][j] * ks[x]);
          if constexpr (SCORED) {
            if (p.score.softcap > 0.f) v = cap2 * tanh_log2(v);
            if (p.score.slopes)
              v -= slope2[mt][j] * fabsf(static_cast<float>(ref[mt][j] - (k0 + g + 8 * x)));
          }
          sv[mt][e] = v;
        }
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = e & 1, key = k0 + g + 8 * (e >> 1);
            const int unit = 8 * (tile0 + mt) + 2 * t4 + j;
            if (SCORED ? key < lim_lo[mt][j] || key >= lim_hi[mt][j]
                       : key >= hi_all + (unit >> gsh))
              sv[mt][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e & 1;
          high = high || sv[mt][e] > m_s[mt][j] + kRescaleLog2 ||
                 sv[mt][e] + ve[e >> 1] > m_w[mt][j] + kRescaleLog2;
        }
      if (__any_sync(0xffffffffu, high)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float a = fmaxf(sv[mt][j], sv[mt][2 + j]);
            float b = fmaxf(sv[mt][j] + ve[0], sv[mt][2 + j] + ve[1]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
              b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
            }
            a = fmaxf(a, m_s[mt][j]);
            b = fmaxf(b, m_w[mt][j]);
            l_run[mt][j] *= exp2f(m_s[mt][j] - a);
            const float alpha = exp2f(m_w[mt][j] - b);
            m_s[mt][j] = a;
            m_w[mt][j] = b;
#pragma unroll
            for (int i2 = 0; i2 < D / 16; ++i2) {
              o[mt][i2][j] *= alpha;
              o[mt][i2][2 + j] *= alpha;
            }
          }
      }
      uint32_t pb[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e & 1;
          l_run[mt][j] += exp2f(sv[mt][e] - m_s[mt][j]);
          pv[e] = exp2f(sv[mt][e] + (ve[e >> 1] - m_w[mt][j]));
        }
        if (!whole) {  // (a masked row may be NaN: its exponent is one then)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sv[mt][e] == -INFINITY) pv[e] = 0.f;
        }
        pb[mt][0] = transpose8(pack_f16x2(pv[0], pv[1]));
        pb[mt][1] = transpose8(pack_f16x2(pv[2], pv[3]));
      }
      // ---- O^T += V^T P^T
      // Rows that no unit sees may hold NaN codes, which weight 0 does not undo: those
      // behind the request's last key, and with key ranges any. (A NaN score counts as
      // unseen: its weight is NaN whatever the codes are.)
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of keys 2 t4, 2 t4 + 1 and those + 8
      const bool edge = SCORED ? !whole : m.w < kChunkKeys;
      if (edge) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          bool lo, hi;
          if constexpr (SCORED) {
            bool seen = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              seen = seen || sv[mt][2 * x] > -INFINITY || sv[mt][2 * x + 1] > -INFINITY;
            const uint32_t b = __ballot_sync(0xffffffffu, seen) >> (8 * t4);  // four lanes a key
            lo = b & 0xfu;
            hi = b & 0xf0u;
          } else {
            const int j = 8 * x + 2 * t4;
            lo = j < m.w;
            hi = j + 1 < m.w;
          }
          keep[x] = (lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int i2 = 0; i2 < D / 32; ++i2) {
        uint32_t w[4], a[2][4];
        ldsm4_trans(v_addr ^ (i2 << 5), w);
        if (edge) {
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] &= keep[x & 1];
        }
        // bytes: (key 2 t4, even dim), (same, odd), (key 2 t4 + 1, even), (same, odd)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          codes_f16(__byte_perm(w[x], 0, 0x3120), a[x >> 1][2 * (x & 1)], a[x >> 1][2 * (x & 1) + 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_f16(o[mt][2 * i2], a[0], pb[mt][0], pb[mt][1]);
          mma_f16(o[mt][2 * i2 + 1], a[1], pb[mt][0], pb[mt][1]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);  // the stage may be refilled

    // ---- end of this CTA's piece of the request
    if ((flags & kLast) && my_tiles > 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l = l_run[mt][j];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
          const int u = 8 * (tile0 + mt) + 2 * t4 + j, i = u >> gsh, h = u & (G - 1);
          if (i >= n) continue;
          const int head = hk * G + h;
          // O's weights are 2^(s + v - m_w): to 2^(s - m_s), by 2^-117 to 2^120
          float up = m_w[mt][j] - m_s[mt][j];
          if (out_base < 0) {
            // The sum l may be 2^20 and more: 2^up / l could be below 2^-126, a zero,
            // where O times it is not. What is below 2^-64 of 2^up comes last (else
            // `last` is 1).
            const float low = fminf(up + 64.f, 0.f), last = exp2f(low);
            const float f = SCORED && l == 0.f ? 0.f : exp2f(up - low) / l;  // no key seen: zeros
            uint16_t* dst =
                p.out + ((static_cast<long long>(t) + i) * p.num_q_heads + head) * D + 2 * g;
#pragma unroll
            for (int i2 = 0; i2 < D / 16; ++i2)
              *reinterpret_cast<uint32_t*>(dst + 16 * i2) =
                  pack_bf16x2(o[mt][i2][j] * f * last, o[mt][i2][2 + j] * f * last);
          } else {
            // The combine sums l * V: a piece of V's above 2^72 or so is kept as 2^-48 of
            // itself under a maximum of 48 more, the same to the combine, so that no sum
            // of fewer than 2^40 weights passes fp32's largest number.
            if (up > 64.f) {
              up -= 48.f;
              l *= 0x1p-48f;
              m_s[mt][j] += 48.f;
            }
            const float f = exp2f(up);
            // n == 1: out_base is (r + c) * V, virtual heads of G or 4 q heads;
            // several rows: a slot of the few-row partials
            const long long slot =
                n == 1 ? static_cast<long long>(out_base) * (p.num_q_heads / p.virt_heads) + head
                       : (static_cast<long long>(out_base) * p.few + i) * p.num_q_heads + head;
            float* dst = (n == 1 ? p.part_o : p.few_o) + slot * D + 2 * g;
            if (g == 0) (n == 1 ? p.part_ml : p.few_ml)[slot] = make_float2(m_s[mt][j], l);
#pragma unroll
            for (int i2 = 0; i2 < D / 16; ++i2)
              *reinterpret_cast<float2*>(dst + 16 * i2) =
                  make_float2(o[mt][i2][j] * f, o[mt][i2][2 + j] * f);
          }
        }
      }
    }
    if (++s == S) {
      s = 0;
      fph ^= 1u;
    }
  }
}

// ------------------------------------------------------------------ host
constexpr int kQuantMinStages = 2, kQuantMaxStages = 8;

// How the kernel is laid out for a call: unit tiles of a consumer warp, warps of a
// kv head, kv heads of a CTA, CTAs an SM is meant to hold (16 consumer warps with one
// tile each, within the 20 warps that their registers allow; one CTA with more
// tiles). `few`: the most rows of a request on the stream.
struct QuantShape {
  int mt, wph, heads, ctas;
};

// More tiles a warp convert a head's K and V fewer times, fewer tiles leave room for
// more warps. A warp takes some 1.5 us for a chunk with one tile among 16 warps, 1.2
// and 1.5 with two and three among 8; the layout with the least time per chunk and
// head wins. 64 requests over some 2300 keys, D = 128, us with tiles of 1, 2 and 3:
// 32 q and 8 kv heads, 4 new tokens 94, 86, 86; 5 tokens 147, 141, 101; 16 tokens
// 286, 257, 305. 128 requests over 9400 keys, 8 q heads and 1 kv head, 3 tokens: 135,
// 391, 449.
static QuantShape quant_shape(int few, int group, int num_kv_heads) {
  const int tiles = (few * group + 7) / 8;
  const float chunk_us[4] = {0.f, 1.5f, 1.2f, 1.5f};
  QuantShape best{};
  float least = 0.f;
  for (int most = 3; most >= 1; --most) {
    QuantShape s;
    s.wph = (tiles + most - 1) / most;
    s.mt = (tiles + s.wph - 1) / s.wph;
    s.heads = kQuantWarps / s.wph < num_kv_heads ? kQuantWarps / s.wph : num_kv_heads;
    while (num_kv_heads % s.heads) --s.heads;
    const int nw = s.heads * s.wph;
    s.ctas = 1;
    if (s.mt == 1) s.ctas = 16 / nw < 20 / (nw + 1) ? 16 / nw : 20 / (nw + 1);
    const float us = chunk_us[s.mt] * s.wph / (nw * s.ctas);
    if (best.mt == 0 || us < least) {
      best = s;
      least = us;
    }
  }
  return best;
}

// Steps whose every request has so few new tokens that their units fit the CTA's
// warps (kFewUnits) stream all of them. In a step with longer chunks those of one
// tile do and the others go to the prefill kernel: most requests of such a step are
// decodes, and one tile a warp streams them at the copy bandwidth (320 decodes of
// 127-2047 keys: 116 us, with two tiles 156).
int quant_few_rows(int max_query_len, int group) {
  if (max_query_len < 1) return 1;
  return max_query_len <= kFewUnits / group ? max_query_len : 8 / group;
}

int quant_slab_heads(int num_kv_heads, int group, int few) {
  return quant_shape(few, group, num_kv_heads).heads;
}

constexpr int kQuantSmem = 227 * 1024;

bool quant_stages_fit(int head_dim, int num_kv_heads, int group, int few) {
  const QuantShape s = quant_shape(few, group, num_kv_heads);
  return QuantLayout(head_dim, s.heads, num_kv_heads, s.heads * s.wph, s.mt, kQuantMinStages).total +
             1024u <= kQuantSmem;
}

// Ranges of the stream by default: the CTAs of all slabs of kv heads are one wave of
// the device. (A wave per slab instead, 64 requests over some 2300 keys: 16 q and kv
// heads, D = 64, 70 us instead of 65; 40 of D = 128 247 instead of 228, four tokens
// each 282 instead of 252; 30 requests over 500 keys, 12 of D = 64, 23 instead of 20.)
static long long quant_wave(int num_sms, int ctas, int slabs) {
  const long long c = static_cast<long long>(num_sms) * ctas / slabs;
  return c > 1 ? c : 1;
}

void quant_most_splits(int num_kv_heads, int group, int num_sms, long long* splits,
                       long long* few_rows) {
  *splits = 1;
  *few_rows = 0;  // (a request of one row leaves its partials elsewhere)
  for (int n = 1; n <= kFewUnits / group; ++n) {
    const QuantShape s = quant_shape(n, group, num_kv_heads);
    const long long c = quant_wave(num_sms, s.ctas, num_kv_heads / s.heads);
    if (c > *splits) *splits = c;
    if (n > 1 && 2 * c * n > *few_rows) *few_rows = 2 * c * n;
  }
}

// Launch shape of one instantiation on one device, worked out once.
struct QuantPrep {
  int dev, kh, hkv, nw, num_sms, stages;
  long long splits;
  size_t smem;
};

template <int D, int SH, int MT, bool SCORED>
static std::vector<QuantPrep> g_quant_prep;
template <int D, int SH, int MT, bool SCORED>
static std::atomic<unsigned long long> g_quant_attr_done{0};
static std::mutex g_quant_prep_mu;

template <int D, int SH, int MT, bool SCORED>
static cudaError_t quant_prepare(int hkv, const QuantShape& shape, int num_sms, QuantPrep* out) {
  auto kern = quant_decode_kernel<D, SH, MT, SCORED>;
  const int kh = shape.heads, nw = kh * shape.wph;
  cudaError_t e = smem_attr_once(kern, kQuantSmem, g_quant_attr_done<D, SH, MT, SCORED>);
  if (e != cudaSuccess) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_quant_prep_mu);
  for (const QuantPrep& d : g_quant_prep<D, SH, MT, SCORED>)
    if (d.dev == dev && d.kh == kh && d.hkv == hkv && d.nw == nw && d.num_sms == num_sms) {
      *out = d;
      return cudaSuccess;
    }
  if constexpr (MT > 1) {
    // the warps' exchange of registers waits for those of the launch
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidKernelImage;
  }
  const int want = shape.ctas;
  auto bytes = [&](int S) { return QuantLayout(D, kh, hkv, nw, MT, S).total + 1024u; };
  int fit = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, quant_threads(nw, MT), bytes(kQuantMinStages));
  if (e != cudaSuccess) return e;
  const int ctas = fit < want ? (fit < 1 ? 1 : fit) : want;
  const size_t budget = 228u * 1024u / ctas - 1024u;
  int S = kQuantMinStages;
  while (S < kQuantMaxStages && bytes(S + 1) <= budget) ++S;
  // more than 1 / (ctas + 1) of the SM's shared memory, see decode_smem_bytes
  const size_t share = 228u * 1024u / (ctas + 1) + 1024u;
  const size_t smem = bytes(S) > share ? bytes(S) : share;
  *out = QuantPrep{dev, kh, hkv, nw, num_sms, S, quant_wave(num_sms, ctas, hkv / kh), smem};
  try {
    g_quant_prep<D, SH, MT, SCORED>.push_back(*out);
  } catch (...) {  // (no memory to keep it: worked out again by the next call)
  }
  return cudaSuccess;
}

// Calls F<D, SH, MT, SCORED>::run(args...) for the instantiated shapes.
template <template <int, int, int, bool> class F, typename... A>
static cudaError_t quant_dispatch(int head_dim, int sh, int mt, bool scored, A&&... args) {
#define PKV_QUANT_CASE(D_, SH_, MT_)                    \
  if (head_dim == D_ && sh == SH_ && mt == MT_)         \
    return scored ? F<D_, SH_, MT_, true>::run(args...) \
                  : F<D_, SH_, MT_, false>::run(args...);
#define PKV_QUANT_MT(D_, SH_) \
  PKV_QUANT_CASE(D_, SH_, 1) PKV_QUANT_CASE(D_, SH_, 2) PKV_QUANT_CASE(D_, SH_, 3)
#define PKV_QUANT_SH(D_) PKV_QUANT_MT(D_, 3) PKV_QUANT_MT(D_, 4) PKV_QUANT_MT(D_, 5)
  PKV_QUANT_SH(128) PKV_QUANT_SH(64)
#undef PKV_QUANT_SH
#undef PKV_QUANT_MT
#undef PKV_QUANT_CASE
  return cudaErrorInvalidValue;
}

template <int D, int SH, int MT, bool SCORED>
struct QuantPrepareOp {
  static cudaError_t run(int hkv, const QuantShape& shape, int sms, long long* splits) {
    QuantPrep d;
    const cudaError_t e = quant_prepare<D, SH, MT, SCORED>(hkv, shape, sms, &d);
    if (e == cudaSuccess) *splits = d.splits;
    return e;
  }
};

template <int D, int SH, int MT, bool SCORED>
struct QuantLaunchOp {
  static cudaError_t run(const QuantDecodeParams& p, const QuantShape& shape, const CUtensorMap& m,
                         int sms, cudaStream_t s) {
    QuantPrep d;
    cudaError_t e = quant_prepare<D, SH, MT, SCORED>(p.num_kv_heads, shape, sms, &d);
    if (e != cudaSuccess) return e;
    QuantDecodeParams q = p;
    q.stages = d.stages;
    const dim3 grid(static_cast<unsigned>(p.splits),
                    static_cast<unsigned>(p.num_kv_heads / shape.heads));
    return launch_pdl(quant_decode_kernel<D, SH, MT, SCORED>, grid,
                      dim3(quant_threads(shape.heads * shape.wph, MT)), d.smem, s, m, q);
  }
};

cudaError_t quant_full_wave_splits(int head_dim, int num_kv_heads, int group, int block_shift,
                                   int few, bool scored, int num_sms, long long* splits) {
  const QuantShape q = quant_shape(few, group, num_kv_heads);
  return quant_dispatch<QuantPrepareOp>(head_dim, block_shift, q.mt, scored, num_kv_heads, q,
                                        num_sms, splits);
}

cudaError_t launch_quant_decode(const AttnArgs& a, const AttnWorkspace& ws,
                                const CUtensorMap& kv_map, long long splits, int num_sms,
                                cudaStream_t stream, void** trace) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const QuantShape shape = quant_shape(a.few, group, a.num_kv_heads);
  QuantDecodeParams p;
  static_cast<DecodeParams&>(p) = decode_params(a, ws, splits);
  p.scales = a.kv_scales;
  p.num_kv_heads = a.num_kv_heads;
  p.group_shift = __builtin_ctz(static_cast<unsigned>(group));
  p.slab_heads = shape.heads;
  p.warps_per_head = shape.wph;
  cudaError_t e = quant_dispatch<QuantLaunchOp>(a.head_dim, a.block_shift, shape.mt, a.scored, p,
                                                shape, kv_map, num_sms, stream);
  if (e == cudaSuccess && trace) e = cudaEventRecord(static_cast<cudaEvent_t>(trace[3]), stream);
  if (e != cudaSuccess) return e;
  return launch_combine(p, a.head_dim, decode_heads_per_warp(group), stream);
}

cudaError_t read_errors_quant_decode(uint32_t* out, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_errors_quant_decode, sizeof(v));
  if (e != cudaSuccess) return e;
  *out |= v;
  if (clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_errors_quant_decode, &z, sizeof(z));
  }
  return e;
}

}  // namespace pkv
