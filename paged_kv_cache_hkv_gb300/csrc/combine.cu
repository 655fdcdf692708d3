// The split-KV combine (sm_103a): merges the partials that the decode kernels
// (decode.cu, quant_decode.cu) leave of requests cut by a range boundary; and the
// parameters that those kernels share.
#include "common.cuh"
#include "decode.cuh"
#include "launch.h"

namespace pkv {

// One CTA per (range boundary c of the split, virtual head vg), one warp per
// q head. A request is split when a boundary falls strictly inside its
// chunks; the first such boundary is the one right after the CTA that owns
// the request's first chunk, and that boundary's CTAs merge the request's
// partials (one per non-empty range that touched it):
//   M = max_p m_p,  o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// CTAs c >= C (one per request of a shared-prefix run) merge such a
// request's decode partials with the shared-prefix items' partials of its
// row; the boundary CTAs leave those requests to them.
// Lanes first read the (m, l) of up to 32 pieces at once, then every lane
// sums its dims over the pieces with independent loads.
//
// DEEP: for requests of many pieces (kDeepPieces), many loads in flight per
// lane, in the same order of sums. It costs registers and, for a few pieces,
// empty loads: the combine of 128 requests of some 5 pieces took 18 us with
// it and 10.6 without; that of one request of 152 pieces 10 and 60.
//
// FEW: requests of several rows are on the stream (8-bit pool), their partials in
// the slots 2 c (a CTA that goes on with the request) and 2 c + 1 (the CTA that
// begins it). The (row, q head) pairs of a request go to FEW warps in turn. Most CTAs
// find nothing to merge, so what counts is that few waves of them run: 4 warps where
// a request has 8 pairs at most, which are mostly decodes (step of 320 decodes and
// two chunks, 32 q and 8 kv heads: 11.5 us cold, with 8 warps 15.1, with 10 15.7), else
// 10, with registers for four CTAs an SM (64 requests of five tokens: 16.7 us, with 8
// warps 20.0, with 4 31, with 20 26). DEEP's registers leave room for 8.
constexpr int kCombineLoads = 32;
constexpr int kFewWarps = 4, kFewPairs = 8, kManyWarps = 10, kManyWarpsDeep = 8;

__host__ __device__ constexpr int combine_threads(int gw, int few) { return (few ? few : gw) * 32; }
__host__ __device__ constexpr int combine_ctas(bool deep, int few) {  // an SM has room for
  return deep || few == 0 ? 0 : few == kFewWarps ? 10 : 4;
}

template <int D, int GW, bool DEEP, int FEW>
__global__ void __launch_bounds__(combine_threads(GW, FEW), combine_ctas(DEEP, FEW))
    combine_kernel(const DecodeParams p) {
  const long long c = blockIdx.x;
  const int vg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long Cn = p.splits;
  pdl_trigger();
  pdl_wait();
  auto in_shared_run = [&](int rr) -> bool {
    const int i = rr - p.shared_first;
    return p.shared_num > 0 && i >= 0 && i < p.shared_num && __ldg(p.shared_use + i);
  };
  int r, si = -1;  // si: the request's place in the shared-prefix run, if it has one
  if (c >= Cn) {
    si = static_cast<int>(c - Cn);
    if (si >= p.shared_num || !__ldg(p.shared_use + si)) return;
    r = p.shared_first + si;
  } else {
    if (c < 1) return;
    r = p.bound[c];
    if (r < 0) return;
  }
  const int pr = __ldg(p.dec_prefix + r);
  const int nblk = __ldg(p.dec_prefix + r + 1) - pr;
  const long long N = p.hdr[kHdrDecodeBlocks];
  const long long cf = owner_cta(pr, N, Cn);
  if (si < 0 && (cf != c - 1 || in_shared_run(r))) return;
  const int row = FEW ? __ldg(p.qsl + r) : 0;
  const int rows = FEW ? __ldg(p.qsl + r + 1) - row : 1;
  const bool few = FEW && rows > 1;
  // pieces j < nd: the decode partial of CTA cf + j, in slot (r + cf + j) * V
  // + vg; pieces nd .. nd + ns - 1: the shared-prefix items' partials
  const int nd = static_cast<int>(owner_cta(pr + nblk - 1, N, Cn) - cf + 1);
  const int ns = si >= 0 ? p.shared_pieces : 0;
  const int npieces = nd + ns;
  auto merge = [&](int item) {
    const int h = FEW ? item % GW : item, i = FEW ? item / GW : 0;
    const long long srow = static_cast<long long>(si) * p.num_q_heads + vg * GW + h;
    const long long sstride = static_cast<long long>(p.shared_num) * p.num_q_heads;

    auto few_slot = [&](int j) -> long long {
      return ((2 * (cf + j) + (j == 0)) * p.few + i) * p.num_q_heads + vg * GW + h;
    };
    // (m, l) of piece j; empty ranges wrote nothing and weigh zero
    auto piece_ml = [&](int j) -> float2 {
      if (j >= npieces) return make_float2(-INFINITY, 0.f);
      if (j >= nd) return p.shared_ml[srow + (j - nd) * sstride];
      const long long cc = cf + j;
      if (cc * N / Cn == (cc + 1) * N / Cn) return make_float2(-INFINITY, 0.f);
      if (few) return p.few_ml[few_slot(j)];
      return p.part_ml[((r + cc) * p.virt_heads + vg) * GW + h];
    };
    auto piece_o = [&](int j) -> const float* {
      if (j >= nd) return p.shared_o + (srow + (j - nd) * sstride) * D;
      if (few) return p.few_o + few_slot(j) * D;
      return p.part_o + (((r + cf + j) * p.virt_heads + vg) * GW + h) * D;
    };
    float M = -INFINITY;
    for (int j0 = 0; j0 < npieces; j0 += 32) M = fmaxf(M, piece_ml(j0 + lane).x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));

    constexpr int E = D / 32;  // dims per lane
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float Ls = 0.f;
    for (int j0 = 0; j0 < npieces; j0 += 32) {
      const float2 ml = piece_ml(j0 + lane);
      const float wgt = (ml.x == -INFINITY) ? 0.f : exp2f(ml.x - M);
      Ls += wgt * ml.y;
      const int cnt = min(32, npieces - j0);
      if constexpr (DEEP) {
        const float* mine = piece_o(wgt == 0.f || j0 + lane >= npieces ? 0 : j0 + lane);
        // kCombineLoads pieces' loads go out before the first is used. A piece of
        // weight 0 (an empty range, which wrote no partial) reads piece 0's slot
        // and is left out of the sum: 0 times an infinity there would be a NaN.
        for (int i0 = 0; i0 < cnt; i0 += kCombineLoads) {
          float vals[kCombineLoads][E], wj[kCombineLoads];
#pragma unroll
          for (int i = 0; i < kCombineLoads; ++i) {
            wj[i] = __shfl_sync(0xffffffffu, wgt, (i0 + i) & 31);
            const float* src = reinterpret_cast<const float*>(__shfl_sync(
                                   0xffffffffu, reinterpret_cast<unsigned long long>(mine), (i0 + i) & 31)) +
                               lane * E;
            if constexpr (E == 4) {
              const float4 v = *reinterpret_cast<const float4*>(src);
              vals[i][0] = v.x;
              vals[i][1] = v.y;
              vals[i][2] = v.z;
              vals[i][3] = v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(src);
              vals[i][0] = v.x;
              vals[i][1] = v.y;
            }
          }
#pragma unroll
          for (int i = 0; i < kCombineLoads; ++i)
            if (wj[i] != 0.f) {  // (nor is there a piece behind the last)
#pragma unroll
              for (int e = 0; e < E; ++e) acc[e] += wj[i] * vals[i][e];
            }
        }
      } else {
        // 8 pieces' loads in flight per lane; a piece of weight 0 as above
#pragma unroll 8
        for (int j = 0; j < cnt; ++j) {
          const float wj = __shfl_sync(0xffffffffu, wgt, j);
          const float* src = piece_o(wj == 0.f ? 0 : j0 + j) + lane * E;
          if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            if (wj != 0.f) {
              acc[0] += wj * v.x;
              acc[1] += wj * v.y;
              acc[2] += wj * v.z;
              acc[3] += wj * v.w;
            }
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            if (wj != 0.f) {
              acc[0] += wj * v.x;
              acc[1] += wj * v.y;
            }
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, off);
    const float inv = p.scored && Ls == 0.f ? 0.f : 1.f / Ls;  // no key seen: zeros
    // (a single row's place is read here: held through the loops it spilled a register)
    const long long out_row = FEW ? static_cast<long long>(row) + i : __ldg(p.qsl + r);
    uint16_t* dst = p.out + (out_row * p.num_q_heads + vg * GW + h) * D + lane * E;
    if constexpr (E == 4) {
      uint2 ov;
      ov.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      ov.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2*>(dst) = ov;
    } else {
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
  };
  if constexpr (FEW > 0) {
    for (int item = warp; item < rows * GW; item += FEW) merge(item);
  } else {
    merge(warp);
  }
}

// ------------------------------------------------------------------ host
// Splits per request from which the combine's DEEP variant is launched (one
// decode of 250 keys, 16 pieces: 11.4 us a step with it, 16.4 without). Not in
// a plain step with prefill rows: such a step's requests are mostly not
// decodes, and where none is the DEEP kernel's registers only make its idle
// launch longer (31.5 instead of 31.0 us for the mixed step's prefill rows).
constexpr long long kDeepPieces = 8;

template <int D, int GW, int FEW, int DEEP_FEW>
static cudaError_t launch_combine_few(const DecodeParams& p, cudaStream_t stream) {
  return launch_pdl(
      p.deep_combine ? combine_kernel<D, GW, true, DEEP_FEW> : combine_kernel<D, GW, false, FEW>,
      dim3(static_cast<unsigned>(p.splits + p.shared_num), static_cast<unsigned>(p.virt_heads)),
      dim3(combine_threads(GW, p.deep_combine ? DEEP_FEW : FEW)), 0, stream, p);
}

template <int D, int GW>
static cudaError_t launch_combine_t(const DecodeParams& p, cudaStream_t stream) {
  return p.few <= 1                ? launch_combine_few<D, GW, 0, 0>(p, stream)
         : p.few * GW <= kFewPairs ? launch_combine_few<D, GW, kFewWarps, kFewWarps>(p, stream)
                                   : launch_combine_few<D, GW, kManyWarps, kManyWarpsDeep>(p, stream);
}

cudaError_t launch_combine(const DecodeParams& p, int head_dim, int gw, cudaStream_t stream) {
  if (head_dim == 128)
    return gw == 4 ? launch_combine_t<128, 4>(p, stream)
                   : gw == 2 ? launch_combine_t<128, 2>(p, stream) : launch_combine_t<128, 1>(p, stream);
  return gw == 4 ? launch_combine_t<64, 4>(p, stream)
                 : gw == 2 ? launch_combine_t<64, 2>(p, stream) : launch_combine_t<64, 1>(p, stream);
}

DecodeParams decode_params(const AttnArgs& a, const AttnWorkspace& ws, long long splits) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const int gw = decode_heads_per_warp(group);
  DecodeParams p;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.out = a.out;
  p.block_table = a.block_table;
  p.max_blocks = a.max_blocks;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.num_reqs = a.num_reqs;
  p.num_q_heads = a.num_q_heads;
  p.num_blocks = a.num_blocks;
  p.head_groups = group / gw;
  p.virt_heads = a.num_kv_heads * p.head_groups;
  decode_slab(a.num_kv_heads, group, &p.slab_vh, &p.slab_kh);
  p.splits = splits;
  p.scale_log2 = a.scale * kLog2e;
  p.scored = a.scored;
  p.score = a.score;
  p.deep_combine =
      splits >= kDeepPieces * a.num_reqs && (a.scored || a.max_query_len <= a.few);
  if (a.score.softcap > 0.f) p.scale_log2 = 2.f * kLog2e * (a.scale / a.score.softcap);
  p.dec_prefix = ws.dec_prefix;
  p.hdr = ws.hdr;
  p.part_ml = ws.part_ml;
  p.part_o = ws.part_o;
  p.bound = ws.bound;
  p.shared_first = a.shared_first;
  p.shared_num = a.shared_num;
  p.shared_chunks = a.shared_len / kChunkKeys;
  p.shared_pieces = a.shared_pieces;
  p.shared_use = ws.casc_use;
  p.shared_ml = ws.casc_ml;
  p.shared_o = ws.casc_o;
  p.few = a.few;
  p.few_ml = ws.few_ml;
  p.few_o = ws.few_o;
  return p;
}

}  // namespace pkv
