// The 8-bit pool's memory moves (sm_103a): rows quantised as they are written,
// rows read back, blocks copied, and the blocks of a step's prompt chunks
// expanded to bf16 for the tensor-core prefill kernel. The format: quant.cuh.
#include "launch.h"
#include "quant.cuh"
#include "row_split.h"
#include "write_rows.cuh"

namespace pkv {

static __device__ uint32_t g_errors_quant;

// The write as one flat stream of 16-byte words (eight bf16 in, eight codes out), in
// the order of the bf16 pool's write: word w = (2 t + kv) * vec_per_row + e. A
// row of one kv head is D / 8 words in as many neighbouring lanes, which find
// its largest magnitude by shuffles; the first of them stores the scale. Every
// thread issues the loads of its kQuantVecs words before it uses the first. A CTA
// per kQuantVecs * kQuantThreads words, however many: 16001 rows of 8 x 128 take
// 21.1 us cold (floor 14.2; with the words stored unconverted 17 of 20.9 on warm
// buffers), the read of 131072 such rows 123 us (floor 119); four words a thread and
// two CTAs an SM were 10% and 15% slower.
constexpr int kQuantVecs = 2;
constexpr int kQuantThreads = 512;

// Pool row (block * 2 + k|v) * B + offset of a slot in the pool (below 2^31 rows).
__device__ __forceinline__ int pool_row(int slot, int kv, int shift) {
  return ((((slot >> shift) * 2) + kv) << shift) + (slot & ((1 << shift) - 1));
}

template <int D>
__device__ __forceinline__ uint32_t row_amax(const uint4& v) {
  uint32_t m = amax8(v);
#pragma unroll
  for (int off = 1; off < D / 8; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

template <int D, typename Index>
__global__ void __launch_bounds__(kQuantThreads)
    quant_write_kernel(uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                       const uint4* __restrict__ key, const uint4* __restrict__ value,
                       long long key_stride_v, long long value_stride_v,
                       const int64_t* __restrict__ slots, Index total, RowSplit split, int shift,
                       int num_slots) {
  pdl_trigger();
  pdl_wait();
  const Index stride = static_cast<Index>(gridDim.x) * blockDim.x;
  const int lane = threadIdx.x & 31;
  // (total is a multiple of D / 8, so a row's lanes are in or out together; the
  // loop goes by the warp's first word, so that all lanes reach the shuffles)
  for (Index w0 = static_cast<Index>(blockIdx.x) * blockDim.x + threadIdx.x; w0 - lane < total;
       w0 += stride * kQuantVecs) {
    uint4 val[kQuantVecs];
    long long slot[kQuantVecs];
    int rem[kQuantVecs];
#pragma unroll
    for (int u = 0; u < kQuantVecs; ++u) {
      const Index w = w0 + u * stride;
      slot[u] = -1;
      val[u] = make_uint4(0, 0, 0, 0);
      rem[u] = 0;
      if (w < total) {
        Index tok;
        rem[u] = split(w, &tok);
        slot[u] = __ldg(slots + tok);
        const uint4* src = rem[u] >= split.vec_per_row
                               ? value + static_cast<long long>(tok) * value_stride_v - split.vec_per_row
                               : key + static_cast<long long>(tok) * key_stride_v;
        val[u] = __ldg(src + rem[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kQuantVecs; ++u) {
      const uint32_t s = scale_byte(row_amax<D>(val[u]));
      if (slot[u] < 0) continue;  // padding row, or past the end
      if (slot[u] >= num_slots) {
        if (rem[u] == 0) atomicOr(&g_errors_quant, kErrSlotRange);
        continue;
      }
      const int kv = rem[u] >= split.vec_per_row, e = rem[u] - kv * split.vec_per_row;
      const long long word =
          static_cast<long long>(pool_row(static_cast<int>(slot[u]), kv, shift)) * split.vec_per_row + e;
      codes[word] = quant8(val[u], s);
      if (e % (D / 8) == 0) scales[word / (D / 8)] = static_cast<uint8_t>(s);
    }
  }
}

// The write with the slots computed on the device: a warp per new token.
constexpr int kQuantMappedWarps = 8;

template <int D>
__global__ void __launch_bounds__(kQuantMappedWarps * 32)
    quant_mapped_write_kernel(const WriteRowsArgs w) {
  pdl_trigger();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kQuantMappedWarps + (threadIdx.x >> 5);
  if (t < w.num_tokens) quant_token_rows<D>(w, t, &g_errors_quant);
}

// Sixteen codes times m to bf16; WIDE: by one store, dst being 32-byte aligned.
// (Stores of half a sector each took the expansion of 32768 rows of 8 x 128 from 33
// to 44 us and the read of 131072 from 144 to 165.)
template <bool WIDE>
__device__ __forceinline__ void store16(uint4* dst, const uint4& codes, float m) {
  const uint2 a = dequant4(codes.x, m), b = dequant4(codes.y, m), c = dequant4(codes.z, m),
              d = dequant4(codes.w, m);
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
                 "r"(a.y), "r"(b.x), "r"(b.y), "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y)
                 : "memory");
  } else {
    dst[0] = make_uint4(a.x, a.y, b.x, b.y);
    dst[1] = make_uint4(c.x, c.y, d.x, d.y);
  }
}

// Rows read back: 16 codes in, 16 bf16 out per thread and word.
template <int D, bool WIDE, typename Index>
__global__ void __launch_bounds__(kQuantThreads)
    quant_read_kernel(uint4* __restrict__ key, uint4* __restrict__ value, long long key_stride_v,
                      long long value_stride_v, const uint4* __restrict__ codes,
                      const uint8_t* __restrict__ scales, const int64_t* __restrict__ slots,
                      Index total, RowSplit split, int shift, int num_slots) {
  pdl_trigger();
  pdl_wait();
  const Index stride = static_cast<Index>(gridDim.x) * blockDim.x;
  for (Index w0 = static_cast<Index>(blockIdx.x) * blockDim.x + threadIdx.x; w0 < total;
       w0 += stride * kQuantVecs) {
    uint4 val[kQuantVecs];
    float m[kQuantVecs];
    uint4* dst[kQuantVecs];
#pragma unroll
    for (int u = 0; u < kQuantVecs; ++u) {
      const Index w = w0 + u * stride;
      dst[u] = nullptr;
      if (w >= total) continue;
      Index tok;
      const int rem = split(w, &tok);
      const int kv = rem >= split.vec_per_row, e = rem - kv * split.vec_per_row;
      const long long at = __ldg(slots + tok);
      if (at < 0) continue;  // a row of padding stays as it is
      if (at >= num_slots) {
        if (rem == 0) atomicOr(&g_errors_quant, kErrSlotRange);
        continue;
      }
      const long long word =
          static_cast<long long>(pool_row(static_cast<int>(at), kv, shift)) * split.vec_per_row + e;
      val[u] = __ldg(codes + word);
      m[u] = scale_value(__ldg(scales + word / (D / 16)));
      dst[u] = (kv ? value + static_cast<long long>(tok) * value_stride_v
                   : key + static_cast<long long>(tok) * key_stride_v) + 2 * e;
    }
#pragma unroll
    for (int u = 0; u < kQuantVecs; ++u)
      if (dst[u]) store16<WIDE>(dst[u], val[u], m[u]);
  }
}

// Whole-block copies, codes and scales; a CTA per pair.
__global__ void quant_copy_kernel(uint4* __restrict__ dst, uint4* __restrict__ dst_scales,
                                  const uint4* __restrict__ src,
                                  const uint4* __restrict__ src_scales,
                                  const int32_t* __restrict__ pairs, int num_pairs,
                                  int dst_num_blocks, int src_num_blocks, int vec_per_block,
                                  int scale_vec_per_block) {
  pdl_trigger();
  pdl_wait();
  for (int i = blockIdx.x; i < num_pairs; i += gridDim.x) {
    const int s = __ldg(pairs + 2 * i), d = __ldg(pairs + 2 * i + 1);
    if (s < 0 || s >= src_num_blocks || d < 0 || d >= dst_num_blocks) {
      if (threadIdx.x == 0) atomicOr(&g_errors_quant, kErrBlockRange);
      continue;
    }
    const uint4* from = src + static_cast<long long>(s) * vec_per_block;
    uint4* to = dst + static_cast<long long>(d) * vec_per_block;
    for (int e = threadIdx.x; e < vec_per_block; e += blockDim.x) to[e] = from[e];
    from = src_scales + static_cast<long long>(s) * scale_vec_per_block;
    to = dst_scales + static_cast<long long>(d) * scale_vec_per_block;
    for (int e = threadIdx.x; e < scale_vec_per_block; e += blockDim.x) to[e] = from[e];
  }
}

// The used blocks of the step's prefill requests turned into bf16 (exactly, see
// quant.cuh), block x of the list into block x of the scratch pool, and a table
// of the scratch blocks in the rows of the requests: the prefill kernel then
// runs as over a bf16 pool. A tile of K and V serves every query tile of a
// chunk, so turning it once costs less than in every tile's way to the tensor
// cores: 6 bytes of traffic per element pair once, against n * G / 128 tiles
// that each would turn 2 x 128 x D elements again. A CTA per block.
constexpr int kExpandThreads = 256;

template <int D>
__global__ void __launch_bounds__(kExpandThreads)
    expand_kernel(ExpandArgs x, const uint4* __restrict__ codes, const uint8_t* __restrict__ scales,
                  const int32_t* __restrict__ block_table, int max_blocks, int num_blocks,
                  int shared_first, int vec_per_block) {
  pdl_trigger();
  pdl_wait();
  const int n_req = static_cast<int>(x.hdr[kHdrPrefillReqs]);
  const int total = n_req > 0 ? __ldg(x.prefix + n_req) : 0;
  for (int b = blockIdx.x; b < total; b += gridDim.x) {
    const int k = warp_upper_index(x.prefix, n_req, b);
    int r = __ldg(x.req + k);
    if (r < 0) r = shared_first;
    const long long entry =
        static_cast<long long>(r) * max_blocks + __ldg(x.first + k) + (b - __ldg(x.prefix + k));
    const int phys = __ldg(block_table + entry);
    const bool ok = phys >= 0 && phys < num_blocks && b < x.capacity;
    if (threadIdx.x == 0) {
      x.table[entry] = ok ? b : -1;  // (the prefill kernel flags an entry that it needs)
      if (b >= x.capacity) atomicOr(&g_errors_quant, kErrChunkKeys);
    }
    if (!ok) continue;
    const uint4* from = codes + static_cast<long long>(phys) * vec_per_block;
    const uint8_t* sc = scales + static_cast<long long>(phys) * (vec_per_block / (D / 16));
    uint4* to = x.pool + static_cast<long long>(b) * vec_per_block * 2;
#pragma unroll 4
    for (int e = threadIdx.x; e < vec_per_block; e += kExpandThreads) {
      const uint4 v = __ldg(from + e);
      const float m = scale_value(__ldg(sc + e / (D / 16)));
      store16<true>(to + 2 * e, v, m);
    }
  }
}

// ------------------------------------------------------------------ host
static int row_grid(long long words) {
  const long long need = (words + kQuantThreads * kQuantVecs - 1) / (kQuantThreads * kQuantVecs);
  return static_cast<int>(need < (1ll << 30) ? need : 1ll << 30);
}

// Whether a launch's word numbers, those past the end included, stay below 2^31.
static bool short_index(long long words) {
  return words + 2ll * row_grid(words) * kQuantThreads * kQuantVecs < (1ll << 31);
}

template <int D>
static cudaError_t launch_quant_write_t(void* codes, uint8_t* scales, const void* key,
                                        const void* value, long long key_stride,
                                        long long value_stride, const int64_t* slots,
                                        int num_tokens, int num_blocks, int shift,
                                        int num_kv_heads, cudaStream_t stream) {
  const RowSplit split = row_split(num_kv_heads * D / 8);
  const long long total = static_cast<long long>(num_tokens) * split.row_pair;
  const dim3 grid(row_grid(total)), block(kQuantThreads);
  const uint4 *k = static_cast<const uint4*>(key), *v = static_cast<const uint4*>(value);
  if (short_index(total))
    return launch_pdl(quant_write_kernel<D, int>, grid, block, 0, stream, static_cast<uint2*>(codes),
                      scales, k, v, key_stride / 8, value_stride / 8, slots,
                      static_cast<int>(total), split, shift, num_blocks << shift);
  return launch_pdl(quant_write_kernel<D, long long>, grid, block, 0, stream,
                    static_cast<uint2*>(codes), scales, k, v, key_stride / 8, value_stride / 8,
                    slots, total, split, shift, num_blocks << shift);
}

cudaError_t launch_quant_write(void* codes, uint8_t* scales, const void* key, const void* value,
                               long long key_stride, long long value_stride, const int64_t* slots,
                               int num_tokens, int num_blocks, int shift, int num_kv_heads,
                               int head_dim, cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  return head_dim == 128
             ? launch_quant_write_t<128>(codes, scales, key, value, key_stride, value_stride,
                                         slots, num_tokens, num_blocks, shift, num_kv_heads, stream)
             : launch_quant_write_t<64>(codes, scales, key, value, key_stride, value_stride, slots,
                                        num_tokens, num_blocks, shift, num_kv_heads, stream);
}

cudaError_t launch_quant_mapped_write(const WriteRowsArgs& w, cudaStream_t stream) {
  if (w.num_tokens == 0) return cudaSuccess;
  const int grid = (w.num_tokens + kQuantMappedWarps - 1) / kQuantMappedWarps;
  return launch_pdl(w.vec_per_head == 16 ? quant_mapped_write_kernel<128>
                                         : quant_mapped_write_kernel<64>,
                    dim3(grid), dim3(kQuantMappedWarps * 32), 0, stream, w);
}

template <int D, bool WIDE>
static cudaError_t launch_quant_read_t(void* key, void* value, long long key_stride,
                                       long long value_stride, const void* codes,
                                       const uint8_t* scales, const int64_t* slots, int num_tokens,
                                       int num_blocks, int shift, int num_kv_heads,
                                       cudaStream_t stream) {
  const RowSplit split = row_split(num_kv_heads * D / 16);
  const long long total = static_cast<long long>(num_tokens) * split.row_pair;
  const dim3 grid(row_grid(total)), block(kQuantThreads);
  uint4 *k = static_cast<uint4*>(key), *v = static_cast<uint4*>(value);
  if (short_index(total))
    return launch_pdl(quant_read_kernel<D, WIDE, int>, grid, block, 0, stream, k, v, key_stride / 8,
                      value_stride / 8, static_cast<const uint4*>(codes), scales, slots,
                      static_cast<int>(total), split, shift, num_blocks << shift);
  return launch_pdl(quant_read_kernel<D, WIDE, long long>, grid, block, 0, stream, k, v,
                    key_stride / 8, value_stride / 8, static_cast<const uint4*>(codes), scales,
                    slots, total, split, shift, num_blocks << shift);
}

cudaError_t launch_quant_read(void* key, void* value, long long key_stride, long long value_stride,
                              const void* codes, const uint8_t* scales, const int64_t* slots,
                              int num_tokens, int num_blocks, int shift, int num_kv_heads,
                              int head_dim, cudaStream_t stream) {
  if (num_tokens == 0) return cudaSuccess;
  const bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0 &&
                    key_stride % 16 == 0 && value_stride % 16 == 0;
  auto run = head_dim == 128 ? (wide ? launch_quant_read_t<128, true> : launch_quant_read_t<128, false>)
                             : (wide ? launch_quant_read_t<64, true> : launch_quant_read_t<64, false>);
  return run(key, value, key_stride, value_stride, codes, scales, slots, num_tokens, num_blocks,
             shift, num_kv_heads, stream);
}

cudaError_t launch_quant_copy(void* dst, uint8_t* dst_scales, int dst_num_blocks, const void* src,
                              const uint8_t* src_scales, int src_num_blocks, const int32_t* pairs,
                              int num_pairs, int block_size, int num_kv_heads, int head_dim,
                              int num_sms, cudaStream_t stream) {
  if (num_pairs == 0) return cudaSuccess;
  const int rows = 2 * block_size * num_kv_heads;  // a multiple of 16
  const long long cap = static_cast<long long>(num_sms) * 8;
  const int grid = static_cast<int>(num_pairs < cap ? num_pairs : cap);
  return launch_pdl(quant_copy_kernel, dim3(grid), dim3(256), 0, stream, static_cast<uint4*>(dst),
                    reinterpret_cast<uint4*>(dst_scales), static_cast<const uint4*>(src),
                    reinterpret_cast<const uint4*>(src_scales), pairs, num_pairs, dst_num_blocks,
                    src_num_blocks, rows * (head_dim / 16), rows / 16);
}

cudaError_t launch_expand(const AttnArgs& a, const ExpandArgs& x, int num_sms,
                          cudaStream_t stream) {
  const int rows = 2 * a.num_kv_heads << a.block_shift;
  const long long cap = static_cast<long long>(num_sms) * 8;
  const int grid = static_cast<int>(x.capacity < cap ? x.capacity : cap);
  return launch_pdl(a.head_dim == 128 ? expand_kernel<128> : expand_kernel<64>, dim3(grid),
                    dim3(kExpandThreads), 0, stream, x, static_cast<const uint4*>(a.kv_cache),
                    a.kv_scales, a.block_table, a.max_blocks, a.num_blocks, a.shared_first,
                    rows * (a.head_dim / 16));
}

cudaError_t read_errors_quant(uint32_t* out, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_errors_quant, sizeof(v));
  if (e != cudaSuccess) return e;
  *out |= v;
  if (clear) {
    const uint32_t z = 0;
    e = cudaMemcpyToSymbol(g_errors_quant, &z, sizeof(z));
  }
  return e;
}

}  // namespace pkv
