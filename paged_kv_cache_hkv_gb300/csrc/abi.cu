// C ABI of libpagedkv.so: argument checks, launch planning, tensor maps.
// Declarations and the contract of every entry point: include/pagedkv.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <map>
#include <mutex>

#include "../../include/pagedkv.h"
#include "launch.h"
#include "write_rows.cuh"

namespace {

thread_local char g_cuda_error[256] = "";

int32_t cuda_fail(cudaError_t e, const char* where) {
  std::snprintf(g_cuda_error, sizeof(g_cuda_error), "%s: %s", where, cudaGetErrorString(e));
  return PKV_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct DeviceInfo {
  int num_sms = 0;
  bool ok = false;
  std::map<long long, long long> full_wave_splits;  // by (D, group, B, kv heads)
};

constexpr int kMaxDevices = 64;
std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
bool g_dev_init[kMaxDevices] = {};

int32_t device_info(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return PKV_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!g_dev_init[dev]) {
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    d.ok = (major == 10 && minor == 3);
    g_dev_init[dev] = true;
  }
  if (!d.ok) return PKV_ERR_DEVICE;
  *out = &d;
  return PKV_OK;
}

// cuTensorMapEncodeTiled, reached through the runtime so that the library
// does not link the driver library directly.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int32_t encode_fn(EncodeTiledFn* fn) {
  static EncodeTiledFn cached = nullptr;
  static std::once_flag once;
  static cudaError_t status = cudaSuccess;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                              cudaEnableDefault, &q);
    if (status == cudaSuccess && q == cudaDriverEntryPointSuccess)
      cached = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (!cached) return cuda_fail(status == cudaSuccess ? cudaErrorSymbolNotFound : status,
                                "cuTensorMapEncodeTiled entry point");
  *fn = cached;
  return PKV_OK;
}

// bf16 map (or one of another type) of `rank` dims (dims[0] contiguous);
// strides[i] is the byte stride of dims[i + 1].
int32_t make_map_n(CUtensorMap* map, const void* base, uint32_t rank, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz,
                   CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  EncodeTiledFn fn;
  int32_t st = encode_fn(&fn);
  if (st != PKV_OK) return st;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, type, rank, const_cast<void*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    std::snprintf(g_cuda_error, sizeof(g_cuda_error), "cuTensorMapEncodeTiled failed (%d)",
                  static_cast<int>(r));
    return PKV_ERR_CUDA;
  }
  return PKV_OK;
}

// 3-D bf16 map: dims {d0, d1, d2} (d0 contiguous), byte strides of dims 1, 2.
int32_t make_map(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                 uint64_t stride1, uint64_t stride2, uint32_t b0, uint32_t b1, uint32_t b2,
                 CUtensorMapSwizzle swz) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {b0, b1, b2};
  return make_map_n(map, base, 3, dims, strides, box, swz);
}

bool block_size_ok(int32_t b) { return b == 8 || b == 16 || b == 32; }

int block_shift_of(int32_t b) { return b == 8 ? 3 : (b == 16 ? 4 : 5); }

int32_t check_layout(const pkv_cache_layout& l) {
  if (l.num_blocks < 1 || l.num_kv_heads < 1 || l.head_dim < 1 || l.block_size < 1)
    return PKV_ERR_BAD_SHAPE;
  if (!block_size_ok(l.block_size)) return PKV_ERR_UNSUPPORTED;
  if (l.head_dim != 64 && l.head_dim != 128) return PKV_ERR_UNSUPPORTED;
  // pool rows (block * 2 + k|v) * B + offset are 32-bit TMA coordinates
  if (static_cast<long long>(l.num_blocks) * 2 * l.block_size >= (1ll << 31))
    return PKV_ERR_BAD_SHAPE;
  return PKV_OK;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The shared-prefix hint of the options, checked (all zero = off).
struct SharedHint {
  int len = 0, first = 0, num = 0, pieces = 0, tpp = 0;
};

int32_t shared_hint(const pkv_attention_options* opt, const pkv_cache_layout& l, int group,
                    int num_reqs, int num_sms, SharedHint* h) {
  *h = SharedHint();
  if (!opt) return PKV_OK;
  const int len = opt->shared_prefix_len, first = opt->shared_first_req,
            num = opt->shared_num_reqs;
  if (len == 0 && first == 0 && num == 0) return PKV_OK;
  if (len <= 0 || first < 0 || num < 1) return PKV_ERR_BAD_SHAPE;
  if (len % 16 || len % l.block_size) return PKV_ERR_BAD_SHAPE;
  if (static_cast<long long>(first) + num > num_reqs) return PKV_ERR_BAD_SHAPE;
  h->len = len;
  h->first = first;
  h->num = num;
  pkv::shared_split(num, group, l.num_kv_heads, len, num_sms, &h->pieces, &h->tpp);
  return PKV_OK;
}

struct Span {
  const void* p;
  long long bytes;
};

// Whether an array that a call writes overlaps one of the others of the list
// (null arrays overlap nothing).
bool overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* v = w + 1; v != written.end(); ++v)
      if (meet(*w, *v)) return true;
    for (const Span& r : read)
      if (meet(*w, r)) return true;
  }
  return false;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The score options of the call, checked: *scored = some field is in use.
int32_t score_params(const pkv_attention_options* opt, float scale, pkv::ScoreParams* s,
                     bool* scored) {
  *s = pkv::ScoreParams{0.f, nullptr, nullptr, nullptr};
  *scored = false;
  if (!opt || opt->reserved[0] == 0) return PKV_OK;
  if (opt->reserved[0] != PKV_OPTIONS_SCORES) return PKV_ERR_BAD_SHAPE;
  const pkv_score_options* o = opt->scores;
  if (!o) return PKV_OK;
  for (int i = 0; i < 4; ++i)
    if (o->reserved[i] != 0) return PKV_ERR_BAD_SHAPE;
  // the kernels' factors softcap * log2(e) and 2 log2(e) scale / softcap stay
  // normal fp32 numbers
  if (o->softcap != 0.f) {
    const float ratio = scale / o->softcap;
    if (!(o->softcap >= 1e-30f && o->softcap <= 1e30f && ratio >= 1e-30f && ratio <= 1e30f))
      return PKV_ERR_BAD_SHAPE;
  }
  if (!aligned4(o->alibi_slopes) || !aligned4(o->key_begin) || !aligned4(o->key_end))
    return PKV_ERR_MISALIGNED;
  s->softcap = o->softcap;
  s->slopes = o->alibi_slopes;
  s->key_begin = o->key_begin;
  s->key_end = o->key_end;
  *scored = s->softcap > 0.f || s->slopes || s->key_begin || s->key_end;
  return PKV_OK;
}

struct WsLayout {
  size_t hdr, dec_prefix, pf_req, pf_prefix, part_ml, part_o, bound, casc_use, casc_ml, casc_o,
      total;
  // 8-bit pool; the expanded blocks take what lies behind
  size_t ex_first, ex_prefix, ex_table, few_ml, few_o, quant_total;
};

WsLayout ws_layout(int num_reqs, int virt_heads, int gw, int head_dim, long long splits,
                   const SharedHint& sh, int num_q_heads) {
  WsLayout w;
  const long long slots = pkv::decode_partial_slots(num_reqs, virt_heads, splits);
  size_t off = 0;
  w.hdr = off;
  off += round256(pkv::kHdrWords * sizeof(uint32_t));
  w.dec_prefix = off;
  off += round256((num_reqs + 1) * sizeof(int32_t));
  w.pf_req = off;
  off += round256((num_reqs + 1) * sizeof(int32_t));
  w.pf_prefix = off;
  off += round256((num_reqs + 2) * sizeof(int32_t));
  w.part_ml = off;
  off += round256(static_cast<size_t>(slots) * gw * sizeof(float2));
  w.part_o = off;
  off += round256(static_cast<size_t>(slots) * gw * head_dim * sizeof(float));
  w.bound = off;
  off += round256(static_cast<size_t>(splits) * sizeof(int));
  const size_t shared_rows = static_cast<size_t>(sh.pieces) * sh.num * num_q_heads;
  w.casc_use = off;
  off += round256(static_cast<size_t>(sh.num) * sizeof(int32_t));
  w.casc_ml = off;
  off += round256(shared_rows * sizeof(float2));
  w.casc_o = off;
  off += round256(shared_rows * head_dim * sizeof(float));
  w.total = off;
  return w;
}

// The further arrays of a call on the 8-bit pool that leaves partials of at most
// `few_rows` rows, two per CTA and row of a request on the decode stream.
void quant_ws_layout(WsLayout* w, int num_reqs, int max_blocks, int num_q_heads, int head_dim,
                     long long few_rows) {
  size_t off = w->total;
  w->ex_first = off;
  off += round256((num_reqs + 1) * sizeof(int32_t));
  w->ex_prefix = off;
  off += round256((num_reqs + 2) * sizeof(int32_t));
  w->ex_table = off;
  off += round256(static_cast<size_t>(num_reqs) * max_blocks * sizeof(int32_t));
  const size_t rows = static_cast<size_t>(few_rows) * num_q_heads;
  w->few_ml = off;
  off += round256(rows * sizeof(float2));
  w->few_o = off;
  off += round256(rows * head_dim * sizeof(float));
  w->quant_total = off;
}

// bytes of a block expanded to bf16
size_t expanded_block_bytes(const pkv_cache_layout& l) {
  return static_cast<size_t>(4) * l.block_size * l.num_kv_heads * l.head_dim;
}

// Ranges and rows of few-row partials that an 8-bit call's workspace is laid out for:
// the most of any number of rows a request (so that one workspace serves every step),
// or with a caller's splits those and as many rows as there can be.
void quant_ws_splits(int num_kv_heads, int group, int num_sms, const pkv_attention_options* opt,
                     long long* splits, long long* few_rows) {
  if (opt && opt->decode_splits > 0) {
    *splits = opt->decode_splits;
    *few_rows = 2ll * opt->decode_splits * (pkv::kFewUnits / group);
  } else {
    pkv::quant_most_splits(num_kv_heads, group, num_sms, splits, few_rows);
  }
}

// Options of a call on the 8-bit pool: the most rows of a request on the decode
// stream (*few: the default is given, 0 = not asked for), and the splits if the
// caller chose them (*splits, else left as it is).
int32_t quant_options(const pkv_attention_options* opt, int group, int* few, long long* splits) {
  if (!opt) return PKV_OK;
  if (opt->reserved[0] != 0 && opt->reserved[0] != PKV_OPTIONS_SCORES) return PKV_ERR_BAD_SHAPE;
  if (opt->reserved[2] != 0 || opt->reserved[3] != 0 || opt->decode_splits < 0)
    return PKV_ERR_BAD_SHAPE;
  const int rows = opt->reserved[PKV_OPTIONS_FEW_ROWS];
  if (rows < 0 || rows > pkv::kFewUnits / group) return PKV_ERR_BAD_SHAPE;
  if (rows > 0) *few = rows;
  if (opt->decode_splits > 0) *splits = opt->decode_splits;
  return PKV_OK;
}

// Ranges (CTAs) the decode stream is split into: the caller's choice, else
// one full wave of the device for the shape (cached per device).
int32_t decode_splits_for(DeviceInfo* d, int head_dim, int num_kv_heads, int group,
                          int block_size, const pkv_attention_options* opt, long long* splits) {
  if (opt) {
    if (opt->reserved[0] != 0 && opt->reserved[0] != PKV_OPTIONS_SCORES) return PKV_ERR_BAD_SHAPE;
    for (int i = 1; i < 4; ++i)
      if (opt->reserved[i] != 0) return PKV_ERR_BAD_SHAPE;
    if (opt->decode_splits < 0) return PKV_ERR_BAD_SHAPE;
    if (opt->decode_splits > 0) {
      *splits = opt->decode_splits;
      return PKV_OK;
    }
  }
  const int sh = block_shift_of(block_size);
  const long long key = ((static_cast<long long>(head_dim) * 16 + group) * 8 + sh) * 65536 +
                        num_kv_heads;
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = d->full_wave_splits.find(key);
  if (it == d->full_wave_splits.end()) {
    long long c = 0;
    cudaError_t e =
        pkv::decode_full_wave_splits(head_dim, num_kv_heads, group, sh, d->num_sms, &c);
    if (e != cudaSuccess) return cuda_fail(e, "decode occupancy");
    it = d->full_wave_splits.emplace(key, c).first;
  }
  *splits = it->second;
  return PKV_OK;
}

int32_t check_group(int num_q_heads, int num_kv_heads) {
  if (num_q_heads < 1 || num_q_heads % num_kv_heads) return PKV_ERR_BAD_SHAPE;
  const int g = num_q_heads / num_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

}  // namespace

extern "C" {

int32_t pkv_abi_version(void) { return PKV_ABI_VERSION; }

const char* pkv_status_string(int32_t status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_ERR_NULL_POINTER: return "a required pointer is NULL";
    case PKV_ERR_BAD_SHAPE: return "a size or count is out of range";
    case PKV_ERR_UNSUPPORTED: return "unsupported block size, head_dim or head grouping";
    case PKV_ERR_MISALIGNED: return "pointer or row stride not 16-byte aligned";
    case PKV_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case PKV_ERR_CUDA: return "CUDA call failed (see pkv_last_cuda_error)";
    case PKV_ERR_DEVICE: return "current device is not an sm_103 GPU";
    case PKV_ERR_SCRATCH_LIMIT:
      return "call needs more scratch than the built-in static workspace holds";
    default: return "unknown status";
  }
}

const char* pkv_last_cuda_error(void) { return g_cuda_error; }

int32_t pkv_slot_mapping(int64_t* slot_mapping, const int32_t* block_table,
                         int32_t max_blocks_per_req, const int32_t* query_start_loc,
                         const int32_t* num_computed_tokens, int32_t num_reqs,
                         int32_t num_tokens, int32_t num_blocks, int32_t block_size,
                         void* stream) {
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0 || num_blocks < 1)
    return PKV_ERR_BAD_SHAPE;
  if (block_size < 1) return PKV_ERR_BAD_SHAPE;
  if (!block_size_ok(block_size)) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!slot_mapping || !query_start_loc) return PKV_ERR_NULL_POINTER;
  if (num_reqs > 0 && (!block_table || !num_computed_tokens)) return PKV_ERR_NULL_POINTER;
  DeviceInfo* d;
  int32_t st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_slot_mapping(slot_mapping, block_table, max_blocks_per_req,
                                           query_start_loc, num_computed_tokens, num_reqs,
                                           num_tokens, num_blocks, block_size,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "slot_mapping launch");
}

int32_t pkv_paged_kv_write(void* kv_cache, const void* key, const void* value,
                           int64_t key_row_stride, int64_t value_row_stride,
                           const int64_t* slot_mapping, int32_t num_tokens,
                           pkv_cache_layout layout, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_BAD_SHAPE;
  const int64_t row = static_cast<int64_t>(layout.num_kv_heads) * layout.head_dim;
  if (key_row_stride == 0) key_row_stride = row;
  if (value_row_stride == 0) value_row_stride = row;
  if (key_row_stride < row || value_row_stride < row) return PKV_ERR_BAD_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!kv_cache || !key || !value || !slot_mapping) return PKV_ERR_NULL_POINTER;
  if (!aligned16(kv_cache) || !aligned16(key) || !aligned16(value) || (key_row_stride % 8) ||
      (value_row_stride % 8))
    return PKV_ERR_MISALIGNED;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_kv_write(kv_cache, key, value, key_row_stride, value_row_stride,
                                       slot_mapping, num_tokens, layout.num_blocks,
                                       layout.block_size, layout.num_kv_heads, layout.head_dim,
                                       d->num_sms,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "kv_write launch");
}

int32_t pkv_slot_mapping_and_write(void* kv_cache, const void* key, const void* value,
                                   int64_t key_row_stride, int64_t value_row_stride,
                                   int64_t* slot_mapping, const int32_t* block_table,
                                   int32_t max_blocks_per_req, const int32_t* query_start_loc,
                                   const int32_t* num_computed_tokens, int32_t num_reqs,
                                   int32_t num_tokens, pkv_cache_layout layout, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0) return PKV_ERR_BAD_SHAPE;
  const int64_t row = static_cast<int64_t>(layout.num_kv_heads) * layout.head_dim;
  if (key_row_stride == 0) key_row_stride = row;
  if (value_row_stride == 0) value_row_stride = row;
  if (key_row_stride < row || value_row_stride < row) return PKV_ERR_BAD_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!kv_cache || !key || !value || !query_start_loc) return PKV_ERR_NULL_POINTER;
  if (num_reqs > 0 && (!block_table || !num_computed_tokens)) return PKV_ERR_NULL_POINTER;
  if (!aligned16(kv_cache) || !aligned16(key) || !aligned16(value) || (key_row_stride % 8) ||
      (value_row_stride % 8))
    return PKV_ERR_MISALIGNED;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  const pkv::WriteRowsArgs w = pkv::write_rows_args(
      kv_cache, key, value, key_row_stride, value_row_stride, slot_mapping, block_table,
      max_blocks_per_req, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
      layout.num_blocks, layout.block_size, layout.num_kv_heads, layout.head_dim);
  cudaError_t e = pkv::launch_mapped_write(w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "slot mapping and write launch");
}

int32_t pkv_copy_blocks(void* dst_pool, int32_t dst_num_blocks, const void* src_pool,
                        int32_t src_num_blocks, const int32_t* block_pairs, int32_t num_pairs,
                        pkv_cache_layout layout, void* stream) {
  pkv_cache_layout l = layout;
  l.num_blocks = dst_num_blocks > 0 ? dst_num_blocks : 1;
  int32_t st = check_layout(l);
  if (st != PKV_OK) return st;
  if (dst_num_blocks < 1 || src_num_blocks < 1 || num_pairs < 0) return PKV_ERR_BAD_SHAPE;
  if (static_cast<long long>(src_num_blocks) * 2 * layout.block_size >= (1ll << 31))
    return PKV_ERR_BAD_SHAPE;
  if (num_pairs == 0) return PKV_OK;
  if (!dst_pool || !src_pool || !block_pairs) return PKV_ERR_NULL_POINTER;
  if (!aligned16(dst_pool) || !aligned16(src_pool)) return PKV_ERR_MISALIGNED;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_copy_blocks(dst_pool, dst_num_blocks, src_pool, src_num_blocks,
                                          block_pairs, num_pairs, layout.block_size,
                                          layout.num_kv_heads, layout.head_dim, d->num_sms,
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "copy_blocks launch");
}

int64_t pkv_attention_workspace_size(int32_t num_reqs, int32_t num_q_heads,
                                     pkv_cache_layout layout,
                                     const pkv_attention_options* options) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_reqs < 0) return PKV_ERR_BAD_SHAPE;
  st = check_group(num_q_heads, layout.num_kv_heads);
  if (st != PKV_OK) return st;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  const int group = num_q_heads / layout.num_kv_heads;
  long long splits = 0;
  st = decode_splits_for(d, layout.head_dim, layout.num_kv_heads, group, layout.block_size,
                         options, &splits);
  if (st != PKV_OK) return st;
  SharedHint sh;
  st = shared_hint(options, layout, group, num_reqs, d->num_sms, &sh);
  if (st != PKV_OK) return st;
  const int gw = pkv::decode_heads_per_warp(group);
  const int virt = layout.num_kv_heads * (group / gw);
  return static_cast<int64_t>(
      ws_layout(num_reqs, virt, gw, layout.head_dim, splits, sh, num_q_heads).total);
}

// pkv_paged_attention, and with `write` the step's slot mapping and cache
// write in the plan's launch (pkv_paged_attention_with_write). With kv_scales the
// pool is the 8-bit one (pkv_quant_paged_attention and its _with_write form).
static int32_t attention_impl(void* out, const void* q, int64_t q_row_stride, const void* kv_cache,
                       const int32_t* block_table, int32_t max_blocks_per_req,
                       const int32_t* seq_lens, const int32_t* query_start_loc,
                       const int32_t* num_computed_tokens, int32_t num_reqs, int32_t num_tokens,
                       int32_t max_query_len, int32_t max_seq_len, int32_t num_q_heads,
                       float scale, pkv_cache_layout layout, void* workspace,
                       size_t workspace_bytes, const pkv_attention_options* options, void* stream,
                       const pkv::WriteRowsArgs* write, bool quant = false,
                       const uint8_t* kv_scales = nullptr) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  st = check_group(num_q_heads, layout.num_kv_heads);
  if (st != PKV_OK) return st;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks_per_req < 0 || max_query_len < 0 ||
      max_seq_len < 0)
    return PKV_ERR_BAD_SHAPE;
  if (!(scale > 0.f) || scale > 3.0e38f) return PKV_ERR_BAD_SHAPE;  // positive and finite
  pkv::AttnArgs a;
  st = score_params(options, scale, &a.score, &a.scored);
  if (st != PKV_OK) return st;
  const int64_t row = static_cast<int64_t>(num_q_heads) * layout.head_dim;
  if (q_row_stride == 0) q_row_stride = row;
  if (q_row_stride < row) return PKV_ERR_BAD_SHAPE;
  if (num_reqs == 0 || num_tokens == 0 || max_query_len == 0) {
    // no attention to do; the write (padding rows: slots -1) still runs
    if (!write) return PKV_OK;
    if (quant) {
      DeviceInfo* d;
      st = device_info(&d);
      if (st != PKV_OK) return st;
    }
    cudaError_t e = quant ? pkv::launch_quant_mapped_write(*write, static_cast<cudaStream_t>(stream))
                          : pkv::launch_mapped_write(*write, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, "slot mapping and write launch");
  }
  if (static_cast<long long>(max_seq_len) >
      static_cast<long long>(max_blocks_per_req) * layout.block_size)
    return PKV_ERR_BAD_SHAPE;
  if (!out || !q || !kv_cache || !block_table || !seq_lens || !query_start_loc ||
      !num_computed_tokens || (quant && !kv_scales))
    return PKV_ERR_NULL_POINTER;
  if (!aligned16(out) || !aligned16(q) || !aligned16(kv_cache) || !aligned16(kv_scales) ||
      (q_row_stride % 8))
    return PKV_ERR_MISALIGNED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PKV_ERR_WORKSPACE;

  const int group = num_q_heads / layout.num_kv_heads;
  long long splits = 0;
  a.few = 1;
  if (quant) {
    a.few = pkv::quant_few_rows(max_query_len, group);
    st = quant_options(options, group, &a.few, &splits);
    if (st != PKV_OK) return st;
    if (!pkv::quant_stages_fit(layout.head_dim, layout.num_kv_heads, group, a.few))
      return PKV_ERR_UNSUPPORTED;
  }
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  if (quant) {
    if (splits == 0) {
      const cudaError_t e = pkv::quant_full_wave_splits(
          layout.head_dim, layout.num_kv_heads, group, block_shift_of(layout.block_size), a.few,
          a.scored, d->num_sms, &splits);
      if (e != cudaSuccess) return cuda_fail(e, "decode occupancy");
    }
  } else {
    st = decode_splits_for(d, layout.head_dim, layout.num_kv_heads, group, layout.block_size,
                           options, &splits);
  }
  if (st != PKV_OK) return st;
  SharedHint sh;
  st = shared_hint(options, layout, group, num_reqs, d->num_sms, &sh);
  if (st != PKV_OK) return st;
  if (static_cast<long long>(sh.len) >
      static_cast<long long>(max_blocks_per_req) * layout.block_size)
    return PKV_ERR_BAD_SHAPE;
  const int gw = pkv::decode_heads_per_warp(group);
  const int virt = layout.num_kv_heads * (group / gw);
  // (8-bit pool: laid out for the most of any step, as its size was asked for)
  long long ws_splits = splits, few_rows = 0;
  if (quant) quant_ws_splits(layout.num_kv_heads, group, d->num_sms, options, &ws_splits, &few_rows);
  WsLayout wl = ws_layout(num_reqs, virt, gw, layout.head_dim, ws_splits, sh, num_q_heads);
  if (quant) {
    quant_ws_layout(&wl, num_reqs, max_blocks_per_req, num_q_heads, layout.head_dim, few_rows);
    if (workspace_bytes < wl.quant_total + expanded_block_bytes(layout)) return PKV_ERR_WORKSPACE;
  }
  if (workspace_bytes < wl.total) return PKV_ERR_WORKSPACE;
  // The decode stream holds at most num_reqs * ceil(max_seq_len / 16)
  // chunks: with the default split, never use more ranges than that (a small
  // batch then launches a few CTAs instead of a full wave). The workspace
  // sized for the full wave still fits.
  if (!(options && options->decode_splits > 0)) {
    const long long bound =
        static_cast<long long>(num_reqs) * ((static_cast<long long>(max_seq_len) + 15) / 16);
    if (bound < splits) splits = bound > 0 ? bound : 1;
  }

  char* wsb = static_cast<char*>(workspace);
  pkv::AttnWorkspace ws;
  ws.hdr = reinterpret_cast<uint32_t*>(wsb + wl.hdr);
  ws.dec_prefix = reinterpret_cast<int32_t*>(wsb + wl.dec_prefix);
  ws.pf_req = reinterpret_cast<int32_t*>(wsb + wl.pf_req);
  ws.pf_prefix = reinterpret_cast<int32_t*>(wsb + wl.pf_prefix);
  ws.part_ml = reinterpret_cast<float2*>(wsb + wl.part_ml);
  ws.part_o = reinterpret_cast<float*>(wsb + wl.part_o);
  ws.bound = reinterpret_cast<int*>(wsb + wl.bound);
  ws.casc_use = reinterpret_cast<int32_t*>(wsb + wl.casc_use);
  ws.casc_ml = reinterpret_cast<float2*>(wsb + wl.casc_ml);
  ws.casc_o = reinterpret_cast<float*>(wsb + wl.casc_o);
  if (quant) {
    ws.ex_first = reinterpret_cast<int32_t*>(wsb + wl.ex_first);
    ws.ex_prefix = reinterpret_cast<int32_t*>(wsb + wl.ex_prefix);
    ws.ex_table = reinterpret_cast<int32_t*>(wsb + wl.ex_table);
    ws.few_ml = reinterpret_cast<float2*>(wsb + wl.few_ml);
    ws.few_o = reinterpret_cast<float*>(wsb + wl.few_o);
    ws.ex_pool = reinterpret_cast<uint4*>(wsb + wl.quant_total);
    const size_t blocks = (workspace_bytes - wl.quant_total) / expanded_block_bytes(layout);
    // (its rows, like the pool's, are 32-bit TMA coordinates)
    const size_t most = ((1ull << 31) - 1) / (2u * layout.block_size);
    ws.ex_capacity = static_cast<int>(blocks < most ? blocks : most);
  } else {
    ws.ex_first = ws.ex_prefix = ws.ex_table = nullptr;
    ws.few_ml = nullptr;
    ws.few_o = nullptr;
    ws.ex_pool = nullptr;
    ws.ex_capacity = 0;
  }

  a.out = static_cast<uint16_t*>(out);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_row_stride;
  a.kv_cache = kv_cache;
  a.kv_scales = kv_scales;
  a.block_table = block_table;
  a.max_blocks = max_blocks_per_req;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.num_computed = num_computed_tokens;
  a.num_reqs = num_reqs;
  a.num_tokens = num_tokens;
  a.max_query_len = max_query_len;
  a.max_seq_len = max_seq_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = layout.num_kv_heads;
  a.head_dim = layout.head_dim;
  a.num_blocks = layout.num_blocks;
  a.block_shift = block_shift_of(layout.block_size);
  a.scale = scale;
  a.shared_len = sh.len;
  a.shared_first = sh.first;
  a.shared_num = sh.num;
  a.shared_pieces = sh.pieces;
  a.shared_tpp = sh.tpp;

  const int D = layout.head_dim, Hkv = layout.num_kv_heads;
  const uint64_t row_bytes = static_cast<uint64_t>(Hkv) * D * 2;
  // pool as rows of one kv head: {d, kv head, (block*2 + k|v)*B + offset}.
  // A decode copy covers the kv heads of one CTA slab and a block's 32 K and
  // V rows (B = 16), 16 rows (half of the K or V rows of a 32-token block)
  // or the 16 K and V rows of an 8-token block.
  const int B = layout.block_size;
  const uint64_t pool_rows = static_cast<uint64_t>(layout.num_blocks) * 2 * B;
  const uint32_t dec_box = B == 16 ? 32u : 16u;
  int slab_vh = 0, slab_kh = 0;
  pkv::decode_slab(Hkv, group, &slab_vh, &slab_kh);
  CUtensorMap kv_map;
  if (quant) {
    // codes as {D, row of a block, kv head, block * 2 + k|v}: a copy takes 16 rows
    // (an 8-token block's 8) of K and V of a CTA's kv heads, and lands them
    // swizzled as [K|V][kv head][row][D]
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(B),
                                static_cast<cuuint64_t>(Hkv),
                                static_cast<cuuint64_t>(layout.num_blocks) * 2};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(Hkv) * D, static_cast<cuuint64_t>(D),
                                   static_cast<cuuint64_t>(B) * Hkv * D};
    const cuuint32_t box[4] = {
        static_cast<cuuint32_t>(D), B < 16 ? 8u : 16u,
        static_cast<cuuint32_t>(pkv::quant_slab_heads(Hkv, group, a.few)), 2};
    st = make_map_n(&kv_map, kv_cache, 4, dims, strides, box,
                    D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_DATA_TYPE_UINT8);
  } else {
    st = make_map(&kv_map, kv_cache, D, Hkv, pool_rows, static_cast<uint64_t>(D) * 2, row_bytes, D,
                  static_cast<uint32_t>(slab_kh), dec_box, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  if (st != PKV_OK) return st;

  a.decode_splits = splits;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void** ev = options ? options->trace_events : nullptr;
  auto mark = [&](int i) -> cudaError_t {
    return ev ? cudaEventRecord(static_cast<cudaEvent_t>(ev[i]), s) : cudaSuccess;
  };
  cudaError_t e = mark(0);
  if (e == cudaSuccess) e = pkv::launch_plan(a, ws, s, write);
  if (e == cudaSuccess) e = mark(1);
  if (e != cudaSuccess) return cuda_fail(e, "plan launch");
  if (max_query_len > a.few || sh.num > 0) {
    // the 8-bit pool's prefill runs over its blocks expanded to bf16
    pkv::AttnArgs pa = a;
    if (quant) {
      e = pkv::launch_expand(a,
                             pkv::ExpandArgs{ws.hdr, ws.pf_req, ws.ex_first, ws.ex_prefix,
                                             ws.ex_table, ws.ex_pool, ws.ex_capacity},
                             d->num_sms, s);
      if (e != cudaSuccess) return cuda_fail(e, "expand launch");
      pa.kv_cache = ws.ex_pool;
      pa.block_table = ws.ex_table;
      pa.num_blocks = ws.ex_capacity;
    }
    const uint64_t pf_rows = static_cast<uint64_t>(pa.num_blocks) * 2 * B;
    // pool for the tensor-core path, as {64-element half row, row within an
    // 8-row group, d half, kv head, 8-row group}: one copy takes the K (or V)
    // rows of one block and one kv head, and lands as 128-byte swizzled
    // 8-row atoms ordered (group, d half, row)
    CUtensorMap kv_map_sw, q_map;
    {
      const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D / 64),
                                  static_cast<cuuint64_t>(Hkv), pf_rows / 8};
      const cuuint64_t strides[4] = {row_bytes, 128, static_cast<uint64_t>(D) * 2, row_bytes * 8};
      const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), 1,
                                 static_cast<cuuint32_t>(B / 8)};
      st = make_map_n(&kv_map_sw, pa.kv_cache, 5, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (st != PKV_OK) return st;
    st = make_map(&q_map, q, D, num_q_heads, num_tokens, static_cast<uint64_t>(D) * 2,
                  static_cast<uint64_t>(q_row_stride) * 2, 64, group, 128 / group,
                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != PKV_OK) return st;
    e = pkv::launch_prefill(pa, ws, kv_map_sw, q_map, d->num_sms, s);
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  }
  e = mark(2);
  if (e == cudaSuccess)
    e = quant ? pkv::launch_quant_decode(a, ws, kv_map, splits, d->num_sms, s, ev)
              : pkv::launch_decode(a, ws, kv_map, splits, d->num_sms, s, ev);
  if (e == cudaSuccess) e = mark(4);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  return PKV_OK;
}

int32_t pkv_paged_attention(void* out, const void* q, int64_t q_row_stride, const void* kv_cache,
                            const int32_t* block_table, int32_t max_blocks_per_req,
                            const int32_t* seq_lens, const int32_t* query_start_loc,
                            const int32_t* num_computed_tokens, int32_t num_reqs,
                            int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
                            int32_t num_q_heads, float scale, pkv_cache_layout layout,
                            void* workspace, size_t workspace_bytes,
                            const pkv_attention_options* options, void* stream) {
  return attention_impl(out, q, q_row_stride, kv_cache, block_table, max_blocks_per_req,
                        seq_lens, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
                        max_query_len, max_seq_len, num_q_heads, scale, layout, workspace,
                        workspace_bytes, options, stream, nullptr);
}

int32_t pkv_paged_attention_with_write(
    void* out, const void* q, int64_t q_row_stride, void* kv_cache, const void* key,
    const void* value, int64_t key_row_stride, int64_t value_row_stride, int64_t* slot_mapping,
    const int32_t* block_table, int32_t max_blocks_per_req, const int32_t* seq_lens,
    const int32_t* query_start_loc, const int32_t* num_computed_tokens, int32_t num_reqs,
    int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len, int32_t num_q_heads,
    float scale, pkv_cache_layout layout, void* workspace, size_t workspace_bytes,
    const pkv_attention_options* options, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0) return PKV_ERR_BAD_SHAPE;
  const int64_t row = static_cast<int64_t>(layout.num_kv_heads) * layout.head_dim;
  if (key_row_stride == 0) key_row_stride = row;
  if (value_row_stride == 0) value_row_stride = row;
  if (key_row_stride < row || value_row_stride < row) return PKV_ERR_BAD_SHAPE;
  if (num_tokens > 0) {
    if (!kv_cache || !key || !value || !query_start_loc) return PKV_ERR_NULL_POINTER;
    if (num_reqs > 0 && (!block_table || !num_computed_tokens)) return PKV_ERR_NULL_POINTER;
    if (!aligned16(kv_cache) || !aligned16(key) || !aligned16(value) || (key_row_stride % 8) ||
        (value_row_stride % 8))
      return PKV_ERR_MISALIGNED;
  }
  const pkv::WriteRowsArgs w = pkv::write_rows_args(
      kv_cache, key, value, key_row_stride, value_row_stride, slot_mapping, block_table,
      max_blocks_per_req, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
      layout.num_blocks, layout.block_size, layout.num_kv_heads, layout.head_dim);
  return attention_impl(out, q, q_row_stride, kv_cache, block_table, max_blocks_per_req,
                        seq_lens, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
                        max_query_len, max_seq_len, num_q_heads, scale, layout, workspace,
                        workspace_bytes, options, stream, num_tokens > 0 ? &w : nullptr);
}

namespace {

// Checks that the 8-bit pool's row calls share; strides of 0 become the
// contiguous ones.
int32_t quant_row_args(const void* kv_cache, const void* kv_scales, const void* key,
                       const void* value, int64_t* key_row_stride, int64_t* value_row_stride,
                       int32_t num_tokens, const pkv_cache_layout& layout) {
  const int64_t row = static_cast<int64_t>(layout.num_kv_heads) * layout.head_dim;
  if (*key_row_stride == 0) *key_row_stride = row;
  if (*value_row_stride == 0) *value_row_stride = row;
  if (*key_row_stride < row || *value_row_stride < row) return PKV_ERR_BAD_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!kv_cache || !kv_scales || !key || !value) return PKV_ERR_NULL_POINTER;
  if (!aligned16(kv_cache) || !aligned16(kv_scales) || !aligned16(key) || !aligned16(value) ||
      (*key_row_stride % 8) || (*value_row_stride % 8))
    return PKV_ERR_MISALIGNED;
  return PKV_OK;
}

}  // namespace

int32_t pkv_quant_kv_write(void* kv_cache, uint8_t* kv_scales, const void* key, const void* value,
                           int64_t key_row_stride, int64_t value_row_stride,
                           const int64_t* slot_mapping, int32_t num_tokens,
                           pkv_cache_layout layout, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_BAD_SHAPE;
  st = quant_row_args(kv_cache, kv_scales, key, value, &key_row_stride, &value_row_stride,
                      num_tokens, layout);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!slot_mapping) return PKV_ERR_NULL_POINTER;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_quant_write(
      kv_cache, kv_scales, key, value, key_row_stride, value_row_stride, slot_mapping, num_tokens,
      layout.num_blocks, block_shift_of(layout.block_size), layout.num_kv_heads, layout.head_dim,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "quant_write launch");
}

int32_t pkv_quant_slot_mapping_and_write(
    void* kv_cache, uint8_t* kv_scales, const void* key, const void* value, int64_t key_row_stride,
    int64_t value_row_stride, int64_t* slot_mapping, const int32_t* block_table,
    int32_t max_blocks_per_req, const int32_t* query_start_loc, const int32_t* num_computed_tokens,
    int32_t num_reqs, int32_t num_tokens, pkv_cache_layout layout, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0) return PKV_ERR_BAD_SHAPE;
  st = quant_row_args(kv_cache, kv_scales, key, value, &key_row_stride, &value_row_stride,
                      num_tokens, layout);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!query_start_loc || (num_reqs > 0 && (!block_table || !num_computed_tokens)))
    return PKV_ERR_NULL_POINTER;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  const pkv::WriteRowsArgs w = pkv::write_rows_args(
      kv_cache, key, value, key_row_stride, value_row_stride, slot_mapping, block_table,
      max_blocks_per_req, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
      layout.num_blocks, layout.block_size, layout.num_kv_heads, layout.head_dim, kv_scales);
  cudaError_t e = pkv::launch_quant_mapped_write(w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "slot mapping and write launch");
}

int32_t pkv_quant_kv_read(void* key, void* value, int64_t key_row_stride, int64_t value_row_stride,
                          const void* kv_cache, const uint8_t* kv_scales,
                          const int64_t* slot_mapping, int32_t num_tokens, pkv_cache_layout layout,
                          void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_BAD_SHAPE;
  st = quant_row_args(kv_cache, kv_scales, key, value, &key_row_stride, &value_row_stride,
                      num_tokens, layout);
  if (st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  if (!slot_mapping) return PKV_ERR_NULL_POINTER;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_quant_read(
      key, value, key_row_stride, value_row_stride, kv_cache, kv_scales, slot_mapping, num_tokens,
      layout.num_blocks, block_shift_of(layout.block_size), layout.num_kv_heads, layout.head_dim,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "quant_read launch");
}

int32_t pkv_quant_copy_blocks(void* dst_pool, uint8_t* dst_scales, int32_t dst_num_blocks,
                              const void* src_pool, const uint8_t* src_scales,
                              int32_t src_num_blocks, const int32_t* block_pairs,
                              int32_t num_pairs, pkv_cache_layout layout, void* stream) {
  pkv_cache_layout l = layout;
  l.num_blocks = dst_num_blocks > 0 ? dst_num_blocks : 1;
  int32_t st = check_layout(l);
  if (st != PKV_OK) return st;
  if (dst_num_blocks < 1 || src_num_blocks < 1 || num_pairs < 0) return PKV_ERR_BAD_SHAPE;
  if (static_cast<long long>(src_num_blocks) * 2 * layout.block_size >= (1ll << 31))
    return PKV_ERR_BAD_SHAPE;
  if (num_pairs == 0) return PKV_OK;
  if (!dst_pool || !dst_scales || !src_pool || !src_scales || !block_pairs)
    return PKV_ERR_NULL_POINTER;
  if (!aligned16(dst_pool) || !aligned16(dst_scales) || !aligned16(src_pool) ||
      !aligned16(src_scales))
    return PKV_ERR_MISALIGNED;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_quant_copy(dst_pool, dst_scales, dst_num_blocks, src_pool, src_scales,
                                         src_num_blocks, block_pairs, num_pairs, layout.block_size,
                                         layout.num_kv_heads, layout.head_dim, d->num_sms,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "quant_copy launch");
}

int32_t pkv_quant_few_rows(int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads) {
  if (max_query_len < 0 || num_kv_heads < 1) return PKV_ERR_BAD_SHAPE;
  const int32_t st = check_group(num_q_heads, num_kv_heads);
  if (st != PKV_OK) return st;
  return pkv::quant_few_rows(max_query_len, num_q_heads / num_kv_heads);
}

int64_t pkv_quant_attention_workspace_size(int32_t num_reqs, int32_t max_blocks_per_req,
                                           int32_t num_q_heads, pkv_cache_layout layout,
                                           int64_t chunk_keys,
                                           const pkv_attention_options* options) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_reqs < 0 || max_blocks_per_req < 0 || chunk_keys < 0) return PKV_ERR_BAD_SHAPE;
  if (chunk_keys >= (1ll << 30)) return PKV_ERR_BAD_SHAPE;
  st = check_group(num_q_heads, layout.num_kv_heads);
  if (st != PKV_OK) return st;
  DeviceInfo* d;
  st = device_info(&d);
  if (st != PKV_OK) return st;
  const int group = num_q_heads / layout.num_kv_heads;
  long long splits = 0, few_rows = 0;
  int few = 0;
  st = quant_options(options, group, &few, &splits);
  if (st != PKV_OK) return st;
  quant_ws_splits(layout.num_kv_heads, group, d->num_sms, options, &splits, &few_rows);
  SharedHint sh;
  st = shared_hint(options, layout, group, num_reqs, d->num_sms, &sh);
  if (st != PKV_OK) return st;
  const int gw = pkv::decode_heads_per_warp(group);
  const int virt = layout.num_kv_heads * (group / gw);
  WsLayout wl = ws_layout(num_reqs, virt, gw, layout.head_dim, splits, sh, num_q_heads);
  quant_ws_layout(&wl, num_reqs, max_blocks_per_req, num_q_heads, layout.head_dim, few_rows);
  const int64_t keys = chunk_keys + sh.len;
  const int64_t blocks = (keys + layout.block_size - 1) / layout.block_size + 1;
  return static_cast<int64_t>(wl.quant_total + blocks * expanded_block_bytes(layout));
}

int32_t pkv_quant_paged_attention(void* out, const void* q, int64_t q_row_stride,
                                  const void* kv_cache, const uint8_t* kv_scales,
                                  const int32_t* block_table, int32_t max_blocks_per_req,
                                  const int32_t* seq_lens, const int32_t* query_start_loc,
                                  const int32_t* num_computed_tokens, int32_t num_reqs,
                                  int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
                                  int32_t num_q_heads, float scale, pkv_cache_layout layout,
                                  void* workspace, size_t workspace_bytes,
                                  const pkv_attention_options* options, void* stream) {
  return attention_impl(out, q, q_row_stride, kv_cache, block_table, max_blocks_per_req,
                        seq_lens, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
                        max_query_len, max_seq_len, num_q_heads, scale, layout, workspace,
                        workspace_bytes, options, stream, nullptr, true, kv_scales);
}

int32_t pkv_quant_paged_attention_with_write(
    void* out, const void* q, int64_t q_row_stride, void* kv_cache, uint8_t* kv_scales,
    const void* key, const void* value, int64_t key_row_stride, int64_t value_row_stride,
    int64_t* slot_mapping, const int32_t* block_table, int32_t max_blocks_per_req,
    const int32_t* seq_lens, const int32_t* query_start_loc, const int32_t* num_computed_tokens,
    int32_t num_reqs, int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
    int32_t num_q_heads, float scale, pkv_cache_layout layout, void* workspace,
    size_t workspace_bytes, const pkv_attention_options* options, void* stream) {
  int32_t st = check_layout(layout);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0) return PKV_ERR_BAD_SHAPE;
  st = quant_row_args(kv_cache, kv_scales, key, value, &key_row_stride, &value_row_stride,
                      num_tokens, layout);
  if (st != PKV_OK) return st;
  if (num_tokens > 0 && (!query_start_loc || (num_reqs > 0 && (!block_table || !num_computed_tokens))))
    return PKV_ERR_NULL_POINTER;
  const pkv::WriteRowsArgs w = pkv::write_rows_args(
      kv_cache, key, value, key_row_stride, value_row_stride, slot_mapping, block_table,
      max_blocks_per_req, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
      layout.num_blocks, layout.block_size, layout.num_kv_heads, layout.head_dim, kv_scales);
  return attention_impl(out, q, q_row_stride, kv_cache, block_table, max_blocks_per_req,
                        seq_lens, query_start_loc, num_computed_tokens, num_reqs, num_tokens,
                        max_query_len, max_seq_len, num_q_heads, scale, layout, workspace,
                        workspace_bytes, options, stream, num_tokens > 0 ? &w : nullptr, true,
                        kv_scales);
}

int32_t pkv_build_step_tables(int32_t* block_table, int32_t max_blocks_per_req,
                              int32_t* query_start_loc, int32_t* seq_lens, int64_t* slot_mapping,
                              const int32_t* num_computed_tokens, const int32_t* query_lens,
                              int32_t num_reqs, int32_t num_tokens, const int32_t* free_queue,
                              const int32_t* free_state, int32_t* free_state_out,
                              int32_t* ref_cnt, int32_t num_blocks, int32_t block_size,
                              void* stream) {
  if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0 || num_blocks < 1 || block_size < 1)
    return PKV_ERR_BAD_SHAPE;
  if (!block_size_ok(block_size)) return PKV_ERR_UNSUPPORTED;
  if (!query_start_loc || !free_queue || !free_state || !free_state_out)
    return PKV_ERR_NULL_POINTER;
  if (num_reqs > 0 && (!seq_lens || !num_computed_tokens || !query_lens ||
                       (max_blocks_per_req > 0 && !block_table)))
    return PKV_ERR_NULL_POINTER;
  for (const void* p : {static_cast<const void*>(block_table),
                        static_cast<const void*>(query_start_loc),
                        static_cast<const void*>(seq_lens),
                        static_cast<const void*>(num_computed_tokens),
                        static_cast<const void*>(query_lens), static_cast<const void*>(free_queue),
                        static_cast<const void*>(free_state),
                        static_cast<const void*>(free_state_out),
                        static_cast<const void*>(ref_cnt)})
    if (!aligned4(p)) return PKV_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return PKV_ERR_MISALIGNED;
  // threads read the inputs while others write (the state may be replaced in place)
  const long long R4 = 4ll * num_reqs;
  if (overlap({{block_table, R4 * max_blocks_per_req}, {query_start_loc, R4 + 4}, {seq_lens, R4},
               {slot_mapping, 8ll * num_tokens}, {ref_cnt, 4ll * num_blocks}, {free_state_out, 8}},
              {{num_computed_tokens, R4}, {query_lens, R4}, {free_queue, 4ll * num_blocks}}) ||
      overlap({{block_table, R4 * max_blocks_per_req}, {query_start_loc, R4 + 4}, {seq_lens, R4},
               {slot_mapping, 8ll * num_tokens}, {ref_cnt, 4ll * num_blocks}}, {{free_state, 8}}))
    return PKV_ERR_BAD_SHAPE;
  DeviceInfo* d;
  int32_t st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_build_tables(
      block_table, max_blocks_per_req, query_start_loc, seq_lens, slot_mapping,
      num_computed_tokens, query_lens, num_reqs, num_tokens, free_queue, free_state,
      free_state_out, ref_cnt, num_blocks, block_size, d->num_sms,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "build_step_tables launch");
}

int64_t pkv_release_workspace_size(int32_t num_released, int32_t max_blocks_per_req) {
  if (num_released < 0 || max_blocks_per_req < 0 ||
      static_cast<long long>(num_released) * max_blocks_per_req >= (1ll << 29))
    return PKV_ERR_BAD_SHAPE;
  return static_cast<int64_t>(pkv::release_workspace_bytes(num_released, max_blocks_per_req));
}

int32_t pkv_release_blocks(const int32_t* block_table, int32_t max_blocks_per_req,
                           int32_t num_reqs, const int32_t* release_rows,
                           const int32_t* release_tokens, int32_t num_released,
                           int32_t* free_queue, const int32_t* free_state,
                           int32_t* free_state_out, int32_t* ref_cnt, int32_t num_blocks,
                           int32_t block_size, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (num_released < 0 || num_reqs < 0 || max_blocks_per_req < 0 || num_blocks < 1 ||
      block_size < 1)
    return PKV_ERR_BAD_SHAPE;
  // the entries of one call are numbered below 2^29
  if (static_cast<long long>(num_released) * max_blocks_per_req >= (1ll << 29))
    return PKV_ERR_BAD_SHAPE;
  if (!block_size_ok(block_size)) return PKV_ERR_UNSUPPORTED;
  if (!free_queue || !free_state || !free_state_out || !ref_cnt) return PKV_ERR_NULL_POINTER;
  if (num_released > 0 && (!release_rows || !release_tokens ||
                           (num_reqs > 0 && max_blocks_per_req > 0 && !block_table)))
    return PKV_ERR_NULL_POINTER;
  for (const void* p : {static_cast<const void*>(block_table),
                        static_cast<const void*>(release_rows),
                        static_cast<const void*>(release_tokens),
                        static_cast<const void*>(free_queue), static_cast<const void*>(free_state),
                        static_cast<const void*>(free_state_out),
                        static_cast<const void*>(ref_cnt)})
    if (!aligned4(p)) return PKV_ERR_MISALIGNED;
  const size_t need = pkv::release_workspace_bytes(num_released, max_blocks_per_req);
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                   workspace_bytes < need))
    return PKV_ERR_WORKSPACE;
  const long long R4 = 4ll * num_reqs, n4 = 4ll * num_released;
  const long long ws = static_cast<long long>(need);
  if (overlap({{free_queue, 4ll * num_blocks}, {ref_cnt, 4ll * num_blocks}, {free_state_out, 8},
               {workspace, ws}},
              {{block_table, R4 * max_blocks_per_req}, {release_rows, n4}, {release_tokens, R4}}) ||
      overlap({{free_queue, 4ll * num_blocks}, {ref_cnt, 4ll * num_blocks}, {workspace, ws}},
              {{free_state, 8}}))
    return PKV_ERR_BAD_SHAPE;
  DeviceInfo* d;
  int32_t st = device_info(&d);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_release_blocks(
      block_table, max_blocks_per_req, num_reqs, release_rows, release_tokens, num_released,
      free_queue, free_state, free_state_out, ref_cnt, num_blocks, block_size, workspace,
      d->num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : cuda_fail(e, "release_blocks launch");
}

int32_t pkv_get_device_errors(uint32_t* flags, int32_t clear, void* stream) {
  if (!flags) return PKV_ERR_NULL_POINTER;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  uint32_t v = 0;
  e = pkv::read_errors_kvwrite(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_decode(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_prefill(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_plan(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_tables(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_quant(&v, clear != 0);
  if (e == cudaSuccess) e = pkv::read_errors_quant_decode(&v, clear != 0);
  if (e != cudaSuccess) return cuda_fail(e, "reading device error word");
  *flags = v;
  return PKV_OK;
}

}  // extern "C"
