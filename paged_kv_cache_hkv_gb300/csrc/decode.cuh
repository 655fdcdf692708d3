// Parameters and helpers that the decode kernels share (sm_103a): the bf16
// pool's (decode.cu) and the 8-bit pool's (quant_decode.cu).
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

struct DecodeParams {
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int num_reqs, num_q_heads, num_blocks;
  int head_groups;  // q-head groups of GW per kv head
  int virt_heads;   // V = num_kv_heads * head_groups
  int slab_vh;      // virtual heads per CTA slab (<= 8); slab s = virtual heads [s*slab_vh, ...)
  int slab_kh;      // kv heads per slab = slab_vh / head_groups
  long long splits; // C: CTAs along the stream (the grid is C x slabs)
  int stages;       // depth of the shared-memory ring of K/V chunks (>= 2)
  float scale_log2;
  const int32_t* dec_prefix;
  const uint32_t* hdr;
  float2* part_ml;
  float* part_o;
  const int* bound;  // [C]: request holding the first position of CTA c's range (-1: none)
  // Shared prefix: request shared_first + i with shared_use[i] streams only
  // its chunks from shared_chunks on and always leaves partials; the combine
  // kernel merges them with the shared items' partials of its row
  // (shared_pieces of them).
  int shared_first, shared_num, shared_chunks, shared_pieces;
  const int32_t* shared_use;
  const float2* shared_ml;
  const float* shared_o;
  // Capped, biased or range-masked scores (the kernel's SCORED variant); with
  // a cap, scale_log2 holds 2 log2(e) scale / softcap instead.
  bool scored;
  ScoreParams score;
  bool deep_combine;  // requests have many pieces each (see the combine kernel)
  // 8-bit pool: most rows of a request on the stream (bf16 pool: 1), and the
  // partials of requests with several rows (see AttnWorkspace)
  int few;
  float2* few_ml;
  float* few_o;
};

// CTA that owns position x of the decode stream: ranges start at floor(c * N / C).
__device__ __forceinline__ long long owner_cta(long long x, long long N, long long C) {
  return ((x + 1) * C + N - 1) / N - 1;
}

enum : int { kFirst = 1, kLast = 2, kInvalid = 4, kEnd = 8 };

// The running max of a head is only moved (and o, l rescaled) when a chunk's
// max exceeds it by more than this many powers of two; in between, p may
// reach 2^8, far inside fp32 range. The result is the same softmax.
constexpr float kRescaleLog2 = 8.f;

// The parameters of a step's decode, but for the K/V copies' shape.
DecodeParams decode_params(const AttnArgs& a, const AttnWorkspace& ws, long long splits);

// The merge of the split requests' partials (combine.cu); gw: q heads per virtual
// head.
cudaError_t launch_combine(const DecodeParams& p, int head_dim, int gw, cudaStream_t stream);

}  // namespace pkv
