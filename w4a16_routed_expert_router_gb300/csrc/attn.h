// Internal interface between the attention operators' C ABI and their kernels.
#pragma once

#include <cuda_fp16.h>

#include "../../include/moe_attn.h"
#include "common.cuh"

namespace moe {
namespace attn {

// one 16-bit element type per kernel instantiation
struct Bf16 {
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return f32_to_bf16_bits(v); }
  // two floats -> one word, `lo` in the low half
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
struct Fp16 {
  static __device__ __forceinline__ float to_f32(uint16_t v) {
    return __half2float(__ushort_as_half(v));
  }
  static __device__ __forceinline__ uint16_t from_f32(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

// 16-bit rows [tokens, heads, head_dim], strides in elements
struct Rows {
  uint16_t* p;
  long long token, head;
};

struct Rotation {
  const long long* freq;
  int rot;          // values of a head that turn
  int interleaved;
  float magnitude;
  float sign;       // +1, or -1 for the inverse
};

// Rotary positions over up to three groups of heads of one token:
// [0, hq) from q, [hq, hq + hk) from k (both turned), the rest from v (copied).
// k and v go to cache slots when `slots` is set.
struct RopeParams {
  Rows q, q_out, k, v;
  uint16_t* k_pages;
  uint16_t* v_pages;
  long long num_slots, page_stride, token_stride, head_stride;
  int page_shift;
  const int* positions;
  const long long* slots;
  Rotation r;
  int tokens, hq, hk, hv, head_dim;
  unsigned* err;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, int sms, cudaStream_t s);

struct Scores {
  float scale;
  float softcap;
  int window;
  const float* slopes;
  const int* prefix;
};

struct Batch {
  const int* cu_q;
  const int* kv_len;
  const int* page_table;
  long long table_stride;
  int columns, num_seqs, num_tokens, max_q;
};

struct AttnParams {
  Rows q, out;
  float* lse;
  const uint16_t* k_pages;
  const uint16_t* v_pages;
  long long num_pages, page_stride, token_stride, head_stride;
  Batch b;
  Scores sc;
  int hq, hk, group, head_dim, page_shift;
  unsigned* err;
};
cudaError_t launch_attn_rows(const AttnParams& p, int dtype, cudaStream_t s);

}  // namespace attn
}  // namespace moe
