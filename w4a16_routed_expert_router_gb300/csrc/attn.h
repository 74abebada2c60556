// Internal interface between the attention operators' C ABI and their kernels.
#pragma once

#include <cuda_fp16.h>

#include "../../include/moe_attn.h"
#include "common.cuh"

namespace moe {
namespace attn {

// one 16-bit element type per kernel instantiation
struct Bf16 {
  static constexpr bool kFp16 = false;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return f32_to_bf16_bits(v); }
  // two floats -> one word, `lo` in the low half
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
struct Fp16 {
  static constexpr bool kFp16 = true;
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
cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t s);

struct Scores {
  float scale;
  float softcap;
  float cap_in;  // scale / softcap, finite; 0 without a cap
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

// How the tensor-core kernel's boxes of K and V are addressed: where `both`,
// one box brings 8-row groups with both 64-value chunks of a head; its group
// coordinate is page * page_groups + group in the page, its head coordinate
// page * page_heads + head.
struct Boxes {
  int both, page_groups, page_heads;
};

struct AttnParams {
  Rows q, out;
  float* lse;
  long long num_pages;
  Batch b;
  Scores sc;
  int hq, hk, group, head_dim, page_shift;
  Boxes boxes;
  unsigned* err;
};

// Split attention: a launch divides its key blocks evenly over the CTAs, in
// the order of the work items, so a CTA holds the end of one item, whole
// items, and the beginning of another; items that several CTAs hold are joined
// by the last of them to finish, in the order of their pieces.
constexpr int kMaxSeqs = 16384;       // a number for each fits the ring of the tensor-core kernel
constexpr int kMaxGrid = 160;         // CTAs of a split launch (152 SMs on GB300)
constexpr int kDecodeRows = 16;       // query rows per kv head of the few-token kernel
// keys per block of that kernel, by 64-value chunks of a head: 32 KB of K and V
__host__ __device__ constexpr int decode_block(int chunks) { return 128 / chunks; }

struct Partials {
  float* o;           // [kMaxGrid][2][rows][head_dim rounded to 64] weighted sums, not normalised
  float2* ml;         // [kMaxGrid][2][rows] maximum (log2 units) and sum
  unsigned* count;    // [kMaxGrid] pieces that arrived, by the item's first CTA (self-resetting)
};

// Keys of one sequence that some query row sees, in blocks of `block` keys:
// block n of `blocks` is key block n, or n + skip from n = near on (a prefix,
// a gap, a window).
struct Span {
  int first, n, kv;       // q rows [first, first + n), keys
  int near, skip, blocks;
};

// The sequence's rows and keys, or n = 0 with the error bit set where they
// leave their ranges.
__device__ __forceinline__ Span read_sequence(const Batch& b, int page_shift, int s,
                                              unsigned* err) {
  Span r{};
  const int q0 = b.cu_q[s], q1 = b.cu_q[s + 1], kv = b.kv_len[s];
  if (q0 < 0 || q1 < q0 || q1 > b.num_tokens || q1 - q0 > b.max_q || kv < 0 ||
      kv > (b.columns << page_shift)) {
    atomicOr(err, kErrRange);
    return r;
  }
  r.first = q0;
  r.n = q1 - q0;
  r.kv = kv;
  return r;
}

__device__ __forceinline__ int prefix_of(const Scores& sc, int s, int kv) {
  return sc.prefix ? min(kv, max(0, sc.prefix[s])) : 0;
}

// Blocks seen by rows at positions [p0, p1] (p1 >= p0), at least one.
__device__ __forceinline__ void span_blocks(Span& r, int p0, int p1, int window, int prefix,
                                            int block) {
  const int end = min(r.kv, max(p1 + 1, prefix));
  const int from = window ? max(0, p0 - window + 1) : 0;
  const int last = (max(end, 1) + block - 1) / block;      // blocks [.., last)
  const int wb = min(from / block, last - 1);
  const int pb = (prefix + block - 1) / block;
  if (prefix == 0) {
    r.near = 0;
    r.skip = wb;
  } else if (wb <= pb) {
    r.near = 0;
    r.skip = 0;
  } else {
    r.near = pb;
    r.skip = wb - pb;
  }
  r.blocks = last - r.skip;
}

// A 64-bit division takes some 400 cycles, a 32-bit one some 80.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Equal shares: CTA c holds [begin(c), begin(c + 1)) of `total`, `per` each, the
// last one what is left; `grid` of them hold something.
struct Shares {
  long long total, per;
  int grid;
  __device__ __forceinline__ Shares(long long all, int most) : total(all), per(1), grid(0) {
    if (all > 0) {
      per = quotient(all + most - 1, most);
      grid = (int)quotient(all + per - 1, per);
    }
  }
  __device__ __forceinline__ long long begin(int c) const { return min(total, c * per); }
  __device__ __forceinline__ int of(long long i) const { return (int)quotient(i, per); }
};

// batches with at most kDecodeRows query rows per sequence and kv head
cudaError_t attn_decode_setup();
cudaError_t launch_attn_decode(const AttnParams& p, const Partials& w, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, int dtype, int grid, cudaStream_t s);


// ---------------------------------------------------------- tensor-core kernel
// An entry is up to two tiles of query tokens of one sequence (all kv heads);
// (entry, kv head) is a work item. A tile's 128 rows are tile_tokens tokens by
// the heads of one group.
constexpr int kTcBlock = 128;  // keys per block
struct Entry {
  int first, ntok;             // q row of the first token, tokens
  int p0, kv;                  // position of the first token, keys of the sequence
  int near, skip, blocks;      // see Span
  int prefix, seq;
};

// What pieces of items leave for each other.
struct TcPieces {
  unsigned* count;  // [kMaxGrid][2][2 tiles] halves of a pair that arrived (self-resetting)
  float* o;         // [kMaxGrid][2 pieces][2 tiles][dim / 4][128 rows][4]
  float2* ml;       // [kMaxGrid][2][2][128] maximum (log2 units), sum
};

__host__ __device__ inline int tile_tokens(int group) { return 128 / group; }

// *usable: the kernels came out of the compiler with what they rely on
cudaError_t attn_tc_setup(bool* usable);
cudaError_t launch_attn_tc(const AttnParams& p, const TcPieces& w, const CUtensorMap& qmap,
                           const CUtensorMap& kmap, const CUtensorMap& vmap, int dtype, int grid,
                           cudaStream_t s);

}  // namespace attn
}  // namespace moe
