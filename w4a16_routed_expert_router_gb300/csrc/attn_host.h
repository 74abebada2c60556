// What the C ABI's files of the attention operators share: the handle, checks of
// arguments, tensor maps.
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <utility>

#include "attn.h"
#include "tensor_map.h"

using namespace moe;
using namespace moe::attn;

struct moe_attn_handle {
  moe_attn_config cfg;
  int device = 0;
  int num_sms = 0;
  void* ws = nullptr;
  int grid = 0;                 // CTAs of a split launch: one per SM
  unsigned* err = nullptr;
  Partials decode{};
  TcPieces tc{};
  bool tc_usable = false;
  // The kernels over an 8-bit cache: 0 until they are set up, 1 those of few tokens, 2
  // all. Threads may make a handle's first calls at once.
  std::atomic<int> ready8{0};
};
// The error word is the workspace's first; tests set its bits through here.
static_assert(offsetof(moe_attn_handle, ws) == sizeof(moe_attn_config) + 8, "place of ws");

namespace moe {
namespace attn {

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_ATTN_OK;
  fprintf(stderr, "moe_attn: CUDA error %s\n", cudaGetErrorString(e));
  return MOE_ATTN_ERR_CUDA;
}

// A handle's device is current within, the caller's again behind.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    error_ = cudaGetDevice(&before_);
    if (error_ == cudaSuccess && before_ != device) {
      error_ = cudaSetDevice(device);
      changed_ = error_ == cudaSuccess;
    }
  }
  ~OnDevice() {
    if (changed_) cudaSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  int status() const { return cuda_status(error_); }

 private:
  int before_ = -1;
  bool changed_ = false;
  cudaError_t error_;
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int validate_config(const moe_attn_config* c) {
  if (!c) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->flags != 0) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->dtype != MOE_ATTN_BF16 && c->dtype != MOE_ATTN_FP16) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->max_tokens < 1 || c->max_tokens > (1 << 20)) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->max_seqs < 1 || c->max_seqs > kMaxSeqs) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 1024 || c->q_heads < c->kv_heads ||
      c->q_heads % c->kv_heads || c->q_heads / c->kv_heads > 64)
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8)
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  return MOE_ATTN_OK;
}

inline int validate_rotation(const moe_attn_rotation* r, int head_dim) {
  if (!r) return MOE_ATTN_ERR_INVALID_ARG;
  if (r->layout != MOE_ATTN_ROPE_HALF && r->layout != MOE_ATTN_ROPE_INTERLEAVED)
    return MOE_ATTN_ERR_INVALID_ARG;
  if (r->inverse != 0 && r->inverse != 1) return MOE_ATTN_ERR_INVALID_ARG;
  if (r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 2)
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (r->rot_dim > 0 && !r->freq) return MOE_ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(r->magnitude)) return MOE_ATTN_ERR_INVALID_ARG;
  return MOE_ATTN_OK;
}

// 16-bit elements: data on 2 bytes at least, strides that do not go backwards
inline int validate_rows(const moe_attn_rows* r) {
  if (!r || !r->data) return MOE_ATTN_ERR_INVALID_ARG;
  if (r->token_stride < 0 || r->head_stride < 0) return MOE_ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(r->data) & 1u) return MOE_ATTN_ERR_MISALIGNED;
  return MOE_ATTN_OK;
}

// Whether [tokens, heads, dim] views share an element: exact where their strides are
// the same (parts of one buffer), else by the first and last byte that each touches.
inline bool overlap(const moe_attn_rows* a, const moe_attn_rows* b, int tokens, int heads, int dim) {
  const auto span = [&](const moe_attn_rows* r) {
    return (uintptr_t)(((tokens - 1) * r->token_stride + (heads - 1) * r->head_stride + dim) * 2);
  };
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a->data);
  const uintptr_t pb = reinterpret_cast<uintptr_t>(b->data);
  if (!(pa < pb + span(b) && pb < pa + span(a))) return false;
  if ((tokens > 1 && a->token_stride != b->token_stride) ||
      (heads > 1 && a->head_stride != b->head_stride))
    return true;
  long long near = heads > 1 ? a->head_stride : dim, far = tokens > 1 ? a->token_stride : near;
  long long n_near = heads, n_far = tokens;
  if (n_far > 1 && far < near) {
    std::swap(near, far);
    std::swap(n_near, n_far);
  }
  if (near <= 0 || far <= 0) return true;
  // rows i of a and j of b are d + (their distance in rows) apart
  const long long d = (long long)(pb - pa) / 2, reach = (n_near - 1) * near + dim;
  const long long f0 = std::max(1 - n_far, (-reach - d) / far - 1);
  const long long f1 = std::min(n_far - 1, (reach - d) / far + 1);
  for (long long f = f0; f <= f1; ++f) {
    const long long r = d + f * far, n = std::min(std::max(-r / near, 1 - n_near), n_near - 1);
    for (long long k = n - 1; k <= n + 1; ++k)
      if (k > -n_near && k < n_near && std::llabs(r + k * near) < dim) return true;
  }
  return false;
}

// rows to be written: no row lies on another (of a broadcast output, whichever row
// came last would stay)
inline bool apart(const moe_attn_rows* r, int tokens, int heads, int dim) {
  long long near = r->head_stride, far = r->token_stride;
  long long n_near = heads, n_far = tokens;
  if (n_far > 1 && (n_near <= 1 || far < near)) {
    std::swap(near, far);
    std::swap(n_near, n_far);
  }
  if (n_near > 1 && near < dim) return false;
  for (long long j = 1; j < n_far && j * far < (n_near - 1) * near + dim; ++j) {
    if (n_near <= 1) return false;
    const long long i = j * far / near, rest = j * far % near;  // between rows i and i + 1
    if ((i < n_near && rest < dim) || (i + 1 < n_near && near - rest < dim)) return false;
  }
  return true;
}

inline bool same(const moe_attn_rows* a, const moe_attn_rows* b) {
  return a->data == b->data && a->token_stride == b->token_stride &&
         a->head_stride == b->head_stride;
}

inline int validate_cache(const moe_attn_cache* c) {
  if (!c || !c->k || !c->v) return MOE_ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > 0x7ffffffeLL) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (c->page_stride <= 0 || c->token_stride <= 0 || c->head_stride <= 0)
    return MOE_ATTN_ERR_INVALID_ARG;
  if (c->page_stride >= (1LL << 39) || c->token_stride >= (1LL << 39) ||
      c->head_stride >= (1LL << 39))
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;  // 2^40 bytes: a tensor map's limit
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride % 8 || c->token_stride % 8 ||
      c->head_stride % 8)
    return MOE_ATTN_ERR_MISALIGNED;
  return MOE_ATTN_OK;
}

// The cap, small enough that it is finite in log2 units, and what brings a product
// to a part of it: at most 1e38, which takes every product but zero to +-1, as
// infinity would.
inline float cap_of(const moe_attn_scores* s) { return fminf(s->softcap, 2.3e38f); }
inline float cap_in_of(const moe_attn_scores* s) {
  if (!(s->softcap > 0.0f)) return 0.0f;
  return fmaxf(fminf(s->scale / cap_of(s), 1e38f), -1e38f);
}

inline Rows rows(const moe_attn_rows* r) {
  return r ? Rows{static_cast<uint16_t*>(r->data), r->token_stride, r->head_stride}
           : Rows{nullptr, 0, 0};
}

inline Rotation rotation(const moe_attn_rotation* r) {
  return Rotation{reinterpret_cast<const long long*>(r->freq), r->rot_dim,
                  r->layout == MOE_ATTN_ROPE_INTERLEAVED, r->magnitude,
                  r->inverse ? -1.0f : 1.0f};
}

inline int log2i(int v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

inline int encode(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims,
           const cuuint64_t* strides, const cuuint32_t* box,
           CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT16,
           CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return MOE_ATTN_ERR_CUDA;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, type, rank, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    fprintf(stderr, "moe_attn: cuTensorMapEncodeTiled failed (%d)\n", (int)r);
    return MOE_ATTN_ERR_CUDA;
  }
  return MOE_ATTN_OK;
}

// stride in bytes of a tensor map's dimension; one of a single element is free
inline cuuint64_t bytes_of(long long stride, long long n, int head_dim) {
  return (cuuint64_t)(n > 1 ? stride : (head_dim + 7) & ~7) * 2;
}

// 3-D view {head_dim, q_heads, tokens} of q, boxes of one tile: its tokens by
// the heads of one group, 64 values wide.
inline int encode_q(CUtensorMap* m, const moe_attn_config& c, const moe_attn_rows* q, int tokens) {
  const int group = c.q_heads / c.kv_heads;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.q_heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {bytes_of(q->head_stride, c.q_heads, c.head_dim),
                                 bytes_of(q->token_stride, tokens, c.head_dim)};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tile_tokens(group)};
  return encode(m, 3, q->data, dims, strides, box);
}

// What a call of attention is checked for before its cache.
inline int check_call(const moe_attn_handle* h, const moe_attn_batch* b, const moe_attn_scores* sc,
                      int sinks) {
  if (!h || !b || !sc) return MOE_ATTN_ERR_INVALID_ARG;
  const moe_attn_config& c = h->cfg;
  if (b->num_tokens < 0 || b->num_seqs < 0 || b->max_q < 0) return MOE_ATTN_ERR_INVALID_ARG;
  if (b->num_tokens > c.max_tokens || b->num_seqs > c.max_seqs)
    return MOE_ATTN_ERR_TOO_MANY_TOKENS;
  if (!std::isfinite(sc->scale) || !std::isfinite(sc->softcap) || sc->softcap < 0.0f ||
      sc->window < 0 || sinks < 0)
    return MOE_ATTN_ERR_INVALID_ARG;
  return MOE_ATTN_OK;
}

// The same behind it, of a batch that is not empty.
inline int check_batch(const moe_attn_config& c, const moe_attn_rows* q, const moe_attn_rows* out,
                       const moe_attn_batch* b) {
  int st;
  if ((st = validate_rows(q)) != MOE_ATTN_OK || (st = validate_rows(out)) != MOE_ATTN_OK) return st;
  if (!aligned16(q->data) || !aligned16(out->data) || q->token_stride % 8 || q->head_stride % 8 ||
      out->token_stride % 8 || out->head_stride % 8)
    return MOE_ATTN_ERR_MISALIGNED;
  if (!apart(out, b->num_tokens, c.q_heads, c.head_dim) ||
      overlap(q, out, b->num_tokens, c.q_heads, c.head_dim))
    return MOE_ATTN_ERR_INVALID_ARG;
  for (const moe_attn_rows* r : {q, out}) {  // broadcast rows are not taken here
    if ((r->token_stride == 0 && b->num_tokens > 1) || (r->head_stride == 0 && c.q_heads > 1))
      return MOE_ATTN_ERR_INVALID_ARG;
    if (r->token_stride >= (1LL << 39) || r->head_stride >= (1LL << 39))
      return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;  // 2^40 bytes: a tensor map's limit
  }
  if (!b->cu_q || !b->kv_len || !b->page_table || b->columns < 1 || b->table_stride < b->columns)
    return MOE_ATTN_ERR_INVALID_ARG;
  if ((long long)b->columns * c.page_size > (1LL << 29))
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;  // int32 sums of positions
  return MOE_ATTN_OK;
}

inline AttnParams params_of(const moe_attn_handle* h, const moe_attn_rows* q,
                            const moe_attn_rows* out, float* lse, long long num_pages,
                            const moe_attn_batch* b, const moe_attn_scores* sc, int sinks) {
  const moe_attn_config& c = h->cfg;
  AttnParams p{};
  p.q = rows(q);
  p.out = rows(out);
  p.lse = lse;
  p.num_pages = num_pages;
  p.b = Batch{b->cu_q, b->kv_len, b->page_table, b->table_stride, b->columns, b->num_seqs,
              b->num_tokens, b->max_q};
  // a window as long as the table hides nothing
  const int window = sc->window >= (long long)b->columns * c.page_size ? 0 : sc->window;
  p.sc = Scores{sc->scale, cap_of(sc), cap_in_of(sc), window, sc->slopes, sc->prefix,
                window ? sinks : 0};
  p.hq = c.q_heads;
  p.hk = c.kv_heads;
  p.group = c.q_heads / c.kv_heads;
  p.head_dim = c.head_dim;
  p.page_shift = log2i(c.page_size);
  p.err = h->err;
  return p;
}

// the tensor-core kernel over a 16-bit cache
int forward_many(moe_attn_handle* h, AttnParams p, const moe_attn_rows* q,
                 const moe_attn_cache* cache, cudaStream_t s);

// moe_attn_forward with first tokens that stay visible behind a window
int forward_sinks(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out, float* lse,
                  const moe_attn_cache* cache, const moe_attn_batch* b, const moe_attn_scores* sc,
                  int sinks, void* stream);

}  // namespace attn
}  // namespace moe
