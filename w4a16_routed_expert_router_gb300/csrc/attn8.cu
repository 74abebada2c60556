// C ABI of include/moe_attn8.h: argument validation and dispatch.
#include "attn_host.h"

namespace {

int validate_norm(const moe_attn_norm* n, int head_dim, int q_heads, int k_heads) {
  if (!n) return MOE_ATTN_ERR_INVALID_ARG;
  if (n->weight_type != MOE_ATTN_WEIGHT_SAME && n->weight_type != MOE_ATTN_WEIGHT_F32)
    return MOE_ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(n->eps) || n->eps < 0.0f || !std::isfinite(n->offset))
    return MOE_ATTN_ERR_INVALID_ARG;
  const uintptr_t odd = n->weight_type == MOE_ATTN_WEIGHT_F32 ? 3u : 1u;
  const struct {
    const void* w;
    int64_t stride;
    int heads;
  } both[2] = {{n->q_weight, n->q_head_stride, q_heads}, {n->k_weight, n->k_head_stride, k_heads}};
  for (const auto& b : both) {
    if (b.heads == 0) continue;
    if (!b.w || b.stride < 0 || (b.stride > 0 && b.stride < head_dim))
      return MOE_ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(b.w) & odd) return MOE_ATTN_ERR_MISALIGNED;
  }
  return MOE_ATTN_OK;
}

Norm norm_of(const moe_attn_norm* n) {
  if (!n) return Norm{nullptr, nullptr, 0, 0, 0.0f, 0.0f, 0, 0};
  return Norm{n->q_weight, n->k_weight, n->q_head_stride, n->k_head_stride, n->eps, n->offset,
              n->weight_type == MOE_ATTN_WEIGHT_F32, 1};
}

// an input and what becomes of it
int validate_pair(const moe_attn_rows* x, const moe_attn_rows* out, int tokens, int heads,
                  int dim) {
  int st;
  if ((st = validate_rows(x)) != MOE_ATTN_OK || (st = validate_rows(out)) != MOE_ATTN_OK) return st;
  if (!apart(out, tokens, heads, dim) || (!same(x, out) && overlap(x, out, tokens, heads, dim)))
    return MOE_ATTN_ERR_INVALID_ARG;
  return MOE_ATTN_OK;
}

// rows of two kinds of heads: whether they share a byte (by their first and last ones;
// parts of one buffer, heads behind heads, are told apart)
bool share(const moe_attn_rows* a, int heads_a, const moe_attn_rows* b, int heads_b, int tokens,
           int dim) {
  const auto span = [&](const moe_attn_rows* r, int heads) {
    return (uintptr_t)(((tokens - 1) * r->token_stride + (heads - 1) * r->head_stride + dim) * 2);
  };
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a->data);
  const uintptr_t pb = reinterpret_cast<uintptr_t>(b->data);
  if (!(pa < pb + span(b, heads_b) && pb < pa + span(a, heads_a))) return false;
  if (tokens > 1 && a->token_stride != b->token_stride) return true;
  // a token's rows of either kind, and where the others begin among them
  const long long wa = (heads_a - 1) * a->head_stride + dim, wb = (heads_b - 1) * b->head_stride + dim;
  const long long step = a->token_stride, d = (long long)(pb - pa) / 2;
  if (tokens == 1) return d < wa && -d < wb;
  if (step <= 0) return true;
  const long long in = ((d % step) + step) % step;
  return in < wa || in + wb > step;
}

int validate_heads(int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                   int32_t dtype) {
  if (tokens < 0 || q_heads < 0 || kv_heads < 0) return MOE_ATTN_ERR_INVALID_ARG;
  if (tokens > (1 << 30)) return MOE_ATTN_ERR_TOO_MANY_TOKENS;
  if (head_dim < 1 || head_dim > 256 || q_heads > 65536 || kv_heads > 65536)
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MOE_ATTN_BF16 && dtype != MOE_ATTN_FP16) return MOE_ATTN_ERR_INVALID_ARG;
  return MOE_ATTN_OK;
}

int validate_cache8(const moe_attn_config& cfg, const moe_attn_cache8* c) {
  if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return MOE_ATTN_ERR_INVALID_ARG;
  if (cfg.head_dim % 16) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (c->num_pages < 1 || c->num_pages > 0x7ffffffeLL) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (c->page_stride <= 0 || c->token_stride <= 0 || c->head_stride <= 0 ||
      c->scale_page_stride < 0 || c->scale_head_stride < 0 || c->scale_block_stride < 0)
    return MOE_ATTN_ERR_INVALID_ARG;
  if (c->page_stride >= (1LL << 40) || c->token_stride >= (1LL << 40) ||
      c->head_stride >= (1LL << 40))
    return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;  // a tensor map's limit
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride % 16 || c->token_stride % 16 ||
      c->head_stride % 16 || ((reinterpret_cast<uintptr_t>(c->k_scales) |
                               reinterpret_cast<uintptr_t>(c->v_scales)) & 3u))
    return MOE_ATTN_ERR_MISALIGNED;
  return MOE_ATTN_OK;
}

// Whether each stride reaches past what lies within it, from `reach` elements on: no two
// places of such a view are one.
struct Dim {
  int64_t n, stride;
};
bool nested(std::initializer_list<Dim> dims, int64_t reach) {
  Dim d[3];
  int n = 0;
  for (const Dim& x : dims)
    if (x.n > 1) d[n++] = x;
  std::sort(d, d + n, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  __int128 within = reach;
  for (int i = 0; i < n; ++i) {
    if (d[i].stride < within) return false;
    within += (__int128)(d[i].n - 1) * d[i].stride;
  }
  return true;
}

// A cache that is written to: blocks whose scales or codes lie on each other, or K's on
// V's, would raise one another's scales, each by its own values.
int validate_written(const moe_attn_config& cfg, const moe_attn_cache8* c) {
  if (c->k == c->v || c->k_scales == c->v_scales) return MOE_ATTN_ERR_INVALID_ARG;
  const int64_t blocks = cfg.page_size / MOE_ATTN8_BLOCK;
  const bool ok = nested({{c->num_pages, c->scale_page_stride},
                          {cfg.kv_heads, c->scale_head_stride},
                          {blocks, c->scale_block_stride}}, 1) &&
                  nested({{c->num_pages, c->page_stride}, {cfg.kv_heads, c->head_stride},
                          {cfg.page_size, c->token_stride}}, cfg.head_dim);
  return ok ? MOE_ATTN_OK : MOE_ATTN_ERR_INVALID_ARG;
}

Cache8 cache_of(const moe_attn_cache8* c) {
  return Cache8{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scales, c->v_scales,
                c->num_pages, c->page_stride, c->token_stride, c->head_stride,
                c->scale_page_stride, c->scale_head_stride, c->scale_block_stride};
}

// 4-D view {head_dim, page_size, kv_heads, pages} of codes, boxes of `rows` rows of one
// page and head, `width` bytes wide (128 or 64: one swizzled row). What a box reaches
// past head_dim, or a page past the cache, is filled with zeros.
int encode_codes(CUtensorMap* m, const moe_attn_config& c, const moe_attn_cache8* k,
                 const void* base, int rows, int width) {
  const auto stride = [&](long long s, long long n) {
    return (cuuint64_t)(n > 1 ? s : c.head_dim);  // of a single element: free
  };
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.kv_heads, (cuuint64_t)k->num_pages};
  const cuuint64_t strides[3] = {stride(k->token_stride, c.page_size),
                                 stride(k->head_stride, c.kv_heads),
                                 stride(k->page_stride, k->num_pages)};
  const cuuint32_t box[4] = {(cuuint32_t)width, (cuuint32_t)rows, 1, 1};
  return encode(m, 4, base, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// The kernels' attributes are set in a handle's first call over an 8-bit cache (handles
// over 16 bits do without). `all`: the tensor-core kernel among them.
int make_ready(moe_attn_handle* h, bool* all) {
  int ready = h->ready8.load(std::memory_order_acquire);
  if (!ready) {
    bool usable = false;
    int st = cuda_status(attn8_decode_setup());
    if (st == MOE_ATTN_OK) st = cuda_status(attn8_tc_setup(&usable));
    if (st != MOE_ATTN_OK) return st;
    ready = usable ? 2 : 1;
    h->ready8.store(ready, std::memory_order_release);
  }
  *all = ready == 2;
  return MOE_ATTN_OK;
}

// Keys and values of a batch in 16 bits, and the page table of them: K, V, table.
struct Scratch {
  size_t half, table, total;
};
Scratch scratch_of(const moe_attn_config& c, const moe_attn_batch* b) {
  const size_t pages = (size_t)b->num_seqs * b->columns;
  Scratch s;
  s.half = align256(pages * c.kv_heads * c.page_size * c.head_dim * 2);
  s.table = 2 * s.half;
  s.total = s.table + align256(pages * 4);
  return s;
}
// Batches of many rows a sequence and kv head are worth it: bringing the keys to 16 bits
// takes the same for any number of rows, and the kernel over 16 bits is faster for each.
// Rows over 32768 keys of 8 kv heads, over codes and so: 400 108 and 113 us, 512 109 and
// 113, 1024 176 and 145, 4000 (over 65536) 1189 and 702; 8 sequences of 8192 keys: 256
// 104 and 146, 512 180 and 189, 1024 330 and 275. Those were sequences of one length; a
// batch goes one way as a whole, by its mean: a chunk beside many single tokens goes over
// codes, and beside few of them their keys are brought along.
// What it rounds: keys and values are exact in either type, but the softmax's numerators
// become bf16 in a bf16 layer (the products there take one type), 2^-8 where fp16 ones
// over codes are 2^-11: results of one batch differ in their last bits between the two.
constexpr long long kExpandRows = 512;
constexpr size_t kScratchMost = size_t(8) << 30;
bool expands(const moe_attn_config& c, const moe_attn_batch* b) {
  const long long group = c.q_heads / c.kv_heads;
  return (long long)b->max_q * group > kDecodeRows &&
         b->num_tokens * group > kExpandRows * b->num_seqs &&
         (long long)b->num_seqs * b->columns <= 0x7ffffffeLL && scratch_of(c, b).total <= kScratchMost;
}

// What moe_attn_append_norm and moe_attn_append8 have in common.
int check_append(const moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                 int32_t T, const moe_attn_rotation* r, const moe_attn_norm* norm) {
  if (!h || T < 0) return MOE_ATTN_ERR_INVALID_ARG;
  const moe_attn_config& c = h->cfg;
  if (T > c.max_tokens) return MOE_ATTN_ERR_TOO_MANY_TOKENS;
  int st = validate_rotation(r, c.head_dim);
  if (st != MOE_ATTN_OK) return st;
  if ((q == nullptr) != (q_out == nullptr)) return MOE_ATTN_ERR_INVALID_ARG;
  return norm ? validate_norm(norm, c.head_dim, q ? c.q_heads : 0, c.kv_heads) : MOE_ATTN_OK;
}
int check_append_rows(const moe_attn_config& c, const moe_attn_rows* q, const moe_attn_rows* q_out,
                      const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                      const int64_t* slots, int32_t T) {
  int st;
  if (q && (st = validate_pair(q, q_out, T, c.q_heads, c.head_dim)) != MOE_ATTN_OK) return st;
  if ((st = validate_rows(k)) != MOE_ATTN_OK || (st = validate_rows(v)) != MOE_ATTN_OK) return st;
  if (q && (share(q_out, c.q_heads, k, c.kv_heads, T, c.head_dim) ||
            share(q_out, c.q_heads, v, c.kv_heads, T, c.head_dim)))
    return MOE_ATTN_ERR_INVALID_ARG;
  return positions && slots ? MOE_ATTN_OK : MOE_ATTN_ERR_INVALID_ARG;
}
NormParams append_params(const moe_attn_handle* h, const moe_attn_rows* q,
                         const moe_attn_rows* q_out, const moe_attn_rows* k,
                         const moe_attn_rows* v, const int32_t* positions, const int64_t* slots,
                         int32_t T, const moe_attn_norm* norm, const moe_attn_rotation* r,
                         long long num_pages) {
  const moe_attn_config& c = h->cfg;
  NormParams p{};
  p.r.q = rows(q);
  p.r.q_out = rows(q_out);
  p.r.k = rows(k);
  p.r.v = rows(v);
  p.r.page_shift = log2i(c.page_size);
  p.r.num_slots = num_pages << p.r.page_shift;
  p.r.positions = positions;
  p.r.slots = reinterpret_cast<const long long*>(slots);
  p.r.r = rotation(r);
  p.r.tokens = T;
  p.r.hq = q ? c.q_heads : 0;
  p.r.hk = p.r.hv = c.kv_heads;
  p.r.head_dim = c.head_dim;
  p.r.err = h->err;
  p.n = norm_of(norm);
  return p;
}

}  // namespace

extern "C" {

int moe_attn_norm_rope(const moe_attn_rows* q, const moe_attn_rows* q_out, const moe_attn_rows* k,
                       const moe_attn_rows* k_out, const int32_t* positions, int32_t T,
                       int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                       const moe_attn_norm* norm, const moe_attn_rotation* r, void* stream) {
  int st = validate_heads(T, q_heads, kv_heads, head_dim, dtype);
  if (st != MOE_ATTN_OK) return st;
  if ((st = validate_rotation(r, head_dim)) != MOE_ATTN_OK) return st;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return MOE_ATTN_ERR_INVALID_ARG;
  const int hq = q ? q_heads : 0, hk = k ? kv_heads : 0;
  if ((st = validate_norm(norm, head_dim, hq, hk)) != MOE_ATTN_OK) return st;
  if (T == 0 || hq + hk == 0) return MOE_ATTN_OK;
  if (hq && (st = validate_pair(q, q_out, T, hq, head_dim)) != MOE_ATTN_OK) return st;
  if (hk && (st = validate_pair(k, k_out, T, hk, head_dim)) != MOE_ATTN_OK) return st;
  if (!positions) return MOE_ATTN_ERR_INVALID_ARG;
  // an output is written while the other's input is read
  if (hq && hk &&
      (share(q_out, hq, k, hk, T, head_dim) || share(k_out, hk, q, hq, T, head_dim) ||
       share(q_out, hq, k_out, hk, T, head_dim)))
    return MOE_ATTN_ERR_INVALID_ARG;
  NormParams p{};
  p.r.q = rows(hq ? q : nullptr);
  p.r.q_out = rows(hq ? q_out : nullptr);
  p.r.k = rows(hk ? k : nullptr);
  p.k_out = rows(hk ? k_out : nullptr);
  p.r.positions = positions;
  p.r.r = rotation(r);
  p.r.tokens = T;
  p.r.hq = hq;
  p.r.hk = hk;
  p.r.head_dim = head_dim;
  p.n = norm_of(norm);
  return cuda_status(launch_norm_rope(p, dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_norm_rope_backward_bytes(int32_t T, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, size_t* bytes) {
  if (!bytes) return MOE_ATTN_ERR_INVALID_ARG;
  const int st = validate_heads(T, q_heads, kv_heads, head_dim, MOE_ATTN_BF16);
  if (st != MOE_ATTN_OK) return st;
  *bytes = T && q_heads + kv_heads ? norm_grad_bytes(T, q_heads + kv_heads, head_dim) : 0;
  return MOE_ATTN_OK;
}

int moe_attn_norm_rope_backward(const moe_attn_rows* dq, const moe_attn_rows* q,
                                const moe_attn_rows* dx_q, float* dw_q, const moe_attn_rows* dk,
                                const moe_attn_rows* k, const moe_attn_rows* dx_k, float* dw_k,
                                const int32_t* positions, int32_t T, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                const moe_attn_norm* norm, const moe_attn_rotation* r,
                                void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate_heads(T, q_heads, kv_heads, head_dim, dtype);
  if (st != MOE_ATTN_OK) return st;
  if ((st = validate_rotation(r, head_dim)) != MOE_ATTN_OK) return st;
  const bool with_q = q || dq || dx_q || dw_q, with_k = k || dk || dx_k || dw_k;
  const int hq = with_q ? q_heads : 0, hk = with_k ? kv_heads : 0;
  if ((st = validate_norm(norm, head_dim, hq, hk)) != MOE_ATTN_OK) return st;
  if ((hq && !dw_q) || (hk && !dw_k)) return MOE_ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dw_q) | reinterpret_cast<uintptr_t>(dw_k)) & 3u)
    return MOE_ATTN_ERR_MISALIGNED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // no token, or no head that has the weight: no gradient of it
  const struct {
    float* dw;
    int64_t stride;
    int heads;
  } weights[2] = {{dw_q, norm->q_head_stride, hq}, {dw_k, norm->k_head_stride, hk}};
  for (const auto& w : weights) {
    const size_t bytes = (size_t)(w.stride ? w.heads : 1) * head_dim * sizeof(float);
    if (w.dw && (T == 0 || w.heads == 0) && bytes &&
        (st = cuda_status(cudaMemsetAsync(w.dw, 0, bytes, s))) != MOE_ATTN_OK)
      return st;
  }
  if (T == 0 || hq + hk == 0) return MOE_ATTN_OK;
  const struct {
    const moe_attn_rows *dy, *x, *dx;
    int heads;
  } both[2] = {{dq, q, dx_q, hq}, {dk, k, dx_k, hk}};
  for (const auto& b : both) {
    if (!b.heads) continue;
    if ((st = validate_pair(b.dy, b.dx, T, b.heads, head_dim)) != MOE_ATTN_OK ||
        (st = validate_pair(b.x, b.dx, T, b.heads, head_dim)) != MOE_ATTN_OK)
      return st;
  }
  if (hq && hk &&
      (share(dx_q, hq, k, hk, T, head_dim) || share(dx_q, hq, dk, hk, T, head_dim) ||
       share(dx_k, hk, q, hq, T, head_dim) || share(dx_k, hk, dq, hq, T, head_dim) ||
       share(dx_q, hq, dx_k, hk, T, head_dim)))
    return MOE_ATTN_ERR_INVALID_ARG;
  if (!positions || !workspace || workspace_bytes < norm_grad_bytes(T, hq + hk, head_dim))
    return MOE_ATTN_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return MOE_ATTN_ERR_MISALIGNED;
  NormGradParams g{};
  g.p.r.q = rows(hq ? q : nullptr);
  g.p.r.q_out = rows(hq ? dx_q : nullptr);
  g.p.r.k = rows(hk ? k : nullptr);
  g.p.k_out = rows(hk ? dx_k : nullptr);
  g.dq = rows(hq ? dq : nullptr);
  g.dk = rows(hk ? dk : nullptr);
  g.p.r.positions = positions;
  g.p.r.r = rotation(r);
  g.p.r.r.sign = -g.p.r.r.sign;  // the opposite rotation
  g.p.r.tokens = T;
  g.p.r.hq = hq;
  g.p.r.hk = hk;
  g.p.r.head_dim = head_dim;
  g.p.n = norm_of(norm);
  g.dw_q = dw_q;
  g.dw_k = dw_k;
  g.parts = static_cast<float*>(workspace);
  return cuda_status(launch_norm_rope_grad(g, dtype, s));
}

int moe_attn_append_norm(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                         const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                         const int64_t* slots, int32_t T, const moe_attn_norm* norm,
                         const moe_attn_rotation* r, const moe_attn_cache* cache, void* stream) {
  if (!norm) return MOE_ATTN_ERR_INVALID_ARG;
  int st = check_append(h, q, q_out, T, r, norm);
  if (st != MOE_ATTN_OK || (st = validate_cache(cache)) != MOE_ATTN_OK || T == 0) return st;
  if ((st = check_append_rows(h->cfg, q, q_out, k, v, positions, slots, T)) != MOE_ATTN_OK)
    return st;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  NormParams p = append_params(h, q, q_out, k, v, positions, slots, T, norm, r, cache->num_pages);
  p.r.k_pages = static_cast<uint16_t*>(cache->k);
  p.r.v_pages = static_cast<uint16_t*>(cache->v);
  p.r.page_stride = cache->page_stride;
  p.r.token_stride = cache->token_stride;
  p.r.head_stride = cache->head_stride;
  return cuda_status(launch_norm_rope(p, h->cfg.dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_append8(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                     const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                     const int64_t* slots, int32_t T, const moe_attn_norm* norm,
                     const moe_attn_rotation* r, const moe_attn_cache8* cache, void* stream) {
  int st = check_append(h, q, q_out, T, r, norm);
  if (st != MOE_ATTN_OK || (st = validate_cache8(h->cfg, cache)) != MOE_ATTN_OK ||
      (st = validate_written(h->cfg, cache)) != MOE_ATTN_OK || T == 0)
    return st;
  if ((st = check_append_rows(h->cfg, q, q_out, k, v, positions, slots, T)) != MOE_ATTN_OK)
    return st;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  Append8Params g{};
  g.p = append_params(h, q, q_out, k, v, positions, slots, T, norm, r, cache->num_pages);
  g.c = cache_of(cache);
  return cuda_status(launch_append8(g, h->cfg.dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_read8(moe_attn_handle* h, const moe_attn_cache8* cache, const moe_attn_extent* e,
                   const moe_attn_rows* k_out, const moe_attn_rows* v_out, void* stream) {
  if (!h || !e || e->num_seqs < 0 || e->num_rows < 0) return MOE_ATTN_ERR_INVALID_ARG;
  const moe_attn_config& c = h->cfg;
  if (e->num_seqs > c.max_seqs || e->num_rows > (1 << 30)) return MOE_ATTN_ERR_TOO_MANY_TOKENS;
  int st = validate_cache8(c, cache);
  if (st != MOE_ATTN_OK || e->num_seqs == 0 || e->num_rows == 0) return st;
  if ((st = validate_rows(k_out)) != MOE_ATTN_OK || (st = validate_rows(v_out)) != MOE_ATTN_OK)
    return st;
  if (!apart(k_out, e->num_rows, c.kv_heads, c.head_dim) ||
      !apart(v_out, e->num_rows, c.kv_heads, c.head_dim) ||
      share(k_out, c.kv_heads, v_out, c.kv_heads, e->num_rows, c.head_dim))
    return MOE_ATTN_ERR_INVALID_ARG;
  if (!e->cu_rows || !e->first || !e->page_table || e->columns < 1 || e->table_stride < e->columns)
    return MOE_ATTN_ERR_INVALID_ARG;
  if ((long long)e->columns * c.page_size > (1LL << 29)) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  Read8Params p{};
  p.c = cache_of(cache);
  p.cu = e->cu_rows;
  p.first = e->first;
  p.page_table = e->page_table;
  p.table_stride = e->table_stride;
  p.columns = e->columns;
  p.num_seqs = e->num_seqs;
  p.rows = e->num_rows;
  p.hk = c.kv_heads;
  p.head_dim = c.head_dim;
  p.page_shift = log2i(c.page_size);
  p.k_out = rows(k_out);
  p.v_out = rows(v_out);
  p.err = h->err;
  return cuda_status(launch_read8(p, c.dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_forward8_scratch_bytes(const moe_attn_handle* h, const moe_attn_batch* b,
                                    size_t* bytes) {
  if (!h || !b || !bytes) return MOE_ATTN_ERR_INVALID_ARG;
  *bytes = 0;
  if (b->num_tokens > 0 && b->num_seqs > 0 && b->columns > 0 && expands(h->cfg, b))
    *bytes = scratch_of(h->cfg, b).total;
  return MOE_ATTN_OK;
}

int moe_attn_forward8(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                      float* lse, const moe_attn_cache8* cache, const moe_attn_batch* b,
                      const moe_attn_scores* sc, int32_t sinks, void* scratch,
                      size_t scratch_bytes, void* stream) {
  int st = check_call(h, b, sc, sinks);
  if (st != MOE_ATTN_OK) return st;
  const moe_attn_config& c = h->cfg;
  if ((st = validate_cache8(c, cache)) != MOE_ATTN_OK) return st;
  if (b->num_tokens == 0 || b->num_seqs == 0) return MOE_ATTN_OK;
  if ((st = check_batch(c, q, out, b)) != MOE_ATTN_OK) return st;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  Attn8Params p{};
  p.a = params_of(h, q, out, lse, cache->num_pages, b, sc, sinks);
  p.c = cache_of(cache);
  p.dtype = c.dtype;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (scratch && expands(c, b) && h->tc_usable) {
    const Scratch room = scratch_of(c, b);
    if (scratch_bytes < room.total) return MOE_ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(scratch) & 255u) return MOE_ATTN_ERR_MISALIGNED;
    uint8_t* at = static_cast<uint8_t*>(scratch);
    Expand8Params e{};
    e.c = p.c;
    e.b = p.a.b;
    e.sc = p.a.sc;
    e.k = reinterpret_cast<uint16_t*>(at);
    e.v = reinterpret_cast<uint16_t*>(at + room.half);
    e.table = reinterpret_cast<int*>(at + room.table);
    e.hk = c.kv_heads;
    e.head_dim = c.head_dim;
    e.page_shift = p.a.page_shift;
    e.err = h->err;
    if ((st = cuda_status(launch_expand8(e, c.dtype, h->grid, s))) != MOE_ATTN_OK) return st;
    const int64_t row = c.head_dim, head = row * c.page_size;
    const moe_attn_cache wide = {e.k, e.v, (int64_t)b->num_seqs * b->columns, head * c.kv_heads,
                                 row, head};
    p.a.num_pages = wide.num_pages;
    p.a.b.page_table = e.table;
    p.a.b.table_stride = b->columns;
    return forward_many(h, p.a, q, &wide, s);
  }
  bool all;
  if ((st = make_ready(h, &all)) != MOE_ATTN_OK) return st;
  // as in moe_attn_forward: one kernel for the whole batch
  CUtensorMap qmap, kmap, vmap;
  const bool few = (long long)b->max_q * p.a.group <= kDecodeRows;
  const int chunks = c.head_dim > 64 ? 2 : 1;
  const int block = few ? decode8_block(chunks) : kTcBlock;
  const int box = c.page_size < block ? c.page_size : block;
  const int width = few ? 64 * chunks : 128;
  if ((st = encode_codes(&kmap, c, cache, cache->k, box, width)) != MOE_ATTN_OK ||
      (st = encode_codes(&vmap, c, cache, cache->v, box, width)) != MOE_ATTN_OK)
    return st;
  if (few) return cuda_status(launch_attn8_decode(p, h->decode, kmap, vmap, h->grid, s));
  if (!all) {  // another compiler: few-token batches go on
    fprintf(stderr, "moe_attn: the tensor-core kernel was built with other registers than it needs\n");
    return MOE_ATTN_ERR_CUDA;
  }
  if ((st = encode_q(&qmap, c, q, b->num_tokens)) != MOE_ATTN_OK) return st;
  return cuda_status(launch_attn8_tc(p, h->tc, qmap, kmap, vmap, h->grid, s));
}

int moe_attn_forward_sinks(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                           float* lse, const moe_attn_cache* cache, const moe_attn_batch* b,
                           const moe_attn_scores* sc, int32_t sinks, void* stream) {
  return forward_sinks(h, q, out, lse, cache, b, sc, sinks, stream);
}

}  // extern "C"
