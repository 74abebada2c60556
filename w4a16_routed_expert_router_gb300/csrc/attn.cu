// C ABI of the attention operators: argument validation, workspace, dispatch.
#include <new>

#include "attn_host.h"

namespace {

// Workspace carve-up; the order is the order of the fields filled in create().
struct Layout {
  size_t off[7], sizes[7];
  size_t total;
};
Layout plan(const moe_attn_config& c) {
  const size_t d = c.head_dim > 64 ? 128 : 64;
  const size_t sizes[] = {
      4,                                        // 0 err
      kMaxGrid * 4,                             // 1 decode: pieces that arrived
      kMaxGrid * 2 * kDecodeRows * 8,           // 2 decode: maximum, sum
      kMaxGrid * 2 * kDecodeRows * d * 4,       // 3 decode: weighted sums
      kMaxGrid * 4 * 4,                         // 4 tensor cores: halves that arrived
      kMaxGrid * 4 * 128 * 8,                   // 5 maximum, sum
      kMaxGrid * 4 * 128 * d * 4,               // 6 weighted sums
  };
  Layout L;
  size_t o = 0;
  for (size_t i = 0; i < sizeof(sizes) / sizeof(sizes[0]); ++i) {
    L.off[i] = o;
    L.sizes[i] = sizes[i];
    o += align256(sizes[i]);
  }
  L.total = o;
  return L;
}

// 4-D view {head_dim, page_size, kv_heads, pages} of K or V, boxes of `rows`
// rows of one page and head, 64 values wide, 128-byte swizzle. A box that
// reaches past head_dim, or a page past the cache, is filled with zeros.
int encode_cache(CUtensorMap* m, const moe_attn_config& c, const moe_attn_cache* k,
                 const void* base, int rows) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.kv_heads, (cuuint64_t)k->num_pages};
  const cuuint64_t strides[3] = {bytes_of(k->token_stride, c.page_size, c.head_dim),
                                 bytes_of(k->head_stride, c.kv_heads, c.head_dim),
                                 bytes_of(k->page_stride, k->num_pages, c.head_dim)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  return encode(m, 4, base, dims, strides, box);
}

// The same with the chunks of 64 values as a dimension behind the rows: where
// head_dim is 128, one box brings both, [chunk][row][64 values]. Otherwise that
// dimension has one element and a box one chunk, as above.
int encode_cache_chunks(CUtensorMap* m, const moe_attn_config& c, const moe_attn_cache* k,
                        const void* base, int rows) {
  const bool both = c.head_dim == 128;
  const cuuint64_t dims[5] = {(cuuint64_t)(both ? 64 : c.head_dim), (cuuint64_t)c.page_size,
                              (cuuint64_t)(both ? 2 : 1), (cuuint64_t)c.kv_heads,
                              (cuuint64_t)k->num_pages};
  const cuuint64_t strides[4] = {bytes_of(k->token_stride, c.page_size, c.head_dim), 128,
                                 bytes_of(k->head_stride, c.kv_heads, c.head_dim),
                                 bytes_of(k->page_stride, k->num_pages, c.head_dim)};
  const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)(both ? 2 : 1), 1, 1};
  return encode(m, 5, base, dims, strides, box);
}

// The tensor-core kernel's boxes of K or V. Heads of 128 values in 16-token pages
// that follow each other evenly: {64, 8 rows, 2 chunks, groups of 8 rows, (page,
// head) or head}, a box for a page with both chunks; otherwise the 4-D view, a
// box for each chunk. The number of boxes bounds caches of small pages (prefill
// of 8192 tokens: 417 us by chunks, 366 us so; from 32-token pages on 364 and
// 367 us, no difference).
Boxes tc_boxes(const moe_attn_config& c, const moe_attn_cache* k) {
  Boxes b{};
  if (c.head_dim != 128 || c.page_size > 16) return b;
  const int groups = c.page_size / 8;
  if ((c.kv_heads == 1 || k->page_stride == c.kv_heads * k->head_stride || k->num_pages == 1) &&
      k->num_pages * c.kv_heads < 0x7fffffffLL - c.kv_heads) {
    b = Boxes{1, 0, c.kv_heads};      // [pages, heads, page, values]
  } else if (k->page_stride == c.page_size * k->token_stride &&
             k->num_pages * groups < 0x7fffffffLL - groups) {
    b = Boxes{1, groups, 0};          // [pages, page, heads, values]
  }
  return b;
}

int encode_tc_cache(CUtensorMap* m, const moe_attn_config& c, const moe_attn_cache* k,
                    const void* base, const Boxes& b) {
  const int rows = c.page_size < kTcBlock ? c.page_size : kTcBlock;
  if (!b.both) return encode_cache(m, c, k, base, rows);
  const bool by_page = b.page_groups == 0;
  const long long heads = by_page ? k->num_pages * c.kv_heads : c.kv_heads;
  const cuuint64_t token = bytes_of(k->token_stride, c.page_size, c.head_dim);
  const long long head_stride = by_page && c.kv_heads == 1 ? k->page_stride : k->head_stride;
  const cuuint64_t dims[5] = {64, 8, 2,
                              (cuuint64_t)(by_page ? 1 : k->num_pages) * (c.page_size / 8),
                              (cuuint64_t)heads};
  const cuuint64_t strides[4] = {token, 128, 8 * token, bytes_of(head_stride, heads, c.head_dim)};
  const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)rows / 8, 1};
  return encode(m, 5, base, dims, strides, box);
}

}  // namespace

int moe::attn::forward_many(moe_attn_handle* h, AttnParams p, const moe_attn_rows* q,
                            const moe_attn_cache* cache, cudaStream_t s) {
  const moe_attn_config& c = h->cfg;
  CUtensorMap qmap, kmap, vmap;
  int st;
  if (!h->tc_usable) {  // another compiler: few-token batches go on
    fprintf(stderr, "moe_attn: the tensor-core kernel was built with other registers than it needs\n");
    return MOE_ATTN_ERR_CUDA;
  }
  p.boxes = tc_boxes(c, cache);
  if ((st = encode_tc_cache(&kmap, c, cache, cache->k, p.boxes)) != MOE_ATTN_OK ||
      (st = encode_tc_cache(&vmap, c, cache, cache->v, p.boxes)) != MOE_ATTN_OK ||
      (st = encode_q(&qmap, c, q, p.b.num_tokens)) != MOE_ATTN_OK)
    return st;
  return cuda_status(launch_attn_tc(p, h->tc, qmap, kmap, vmap, c.dtype, h->grid, s));
}

int moe::attn::forward_sinks(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                             float* lse, const moe_attn_cache* cache, const moe_attn_batch* b,
                             const moe_attn_scores* sc, int sinks, void* stream) {
  int st = check_call(h, b, sc, sinks);
  if (st != MOE_ATTN_OK) return st;
  const moe_attn_config& c = h->cfg;
  if ((st = validate_cache(cache)) != MOE_ATTN_OK) return st;
  // (with a max_q of 0 the device finds out whether the sequences are empty)
  if (b->num_tokens == 0 || b->num_seqs == 0) return MOE_ATTN_OK;
  if ((st = check_batch(c, q, out, b)) != MOE_ATTN_OK) return st;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  AttnParams p = params_of(h, q, out, lse, cache->num_pages, b, sc, sinks);
  // One kernel takes the whole batch: the few-token kernel where every sequence
  // has few rows, else the tensor-core kernel, whose single tokens run beside the
  // chunks (16 sequences, 4 of them chunks, 104 us in two launches, 90 us so).
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((long long)b->max_q * p.group <= kDecodeRows) {
    CUtensorMap kmap, vmap;
    const int block = decode_block(c.head_dim > 64 ? 2 : 1);
    const int box = c.page_size < block ? c.page_size : block;
    if ((st = encode_cache_chunks(&kmap, c, cache, cache->k, box)) != MOE_ATTN_OK ||
        (st = encode_cache_chunks(&vmap, c, cache, cache->v, box)) != MOE_ATTN_OK)
      return st;
    return cuda_status(launch_attn_decode(p, h->decode, kmap, vmap, c.dtype, h->grid, s));
  }
  return forward_many(h, p, q, cache, s);
}

extern "C" {

int moe_attn_rope_frequencies(int32_t rot_dim, double base, double factor, int32_t by_parts,
                              double original_len, double beta_fast, double beta_slow,
                              int64_t* freq, float* magnitude) {
  if (!magnitude || (rot_dim > 0 && !freq)) return MOE_ATTN_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > 256 || rot_dim % 2) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
    return MOE_ATTN_ERR_INVALID_ARG;
  if (by_parts != 0 && by_parts != 1) return MOE_ATTN_ERR_INVALID_ARG;
  if (by_parts && !(original_len > 0.0 && std::isfinite(original_len) && beta_slow >= 0.0 &&
                    beta_fast > beta_slow && std::isfinite(beta_fast)))
    return MOE_ATTN_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double theta = std::pow(base, -2.0 * i / rot_dim);
    if (by_parts) {
      double keep = (original_len * theta / two_pi - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      theta = theta * keep + theta / factor * (1.0 - keep);
    } else {
      theta /= factor;
    }
    // theta <= 1 radian: below 2^62, inside int64
    freq[i] = (int64_t)std::ldexp(theta / two_pi, 64);
  }
  *magnitude = by_parts && factor > 1.0 ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
  return MOE_ATTN_OK;
}

int moe_attn_rope(const moe_attn_rows* x, const moe_attn_rows* out, const int32_t* positions,
                  int32_t T, int32_t heads, int32_t head_dim, int32_t dtype,
                  const moe_attn_rotation* r, void* stream) {
  if (T < 0 || heads < 0) return MOE_ATTN_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 256 || heads > 65536) return MOE_ATTN_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MOE_ATTN_BF16 && dtype != MOE_ATTN_FP16) return MOE_ATTN_ERR_INVALID_ARG;
  int st = validate_rotation(r, head_dim);
  if (st != MOE_ATTN_OK) return st;
  if (T == 0 || heads == 0) return MOE_ATTN_OK;
  if ((st = validate_rows(x)) != MOE_ATTN_OK || (st = validate_rows(out)) != MOE_ATTN_OK) return st;
  if (!positions) return MOE_ATTN_ERR_INVALID_ARG;
  if (!apart(out, T, heads, head_dim) ||
      (!same(x, out) && overlap(x, out, T, heads, head_dim)))
    return MOE_ATTN_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = rows(x);
  p.q_out = rows(out);
  p.positions = positions;
  p.r = rotation(r);
  p.tokens = T;
  p.hq = heads;
  p.head_dim = head_dim;
  return cuda_status(launch_rope(p, dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_workspace_bytes(const moe_attn_config* cfg, size_t* bytes) {
  if (!bytes) return MOE_ATTN_ERR_INVALID_ARG;
  const int st = validate_config(cfg);
  if (st != MOE_ATTN_OK) return st;
  *bytes = plan(*cfg).total;
  return MOE_ATTN_OK;
}

int moe_attn_create(const moe_attn_config* cfg, int device, moe_attn_handle** out) {
  if (!out) return MOE_ATTN_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_config(cfg);
  if (st != MOE_ATTN_OK) return st;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev <= 0) {
    cudaGetLastError();
    return MOE_ATTN_ERR_NO_DEVICE;
  }
  if (device < 0 || device >= ndev) return MOE_ATTN_ERR_INVALID_ARG;
  cudaDeviceProp prop;
  if ((st = cuda_status(cudaGetDeviceProperties(&prop, device))) != MOE_ATTN_OK) return st;
  if (prop.major != 10 || prop.minor != 3) return MOE_ATTN_ERR_NO_DEVICE;
  const OnDevice on(device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  moe_attn_handle* h = new (std::nothrow) moe_attn_handle();
  if (!h) return MOE_ATTN_ERR_CUDA;
  h->cfg = *cfg;
  h->device = device;
  h->num_sms = prop.multiProcessorCount;
  h->grid = h->num_sms < kMaxGrid ? h->num_sms : kMaxGrid;
  const Layout L = plan(*cfg);
  if ((st = cuda_status(attn_decode_setup())) != MOE_ATTN_OK ||
      (st = cuda_status(attn_tc_setup(&h->tc_usable))) != MOE_ATTN_OK ||
      (st = cuda_status(cudaMalloc(&h->ws, L.total))) != MOE_ATTN_OK ||
      (st = cuda_status(cudaMemset(h->ws, 0, L.total))) != MOE_ATTN_OK ||
      // cudaMemset does not wait, and other streams do not wait for it
      (st = cuda_status(cudaDeviceSynchronize())) != MOE_ATTN_OK) {
    moe_attn_destroy(h);
    return st;
  }
  uint8_t* b = static_cast<uint8_t*>(h->ws);
  h->err = reinterpret_cast<unsigned*>(b + L.off[0]);
  h->decode.count = reinterpret_cast<unsigned*>(b + L.off[1]);
  h->decode.ml = reinterpret_cast<float2*>(b + L.off[2]);
  h->decode.o = reinterpret_cast<float*>(b + L.off[3]);
  h->tc.count = reinterpret_cast<unsigned*>(b + L.off[4]);
  h->tc.ml = reinterpret_cast<float2*>(b + L.off[5]);
  h->tc.o = reinterpret_cast<float*>(b + L.off[6]);
  *out = h;
  return MOE_ATTN_OK;
}

int moe_attn_destroy(moe_attn_handle* h) {
  if (!h) return MOE_ATTN_OK;
  const OnDevice on(h->device);
  cudaDeviceSynchronize();
  if (h->ws) cudaFree(h->ws);
  delete h;
  return MOE_ATTN_OK;
}

int moe_attn_append(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                    const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                    const int64_t* slots, int32_t T, const moe_attn_rotation* r,
                    const moe_attn_cache* cache, void* stream) {
  if (!h || T < 0) return MOE_ATTN_ERR_INVALID_ARG;
  const moe_attn_config& c = h->cfg;
  if (T > c.max_tokens) return MOE_ATTN_ERR_TOO_MANY_TOKENS;
  int st = validate_rotation(r, c.head_dim);
  if (st != MOE_ATTN_OK) return st;
  if ((st = validate_cache(cache)) != MOE_ATTN_OK) return st;
  if ((q == nullptr) != (q_out == nullptr)) return MOE_ATTN_ERR_INVALID_ARG;
  if (T == 0) return MOE_ATTN_OK;
  if (q && ((st = validate_rows(q)) != MOE_ATTN_OK || (st = validate_rows(q_out)) != MOE_ATTN_OK))
    return st;
  if ((st = validate_rows(k)) != MOE_ATTN_OK || (st = validate_rows(v)) != MOE_ATTN_OK) return st;
  if (!positions || !slots) return MOE_ATTN_ERR_INVALID_ARG;
  if (q && (!apart(q_out, T, c.q_heads, c.head_dim) ||
            (!same(q, q_out) && overlap(q, q_out, T, c.q_heads, c.head_dim))))
    return MOE_ATTN_ERR_INVALID_ARG;
  const OnDevice on(h->device);
  if ((st = on.status()) != MOE_ATTN_OK) return st;
  RopeParams p{};
  p.q = rows(q);
  p.q_out = rows(q_out);
  p.k = rows(k);
  p.v = rows(v);
  p.k_pages = static_cast<uint16_t*>(cache->k);
  p.v_pages = static_cast<uint16_t*>(cache->v);
  p.page_shift = log2i(c.page_size);
  p.num_slots = cache->num_pages << p.page_shift;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.positions = positions;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.r = rotation(r);
  p.tokens = T;
  p.hq = q ? c.q_heads : 0;
  p.hk = p.hv = c.kv_heads;
  p.head_dim = c.head_dim;
  p.err = h->err;
  return cuda_status(launch_rope(p, c.dtype, static_cast<cudaStream_t>(stream)));
}

int moe_attn_forward(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                     float* lse, const moe_attn_cache* cache, const moe_attn_batch* b,
                     const moe_attn_scores* sc, void* stream) {
  return forward_sinks(h, q, out, lse, cache, b, sc, 0, stream);
}

int moe_attn_check_device_errors(moe_attn_handle* h, uint32_t* flags) {
  if (!h || !flags) return MOE_ATTN_ERR_INVALID_ARG;
  *flags = 0;
  const OnDevice on(h->device);
  int st = on.status();
  if (st != MOE_ATTN_OK) return st;
  if ((st = cuda_status(cudaDeviceSynchronize())) != MOE_ATTN_OK) return st;
  uint32_t v = 0;
  if ((st = cuda_status(cudaMemcpy(&v, h->err, 4, cudaMemcpyDeviceToHost))) != MOE_ATTN_OK)
    return st;
  // A launch that gave up leaves counters of joins raised, which only the second
  // half of a pair resets; the next launch would take old sums for that half.
  if (v & kErrTimeout) {
    const Layout L = plan(h->cfg);
    uint8_t* b = static_cast<uint8_t*>(h->ws);
    for (int i : {1, 4})
      if ((st = cuda_status(cudaMemset(b + L.off[i], 0, L.sizes[i]))) != MOE_ATTN_OK) return st;
  }
  // and a bit that the next launch sets must not be cleared by a late memset
  if (v && ((st = cuda_status(cudaMemset(h->err, 0, 4))) != MOE_ATTN_OK ||
            (st = cuda_status(cudaDeviceSynchronize())) != MOE_ATTN_OK))
    return st;
  *flags = v;
  return v ? MOE_ATTN_ERR_DEVICE : MOE_ATTN_OK;
}

}  // extern "C"
