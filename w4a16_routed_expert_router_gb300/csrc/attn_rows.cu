// Attention over the paged cache, one warp per (token, query head): the
// definition with a running maximum and sum, every key read once per row. The
// plain kernel the others are checked against; bound by issue slots.
#include "attn.h"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attn_rows_kernel(const AttnParams p) {
  const int lane = threadIdx.x & 31;
  const long long job = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (job >= (long long)p.b.num_tokens * p.hq) return;
  const int tok = (int)(job / p.hq), h = (int)(job - (long long)tok * p.hq);
  // sequence of this token: the last one that begins at or before it
  int lo = 0, hi = p.b.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.b.cu_q[mid] <= tok)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int first = p.b.cu_q[lo], n = p.b.cu_q[lo + 1] - first;
  const int kv = p.b.kv_len[lo];
  if (n >= 0 && (tok < first || tok >= first + n)) return;
  if (n < 0 || kv < 0 || kv > (p.b.columns << p.page_shift) || n > p.b.max_q) {
    if (lane == 0) atomicOr(p.err, kErrRange);
    return;
  }
  if (n * p.group <= kDecodeRows) return;
  const int pos = kv - n + (tok - first);
  const int prefix = p.sc.prefix ? min(kv, max(0, p.sc.prefix[lo])) : 0;
  const float slope = p.sc.slopes ? p.sc.slopes[h] : 0.0f;
  const uint16_t* q = p.q.p + (long long)tok * p.q.token + (long long)h * p.q.head;
  float qv[4], acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane + 32 * i;
    qv[i] = d < p.head_dim ? T::to_f32(q[d]) : 0.0f;
    acc[i] = 0.0f;
  }
  const int* table = p.b.page_table + (long long)lo * p.b.table_stride;
  const int mask = (1 << p.page_shift) - 1;
  float m = -INFINITY, l = 0.0f;
  const int end = max(min(pos + 1, kv), prefix);
  for (int j = 0; j < end; ++j) {
    const bool seen = j < prefix || (j <= pos && (p.sc.window == 0 || j > pos - p.sc.window));
    if (!seen) continue;
    const int page = table[j >> p.page_shift];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(p.err, kErrRange);
      return;
    }
    const long long row = (long long)page * p.page_stride + (long long)(j & mask) * p.token_stride +
                          (long long)(h / p.group) * p.head_stride;
    float x = 0.0f, vv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = lane + 32 * i;
      const bool in = d < p.head_dim;
      x = fmaf(qv[i], in ? T::to_f32(p.k_pages[row + d]) : 0.0f, x);
      vv[i] = in ? T::to_f32(p.v_pages[row + d]) : 0.0f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= p.sc.scale;
    if (p.sc.softcap > 0.0f) x = p.sc.softcap * tanhf(x / p.sc.softcap);
    x -= slope * (float)abs(pos - j);
    const float m2 = fmaxf(m, x);
    const float base = m2 == -INFINITY ? 0.0f : m2;
    const float a = expf(m - base), e = expf(x - base);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = acc[i] * a + e * vv[i];
    m = m2;
  }
  uint16_t* o = p.out.p + (long long)tok * p.out.token + (long long)h * p.out.head;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane + 32 * i;
    if (d < p.head_dim) o[d] = T::from_f32(acc[i] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[(long long)tok * p.hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnParams& p, int dtype, cudaStream_t s) {
  const long long jobs = (long long)p.b.num_tokens * p.hq;
  const unsigned grid = (unsigned)((jobs + kWarps - 1) / kWarps);
  if (dtype == MOE_ATTN_BF16)
    attn_rows_kernel<Bf16><<<grid, kWarps * 32, 0, s>>>(p);
  else
    attn_rows_kernel<Fp16><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
