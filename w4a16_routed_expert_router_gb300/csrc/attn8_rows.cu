// Attention over an 8-bit cache, a warp for each query row (token, head): 4 values of
// a head to a lane, keys one after the other.
#include "attn_common.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void values4(uint32_t w, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) attn8_rows_kernel(const Attn8Params g) {
  const AttnParams& p = g.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int token = blockIdx.x, h = blockIdx.y * kWarps + warp;
  if (h >= p.hq) return;
  Span s{};
  int seq = 0;
  for (; seq < p.b.num_seqs; ++seq) {
    s = read_sequence(p.b, p.page_shift, seq, p.err);
    if (s.n > 0 && token >= s.first && token < s.first + s.n) break;
  }
  if (seq == p.b.num_seqs) return;
  const int pos = s.kv - s.n + token - s.first, hk = h / p.group;
  const int prefix = prefix_of(p.sc, seq, s.kv), kept = kept_of(p.sc, prefix, pos);
  const float slope = p.sc.slopes ? p.sc.slopes[h] : 0.0f;
  const int c = lane * 4;
  const bool on = c < p.head_dim;
  float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
  if (on)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = T::to_f32(p.q.p[(long long)token * p.q.token + (long long)h * p.q.head + c + i]);
  const int end = min(s.kv, max(pos + 1, prefix));
  const int from = p.sc.window ? max(0, pos - p.sc.window + 1) : 0;
  for (int j = 0; j < end; ++j) {
    if (j >= kept && j < from) j = from;
    if (j >= end) break;
    const int page = p.b.page_table[seq * p.b.table_stride + (j >> p.page_shift)];
    float k[4] = {}, v[4] = {};
    if (page < 0 || page >= p.num_pages) {
      atomicOr(p.err, kErrRange);
    } else if (on) {
      const int row = j & ((1 << p.page_shift) - 1);
      const long long at = page * g.c.page + (long long)hk * g.c.head + row * g.c.token + c;
      const long long sc = page * g.c.scale_page + hk * g.c.scale_head +
                           row / kScaleBlock * g.c.scale_block;
      values4(*reinterpret_cast<const uint32_t*>(g.c.k + at), g.c.k_scales[sc], k);
      values4(*reinterpret_cast<const uint32_t*>(g.c.v + at), g.c.v_scales[sc], v);
    }
    float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x = p.sc.softcap > kWideCap ? score<kWide>(p.sc, x, slope, pos - j)
                                : score<kGeneral>(p.sc, x, slope, pos - j);
    const float m2 = fmaxf(m, x), base = m2 == -INFINITY ? 0.0f : m2;
    const float a = ex2(m - base), b = ex2(x - base);
    m = m2;
    l = l * a + b;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * a + v[i] * b;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (on)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p.out.p[(long long)token * p.out.token + (long long)h * p.out.head + c + i] =
          T::from_f32(o[i] * inv);
  if (p.lse && lane == 0)
    p.lse[(long long)token * p.hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_attn8_rows(const Attn8Params& g, cudaStream_t s) {
  const dim3 grid(g.a.b.num_tokens, (g.a.hq + kWarps - 1) / kWarps), block(kWarps * 32);
  if (g.dtype == MOE_ATTN_BF16)
    attn8_rows_kernel<Bf16><<<grid, block, 0, s>>>(g);
  else
    attn8_rows_kernel<Fp16><<<grid, block, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
