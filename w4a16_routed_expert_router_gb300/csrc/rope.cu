// Rotary positions, alone or with the append of keys and values to a paged
// cache.
//
// The angle of pair i at position p is 2 pi frac(p * freq[i] / 2^64): the
// product wraps as a 64-bit integer, which drops whole turns exactly, and its
// signed value is the angle's fraction of a turn in [-1/2, 1/2). sincospif of
// twice that needs no range reduction, at a position of 3 as at one of 2^31.
//
// One CTA turns all heads of one or more tokens: its threads first put the
// cosines and sines of the tokens' pairs into shared memory (one evaluation
// for all heads), then each thread moves one chunk of a head (V values, or V
// pairs in the half layout) for head after head. Bound by memory.
#include "attn.h"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <int V>
struct Vec;
template <>
struct Vec<8> {
  typedef uint4 type;
};
template <>
struct Vec<4> {
  typedef uint2 type;
};
template <>
struct Vec<1> {
  typedef uint16_t type;
};

template <int V>
union Chunk {
  typename Vec<V>::type v;
  uint16_t e[V];
};

// V values (half layout: of each half) or V / 2 pairs (interleaved, V > 1) of
// one head; V = 1 interleaved takes one pair as two single values.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int tokens_per_cta,
                                                        int units, int turn_units) {
  extern __shared__ float2 cs[];  // [tokens_per_cta][rot / 2]
  typedef typename Vec<V>::type W;
  const int pairs = p.r.rot >> 1;
  const int t0 = blockIdx.x * tokens_per_cta;
  const int nt = min(tokens_per_cta, p.tokens - t0);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int i = tid; i < nt * pairs; i += blockDim.x * blockDim.y) {
    const int t = i / pairs, c = i - t * pairs;
    const long long phase = (long long)((unsigned long long)(long long)p.positions[t0 + t] *
                                        (unsigned long long)p.r.freq[c]);
    float sn, cn;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &sn, &cn);
    cs[i] = make_float2(cn * p.r.magnitude, sn * p.r.magnitude * p.r.sign);
  }
  __syncthreads();
  const int u = threadIdx.x;
  if (u >= units) return;
  const int heads = p.hq + p.hk + p.hv;
  for (int t = 0; t < nt; ++t) {
    const int tok = t0 + t;
    long long slot = 0, row = 0;
    if (p.slots) {
      slot = p.slots[tok];
      if (slot >= p.num_slots) {
        if (tid == 0) atomicOr(p.err, kErrRange);
        slot = -1;
      }
      const long long page = slot >> p.page_shift;
      row = page * p.page_stride + (slot - (page << p.page_shift)) * p.token_stride;
    }
    for (int hd = threadIdx.y; hd < heads; hd += blockDim.y) {
      const uint16_t* src;
      uint16_t* dst;
      bool turn = true;
      if (hd < p.hq) {
        src = p.q.p + (long long)tok * p.q.token + (long long)hd * p.q.head;
        dst = p.q_out.p + (long long)tok * p.q_out.token + (long long)hd * p.q_out.head;
      } else if (slot < 0) {
        continue;
      } else if (hd < p.hq + p.hk) {
        const int h = hd - p.hq;
        src = p.k.p + (long long)tok * p.k.token + (long long)h * p.k.head;
        dst = p.k_pages + row + (long long)h * p.head_stride;
      } else {
        const int h = hd - p.hq - p.hk;
        src = p.v.p + (long long)tok * p.v.token + (long long)h * p.v.head;
        dst = p.v_pages + row + (long long)h * p.head_stride;
        turn = false;
      }
      if (u >= turn_units) {  // behind the turned part: one chunk, copied
        const int o = p.r.rot + (u - turn_units) * V;
        *reinterpret_cast<W*>(dst + o) = *reinterpret_cast<const W*>(src + o);
        continue;
      }
      const float2* c = cs + t * pairs;
      if (!p.r.interleaved || V == 1) {
        // unit u holds pairs [u V, (u + 1) V): half layout values (i, i + rot / 2),
        // or the one interleaved pair (2u, 2u + 1)
        const int oa = p.r.interleaved ? 2 * u : u * V;
        const int ob = p.r.interleaved ? 2 * u + 1 : oa + pairs;
        Chunk<V> a, b;
        a.v = *reinterpret_cast<const W*>(src + oa);
        b.v = *reinterpret_cast<const W*>(src + ob);
        if (turn) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 w = c[u * V + i];
            const float x = T::to_f32(a.e[i]), y = T::to_f32(b.e[i]);
            a.e[i] = T::from_f32(x * w.x - y * w.y);
            b.e[i] = T::from_f32(y * w.x + x * w.y);
          }
        }
        *reinterpret_cast<W*>(dst + oa) = a.v;
        *reinterpret_cast<W*>(dst + ob) = b.v;
      } else {
        Chunk<V> a;
        a.v = *reinterpret_cast<const W*>(src + u * V);
        if (turn) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float2 w = c[u * (V / 2) + i];
            const float x = T::to_f32(a.e[2 * i]), y = T::to_f32(a.e[2 * i + 1]);
            a.e[2 * i] = T::from_f32(x * w.x - y * w.y);
            a.e[2 * i + 1] = T::from_f32(y * w.x + x * w.y);
          }
        }
        *reinterpret_cast<W*>(dst + u * V) = a.v;
      }
    }
  }
}

bool aligned(const Rows& r, int v) {
  return r.p == nullptr || ((reinterpret_cast<uintptr_t>(r.p) % (2 * v)) == 0 && r.token % v == 0 &&
                            r.head % v == 0);
}

// the widest access every address of the call allows
bool fits(const RopeParams& p, int v) {
  const int half = p.r.rot / 2;
  if ((p.r.interleaved ? p.r.rot : half) % v || (p.head_dim - p.r.rot) % v) return false;
  if (p.slots && (p.page_stride % v || p.token_stride % v || p.head_stride % v)) return false;
  return aligned(p.q, v) && aligned(p.q_out, v) && aligned(p.k, v) && aligned(p.v, v);
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  const int turn_units = p.r.interleaved && V > 1 ? p.r.rot / V : p.r.rot / 2 / V;
  const int units = turn_units + (p.head_dim - p.r.rot) / V;
  const int tokens_per_cta = 1;
  dim3 block(units, 1);
  const int heads = p.hq + p.hk + p.hv;
  while ((int)(block.x * block.y * 2) <= kThreads && (int)block.y < heads) block.y *= 2;
  rope_kernel<T, V><<<(p.tokens + tokens_per_cta - 1) / tokens_per_cta, block,
                      tokens_per_cta * (p.r.rot / 2) * sizeof(float2), s>>>(p, tokens_per_cta,
                                                                            units, turn_units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t s) {
  if (fits(p, 8)) return launch<T, 8>(p, s);
  if (fits(p, 4)) return launch<T, 4>(p, s);
  return launch<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int sms, cudaStream_t s) {
  (void)sms;
  return dtype == MOE_ATTN_BF16 ? launch_t<Bf16>(p, s) : launch_t<Fp16>(p, s);
}

}  // namespace attn
}  // namespace moe
