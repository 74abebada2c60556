// Rotary positions, alone or with the append of keys and values to a paged
// cache.
//
// The angle of pair i at position p is 2 pi frac(p * freq[i] / 2^64): the
// product wraps as a 64-bit integer, which drops whole turns exactly, and its
// signed value is the angle's fraction of a turn in [-1/2, 1/2). sincospif of
// twice that needs no range reduction, at a position of 3 as at one of 2^31.
//
// A thread has one chunk of one head (V values, or V pairs in the half layout)
// and takes it for a few tokens: addresses and the kind of head are
// worked out once, and all its loads are under way while the CTA puts the
// cosines and sines of its tokens' pairs into shared memory, one evaluation for
// all heads. Bound by memory: q, k and v of 8192 tokens (32, 8 and 8 heads of 128),
// not in the caches, take 32.8 us, 6.1 TB/s, 0.90 of the measured copy rate (replayed
// on the same inputs 35.6 us); by flat chunk numbers, divided out per chunk, 60 us.
#include "attn_common.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kMaxThreads = 512;
// Tokens of a thread: four chunks under way either way. Registers for three
// CTAs of 512 threads on an SM (with two, 8192 tokens took 8 % longer).
constexpr int tokens_of(bool two_chunks) { return two_chunks ? 2 : 4; }
constexpr int kSms = 152;

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

// N consecutive values of a table in shared memory
template <int N>
__device__ __forceinline__ void read_table(const float* src, float* v) {
  if (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      *reinterpret_cast<float4*>(v + 4 * i) = *reinterpret_cast<const float4*>(src + 4 * i);
  } else if (N == 2) {
    *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
  } else {
    v[0] = src[0];
  }
}

// IL: interleaved pairs (V > 1: V / 2 of them in a chunk; V = 1: one pair as
// two single values, as in the half layout)
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kMaxThreads, 3)
    rope_kernel(const RopeParams p, int tokens_per_thread, int units, int turn_units) {
  extern __shared__ float4 table4[];  // cosines, then sines: [tokens of the CTA][rot / 2]
  float* cosines = reinterpret_cast<float*>(table4);
  typedef typename Vec<V>::type W;
  constexpr bool kInChunk = IL && V > 1;            // both values of a pair in one chunk
  constexpr int kPairs = kInChunk ? V / 2 : V;
  constexpr int kTokens = tokens_of(!kInChunk);
  const int pairs = p.r.rot >> 1;
  // this CTA's tokens, and this thread's among them
  const int tokens_per_cta = tokens_per_thread * blockDim.z;
  const int cta0 = blockIdx.x * tokens_per_cta;
  const int cta_tokens = min(tokens_per_cta, p.tokens - cta0);
  const int first = threadIdx.z * tokens_per_thread, t0 = cta0 + first;
  const int nt = min(tokens_per_thread, cta_tokens - first);
  float* sines = cosines + tokens_per_cta * pairs;

  wait_prior_launch();
  let_next_launch();
  const int u = threadIdx.x, hd = blockIdx.y * blockDim.y + threadIdx.y;
  const bool active = hd < p.hq + p.hk + p.hv;
  const bool key = hd >= p.hq && hd < p.hq + p.hk, value = hd >= p.hq + p.hk;
  const bool pass = u >= turn_units;                // behind the turned part: copied
  const bool two = !pass && !kInChunk;              // a chunk of each half
  const int h = hd - (value ? p.hq + p.hk : key ? p.hq : 0);
  const Rows& in = value ? p.v : key ? p.k : p.q;
  const int oa = pass ? p.r.rot + (u - turn_units) * V : (IL && V == 1) ? 2 * u : u * V;
  const int gap = (IL && V == 1) ? 1 : pairs;       // to the other half's chunk
  const uint16_t* src = in.p + (long long)t0 * in.token + (long long)h * in.head + oa;
  Chunk<V> a[kTokens], b[kTokens];
  if (active) {
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      if (t < nt) {
        a[t].v = *reinterpret_cast<const W*>(src + t * in.token);
        if (two) b[t].v = *reinterpret_cast<const W*>(src + t * in.token + gap);
      }
  }
  const int tid = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x;
  const int threads = blockDim.x * blockDim.y * blockDim.z;
  for (int i = tid; i < cta_tokens * pairs; i += threads) {
    const int t = i / pairs, c = i - t * pairs;
    const long long phase = (long long)((unsigned long long)(long long)p.positions[cta0 + t] *
                                        (unsigned long long)p.r.freq[c]);
    float sn, cn;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &sn, &cn);
    cosines[i] = cn * p.r.magnitude;
    sines[i] = sn * p.r.magnitude * p.r.sign;
  }
  __syncthreads();
  if (!active) return;
  const bool turns = !pass && !value;
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    if (t >= nt) break;
    uint16_t* dst;
    if (key || value) {  // to the token's slot
      const long long slot = p.slots[t0 + t];
      if (slot < 0) continue;
      if (slot >= p.num_slots) {
        atomicOr(p.err, kErrRange);
        continue;
      }
      const long long page = slot >> p.page_shift;
      dst = (key ? p.k_pages : p.v_pages) + page * p.page_stride +
            (slot - (page << p.page_shift)) * p.token_stride + (long long)h * p.head_stride + oa;
    } else {
      dst = p.q_out.p + (long long)(t0 + t) * p.q_out.token + (long long)h * p.q_out.head + oa;
    }
    if (turns) {
      float c[kPairs], s[kPairs];
      read_table<kPairs>(cosines + (first + t) * pairs + u * kPairs, c);
      read_table<kPairs>(sines + (first + t) * pairs + u * kPairs, s);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        uint16_t& ea = a[t].e[kInChunk ? 2 * i : i];
        uint16_t& eb = kInChunk ? a[t].e[2 * i + 1] : b[t].e[i];
        const float x = T::to_f32(ea), y = T::to_f32(eb);
        ea = T::from_f32(x * c[i] - y * s[i]);
        eb = T::from_f32(y * c[i] + x * s[i]);
      }
    }
    *reinterpret_cast<W*>(dst) = a[t].v;
    if (two) *reinterpret_cast<W*>(dst + gap) = b[t].v;
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

template <typename T, int V, bool IL>
cudaError_t launch_il(const RopeParams& p, cudaStream_t s) {
  const int turn_units = IL && V > 1 ? p.r.rot / V : p.r.rot / 2 / V;
  const int units = turn_units + (p.head_dim - p.r.rot) / V;
  const int heads = p.hq + p.hk + p.hv;
  // groups of heads of at most kMaxThreads threads, as even as they come
  const int most = kMaxThreads / units;  // units <= 256
  const int groups = (heads + most - 1) / most;
  dim3 block(units, (heads + groups - 1) / groups, 1);
  // few heads: tokens side by side, up to 256 threads, while every SM has two
  // CTAs and the table stays within 16 KB; then several tokens to a thread,
  // while every SM has four (2047 tokens of 8 heads: 32 threads a CTA took
  // 6.2 us)
  const long long all = (long long)p.tokens * groups;
  while (block.x * block.y * block.z <= 128 && block.z < 64 && all >= 4LL * kSms * block.z &&
         2 * block.z * p.r.rot <= 4096)
    block.z *= 2;
  int tokens = 1;
  while (tokens < tokens_of(!(IL && V > 1)) && all >= 8LL * kSms * block.z * tokens &&
         2 * tokens * block.z * p.r.rot <= 4096)
    tokens *= 2;
  const int cta = tokens * block.z;
  return launch_after(rope_kernel<T, V, IL>, dim3((p.tokens + cta - 1) / cta, groups), block,
                      cta * p.r.rot * (int)sizeof(float), s, p, tokens, units, turn_units);
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  return p.r.interleaved ? launch_il<T, V, true>(p, s) : launch_il<T, V, false>(p, s);
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t s) {
  if (fits(p, 8)) return launch<T, 8>(p, s);
  if (fits(p, 4)) return launch<T, 4>(p, s);
  return launch<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_ATTN_BF16 ? launch_t<Bf16>(p, s) : launch_t<Fp16>(p, s);
}

}  // namespace attn
}  // namespace moe
