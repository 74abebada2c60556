// What a thread has of a head in the kernels of norms and rotary positions.
//
// Fast form: a head's values are cut into units, one a lane of a group of `lanes`
// (a power of two, 32 at most). In the half layout a unit of the turned part is a
// chunk of 8 values of either half, so that both values of a pair are in one lane, and
// of the part that does not turn two neighbouring chunks; interleaved pairs lie in one
// chunk, and so units are single chunks there. Every access is 16 bytes, and a sum over
// a head is a few shuffles.
#pragma once

#include "attn_common.cuh"

namespace moe {
namespace attn {

struct Units {
  int count, turned, lanes;
};
template <bool IL>
__host__ __device__ __forceinline__ Units units_of_head(int head_dim, int rot) {
  Units u;
  u.turned = IL ? rot / 8 : rot / 16;
  u.count = u.turned + (IL ? (head_dim - rot) / 8 : (head_dim - rot + 8) / 16);
  u.lanes = 1;
  while (u.lanes < u.count) u.lanes *= 2;
  return u;
}

union Chunk8 {
  uint4 v;
  uint16_t e[8];
};

__device__ __forceinline__ float group_sum(float x, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cosines and sines of the pairs of positions[0 .. tokens), by all threads of the CTA
__device__ __forceinline__ void fill_table(const Rotation& r, const int* positions, int tokens,
                                           float* cosines, float* sines, int tid, int threads) {
  const int pairs = r.rot >> 1;
  for (int i = tid; i < tokens * pairs; i += threads) {
    const int t = i / pairs, c = i - t * pairs;
    const long long phase = (long long)((unsigned long long)(long long)positions[t] *
                                        (unsigned long long)r.freq[c]);
    // (the upper half says it to 2^-32 turns; all of it takes a conversion of 64 bits)
    float sn, cn;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn, &cn);
    cosines[i] = cn * r.magnitude;
    sines[i] = sn * r.magnitude * r.sign;
  }
}

// A lane's unit: chunk `a`, and where `two` chunk `b` `gap` values behind it.
template <bool IL>
struct Lane {
  int at, gap, pair;   // first value, pairs of a half, first pair
  bool turns, two;
  __device__ __forceinline__ Lane(int u, int turned, int rot, int head_dim) {
    turns = u < turned;
    at = turns ? u * 8 : rot + (u - turned) * (IL ? 8 : 16);
    gap = turns ? rot >> 1 : 8;
    two = !IL && (turns || at + 8 < head_dim);
    pair = turns ? u * (IL ? 4 : 8) : 0;
  }
  // fp32 weights plus offset of the unit's values
  template <typename T>
  __device__ __forceinline__ void weights(const void* w, long long head, int wide, float offset,
                                          float* wa, float* wb) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float* to = half ? wb : wa;
      if (half && !two) break;
      const long long i = head + at + (half ? gap : 0);
      if (wide) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + i);
        const float4 x = __ldg(f), y = __ldg(f + 1);
        to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
        to[4] = y.x, to[5] = y.y, to[6] = y.z, to[7] = y.w;
      } else {
        Chunk8 c;
        c.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + i));
#pragma unroll
        for (int k = 0; k < 8; ++k) to[k] = T::to_f32(c.e[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) to[k] += offset;
    }
  }
  // the unit's pairs turned; cosines and sines of its token
  __device__ __forceinline__ void turn(float* a, float* b, const float* cosines,
                                       const float* sines) const {
    constexpr int kPairs = IL ? 4 : 8;
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs / 4; ++i) {
      *reinterpret_cast<float4*>(c + 4 * i) = *reinterpret_cast<const float4*>(cosines + pair + 4 * i);
      *reinterpret_cast<float4*>(s + 4 * i) = *reinterpret_cast<const float4*>(sines + pair + 4 * i);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float& x = a[IL ? 2 * i : i];
      float& y = IL ? a[2 * i + 1] : b[i];
      const float x0 = x, y0 = y;
      x = x0 * c[i] - y0 * s[i];
      y = y0 * c[i] + x0 * s[i];
    }
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(const Chunk8& c, float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = T::to_f32(c.e[k]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(T::pack(f[0], f[1]), T::pack(f[2], f[3]), T::pack(f[4], f[5]),
                    T::pack(f[6], f[7]));
}

// Any form: a warp a head, lane l values l, l + 32, ...; partners through shared
// memory. For head sizes, rotations and addresses that the fast form does not take.
constexpr int kAnyValues = 8;  // of a lane: head sizes up to 256

// value i of a row, turned; `row` holds the row's values in shared memory
__device__ __forceinline__ float turned_any(const Rotation& r, int position, const float* row,
                                            int i) {
  if (i >= r.rot) return row[i];
  const int half = r.rot >> 1;
  const int pair = r.interleaved ? i >> 1 : i < half ? i : i - half;
  const bool second = r.interleaved ? i & 1 : i >= half;
  const long long phase = (long long)((unsigned long long)(long long)position *
                                      (unsigned long long)r.freq[pair]);
  float sn, cn;
  sincospif(__ll2float_rn(phase) * 0x1p-63f, &sn, &cn);
  cn *= r.magnitude;
  sn *= r.magnitude * r.sign;
  const float other = row[r.interleaved ? i ^ 1 : second ? i - half : i + half];
  return second ? row[i] * cn + other * sn : row[i] * cn - other * sn;
}

template <typename T>
__device__ __forceinline__ float weight_any(const void* w, long long i, int wide, float offset) {
  return (wide ? static_cast<const float*>(w)[i]
               : T::to_f32(static_cast<const uint16_t*>(w)[i])) + offset;
}

inline bool rows_aligned(const Rows& r) {
  return r.p == nullptr ||
         ((reinterpret_cast<uintptr_t>(r.p) & 15u) == 0 && r.token % 8 == 0 && r.head % 8 == 0);
}
inline bool weights_aligned(const Norm& n) {
  const int per = n.wide ? 4 : 8;
  const auto ok = [&](const void* w, long long head) {
    return !w || ((reinterpret_cast<uintptr_t>(w) & 15u) == 0 && head % per == 0);
  };
  return !n.on || (ok(n.q_weight, n.q_head) && ok(n.k_weight, n.k_head));
}
// the fast form takes these heads
inline bool units_fit(const Rotation& r, int head_dim) {
  return (r.interleaved ? r.rot : r.rot / 2) % 8 == 0 && (head_dim - r.rot) % 8 == 0;
}

}  // namespace attn
}  // namespace moe
