// What a thread has of a head in the kernels of norms and rotary positions.
//
// Fast form: a head's values are cut into units, one a lane of a group of `lanes`
// (a power of two, 16 at most). A unit of the turned part is a chunk of 8 values of
// either half, which in the half layout brings both values of a pair to one lane
// (interleaved pairs lie in one chunk anyway), and of the part that does not turn two
// neighbouring chunks. Every access is 16 bytes, and a sum over a head is a few
// shuffles.
#pragma once

#include "attn_common.cuh"

namespace moe {
namespace attn {

struct Units {
  int count, turned, lanes;
};
__host__ __device__ __forceinline__ Units units_of_head(int head_dim, int rot) {
  Units u;
  u.turned = rot / 16;
  u.count = u.turned + (head_dim - rot + 8) / 16;
  u.lanes = 1;
  while (u.lanes < u.count) u.lanes *= 2;
  return u;
}

union Chunk8 {
  uint4 v;
  uint32_t w[4];
  uint16_t e[8];
};

__device__ __forceinline__ float group_sum(float x, int lanes) {
  // (a branch for each step costs more than the steps that a small group leaves out)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = o < lanes ? x + y : x;
  }
  return x;
}

__device__ __forceinline__ void cos_sin(const Rotation& r, int position, int pair, float& cosine,
                                        float& sine) {
  const long long phase = (long long)((unsigned long long)(long long)position *
                                      (unsigned long long)r.freq[pair]);
  // (the upper half says it to 2^-32 turns; all of it takes a conversion of 64 bits)
  float sn, cn;
  sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn, &cn);
  cosine = cn * r.magnitude;
  sine = sn * r.magnitude * r.sign;
}
// The pairs of a head, and which token's an entry of a table is: entries are below 4096
// and pairs 8 to 128 of them, so the quotient is exact in 32 bits (a division takes about
// as long as the rest of an entry).
struct Pairs {
  int count;
  unsigned inverse;
  __device__ __forceinline__ explicit Pairs(int rot)
      : count(rot >> 1), inverse(count ? ((1u << 22) + count - 1) / count : 0) {}
  __device__ __forceinline__ int token(int entry) const { return entry * inverse >> 22; }
};
// cosines and sines of the pairs of positions[0 .. tokens), by all threads of the CTA
__device__ __forceinline__ void fill_table(const Rotation& r, const int* positions, int tokens,
                                           float* cosines, float* sines, int tid, int threads) {
  const Pairs pairs(r.rot);
  for (int i = tid; i < tokens * pairs.count; i += threads) {
    const int t = pairs.token(i), c = i - t * pairs.count;
    cos_sin(r, positions[t], c, cosines[i], sines[i]);
  }
}

// A lane's unit: chunk `a`, and where `two` chunk `b` `gap` values behind it.
template <bool IL>
struct Lane {
  int at, gap, pair;   // first value, from chunk to chunk, first pair
  bool turns, two;
  __device__ __forceinline__ Lane(int u, int turned, int rot, int head_dim) {
    turns = u < turned;
    at = turns ? u * 8 : rot + (u - turned) * 16;
    gap = turns ? rot >> 1 : 8;
    two = turns || at + 8 < head_dim;
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
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // interleaved: the pairs of either chunk
      const int from = pair + i * (IL ? gap >> 1 : 4);
      *reinterpret_cast<float4*>(c + 4 * i) = *reinterpret_cast<const float4*>(cosines + from);
      *reinterpret_cast<float4*>(s + 4 * i) = *reinterpret_cast<const float4*>(sines + from);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& x = IL ? (i < 4 ? a : b)[2 * (i & 3)] : a[i];
      float& y = IL ? (i < 4 ? a : b)[2 * (i & 3) + 1] : b[i];
      const float x0 = x, y0 = y;
      x = x0 * c[i] - y0 * s[i];
      y = y0 * c[i] + x0 * s[i];
    }
  }
};

template <typename T>
__device__ __forceinline__ void unpack8(const Chunk8& c, float* f) {
  // (by words: an instruction less for each value than halves of them take)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (T::kFp16) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&c.w[k]));
      f[2 * k] = x.x, f[2 * k + 1] = x.y;
    } else {
      f[2 * k] = __uint_as_float(c.w[k] << 16);
      f[2 * k + 1] = __uint_as_float(c.w[k] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(T::pack(f[0], f[1]), T::pack(f[2], f[3]), T::pack(f[4], f[5]),
                    T::pack(f[6], f[7]));
}

// Threads of a CTA walk along the tokens: thread (unit, head, z) has its unit of its head
// for tokens c0 + z, c0 + step + z, ... Its chunks come through a ring of its own in
// shared memory, kAhead - 1 tokens ahead, so that loads are under way without registers
// and nobody waits for anybody but for the tables, which are made for kAhead steps at
// once. What bounds it is instructions, so addresses go on by additions and slots are
// told apart at compile time.
constexpr int kAhead = 4, kWalkThreads = 256;
// Turned values of the tokens side by side, where they are more than one: ring and
// tables then take the 48 KB that a kernel has without asking, to the byte.
constexpr int kWalkTurned = 1024;
static_assert(kAhead * (kWalkTurned * 4 + kWalkThreads * 32) <= 48 * 1024,
              "shared memory of a walk");

__device__ __forceinline__ void copy_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

struct Walk {
  int tid, threads, lanes;   // of the CTA, up to kWalkThreads; lanes of a head
  int z, zs;                 // token side by side, and how many (a power of two)
  int c0, step;
  __host__ __device__ static int table_floats(int zs, int rot) { return kAhead * zs * rot; }
  static size_t bytes(int zs, int rot) {
    return (size_t)table_floats(zs, rot) * 4 + (size_t)kAhead * kWalkThreads * 32;
  }
};

// Where a walk's rows go: one behind the other.
struct RowRun {
  uint16_t* to;
  long long step;
  __device__ __forceinline__ uint16_t* next(int) {
    uint16_t* at = to;
    to += step;
    return at;
  }
};

// Norm and rotation. `plain`: the rows are copied as they are. src: the thread's unit of
// its first token; out.next(t): where token t's goes, or null. w, w_head: the weight and
// where the head's begins. smem: of Walk::bytes.
template <typename T, bool IL, class Out>
__device__ __forceinline__ void norm_walk(const Walk& k, const Rotation& rot,
                                          const int* positions, int tokens, int head_dim,
                                          const Norm& n, const Lane<IL>& lane, bool active,
                                          bool plain, const uint16_t* src, long long src_token,
                                          const void* w, long long w_head, float* smem, Out out) {
  const Pairs table(rot.rot);
  const int pairs = table.count, z_shift = __ffs(k.zs) - 1;
  constexpr int kHalf = kWalkThreads, kSlot = 2 * kHalf;   // of the ring, chunks
  const uint4* ring = reinterpret_cast<uint4*>(smem + Walk::table_floats(k.zs, rot.rot)) + k.tid;
  const uint32_t ring_at = smem_u32(ring);
  const long long src_step = src_token * k.step;
  int coming = active ? k.c0 + k.z : tokens;               // token of the next copy
  const auto fetch = [&](int slot) {
    if (coming < tokens) {
      copy_async16(ring_at + slot * kSlot * 16, src);
      if (lane.two) copy_async16(ring_at + (slot * kSlot + kHalf) * 16, src + lane.gap);
      src += src_step;
      coming += k.step;
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch(i);
  float wa[8], wb[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) wa[q] = wb[q] = 0.0f;
  if (active && !plain && n.on)
    lane.template weights<T>(w, w_head, n.wide, n.offset, wa, wb);
  const float mean = 1.0f / (float)head_dim;
  int t = k.c0 + k.z;
  for (int c0 = k.c0; c0 < tokens;) {
    __syncthreads();
    for (int e = k.tid; e < kAhead * k.zs * pairs; e += k.threads) {
      const int row = table.token(e), c = e - row * pairs;
      const int of = c0 + (row >> z_shift) * k.step + (row & (k.zs - 1));
      if (of < tokens) cos_sin(rot, positions[of], c, smem[e], smem[kAhead * k.zs * pairs + e]);
    }
    __syncthreads();
    const float* cosines = smem + k.z * pairs;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c0 >= tokens) break;                             // (of all threads)
      fetch((i + kAhead - 1) % kAhead);
      copies_wait<kAhead - 1>();
      const bool on = active && t < tokens;
      Chunk8 a, b;
      a.v = b.v = make_uint4(0, 0, 0, 0);
      if (on) {
        a.v = ring[i * kSlot];
        if (lane.two) b.v = ring[i * kSlot + kHalf];
      }
      float fa[8], fb[8], f = 1.0f;
      unpack8<T>(a, fa);
      unpack8<T>(b, fb);
      if (n.on) {  // (all lanes: heads that are copied may share a warp with others)
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) sum = fmaf(fa[q], fa[q], fmaf(fb[q], fb[q], sum));
        f = rsqrtf(fmaf(group_sum(sum, k.lanes), mean, n.eps));
      }
      if (!plain) {
        if (n.on) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            fa[q] = fa[q] * f * wa[q];
            fb[q] = fb[q] * f * wb[q];
          }
        }
        if (lane.turns) lane.turn(fa, fb, cosines, cosines + kAhead * k.zs * pairs);
        a.v = pack8<T>(fa);
        b.v = pack8<T>(fb);
      }
      if (on) {
        uint16_t* to = out.next(t);
        if (to) {
          *reinterpret_cast<uint4*>(to) = a.v;
          if (lane.two) *reinterpret_cast<uint4*>(to + lane.gap) = b.v;
        }
      }
      cosines += k.zs * pairs;
      c0 += k.step;
      t += k.step;
    }
  }
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
  return r.rot % 16 == 0 && head_dim % 8 == 0;
}

}  // namespace attn
}  // namespace moe
