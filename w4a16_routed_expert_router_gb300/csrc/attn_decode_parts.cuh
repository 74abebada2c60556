// What the kernels for few query rows share, over a 16-bit cache and an 8-bit one:
// dividing the key blocks over the CTAs, and joining what they and their warps have.
#pragma once

#include "attn_common.cuh"

namespace moe {
namespace attn {

using namespace tc;

constexpr int kRows = kDecodeRows;
constexpr int kStateRows = 4 * kRows;
constexpr int kAhead = 12;  // pieces whose loads are under way together in a join

template <typename T>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<Bf16>(float* d, const uint32_t* a, uint32_t b0,
                                            uint32_t b1) {
  mma_bf16_16816(d, a, b0, b1, d);
}
template <>
__device__ __forceinline__ void mma16<Fp16>(float* d, const uint32_t* a, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int CONSUMERS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
}

// How a kernel divides the work: kBlk keys a block, and kItem, an item's fixed cost in
// blocks.
template <class C>
__device__ __forceinline__ int units_of(const Span& r) {
  return r.blocks ? r.blocks + C::kItem : 0;
}

template <class C>
__device__ __forceinline__ Span item_of(const AttnParams& p, int s) {
  Span r = read_sequence(p.b, p.page_shift, s, p.err);
  r.blocks = 0;
  if (r.n > 0)  // and at most max_q, which is kRows / group or less
    span_blocks(r, r.kv - r.n, r.kv - 1, p.sc, prefix_of(p.sc, s, r.kv), C::kBlk);
  return r;
}

// A role's way through its CTA's share: units [w, hi), `at` the first unit of
// (seq, head 0).
struct Walk {
  long long at, w, hi;
  int seq, head;         // head -1: to be worked out
};
// Blocks [n0, end) of an item that begins at unit `first`.
struct Piece {
  Span it;
  long long first;
  int seq, head, n0, end;
};
template <class C>
__device__ __forceinline__ bool next_piece(const AttnParams& p, Walk& k, Piece& g) {
  while (k.w < k.hi) {
    g.it = item_of<C>(p, k.seq);
    const int units = units_of<C>(g.it);
    if (units == 0) {
      ++k.seq;
      continue;
    }
    if (k.head < 0) k.head = (int)quotient(k.w - k.at, units);
    g.seq = k.seq;
    g.head = k.head;
    g.first = k.at + (long long)k.head * units;
    const int u0 = (int)(k.w - g.first), u1 = (int)min((long long)units, u0 + (k.hi - k.w));
    g.n0 = max(0, u0 - C::kItem);
    g.end = max(0, u1 - C::kItem);
    k.w = g.first + u1;
    if (++k.head == p.hk) {  // (a share's last item may end early; nothing follows it)
      k.head = 0;
      k.at = k.w;
      ++k.seq;
    }
    if (g.end > g.n0) return true;
  }
  return false;
}

// Units of all sequences, and where this CTA's share begins; false where it has none.
// The CTA's barriers are set up behind it.
template <class C, int THREADS, class S>
__device__ __forceinline__ bool begin_share(const AttnParams& p, S& s, long long& total,
                                            Walk& walk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  total = 0;
  long long lo = 0, at = 0;
  int seq = 0;
  if (p.b.num_seqs <= 32) {  // each warp for itself
    const long long mine = lane < p.b.num_seqs ? (long long)units_of<C>(item_of<C>(p, lane)) * p.hk : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const Shares sh(total, gridDim.x);
    if ((int)blockIdx.x >= sh.grid) return false;
    lo = sh.begin(blockIdx.x);
    seq = __ffs(__ballot_sync(0xffffffffu, lo < incl)) - 1;
    at = __shfl_sync(0xffffffffu, incl - mine, seq);
    __syncthreads();  // the barriers are set up
  } else {
    const int per = (p.b.num_seqs + THREADS - 1) / THREADS;
    const int s0 = min(p.b.num_seqs, (int)threadIdx.x * per);
    const int s1 = min(p.b.num_seqs, s0 + per);
    long long mine = 0;
    for (int q = s0; q < s1; ++q) mine += (long long)units_of<C>(item_of<C>(p, q)) * p.hk;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += s.scan[i];
      total += s.scan[i];
    }
    const Shares sh(total, gridDim.x);
    if ((int)blockIdx.x >= sh.grid) return false;
    lo = sh.begin(blockIdx.x);
    if (lo >= before && lo < before + mine) {
      long long first = before;
      for (int q = s0; q < s1; ++q) {
        const long long c = (long long)units_of<C>(item_of<C>(p, q)) * p.hk;
        if (lo < first + c) {
          s.begin_seq = q;
          s.begin_at = first;
          break;
        }
        first += c;
      }
    }
    __syncthreads();
    seq = s.begin_seq;
    at = s.begin_at;
  }
  const Shares sh(total, gridDim.x);
  walk = Walk{at, lo, sh.begin(blockIdx.x + 1), seq, -1};
  return true;
}

// The end of an item: the warps' states joined in shared memory, and its results
// written, or left as a piece, which the last CTA of the item joins. L: which rows a
// thread has and where the values of a state lie in it; FIRST: first consumer thread;
// D: row length of the pieces.
template <class C, class L, int FIRST, int CONSUMERS, int D, class S, class Pack>
__device__ __forceinline__ void finish_item(const AttnParams& p, const Partials& ws, S& s,
                                            const Shares& sh, const Piece& g, int cw,
                                            typename L::Values& o, float (&m)[L::kRows],
                                            float (&l)[L::kRows], const Pack& pack) {
  const int lane = threadIdx.x & 31;
  const Span& it = g.it;
  const int head = g.head, n0 = g.n0, end = g.end, rows = it.n * p.group;
#pragma unroll
  for (int r = 0; r < L::kRows; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], L::kLanes);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2 * L::kLanes);
    if (L::kLanes == 4) l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
  }
  // Join the warps' states: where they are more than there is room for, the upper half
  // of the warps first hand theirs to the lower half; then all states lie in shared
  // memory and every thread adds up its values of them.
  const auto put = [&](int state, int per_state) {
#pragma unroll
    for (int r = 0; r < L::kRows; ++r) {
      const int row = L::row(r, lane);
      if (row >= rows) continue;
      const int at_row = state * per_state + row;
      if (L::first(lane)) s.ml[at_row] = make_float2(m[r], l[r]);
      L::put(s.o[at_row], o, r, lane);
    }
  };
  const bool many = rows > 8, fold = many || CONSUMERS > 8;
  const int states = fold ? CONSUMERS / 2 : CONSUMERS, per_state = many ? kRows : 8;
  static_assert(CONSUMERS <= 16, "eight states of 8 rows have room");
  if (fold) {
    if (cw >= CONSUMERS / 2) put(cw - CONSUMERS / 2, per_state);
    consumers_sync<CONSUMERS>();
    if (cw < CONSUMERS / 2) {
#pragma unroll
      for (int r = 0; r < L::kRows; ++r) {
        const int row = L::row(r, lane);
        if (row >= rows) continue;
        const float2 x = s.ml[cw * per_state + row];
        const float mm = fmaxf(m[r], x.x), base = mm == -INFINITY ? 0.0f : mm;
        const float a = ex2(m[r] - base), b = ex2(x.x - base);
        m[r] = mm;
        l[r] = l[r] * a + x.y * b;
        L::add(s.o[cw * per_state + row], o, r, lane, a, b);
      }
    }
    consumers_sync<CONSUMERS>();
  }
  if (cw < states) put(cw, per_state);
  consumers_sync<CONSUMERS>();

  const bool split = end - n0 < it.blocks;
  const int c0 = split ? sh.of(g.first + C::kItem) : 0;  // CTA of the item's first block
  const long long slot = 2LL * blockIdx.x + ((int)blockIdx.x == c0 ? 1 : 0);
  const int half_d = p.head_dim >> 1;
  const auto write = [&](int row, int c, float x, float y, float mm, float sum) {
    const int tok = row / p.group, h = head * p.group + (row - tok * p.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<uint32_t*>(p.out.p + (long long)(it.first + tok) * p.out.token +
                                 (long long)h * p.out.head + c) = pack(x * inv, y * inv);
    if (p.lse && c == 0)
      p.lse[(long long)(it.first + tok) * p.hq + h] =
          sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
  };
  for (int e = threadIdx.x - FIRST; e < rows * half_d; e += CONSUMERS * 32) {
    const int row = e / half_d, c = 2 * (e - row * half_d);
    float2 q[8], v[8];
    float mm = -INFINITY, sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = make_float2(-INFINITY, 0.0f);
      v[i] = make_float2(0.0f, 0.0f);
      if (i < states) {
        q[i] = s.ml[i * per_state + row];
        v[i] = *reinterpret_cast<const float2*>(&s.o[i * per_state + row][c]);
      }
      mm = fmaxf(mm, q[i].x);
    }
    const float base = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ex2(q[i].x - base);
      sum = fmaf(q[i].y, f, sum);
      x = fmaf(v[i].x, f, x);
      y = fmaf(v[i].y, f, y);
    }
    if (!split) {
      write(row, c, x, y, mm, sum);
    } else {
      // a piece: left in the workspace
      __stcg(reinterpret_cast<float2*>(ws.o + (slot * kRows + row) * D + c),
             make_float2(x, y));
      if (c == 0) __stcg(ws.ml + slot * kRows + row, make_float2(mm, sum));
    }
  }
  if (split) __threadfence();
  consumers_sync<CONSUMERS>();  // the states are read, and a piece is written
  if (split) {
    // the last CTA of the item joins the pieces, in their order
    const int c1 = sh.of(g.first + units_of<C>(it) - 1);
    if (cw == 0 && lane == 0) {
      const unsigned got = atomicAdd(ws.count + c0, 1u);
      s.last = got == (unsigned)(c1 - c0);
      if (s.last) ws.count[c0] = 0;
      __threadfence();
    }
    consumers_sync<CONSUMERS>();
    if (s.last) {
      const int pieces = c1 - c0 + 1;
      for (int e = threadIdx.x - FIRST; e < rows * half_d; e += CONSUMERS * 32) {
        const int row = e / half_d, c = 2 * (e - row * half_d);
        float mm = -INFINITY, sum = 0.0f, x = 0.0f, y = 0.0f;
        for (int i0 = 0; i0 < pieces; i0 += kAhead) {
          float2 q[kAhead], v[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const long long at_row =
                (2LL * (c0 + i0 + i) + (i0 + i == 0 ? 1 : 0)) * kRows + row;
            q[i] = make_float2(-INFINITY, 0.0f);
            v[i] = make_float2(0.0f, 0.0f);
            if (i0 + i < pieces) {
              q[i] = __ldcg(ws.ml + at_row);
              v[i] = __ldcg(reinterpret_cast<const float2*>(ws.o + at_row * D + c));
            }
          }
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const float m2 = fmaxf(mm, q[i].x), base = m2 == -INFINITY ? 0.0f : m2;
            const float a = ex2(mm - base), b = ex2(q[i].x - base);
            mm = m2;
            sum = sum * a + q[i].y * b;
            x = x * a + v[i].x * b;
            y = y * a + v[i].y * b;
          }
        }
        write(row, c, x, y, mm, sum);
      }
    }
  }
}

}  // namespace attn
}  // namespace moe
