// Attention of a few new tokens per sequence over the paged cache (at most 16
// query rows per kv head): decode steps and short drafts.
//
// Bound by the cache's bytes. The key blocks of all (sequence, kv head) items
// are divided evenly over one persistent CTA per SM, so ragged lengths, one
// long sequence and many short ones all keep every SM loading; an item that
// several CTAs hold is joined by the last of them.
//
// Per CTA: warp 0 brings blocks of 64 keys (128 at head sizes up to 64; K and V,
// 128-byte-swizzled boxes of a page) by TMA into a ring of stages. Warps 1-8
// consume: two groups of four take alternate blocks, and each warp a quarter of
// its block's keys, with a running maximum, sum and weighted value sum of its own, so no warp waits for
// another inside an item. The 16 query rows are the M side of mma.sync
// m16n8k16; rows of other tokens and heads of the group fill it. (mma.sync is
// enough: 64 keys take about 500 of its cycles an SM, their bytes 1400 at the
// HBM rate.) At an item's end the eight states are joined in shared memory.
#include "attn_common.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tc;

constexpr int kConsumers = 8;
constexpr int kThreads = (1 + kConsumers) * 32;
constexpr int kRows = kDecodeRows;
constexpr int kStateRows = 4 * kRows;
constexpr int kAhead = 12;  // pieces whose loads are under way together in a join

template <int ND>  // 64-value chunks of a head
struct Smem {
  static constexpr int kD = ND * 64;
  static constexpr int kSub = decode_block(ND) / 64;  // 16-key tiles of a warp in a block
  static constexpr int kTile = 16 * 1024;             // K or V of a block
  static constexpr int kStages = 6;                   // 192 KB in flight
  // A group of warps takes every second block, so every second stage, always
  // the same ones: a warp has to wait for every phase of a barrier it uses.
  static_assert(kStages % 2 == 0, "stages belong to one consumer group each");
  static constexpr int kPad = kD + 4;               // row stride of a state
  uint8_t ring[kStages][2 * kTile];
  // states to be joined: [state][row] with 8 states of 8 rows or 4 of 16
  float o[kStateRows][kPad];
  float2 ml[kStateRows];
  uint64_t full[kStages], empty[kStages];
  long long scan[kThreads / 32];
  long long begin_at;
  int begin_seq, last;
};

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
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

// An item's fixed cost in blocks, counted when the work is divided (four tokens of
// 33 sequences: without it 28.8 us, 28.1 at 3, 24.6 at 6, 26.7 at 9).
constexpr int kItemUnits = 6;
__device__ __forceinline__ int units_of(const Span& r) {
  return r.blocks ? r.blocks + kItemUnits : 0;
}

template <int ND>
__device__ __forceinline__ Span item_of(const AttnParams& p, int s) {
  Span r = read_sequence(p.b, p.page_shift, s, p.err);
  r.blocks = 0;
  if (r.n > 0)  // and at most max_q, which is kRows / group or less
    span_blocks(r, r.kv - r.n, r.kv - 1, p.sc.window, prefix_of(p.sc, s, r.kv), decode_block(ND));
  return r;
}

// The boxes of a page: 64 values of both chunks of a head at once where the
// head has 128 (half as many copies: 16-token pages went from 5.7 to 6.9 TB/s),
// one chunk otherwise.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                        int c0, int row, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(row), "r"(0),
      "r"(head), "r"(page)
      : "memory");
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
template <int ND>
__device__ __forceinline__ bool next_piece(const AttnParams& p, Walk& k, Piece& g) {
  while (k.w < k.hi) {
    g.it = item_of<ND>(p, k.seq);
    const int units = units_of(g.it);
    if (units == 0) {
      ++k.seq;
      continue;
    }
    if (k.head < 0) k.head = (int)quotient(k.w - k.at, units);
    g.seq = k.seq;
    g.head = k.head;
    g.first = k.at + (long long)k.head * units;
    const int u0 = (int)(k.w - g.first), u1 = (int)min((long long)units, u0 + (k.hi - k.w));
    g.n0 = max(0, u0 - kItemUnits);
    g.end = max(0, u1 - kItemUnits);
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

template <typename T, int ND, int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const AttnParams p,
                       const Partials ws) {
  typedef Smem<ND> S;
  constexpr int kBlk = decode_block(ND), kSub = S::kSub;
  // Weights are in units of 2^m, m the running maximum less kUp: fp16 keeps all bits
  // of those down to 2^-29 of the largest then, and not 2^-14 (below 2^-25 they would
  // vanish).
  constexpr float kUp = T::kFp16 ? 15.0f : 0.0f;
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kConsumers / 2);
    }
    fence_mbar_init();
  }
  wait_prior_launch();
  let_next_launch();
  // units of all sequences, and the sequence at which this CTA's share begins
  long long total = 0, lo = 0, at = 0;
  int seq = 0;
  if (p.b.num_seqs <= 32) {  // each warp for itself
    const long long mine = lane < p.b.num_seqs ? (long long)units_of(item_of<ND>(p, lane)) * p.hk : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const Shares sh(total, gridDim.x);
    if ((int)blockIdx.x >= sh.grid) return;
    lo = sh.begin(blockIdx.x);
    seq = __ffs(__ballot_sync(0xffffffffu, lo < incl)) - 1;
    at = __shfl_sync(0xffffffffu, incl - mine, seq);
    __syncthreads();  // the barriers are set up
  } else {
    const int per = (p.b.num_seqs + kThreads - 1) / kThreads;
    const int s0 = min(p.b.num_seqs, (int)threadIdx.x * per);
    const int s1 = min(p.b.num_seqs, s0 + per);
    long long mine = 0;
    for (int q = s0; q < s1; ++q) mine += (long long)units_of(item_of<ND>(p, q)) * p.hk;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += s.scan[i];
      total += s.scan[i];
    }
    const Shares sh(total, gridDim.x);
    if ((int)blockIdx.x >= sh.grid) return;
    lo = sh.begin(blockIdx.x);
    if (lo >= before && lo < before + mine) {
      long long first = before;
      for (int q = s0; q < s1; ++q) {
        const long long c = (long long)units_of(item_of<ND>(p, q)) * p.hk;
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
  Walk walk{at, lo, sh.begin(blockIdx.x + 1), seq, -1};
  Piece g;
  uint32_t stage = 0, ph = 0;
  // a stage holds its boxes one after the other, each [chunk][box_rows][64 values]
  const int ps = 1 << p.page_shift;
  const int box_rows = min(ps, kBlk);
  const int box_bytes = ND * box_rows * 128;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&vmap);
    }
    const int ppb = kBlk / box_rows;                  // boxes of a block
    const bool both = p.head_dim == ND * 64;          // all chunks of a head in one box
    const int per_batch = 32 / ppb;
    uint32_t filled = 0, last_ph = 0;
    bool ok = true;
    while (ok && next_piece<ND>(p, walk, g)) {
      const Span& it = g.it;
      const int head = g.head, end = g.end;
      int n = g.n0;
      const int* table = p.b.page_table + (long long)g.seq * p.b.table_stride;
      const int bi = lane / ppb, pi = lane - bi * ppb;
      // a lane holds the page of box pi of block (batch start + bi), one batch ahead
      const auto fetch = [&](int n0) {
        const int nn = n0 + bi;
        const int kb = (nn < it.near ? nn : nn + it.skip) * kBlk;
        const int key = kb + pi * box_rows;
        int id = 0;
        if (nn < end && key < it.kv) {
          id = __ldg(table + (key >> p.page_shift));
          if (id < 0 || id >= p.num_pages) {
            atomicOr(p.err, kErrRange);
            id = (int)p.num_pages;  // outside the tensor: the box is filled with zeros
          }
        }
        return id;
      };
      int ids = fetch(n);
      while (n < end && ok) {
        const int batch = min(per_batch, end - n);
        const int next = n + batch < end ? fetch(n + batch) : 0;
        for (int i = 0; i < batch; ++i) {
          const int nn = n + i;
          const int kb = (nn < it.near ? nn : nn + it.skip) * kBlk;
          const int boxes = min(ppb, max(0, it.kv - kb + box_rows - 1) / box_rows);
          const int page = __shfl_sync(0xffffffffu, ids, i * ppb + min(lane, ppb - 1));
          int go = 1;
          if (lane == 0) {
            go = bwait(&s.empty[stage], ph ^ 1u, p.err);
            if (go) mbar_arrive_expect_tx(&s.full[stage], 2 * boxes * box_bytes);
          }
          go = __shfl_sync(0xffffffffu, go, 0);
          if (!go) {
            ok = false;
            break;
          }
          if (lane < boxes) {
            const int row = (kb + lane * box_rows) & (ps - 1);
            const uint32_t dst = smem_u32(s.ring[stage]) + lane * box_bytes;
            for (int c = 0; c < (both ? 1 : ND); ++c) {
              const uint32_t to = dst + c * box_rows * 128;
              tma_box(to, &kmap, &s.full[stage], c * 64, row, head, page);
              tma_box(to + S::kTile, &vmap, &s.full[stage], c * 64, row, head, page);
            }
          }
          filled |= 1u << stage;
          last_ph = (last_ph & ~(1u << stage)) | (ph << stage);
          if (++stage == S::kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
        n += batch;
        ids = next;
      }
    }
    // wind down: no TMA copy may still be landing when the CTA exits
    if (lane == 0)
      for (int i = 0; i < S::kStages; ++i)
        if (filled & (1u << i)) mbar_wait(&s.full[i], (last_ph >> i) & 1u, p.err);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int cw = warp - 1, grp = cw >> 2;
  const int gid = lane >> 2, tig = lane & 3;
  const int krow = (cw & 3) * 16 * kSub;                // this warp's keys in a block
  // where its 16-key tiles lie in a stage, and the ldmatrix lane addresses in a
  // tile: K rows by key, V rows by key (transposed on load)
  uint32_t tile_at[kSub];
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int r = krow + 16 * i;
    tile_at[i] = (r / box_rows) * box_bytes + (r % box_rows) * 128;
  }
  const uint32_t chunk = box_rows * 128;
  const int lk_row = (lane & 7) + ((lane >> 4) << 3), lk_c = (lane >> 3) & 1;
  const int lv_row = (lane & 7) + (((lane >> 3) & 1) << 3), lv_c = lane >> 4;
  int parity = 0;                                       // blocks this CTA took so far, mod 2
  bool ok = true;
  while (next_piece<ND>(p, walk, g)) {
    const Span& it = g.it;
    const int head = g.head, n0 = g.n0, end = g.end;
    const int rows = it.n * p.group;
    const int prefix = prefix_of(p.sc, g.seq, it.kv);
    // Q fragments; rows gid and gid + 8 are (token r / group, head r % group)
    uint32_t qf[ND * 4][4];
    int pos[2];
    float slope[2];
    const uint16_t* qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(gid + 8 * i, rows - 1);
      const int tok = r / p.group, h = head * p.group + (r - tok * p.group);
      pos[i] = it.kv - it.n + tok;
      slope[i] = FORM != kPlain && p.sc.slopes ? p.sc.slopes[h] : 0.0f;
      qp[i] = p.q.p + (long long)(it.first + tok) * p.q.token + (long long)h * p.q.head;
    }
#pragma unroll
    for (int k = 0; k < ND * 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = k * 16 + (i >> 1) * 8 + 2 * tig;
        qf[k][i] = c < p.head_dim && gid + 8 * (i & 1) < rows
                       ? __ldg(reinterpret_cast<const uint32_t*>(qp[i & 1] + c))
                       : 0u;
      }
    float o[ND * 8][4];
#pragma unroll
    for (int i = 0; i < ND * 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int n = n0; n < end; ++n) {
      if (parity == grp) {
        if (ok) ok = warp_wait(&s.full[stage], ph, p.err);
        const int k0 = (n < it.near ? n : n + it.skip) * kBlk + krow;
        if (ok && k0 < it.kv) {
          const uint32_t kt = smem_u32(s.ring[stage]), vt = kt + S::kTile;
          if (k0 + 16 * kSub > it.kv) {
            // rows behind the last key may hold anything: V takes part in the
            // product with weight zero, so it is cleared here
            const int from = it.kv - k0;
            for (int i = lane; i < (16 * kSub - from) * ND * 8; i += 32) {
              const int r = krow + from + i / (ND * 8), c = i % (ND * 8);
              sts128(vt + (r / box_rows) * box_bytes + (c >> 3) * chunk + (r % box_rows) * 128 +
                         (c & 7) * 16,
                     0, 0, 0, 0);
            }
            __syncwarp();
          }
          float sacc[2 * kSub][4] = {};
#pragma unroll
          for (int k = 0; k < ND * 4; ++k) {
            const int c = (k & 3) * 2 + lk_c;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4];
              ldsm4(kt + tile_at[i] + (k >> 2) * chunk + lk_row * 128 + ((c ^ (lk_row & 7)) << 4),
                    b);
              mma16<T>(sacc[2 * i], qf[k], b[0], b[1]);
              mma16<T>(sacc[2 * i + 1], qf[k], b[2], b[3]);
            }
          }
          if (FORM != kPlain || !(k0 + 16 * kSub <= it.kv - it.n + 1 && p.sc.window == 0)) {
#pragma unroll
            for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = k0 + t * 8 + 2 * tig + (i & 1), r = i >> 1;
                const int away = pos[r] - key;
                const bool seen =
                    key < it.kv && (key < prefix || (away >= 0 && (p.sc.window == 0 ||
                                                                  away < p.sc.window)));
                sacc[t][i] = seen ? score<FORM>(p.sc, sacc[t][i], slope[r], away) : -INFINITY;
              }
          } else {  // every row sees every key
#pragma unroll
            for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) sacc[t][i] = score<kPlain>(p.sc, sacc[t][i], 0.0f, 0);
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i >> 1] = fmaxf(mx[i >> 1], sacc[t][i]);
          float base[2], scale[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            // up: no numerator above 2^kUp
            mx[r] = fmaxf(m[r], __fadd_ru(mx[r], -kUp));
            base[r] = mx[r] == -INFINITY ? 0.0f : mx[r];
            scale[r] = ex2(m[r] - base[r]);
            m[r] = mx[r];
            l[r] *= scale[r];
          }
          uint32_t pf[kSub][4];
#pragma unroll
          for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float e0 = ex2(sacc[t][2 * r] - base[r]);
              const float e1 = ex2(sacc[t][2 * r + 1] - base[r]);
              l[r] += e0 + e1;
              pf[t >> 1][2 * (t & 1) + r] = T::pack(e0, e1);
            }
          if (__any_sync(0xffffffffu, scale[0] != 1.0f || scale[1] != 1.0f)) {
#pragma unroll
            for (int i = 0; i < ND * 8; ++i) {
              o[i][0] *= scale[0];
              o[i][1] *= scale[0];
              o[i][2] *= scale[1];
              o[i][3] *= scale[1];
            }
          }
#pragma unroll
          for (int d = 0; d < ND * 4; ++d) {
            const int c = (d & 3) * 2 + lv_c;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4];
              ldsm4t(vt + tile_at[i] + (d >> 2) * chunk + lv_row * 128 + ((c ^ (lv_row & 7)) << 4),
                     b);
              mma16<T>(o[2 * d], pf[i], b[0], b[1]);
              mma16<T>(o[2 * d + 1], pf[i], b[2], b[3]);
            }
          }
        }
        // the generic reads (and the cleared rows) come before the next fill
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[stage]);
      }
      parity ^= 1;
      if (++stage == S::kStages) {
        stage = 0;
        ph ^= 1u;
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    // Join the warps' states: with more than 8 rows warps 4-7 first hand theirs
    // to warps 0-3, then all states lie in shared memory and every thread adds up
    // its values of them.
    const auto put = [&](int state, int per_state) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gid + 8 * r;
        if (row >= rows) continue;
        const int at_row = state * per_state + row;
        if (tig == 0) s.ml[at_row] = make_float2(m[r], l[r]);
#pragma unroll
        for (int i = 0; i < ND * 8; ++i)
          *reinterpret_cast<float2*>(&s.o[at_row][i * 8 + 2 * tig]) =
              make_float2(o[i][2 * r], o[i][2 * r + 1]);
      }
    };
    const int states = rows > 8 ? 4 : 8, per_state = rows > 8 ? kRows : 8;
    if (rows > 8) {
      if (cw >= 4) put(cw - 4, kRows);
      consumers_sync();
      if (cw < 4) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = gid + 8 * r;
          if (row >= rows) continue;
          const float2 x = s.ml[cw * kRows + row];
          const float mm = fmaxf(m[r], x.x), base = mm == -INFINITY ? 0.0f : mm;
          const float a = ex2(m[r] - base), b = ex2(x.x - base);
          m[r] = mm;
          l[r] = l[r] * a + x.y * b;
#pragma unroll
          for (int i = 0; i < ND * 8; ++i) {
            const float2 v =
                *reinterpret_cast<const float2*>(&s.o[cw * kRows + row][i * 8 + 2 * tig]);
            o[i][2 * r] = o[i][2 * r] * a + v.x * b;
            o[i][2 * r + 1] = o[i][2 * r + 1] * a + v.y * b;
          }
        }
      }
      consumers_sync();
    }
    if (cw < states) put(cw, per_state);
    consumers_sync();

    const bool split = end - n0 < it.blocks;
    const int c0 = split ? sh.of(g.first + kItemUnits) : 0;  // CTA of the item's first block
    const long long slot = 2LL * blockIdx.x + ((int)blockIdx.x == c0 ? 1 : 0);
    const int half_d = p.head_dim >> 1;
    const auto write = [&](int row, int c, float x, float y, float mm, float sum) {
      const int tok = row / p.group, h = head * p.group + (row - tok * p.group);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<uint32_t*>(p.out.p + (long long)(it.first + tok) * p.out.token +
                                   (long long)h * p.out.head + c) = T::pack(x * inv, y * inv);
      if (p.lse && c == 0)
        p.lse[(long long)(it.first + tok) * p.hq + h] =
            sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * kLn2;
    };
    for (int e = threadIdx.x - 32; e < rows * half_d; e += kConsumers * 32) {
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
        __stcg(reinterpret_cast<float2*>(ws.o + (slot * kRows + row) * S::kD + c),
               make_float2(x, y));
        if (c == 0) __stcg(ws.ml + slot * kRows + row, make_float2(mm, sum));
      }
    }
    if (split) __threadfence();
    consumers_sync();  // the states are read, and a piece is written
    if (split) {
      // the last CTA of the item joins the pieces, in their order
      const int c1 = sh.of(g.first + units_of(it) - 1);
      if (cw == 0 && lane == 0) {
        const unsigned got = atomicAdd(ws.count + c0, 1u);
        s.last = got == (unsigned)(c1 - c0);
        if (s.last) ws.count[c0] = 0;
        __threadfence();
      }
      consumers_sync();
      if (s.last) {
        const int pieces = c1 - c0 + 1;
        for (int e = threadIdx.x - 32; e < rows * half_d; e += kConsumers * 32) {
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
                v[i] = __ldcg(reinterpret_cast<const float2*>(ws.o + at_row * S::kD + c));
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
}

template <int ND>
constexpr int smem_bytes() {
  return (int)sizeof(Smem<ND>) + 1024;
}
static_assert(smem_bytes<1>() <= 227 * 1024 && smem_bytes<2>() <= 227 * 1024,
              "shared memory of a CTA");

template <typename F>
cudaError_t setup_one(F f, int bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <typename T, int ND>
cudaError_t setup_nd() {
  cudaError_t e;
  if ((e = setup_one(attn_decode_kernel<T, ND, kPlain>, smem_bytes<ND>())) != cudaSuccess) return e;
  if ((e = setup_one(attn_decode_kernel<T, ND, kGeneral>, smem_bytes<ND>())) != cudaSuccess)
    return e;
  return setup_one(attn_decode_kernel<T, ND, kWide>, smem_bytes<ND>());
}

template <typename T, int ND>
cudaError_t launch_one(const AttnParams& p, const Partials& w, const CUtensorMap& kmap,
                       const CUtensorMap& vmap, int grid, cudaStream_t s) {
  const Form form = form_of(p.sc);
  return launch_after(form == kPlain     ? attn_decode_kernel<T, ND, kPlain>
                      : form == kGeneral ? attn_decode_kernel<T, ND, kGeneral>
                                         : attn_decode_kernel<T, ND, kWide>,
                      dim3(grid), dim3(kThreads), smem_bytes<ND>(), s, kmap, vmap, p, w);
}

}  // namespace

cudaError_t attn_decode_setup() {
  cudaError_t e;
  if ((e = setup_nd<Bf16, 1>()) != cudaSuccess) return e;
  if ((e = setup_nd<Bf16, 2>()) != cudaSuccess) return e;
  if ((e = setup_nd<Fp16, 1>()) != cudaSuccess) return e;
  return setup_nd<Fp16, 2>();
}

cudaError_t launch_attn_decode(const AttnParams& p, const Partials& w, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, int dtype, int grid, cudaStream_t s) {
  const bool wide = p.head_dim > 64;
  if (dtype == MOE_ATTN_BF16)
    return wide ? launch_one<Bf16, 2>(p, w, kmap, vmap, grid, s)
                : launch_one<Bf16, 1>(p, w, kmap, vmap, grid, s);
  return wide ? launch_one<Fp16, 2>(p, w, kmap, vmap, grid, s)
              : launch_one<Fp16, 1>(p, w, kmap, vmap, grid, s);
}

}  // namespace attn
}  // namespace moe
