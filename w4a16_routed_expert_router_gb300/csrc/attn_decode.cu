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
#include "attn_decode_parts.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = (1 + kConsumers) * 32;

template <int ND>
struct Split {
  static constexpr int kBlk = decode_block(ND);
  // four tokens of 33 sequences: without it 28.8 us, 28.1 at 3, 24.6 at 6, 26.7 at 9
  static constexpr int kItem = 6;
};

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

// A state in a warp: rows gid and gid + 8, two columns of each 8-value tile of the
// products.
template <int ND>
struct StateOf {
  typedef float Values[ND * 8][4];
  static constexpr int kRows = 2, kLanes = 1;  // lanes 1 and 2 apart have other keys of a row
  static __device__ __forceinline__ int row(int r, int lane) { return (lane >> 2) + 8 * r; }
  static __device__ __forceinline__ bool first(int lane) { return (lane & 3) == 0; }
  static __device__ __forceinline__ void put(float* row, const Values& o, int r, int lane) {
#pragma unroll
    for (int i = 0; i < ND * 8; ++i)
      *reinterpret_cast<float2*>(row + i * 8 + 2 * (lane & 3)) =
          make_float2(o[i][2 * r], o[i][2 * r + 1]);
  }
  // o = o a + row b
  static __device__ __forceinline__ void add(const float* row, Values& o, int r, int lane, float a,
                                             float b) {
#pragma unroll
    for (int i = 0; i < ND * 8; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(row + i * 8 + 2 * (lane & 3));
      o[i][2 * r] = o[i][2 * r] * a + v.x * b;
      o[i][2 * r + 1] = o[i][2 * r + 1] * a + v.y * b;
    }
  }
};

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
  long long total;
  Walk walk;
  if (!begin_share<Split<ND>, kThreads>(p, s, total, walk)) return;
  const Shares sh(total, gridDim.x);
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
    while (ok && next_piece<Split<ND>>(p, walk, g)) {
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
  while (next_piece<Split<ND>>(p, walk, g)) {
    const Span& it = g.it;
    const int head = g.head, n0 = g.n0, end = g.end;
    const int rows = it.n * p.group;
    const int prefix = prefix_of(p.sc, g.seq, it.kv);
    // Q fragments; rows gid and gid + 8 are (token r / group, head r % group)
    uint32_t qf[ND * 4][4];
    int pos[2], kept[2];
    float slope[2];
    const uint16_t* qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(gid + 8 * i, rows - 1);
      const int tok = r / p.group, h = head * p.group + (r - tok * p.group);
      pos[i] = it.kv - it.n + tok;
      kept[i] = kept_of(p.sc, prefix, pos[i]);
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
                    key < it.kv && (key < kept[r] || (away >= 0 && (p.sc.window == 0 ||
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
    finish_item<Split<ND>, StateOf<ND>, 32, kConsumers, S::kD>(
        p, ws, s, sh, g, cw, o, m, l, [](float x, float y) { return T::pack(x, y); });
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
