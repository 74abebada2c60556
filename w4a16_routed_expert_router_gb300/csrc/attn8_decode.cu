// Attention of a few new tokens per sequence (at most 16 query rows per kv head) over
// the 8-bit cache: decode steps and short drafts.
//
// Bound by the cache's bytes; the division of the work, the roles and the joins are
// those of attn_decode.cu, on blocks of 128 keys (256 at head sizes up to 64), 32 KB of
// codes, in a ring of 6 stages. A key's codes are 128 (64) bytes: one swizzled row, and
// one box brings a page's rows whole. The scales, one for 16 keys, come with the block
// by asynchronous copies of 4 bytes.
//
// The keys are the M side of mma.sync m16n8k16 and the query rows the N side, 8 or 16
// of them (S^T = K Q^T, O^T = V^T P^T): codes are converted once for all rows, and up
// to 8 rows take half of the products, sums and registers of 16, so that more
// warps fit. (With the rows as the M side, 8 warps took 373 us for 64 sequences of up to
// 16384 keys, at a third of the issue slots and 16 % of the matrix unit: latency.)
//
// Codes go to fp16 in registers, two an instruction. ldmatrix deals in units of 16
// bits, so a thread gets 4 values of a key in a row, (4 tig .. 4 tig + 3) of a 16-value
// step: the sum over a head does not mind the order, and Q is laid out alike. Of V it
// gets 2 values of 2 keys; their middle bytes change places, and rows gid and gid + 8 of
// the product are values 2 gid and 2 gid + 1 of 16.
//
// Scales. S = (q.k) (scale sk) with the key's scale sk. With v = code * sv, weights
// enter the product as p sv: the exponent takes log2 sv, the running maximum is of
// x + log2 sv, so that no numerator leaves fp16's range however the scales differ, and
// the sum of weights takes 1 / sv back, once for 16 keys. bf16 queries become fp16 by a
// power of two of their own for each row.
//
// 64 sequences of up to 16384 keys, 8 kv heads of 128, take 185 us (1.1 GB, 5.9 TB/s of
// codes and scales; 16-bit keys take 331). Four drafted tokens of 48 sequences under a
// window of 4096, heads of 64, take 45 us for 100 MB: a block of 32 KB takes 0.9 us an SM,
// 23 of them 20 us, and the ends and joins of two to three pieces an SM most of the rest.
// 9 to 16 rows of heads of 128 (64 sequences of up to 16384 keys, 4 tokens each, 1.4 GB)
// take 354 us, 225 with one token: twice the products and sums on eight warps of 168
// registers, of which 80 to 130 bytes a thread go to memory and back.
// One token over 4096 keys is a chain of latencies as in attn_decode.cu, 11 us.
#include "attn8_parts.cuh"
#include "attn_decode_parts.cuh"

namespace moe {
namespace attn {
namespace {

// Warps that consume, in groups of four that take blocks in turn. (Twelve for two row
// tiles of small heads, whose registers then spill: 45 -> 64 us for 48 drafts.)
template <int NT>
constexpr int kConsumers = NT == 1 ? 12 : 8;
// Before them four that produce: K, V, scales; the last of them fills the warpgroup. (One
// warp for all issued a box in 75 cycles and took 1000 for a block with its scales: 363
// us for 64 sequences in 16-token pages, 216 without any arithmetic in 64-token pages.)
constexpr int kProducers = 4;
template <int NT>
constexpr int kThreads = (kProducers + kConsumers<NT>) * 32;

template <int ND>
struct Split {
  static constexpr int kBlk = decode8_block(ND);
  static constexpr int kItem = 3;  // as much as in attn_decode.cu
};

template <int ND, int NT>  // 64-value chunks of a head, row tiles
struct Smem {
  static constexpr int kD = ND * 64;
  static constexpr int kRow = ND * 64;                // bytes of a key's codes
  static constexpr int kBlk = decode8_block(ND);
  static constexpr int kSub = kBlk / 64;              // 16-key tiles of a warp in a block
  static constexpr int kTile = 16 * 1024;             // K or V of a block
  static constexpr int kGroupsOfWarps = kConsumers<NT> / 4;
  static constexpr int kStages = ND * NT <= 2 ? 6 : 4;  // 192 or 128 KB in flight
  static constexpr int kStateRows = kConsumers<NT> / 2 * 8 * NT;
  static_assert(kTile == kBlk * kRow, "a block's codes");
  // a warp has to wait for every phase of a barrier it uses
  static_assert(kStages % kGroupsOfWarps == 0, "stages belong to one consumer group each");
  static constexpr int kPad = kD + 4;                 // row stride of a state
  uint8_t ring[kStages][2 * kTile];
  float scales[kStages][2][kBlk / kScaleBlock];       // K's, V's
  // states to be joined: [state][row] with 8 states of 8 rows or 4 of 16
  float o[kStateRows][kPad];
  float2 ml[kStateRows];
  uint64_t full[kStages], empty[kStages];
  long long scan[kThreads<NT> / 32];
  long long begin_at;
  int begin_seq, last;
};

// A state in a warp: rows 2 tig and 2 tig + 1 of each tile, of 16 values 2 gid and the
// next.
template <int ND, int NT>
struct State8 {
  typedef float Values[NT][ND * 4][4];
  static constexpr int kRows = 2 * NT, kLanes = 4;  // lanes 4, 8, 16 apart: other keys of a row
  static __device__ __forceinline__ int row(int r, int lane) {
    return 8 * (r >> 1) + 2 * (lane & 3) + (r & 1);
  }
  static __device__ __forceinline__ bool first(int lane) { return lane < 4; }
  static __device__ __forceinline__ void put(float* row, const Values& o, int r, int lane) {
#pragma unroll
    for (int i = 0; i < ND * 4; ++i)
      *reinterpret_cast<float2*>(row + i * 16 + 2 * (lane >> 2)) =
          make_float2(o[r >> 1][i][r & 1], o[r >> 1][i][2 + (r & 1)]);
  }
  // o = o a + row b
  static __device__ __forceinline__ void add(const float* row, Values& o, int r, int lane, float a,
                                             float b) {
#pragma unroll
    for (int i = 0; i < ND * 4; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(row + i * 16 + 2 * (lane >> 2));
      float(&to)[4] = o[r >> 1][i];
      to[r & 1] = to[r & 1] * a + v.x * b;
      to[2 + (r & 1)] = to[2 + (r & 1)] * a + v.y * b;
    }
  }
};

// an 8 x 8 tile of 16-bit values, rows by columns, turned over its diagonal
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int ND>
__device__ __forceinline__ uint32_t swizzled(int row, int unit) {
  return (unit ^ (ND == 2 ? row & 7 : (row >> 1) & 3)) << 4;
}

template <int ND, int NT, int FORM>
__global__ void __launch_bounds__(kThreads<NT>, 1)
    attn8_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ Attn8Params g8,
                        const __grid_constant__ Partials ws) {
  typedef Smem<ND, NT> S;
  typedef State8<ND, NT> State;
  constexpr int R = State::kRows;
  const AttnParams& p = g8.a;
  constexpr int kBlk = S::kBlk, kSub = S::kSub, kUnits = ND * 4;
  constexpr float kUp = 15.0f;  // see attn_decode.cu
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s.full[i], 2 + 32);  // K, V, and each lane's scales
      mbar_init(&s.empty[i], 4);
    }
    fence_mbar_init();
  }
  wait_prior_launch();
  let_next_launch();
  long long total;
  Walk walk;
  if (!begin_share<Split<ND>, kThreads<NT>>(p, s, total, walk)) return;
  const Shares sh(total, gridDim.x);
  Piece g;
  uint32_t stage = 0, ph = 0;
  // a stage holds its boxes one after the other, each [box_rows][kRow bytes]
  const int ps = 1 << p.page_shift;
  const int box_rows = min(ps, kBlk);
  const int box_bytes = box_rows * S::kRow;

  if (warp < kProducers) {
    // ---------------------------------------------------------------- producers
    if (warp == kProducers - 1) return;
    const bool scaler = warp == 2;
    const CUtensorMap* map = warp == 0 ? &kmap : &vmap;
    if (lane == 0 && !scaler) prefetch_tmap(map);
    const int ppb = kBlk / box_rows;                  // boxes of a block
    const int per_batch = 32 / ppb;
    // scales: lanes 0 .. 2 kGroups - 1 bring those of 16 keys each, K's then V's
    constexpr int kGroups = kBlk / kScaleBlock;
    const int grp = lane & (kGroups - 1);
    const float* scale_base = lane < kGroups ? g8.c.k_scales : g8.c.v_scales;
    const int grp_box = min(grp * kScaleBlock / box_rows, ppb - 1);  // the box of its scale
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
          if (!(ok = warp_wait(&s.empty[stage], ph ^ 1u, p.err))) break;
          if (scaler) {
            const int page = __shfl_sync(0xffffffffu, ids, i * ppb + grp_box);
            if (lane < 2 * kGroups) {
              const int key = kb + grp * kScaleBlock;
              const bool there = key < it.kv && page < p.num_pages;
              const long long at = there ? page * g8.c.scale_page + head * g8.c.scale_head +
                                               ((key & (ps - 1)) / kScaleBlock) * g8.c.scale_block
                                         : 0;
              copy4_async(smem_u32(&s.scales[stage][0][0]) + lane * 4, scale_base + at, there);
            }
            arrive_after_copies(&s.full[stage]);
          } else {
            uint32_t dst = smem_u32(s.ring[stage]) + (warp == 1 ? S::kTile : 0);
            if (one_thread()) mbar_arrive_expect_tx(&s.full[stage], boxes * box_bytes);
            for (int j = 0; j < boxes; ++j, dst += box_bytes) {
              const int page = __shfl_sync(0xffffffffu, ids, i * ppb + j);
              if (one_thread())
                tma_page(dst, map, &s.full[stage], 0, (kb + j * box_rows) & (ps - 1), head, page);
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
    // wind down: no copy may still be landing when the CTA exits
    if (lane == 0)
      for (int i = 0; i < S::kStages; ++i)
        if (filled & (1u << i)) mbar_wait(&s.full[i], (last_ph >> i) & 1u, p.err);
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int cw = warp - kProducers, grp = cw >> 2;
  const int gid = lane >> 2, tig = lane & 3;
  const int krow = (cw & 3) * 16 * kSub;                // this warp's keys in a block
  // where its 16-key tiles lie in a stage, and the ldmatrix lane addresses in a
  // tile: K rows by key, V rows by key (transposed on load)
  uint32_t tile_at[kSub];
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int r = krow + 16 * i;
    tile_at[i] = (r / box_rows) * box_bytes + (r % box_rows) * S::kRow;
  }
  const int lk_row = (lane & 7) + ((lane >> 4) << 3), lk_c = (lane >> 3) & 1;
  const int lv_row = (lane & 7) + (((lane >> 3) & 1) << 3), lv_c = lane >> 4;
  const int units = p.head_dim >> 4;
  const bool bf16 = g8.dtype == MOE_ATTN_BF16;
  int turn = 0;                                         // blocks this CTA took so far, mod groups
  bool ok = true;
  while (next_piece<Split<ND>>(p, walk, g)) {
    const Span& it = g.it;
    const int head = g.head, n0 = g.n0, end = g.end;
    const int rows = it.n * p.group;
    const int prefix = prefix_of(p.sc, g.seq, it.kv);
    // Q fragments: row gid of each tile, (token r / group, head r % group)
    uint32_t qf[NT][kUnits][2];
    float down[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = min(gid + 8 * t, rows - 1);
      const int tok = r / p.group, h = head * p.group + (r - tok * p.group);
      const uint16_t* qp =
          p.q.p + (long long)(it.first + tok) * p.q.token + (long long)h * p.q.head + 4 * tig;
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const uint2 w = k < units && gid + 8 * t < rows
                            ? __ldg(reinterpret_cast<const uint2*>(qp + 16 * k))
                            : make_uint2(0, 0);
        qf[t][k][0] = w.x;
        qf[t][k][1] = w.y;
        if (bf16) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = fmaxf(top, fmaxf(fabsf(bf16_bits_to_f32((uint16_t)qf[t][k][i])),
                                   fabsf(bf16_bits_to_f32((uint16_t)(qf[t][k][i] >> 16)))));
        }
      }
      down[t] = 1.0f;
      if (bf16) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const RowUnit u(top);
        down[t] = u.down;
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[t][k][i] = Fp16::pack(bf16_bits_to_f32((uint16_t)qf[t][k][i]) * u.up,
                                     bf16_bits_to_f32((uint16_t)(qf[t][k][i] >> 16)) * u.up);
      }
    }
    // the rows whose scores this thread gets, see State8
    int pos[R], kept[R];
    float slope[R], unit[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = min(State::row(i, lane), rows - 1);
      const int tok = r / p.group, h = head * p.group + (r - tok * p.group);
      pos[i] = it.kv - it.n + tok;
      kept[i] = kept_of(p.sc, prefix, pos[i]);
      slope[i] = FORM != kPlain && p.sc.slopes ? p.sc.slopes[h] : 0.0f;
      unit[i] = __shfl_sync(0xffffffffu, down[i >> 1], (2 * tig + (i & 1)) * 4);
      if (FORM == kPlain) unit[i] *= p.sc.scale * kLog2e;
    }
    typename State::Values o;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][i][j] = 0.0f;
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = -INFINITY, l[r] = 0.0f;

    for (int n = n0; n < end; ++n) {
      if (turn == grp) {
        if (ok) ok = warp_wait(&s.full[stage], ph, p.err);
        const int k0 = (n < it.near ? n : n + it.skip) * kBlk + krow;
        if (ok && k0 < it.kv) {
          const uint32_t kt = smem_u32(s.ring[stage]), vt = kt + S::kTile;
          if (k0 + 16 * kSub > it.kv) {
            // rows behind the last key may hold anything: V takes part in the
            // product with weight zero, so it is cleared here
            const int from = it.kv - k0;
            for (int i = lane; i < (16 * kSub - from) * kUnits; i += 32) {
              const int r = krow + from + i / kUnits, c = i % kUnits;
              sts128(vt + (r / box_rows) * box_bytes + (r % box_rows) * S::kRow + c * 16, 0, 0, 0,
                     0);
            }
            __syncwarp();
          }
          float sk[kSub], lv[kSub], back[kSub];  // scale of K, log2 of V's, its inverse
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            sk[i] = scale_in_range(s.scales[stage][0][krow / 16 + i]);
            lv[i] = log2_of_scale(scale_in_range(s.scales[stage][1][krow / 16 + i]));
            back[i] = ex2(-lv[i]);
          }
          float x[kSub][NT][4] = {};
#pragma unroll
          for (int k = 0; k < kUnits / 2; ++k) {
            if (2 * k >= units) break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4], a[2][4];
              ldsm4(kt + tile_at[i] + lk_row * S::kRow + swizzled<ND>(lk_row, 2 * k + lk_c), b);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                a[u][0] = f16_of_codes(b[u], false);
                a[u][1] = f16_of_codes(b[2 + u], false);
                a[u][2] = f16_of_codes(b[u], true);
                a[u][3] = f16_of_codes(b[2 + u], true);
              }
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma16<Fp16>(x[i][t], a[u], qf[t][2 * k + u][0], qf[t][2 * k + u][1]);
            }
          }
          // x[i][t][j]: key 16 i + gid + 8 (j >> 1), row 2 tig + (j & 1) of tile t
          // every row of the sequence sees every key of the warp's, or not
          const bool whole = k0 + 16 * kSub <= it.kv - it.n + 1 &&
                             (p.sc.window == 0 || k0 > it.kv - 1 - p.sc.window);
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = 2 * t + (j & 1);
                x[i][t][j] *= unit[r] * sk[i];
                if (FORM != kPlain)
                  x[i][t][j] = score<FORM>(p.sc, x[i][t][j], slope[r],
                                           pos[r] - (k0 + 16 * i + gid + 8 * (j >> 1)));
              }
          if (!whole) {
#pragma unroll
            for (int i = 0; i < kSub; ++i)
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int r = 2 * t + (j & 1);
                  const int key = k0 + 16 * i + gid + 8 * (j >> 1), away = pos[r] - key;
                  const bool seen =
                      key < it.kv && (key < kept[r] || (away >= 0 && (p.sc.window == 0 ||
                                                                      away < p.sc.window)));
                  if (!seen) x[i][t][j] = -INFINITY;
                }
          }
          float base[R], scale[R];
          bool moved = false;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < kSub; ++i)
              mx = fmaxf(mx, fmaxf(x[i][r >> 1][r & 1], x[i][r >> 1][2 + (r & 1)]) + lv[i]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            // up: no numerator above 2^kUp
            mx = fmaxf(m[r], __fadd_ru(mx, -kUp));
            base[r] = mx == -INFINITY ? 0.0f : mx;
            scale[r] = ex2(m[r] - base[r]);
            m[r] = mx;
            l[r] *= scale[r];
            moved |= scale[r] != 1.0f;
          }
          uint32_t pf[kSub][NT][2];
#pragma unroll
          for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float e[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) e[j] = ex2(x[i][t][j] - (base[2 * t + (j & 1)] - lv[i]));
              l[2 * t] = fmaf(e[0] + e[2], back[i], l[2 * t]);
              l[2 * t + 1] = fmaf(e[1] + e[3], back[i], l[2 * t + 1]);
              pf[i][t][0] = transposed(Fp16::pack(e[0], e[1]));
              pf[i][t][1] = transposed(Fp16::pack(e[2], e[3]));
            }
          if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < kUnits; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][i][j] *= scale[2 * t + (j & 1)];
          }
#pragma unroll
          for (int d = 0; d < kUnits / 2; ++d) {
            if (2 * d >= units) break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4];
              ldsm4t(vt + tile_at[i] + lv_row * S::kRow + swizzled<ND>(lv_row, 2 * d + lv_c), b);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint32_t lo = __byte_perm(b[2 * u], 0, 0x3120);
                const uint32_t hi = __byte_perm(b[2 * u + 1], 0, 0x3120);
                const uint32_t a[4] = {f16_of_codes(lo, false), f16_of_codes(lo, true),
                                       f16_of_codes(hi, false), f16_of_codes(hi, true)};
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma16<Fp16>(o[t][2 * d + u], a, pf[i][t][0], pf[i][t][1]);
              }
            }
          }
        }
        // the generic reads (and the cleared rows) come before the next fill
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[stage]);
      }
      if (++turn == S::kGroupsOfWarps) turn = 0;
      if (++stage == S::kStages) {
        stage = 0;
        ph ^= 1u;
      }
    }
    finish_item<Split<ND>, State, kProducers * 32, kConsumers<NT>, S::kD>(
        p, ws, s, sh, g, cw, o, m, l,
        [bf16](float x, float y) { return bf16 ? Bf16::pack(x, y) : Fp16::pack(x, y); });
  }
}

template <int ND, int NT>
constexpr int smem_bytes() {
  return (int)sizeof(Smem<ND, NT>) + 1024;
}
static_assert(smem_bytes<1, 1>() <= 227 * 1024 && smem_bytes<2, 1>() <= 227 * 1024 &&
                  smem_bytes<1, 2>() <= 227 * 1024 && smem_bytes<2, 2>() <= 227 * 1024,
              "shared memory of a CTA");

template <int ND, int NT>
cudaError_t setup_nd() {
  cudaError_t e = cudaSuccess;
  for (auto f : {attn8_decode_kernel<ND, NT, kPlain>, attn8_decode_kernel<ND, NT, kGeneral>,
                 attn8_decode_kernel<ND, NT, kWide>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               smem_bytes<ND, NT>());
  return e;
}

template <int ND, int NT>
cudaError_t launch_nd(const Attn8Params& p, const Partials& w, const CUtensorMap& kmap,
                      const CUtensorMap& vmap, int grid, cudaStream_t s) {
  const Form form = form_of(p.a.sc);
  return launch_after(form == kPlain     ? attn8_decode_kernel<ND, NT, kPlain>
                      : form == kGeneral ? attn8_decode_kernel<ND, NT, kGeneral>
                                         : attn8_decode_kernel<ND, NT, kWide>,
                      dim3(grid), dim3(kThreads<NT>), smem_bytes<ND, NT>(), s, kmap, vmap, p, w);
}

}  // namespace

cudaError_t attn8_decode_setup() {
  cudaError_t e = setup_nd<1, 1>();
  if (e == cudaSuccess) e = setup_nd<1, 2>();
  if (e == cudaSuccess) e = setup_nd<2, 1>();
  return e != cudaSuccess ? e : setup_nd<2, 2>();
}

cudaError_t launch_attn8_decode(const Attn8Params& p, const Partials& w, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, int grid, cudaStream_t s) {
  const bool wide = p.a.head_dim > 64;
  if ((long long)p.a.b.max_q * p.a.group <= 8)
    return wide ? launch_nd<2, 1>(p, w, kmap, vmap, grid, s)
                : launch_nd<1, 1>(p, w, kmap, vmap, grid, s);
  return wide ? launch_nd<2, 2>(p, w, kmap, vmap, grid, s)
              : launch_nd<1, 2>(p, w, kmap, vmap, grid, s);
}

}  // namespace attn
}  // namespace moe
