// Attention of a few new tokens per sequence (at most 16 query rows per kv head) over
// the 8-bit cache: decode steps and short drafts.
//
// Bound by the cache's bytes; the division of the work, the roles and the joins are
// those of attn_decode.cu, on blocks of 64 keys (128 at head sizes up to 64), 16 KB of
// codes, in a ring of 10 stages. A key's codes are 128 (64) bytes: one swizzled row, and
// one box brings a page's rows whole. The scales, one for 16 keys, come with the block
// by asynchronous copies of 4 bytes.
//
// Codes go to fp16 in registers, two an instruction. ldmatrix deals in units of 16
// bits, so a thread gets 4 values of a key in a row, (4 tig .. 4 tig + 3) of a 16-value
// step: the sum over a head does not mind the order, and Q is laid out alike. Of V it
// gets 2 values of 2 keys; their middle bytes change places, and the columns of two
// neighbouring tiles of the result are the even and the odd values of 16.
//
// Scales. S = (q.k) (scale sk) with the key's scale sk. With v = code * sv, weights
// enter the product as p sv: the exponent takes log2 sv, the running maximum is of
// x + log2 sv, so that no numerator leaves fp16's range however the scales differ, and
// the sum of weights takes 1 / sv back, once for 16 keys. bf16 queries become fp16 by a
// power of two of their own for each row.
#include "attn8_parts.cuh"
#include "attn_decode_parts.cuh"

namespace moe {
namespace attn {
namespace {

template <int ND>  // 64-value chunks of a head
struct Smem {
  static constexpr int kD = ND * 64;
  static constexpr int kRow = ND * 64;                // bytes of a key's codes
  static constexpr int kBlk = decode8_block(ND);
  static constexpr int kSub = kBlk / 64;              // 16-key tiles of a warp in a block
  static constexpr int kTile = 8 * 1024;              // K or V of a block
  static constexpr int kStages = 10;                  // 160 KB in flight
  static_assert(kTile == kBlk * kRow, "a block's codes");
  static_assert(kStages % 2 == 0, "stages belong to one consumer group each");
  static constexpr int kPad = kD + 4;                 // row stride of a state
  uint8_t ring[kStages][2 * kTile];
  float scales[kStages][2][kBlk / kScaleBlock];       // K's, V's
  // states to be joined: [state][row] with 8 states of 8 rows or 4 of 16
  float o[kStateRows][kPad];
  float2 ml[kStateRows];
  uint64_t full[kStages], empty[kStages];
  long long scan[kThreads / 32];
  long long begin_at;
  int begin_seq, last;
};

// A state's values in a warp: of 16 values, a thread has 4 in a row.
template <int ND>
struct State8 {
  typedef float Values[ND * 8][4];
  static __device__ __forceinline__ void put(float* row, const Values& o, int r, int tig) {
#pragma unroll
    for (int i = 0; i < ND * 4; ++i)
      *reinterpret_cast<float4*>(row + i * 16 + 4 * tig) =
          make_float4(o[2 * i][2 * r], o[2 * i + 1][2 * r], o[2 * i][2 * r + 1],
                      o[2 * i + 1][2 * r + 1]);
  }
  // o = o a + row b
  static __device__ __forceinline__ void add(const float* row, Values& o, int r, int tig, float a,
                                             float b) {
#pragma unroll
    for (int i = 0; i < ND * 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(row + i * 16 + 4 * tig);
      o[2 * i][2 * r] = o[2 * i][2 * r] * a + v.x * b;
      o[2 * i + 1][2 * r] = o[2 * i + 1][2 * r] * a + v.y * b;
      o[2 * i][2 * r + 1] = o[2 * i][2 * r + 1] * a + v.z * b;
      o[2 * i + 1][2 * r + 1] = o[2 * i + 1][2 * r + 1] * a + v.w * b;
    }
  }
};

template <int ND>
__device__ __forceinline__ uint32_t swizzled(int row, int unit) {
  return (unit ^ (ND == 2 ? row & 7 : (row >> 1) & 3)) << 4;
}

template <int ND, int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    attn8_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ Attn8Params g8,
                        const __grid_constant__ Partials ws) {
  typedef Smem<ND> S;
  const AttnParams& p = g8.a;
  constexpr int kBlk = S::kBlk, kSub = S::kSub, kUnits = ND * 4;
  constexpr float kUp = 15.0f;  // see attn_decode.cu
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s.full[i], 1 + 32);  // the codes, and each lane's scales
      mbar_init(&s.empty[i], kConsumers / 2);
    }
    fence_mbar_init();
  }
  wait_prior_launch();
  let_next_launch();
  long long total;
  Walk walk;
  if (!begin_share<kBlk>(p, s, total, walk)) return;
  const Shares sh(total, gridDim.x);
  Piece g;
  uint32_t stage = 0, ph = 0;
  // a stage holds its boxes one after the other, each [box_rows][kRow bytes]
  const int ps = 1 << p.page_shift;
  const int box_rows = min(ps, kBlk);
  const int box_bytes = box_rows * S::kRow;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&vmap);
    }
    const int ppb = kBlk / box_rows;                  // boxes of a block
    const int per_batch = 32 / ppb;
    // lanes 0 .. 2 kGroups - 1 bring the scales of 16 keys each, K's then V's
    constexpr int kGroups = kBlk / kScaleBlock;
    const int grp = lane & (kGroups - 1);
    const bool scaler = lane < 2 * kGroups;
    const float* scale_base = lane < kGroups ? g8.c.k_scales : g8.c.v_scales;
    uint32_t filled = 0, last_ph = 0;
    bool ok = true;
    while (ok && next_piece<kBlk>(p, walk, g)) {
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
          const int scale_page =
              __shfl_sync(0xffffffffu, ids, i * ppb + min(grp * kScaleBlock / box_rows, ppb - 1));
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
          __syncwarp();
          if (scaler) {
            const int key = kb + grp * kScaleBlock;
            const bool there = key < it.kv && scale_page < p.num_pages;
            const long long at = there ? scale_page * g8.c.scale_page + head * g8.c.scale_head +
                                             ((key & (ps - 1)) / kScaleBlock) * g8.c.scale_block
                                       : 0;
            copy4_async(smem_u32(&s.scales[stage][0][0]) + lane * 4, scale_base + at, there);
          }
          arrive_after_copies(&s.full[stage]);
          if (lane < boxes) {
            const int row = (kb + lane * box_rows) & (ps - 1);
            const uint32_t dst = smem_u32(s.ring[stage]) + lane * box_bytes;
            tma_page(dst, &kmap, &s.full[stage], 0, row, head, page);
            tma_page(dst + S::kTile, &vmap, &s.full[stage], 0, row, head, page);
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
  const int cw = warp - 1, grp = cw >> 2;
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
  int parity = 0;                                       // blocks this CTA took so far, mod 2
  bool ok = true;
  while (next_piece<kBlk>(p, walk, g)) {
    const Span& it = g.it;
    const int head = g.head, n0 = g.n0, end = g.end;
    const int rows = it.n * p.group;
    const int prefix = prefix_of(p.sc, g.seq, it.kv);
    // Q fragments; rows gid and gid + 8 are (token r / group, head r % group)
    uint32_t qf[kUnits][4];
    int pos[2], kept[2];
    float slope[2], unit[2] = {1.0f, 1.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(gid + 8 * i, rows - 1);
      const int tok = r / p.group, h = head * p.group + (r - tok * p.group);
      pos[i] = it.kv - it.n + tok;
      kept[i] = kept_of(p.sc, prefix, pos[i]);
      slope[i] = FORM != kPlain && p.sc.slopes ? p.sc.slopes[h] : 0.0f;
      const uint16_t* qp =
          p.q.p + (long long)(it.first + tok) * p.q.token + (long long)h * p.q.head + 4 * tig;
      uint2 w[kUnits];
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        w[k] = k < units && gid + 8 * i < rows ? __ldg(reinterpret_cast<const uint2*>(qp + 16 * k))
                                               : make_uint2(0, 0);
        if (bf16)
          top = fmaxf(fmaxf(top, fmaxf(fabsf(bf16_bits_to_f32((uint16_t)w[k].x)),
                                       fabsf(bf16_bits_to_f32((uint16_t)(w[k].x >> 16))))),
                      fmaxf(fabsf(bf16_bits_to_f32((uint16_t)w[k].y)),
                            fabsf(bf16_bits_to_f32((uint16_t)(w[k].y >> 16)))));
      }
      if (bf16) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const RowUnit u(top);
        unit[i] = u.down;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
          w[k].x = Fp16::pack(bf16_bits_to_f32((uint16_t)w[k].x) * u.up,
                              bf16_bits_to_f32((uint16_t)(w[k].x >> 16)) * u.up);
          w[k].y = Fp16::pack(bf16_bits_to_f32((uint16_t)w[k].y) * u.up,
                              bf16_bits_to_f32((uint16_t)(w[k].y >> 16)) * u.up);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        qf[k][i] = w[k].x;
        qf[k][2 + i] = w[k].y;
      }
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
            const int t = krow / 16 + i;
            sk[i] = scale_in_range(s.scales[stage][0][t]);
            lv[i] = log2_of_scale(scale_in_range(s.scales[stage][1][t]));
            back[i] = ex2(-lv[i]);
          }
          float sacc[2 * kSub][4] = {};
#pragma unroll
          for (int k = 0; k < kUnits / 2; ++k) {
            if (2 * k >= units) break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4];
              ldsm4(kt + tile_at[i] + lk_row * S::kRow + swizzled<ND>(lk_row, 2 * k + lk_c), b);
              mma16<Fp16>(sacc[2 * i], qf[2 * k], f16_of_codes(b[0], false),
                          f16_of_codes(b[0], true));
              mma16<Fp16>(sacc[2 * i + 1], qf[2 * k], f16_of_codes(b[2], false),
                          f16_of_codes(b[2], true));
              mma16<Fp16>(sacc[2 * i], qf[2 * k + 1], f16_of_codes(b[1], false),
                          f16_of_codes(b[1], true));
              mma16<Fp16>(sacc[2 * i + 1], qf[2 * k + 1], f16_of_codes(b[3], false),
                          f16_of_codes(b[3], true));
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
                sacc[t][i] = seen ? score<FORM>(p.sc, sacc[t][i] * (unit[r] * sk[t >> 1]),
                                                slope[r], away)
                                  : -INFINITY;
              }
          } else {  // every row sees every key
#pragma unroll
            for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sacc[t][i] *= (p.sc.scale * kLog2e) * unit[i >> 1] * sk[t >> 1];
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int t = 0; t < kSub; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              mx[r] = fmaxf(mx[r], fmaxf(fmaxf(sacc[2 * t][2 * r], sacc[2 * t][2 * r + 1]),
                                         fmaxf(sacc[2 * t + 1][2 * r], sacc[2 * t + 1][2 * r + 1])) +
                                       lv[t]);
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
          for (int t = 0; t < kSub; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float b = base[r] - lv[t];
              float e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = ex2(sacc[2 * t + (i >> 1)][2 * r + (i & 1)] - b);
              l[r] = fmaf((e[0] + e[1]) + (e[2] + e[3]), back[t], l[r]);
              pf[t][r] = Fp16::pack(e[0], e[1]);
              pf[t][2 + r] = Fp16::pack(e[2], e[3]);
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
          for (int d = 0; d < kUnits / 2; ++d) {
            if (2 * d >= units) break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              uint32_t b[4];
              ldsm4t(vt + tile_at[i] + lv_row * S::kRow + swizzled<ND>(lv_row, 2 * d + lv_c), b);
#pragma unroll
              for (int k = 0; k < 4; ++k) b[k] = __byte_perm(b[k], 0, 0x3120);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float(*to)[4] = &o[4 * d + 2 * k];
                mma16<Fp16>(to[0], pf[i], f16_of_codes(b[2 * k], false),
                            f16_of_codes(b[2 * k + 1], false));
                mma16<Fp16>(to[1], pf[i], f16_of_codes(b[2 * k], true),
                            f16_of_codes(b[2 * k + 1], true));
              }
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
    finish_item<State8<ND>, S::kD>(p, ws, s, sh, g, cw, o, m, l, [bf16](float x, float y) {
      return bf16 ? Bf16::pack(x, y) : Fp16::pack(x, y);
    });
  }
}

template <int ND>
constexpr int smem_bytes() {
  return (int)sizeof(Smem<ND>) + 1024;
}
static_assert(smem_bytes<1>() <= 227 * 1024 && smem_bytes<2>() <= 227 * 1024,
              "shared memory of a CTA");

template <int ND>
cudaError_t setup_nd() {
  cudaError_t e = cudaSuccess;
  for (auto f : {attn8_decode_kernel<ND, kPlain>, attn8_decode_kernel<ND, kGeneral>,
                 attn8_decode_kernel<ND, kWide>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<ND>());
  return e;
}

template <int ND>
cudaError_t launch_nd(const Attn8Params& p, const Partials& w, const CUtensorMap& kmap,
                      const CUtensorMap& vmap, int grid, cudaStream_t s) {
  const Form form = form_of(p.a.sc);
  return launch_after(form == kPlain     ? attn8_decode_kernel<ND, kPlain>
                      : form == kGeneral ? attn8_decode_kernel<ND, kGeneral>
                                         : attn8_decode_kernel<ND, kWide>,
                      dim3(grid), dim3(kThreads), smem_bytes<ND>(), s, kmap, vmap, p, w);
}

}  // namespace

cudaError_t attn8_decode_setup() {
  const cudaError_t e = setup_nd<1>();
  return e != cudaSuccess ? e : setup_nd<2>();
}

cudaError_t launch_attn8_decode(const Attn8Params& p, const Partials& w, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, int grid, cudaStream_t s) {
  return p.a.head_dim > 64 ? launch_nd<2>(p, w, kmap, vmap, grid, s)
                           : launch_nd<1>(p, w, kmap, vmap, grid, s);
}

}  // namespace attn
}  // namespace moe
