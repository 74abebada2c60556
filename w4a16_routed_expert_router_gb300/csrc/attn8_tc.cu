// Attention of many new tokens per sequence over the 8-bit cache, on the 5th-generation
// tensor core: attn_tc.cu with four warps more, which make codes into fp16.
//
// Division of the work, pieces, joins and the order of the products are those of
// attn_tc.cu, and so is the ring of slots: a slot has room for 128 keys in 16 bits, a
// box brings their codes (128 bytes a key, one swizzled row) to its first half, and the
// converting warps spread them out in place: the 16-bit rows of a warp's 32 keys, of both
// chunks of 64 values, lie over nothing but the codes of those keys, so no warp waits
// for another. All codes are fp16 numbers, so nothing is rounded. (Codes fed to the
// tensor core as they are would need queries and numerators in 8 bits, or each in two
// terms, which takes as many products as fp16 and a longer softmax.)
//   warps 0-3, 4-7  softmax of tile 0 / 1
//   warp 8    TMA producer: Q, K and V codes, and the scales
//   warp 9    MMA issuer
//   warp 10   (idle)
//   warp 11   walks the share
//   warps 12-15  codes to fp16; V rows behind the last key become zeros. bf16 queries
//             become fp16 in place, each row by a power of two of its own.
// Scales: see attn8_decode.cu. A score is (q.k) (scale 2^e sk), e the row's power of two;
// the exponent takes log2 sv, the running maximum is of x + log2 sv, and the sum of
// weights takes 1 / sv back, once for 16 keys.
//
// For batches of up to 512 rows a sequence and kv head, or where there is no room for the
// keys in 16 bits, heads of 128, 4 to a kv head: 64 tokens over 32768 keys take 75 us (18
// at the matrix products' rate), 100 102 (28), 8 sequences of 64 over 8192 keys 98 (36).
// No unit bounds it: in the last, 6700 cycles a block of two tiles with the matrix unit
// at 30 % of them, issue slots at 35, shared memory at 24 (of the threads' accesses) and
// DRAM at 18. It is the way of a block from the copy over the converters, products and
// softmax, one behind the other. (Slots of codes beside those of 16 bits, converters in
// pairs, the ratio of scales applied by the converters, and V's slots given back early:
// none was faster.)
#define MOE_ATTN8_TC
#include "attn_tc.cu"
#include "attn8_parts.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads8 = 16 * 32;
constexpr int kFirstConverter = 12, kConverters = 4;
constexpr int kPieceReaders8 = kSoftmaxWarps + 2 + kConverters;
// Registers a thread: 128 at the launch, then 192 for the softmax, and what is left.
constexpr int kLaunchRegs8 = 128, kSoftmaxRegs8 = 192, kOtherRegs8 = 80, kConverterRegs = 48;
static_assert(2 * kSoftmaxRegs8 + kOtherRegs8 + kConverterRegs <= 4 * kLaunchRegs8,
              "setmaxnreg draws on the launch");
constexpr int kGroups = kBlk / kScaleBlock;   // scales of a block

template <int ND>
struct Smem8 {
  static constexpr int kSlots = ND == 2 ? 5 : 8;
  // Scales of so many blocks: those of block n + kScales may come once the slot of its K
  // is free, which held V of a block from n on, so that the softmax is through with n.
  static constexpr int kScales = ND == 2 ? 4 : 8;
  static_assert(2 * kScales > kSlots, "see kScales");
  uint8_t kv[kSlots][ND * kChunk];
  uint8_t q[2][ND * kChunk];
  uint8_t piece[kPieces][kPieceBytes];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  // scale of K, log2 of V's and its inverse (before they are converted: K's and V's)
  float4 scales[kScales][kGroups];
  int8_t q_exp[2][2][128];      // by piece: the rows' powers of two
  Scan<kThreads8> scan;
  Share share;
  unsigned there[2];
  uint64_t kv_full[kSlots], kv_ready[kSlots], kv_empty[kSlots];
  uint64_t sc_full[kScales], sc_ready[kScales];
  uint64_t q_full, q_ready, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], drain;
  uint32_t tmem_base;
};

// 16 bytes of shared memory
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 32 keys of a slot, codes to fp16 in place; keys from `left` on become zeros. A lane
// has 16 codes of a key at a time, 8 lanes a key (4 at head sizes up to 64); the codes
// of the keys at hand are read before any of their 16-bit rows is written.
template <int ND>
__device__ __forceinline__ void spread(uint32_t slot, int row0, int left) {
  constexpr int kLanes = ND * 4, kRows = 32 / kLanes;  // lanes a key, keys at a time
  const int lane = threadIdx.x & 31;
  const int u = lane & (kLanes - 1), sub = lane / kLanes;
  constexpr int kAhead = 4;                            // loads under way
#pragma unroll 1
  for (int i = 0; i < 32; i += kRows * kAhead) {
    uint4 c[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int row = row0 + i + j * kRows + sub;
      c[j] = lds128(slot + row * 128 + ((u ^ (row & 7)) << 4));
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int row = row0 + i + j * kRows + sub, x = row & 7;
      if (row >= left) c[j] = make_uint4(0, 0, 0, 0);
      // 8 lanes together write to all banks: of the second chunk the odd units first
      const bool odd = ND == 2 && u >= 4;
      const uint32_t to = slot + row * 128 + (ND == 2 ? (u >> 2) * kChunk : 0);
      const uint32_t a0 = odd ? c[j].z : c[j].x, a1 = odd ? c[j].w : c[j].y;
      const uint32_t b0 = odd ? c[j].x : c[j].z, b1 = odd ? c[j].y : c[j].w;
      const int unit = (u & 3) * 2;
      sts128(to + (((unit + odd) ^ x) << 4), f16_of_codes(a0, false), f16_of_codes(a0, true),
             f16_of_codes(a1, false), f16_of_codes(a1, true));
      sts128(to + (((unit + !odd) ^ x) << 4), f16_of_codes(b0, false), f16_of_codes(b0, true),
             f16_of_codes(b1, false), f16_of_codes(b1, true));
    }
  }
}

// A row of Q, bf16 to fp16 in place; its power of two (x = fp16 * 2^-e).
template <int ND>
__device__ __forceinline__ int convert_q(uint32_t tile, int row) {
  const uint32_t at = tile + row * 128, x = row & 7;
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < ND; ++c)
#pragma unroll 2
    for (int u = 0; u < 8; ++u) {
      const uint4 v = lds128(at + c * kChunk + ((u ^ x) << 4));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = max3(top, fabsf(bf16_bits_to_f32((uint16_t)w[k])),
                   fabsf(bf16_bits_to_f32((uint16_t)(w[k] >> 16))));
    }
  const RowUnit unit(top);
#pragma unroll
  for (int c = 0; c < ND; ++c)
#pragma unroll 2
    for (int u = 0; u < 8; ++u) {
      const uint32_t to = at + c * kChunk + ((u ^ x) << 4);
      const uint4 v = lds128(to);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        h[k] = Fp16::pack(bf16_bits_to_f32((uint16_t)w[k]) * unit.up,
                          bf16_bits_to_f32((uint16_t)(w[k] >> 16)) * unit.up);
      sts128(to, h[0], h[1], h[2], h[3]);
    }
  return (__float_as_int(unit.up) >> 23) - 127;
}

template <typename T, int ND, int FORM>
__global__ void __launch_bounds__(kThreads8, 1)
    attn8_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ Attn8Params g8, const __grid_constant__ TcPieces ws) {
  typedef Smem8<ND> S;
  typedef BlockLayout<false> L;
  const AttnParams& p = g8.a;
  constexpr bool kHalves = ND == 1;  // see attn_tc.cu
  constexpr bool GEN = FORM != kPlain;
  constexpr bool kCut = ND == 2 && !GEN;
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_ready[i], kConverters);
      mbar_init(&s.kv_empty[i], 1);
    }
    for (int i = 0; i < S::kScales; ++i) {
      mbar_init(&s.sc_full[i], 32);
      mbar_init(&s.sc_ready[i], kConverters);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&s.piece_full[i], 1);
      mbar_init(&s.piece_empty[i], kPieceReaders8);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_ready, kConverters);
    mbar_init(&s.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_half[t], 4);
      mbar_init(&s.p_full[t], 4);
      mbar_init(&s.o_full[t], 1);
      mbar_init(&s.o_empty[t], 4);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == kMmaWarp) tmem_alloc(&s.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  wait_prior_launch();

  const int tpt = tile_tokens(p.group);
  divide<kCut>(p, s.scan, &s.kv[0][0], s.share, tpt);
  Piece g;
  fence_async_shared();  // the ring's first use was that one
  __syncthreads();

  if (warp >= kFirstConverter) {
    // ---------------------------------------------------------------- codes to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConverterRegs));
    const int cw = warp - kFirstConverter;
    uint32_t slot = 0, ph = 0, qph = 0, block = 0, odd = 0;
    bool ok = true;
    Pieces<S, true> pieces{s, p.err};
    while (ok && pieces.next(g)) {
      if (!(ok = __all_sync(0xffffffffu, bwait_piece(&s.q_full, qph, p.err)))) break;
      qph ^= 1u;
      if (!T::kFp16) {
        const int row = cw * 32 + lane;
        for (int t = 0; t < (g.ntok > tpt ? 2 : 1); ++t)
          s.q_exp[odd][t][row] = (int8_t)convert_q<ND>(smem_u32(s.q[t]), row);
        fence_async_shared();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_ready);
      odd ^= 1u;
      for (int n = g.n0; n < g.end && ok; ++n, ++block) {
        const int left = g.kv - key_block(g, n) * kBlk;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (!(ok = warp_wait(&s.kv_full[slot], ph, p.err))) break;
          spread<ND>(smem_u32(s.kv[slot]), cw * 32, kv ? left : kBlk);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.kv_ready[slot]);
          if (++slot == S::kSlots) {
            slot = 0;
            ph ^= 1u;
          }
          if (kv == 0) {
            const uint32_t at = block % S::kScales, sph = block / S::kScales & 1u;
            if (cw == 0) {
              if (!(ok = warp_wait(&s.sc_full[at], sph, p.err))) break;
              if (lane < kGroups) {
                float4& v = s.scales[at][lane];
                const float sk = scale_in_range(v.x), lv = log2_of_scale(scale_in_range(v.y));
                v = make_float4(sk, lv, ex2(-lv), 0.0f);
              }
              __syncwarp();
            }
            // every converting warp: the rows' powers of two go with them
            if (lane == 0) mbar_arrive(&s.sc_ready[at]);
          }
        }
      }
    }
  } else if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs8));
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- producer
      const int ps = 1 << p.page_shift;
      const int ppb = ps < kBlk ? kBlk / ps : 1;
      const int box_rows = min(ps, kBlk);
      const int per_batch = 32 / ppb;
      const int grp = lane & (kGroups - 1), grp_box = min(grp * kScaleBlock / box_rows, ppb - 1);
      const float* scale_base = lane < kGroups ? g8.c.k_scales : g8.c.v_scales;
      uint32_t slot = 0, ph = 0, filled = 0, last_ph = 0, qph = 0, block = 0;
      bool ok = true, q_used = false;
      Pieces<S, true> pieces{s, p.err};
      while (ok && pieces.next(g)) {
        const int* table = p.b.page_table + (long long)g.seq * p.b.table_stride;
        const int bi = lane / ppb, pi = lane - bi * ppb;
        const auto fetch = [&](int n0) {
          const int nn = n0 + bi;
          const int key = key_block(g, nn) * kBlk + pi * box_rows;
          int id = 0;
          if (nn < g.end && key < g.kv) {
            id = __ldg(table + (key >> p.page_shift));
            if (id < 0 || id >= p.num_pages) {
              atomicOr(p.err, kErrRange);
              id = (int)p.num_pages;  // outside the tensor: the box is filled with zeros
            }
          }
          return id;
        };
        int ids = fetch(g.n0);
        // Q: tile t's tokens by the group's heads
        if (!(ok = __all_sync(0xffffffffu, bwait_piece(&s.q_empty, qph ^ 1u, p.err)))) break;
        if (elect_one()) {
          const int tiles = g.ntok > tpt ? 2 : 1;
          mbar_arrive_expect_tx(&s.q_full, tiles * ND * tpt * p.group * 128);
          for (int t = 0; t < tiles; ++t)
#pragma unroll
            for (int c = 0; c < ND; ++c)
              tma_q(smem_u32(s.q[t]) + c * kChunk, &qmap, &s.q_full, c * 64, g.head * p.group,
                    g.first + t * tpt);
        }
        __syncwarp();
        q_used = true;
        qph ^= 1u;
        for (int n = g.n0; n < g.end && ok;) {
          const int batch = min(per_batch, g.end - n);
          const int next = n + batch < g.end ? fetch(n + batch) : 0;
          for (int i = 0; i < batch && ok; ++i, ++block) {
            const int kb = key_block(g, n + i) * kBlk;
            const int boxes = min(ppb, max(0, g.kv - kb + box_rows - 1) / box_rows);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (!(ok = warp_wait(&s.kv_empty[slot], ph ^ 1u, p.err))) break;
              if (elect_one()) mbar_arrive_expect_tx(&s.kv_full[slot], boxes * box_rows * 128);
              const uint32_t dst = smem_u32(s.kv[slot]);
              for (int j = 0; j < boxes; ++j) {
                const int page = __shfl_sync(0xffffffffu, ids, i * ppb + j);
                if (elect_one())
                  tma_page(dst + j * box_rows * 128, kv ? &vmap : &kmap, &s.kv_full[slot], 0,
                           (kb + j * box_rows) & (ps - 1), g.head, page);
              }
              if (kv == 0) {
                const uint32_t at = block % S::kScales;
                const int page = __shfl_sync(0xffffffffu, ids, i * ppb + grp_box);
                if (lane < 2 * kGroups) {
                  const int key = kb + grp * kScaleBlock;
                  const bool there = key < g.kv && page < p.num_pages;
                  const long long from =
                      there ? page * g8.c.scale_page + g.head * g8.c.scale_head +
                                  ((key & (ps - 1)) / kScaleBlock) * g8.c.scale_block
                            : 0;
                  copy4_async(smem_u32(&s.scales[at][grp]) + (lane < kGroups ? 0 : 4),
                              scale_base + from, there);
                }
                arrive_after_copies(&s.sc_full[at]);
              }
              filled |= 1u << slot;
              last_ph = (last_ph & ~(1u << slot)) | (ph << slot);
              if (++slot == S::kSlots) {
                slot = 0;
                ph ^= 1u;
              }
            }
          }
          n += batch;
          ids = next;
        }
      }
      // wind down: no copy may still be landing when the CTA exits
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        for (int i = 0; i < S::kSlots; ++i)
          if (filled & (1u << i)) mbar_wait(&s.kv_full[i], (last_ph >> i) & 1u, p.err);
        if (q_used) mbar_wait(&s.q_full, qph ^ 1u, p.err);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      const int ksteps = (p.head_dim + 15) / 16;
      const int dn = (p.head_dim + 15) & ~15;
      const uint32_t id_qk = idesc_of<Fp16>(kBlk, false), id_pv = idesc_of<Fp16>(dn, true);
      if (elect_one()) {
        uint32_t slot = 0, ph = 0, qph = 0;
        uint32_t pph[2] = {0, 0}, oph[2] = {0, 0};
        bool ok = true;
        Pieces<S, false> pieces{s, p.err};
        const auto wait_slot = [&]() { return bwait(&s.kv_ready[slot], ph, p.err); };
        const auto advance = [&]() {
          if (++slot == S::kSlots) {
            slot = 0;
            ph ^= 1u;
          }
        };
        const auto issue_qk = [&](int t, uint32_t kslot) {
          const uint64_t qd = smem_desc_sw128(smem_u32(s.q[t]));
          const uint64_t kd = L::k(smem_u32(s.kv[kslot]));
#pragma unroll
          for (int k = 0; k < ND * 4; ++k)
            if (k < ksteps)
              mma_bf16(tmem + t * 128, qd + (((k >> 2) * kChunk + (k & 3) * 32) >> 4),
                       kd + (((k >> 2) * L::kNext + (k & 3) * 32) >> 4), id_qk, k != 0);
          mma_commit(&s.s_full[t]);
        };
        while (ok && pieces.next(g)) {
          const int blocks = g.end - g.n0;
          const int cnt[2] = {g.cnt[0], g.cnt[1]};
          if (!bwait(&s.q_ready, qph, p.err) || !wait_slot()) break;
          qph ^= 1u;
          tc_fence_after();
          if (cnt[0] > 0) issue_qk(0, slot);
          if (cnt[1] > 0) issue_qk(1, slot);
          mma_commit(&s.kv_empty[slot]);
          if (blocks == 1) mma_commit(&s.q_empty);
          advance();
          for (int j = 0; j < blocks; ++j) {
            const uint32_t vslot = slot;
            if (!(ok = wait_slot())) break;
            advance();
            const bool more = j + 1 < blocks;
            const uint32_t kslot = slot;
            if (more) {
              if (!(ok = wait_slot())) break;
              advance();
            }
            const uint64_t vd = L::v(smem_u32(s.kv[vslot]));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (j >= cnt[t]) continue;
              if (j == 0) {  // the last piece's O has been read
                if (!(ok = bwait(&s.o_empty[t], oph[t] ^ 1u, p.err))) break;
                oph[t] ^= 1u;
              }
              if (kHalves) {
                if (!(ok = bwait(&s.p_half[t], pph[t], p.err))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kBlk / 32; ++k)
                  mma_ts(tmem + 256 + t * ND * 64, tmem + t * 128 + k * 8,
                         vd + k * (L::kGroup >> 3), id_pv, (j | k) != 0);
              }
              if (!(ok = bwait(&s.p_full[t], pph[t], p.err))) break;
              pph[t] ^= 1u;
              tc_fence_after();
#pragma unroll
              for (int k = kHalves ? kBlk / 32 : 0; k < kBlk / 16; ++k)
                mma_ts(tmem + 256 + t * ND * 64, tmem + t * 128 + k * 8, vd + k * (L::kGroup >> 3),
                       id_pv, (j | k) != 0);
              if (j + 1 == cnt[t]) mma_commit(&s.o_full[t]);
              if (j + 1 < cnt[t]) issue_qk(t, kslot);
            }
            if (!ok) break;
            mma_commit(&s.kv_empty[vslot]);
            if (more) mma_commit(&s.kv_empty[kslot]);
            if (j + 2 == blocks) mma_commit(&s.q_empty);
          }
        }
        // wind down: every MMA issued here has completed before the exit
        mma_commit(&s.drain);
        mbar_wait(&s.drain, 0, p.err);
      }
      __syncwarp();
    } else if (warp == kSoftmaxWarps + 3 && lane == 0) {
      walk_share<kCut>(p, s, tpt);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs8));
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + t * 128;
    const uint32_t o_tm = tmem + lane_base + 256 + t * ND * 64;
    const int tok = row / p.group, hg = row - tok * p.group;  // token of the tile, head of the group
    const float scale2 = p.sc.scale * kLog2e;
    uint32_t sph = 0, oph = 0, block = 0, odd = 0;
    Pieces<S, true> pieces{s, p.err};
    for (;;) {
      const Piece* held = pieces.hold();
      if (!group_all(t, held != nullptr)) break;  // the end of the share, or a timeout
      const uint32_t block0 = block;
      block += held->end - held->n0;
      odd ^= 1u;
      const int ntok = min(tpt, held->ntok - t * tpt);    // tokens of this tile
      if (ntok <= 0) {
        pieces.release();
        continue;
      }
      const int cnt = held->cnt[t];
      const int n0 = held->n0, near = held->near, skip = held->skip, prefix = held->prefix;
      const int kv = held->kv;
      const int p_first = held->p0 + t * tpt;
      const int pos = p_first + tok;
      const int lo_last = p.sc.window ? p_first + ntok - 1 - p.sc.window : -1;
      const float slope =
          GEN && p.sc.slopes ? p.sc.slopes[held->head * p.group + hg] * kLog2e : 0.0f;
      const bool mine = tok < ntok;                       // this row exists
      float unit = 1.0f;                                  // of a product, see convert_q
      float ref = -INFINITY, l = 0.0f;                    // 2^ref is the sums' unit
      bool ok = true;
      for (int j = 0; j < cnt; ++j) {
        // The products first: K of this block has then been spread by every converter, and
        // the scales of all blocks before it are ready, so that the parity below can only
        // mean this block's. (A tile without tokens passes its pieces over and may be
        // whole phases ahead of the converters, where the parity says nothing.)
        if (!(ok = warp_wait(&s.s_full[t], sph, p.err))) break;
        sph ^= 1u;
        tc_fence_after();
        const uint32_t at = (block0 + j) % S::kScales;
        if (!(ok = warp_wait(&s.sc_ready[at], (block0 + j) / S::kScales & 1u, p.err))) break;
        if (!T::kFp16 && j == 0)
          unit = __int_as_float((127 - (int)s.q_exp[odd ^ 1u][t][row]) << 23);
        const int n = n0 + j, kb = (n < near ? n : n + skip) * kBlk;
        float x[kBlk];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tmem_ld32_nowait(s_tm + i * 32, reinterpret_cast<uint32_t*>(x) + i * 32);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) loaded16(reinterpret_cast<uint32_t*>(x) + i * 16);
        // every row of the tile sees every key of the block, or not
        const bool whole = (kb + kBlk - 1 <= p_first && kb > lo_last) || kb + kBlk <= prefix;
        if (GEN) {
#pragma unroll
          for (int i = 0; i < kBlk / 2; ++i) {
            const float f = s.scales[at][i / (kScaleBlock / 2)].x * unit;
            unpack2(mul2(pack2(x[2 * i], x[2 * i + 1]), pack2(f, f)), x[2 * i], x[2 * i + 1]);
          }
          general_scores<FORM>(p, x, scale2, kb, kv, mine, pos, p_first, slope);
        }
        if (!whole) mask_row(p, x, kb, prefix, pos);
        // plain scores are products until the exponent, of unit f times K's scale
        // (positive, so that what is masked stays so, however small the two are)
        const float f = GEN ? 1.0f : scale2 * unit;
        const auto times = [&](float sk) { return GEN ? 1.0f : fmaxf(f * sk, 1e-37f); };
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const float* y = x + i * kScaleBlock;
          const float4 sc = s.scales[at][i];
          const float top = max3(max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), y[6]),
                                 max3(max3(y[7], y[8], y[9]), max3(y[10], y[11], y[12]), y[13]),
                                 fmaxf(y[14], y[15]));
          mx = fmaxf(mx, GEN ? top + sc.y : fmaf(top, times(sc.x), sc.y));
        }
        // each row by its own scores, see attn_tc.cu; in log2 units
        const float to = __fadd_ru(mx, -kUp<Fp16>);
        const bool up = to > __fadd_rd(ref, kRaise<Fp16>);
        if (__any_sync(0xffffffffu, up)) {
          const float a = up ? ex2(ref - to) : 1.0f;
          l *= a;
          ref = up ? to : ref;
          if (j > 0) {
#pragma unroll
            for (int i = 0; i < ND * 4; ++i) {
              uint32_t r[16];
              tmem_ld16_nowait(o_tm + i * 16, r);
              tmem_ld_wait();
              loaded16(r);
#pragma unroll
              for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * a);
              tmem_st16(o_tm + i * 16, r);
            }
          }
        }
        const float base = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          uint32_t r[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 sc = s.scales[at][part * 2 + h];
            const float c = times(sc.x), b = sc.y - base;
            const uint64_t c2 = pack2(c, c), b2 = pack2(b, b);
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = part * 32 + h * 16 + 2 * i;
              float e0, e1;
              unpack2(GEN ? add2(pack2(x[k], x[k + 1]), b2) : fma2(pack2(x[k], x[k + 1]), c2, b2),
                      e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum = add2(sum, pack2(e0, e1));
              r[h * 8 + i] = Fp16::pack(e0, e1);
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            l = fmaf(s0 + s1, sc.z, l);
          }
          tmem_st16(s_tm + part * 16, r);
          if (kHalves && part == 1) {  // the product with the first 64 keys may begin
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_half[t]);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[t]);
      }
      if (ok && cnt > 0) {
        ok = warp_wait(&s.o_full[t], oph, p.err);
        oph ^= 1u;
        tc_fence_after();
      }
      // see attn_tc.cu
      if ((!ok || held->pieces) && !group_all(t, ok)) break;
      finish_piece<T, ND, kCut>(p, ws, s, held, t, o_tm, cnt, ref, l);
      if (cnt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_empty[t]);
      }
      pieces.release();
    }
  }

  tc_fence_before();
  __syncthreads();
  let_next_launch();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <int ND>
constexpr int smem_bytes8() {
  return (int)sizeof(Smem8<ND>) + 1024;
}
static_assert(2 * smem_bytes8<1>() > 228 * 1024 && 2 * smem_bytes8<2>() > 228 * 1024,
              "attn8_tc_kernel must stay at one CTA per SM");
static_assert(smem_bytes8<1>() <= 227 * 1024 && smem_bytes8<2>() <= 227 * 1024,
              "shared memory of a CTA");

template <typename F>
cudaError_t setup_one(F f, int bytes, bool* usable) {
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, f)) != cudaSuccess) return e;
  int n = 0;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, kThreads8, bytes)) != cudaSuccess)
    return e;
  if (attr.numRegs != kLaunchRegs8 || n != 1) *usable = false;  // see attn_tc.cu
  return cudaSuccess;
}

template <typename T, int ND>
cudaError_t setup_nd(bool* usable) {
  const int bytes = smem_bytes8<ND>();
  cudaError_t e = setup_one(attn8_tc_kernel<T, ND, kPlain>, bytes, usable);
  if (e == cudaSuccess) e = setup_one(attn8_tc_kernel<T, ND, kGeneral>, bytes, usable);
  return e != cudaSuccess ? e : setup_one(attn8_tc_kernel<T, ND, kWide>, bytes, usable);
}

template <typename T, int ND>
cudaError_t launch_nd(const Attn8Params& p, const TcPieces& w, const CUtensorMap& qmap,
                      const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  Form form = form_of(p.a.sc);
  // Plain scores are told from the maximum by one fused multiply-add (see attn_tc.cu), and
  // the scale times that of K and a row's power of two has to be a positive number.
  if (form == kPlain && !(p.a.sc.scale > 1e-8f && p.a.sc.scale <= 16.0f)) form = kGeneral;
  return launch_after(form == kPlain     ? attn8_tc_kernel<T, ND, kPlain>
                      : form == kGeneral ? attn8_tc_kernel<T, ND, kGeneral>
                                         : attn8_tc_kernel<T, ND, kWide>,
                      dim3(grid), dim3(kThreads8), smem_bytes8<ND>(), s, qmap, kmap, vmap, p, w);
}

}  // namespace

cudaError_t attn8_tc_setup(bool* usable) {
  *usable = true;
  cudaError_t e;
  if ((e = setup_nd<Bf16, 1>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Bf16, 2>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Fp16, 1>(usable)) != cudaSuccess) return e;
  return setup_nd<Fp16, 2>(usable);
}

cudaError_t launch_attn8_tc(const Attn8Params& p, const TcPieces& w, const CUtensorMap& qmap,
                            const CUtensorMap& kmap, const CUtensorMap& vmap, int grid,
                            cudaStream_t s) {
  const bool wide = p.a.head_dim > 64;
  if (p.dtype == MOE_ATTN_BF16)
    return wide ? launch_nd<Bf16, 2>(p, w, qmap, kmap, vmap, grid, s)
                : launch_nd<Bf16, 1>(p, w, qmap, kmap, vmap, grid, s);
  return wide ? launch_nd<Fp16, 2>(p, w, qmap, kmap, vmap, grid, s)
              : launch_nd<Fp16, 1>(p, w, qmap, kmap, vmap, grid, s);
}

}  // namespace attn
}  // namespace moe
