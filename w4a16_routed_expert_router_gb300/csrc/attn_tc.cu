// Attention of many new tokens per sequence over the paged cache: prompts and
// chunks of prompts, on the 5th-generation tensor core.
//
// One persistent CTA per SM over an equal share of all key blocks of all items,
// an item being up to two tiles of query tokens of one sequence (an entry) and a
// kv head. Equal shares keep every SM busy to the end under a causal mask, ragged
// lengths or a single chunk over a long cache; few items over many keys are cut in
// step (kCutShare). The pieces of an item that more than one CTA holds are joined
// by pairs, by whichever of the two comes second (which has its own piece in TMEM
// still), in an order that does not depend on who that is. (A launch of its own
// that added them took 8 to 15 us.)
//
// One item: two tiles of 128 query rows (token, head of the group)
// against blocks of 128 keys, S = Q K^T and O += P V with tcgen05.mma; S and O
// of both tiles fill the 512 columns of TMEM, and P (16 bits) takes the place
// of S, whose row a thread has in registers by then, as the A operand in TMEM.
//   warps 0-3, 4-7  softmax of tile 0 / 1: one row per thread. The running
//             maximum is only raised when a row exceeds it by 2^8 (2^3 in fp16), so
//             that O is rescaled (by the same threads, in TMEM) in few blocks;
//             numerators stay below that and the result is exact either way.
//   warp 8    TMA producer: Q, and K and V blocks into one ring of slots.
//   warp 9    MMA issuer. While one tile's softmax runs, the tensor core works
//             on the other: PV0(j) QK0(j+1) PV1(j) QK1(j+1) ... (A thread for
//             each tile was slower, 836 to 804 us for 1000 tokens over 65536
//             keys: the tiles' MMAs interleave and both results come late.)
//   warp 10   clears V rows behind a sequence's last key.
//   warp 11   walks the share and hands its pieces to the others.
// Every wait on an mbarrier is bounded; a timeout sets the error bit and the kernel
// winds down. The four warps of a softmax group meet at named barriers, which have
// no limit, so they go on or leave as one (group_all): a warp whose wait gave up
// takes part in the next vote before it leaves.
#include "attn_common.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tc;

constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;  // whole warpgroups: setmaxnreg
constexpr int kTmaWarp = 8, kMmaWarp = 9, kClearWarp = 10;  // and 11, which walks the share
constexpr int kPieceReaders = kSoftmaxWarps + 3;
// Registers a thread: the launch gives every thread kLaunchRegs; the producer
// warpgroup hands most of its share to the two softmax warpgroups, whose rows
// of 128 scores do not fit otherwise. (216 and 72 spill in the issuing thread:
// prefill of 8192 tokens 407 us, 390 us with these.)
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "setmaxnreg draws on the launch");
constexpr int kBlk = kTcBlock;
constexpr int kChunk = 128 * 128;   // 128 rows of 64 values
// Where items are no more than CTAs, sequences have two entries or more and items
// kCutItem units (means), items are cut from their first key on, a share a CTA: the
// CTAs of a kv head then read the same keys at the same time, and its cache comes
// from DRAM about once and not for each of them. 1000 tokens over 65536 keys: 2.69
// -> 0.38 GB read, and with the power that saves 786 -> 695 us back to back; 700
// over 32768 262 -> 249, 100 over 65536 122 -> 114, 100 over 32768 76.8 -> 74.8.
// Shorter items lost (100 over 16384 keys, 131 units: 54.7 -> 55.4; 500 over 8192:
// 61.9 -> 62.9) or stayed (1000 over 16384), and so did single entries, which share
// no keys (64 over 131072: 126.2 -> 128.7). Bounded by their softmax, capped scores
// lost (1178 -> 1199), as did biased ones (980 -> 1043) and head sizes up to 64
// (511 -> 514): not cut. What is left of the items makes the remaining shares;
// kRestUnits is its fixed cost there. A share has kCutShare units at least: a chunk
// must hold more than an item's fixed cost.
constexpr int kCutItem = 192, kCutShare = 8, kRestUnits = 5;
// An item's fixed cost, in blocks (prefill of 8192 tokens: 2 -> 405 us, 4 -> 399,
// 5 -> 402; 16 prompts of 1024: 196, 206, 203; without it 902 and 387 before the
// cost itself was cut).
constexpr int kItemUnits = 2;
static_assert(kCutShare > kItemUnits, "every chunk reads something");
// tanh(y) = y P(y^2) for |y| < 0.6: the fit of tanh(y) / y in y^2 with the least
// relative error, 7.4e-8, and 1.8e-7 with fp32 arithmetic. (Up to 0.75 it takes a
// coefficient more.)
constexpr float kTanhMax = 0.6f;
constexpr int kTanhTerms = 5;
__device__ constexpr float kTanh[kTanhTerms] = {0.99999992687f, -0.3333230997f, 0.13310173604f,
                                                -0.052101477875f, 0.01547542443f};
// A row's maximum is raised when scores exceed it by kRaise (log2 units). Numerators,
// and so their sums, are 2^kUp times what they would be by the maximum: fp16 holds
// up to 2^15 and, with all its bits, down to 2^-14, so weights of 2^-26 of the
// largest and above keep theirs (without it they lose them below 2^-14, and vanish
// below 2^-25: a hundred thousand keys each 2^-25 of one were not there).
template <typename T>
constexpr float kRaise = T::kFp16 ? 3.0f : 8.0f;
template <typename T>
constexpr float kUp = T::kFp16 ? 12.0f : 0.0f;

// one value per warp of a scan over the CTA
struct Scan {
  long long part[kThreads / 32];
};
// What an entry needs of its sequence: n = 0 where its lengths leave their ranges.
struct alignas(16) Seq {
  int first, n, kv, prefix;
};

// A CTA's share: units [at, hi) of the list of items, from entry `index` of
// sequence `seq` on, whose first unit is number `entry_at`. With `cut`, items are
// first cut into chunks of `per` units, the first `cuts` CTAs have one chunk each,
// and the list is of what is left of the items; `cut_at` is the number of the
// entry's first chunk.
struct Share {
  long long per, at, hi, entry_at;
  Seq s;
  int seq, index;
  int cut, cuts, cut_at;
};

constexpr int kPieceBytes = 80, kPieces = 4;  // pieces handed out ahead

template <int ND>
struct Smem {
  static constexpr int kSlots = ND == 2 ? 5 : 8;
  uint8_t kv[kSlots][ND * kChunk];
  uint8_t q[2][ND * kChunk];
  uint8_t piece[kPieces][kPieceBytes];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  Scan scan;
  Share share;
  unsigned there[2];
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], drain, clear, cleared;
  uint32_t tmem_base;
};

// A operand (16-bit, K packed two per column) in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// How a block of keys lies in its slot: atoms of 8 rows of 64 values (1024 B,
// 128-byte swizzle), kGroup bytes from 8 rows to the next, kNext bytes from 64
// values to the next. BOTH: one box brings both chunks of a head, 8 rows by 8
// rows; else a box a chunk. (As numbers known at run time they cost the issuing
// thread 5 % of a prefill.)
template <bool BOTH>
struct BlockLayout {
  static constexpr uint32_t kGroup = BOTH ? 2048 : 1024, kNext = BOTH ? 1024 : kChunk;
  // shared-memory descriptors: K, values along the sum
  static __device__ __forceinline__ uint64_t k(uint32_t addr) {
    return (smem_desc_sw128(addr) & ~((uint64_t)0x3FFF << 32)) | (uint64_t)(kGroup >> 4) << 32;
  }
  // V, keys along the sum and values contiguous: the leading offset goes from 64
  // values to the next, the stride offset from 8 keys to the next
  static __device__ __forceinline__ uint64_t v(uint32_t addr) {
    return (k(addr) & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(kNext >> 4) << 16;
  }
};

template <typename T>
__device__ __forceinline__ uint32_t idesc_of(int n, bool b_mn) {
  uint32_t d = idesc_bf16(128, n);
  if (T::kFp16) d &= ~((1u << 7) | (1u << 10));
  return d | (b_mn ? 1u << 16 : 0u);
}

// 32 columns of this thread's TMEM lane, without the wait
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// After the wait: values of a load before it, so that no use of them moves
// above the wait.
__device__ __forceinline__ void loaded16(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// 16 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Whether `ok` holds in all four warps of softmax group t. Every warp of the group
// takes part in every vote, whatever became of its own waits.
__device__ __forceinline__ bool group_all(int t, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + t)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// the n lowest bits, none below 0 and all from 32 on
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// two fp32 values in one 64-bit register
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// groups of 8 rows, both chunks of a head
__device__ __forceinline__ void tma_groups(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                           int group, int head) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(group), "r"(head)
      : "memory");
}

__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                      int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(head), "r"(token)
      : "memory");
}

// One thread of the converged warp, the same one every time. (Under elect.sync the
// compiler knows that one thread issues the MMAs below; under `lane == 0` the
// same 32 MMAs of a block took 3700 cycles to issue, more than they run.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------------ the share of a CTA
// Shares are counted in units: kItemUnits for an item's fixed cost (Q, the
// results), then one for each of its blocks.
__device__ __forceinline__ int units_of(const Entry& e) { return e.blocks + kItemUnits; }

// One piece: blocks [n0, end) of an item, as one warp hands it to the others.
struct alignas(16) Piece {
  int first, ntok, p0, kv;          // see Entry
  int near, skip, blocks, prefix;
  int head, n0, end, seq;
  int cnt[2];                       // blocks of the piece that tile 0 / 1 takes
  // of a split item: pieces (0: it is whole), number of this one; the first
  // `chunks` of them on CTAs from `chunk0` on, the others on those from cta0 on
  // (both from cta0 where there are no chunks)
  int pieces, number, chunks, chunk0, cta0;
  int pad;
};
static_assert(sizeof(Piece) == kPieceBytes, "shared memory of a piece");

// One role's way through the pieces; `whole` warps or single threads.
template <int ND, bool kWarp>
struct Pieces {
  Smem<ND>& s;
  unsigned* err;
  int i = 0;
  uint32_t ph = 0;
  // the next piece, or null at the end of the share or after a timeout
  __device__ __forceinline__ const Piece* hold() {
    const bool there = bwait_piece(&s.piece_full[i], ph, err);
    if (!(kWarp ? __all_sync(0xffffffffu, there) : there)) return nullptr;
    const Piece* g = reinterpret_cast<const Piece*>(s.piece[i]);
    return g->end > 0 ? g : nullptr;
  }
  // done with it
  __device__ __forceinline__ void release() {
    if (kWarp) __syncwarp();
    if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&s.piece_empty[i]);
    if (++i == kPieces) {
      i = 0;
      ph ^= 1u;
    }
  }
  // a copy of the next piece
  __device__ __forceinline__ bool next(Piece& g) {
    const Piece* held = hold();
    if (!held) return false;
    g = *held;
    release();
    return true;
  }
};

__device__ __forceinline__ int key_block(const Piece& e, int n) {
  return n < e.near ? n : n + e.skip;
}

// listed blocks that rows of tile 0 see (tile 1 sees all, where it has tokens)
__device__ __forceinline__ int blocks_of_tile0(const Entry& e, int tpt) {
  const int p1 = e.p0 + min(e.ntok, tpt) - 1;
  const int end = min(e.kv, max(p1 + 1, e.prefix));
  const int kb = (max(end, 1) + kBlk - 1) / kBlk;
  return min(e.blocks, kb <= e.near ? kb : max(max(e.near, 1), kb - e.skip));
}

// ------------------------------------------------------------------ dividing the work
__device__ __forceinline__ Seq sequence_of(const AttnParams& p, int q) {
  const Span r = read_sequence(p.b, p.page_shift, q, p.err);
  return Seq{r.first, r.n, r.kv, prefix_of(p.sc, q, r.kv)};
}
__device__ __forceinline__ int entries_of(const Seq& r, int tpt) {
  return (int)((unsigned)(r.n + 2 * tpt - 1) / (unsigned)(2 * tpt));
}

// entry i of a sequence
__device__ __forceinline__ Entry entry_of(const AttnParams& p, const Seq& q, int seq, int i,
                                          int tpt) {
  const int t0 = i * 2 * tpt;
  Entry e;
  e.seq = seq;
  e.first = q.first + t0;
  e.ntok = min(2 * tpt, q.n - t0);
  e.p0 = q.kv - q.n + t0;
  e.kv = q.kv;
  e.prefix = q.prefix;
  Span r;
  r.kv = q.kv;
  span_blocks(r, e.p0, e.p0 + e.ntok - 1, p.sc.window, e.prefix, kBlk);
  e.near = r.near;
  e.skip = r.skip;
  e.blocks = r.blocks;
  return e;
}

// Exclusive scan of a value per thread over the CTA; the sum in `whole`.
__device__ __forceinline__ long long cta_scan(Scan& sc, long long mine, long long& whole) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) sc.part[warp] = v;
  __syncthreads();
  long long before = v - mine;
  whole = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sc.part[i];
    whole += sc.part[i];
  }
  return before;
}

// units on the list of what cutting leaves of an item
__device__ __forceinline__ int rest_of(int units) { return units ? units + kRestUnits : 0; }

// Every CTA divides the work for itself (a launch that did it once took longer):
// the entries of all sequences, a run of sequences a thread, then their units, a
// run of entries a thread. `room` is shared memory for a number per sequence and
// one more, and for the sequences themselves while they are few.
constexpr int kSeqsKept = 4096;
template <bool CUT>
__device__ __forceinline__ void divide(const AttnParams& p, Scan& sc, uint8_t* room, Share& share,
                                       int tpt) {
  const int tid = threadIdx.x, seqs = p.b.num_seqs;
  Seq* kept = reinterpret_cast<Seq*>(room);
  int* first = reinterpret_cast<int*>(room + (seqs <= kSeqsKept ? seqs * sizeof(Seq) : 0));
  const int per = (seqs + kThreads - 1) / kThreads;
  const int s0 = min(seqs, tid * per), s1 = min(seqs, s0 + per);
  const auto get = [&](int q) { return seqs <= kSeqsKept ? kept[q] : sequence_of(p, q); };
  long long mine = 0, n = 0;
  for (int q = s0; q < s1; ++q) {
    const Seq r = sequence_of(p, q);
    if (seqs <= kSeqsKept) kept[q] = r;
    mine += entries_of(r, tpt);
  }
  long long at = cta_scan(sc, mine, n);
  for (int q = s0; q < s1; ++q) {
    first[q] = (int)at;
    at += s1 - s0 == 1 ? mine : entries_of(get(q), tpt);
  }
  if (tid == 0) first[seqs] = (int)n;
  __syncthreads();
  const int run = ((int)n + kThreads - 1) / kThreads;
  const int e0 = min((int)n, tid * run), e1 = min((int)n, e0 + run);
  int seq = 0;
  if (e0 < e1) {  // last sequence with first <= e0
    int hi = seqs - 1;
    while (seq < hi) {
      const int mid = (seq + hi + 1) >> 1;
      if (first[mid] <= e0)
        seq = mid;
      else
        hi = mid - 1;
    }
  }
  const auto units = [&](int q, int e) {
    return (long long)units_of(entry_of(p, get(q), q, e - first[q], tpt)) * p.hk;
  };
  long long sum = 0, total;
  int q = seq;
  for (int e = e0; e < e1; ++e) {
    while (first[q + 1] <= e) ++q;
    sum += units(q, e);
  }
  if (tid == 0) share.at = share.hi = 0;  // nothing, unless a thread below finds more
  at = cta_scan(sc, sum, total);
  const Shares sh(total, gridDim.x);
  const int cta = blockIdx.x;
  if (CUT && n * p.hk <= gridDim.x && n >= 2 * seqs && sh.per >= kCutShare &&
      total >= n * p.hk * kCutItem) {  // at most one entry a thread
    const Shares cut(total + n * p.hk * kRestUnits, gridDim.x);
    const int per = (int)cut.per;  // at least one item's units in all: int
    const int u = e0 < e1 ? (int)quotient(sum, p.hk) : 0;
    const int chunks = u / per, rest = u - chunks * per;
    const long long mine2 = (long long)rest_of(rest) * p.hk;
    long long both;  // chunks in the low bits, no more than CTAs
    const long long at2 = cta_scan(sc, mine2 << 8 | chunks * p.hk, both);
    const int cut_at = (int)(at2 & 255), cuts = (int)(both & 255);
    const long long lo = cta < cuts ? 0 : (long long)(cta - cuts) * per;
    const bool here = cta < cuts ? cut_at <= cta && cta < cut_at + chunks * p.hk
                                 : at2 >> 8 <= lo && lo < (at2 >> 8) + mine2;
    if (here)
      share = Share{per, lo, cta < cuts ? 1 : min(both >> 8, lo + per), at2 >> 8, get(q), q,
                    e0 - first[q], 1, cuts, cut_at};
    return;
  }
  const long long lo = sh.begin(cta);
  if (lo >= at && lo < at + sum) {
    q = seq;
    for (int e = e0; e < e1; ++e) {
      while (first[q + 1] <= e) ++q;
      const long long u = e1 - e0 == 1 ? sum : units(q, e);
      if (lo < at + u) {
        share = Share{sh.per, lo, sh.begin(cta + 1), at, get(q), q, e - first[q], 0, 0, 0};
        break;
      }
      at += u;
    }
  }
}

// What a softmax group does with the rows of a piece when its blocks are done: of
// this thread's row, m, the logarithm of its sums' unit, and l, its sum of weights;
// O in TMEM (cnt > 0). Its loops are not unrolled: the code runs once a piece, and
// what it takes is mostly the fetching of its instructions (unrolled, a whole
// item's results took 6500 cycles to store, 3300 so).
template <typename T, int ND, bool CUT>
__device__ __forceinline__ void finish_piece(const AttnParams& p, const TcPieces& ws, Smem<ND>& s,
                                          const Piece* piece, int t, uint32_t o_tm, int cnt,
                                          float m, float l) {
  const Piece& g = *piece;
  const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const int tpt = tile_tokens(p.group);
  const int tok = row / p.group, h = g.head * p.group + (row - tok * p.group);
  const bool mine = tok < min(tpt, g.ntok - t * tpt);  // this row exists
  bool holds = true;  // this group has what is known of the item's rows
  if (g.pieces) {
    bool have = cnt > 0;  // O lies in TMEM
    int a = g.number;  // first piece of what it has
    // Where piece i is left, and where the second half of a pair is counted that
    // begins with it: slot 0 of its CTA, or slot 1 of the item's first CTA for the
    // first piece behind its chunks, as its own CTA may end one item there and
    // begin the next.
    const auto slot = [&](int i) {
      const int chunks = CUT ? g.chunks : 0;
      const int n = i == chunks ? 2 * g.chunk0 + 1
                                  : 2 * (i < chunks ? g.chunk0 + i : g.cta0 + (i - chunks));
      return n * 2 + t;
    };
    const auto group_sync = [&]() {
      asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
    };
    const bool first_thread = (threadIdx.x & 127) == 0;
    for (int size = 1; size < g.pieces && holds; size <<= 1) {
      // pieces [a, a + size) are here; the other half of their pair
      const bool left = (a & size) == 0;
      const int other = left ? a + size : a - size;
      if (other >= g.pieces) continue;
      unsigned* node = ws.count + slot(max(a, other));
      if (first_thread) {
        unsigned v;
        asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(node) : "memory");
        s.there[t] = v;
      }
      group_sync();
      bool there = s.there[t] != 0;
      if (!there) {
        // leave it in the workspace, unless the other half came meanwhile
        const long long at = slot(a);
        __stcg(ws.ml + at * 128 + row, make_float2(m, l));
        if (have) {
          float4* dst = reinterpret_cast<float4*>(ws.o) + at * (ND * 16) * 128 + row;
#pragma unroll 1
          for (int i = 0; i < ND * 2; ++i) {
            uint32_t r[32];
            tmem_ld32_nowait(o_tm + i * 32, r);
            tmem_ld_wait();
            loaded16(r);
            loaded16(r + 16);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(dst + (i * 8 + k) * 128,
                     make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                 __uint_as_float(r[4 * k + 2]),
                                 __uint_as_float(r[4 * k + 3])));
          }
        }
        __threadfence();
        group_sync();
        if (first_thread) {
          s.there[t] = atomicAdd(node, 1u);
          __threadfence();
        }
        group_sync();
        there = s.there[t] != 0;
      }
      if (!there) {
        holds = false;
      } else {
        const long long at = slot(other);
        const float2 x = __ldcg(ws.ml + at * 128 + row);
        const float4* src = reinterpret_cast<const float4*>(ws.o) + at * (ND * 16) * 128 + row;
        const float m2 = fmaxf(m, x.x), base = m2 == -INFINITY ? 0.0f : m2;
        const float f = ex2(m - base), fx = ex2(x.x - base);
        m = m2;
        l = left ? fmaf(x.y, fx, l * f) : fmaf(l, f, x.y * fx);
        const bool nothing = x.y == 0.0f;  // saw no key: its sums may not have been written
#pragma unroll 1
        for (int i = 0; i < ND; ++i) {     // 64 values: 16 loads under way
          float4 v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __ldcg(src + (i * 16 + k) * 128);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16];
            if (have) {
              tmem_ld16_nowait(o_tm + i * 64 + c * 16, r);
              tmem_ld_wait();
              loaded16(r);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float* q = reinterpret_cast<const float*>(&v[c * 4 + (k >> 2)]);
              const float y = nothing ? 0.0f : q[k & 3];
              const float o = have ? __uint_as_float(r[k]) : 0.0f;
              r[k] = __float_as_uint(left ? fmaf(y, fx, o * f) : fmaf(o, f, y * fx));
            }
            tmem_st16(o_tm + i * 64 + c * 16, r);
          }
        }
        tmem_st_wait();
        if (first_thread) *node = 0;  // for the next launch
        have = true;
        a = min(a, other);
      }
      group_sync();  // s.there is free again
    }
  }
  if (holds) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    // A thread has a row; four neighbours exchange 16-byte units, so that
    // they store 64 bytes of one row at a time (by rows alone, a warp's
    // store touched 32 lines, 4500 cycles a tile).
    long long own = -1, off[4];
    if (mine)
      own = (long long)(g.first + t * tpt + tok) * p.out.token + (long long)h * p.out.head;
#pragma unroll
    for (int k = 0; k < 4; ++k) off[k] = __shfl_sync(0xffffffffu, own, (lane & ~3) + k);
    const bool odd = lane & 1, upper = lane & 2;
#pragma unroll 1
    for (int i = 0; i < ND * 2; ++i) {
      uint32_t r[32], u[4][4];
      tmem_ld32_nowait(o_tm + i * 32, r);
      tmem_ld_wait();
      loaded16(r);
      loaded16(r + 16);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        u[k >> 2][k & 3] = T::pack(__uint_as_float(r[2 * k]) * inv,
                                   __uint_as_float(r[2 * k + 1]) * inv);
#pragma unroll
      for (int k = 0; k < 4; k += 2)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t v = __shfl_xor_sync(0xffffffffu, odd ? u[k][w] : u[k + 1][w], 1);
          u[k][w] = odd ? v : u[k][w];
          u[k + 1][w] = odd ? u[k + 1][w] : v;
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t v = __shfl_xor_sync(0xffffffffu, upper ? u[k][w] : u[k + 2][w], 2);
          u[k][w] = upper ? v : u[k][w];
          u[k + 2][w] = upper ? u[k + 2][w] : v;
        }
      // u[k] is now this lane's unit of row k of the four
      const int c0 = i * 32 + (lane & 3) * 8;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (off[k] >= 0 && c0 < p.head_dim)
          *reinterpret_cast<uint4*>(p.out.p + off[k] + c0) =
              make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
    }
    if (mine && p.lse)
      p.lse[(long long)(g.first + t * tpt + tok) * p.hq + h] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// ------------------------------------------------------------------ attention
template <typename T, int ND, int FORM, bool BOTH>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AttnParams p,
                   const __grid_constant__ TcPieces ws) {
  typedef Smem<ND> S;
  typedef BlockLayout<BOTH> L;
  // Half of a block's numerators handed over early: at head sizes up to 64 the
  // softmax is the longer way (16384 tokens 1107 -> 1057 us); above, the tensor
  // core is (8192 tokens 376 -> 391 us with it).
  constexpr bool kHalves = ND == 1;
  constexpr bool GEN = FORM != kPlain;
  constexpr bool kCut = ND == 2 && !GEN;  // what the softmax does not bound, see kCutShare
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&s.piece_full[i], 1);
      mbar_init(&s.piece_empty[i], kPieceReaders);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.clear, 1);
    mbar_init(&s.cleared, 1);
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

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- producer
      const int ps = 1 << p.page_shift;
      const int ppb = ps < kBlk ? kBlk / ps : 1;
      const int box_rows = min(ps, kBlk);
      const int per_batch = 32 / ppb;
      uint32_t slot = 0, ph = 0, filled = 0, last_ph = 0, qph = 0;
      bool ok = true, q_used = false;
      Pieces<ND, true> pieces{s, p.err};
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
        if (lane == 0) {
          ok = bwait_piece(&s.q_empty, qph ^ 1u, p.err);
          if (ok) {
            const int tiles = g.ntok > tpt ? 2 : 1;
            mbar_arrive_expect_tx(&s.q_full, tiles * ND * tpt * p.group * 128);
            for (int t = 0; t < tiles; ++t)
  #pragma unroll
              for (int c = 0; c < ND; ++c)
                tma_q(smem_u32(s.q[t]) + c * kChunk, &qmap, &s.q_full, c * 64, g.head * p.group,
                      g.first + t * tpt);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        q_used = true;
        qph ^= 1u;
        for (int n = g.n0; n < g.end && ok;) {
          const int batch = min(per_batch, g.end - n);
          const int next = n + batch < g.end ? fetch(n + batch) : 0;
          for (int i = 0; i < batch && ok; ++i) {
            const int kb = key_block(g, n + i) * kBlk;
            const int boxes = min(ppb, max(0, g.kv - kb + box_rows - 1) / box_rows);
            const int page = __shfl_sync(0xffffffffu, ids, i * ppb + min(lane, ppb - 1));
            const int row = (kb + lane * box_rows) & (ps - 1);
  #pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (lane == 0) {
                ok = bwait(&s.kv_empty[slot], ph ^ 1u, p.err);
                if (ok) mbar_arrive_expect_tx(&s.kv_full[slot], boxes * box_rows * 128 * ND);
              }
              ok = __shfl_sync(0xffffffffu, ok, 0);
              if (!ok) break;
              if (lane < boxes) {
                const uint32_t dst = smem_u32(s.kv[slot]) + lane * (box_rows >> 3) * L::kGroup;
                const CUtensorMap* map = kv ? &vmap : &kmap;
                if (BOTH) {
                  tma_groups(dst, map, &s.kv_full[slot],
                             page * p.boxes.page_groups + (row >> 3),
                             page * p.boxes.page_heads + g.head);
                } else {
#pragma unroll
                  for (int c = 0; c < ND; ++c)
                    tma_page(dst + c * kChunk, map, &s.kv_full[slot], c * 64, row, g.head, page);
                }
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
      // wind down: no TMA copy may still be landing when the CTA exits
      if (lane == 0) {
        for (int i = 0; i < S::kSlots; ++i)
          if (filled & (1u << i)) mbar_wait(&s.kv_full[i], (last_ph >> i) & 1u, p.err);
        if (q_used) mbar_wait(&s.q_full, qph ^ 1u, p.err);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      // One thread; what it waits for is there already when the softmax keeps
      // up, and a wait by a whole warp costs it about 150 cycles more.
      const int ksteps = (p.head_dim + 15) / 16;
      const int dn = (p.head_dim + 15) & ~15;
      const uint32_t id_qk = idesc_of<T>(kBlk, false), id_pv = idesc_of<T>(dn, true);
      if (elect_one()) {
        uint32_t slot = 0, ph = 0, qph = 0, cph = 0;
        uint32_t pph[2] = {0, 0}, oph[2] = {0, 0};
        bool ok = true;
        Pieces<ND, false> pieces{s, p.err};
        const auto wait_slot = [&]() { return bwait(&s.kv_full[slot], ph, p.err); };
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
          if (!bwait(&s.q_full, qph, p.err) || !wait_slot()) break;
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
            if (g.kv - key_block(g, g.n0 + j) * kBlk < kBlk) {
              mbar_arrive(&s.clear);
              if (!(ok = bwait(&s.cleared, cph, p.err))) break;
              cph ^= 1u;
            }
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
    } else if (warp == kClearWarp) {
      // ---------------------------------------------------------------- cleared rows
      // V rows behind the last key may hold anything, and take part in the
      // product with weight zero: clear them in the block that has them, once
      // the issuer has seen it arrive.
      uint32_t slot = 0, cph = 0;
      bool ok = true;
      Pieces<ND, true> pieces{s, p.err};
      while (ok && pieces.next(g)) {
        for (int n = g.n0; n < g.end; ++n) {
          const uint32_t vslot = (slot + 1) % S::kSlots;
          slot = (slot + 2) % S::kSlots;
          const int left = g.kv - key_block(g, n) * kBlk;
          if (left >= kBlk) continue;
          if (!(ok = __all_sync(0xffffffffu, bwait_piece(&s.clear, cph, p.err)))) break;
          cph ^= 1u;
          const uint32_t v = smem_u32(s.kv[vslot]);
          const int from = max(left, 0);
          for (int i = lane; i < (kBlk - from) * ND * 8; i += 32) {
            const int r = from + i / (ND * 8), c = i % (ND * 8);
            sts128(v + (c >> 3) * L::kNext + (r >> 3) * L::kGroup + (r & 7) * 128 + (c & 7) * 16, 0,
                   0, 0, 0);
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.cleared);
        }
      }
    } else if (lane == 0) {
      // ---------------------------------------------------------------- the share, piece by piece
      const Share& sh = s.share;
      const int cta = blockIdx.x;
      const bool chunk = kCut && cta < sh.cuts;  // a chunk of an item, and nothing else
      long long at = sh.at, entry_at = sh.entry_at;
      const long long hi = sh.hi;
      int seq = sh.seq, index = sh.index, cut_at = sh.cut_at;
      Entry e;
      Seq r = sh.s;
      // an item of the entry: its chunks; the units it has on the list, the first
      // of which read nothing, and the block that the others begin with
      int chunks = 0, listed = 0, fixed = 0, behind = 0;
      int head = -1, i = 0;   // head -2: the sequence is to be read, -1: the entry made
      uint32_t ph = 0;
      bool ok = true;
      while (ok) {
        Piece o = {};
        while (at < hi) {
          if (head < 0) {
            if (head == -2) r = sequence_of(p, seq);
            if (index == entries_of(r, tpt)) {
              ++seq;
              index = 0;
              head = -2;
              continue;
            }
            e = entry_of(p, r, seq, index, tpt);
            listed = units_of(e);
            if (kCut && sh.cut) {
              chunks = listed / (int)sh.per;
              listed = rest_of(listed - chunks * (int)sh.per);
              behind = max(0, chunks * (int)sh.per - kItemUnits);
            }
            fixed = listed - (e.blocks - behind);
            head = chunk ? (cta - cut_at) / chunks
                         : listed ? (int)quotient(at - entry_at, listed) : p.hk;
          }
          const long long item = entry_at + (long long)head * listed;
          if (chunk) {
            o.number = cta - cut_at - head * chunks;
            o.n0 = max(0, o.number * (int)sh.per - kItemUnits);
            o.end = (o.number + 1) * (int)sh.per - kItemUnits;
            at = hi;
          } else if (listed) {
            const int u0 = (int)(at - item), u1 = (int)min((long long)listed, u0 + (hi - at));
            at = item + u1;
            o.n0 = behind + max(0, u0 - fixed);
            o.end = behind + max(0, u1 - fixed);
          }
          if (o.end <= o.n0) o.end = 0;  // nothing to read: no piece
          if (o.end) {
            o.head = head;
            o.first = e.first, o.ntok = e.ntok, o.p0 = e.p0, o.kv = e.kv;
            o.near = e.near, o.skip = e.skip, o.blocks = e.blocks, o.prefix = e.prefix;
            o.seq = e.seq;
            o.cnt[0] = min(o.end, blocks_of_tile0(e, tpt)) - o.n0;
            o.cnt[1] = e.ntok > tpt ? o.end - o.n0 : 0;
            if (o.end - o.n0 < e.blocks) {
              o.cta0 = sh.cuts + (int)quotient(item + fixed, sh.per);
              const int last = sh.cuts + (int)quotient(item + listed - 1, sh.per);
              o.pieces = chunks + (listed ? last - o.cta0 + 1 : 0);
              o.chunks = chunks;
              o.chunk0 = chunks ? cut_at + head * chunks : o.cta0;
              if (!chunk) o.number = chunks + cta - o.cta0;
            }
          }
          if (listed == 0 || at == item + listed) ++head;
          if (head >= p.hk) {
            head = -1;
            ++index;
            entry_at += (long long)listed * p.hk;
            cut_at += chunks * p.hk;
          }
          if (o.end) break;
        }
        ok = bwait_piece(&s.piece_empty[i], ph ^ 1u, p.err);
        if (!ok) break;
        *reinterpret_cast<Piece*>(s.piece[i]) = o;
        mbar_arrive(&s.piece_full[i]);
        if (++i == kPieces) {
          i = 0;
          ph ^= 1u;
        }
        if (o.end == 0) break;  // the end of the share, told to all
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + t * 128;
    const uint32_t o_tm = tmem + lane_base + 256 + t * ND * 64;
    const int tok = row / p.group, hg = row - tok * p.group;  // token of the tile, head of the group
    const float scale2 = p.sc.scale * kLog2e;
    // scores are dot products until the exponent (plain), or log2 units (GEN)
    const float c = GEN ? 1.0f : scale2, raise = GEN ? kRaise<T> : kRaise<T> / c;
    const float cap_in = p.sc.cap_in;
    const float cap_out = p.sc.softcap * kLog2e;
    uint32_t sph = 0, oph = 0;
    Pieces<ND, true> pieces{s, p.err};
    for (;;) {
      const Piece* held = pieces.hold();
      if (!group_all(t, held != nullptr)) break;  // the end of the share, or a timeout
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
      float m = -INFINITY, ref = -INFINITY, l = 0.0f;  // ref: 2^ref is the sums' unit
      bool ok = true;
      for (int j = 0; j < cnt; ++j) {
        if (!(ok = warp_wait(&s.s_full[t], sph, p.err))) break;
        sph ^= 1u;
        tc_fence_after();
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
          if (p.sc.softcap > 0.0f) {
            // cap tanh(y) in log2 units, y = x scale / cap. While every |y| of the
            // warp's rows is below kTanhMax, it is y times a polynomial in y^2, two
            // keys to an instruction; else as FORM has it. Rows and keys that do
            // not exist have no part in the choice: the block with the last key takes
            // the second form. (The powers of scale / cap do not go into the
            // coefficients, which saves a product but lets the highest ones vanish
            // where scale / cap is small: scores were 0.3 off at a cap of 2000.)
            float top = fabsf(x[0]);
#pragma unroll
            for (int i = 1; i < kBlk - 1; i += 2) top = max3(top, fabsf(x[i]), fabsf(x[i + 1]));
            top = fmaxf(top, fabsf(x[kBlk - 1]));
            if (kb + kBlk <= kv &&
                __all_sync(0xffffffffu, !mine || top * fabsf(cap_in) < kTanhMax)) {
              const uint64_t in2 = pack2(cap_in, cap_in);
              float f[kTanhTerms];
#pragma unroll
              for (int k = 0; k < kTanhTerms; ++k) f[k] = kTanh[k] * cap_out;
#pragma unroll
              for (int i = 0; i < kBlk / 2; ++i) {
                const uint64_t y = mul2(pack2(x[2 * i], x[2 * i + 1]), in2);
                const uint64_t t = mul2(y, y);
                uint64_t r = pack2(f[kTanhTerms - 1], f[kTanhTerms - 1]);
#pragma unroll
                for (int k = kTanhTerms - 2; k >= 0; --k) r = fma2(r, t, pack2(f[k], f[k]));
                unpack2(mul2(r, y), x[2 * i], x[2 * i + 1]);
              }
            } else if (FORM == kWide) {
#pragma unroll
              for (int i = 0; i < kBlk / 2; ++i) {
                const uint64_t y = pack2(tanh_range(x[2 * i] * cap_in),
                                         tanh_range(x[2 * i + 1] * cap_in));
                const uint64_t t = mul2(y, y);
                uint64_t a = pack2(kTanhP[4], kTanhP[4]), b = pack2(kTanhQ[4], kTanhQ[4]);
#pragma unroll
                for (int k = 3; k >= 0; --k) {
                  a = fma2(a, t, pack2(kTanhP[k], kTanhP[k]));
                  b = fma2(b, t, pack2(kTanhQ[k], kTanhQ[k]));
                }
                float b0, b1;
                unpack2(b, b0, b1);
                a = mul2(mul2(a, y), pack2(rcp(b0), rcp(b1)));
                unpack2(mul2(a, pack2(cap_out, cap_out)), x[2 * i], x[2 * i + 1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < kBlk; ++i) {
                const float e = ex2(x[i] * (2.0f * kLog2e * cap_in));
                x[i] = fmaf(-2.0f * cap_out, rcp(1.0f + e), cap_out);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < kBlk / 2; ++i) {
              const uint64_t r = mul2(pack2(x[2 * i], x[2 * i + 1]), pack2(scale2, scale2));
              unpack2(r, x[2 * i], x[2 * i + 1]);
            }
          }
          if (p.sc.slopes) {
            // distances are whole numbers: exact steps of -1 from key to key, where
            // fp32 holds them all and no key lies ahead of its query
            const float far = (float)(pos - kb);
            if (kb + kBlk - 1 <= p_first && p_first - kb < (1 << 24) - 128) {
              uint64_t away = pack2(far, far - 1.0f);
#pragma unroll
              for (int i = 0; i < kBlk / 2; ++i) {
                const uint64_t r =
                    fma2(away, pack2(-slope, -slope), pack2(x[2 * i], x[2 * i + 1]));
                unpack2(r, x[2 * i], x[2 * i + 1]);
                away = add2(away, pack2(-2.0f, -2.0f));
              }
            } else {
#pragma unroll
              for (int i = 0; i < kBlk; ++i) x[i] = fmaf(-slope, fabsf(far - (float)i), x[i]);
            }
          }
        }
        if (!whole) {
          // bit i of word w: this row sees key kb + 32 w + i
          const int a = pos - kb + 1, b = p.sc.window ? pos - p.sc.window - kb + 1 : 0;
          const int pre = prefix - kb;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t bits = (below(a - 32 * w) & ~below(b - 32 * w)) | below(pre - 32 * w);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(bits & (1u << i))) x[32 * w + i] = -INFINITY;
          }
        }
        float mt[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < kBlk - 4; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mt[k] = max3(mt[k], x[i + 2 * k], x[i + 2 * k + 1]);
        const float mx = fmaxf(max3(max3(mt[0], x[124], x[125]), mt[1], mt[2]),
                               max3(mt[3], x[126], x[127]));
        // each row by its own scores: what shares its warp does not change it (rounded
        // so that no numerator passes its limit, however large the scores)
        const bool up = mx > __fadd_rd(m, raise);
        if (__any_sync(0xffffffffu, up)) {
          const float to = __fmaf_ru(mx, c, -kUp<T>);
          const float a = up ? ex2(ref - to) : 1.0f;
          l *= a;
          m = up ? mx : m;
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
        const uint64_t c2 = pack2(c, c), base2 = pack2(-base, -base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            unpack2(fma2(pack2(x[part * 32 + 2 * i], x[part * 32 + 2 * i + 1]), c2, base2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
            r[i] = T::pack(e0, e1);
          }
          tmem_st16(s_tm + part * 16, r);
          if (kHalves && part == 1) {  // the product with the first 64 keys may begin
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_half[t]);
          }
        }
        {
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
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
      // A piece of a split item meets barriers in there: a vote first. A whole item
      // has none, and a warp that gave up takes part in the group's next vote, the
      // one above, from here.
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
constexpr int smem_bytes() {
  return (int)sizeof(Smem<ND>) + 1024;
}
// A CTA holds all of TMEM, so there may be one per SM only.
static_assert(2 * smem_bytes<1>() > 228 * 1024 && 2 * smem_bytes<2>() > 228 * 1024,
              "attn_tc_kernel must stay at one CTA per SM");
static_assert(smem_bytes<2>() <= 227 * 1024, "shared memory of a CTA");

template <typename F>
cudaError_t setup_one(F f, int bytes, bool* usable) {
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, f)) != cudaSuccess) return e;
  int n = 0;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, kThreads, bytes)) != cudaSuccess)
    return e;
  // With fewer registers at launch the softmax warps would wait for more for ever,
  // and a CTA holds all of its SM's TMEM.
  if (attr.numRegs != kLaunchRegs || n != 1) *usable = false;
  return cudaSuccess;
}

template <typename T, int ND, bool BOTH>
cudaError_t setup_nd(bool* usable) {
  const int bytes = smem_bytes<ND>();
  cudaError_t e = setup_one(attn_tc_kernel<T, ND, kPlain, BOTH>, bytes, usable);
  if (e == cudaSuccess) e = setup_one(attn_tc_kernel<T, ND, kGeneral, BOTH>, bytes, usable);
  return e != cudaSuccess ? e : setup_one(attn_tc_kernel<T, ND, kWide, BOTH>, bytes, usable);
}

template <typename T, int ND, bool BOTH>
cudaError_t launch_nd(const AttnParams& p, const TcPieces& w, const CUtensorMap& qmap,
                      const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  Form form = form_of(p.sc);
  // The plain form takes the maximum before it scales (kRaise over the scale has to be
  // a number), and tells a score's distance from it by one fused multiply-add, whose
  // parts should stay below 2^26.
  if (form == kPlain && !(p.sc.scale > 1e-30f && p.sc.scale <= 16.0f)) form = kGeneral;
  return launch_after(form == kPlain     ? attn_tc_kernel<T, ND, kPlain, BOTH>
                      : form == kGeneral ? attn_tc_kernel<T, ND, kGeneral, BOTH>
                                         : attn_tc_kernel<T, ND, kWide, BOTH>,
                      dim3(grid), dim3(kThreads), smem_bytes<ND>(), s, qmap, kmap, vmap, p, w);
}

template <typename T>
cudaError_t launch_t(const AttnParams& p, const TcPieces& w, const CUtensorMap& qmap,
                     const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  if (p.head_dim <= 64) return launch_nd<T, 1, false>(p, w, qmap, kmap, vmap, grid, s);
  return p.boxes.both ? launch_nd<T, 2, true>(p, w, qmap, kmap, vmap, grid, s)
                      : launch_nd<T, 2, false>(p, w, qmap, kmap, vmap, grid, s);
}

}  // namespace

cudaError_t attn_tc_setup(bool* usable) {
  *usable = true;
  cudaError_t e;
  if ((e = setup_nd<Bf16, 1, false>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Bf16, 2, false>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Bf16, 2, true>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Fp16, 1, false>(usable)) != cudaSuccess) return e;
  if ((e = setup_nd<Fp16, 2, false>(usable)) != cudaSuccess) return e;
  return setup_nd<Fp16, 2, true>(usable);
}

cudaError_t launch_attn_tc(const AttnParams& p, const TcPieces& w, const CUtensorMap& qmap,
                           const CUtensorMap& kmap, const CUtensorMap& vmap, int dtype, int grid,
                           cudaStream_t s) {
  return dtype == MOE_ATTN_BF16 ? launch_t<Bf16>(p, w, qmap, kmap, vmap, grid, s)
                                : launch_t<Fp16>(p, w, qmap, kmap, vmap, grid, s);
}

}  // namespace attn
}  // namespace moe
