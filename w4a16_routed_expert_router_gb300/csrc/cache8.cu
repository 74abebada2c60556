// Writing keys and values to the 8-bit cache, and reading them back.
//
// Append. Tokens of one block (16 rows of a page) follow each other in a call, so a
// block's new tokens are a run of at most 16 consecutive tokens. Two warps have one run
// and one kv head, of K or of V, 8 rows each: they read the rows, raise the block's scale
// to the power of two that their largest value needs, write their codes, and where the
// scale has grown re-express the codes of the block's other rows. A CTA looks at a
// window of 16 tokens for the runs that begin there (one, in a prompt; up to 16, in a
// decode step, which `split` CTAs share), so nothing is planned on the host. Keys are
// normed and turned on the way, and kept in registers between the largest value and the
// codes. Queries are normed and turned by CTAs of the same launch, as in norm_rope.cu.
//
// Bound by instructions at 72 % of the issue slots: 8191 tokens of 32 + 8 heads of 128,
// with norms, take 41 us (185 MB, 4.5 TB/s; 27 us at the copy rate). A choice between
// product and division for each value cost 15 us of 94, four CTAs of 64 registers with
// some spills save 2 us over three of 80, heads that share a window's plan and its table
// of cosines 6 us. A decode step of 64 tokens is bound by latency, 6 us. The form for any
// rows (see norm_rope.cu): heads of 80 with 40 turned 139 us for 8192 tokens, of 96 with 24
// turned 123 (17 and 20 at the copy rate).
#include <algorithm>

#include "norm_parts.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = kWalkThreads, kWarps = kThreads / 32;
constexpr int kSms = 152;
constexpr int kRun = kScaleBlock;

// ------------------------------------------------------------------ codes
// two values as e4m3 codes, `lo` in the low byte; what is above 448 becomes 448
__device__ __forceinline__ uint16_t to_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t codes_to_f16(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ float2 codes_to_f32(uint16_t c) {
  const uint32_t h = codes_to_f16(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The least power of two s in 2^-64 .. 2^64 with top <= 448 s: 448 is 1.75 2^8.
__device__ __forceinline__ float scale_for(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return __int_as_float((min(max(e, -kScaleExp), kScaleExp) + 127) << 23);
}
// |x|, or 0 where that is no number
__device__ __forceinline__ float size_of(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}
__device__ __forceinline__ bool power_of_two(float s) {
  return (__float_as_int(s) & 0x807fffff) == 0;
}
// what x / scale is: exactly the product where the scale is a power of two (all scales
// that append wrote); chosen once for a run
struct Times {
  float inverse;
  __device__ __forceinline__ float operator()(float x) const { return x * inverse; }
};
struct Divide {
  float scale;
  __device__ __forceinline__ float operator()(float x) const { return __fdiv_rn(x, scale); }
};

// ------------------------------------------------------------------ append
struct Dims {  // of a launch
  int kv_ctas, token_groups;          // CTAs of keys and values; of queries along the tokens
  int q_heads, q_z;                   // heads of one, tokens side by side
  int q_rows;                         // groups of heads
  int split, combos, loops;           // CTAs that share a window's runs; of `loops` times
                                      // 4 (half, head)s
  int units, turned, lanes;
};

// A warp's rows of a run, in either form: in a lane, of each of its kSteps rows kValues
// values (chunks `a` and `b`, or single values).
constexpr int kWarpRows = kRun / 2;

template <typename T, bool IL, bool FAST>
struct RowsOf;

template <typename T, bool IL>
struct RowsOf<T, IL, true> {
  // 8 lanes a row or fewer: 4 rows at a time
  static constexpr int kSteps = 2, kValues = 16;
  Lane<IL> lane;
  int lanes, group, rows;
  bool active;
  float w[kValues];
  float v[kSteps][kValues];
  __device__ __forceinline__ RowsOf(const Dims& d, const RopeParams& r, float*)
      : lane((threadIdx.x & (d.lanes - 1)) < d.units ? threadIdx.x & (d.lanes - 1) : 0, d.turned,
             r.r.rot, r.head_dim),
        lanes(d.lanes),
        group((threadIdx.x & 31) / d.lanes),
        rows(32 / d.lanes),
        active((int)(threadIdx.x & (d.lanes - 1)) < d.units) {}
  // rows [0, n) from `first` on, `stride` apart, without norm and rotation
  __device__ __forceinline__ void load(const uint16_t* first, long long stride, int n) {
    Chunk8 a[kSteps], b[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = i * rows + group;
      a[i].v = b[i].v = make_uint4(0, 0, 0, 0);
      if (active && k < n) {
        a[i].v = *reinterpret_cast<const uint4*>(first + k * stride + lane.at);
        if (lane.two) b[i].v = *reinterpret_cast<const uint4*>(first + k * stride + lane.at + lane.gap);
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      unpack8<T>(a[i], v[i]);
      unpack8<T>(b[i], v[i] + 8);
    }
  }
  __device__ __forceinline__ void norm(const Norm& n, int h, float mean) {
    float sum[kSteps];
    lane.template weights<T>(n.k_weight, h * n.k_head, n.wide, n.offset, w, w + 8);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      sum[i] = 0.0f;
#pragma unroll
      for (int k = 0; k < kValues; ++k) sum[i] = fmaf(v[i][k], v[i][k], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) sum[i] = group_sum(sum[i], lanes);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const float f = rsqrtf(fmaf(sum[i], mean, n.eps));
#pragma unroll
      for (int k = 0; k < kValues; ++k)
        if (k < 8 || lane.two) v[i][k] = v[i][k] * f * w[k];
    }
  }
  __device__ __forceinline__ void turn(const RopeParams& r, const float* cosines,
                                       const float* sines, int, int n) {
    const int pairs = r.r.rot >> 1;
    if (!lane.turns) return;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = min(i * rows + group, n - 1);
      lane.turn(v[i], v[i] + 8, cosines + k * pairs, sines + k * pairs);
    }
  }
  __device__ __forceinline__ float top() const {
    float m = 0.0f;
    if (active) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int k = 0; k < kValues; ++k)
          if (k < 8 || lane.two) m = fmaxf(m, size_of(v[i][k]));
    }
    return m;
  }
  template <class By>
  static __device__ __forceinline__ uint2 codes(const float* f, const By& by) {
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c[i] = to_codes(by(f[4 * i]), by(f[4 * i + 1])) |
             (uint32_t)to_codes(by(f[4 * i + 2]), by(f[4 * i + 3])) << 16;
    return make_uint2(c[0], c[1]);
  }
  // row_of(k): the block's row that row k goes to, asked for by all lanes at once
  template <class By, class RowOf>
  __device__ __forceinline__ void store(const By& by, int n, uint8_t* block, long long token,
                                        const RowOf& row_of) const {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = i * rows + group, to = row_of(k);
      if (!active || k >= n) continue;
      uint8_t* row = block + to * token + lane.at;
      *reinterpret_cast<uint2*>(row) = codes(v[i], by);
      if (lane.two) *reinterpret_cast<uint2*>(row + lane.gap) = codes(v[i] + 8, by);
    }
  }
};

template <typename T>
struct RowsOf<T, false, false> {
  static constexpr int kLane = 4;
  int dim;
  float* row;
  float v[kWarpRows][kLane];
  __device__ __forceinline__ RowsOf(const Dims&, const RopeParams& r, float* smem)
      : dim(r.head_dim), row(smem + (threadIdx.x >> 5) * 128) {}
  __device__ __forceinline__ int index(int k) const { return (threadIdx.x & 31) + 32 * k; }
  __device__ __forceinline__ void load(const uint16_t* first, long long stride, int n) {
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
      for (int k = 0; k < kLane; ++k)
        v[i][k] = i < n && index(k) < dim ? T::to_f32(first[i * stride + index(k)]) : 0.0f;
  }
  __device__ __forceinline__ void norm(const Norm& n, int h, float mean) {
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kLane; ++k) sum = fmaf(v[i][k], v[i][k], sum);
      const float f = rsqrtf(fmaf(group_sum(sum, 32), mean, n.eps));
#pragma unroll
      for (int k = 0; k < kLane; ++k)
        if (index(k) < dim)
          v[i][k] *= f * weight_any<T>(n.k_weight, h * n.k_head + index(k), n.wide, n.offset);
    }
  }
  __device__ __forceinline__ void turn(const RopeParams& r, const float*, const float*, int t0,
                                       int n) {
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      if (i >= n) break;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kLane; ++k) row[index(k)] = v[i][k];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kLane; ++k)
        if (index(k) < dim) v[i][k] = turned_any(r.r, r.positions[t0 + i], row, index(k));
    }
  }
  __device__ __forceinline__ float top() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
      for (int k = 0; k < kLane; ++k) m = fmaxf(m, size_of(v[i][k]));
    return m;
  }
  template <class By, class RowOf>
  __device__ __forceinline__ void store(const By& by, int n, uint8_t* block, long long token,
                                        const RowOf& row_of) const {
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      uint8_t* row = block + row_of(i) * token;
#pragma unroll
      for (int k = 0; k < kLane; ++k)
        if (i < n && index(k) < dim) row[index(k)] = (uint8_t)to_codes(by(v[i][k]), 0.0f);
    }
  }
};

// Codes of a block's rows that are not in `written` (a bit a row), by a new scale; two
// warps, `sub` of them.
__device__ __forceinline__ void reexpress(uint8_t* block, long long token, int dim,
                                          unsigned written, float ratio, int sub) {
  const int chunks = dim >> 4;
  for (int i = (threadIdx.x & 31) + 32 * sub; i < kScaleBlock * chunks; i += 64) {
    const int r = i / chunks, c = i - r * chunks;
    if (written >> r & 1) continue;
    uint4* at = reinterpret_cast<uint4*>(block + r * token + c * 16);
    uint4 w = *at;
    uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 lo = codes_to_f32((uint16_t)x[k]), hi = codes_to_f32((uint16_t)(x[k] >> 16));
      x[k] = to_codes(lo.x * ratio, lo.y * ratio) |
             (uint32_t)to_codes(hi.x * ratio, hi.y * ratio) << 16;
    }
    *at = w;
  }
}

// Queries: norm and rotation, a lane group a head, as in norm_rope.cu.
template <typename T, bool IL>
__device__ __forceinline__ void queries(const Append8Params& g, const Dims& d, int cta,
                                        float* smem) {
  const RopeParams& r = g.p.r;
  const int tg = cta % d.token_groups, hg = cta / d.token_groups;
  const int u = threadIdx.x & (d.lanes - 1), y = threadIdx.x / d.lanes;
  Walk k;
  k.tid = threadIdx.x;
  k.threads = kThreads;
  k.lanes = d.lanes;
  k.z = y / d.q_heads;
  k.zs = d.q_z;
  k.c0 = tg * d.q_z;
  k.step = d.token_groups * d.q_z;
  const int hd = hg * d.q_heads + (y - k.z * d.q_heads);
  const bool active = k.z < d.q_z && hd < r.hq && u < d.units;
  if (!active) k.z = 0;
  const Lane<IL> lane(u < d.units ? u : 0, d.turned, r.r.rot, r.head_dim);
  const long long first = k.c0 + k.z, h = active ? hd : 0;
  norm_walk<T, IL>(
      k, r.r, r.positions, r.tokens, r.head_dim, g.p.n, lane, active, false,
      r.q.p + first * r.q.token + h * r.q.head + lane.at, r.q.token, g.p.n.q_weight,
      h * g.p.n.q_head, smem,
      RowRun{r.q_out.p + first * r.q_out.token + h * r.q_out.head + lane.at, r.q_out.token * k.step});
}

// Queries in the form for any rows: a warp a head.
template <typename T>
__device__ __forceinline__ void queries_any(const Append8Params& g, const Dims& d, int cta,
                                            float* smem) {
  const RopeParams& r = g.p.r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = cta % d.token_groups;
  const int hd = cta / d.token_groups * kWarps + warp;
  if (hd >= r.hq) return;
  float* row = smem + warp * 128;
  const uint16_t* src = r.q.p + (long long)t * r.q.token + (long long)hd * r.q.head;
  float v[4], sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    v[k] = i < r.head_dim ? T::to_f32(src[i]) : 0.0f;
    sum = fmaf(v[k], v[k], sum);
  }
  if (g.p.n.on) {
    const float f = rsqrtf(fmaf(group_sum(sum, 32), 1.0f / (float)r.head_dim, g.p.n.eps));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = lane + 32 * k;
      if (i < r.head_dim)
        v[k] *= f * weight_any<T>(g.p.n.q_weight, hd * g.p.n.q_head + i, g.p.n.wide,
                                  g.p.n.offset);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) row[lane + 32 * k] = v[k];
  __syncwarp();
  uint16_t* dst = r.q_out.p + (long long)t * r.q_out.token + (long long)hd * r.q_out.head;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    if (i < r.head_dim) dst[i] = T::from_f32(turned_any(r.r, r.positions[t], row, i));
  }
}

template <typename T, bool IL, bool FAST>
__global__ void __launch_bounds__(kThreads, 4)
    append8_kernel(const __grid_constant__ Append8Params g, const Dims d) {
  // (nothing static beside it: the queries' ring and tables may take all there is)
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  const RopeParams& r = g.p.r;
  wait_prior_launch();
  let_next_launch();
  int cta = blockIdx.x;                 // keys and values, which take longest, come first
  if (cta >= d.kv_ctas) {
    if constexpr (FAST)
      queries<T, IL>(g, d, cta - d.kv_ctas, smem);
    else
      queries_any<T>(g, d, cta - d.kv_ctas, smem);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & 1;
  const int first_combo = cta % d.combos * d.loops * (kWarps / 2);  // K heads, then V heads
  cta /= d.combos;
  const int part = cta % d.split, w0 = cta / d.split * kRun;
  // lane l has token w0 - 1 + l: the one before the window, the window, and what runs
  // that begin there may go on with
  const int t = w0 - 1 + lane;
  long long slot = -1;
  if (t >= 0 && t < r.tokens) {
    slot = r.slots[t];
    if (slot >= r.num_slots) {
      if (lane > 0 && lane <= kRun) atomicOr(r.err, kErrRange);
      slot = -1;
    }
  }
  const long long prev = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool follows = lane > 0 && slot >= 0 && prev >= 0 && prev < slot &&
                       prev / kScaleBlock == slot / kScaleBlock;
  const unsigned go_on = __ballot_sync(0xffffffffu, follows);
  unsigned begin = __ballot_sync(0xffffffffu, slot >= 0 && !follows && lane > 0 && lane <= kRun);
  const bool any_keys = first_combo < r.hk;            // in the CTA
  const int pairs = r.r.rot >> 1;
  float *tops = smem, *cosines = smem + kWarps, *sines = cosines + kRun * pairs;
  for (int i = 0; begin; ++i) {
    const int at = __ffs(begin) - 1;
    begin &= begin - 1;
    if (i % d.split != part) continue;
    // the run [t0, t0 + n) goes on while the bits behind its first token are set; this
    // warp has `mine` rows from k0 on
    const int n = at == 31 ? 1 : __ffs(~(go_on >> (at + 1)));
    const int t0 = w0 - 1 + at, k0 = sub * kWarpRows, mine = min(kWarpRows, n - k0);
    const long long slot0 = __shfl_sync(0xffffffffu, slot, at);
    // rows of the block that the run has, and the row of each of its tokens
    const int row_of = (int)(slot - slot0) + (int)(slot0 & (kScaleBlock - 1));
    const unsigned written =
        __reduce_or_sync(0xffffffffu, lane >= at && lane < at + n ? 1u << (row_of & 31) : 0u);
    const long long page = slot0 >> r.page_shift;
    const int in_page = (int)(slot0 - (page << r.page_shift));
    const int first = in_page & (kScaleBlock - 1), block = in_page / kScaleBlock;
    if (FAST && any_keys)
      fill_table(r.r, r.positions + t0, n, cosines, sines, threadIdx.x, kThreads);
    for (int loop = 0; loop < d.loops; ++loop) {
      const int combo = first_combo + loop * (kWarps / 2) + (warp >> 1);
      const bool key = combo < r.hk, on = combo < 2 * r.hk;
      const int h = key ? combo : combo - r.hk;
      const Rows& in = key ? r.k : r.v;
      uint8_t* codes = (key ? g.c.k : g.c.v) + page * g.c.page + (long long)h * g.c.head +
                       (long long)(in_page - first) * g.c.token;
      float* scale_at = (key ? g.c.k_scales : g.c.v_scales) + page * g.c.scale_page +
                        h * g.c.scale_head + block * g.c.scale_block;
      RowsOf<T, IL, FAST> of(d, r, smem + kWarps);
      float top = 0.0f, before = 0.0f;
      if (on) {
        if (first) before = *scale_at;
        if (mine > 0)
          of.load(in.p + (long long)(t0 + k0) * in.token + (long long)h * in.head, in.token, mine);
      }
      if (FAST && any_keys && loop == 0) __syncthreads();  // the table is there
      if (on && mine > 0) {
        if (key) {
          if (g.p.n.on) of.norm(g.p.n, h, 1.0f / (float)r.head_dim);
          of.turn(r, cosines + k0 * pairs, sines + k0 * pairs, t0 + k0, mine);
        }
        top = of.top();
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) tops[warp] = top;
      __syncthreads();  // (and the old scale is read)
      float scale = scale_for(fmaxf(top, tops[warp ^ 1]));
      if (on) {
        if (first && before > 0.0f && before < INFINITY) {
          if (before >= scale)
            scale = before;
          else
            reexpress(codes, g.c.token, r.head_dim, written, before / scale, sub);
        }
        if (lane == 0 && sub == 0) *scale_at = scale;
      }
      // (all lanes: they hand out the rows)
      const auto row = [&](int k) { return __shfl_sync(0xffffffffu, row_of, (at + k0 + k) & 31); };
      if (on && mine > 0) {
        if (power_of_two(scale))
          of.store(Times{1.0f / scale}, mine, codes, g.c.token, row);
        else
          of.store(Divide{scale}, mine, codes, g.c.token, row);
      }
      __syncthreads();  // tops is free again, and at the end the table
    }
  }
}

template <typename T, bool IL, bool FAST>
cudaError_t launch_append(const Append8Params& g, cudaStream_t s) {
  const RopeParams& r = g.p.r;
  Dims d{};
  int smem;
  if (FAST) {
    const Units u = units_of_head(r.head_dim, r.r.rot);
    d.units = u.count;
    d.turned = u.turned;
    d.lanes = u.lanes;
    const int most = kThreads / u.lanes;
    d.q_rows = (r.hq + most - 1) / most;
    d.q_heads = d.q_rows ? (r.hq + d.q_rows - 1) / d.q_rows : 1;
    d.q_z = 1;
    while (2 * d.q_z * d.q_heads <= most && 2 * d.q_z * r.r.rot <= kWalkTurned &&
           (long long)r.tokens * d.q_rows >= 8LL * kSms * d.q_z)
      d.q_z *= 2;
    // up to 8 tokens to a thread, where every SM has CTAs enough
    const int all = (r.tokens + d.q_z - 1) / d.q_z;
    const int few = d.q_rows ? (4 * kSms + d.q_rows - 1) / d.q_rows : 1;
    d.token_groups = std::min(all, std::max(few, (all + 7) / 8));
    smem = std::max((kWarps + kRun * r.r.rot) * (int)sizeof(float),
                    r.hq ? (int)Walk::bytes(d.q_z, r.r.rot) : 0);
  } else {
    d.q_rows = (r.hq + kWarps - 1) / kWarps;
    d.token_groups = r.tokens;
    smem = kWarps * (1 + 128) * (int)sizeof(float);
  }
  d.combos = (2 * r.hk + kWarps / 2 - 1) / (kWarps / 2);
  const int windows = (r.tokens + kRun - 1) / kRun;
  // in long calls up to four times four, which share a window's plan and its table
  d.loops = 1;
  while (d.loops < 4 && d.combos > 1 && (long long)windows * d.combos > 4 * kSms) {
    d.loops *= 2;
    d.combos = (d.combos + 1) / 2;
  }
  // a window's runs to as many CTAs as the GPU takes at once: decode steps have a run
  // for each token, prompts one for each window
  d.split = kRun;
  while (d.split > 1 && (long long)windows * d.combos * d.split > 4 * kSms) d.split /= 2;
  d.kv_ctas = windows * d.combos * d.split;
  const long long ctas = d.kv_ctas + (long long)d.token_groups * d.q_rows;
  return launch_after(append8_kernel<T, IL, FAST>, dim3((unsigned)ctas), dim3(kThreads), smem, s, g,
                      d);
}

// ------------------------------------------------------------------ read back
// A CTA has up to 32 rows of the outputs, all heads: it brings the sequences' first rows
// to shared memory (as many as there is room for; every thread then counts some of those
// that begin at or before its first row), a lane a row finds its sequence by bisection and
// looks up its page, then all threads bring 16 codes at a time to 32 bytes of the
// outputs. Bound by memory: 16 sequences of up to 16384 tokens, 8 heads of 128, 931 MB
// take 148 us (6.3 TB/s).
constexpr int kReadRows = 32, kReadSeqs = 1024;

// Two values of the cache in 16 bits. A finite value stays finite: fp16 takes what is
// above 65504 as that (append holds 65000 as 256 * 256, half a step of the codes above
// it). bf16 has room for every code by every scale.
template <typename T>
__device__ __forceinline__ uint32_t pack_held(float lo, float hi) {
  if (!T::kFp16) return T::pack(lo, hi);
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T>
__device__ __forceinline__ void read16(const uint4& w, float scale, uint16_t* to, bool wide) {
  const uint32_t* x = reinterpret_cast<const uint32_t*>(&w);
  uint32_t y[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 lo = codes_to_f32((uint16_t)x[k]), hi = codes_to_f32((uint16_t)(x[k] >> 16));
    y[2 * k] = pack_held<T>(lo.x * scale, lo.y * scale);
    y[2 * k + 1] = pack_held<T>(hi.x * scale, hi.y * scale);
  }
  if (wide) {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(y[4], y[5], y[6], y[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) to[k] = (uint16_t)(y[k >> 1] >> (16 * (k & 1)));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read8_kernel(const Read8Params p, int rows_shift,
                                                         int wide) {
  __shared__ long long code_at[kReadRows], scale_at[kReadRows];
  __shared__ int cu[kReadSeqs + 1];
  __shared__ int counts[kWarps];
  const int cta_rows = 1 << rows_shift, row0 = blockIdx.x << rows_shift;
  wait_prior_launch();
  let_next_launch();
  // the sequences from s0 on, the first of them the one that row0 may be in
  int s0 = 0;
  if (p.num_seqs > kReadSeqs) {
    int mine = 0;
    for (int s = 1 + threadIdx.x; s <= p.num_seqs; s += kThreads) mine += p.cu[s] <= row0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s0 += counts[i];
  }
  const int kept = min(p.num_seqs - s0, kReadSeqs);
  for (int i = threadIdx.x; i <= kept; i += kThreads) cu[i] = p.cu[s0 + i];
  __syncthreads();
  if (threadIdx.x < cta_rows) {
    const int row = row0 + threadIdx.x;
    int lo = 0, hi = kept;                             // last sequence with cu <= row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= row)
        lo = mid;
      else
        hi = mid - 1;
    }
    // (behind what is kept, where thousands of sequences have no rows)
    int s = s0 + lo;
    while (s < p.num_seqs && p.cu[s + 1] <= row) ++s;
    long long at = -1, sc = 0;
    const int begin = s < p.num_seqs ? p.cu[s] : 0;
    if (row < p.rows && s < p.num_seqs && begin >= 0 && row >= begin) {
      const long long pos = (long long)p.first[s] + (row - begin);
      const long long limit = (long long)p.columns << p.page_shift;
      int page = -1;
      if (p.first[s] >= 0 && pos < limit)
        page = p.page_table[s * p.table_stride + (pos >> p.page_shift)];
      if (page < 0 || page >= p.c.num_pages) {
        atomicOr(p.err, kErrRange);
      } else {
        const int in_page = (int)(pos & ((1 << p.page_shift) - 1));
        at = page * p.c.page + in_page * p.c.token;
        sc = page * p.c.scale_page + in_page / kScaleBlock * p.c.scale_block;
      }
    }
    code_at[threadIdx.x] = at;
    scale_at[threadIdx.x] = sc;
  }
  __syncthreads();
  const int chunks = p.head_dim >> 4, items = (p.hk * chunks) << rows_shift;
#pragma unroll 4
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int rest = i / chunks, c = i - rest * chunks;
    const int r = rest & (cta_rows - 1), h = rest >> rows_shift;
    if (code_at[r] < 0) continue;
    const long long at = code_at[r] + h * p.c.head + c * 16, sc = scale_at[r] + h * p.c.scale_head;
    const float ks = __ldg(p.c.k_scales + sc), vs = __ldg(p.c.v_scales + sc);
    const uint4 k = __ldg(reinterpret_cast<const uint4*>(p.c.k + at));
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.c.v + at));
    read16<T>(k, ks,
              p.k_out.p + (long long)(row0 + r) * p.k_out.token + h * p.k_out.head + c * 16, wide);
    read16<T>(v, vs,
              p.v_out.p + (long long)(row0 + r) * p.v_out.token + h * p.v_out.head + c * 16, wide);
  }
}

// ------------------------------------------------------------------ a batch's keys in 16 bits
// Persistent CTAs over parts of the pages of all sequences, dealt out in turn: every CTA
// adds up the sequences' pages for itself, keeps the first page of each while they are
// few, and finds a page's sequence by bisection. A part is what a CTA's threads bring with
// their loads under way at once. Blocks of kTcBlock keys that no query sees are passed
// over. Bound by memory. (Whole pages to a CTA left most of them without work where pages
// are few: a chunk of 256 tokens over 32768 keys, with its attention, 158 us, 146 so.)
constexpr int kFirstKept = 2048, kPartItems = 2 * kThreads;   // of 16 values of K and of V

template <typename T>
__global__ void __launch_bounds__(kThreads) expand8_kernel(const Expand8Params p) {
  __shared__ int first[kFirstKept + 1];
  __shared__ int sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, seqs = p.b.num_seqs;
  const int page_rows = 1 << p.page_shift, chunks = p.head_dim >> 4;
  const int row_chunks = page_rows * chunks, items = p.hk * row_chunks;
  const int parts = (items + kPartItems - 1) / kPartItems;   // of a page
  wait_prior_launch();
  let_next_launch();
  // Pages of sequence s. (A sequence whose lengths leave their ranges has none.)
  const auto pages_of = [&](int s) {
    const Span r = read_sequence(p.b, p.page_shift, s, p.err);
    return r.n > 0 ? (r.kv + page_rows - 1) >> p.page_shift : 0;
  };
  int base = 0;                                        // pages before sequence s0
  for (int s0 = 0; s0 < seqs; s0 += kFirstKept) {
    const int n = min(kFirstKept, seqs - s0);
    const int per = (n + kThreads - 1) / kThreads;
    const int a = min(n, tid * per), b = min(n, a + per);
    int mine = 0;
    for (int i = a; i < b; ++i) mine += pages_of(s0 + i);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int at = base + incl - mine, total = base;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += sums[i];
      total += sums[i];
    }
    for (int i = a; i < b; ++i) {
      first[i] = at;
      at += pages_of(s0 + i);
    }
    if (tid == 0) first[n] = total;
    __syncthreads();
    // this CTA's parts of pages [base, total)
    const long long u0 = (long long)base * parts, u1 = (long long)total * parts;
    long long u = u0 + (blockIdx.x + gridDim.x - u0 % gridDim.x) % gridDim.x;
    int lo = 0;
    for (; u < u1; u += gridDim.x) {
      const int i = (int)(u / parts), part = (int)(u - (long long)i * parts);
      int hi = n - 1;                                  // last sequence with first <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int seq = s0 + lo, column = i - first[lo], key0 = column << p.page_shift;
      if (tid == 0 && part == 0) p.table[(long long)seq * p.b.columns + column] = i;
      const int kv = p.b.kv_len[seq], n_new = p.b.cu_q[seq + 1] - p.b.cu_q[seq];
      const int kept = kept_of(p.sc, prefix_of(p.sc, seq, kv), kv - 1);
      const int from = p.sc.window ? max(0, kv - n_new - p.sc.window + 1) : 0;
      if (key0 + page_rows <= from / kTcBlock * kTcBlock &&
          key0 >= (kept + kTcBlock - 1) / kTcBlock * kTcBlock)
        continue;
      const int page = p.b.page_table[seq * p.b.table_stride + column];
      const bool bad = page < 0 || page >= p.c.num_pages;
      if (bad && tid == 0) atomicOr(p.err, kErrRange);
      const int rows = min(page_rows, kv - key0);
      const long long out = (long long)i * p.hk * page_rows * p.head_dim;
      constexpr int kItems = kPartItems / kThreads;
      uint4 k[kItems], v[kItems];
      float ks[kItems], vs[kItems];
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int e = part * kPartItems + q * kThreads + tid;
        const int row = e / chunks, c = e - row * chunks;
        const int h = row >> p.page_shift, r = row & (page_rows - 1);
        k[q] = v[q] = make_uint4(0, 0, 0, 0);
        ks[q] = vs[q] = 0.0f;
        if (e < items && r < rows && !bad) {
          const long long code = page * p.c.page + h * p.c.head + r * p.c.token + c * 16;
          const long long scale =
              page * p.c.scale_page + h * p.c.scale_head + r / kScaleBlock * p.c.scale_block;
          k[q] = __ldg(reinterpret_cast<const uint4*>(p.c.k + code));
          v[q] = __ldg(reinterpret_cast<const uint4*>(p.c.v + code));
          ks[q] = __ldg(p.c.k_scales + scale);
          vs[q] = __ldg(p.c.v_scales + scale);
        }
      }
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int e = part * kPartItems + q * kThreads + tid;
        if (e >= items || (e / chunks & (page_rows - 1)) >= rows) continue;
        read16<T>(k[q], ks[q], p.k + out + (long long)e * 16, true);
        read16<T>(v[q], vs[q], p.v + out + (long long)e * 16, true);
      }
    }
    base = total;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_append8(const Append8Params& g, int dtype, cudaStream_t s) {
  const RopeParams& r = g.p.r;
  const bool fast = units_fit(r.r, r.head_dim) && weights_aligned(g.p.n) && rows_aligned(r.q) &&
                    rows_aligned(r.q_out) && rows_aligned(r.k) && rows_aligned(r.v);
  const bool il = r.r.interleaved;
  if (dtype == MOE_ATTN_BF16)
    return !fast ? launch_append<Bf16, false, false>(g, s)
           : il  ? launch_append<Bf16, true, true>(g, s)
                 : launch_append<Bf16, false, true>(g, s);
  return !fast ? launch_append<Fp16, false, false>(g, s)
         : il  ? launch_append<Fp16, true, true>(g, s)
               : launch_append<Fp16, false, true>(g, s);
}

cudaError_t launch_read8(const Read8Params& p, int dtype, cudaStream_t s) {
  // fewer rows a CTA until every SM has four CTAs (8191 rows with their append: 58.6 us
  // until it has two, 54.9 so, 55.9 until it has 16)
  int shift = 5;
  while (shift > 1 && (p.rows >> shift) < 4 * kSms) --shift;
  const dim3 grid((p.rows + (1 << shift) - 1) >> shift), block(kThreads);
  const int wide = rows_aligned(p.k_out) && rows_aligned(p.v_out);
  return dtype == MOE_ATTN_BF16
             ? launch_after(read8_kernel<Bf16>, grid, block, 0, s, p, shift, wide)
             : launch_after(read8_kernel<Fp16>, grid, block, 0, s, p, shift, wide);
}

cudaError_t launch_expand8(const Expand8Params& p, int dtype, int grid, cudaStream_t s) {
  // 16 CTAs for each SM, as far as the table's pages have parts for them (prompts of 8192
  // tokens, with their attention: 378 us with the 4 or 6 that run at once, 372 with 16,
  // 376 with 32)
  const long long items = (long long)p.hk * p.head_dim / 16 << p.page_shift;
  const long long parts = (items + kPartItems - 1) / kPartItems * p.b.num_seqs * p.b.columns;
  const dim3 ctas((unsigned)std::min(16LL * grid, parts)), block(kThreads);
  return dtype == MOE_ATTN_BF16 ? launch_after(expand8_kernel<Bf16>, ctas, block, 0, s, p)
                                : launch_after(expand8_kernel<Fp16>, ctas, block, 0, s, p);
}

}  // namespace attn
}  // namespace moe
