// Norms of queries and keys for each head with the rotary positions in the same
// pass, and their gradient.
//
// Forward: y = R_p(x rsqrt(mean x^2 + eps) (w + offset)), read once, written once. A
// group of lanes has a head and walks along the tokens (norm_walk in norm_parts.cuh). The
// CTA makes the tables of cosines and sines, one evaluation for its heads. 8192 tokens of
// 40 heads of 128 take 35 us (168 MB, 4.8 TB/s; the same kernel without sums, rotation
// and weights takes 28, the copy rate 25): latency and instructions, 260 for 16 values of a
// lane, at 55 % of the issue slots. (A few tokens a thread, loaded to registers first, took 44 us:
// a third of its instructions prepared a thread for them. Rows in units of one chunk for
// interleaved pairs cost as many sums and addresses again.) Into 16-bit pages, with 8
// heads of values beside them, 42 us (201 MB; 30 at the copy rate).
//
// Rotations that are not a multiple of 16 values, and rows that are not aligned, go a warp
// a head, which evaluates an angle for each value of each head: 8192 tokens of 40 heads of
// 80 with 40 turned 147 us (15.5 at the copy rate; all 80 turned, in the fast form, 30), of
// 96 with 24 turned 129 (18.6); their gradient 390 (23) and 364 (28).
//
// Gradient: with u = R_p^T dy, n = x r and h = u (w + offset),
//   dx = r (h - n mean(h n)),  dw = sum u n.
// mean(h n) = r mean(h x), so both sums over a head, of x^2 and of h x, are taken
// together. Each thread keeps one unit of one head for many tokens and adds up that
// unit's dw; a CTA adds its rows in order, and a second launch the CTAs (8 of 16 us for
// 2047 tokens of 20 heads of 64: 456 rows). 16384 tokens of
// 40 heads of 128 take 107 us (503 MB, 4.7 TB/s; 75 at the copy rate): latency, with 15
// warps an SM at 122 registers; two values to an instruction change nothing. (The
// forward's ring of copies in place of registers: 134 us, for its instructions and spills.)
#include <algorithm>

#include "norm_parts.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSms = 152;

// where a key or value of token t goes in the pages, or null
__device__ __forceinline__ uint16_t* page_row(const RopeParams& r, bool key, int t, int h) {
  const long long slot = r.slots[t];
  if (slot < 0) return nullptr;
  if (slot >= r.num_slots) {
    atomicOr(r.err, kErrRange);
    return nullptr;
  }
  const long long page = slot >> r.page_shift;
  return (key ? r.k_pages : r.v_pages) + page * r.page_stride +
         (slot - (page << r.page_shift)) * r.token_stride + (long long)h * r.head_stride;
}

// What row (token, head) is: queries, then keys, then values.
struct Head {
  int h;
  bool key, value;
  __device__ __forceinline__ Head(const RopeParams& r, int hd) {
    key = hd >= r.hq && hd < r.hq + r.hk;
    value = hd >= r.hq + r.hk;
    h = hd - (value ? r.hq + r.hk : key ? r.hq : 0);
  }
  // (by value: a reference makes every use a load from an address among the parameters)
  static __device__ __forceinline__ Rows pick(bool first, const Rows& a, const Rows& b) {
    return Rows{first ? a.p : b.p, first ? a.token : b.token, first ? a.head : b.head};
  }
  __device__ __forceinline__ Rows in(const RopeParams& r) const {
    return pick(value, r.v, pick(key, r.k, r.q));
  }
  __device__ __forceinline__ uint16_t* out(const NormParams& p, int t) const {
    if ((key || value) && p.r.slots) return page_row(p.r, key, t, h);
    const Rows o = pick(key, p.k_out, p.r.q_out);
    return o.p + (long long)t * o.token + (long long)h * o.head;
  }
};

// Where rows go in a launch that writes keys and values to pages.
struct PagedRun {
  const RopeParams& r;
  RowRun run;
  bool key, paged;
  int h, at;
  __device__ __forceinline__ uint16_t* next(int t) {
    if (!paged) return run.next(t);
    uint16_t* row = page_row(r, key, t, h);
    return row ? row + at : nullptr;
  }
};

template <typename T, bool IL, bool PAGES>
__global__ void __launch_bounds__(kWalkThreads, 3)
    norm_rope_kernel(const __grid_constant__ NormParams p, int units, int turned) {
  extern __shared__ float4 smem4[];
  const RopeParams& r = p.r;
  wait_prior_launch();
  let_next_launch();
  const int u = threadIdx.x, hd = blockIdx.y * blockDim.y + threadIdx.y;
  const bool active = hd < r.hq + r.hk + r.hv && u < units;
  const Head hh(r, active ? hd : 0);
  const Lane<IL> lane(active ? u : 0, turned, r.r.rot, r.head_dim);
  Walk k;
  k.tid = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x;
  k.threads = blockDim.x * blockDim.y * blockDim.z;
  k.lanes = blockDim.x;
  k.z = threadIdx.z;
  k.zs = blockDim.z;
  k.c0 = blockIdx.x * k.zs;
  k.step = gridDim.x * k.zs;
  const Rows in = hh.in(r), o = Head::pick(hh.key, p.k_out, r.q_out);
  const long long first = k.c0 + k.z;
  const RowRun run = {o.p + first * o.token + (long long)hh.h * o.head + lane.at, o.token * k.step};
  const auto walk = [&](auto out) {
    norm_walk<T, IL>(k, r.r, r.positions, r.tokens, r.head_dim, p.n, lane, active, hh.value,
                     in.p + first * in.token + (long long)hh.h * in.head + lane.at, in.token,
                     hh.key ? p.n.k_weight : p.n.q_weight,
                     hh.h * (hh.key ? p.n.k_head : p.n.q_head), reinterpret_cast<float*>(smem4),
                     out);
  };
  if constexpr (PAGES)
    walk(PagedRun{r, run, hh.key, hh.key || hh.value, hh.h, lane.at});
  else
    walk(run);
}

constexpr int kAnyWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kAnyWarps * 32)
    norm_rope_any_kernel(const __grid_constant__ NormParams p, int tokens_per_warp) {
  __shared__ float row[kAnyWarps][32 * kAnyValues];
  const RopeParams& r = p.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hd = blockIdx.y * kAnyWarps + warp;
  wait_prior_launch();
  let_next_launch();
  if (hd >= r.hq + r.hk + r.hv) return;
  const Head hh(r, hd);
  const Rows in = hh.in(r);
  const void* w = hh.key ? p.n.k_weight : p.n.q_weight;
  const long long wh = hh.h * (hh.key ? p.n.k_head : p.n.q_head);
  const int t1 = min(r.tokens, (int)(blockIdx.x + 1) * tokens_per_warp);
  for (int t = blockIdx.x * tokens_per_warp; t < t1; ++t) {
    const uint16_t* src = in.p + (long long)t * in.token + (long long)hh.h * in.head;
    uint16_t x[kAnyValues];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kAnyValues; ++k) {
      const int i = lane + 32 * k;
      x[k] = i < r.head_dim ? src[i] : (uint16_t)0;
      sum = fmaf(T::to_f32(x[k]), T::to_f32(x[k]), sum);
    }
    sum = group_sum(sum, 32);
    const float f = rsqrtf(fmaf(sum, 1.0f / (float)r.head_dim, p.n.eps));
    uint16_t* dst = hh.out(p, t);
    if (!hh.value) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kAnyValues; ++k) {
        const int i = lane + 32 * k;
        if (i < r.head_dim)
          row[warp][i] = T::to_f32(x[k]) * f * weight_any<T>(w, wh + i, p.n.wide, p.n.offset);
      }
      __syncwarp();
    }
    if (!dst) continue;
#pragma unroll
    for (int k = 0; k < kAnyValues; ++k) {
      const int i = lane + 32 * k;
      if (i < r.head_dim)
        dst[i] = hh.value ? x[k] : T::from_f32(turned_any(r.r, r.positions[t], row[warp], i));
    }
  }
}

template <typename T, bool IL>
cudaError_t launch_fast(const NormParams& p, cudaStream_t s) {
  const RopeParams& r = p.r;
  const Units u = units_of_head(r.head_dim, r.r.rot);
  const int heads = r.hq + r.hk + r.hv;
  // groups of heads of at most kWalkThreads threads, tokens side by side where heads are
  // few, and as many CTAs along the tokens as the GPU takes at once
  const int most = kWalkThreads / u.lanes;
  const int groups = (heads + most - 1) / most;
  dim3 block(u.lanes, (heads + groups - 1) / groups, 1);
  while (2 * block.x * block.y * block.z <= kWalkThreads && block.z < 64 &&
         2 * block.z * r.r.rot <= kWalkTurned &&
         (long long)r.tokens * groups >= 8LL * kSms * block.z)
    block.z *= 2;
  const int threads = block.x * block.y * block.z;
  const int want = std::max(1, kSms * (3 * kWalkThreads / threads) / groups);
  const int all = (r.tokens + block.z - 1) / block.z;
  return launch_after(r.slots ? norm_rope_kernel<T, IL, true> : norm_rope_kernel<T, IL, false>,
                      dim3(std::min(want, all), groups), block,
                      (int)Walk::bytes(block.z, r.r.rot), s, p, u.count, u.turned);
}

bool fits(const NormParams& p) {
  const RopeParams& r = p.r;
  if (!units_fit(r.r, r.head_dim) || !weights_aligned(p.n)) return false;
  if (r.slots && (r.page_stride % 8 || r.token_stride % 8 || r.head_stride % 8)) return false;
  return rows_aligned(r.q) && rows_aligned(r.q_out) && rows_aligned(r.k) && rows_aligned(p.k_out) &&
         rows_aligned(r.v);
}

template <typename T>
cudaError_t launch_t(const NormParams& p, cudaStream_t s) {
  if (fits(p)) return p.r.r.interleaved ? launch_fast<T, true>(p, s) : launch_fast<T, false>(p, s);
  const int heads = p.r.hq + p.r.hk + p.r.hv, groups = (heads + kAnyWarps - 1) / kAnyWarps;
  const int tokens = p.r.tokens >= 16 * kSms ? 4 : 1;
  return launch_after(norm_rope_any_kernel<T>, dim3((p.r.tokens + tokens - 1) / tokens, groups),
                      dim3(kAnyWarps * 32), 0, s, p, tokens);
}

// ------------------------------------------------------------------ gradient

constexpr int kGradThreads = 256, kTables = 4;

template <typename T, bool IL>
__global__ void __launch_bounds__(kGradThreads, 2)
    norm_grad_kernel(const __grid_constant__ NormGradParams g, int units, int turned, int shared) {
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  const NormParams& p = g.p;
  const RopeParams& r = p.r;
  const Pairs head(r.r.rot);
  const int pairs = head.count, z = blockDim.z, z_shift = __ffs(z) - 1, heads = r.hq + r.hk;
  wait_prior_launch();
  let_next_launch();
  const int u = threadIdx.x, hd = blockIdx.y * blockDim.y + threadIdx.y;
  const bool active = hd < heads && u < units;
  const Head hh(r, active ? hd : 0);
  const Lane<IL> lane(active ? u : 0, turned, r.r.rot, r.head_dim);
  const Rows in = hh.in(r), dy = Head::pick(hh.key, g.dk, g.dq),
             dx = Head::pick(hh.key, p.k_out, r.q_out);
  const long long hi = hh.h * in.head + lane.at, hy = hh.h * dy.head + lane.at,
                  ho = hh.h * dx.head + lane.at;
  float wa[8], wb[8], da[8], db[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) da[k] = db[k] = wa[k] = wb[k] = 0.0f;
  if (active)
    lane.template weights<T>(hh.key ? p.n.k_weight : p.n.q_weight,
                             hh.h * (hh.key ? p.n.k_head : p.n.q_head), p.n.wide, p.n.offset, wa,
                             wb);
  const int tid = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x;
  const int threads = blockDim.x * blockDim.y * blockDim.z;
  const float mean = 1.0f / (float)r.head_dim;
  // a token's chunks, one iteration ahead
  const int step = gridDim.x * z;
  int t = blockIdx.x * z + threadIdx.z, coming = active ? t : r.tokens;
  const uint16_t* x = in.p + (long long)t * in.token + hi;
  const uint16_t* y = dy.p + (long long)t * dy.token + hy;
  uint16_t* out = dx.p + (long long)t * dx.token + ho;
  const long long x_step = in.token * step, y_step = dy.token * step, out_step = dx.token * step;
  Chunk8 next[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) next[k].v = make_uint4(0, 0, 0, 0);
  const auto load = [&]() {
    if (coming < r.tokens) {
      next[0].v = *reinterpret_cast<const uint4*>(x);
      next[1].v = *reinterpret_cast<const uint4*>(y);
      if (lane.two) {
        next[2].v = *reinterpret_cast<const uint4*>(x + lane.gap);
        next[3].v = *reinterpret_cast<const uint4*>(y + lane.gap);
      }
      x += x_step;
      y += y_step;
      coming += step;
    }
  };
  // of kTables iterations at once, which takes most threads
  const auto table = [&](int c0) {
    for (int i = tid; i < kTables * z * pairs; i += threads) {
      const int row = head.token(i), c = i - row * pairs;
      const int t = c0 + (row >> z_shift) * step + (row & (z - 1));
      if (t >= r.tokens) continue;
      cos_sin(r.r, r.positions[t], c, smem[i], smem[kTables * z * pairs + i]);
    }
  };
  const float* cosines = smem;
  load();
  for (int c0 = blockIdx.x * z, turn = 0; c0 < r.tokens; c0 += step, t += step) {
    const bool on = active && t < r.tokens;
    const Chunk8 xa = next[0], ya = next[1], xb = next[2], yb = next[3];
    load();
    if (turn == 0) {
      __syncthreads();
      table(c0);
      __syncthreads();
      turn = kTables;
      cosines = smem + threadIdx.z * pairs;
    }
    float fx[8], gx[8], ua[8], ub[8];
    unpack8<T>(xa, fx);
    unpack8<T>(xb, gx);
    unpack8<T>(ya, ua);
    unpack8<T>(yb, ub);
    if (on && lane.turns)
      lane.turn(ua, ub, cosines, cosines + kTables * z * pairs);
    --turn;
    cosines += z * pairs;
    float sq = 0.0f, dot = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sq = fmaf(fx[k], fx[k], sq);
      sq = fmaf(gx[k], gx[k], sq);
      dot = fmaf(ua[k] * wa[k], fx[k], dot);
      dot = fmaf(ub[k] * wb[k], gx[k], dot);
    }
    sq = group_sum(sq, blockDim.x);
    dot = group_sum(dot, blockDim.x);
    if (!on) continue;
    const float f = rsqrtf(fmaf(sq, mean, p.n.eps));
    const float c = -(dot * mean * f * f) * f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ua[k] *= f;
      da[k] = fmaf(ua[k], fx[k], da[k]);
      ua[k] = fmaf(c, fx[k], ua[k] * wa[k]);
      if (lane.two) {
        ub[k] *= f;
        db[k] = fmaf(ub[k], gx[k], db[k]);
        ub[k] = fmaf(c, gx[k], ub[k] * wb[k]);
      }
    }
    *reinterpret_cast<uint4*>(out) = pack8<T>(ua);
    if (lane.two) *reinterpret_cast<uint4*>(out + lane.gap) = pack8<T>(ub);
    out += out_step;
  }
  // the CTA's rows in order: tokens side by side, then the heads that share a weight
  __syncthreads();
  const int d = r.head_dim, ny = blockDim.y;
  if (active) {
    float* to = smem + (threadIdx.z * ny + threadIdx.y) * d + lane.at;
#pragma unroll
    for (int k = 0; k < 8; ++k) to[k] = da[k];
    if (lane.two) {
#pragma unroll
      for (int k = 0; k < 8; ++k) to[lane.gap + k] = db[k];
    }
  }
  __syncthreads();
  const int h0 = blockIdx.y * ny, h1 = min(heads, h0 + ny);
  const long long cta = (long long)blockIdx.x * gridDim.y + blockIdx.y;
  const int rows = shared ? 2 : ny;
  for (int i = tid; i < rows * d; i += threads) {
    const int w = i / d, v = i - w * d;
    int y0 = w, y1 = w + 1;
    if (shared) {  // queries, or keys, of this CTA
      y0 = w == 0 ? 0 : max(0, r.hq - h0);
      y1 = w == 0 ? min(h1, r.hq) - h0 : h1 - h0;
    } else if (h0 + w >= h1) {
      y1 = y0;
    }
    float sum = 0.0f;
    for (int y = y0; y < y1; ++y)
      for (int k = 0; k < z; ++k) sum += smem[(k * ny + y) * d + v];
    g.parts[(cta * rows + w) * d + v] = sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(kAnyWarps * 32) norm_grad_any_kernel(const __grid_constant__ NormGradParams g) {
  __shared__ float row[kAnyWarps][32 * kAnyValues];
  const NormParams& p = g.p;
  const RopeParams& r = p.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = r.hq + r.hk;
  const int hd = blockIdx.y * kAnyWarps + warp;
  wait_prior_launch();
  let_next_launch();
  if (hd >= heads) return;
  const Head hh(r, hd);
  const Rows in = hh.in(r), dy = Head::pick(hh.key, g.dk, g.dq),
             dx = Head::pick(hh.key, p.k_out, r.q_out);
  const void* w = hh.key ? p.n.k_weight : p.n.q_weight;
  const long long wh = hh.h * (hh.key ? p.n.k_head : p.n.q_head);
  const float mean = 1.0f / (float)r.head_dim;
  float dw[kAnyValues] = {};
  for (int t = blockIdx.x; t < r.tokens; t += gridDim.x) {
    const uint16_t* x = in.p + (long long)t * in.token + hh.h * in.head;
    const uint16_t* y = dy.p + (long long)t * dy.token + hh.h * dy.head;
    float f[kAnyValues], sq = 0.0f, dot = 0.0f;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAnyValues; ++k) {
      const int i = lane + 32 * k;
      f[k] = i < r.head_dim ? T::to_f32(x[i]) : 0.0f;
      if (i < r.head_dim) row[warp][i] = T::to_f32(y[i]);
      sq = fmaf(f[k], f[k], sq);
    }
    __syncwarp();
    float u[kAnyValues], h[kAnyValues];
#pragma unroll
    for (int k = 0; k < kAnyValues; ++k) {
      const int i = lane + 32 * k;
      u[k] = h[k] = 0.0f;
      if (i < r.head_dim) {
        u[k] = turned_any(r.r, r.positions[t], row[warp], i);
        h[k] = u[k] * weight_any<T>(w, wh + i, p.n.wide, p.n.offset);
      }
      dot = fmaf(h[k], f[k], dot);
    }
    sq = group_sum(sq, 32);
    dot = group_sum(dot, 32);
    const float n = rsqrtf(fmaf(sq, mean, p.n.eps)), c = dot * mean * n * n;
    uint16_t* out = dx.p + (long long)t * dx.token + hh.h * dx.head;
#pragma unroll
    for (int k = 0; k < kAnyValues; ++k) {
      const int i = lane + 32 * k;
      dw[k] = fmaf(u[k], f[k] * n, dw[k]);
      if (i < r.head_dim) out[i] = T::from_f32(n * fmaf(-c, f[k], h[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < kAnyValues; ++k)
    if (lane + 32 * k < r.head_dim)
      g.parts[((long long)blockIdx.x * heads + hd) * r.head_dim + lane + 32 * k] = dw[k];
}

constexpr int kAddRows = 16;

// dw of the queries' and the keys' weights: outputs [0, n_q) and [n_q, n_q + n_k); the
// sums of `outer` CTAs, `rows` rows each; a weight's are rows [row0, row0 + inner).
struct AddParams {
  const float* parts;
  float *dw_q, *dw_k;
  int d, outer, rows;
  int weights_q, weights_k, inner_q, inner_k;
  // rows of the CTAs' heads where each has its own: head = group * per + row
  int per, groups, heads_q;
};
__global__ void __launch_bounds__(32 * kAddRows) norm_grad_add_kernel(const AddParams a) {
  __shared__ float part[kAddRows][32];
  wait_prior_launch();
  let_next_launch();
  const int n_q = a.weights_q * a.d, i = blockIdx.x * 32 + threadIdx.x;
  const bool on = i < n_q + a.weights_k * a.d, key = i >= n_q;
  float sum = 0.0f;
  if (on) {
    const int j = key ? i - n_q : i, w = j / a.d, v = j - w * a.d;
    // the weight's rows, one behind the other; CTAs dealt out over threadIdx.y
    const int h0 = a.per ? (key ? a.heads_q : 0) + w : (key ? 1 : 0);
    const int inner = key ? a.inner_k : a.inner_q;
    const long long stride = (long long)a.rows * (a.per ? a.groups : 1) * a.d;
    for (int h = h0; h < h0 + inner; ++h) {
      const int at = a.per ? h / a.per * a.rows + h % a.per : h;
      const float* from = a.parts + (long long)at * a.d + v;
#pragma unroll 4
      for (int o = threadIdx.y; o < a.outer; o += kAddRows) sum += from[o * stride];
    }
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && on) {
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kAddRows; ++k) sum += part[k][threadIdx.x];
    (key ? a.dw_k : a.dw_q)[key ? i - n_q : i] = sum;
  }
}

template <typename T, bool IL>
cudaError_t launch_grad_fast(const NormGradParams& g, const NormGradPlan& n, cudaStream_t s) {
  const RopeParams& r = g.p.r;
  const Units u = units_of_head(r.head_dim, r.r.rot);
  const int shared = (!r.hq || g.p.n.q_head == 0) && (!r.hk || g.p.n.k_head == 0);
  const int table = 2 * kTables * n.z * (r.r.rot / 2), sums = n.rows * n.z * r.head_dim;
  cudaError_t e = launch_after(norm_grad_kernel<T, IL>, dim3(n.parts, n.groups),
                               dim3(u.lanes, n.rows, n.z),
                               (table > sums ? table : sums) * (int)sizeof(float), s, g, u.count,
                               u.turned, shared);
  return e;
}

}  // namespace

cudaError_t launch_norm_rope(const NormParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_ATTN_BF16 ? launch_t<Bf16>(p, s) : launch_t<Fp16>(p, s);
}

// Heads of a CTA and tokens side by side, up to kGradThreads; CTAs along the tokens
// until every SM has three.
NormGradPlan norm_grad_plan(int tokens, int heads, int lanes) {
  NormGradPlan n;
  const int most = kGradThreads / lanes;
  n.groups = (heads + most - 1) / most;
  n.rows = (heads + n.groups - 1) / n.groups;
  n.groups = (heads + n.rows - 1) / n.rows;
  n.z = 1;
  while (lanes < 32 * kAnyWarps && 2 * n.z * n.rows * lanes <= kGradThreads && n.z < 8) n.z *= 2;
  const int want = (3 * kSms + n.groups - 1) / n.groups, all = (tokens + n.z - 1) / n.z;
  n.parts = want < all ? want : all;
  return n;
}

size_t norm_grad_bytes(int tokens, int heads, int head_dim) {
  size_t most = 0;
  for (int lanes = 1; lanes <= 32; lanes *= 2) {
    const NormGradPlan n = norm_grad_plan(tokens, heads, lanes);
    const size_t rows = (size_t)n.parts * n.groups * (n.rows > 2 ? n.rows : 2);
    most = rows > most ? rows : most;
  }
  return most * head_dim * sizeof(float);
}

cudaError_t launch_norm_rope_grad(const NormGradParams& g, int dtype, cudaStream_t s) {
  const NormParams& p = g.p;
  const RopeParams& r = p.r;
  const int heads = r.hq + r.hk;
  const bool fast = fits(p) && rows_aligned(g.dq) && rows_aligned(g.dk);
  const bool each_q = r.hq && p.n.q_head, each_k = r.hk && p.n.k_head;
  const bool shared = !each_q && !each_k;
  AddParams a{};
  a.parts = g.parts;
  a.dw_q = g.dw_q;
  a.dw_k = g.dw_k;
  a.d = r.head_dim;
  a.weights_q = r.hq ? (each_q ? r.hq : 1) : 0;
  a.weights_k = r.hk ? (each_k ? r.hk : 1) : 0;
  a.inner_q = each_q ? 1 : r.hq;
  a.inner_k = each_k ? 1 : r.hk;
  a.heads_q = r.hq;
  cudaError_t e;
  if (fast) {
    const int lanes = units_of_head(r.head_dim, r.r.rot).lanes;
    const NormGradPlan n = norm_grad_plan(r.tokens, heads, lanes);
    if (shared) {  // two rows a CTA, of the queries and of the keys
      a.outer = n.parts * n.groups;
      a.rows = 2;
      a.inner_q = a.inner_k = 1;
    } else {
      a.outer = n.parts;
      a.rows = a.per = n.rows;
      a.groups = n.groups;
    }
    if (dtype == MOE_ATTN_BF16)
      e = r.r.interleaved ? launch_grad_fast<Bf16, true>(g, n, s)
                          : launch_grad_fast<Bf16, false>(g, n, s);
    else
      e = r.r.interleaved ? launch_grad_fast<Fp16, true>(g, n, s)
                          : launch_grad_fast<Fp16, false>(g, n, s);
  } else {
    const NormGradPlan n = norm_grad_plan(r.tokens, heads, 32);
    a.outer = n.parts;
    a.rows = a.per = heads;
    a.groups = 1;
    const dim3 grid(n.parts, (heads + kAnyWarps - 1) / kAnyWarps), block(kAnyWarps * 32);
    e = dtype == MOE_ATTN_BF16 ? launch_after(norm_grad_any_kernel<Bf16>, grid, block, 0, s, g)
                               : launch_after(norm_grad_any_kernel<Fp16>, grid, block, 0, s, g);
  }
  if (e != cudaSuccess) return e;
  const int outputs = (a.weights_q + a.weights_k) * a.d;
  return launch_after(norm_grad_add_kernel, dim3((outputs + 31) / 32), dim3(32, kAddRows), 0, s, a);
}

}  // namespace attn
}  // namespace moe
