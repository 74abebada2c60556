// Device helpers shared by the attention kernels.
#pragma once

#include "attn.h"
#include "tc_common.cuh"

namespace moe {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tc::bwait for what another role of the CTA does only once a piece of its work,
// which may take seconds over hundreds of millions of keys; the waits inside a
// piece keep the short limit.
__device__ __forceinline__ bool bwait_piece(uint64_t* bar, uint32_t parity, unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if ((i & 15u) == 0) {
      if (tc::aborted(err)) return false;
      if (global_ns() - t0 > 30 * kWaitLimitNs) {
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
}

// Waits until the launch before this one is complete and its writes are visible.
__device__ __forceinline__ void wait_prior_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next launch's CTAs start where there is room; they wait as above.
__device__ __forceinline__ void let_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// one box of a page: rows from `row`, values from `c0`, of a kv head
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                         int c0, int row, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(row), "r"(head),
      "r"(page)
      : "memory");
}

// What a kernel is compiled for: plain scores; scores with a bias or a cap of
// ordinary size, 1 - 2 / (1 + e^2y) with an error of 1.3e-7 of the cap; scores under
// a cap above kWideCap, of which that would be more than scores may be off, by
// tanh_of. (tanh_of for all: a prompt of 8192 tokens near its cap 823 -> 1112 us,
// decode of 64 sequences under a cap of 50 358 -> 400 us.)
enum Form { kPlain, kGeneral, kWide };
constexpr float kWideCap = 64.0f;
inline Form form_of(const Scores& s) {
  return s.softcap > kWideCap ? kWide : s.softcap > 0.0f || s.slopes ? kGeneral : kPlain;
}

// tanh(y), to 4e-7 of itself at any size of y: y P(y^2) / Q(y^2) for |y| < 9.02,
// where it is 1 - 3e-8, a fit of tanh(y) / y with the least relative error (2.1e-8).
// All coefficients are positive, so nothing cancels.
constexpr float kTanhEnd = 9.02f;
__device__ constexpr float kTanhP[5] = {0.999999979f, 0.1337970922f, 0.003494024105f,
                                        2.058330581e-05f, 1.331882452e-08f};
__device__ constexpr float kTanhQ[5] = {1.0f, 0.4671302446f, 0.02587103368f, 0.0003283075583f,
                                        7.761918968e-07f};
__device__ __forceinline__ float tanh_range(float y) {  // keeps a NaN
  float r;
  asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, %2;\n min.NaN.f32 %0, t, %3;\n}\n"
      : "=f"(r)
      : "f"(y), "f"(-kTanhEnd), "f"(kTanhEnd));
  return r;
}
__device__ __forceinline__ float tanh_of(float y) {
  y = tanh_range(y);
  const float t = y * y;
  float a = kTanhP[4], b = kTanhQ[4];
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    a = fmaf(a, t, kTanhP[k]);
    b = fmaf(b, t, kTanhQ[k]);
  }
  return a * y * rcp(b);
}

// log2-space score of a product
template <int FORM>
__device__ __forceinline__ float score(const Scores& sc, float dot, float slope, int away) {
  if (FORM == kPlain) return dot * (sc.scale * kLog2e);
  float x = dot * sc.scale;
  if (FORM == kWide) {
    x = sc.softcap * tanh_of(dot * sc.cap_in);
  } else if (sc.softcap > 0.0f) {
    // tanh(y) = 1 - 2 / (1 + e^2y): absolute error of a few 2^-24
    const float e = ex2(dot * (2.0f * kLog2e * sc.cap_in));
    x = sc.softcap * (1.0f - __fdividef(2.0f, 1.0f + e));
  }
  return (x - slope * (float)abs(away)) * kLog2e;
}

// A launch that may begin while the one before it ends: every kernel launched so
// waits (wait_prior_launch) before it reads or writes memory.
template <typename... A, typename... B>
inline cudaError_t launch_after(void (*f)(A...), dim3 grid, dim3 block, int smem, cudaStream_t s,
                         B... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}

}  // namespace attn
}  // namespace moe
