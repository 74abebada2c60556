// What the attention kernels over the 8-bit cache share: codes as fp16, scales.
#pragma once

#include "attn_common.cuh"

namespace moe {
namespace attn {

// Every e4m3 code is an fp16 number: the products run in fp16, whatever the type of
// the queries and the results. (bf16 would hold them as well, but takes three more
// instructions for two codes, and keeps less of the softmax's numerators.)
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t codes, bool upper) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, %2;\n}\n"
      : "=r"(r)
      : "r"(codes), "h"((uint16_t)(upper ? codes >> 16 : codes)));
  return r;
}

// A scale of K or V, kept within what caches may have: what is 0, or no number, behind
// the last key then hurts nothing.
__device__ __forceinline__ float scale_in_range(float s) {
  return fminf(fmaxf(s, 0x1p-64f), 0x1p64f);
}
// log2 of a scale in range, exact for powers of two
__device__ __forceinline__ float log2_of_scale(float s) {
  const int bits = __float_as_int(s);
  float m;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(m) : "f"(__int_as_float((bits & 0x7fffff) | 0x3f800000)));
  return (float)((bits >> 23) - 127) + m;
}

// One thread of the converged warp, the same one every time: the compiler then knows
// that a single thread issues what follows.
__device__ __forceinline__ bool one_thread() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(p));
  return p != 0;
}

// 4 bytes from global to shared memory, or zeros where `on` is false
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 4 : 0)
               : "memory");
}
// arrives at the barrier once this thread's copies above have landed
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// The power of two that brings a row whose largest |value| is `top` to 2^14 .. 2^15, and
// its inverse: bf16 values as fp16, of which those down to 2^-32 of the largest keep
// all their bits. 1 for a row that holds what is no number.
struct RowUnit {
  float up, down;
  __device__ __forceinline__ explicit RowUnit(float top) {
    int e = 14 - ((__float_as_int(top) >> 23) - 127);
    e = top < INFINITY ? min(e, 100) : 0;
    up = __int_as_float((e + 127) << 23);
    down = __int_as_float((127 - e) << 23);
  }
};

}  // namespace attn
}  // namespace moe
