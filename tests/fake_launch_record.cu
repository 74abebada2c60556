// A CUDA runtime that records launches in place of running them, and calls of the
// launching functions in csrc/norm_rope.cu and csrc/cache8.cu, for tests of what they ask
// for. No GPU takes part.
#include <cstdio>
#include <map>
#include <string>

#include "attn.h"

// (made by the first kernel that is registered, before this file's own variables)
static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static std::string launches;  // "name grid.x grid.y block.x block.y block.z bytes;" each

using namespace moe;
using namespace moe::attn;

static Rows rows(int heads, int dim) {
  static uint16_t* const p = reinterpret_cast<uint16_t*>(1 << 20);
  return Rows{p, (long long)heads * dim, dim};
}
static NormParams params(int tokens, int hq, int hk, int dim, int rot, int interleaved) {
  NormParams p{};
  p.r.q = p.r.q_out = hq ? rows(hq, dim) : Rows{};
  p.r.k = p.r.v = p.k_out = hk ? rows(hk, dim) : Rows{};
  p.r.r = Rotation{nullptr, rot, interleaved, 1.0f, 1.0f};
  p.r.tokens = tokens, p.r.hq = hq, p.r.hk = hk, p.r.head_dim = dim;
  p.n.on = 1;
  return p;
}

extern "C" {
const char* record_take() {
  static std::string taken;
  taken.swap(launches);
  launches.clear();
  return taken.c_str();
}
int record_append8(int tokens, int hq, int hk, int dim, int rot, int interleaved) {
  Append8Params g{};
  g.p = params(tokens, hq, hk, dim, rot, interleaved);
  g.p.r.hv = hk;
  return launch_append8(g, MOE_ATTN_BF16, nullptr);
}
int record_norm(int tokens, int hq, int hk, int dim, int rot, int interleaved) {
  return launch_norm_rope(params(tokens, hq, hk, dim, rot, interleaved), MOE_ATTN_BF16, nullptr);
}
int record_append_norm(int tokens, int hq, int hk, int dim, int rot, int interleaved) {
  NormParams p = params(tokens, hq, hk, dim, rot, interleaved);
  p.r.hv = hk;
  p.r.slots = reinterpret_cast<const long long*>(64);
  return launch_norm_rope(p, MOE_ATTN_BF16, nullptr);
}
int record_gradient(int tokens, int hq, int hk, int dim, int rot, int interleaved) {
  NormGradParams g{};
  g.p = params(tokens, hq, hk, dim, rot, interleaved);
  g.dq = g.p.r.q, g.dk = g.p.r.k;
  return launch_norm_rope_grad(g, MOE_ATTN_BF16, nullptr);
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  char line[160];
  snprintf(line, sizeof line, " %u %u %u %u %u %zu;", c->gridDim.x, c->gridDim.y, c->blockDim.x,
           c->blockDim.y, c->blockDim.z, c->dynamicSmemBytes);
  launches += names().at(f) + line;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*,
                            dim3*, dim3*, int*) {
  names()[host] = name;
}
}
