// The attention kernels' launches for tests of their host side: recorded, not run
// (see fake_cudart.cpp).
#include "attn.h"

cudaError_t fake_call(const char* what, bool with_device);

static void* counters[2];  // what the last launches of either kernel got

extern "C" void* fake_counters(int kernel) { return counters[kernel]; }
extern "C" int fake_counter_words(int kernel) { return moe::attn::kMaxGrid * (kernel ? 4 : 1); }

namespace moe {
namespace attn {
cudaError_t launch_rope(const RopeParams&, int, cudaStream_t) { return fake_call("rope", true); }
cudaError_t attn_decode_setup() { return fake_call("decode setup", false); }
cudaError_t attn_tc_setup(bool* usable) {
  *usable = fake_call("tc usable", false) == cudaSuccess;
  return fake_call("tc setup", false);
}
cudaError_t launch_attn_decode(const AttnParams&, const Partials& w, const CUtensorMap&,
                               const CUtensorMap&, int, int, cudaStream_t) {
  counters[0] = w.count;
  return fake_call("decode", true);
}
cudaError_t launch_attn_tc(const AttnParams&, const TcPieces& w, const CUtensorMap&,
                           const CUtensorMap&, const CUtensorMap&, int, int, cudaStream_t) {
  counters[1] = w.count;
  return fake_call("tc", true);
}
}  // namespace attn
}  // namespace moe
