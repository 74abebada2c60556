// The launches of include/moe_attn8.h for tests of their host side: recorded, not run
// (see fake_cudart.cpp).
#include "attn.h"

cudaError_t fake_call(const char* what, bool with_device);

namespace moe {
namespace attn {
cudaError_t launch_norm_rope(const NormParams&, int, cudaStream_t) { return fake_call("norm", true); }
size_t norm_grad_bytes(int, int, int) { return 16; }
cudaError_t launch_norm_rope_grad(const NormGradParams&, int, cudaStream_t) {
  return fake_call("gradient", true);
}
cudaError_t launch_append8(const Append8Params&, int, cudaStream_t) {
  return fake_call("append8", true);
}
cudaError_t launch_read8(const Read8Params&, int, cudaStream_t) { return fake_call("read8", true); }
cudaError_t launch_expand8(const Expand8Params&, int, int, cudaStream_t) {
  return fake_call("expand8", true);
}
cudaError_t attn8_decode_setup() { return fake_call("decode8 setup", false); }
cudaError_t attn8_tc_setup(bool* usable) {
  *usable = fake_call("tc8 usable", false) == cudaSuccess;
  return fake_call("tc8 setup", false);
}
cudaError_t launch_attn8_decode(const Attn8Params&, const Partials&, const CUtensorMap&,
                                const CUtensorMap&, int, cudaStream_t) {
  return fake_call("decode8", true);
}
cudaError_t launch_attn8_tc(const Attn8Params&, const TcPieces&, const CUtensorMap&,
                            const CUtensorMap&, const CUtensorMap&, int, cudaStream_t) {
  return fake_call("tc8", true);
}
}  // namespace attn
}  // namespace moe
