// A CUDA runtime for the host side of the attention operators (csrc/attn.cu): two
// devices without a GPU, device memory on the host, every call on record, and
// errors on demand. Kernels are not run; fake_launches.cu records their launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

namespace {
std::string calls, failing;
int device = 0;

void record(const char* what) {
  calls += what;
  calls += ';';
}
cudaError_t done(const char* what) {
  record(what);
  return failing == what ? cudaErrorUnknown : cudaSuccess;
}
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

// a launch or a set-up call of fake_launches.cu
cudaError_t fake_call(const char* what, bool with_device) {
  record(with_device ? (std::string(what) + " on " + std::to_string(device)).c_str() : what);
  return failing == what ? cudaErrorUnknown : cudaSuccess;
}

extern "C" {
const char* fake_calls() { return calls.c_str(); }
void fake_reset() { calls.clear(), failing.clear(); }
void fake_fail(const char* what) { failing = what; }
int fake_device() { return device; }
void fake_use(int d) { device = d; }

cudaError_t cudaGetDeviceCount(int* n) { return *n = 2, cudaSuccess; }
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
  memset(p, 0, sizeof *p);
  p->major = 10, p->minor = 3, p->multiProcessorCount = 152;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaSetDevice(int d) {
  device = d;
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() { return done("sync"); }
cudaError_t cudaMalloc(void** p, size_t n) {
  if (failing == "malloc") return done("malloc");
  *p = malloc(n);
  memset(*p, 0xab, n);
  return done("malloc");
}
cudaError_t cudaFree(void* p) {
  free(p);
  return done("free");
}
cudaError_t cudaMemset(void* p, int v, size_t n) {
  if (failing == "memset") return done("memset");
  memset(p, v, n);
  return done("memset");
}
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) {
  memcpy(d, s, n);
  return done("memcpy");
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "an error of the stand-in"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}
