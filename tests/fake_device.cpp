// What api.cu needs of the CUDA runtime and of the kernels' files, without a GPU: devices that only exist as numbers, and
// launches that are noted instead of run. Linked with api.cu's object into a library of its own for the host tests.
#include <cuda_runtime.h>

#include <cstring>

#include "internal.cuh"

namespace {
int g_device = 0, g_failing = -1;
unsigned g_parts;  // of a unit, at most, in the last decode step over a 4-bit cache
int g_sms = 152;
int g_set[64][5];  // attributes set, by device: attention, prologue, linear, decode, 4-bit (its decode step and attention)
struct Launch {
  uint64_t counters, counters_end, scratch, scratch_end;  // words that a call needs at zero; what it writes besides
};
Launch g_last;
cudaError_t set(int what) {
  ++g_set[g_device][what];
  return g_device == g_failing ? cudaErrorInvalidValue : cudaSuccess;
}
uint64_t at(const void* p) { return reinterpret_cast<uint64_t>(p); }
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
void fake_device(int d, int failing) {
  g_device = d;
  g_failing = failing;
}
int fake_set(int d, int what) { return g_set[d][what]; }
void fake_sms(int n) { g_sms = n; }
int fake_parts() { return static_cast<int>(g_parts); }
void fake_last(uint64_t* out) { std::memcpy(out, &g_last, sizeof(g_last)); }

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : g_sms;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void**, const void*) { return cudaErrorInvalidSymbol; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *f = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 0; }
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
}

namespace ea {
cudaError_t attention_set_attributes() { return set(0); }
cudaError_t prologue_set_attributes() { return set(1); }
cudaError_t linear_set_attributes() { return set(2); }
cudaError_t decode_set_attributes() { return set(3); }
cudaError_t mxfp4_decode_set_attributes() { return set(4); }
cudaError_t mxfp4_attention_set_attributes() { return set(4); }

cudaError_t launch_linear(const LinearParams&, int, int, cudaLaunchConfig_t) { return cudaSuccess; }
cudaError_t launch_quantize_mxfp4(const __nv_bfloat16*, uint8_t*, uint8_t*, int, int, cudaStream_t) { return cudaSuccess; }
void quantize_cache_kernel(const __nv_bfloat16*, uint8_t*, float*, int, int) {}
template <int CAP>
cudaError_t launch_prologue_kernel(const PrologueParams<CAP>&, bool, int, cudaLaunchConfig_t) {
  return cudaSuccess;
}
template cudaError_t launch_prologue_kernel(const PrologueParams<kSmallCap>&, bool, int, cudaLaunchConfig_t);
template cudaError_t launch_prologue_kernel(const PrologueParams<kMaxLayersPerLaunch>&, bool, int, cudaLaunchConfig_t);
template <int CAP>
cudaError_t launch_attention_kernel(const AttnParams<CAP>& p, bool f8, cudaLaunchConfig_t cfg) {
  g_last = {at(p.unit_sync), at(p.unit_sync + 2 * (p.W / p.T)), f8 ? at(p.q_scale) : at(p.part_o),
            at(p.part_lse + static_cast<size_t>(cfg.gridDim.x) * 6 * kRows)};
  return cudaSuccess;
}
template cudaError_t launch_attention_kernel(const AttnParams<kSmallCap>&, bool, cudaLaunchConfig_t);
template cudaError_t launch_attention_kernel(const AttnParams<kMaxLayersPerLaunch>&, bool, cudaLaunchConfig_t);
template <int CAP>
cudaError_t launch_decode_kernel(const DecodeParams<CAP>& p, cudaLaunchConfig_t cfg) {
  g_last = {at(p.unit_cnt), at(p.unit_cnt + p.W / p.T), at(p.part_o), at(p.part_ml + static_cast<size_t>(cfg.gridDim.x) * 4 * kRepText)};
  return cudaSuccess;
}
template cudaError_t launch_decode_kernel(const DecodeParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_decode_kernel(const DecodeParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);
cudaError_t launch_mxfp4_rows(const MxRowsParams&, int, int, bool, cudaLaunchConfig_t) { return cudaSuccess; }
cudaError_t launch_mxfp4_prologue(const MxPrologueParams&, int, cudaLaunchConfig_t) { return cudaSuccess; }
cudaError_t launch_mxfp4_attention(const MxExpertParams&, cudaLaunchConfig_t) { return cudaSuccess; }
cudaError_t launch_mxfp4_merge(const MxMergeParams&, int, cudaLaunchConfig_t) { return cudaSuccess; }
cudaError_t launch_mxfp4_decode(const MxDecodeParams& p, cudaLaunchConfig_t cfg) {
  // the parts that the kernel will count, from the ranges' starts
  auto start = [&](uint32_t c) {
    return p.parts > 0 ? c / p.parts * p.T + c % p.parts * p.T / p.parts : c * p.per_cta + (c < p.extra ? c : p.extra);
  };
  g_parts = 0;
  uint32_t unit = 0, n = 0;
  for (uint32_t c = 0; c < cfg.gridDim.x; ++c) {
    for (uint32_t u = start(c) / p.T; u <= (start(c + 1) - 1) / p.T; ++u, ++n) {
      if (u != unit) n = 0;
      unit = u;
      g_parts = n + 1 > g_parts ? n + 1 : g_parts;
    }
  }
  g_last = {at(p.unit_cnt), at(p.unit_cnt + kMaxLayersPerLaunch * kHkv), at(p.part_o),
            at(p.part_lse + static_cast<size_t>(cfg.gridDim.x) * 2 * kRepText)};
  return cudaSuccess;
}
}  // namespace ea
