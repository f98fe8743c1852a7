// What api_fp8.cu needs of the 8-bit cache's kernels, without a GPU: launches that are noted instead of run. Linked with api.cu's and
// api_fp8.cu's objects and fake_device.cpp into a library of its own for the host tests.
#include <cuda_runtime.h>

#include <cstring>

#include "internal.cuh"

namespace {
struct Launch {
  uint64_t counters, counters_end, scratch, scratch_end;  // words that a call needs at zero; what it writes besides
};
Launch g_last;
int g_set[64][2];  // attributes set, by device: decode, evict
int g_failing = -1, g_parts, g_kernel, g_weights;
uint64_t at(const void* p) { return reinterpret_cast<uint64_t>(p); }
int device() {
  int d = 0;
  cudaGetDevice(&d);
  return d;
}
cudaError_t set(int what) {
  ++g_set[device()][what];
  return device() == g_failing ? cudaErrorInvalidValue : cudaSuccess;
}
}  // namespace

extern "C" {
void fake_fp8_failing(int d) { g_failing = d; }
int fake_fp8_set(int d, int what) { return g_set[d][what]; }
void fake_fp8_last(uint64_t* out) { std::memcpy(out, &g_last, sizeof(g_last)); }
int fake_fp8_parts() { return g_parts; }      // of a unit in the last call of little work
int fake_fp8_kernel() { return g_kernel; }    // 1: little work, 2: the other one
int fake_fp8_weights() { return g_weights; }  // launches of the weights' kernel so far
}

namespace ea {
cudaError_t fp8_decode_set_attributes() { return set(0); }
cudaError_t fp8_decode_small_set_attributes() { return set(0); }
cudaError_t fp8_evict_set_attributes() { return set(1); }
cudaError_t launch_fp8_rows(const F8RowsParams&, int, int, bool, cudaLaunchConfig_t) { return cudaSuccess; }

static void note(const uint32_t* cnt, const float* lse, const float* part_ml, size_t slots, const float* scores, size_t keys) {
  g_last = {at(cnt), at(cnt + kDecodeMaxLayers * kHkv), at(lse), at(part_ml + slots * kRepText * 2)};
  if (scores != nullptr) g_last.scratch_end = at(scores + keys * kRepText);
}
template <int CAP>
cudaError_t launch_fp8_decode(const F8DecodeParams<CAP>& p, cudaLaunchConfig_t cfg) {
  g_kernel = 2;
  note(p.unit_cnt, p.lse, p.part_ml, static_cast<size_t>(cfg.gridDim.x) * 2, p.scores, static_cast<size_t>(p.W) * kKeyTile);
  return cudaSuccess;
}
template cudaError_t launch_fp8_decode(const F8DecodeParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode(const F8DecodeParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);
template <int CAP>
cudaError_t launch_fp8_decode_small(const F8SmallParams<CAP>& p, cudaLaunchConfig_t) {
  g_kernel = 1;
  g_parts = p.parts;
  const size_t units = static_cast<size_t>(p.n_layers) * kHkv;
  note(p.unit_cnt, p.lse, p.part_ml, p.parts > 1 ? units * p.parts : 0, p.scores, units * p.T * kKeyTile);
  return cudaSuccess;
}
template cudaError_t launch_fp8_decode_small(const F8SmallParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode_small(const F8SmallParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);
cudaError_t launch_fp8_weights(const F8WeightsParams&, cudaLaunchConfig_t) {
  ++g_weights;
  return cudaSuccess;
}
cudaError_t launch_fp8_evict(F8EvictParams& p, int, cudaLaunchConfig_t) {
  g_last = {at(p.status), at(p.status + 1), at(p.ticket), at(p.loaded + static_cast<size_t>(p.n_layers) * kHkv * p.blocks)};
  return cudaSuccess;
}
}  // namespace ea
