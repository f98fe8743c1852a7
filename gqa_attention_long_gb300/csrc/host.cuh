// host.cuh — what the host side's files share: the device's description, once-per-device set-up, cached tensor maps, launch
// attributes, the check that a call's outputs are all different, and a position's rotations in 64 bits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <array>
#include <cmath>
#include <mutex>

#include "internal.cuh"

namespace ea {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool init = false;
  bool ok = false;
  int sm_count = 0;
};

// What a kernel's attributes need: done once for each device (they hold for the current device alone), and again where it
// failed.
class OncePerDevice {
 public:
  template <class Set>
  bool operator()(int dev, Set set) {
    std::lock_guard<std::mutex> lk(mu_);
    if (!done_[dev]) done_[dev] = set();
    return done_[dev];
  }

 private:
  std::mutex mu_;
  bool done_[kMaxDevices] = {};
};

// The current device, if it is an sm_103 part (see api.cu).
bool device_info(int* dev_out, DeviceInfo* info);
// A cache's tensor map: see api.cu.
bool cache_map(const void* base, int S, int Smax, bool f8, CUtensorMap* out);
cudaLaunchConfig_t launch_config(cudaStream_t st, cudaLaunchAttribute* attr, bool pdl);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct MxNone {
  template <class A>
  std::array<const void*, 0> operator()(const A&) const {
    return {};
  }
};
// Whether the arrays that one call writes, writes(a[l])[0 .. N) of every layer, are all different (what stands twice
// would be written twice, in any order), and none of those that it only reads, reads(a[l]), is among them (which may stand in several
// layers). Null entries (outputs that are not asked for) are passed over.
template <int N, class A, class Writes, class Reads = MxNone>
bool mx_distinct(const A* a, int n, Writes writes, Reads reads = {}) {
  constexpr int kBits = N <= 4 ? 9 : N <= 8 ? 10 : 11;
  constexpr uint32_t kSlots = 1u << kBits;
  static_assert(N * kMaxLayersPerLaunch <= kSlots / 2, "table");
  for (int l0 = 0; l0 < n; l0 += kMaxLayersPerLaunch) {
    const void* seen[kSlots] = {};
    auto find = [&](const void* p) {  // p's place, or the free one where it belongs
      uint32_t h = static_cast<uint32_t>((reinterpret_cast<uintptr_t>(p) >> 4) * 0x9E3779B97F4A7C15ull >> (64 - kBits));
      while (seen[h] != nullptr && seen[h] != p) h = (h + 1) % kSlots;
      return h;
    };
    const int l1 = l0 + kMaxLayersPerLaunch < n ? l0 + kMaxLayersPerLaunch : n;
    for (int l = l0; l < n; ++l)  // 64 layers into the table, the later ones against it
      for (const void* p : writes(a[l])) {
        if (p == nullptr) continue;
        const uint32_t h = find(p);
        if (seen[h] != nullptr) return false;
        if (l < l1) seen[h] = p;
      }
    for (int l = 0; l < n; ++l)
      for (const void* p : reads(a[l]))
        if (p != nullptr && seen[find(p)] != nullptr) return false;
  }
  return true;
}

// Cosines and sines of pos * 5e6^(-j/64), |pos| < 2^24, in 64 bits (a far position's angle needs them): the product of
// four rotations, by the position's base-64 digits, from a table that is formed once per process (64 library
// sines and cosines would be half of a small call's time on the host).
class MxRotations {
 public:
  struct Cis {
    double c, s;
  };
  static const MxRotations& get() {
    static const MxRotations r;
    return r;
  }
  Cis at(long long pos, int j) const {
    const uint32_t a = static_cast<uint32_t>(pos < 0 ? -pos : pos);
    Cis r = t_[0][a & 63][j];
    for (int d = 1; d < 4; ++d)
      if (const uint32_t k = (a >> (6 * d)) & 63) r = mul(r, t_[d][k][j]);
    if (pos < 0) r.s = -r.s;
    return r;
  }
  static Cis mul(const Cis& a, const Cis& b) { return {a.c * b.c - a.s * b.s, a.s * b.c + a.c * b.s}; }
  // as fp32 pairs: cosine x + y, sine z + w
  static float4 split(const Cis& a) {
    const float c = static_cast<float>(a.c), s = static_cast<float>(a.s);
    return make_float4(c, static_cast<float>(a.c - c), s, static_cast<float>(a.s - s));
  }

 private:
  MxRotations() {
    for (int j = 0; j < kD / 2; ++j) {
      const double f = std::pow(5.0e6, -static_cast<double>(j) / (kD / 2));
      for (int d = 0; d < 4; ++d)
        for (int k = 0; k < 64; ++k) {
          const double x = std::ldexp(static_cast<double>(k), 6 * d) * f;
          t_[d][k][j] = {std::cos(x), std::sin(x)};
        }
    }
  }
  Cis t_[4][64][kD / 2];
};

}  // namespace ea
