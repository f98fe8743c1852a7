// mxfp4.cu — the 4-bit cache's writer and reader.
//
// Writer: rows [row0, row0 + n) of K and V, as they come (bf16, fp16 or fp32; any head and row
// strides), become E2M1 codes and scale bytes in the same rows of the cache. Reader: the same rows as
// numbers. Both are one pass over the data, bound by HBM: 16 threads take a row, 8 channels each.
// 16 layers x 4700 rows in bf16 (390 MB a call): written in 60 us (6.4 TB/s; the encoder's instructions come close
// behind, 75 % of the issue slots), read in 58.6 us (6.65 TB/s, 98 % of a plain copy); in fp32 written in 98.8 us, read in
// 145 (71 %: a thread's 32 bytes are two stores of 16, each of which fills half of its sectors). 64 layers x 1 row, written
// and read back: 3.1 us, two launches.
#include <type_traits>

#include "mxfp4.cuh"
#include "rope.cuh"

namespace ea {
namespace mx {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;  // (write, 16 layers x 4700 rows: 137 us with 1, 124 with 2, 131 with 4)
constexpr int kRowStep = kThreads / 16;           // rows side by side in a CTA
constexpr int kRowsPerCta = kUnroll * kRowStep;

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    if constexpr (std::is_same<T, __half>::value) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_f16x2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
      unpack_bf16x8(v, x);
    }
  }
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = pack8(x, std::is_same<T, __half>::value);
  }
}

}  // namespace mx

// grid (row blocks, kv heads, layers); thread = 8 channels of kUnroll rows of K, then of V: the rows' loads go out
// together, so that a thread has kUnroll of them in flight.
template <class T>
__global__ void __launch_bounds__(mx::kThreads) mxfp4_write_kernel(const __grid_constant__ MxRowsParams p) {
  using namespace mx;
  const int c = threadIdx.x & 15;
  const int r0 = blockIdx.x * kRowsPerCta + (threadIdx.x >> 4);
  const int g = blockIdx.y;
  const MxRowsLayer& L = p.layer[blockIdx.z];
  pdl_wait_primary();
  pdl_launch_dependents();
  if ((r0 & ~1) >= p.n_rows) return;  // the warp's first row
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = static_cast<const T*>(kv ? L.v : L.k) + g * p.head_stride + 8 * c;
    uint8_t* codes = kv ? L.vc : L.kc;
    uint8_t* scales = kv ? L.vs : L.ks;
    float x[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {  // a row past the end repeats the last one: its threads shuffle along
      const int r = min(r0 + u * kRowStep, p.n_rows - 1);
      load8(src + r * p.row_stride, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      auto block_max = [&] {
        const float a = mx_amax8<true>(x[u]), b = mx_max<true>(a, __shfl_xor_sync(0xffffffffu, a, 1));
        return mx_max<true>(b, __shfl_xor_sync(0xffffffffu, b, 2));
      };
      float amax = block_max();
      if (__any_sync(0xffffffffu, amax != amax)) {
        mx_clean8(x[u]);
        amax = block_max();
      }
      const int e = mx_exponent(amax);
      const uint32_t w = mx_pack8<true>(x[u], mx_pow2(-e));
      // the row's four scale bytes (lanes 0, 4, 8, 12 of its 16) in one word
      uint32_t sc = static_cast<uint32_t>(e + 127) << (8 * (c >> 2));
      sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
      sc |= __shfl_xor_sync(0xffffffffu, sc, 8);
      const int r = r0 + u * kRowStep;
      if (r < p.n_rows) {
        const size_t row = static_cast<size_t>(g) * p.Smax + p.row0 + r;
        *reinterpret_cast<uint32_t*>(codes + row * kMxRowBytes + 4 * c) = w;
        if (c == 0) *reinterpret_cast<uint32_t*>(scales + row * kMxRowScales) = sc;
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(mx::kThreads) mxfp4_read_kernel(const __grid_constant__ MxRowsParams p) {
  using namespace mx;
  const int c = threadIdx.x & 15;
  const int r0 = blockIdx.x * kRowsPerCta + (threadIdx.x >> 4);
  const int g = blockIdx.y;
  const MxRowsLayer& L = p.layer[blockIdx.z];
  pdl_wait_primary();
  pdl_launch_dependents();
  if (r0 >= p.n_rows) return;
  uint32_t w[2][kUnroll], b[2][kUnroll];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const size_t row = static_cast<size_t>(g) * p.Smax + p.row0 + min(r0 + u * kRowStep, p.n_rows - 1);
      w[kv][u] = *reinterpret_cast<const uint32_t*>((kv ? L.vc : L.kc) + row * kMxRowBytes + 4 * c);
      b[kv][u] = (kv ? L.vs : L.ks)[row * kMxRowScales + (c >> 2)];
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* dst = static_cast<T*>(kv ? L.v : L.k) + g * p.head_stride + 8 * c;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kRowStep;
      float x[8];
      mx_values8(w[kv][u], mx_scale(b[kv][u]), x);
      if (r < p.n_rows) store8(dst + r * p.row_stride, x);
    }
  }
}

cudaError_t launch_mxfp4_rows(const MxRowsParams& p, int n_layers, int dtype, bool write, cudaLaunchConfig_t cfg) {
  cfg.gridDim = dim3((p.n_rows + mx::kRowsPerCta - 1) / mx::kRowsPerCta, kHkv, n_layers);
  cfg.blockDim = dim3(mx::kThreads);
  if (dtype == 0)
    return cudaLaunchKernelEx(&cfg, write ? mxfp4_write_kernel<__nv_bfloat16> : mxfp4_read_kernel<__nv_bfloat16>, p);
  if (dtype == 1) return cudaLaunchKernelEx(&cfg, write ? mxfp4_write_kernel<__half> : mxfp4_read_kernel<__half>, p);
  return cudaLaunchKernelEx(&cfg, write ? mxfp4_write_kernel<float> : mxfp4_read_kernel<float>, p);
}

}  // namespace ea
