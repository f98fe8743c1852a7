// fp8.cu — the 8-bit cache's writer and reader.
//
// Writer: rows [row0, row0 + n) of K and V, as they come (bf16, fp16 or fp32; any head and row strides), are appended to
// a cache that holds rows [0, row0). One CTA takes one head's rows of one 128-row block, of K or of V: it finds their largest
// magnitude, which says what becomes of the block's scale (fp8.cuh), rounds the block's earlier rows again if that has
// moved, and encodes. Reader: rows as numbers. Both are one pass over the data, bound by HBM: 4700 bf16 rows of 16 layers (463 MB) 62 us
// written and 65 read back (the copy's rate over both is 137; some of what is written stays in L2).
#include <type_traits>

#include "fp8.cuh"
#include "rope.cuh"

namespace ea {
namespace f8 {

constexpr int kThreads = 256;
constexpr int kChunks = kScaleBlock * kD / 8 / kThreads;  // pieces of 8 channels that a thread holds of a block

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

// Eight values of a row as they come: kept so until the block's scale is known, which takes half the registers of fp32.
template <class T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { load8(reinterpret_cast<const T*>(v), x); }
};

__device__ __forceinline__ float amax8(const float (&x)[8], float amax) {  // (a NaN is passed over)
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
  return amax;
}
template <class F>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], F q) {
  return make_uint2(f8_pack4(q(x[0]), q(x[1]), q(x[2]), q(x[3])), f8_pack4(q(x[4]), q(x[5]), q(x[6]), q(x[7])));
}
// Codes of n pieces of 16 bytes times f, rounded again: kBatch of them under way in a thread.
template <int kBatch>
__device__ __forceinline__ void rescale(uint8_t* codes, int n, float f, int first, int step) {
  uint4* c = reinterpret_cast<uint4*>(codes) + first;
  for (int i = first; i < n; i += kBatch * step, c += kBatch * step) {
    uint4 w[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (i + e * step < n) w[e] = c[e * step];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      if (i + e * step < n) c[e * step] = f8_rescale16(w[e], f);
  }
}

}  // namespace f8

// grid (touched blocks, 2 * kv head + (0: K, 1: V), layers)
template <class T>
__global__ void __launch_bounds__(f8::kThreads, sizeof(T) == 2 ? 4 : 2) fp8_write_kernel(const __grid_constant__ F8RowsParams p) {
  using namespace f8;
  __shared__ float red[kThreads / 32];
  const int kv = blockIdx.y & 1, g = blockIdx.y >> 1, tid = threadIdx.x;
  const F8RowsLayer& L = p.layer[blockIdx.z];
  const int b = p.row0 / kScaleBlock + blockIdx.x;
  const int r0 = max(p.row0, b * kScaleBlock), r1 = min(p.row0 + p.n_rows, (b + 1) * kScaleBlock);
  const int before = r0 - b * kScaleBlock, n = r1 - r0;  // rows that the block holds, and that it gets
  float* scale = (kv ? L.vs : L.ks) + g * (p.Smax / kScaleBlock + 1) + b;
  const T* src = static_cast<const T*>(kv ? L.v : L.k) + g * p.head_stride + (r0 - p.row0) * p.row_stride + 8 * (tid & 15);
  uint8_t* codes = (kv ? L.vc : L.kc) + (static_cast<size_t>(g) * p.Smax + static_cast<size_t>(b) * kScaleBlock) * kD;
  pdl_wait_primary();
  pdl_launch_dependents();
  Raw8<T> raw[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = (tid >> 4) + (kThreads / 16) * i;
    if (r < n) raw[i].load(src + r * p.row_stride);
  }
  const float s = before > 0 ? *scale : f8_pow2(kF8FirstExp);
  float amax = 0.f, x[8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    if ((tid >> 4) + (kThreads / 16) * i < n) {
      raw[i].get(x);
      amax = amax8(x, amax);
    }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();  // (the scale has been read, too)
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const int k = f8_growth(amax, s);
  const float s1 = f8_grown(s, k);
  if (tid == 0 && (k > 0 || before == 0)) *scale = s1;
  if (k > 0 && before > 0) rescale<2>(codes, before * kD / 16, f8_shrink(k), tid, kThreads);
  auto encode = [&](auto q) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + kThreads * i;
      if ((c >> 4) < n) {
        raw[i].get(x);
        *reinterpret_cast<uint2*>(codes + before * kD + 8 * c) = encode8(x, q);
      }
    }
  };
  const F8Quotient q(s1);
  if (q.pow2) encode([&](float v) { return v * q.inv; });
  else encode([&](float v) { return __fdiv_rn(v, q.s); });
}

// A few rows (at most kFew, within one block or two): a warp takes one head's rows of one block, of K or of V. grid (blocks, heads and K, V in fours,
// layers)
namespace f8 {
constexpr int kFew = 4, kFewThreads = 128;
}
template <class T>
__global__ void __launch_bounds__(f8::kFewThreads) fp8_write_few_kernel(const __grid_constant__ F8RowsParams p) {
  using namespace f8;
  const int y = blockIdx.y * (kFewThreads / 32) + (threadIdx.x >> 5), kv = y & 1, g = y >> 1, lane = threadIdx.x & 31;
  const F8RowsLayer& L = p.layer[blockIdx.z];
  const int b = p.row0 / kScaleBlock + blockIdx.x;
  const int r0 = max(p.row0, b * kScaleBlock), r1 = min(p.row0 + p.n_rows, (b + 1) * kScaleBlock);
  const int before = r0 - b * kScaleBlock, n = r1 - r0;
  float* scale = (kv ? L.vs : L.ks) + g * (p.Smax / kScaleBlock + 1) + b;
  const T* src = static_cast<const T*>(kv ? L.v : L.k) + g * p.head_stride + (r0 - p.row0) * p.row_stride + 8 * (lane & 15);
  uint8_t* codes = (kv ? L.vc : L.kc) + (static_cast<size_t>(g) * p.Smax + static_cast<size_t>(b) * kScaleBlock) * kD;
  pdl_wait_primary();
  pdl_launch_dependents();
  Raw8<T> raw[kFew / 2];  // half a warp to a row
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i)
    if ((lane >> 4) + 2 * i < n) raw[i].load(src + ((lane >> 4) + 2 * i) * p.row_stride);
  const float s = before > 0 ? *scale : f8_pow2(kF8FirstExp);
  float amax = 0.f, x[8];
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i)
    if ((lane >> 4) + 2 * i < n) {
      raw[i].get(x);
      amax = amax8(x, amax);
    }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  const int k = f8_growth(amax, s);
  const float s1 = f8_grown(s, k);
  __syncwarp();  // (every lane has read the scale)
  if (lane == 0 && (k > 0 || before == 0)) *scale = s1;
  if (k > 0 && before > 0) rescale<8>(codes, before * kD / 16, f8_shrink(k), lane, 32);
  const F8Quotient q(s1);
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i)
    if ((lane >> 4) + 2 * i < n) {
      raw[i].get(x);
      *reinterpret_cast<uint2*>(codes + (before + (lane >> 4) + 2 * i) * kD + 8 * (lane & 15)) = encode8(x, q);
    }
}

// grid (row blocks, kv heads, layers); thread = 8 channels of kUnroll rows of K and of V
namespace f8 {
constexpr int kReadThreads = 128, kUnroll = 2, kRowStep = kReadThreads / 16, kRowsPerCta = kUnroll * kRowStep;
}
template <class T>
__global__ void __launch_bounds__(f8::kReadThreads) fp8_read_kernel(const __grid_constant__ F8RowsParams p) {
  using namespace f8;
  const int c = threadIdx.x & 15, r0 = blockIdx.x * kRowsPerCta + (threadIdx.x >> 4), g = blockIdx.y;
  const F8RowsLayer& L = p.layer[blockIdx.z];
  pdl_wait_primary();
  pdl_launch_dependents();
  if (r0 >= p.n_rows) return;
  uint2 w[2][kUnroll];
  float s[2][kUnroll];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int row = p.row0 + min(r0 + u * kRowStep, p.n_rows - 1);
      w[kv][u] = *reinterpret_cast<const uint2*>((kv ? L.vc : L.kc) + (static_cast<size_t>(g) * p.Smax + row) * kD + 8 * c);
      s[kv][u] = (kv ? L.vs : L.ks)[g * (p.Smax / kScaleBlock + 1) + row / kScaleBlock];
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* dst = static_cast<T*>(kv ? L.v : L.k) + g * p.head_stride + 8 * c;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kRowStep;
      float a[4], b[4], x[8];
      f8_unpack4(w[kv][u].x, a);
      f8_unpack4(w[kv][u].y, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = a[e] * s[kv][u];
        x[4 + e] = b[e] * s[kv][u];
      }
      if (r < p.n_rows) store8(dst + r * p.row_stride, x);
    }
  }
}

template <class T>
static cudaError_t launch_rows(const F8RowsParams& p, int n_layers, bool write, cudaLaunchConfig_t cfg) {
  const int blocks = (p.row0 + p.n_rows - 1) / kScaleBlock - p.row0 / kScaleBlock + 1;
  if (!write) {
    cfg.gridDim = dim3((p.n_rows + f8::kRowsPerCta - 1) / f8::kRowsPerCta, kHkv, n_layers);
    cfg.blockDim = dim3(f8::kReadThreads);
    return cudaLaunchKernelEx(&cfg, fp8_read_kernel<T>, p);
  }
  if (p.n_rows <= f8::kFew) {
    cfg.gridDim = dim3(blocks, 2 * kHkv / (f8::kFewThreads / 32), n_layers);
    cfg.blockDim = dim3(f8::kFewThreads);
    return cudaLaunchKernelEx(&cfg, fp8_write_few_kernel<T>, p);
  }
  cfg.gridDim = dim3(blocks, 2 * kHkv, n_layers);
  cfg.blockDim = dim3(f8::kThreads);
  return cudaLaunchKernelEx(&cfg, fp8_write_kernel<T>, p);
}

cudaError_t launch_fp8_rows(const F8RowsParams& p, int n_layers, int dtype, bool write, cudaLaunchConfig_t cfg) {
  if (dtype == 0) return launch_rows<__nv_bfloat16>(p, n_layers, write, cfg);
  if (dtype == 1) return launch_rows<__half>(p, n_layers, write, cfg);
  return launch_rows<float>(p, n_layers, write, cfg);
}

}  // namespace ea
