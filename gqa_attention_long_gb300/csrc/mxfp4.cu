// mxfp4.cu — the 4-bit cache's writer and reader, and the attention over it.
//
// Writer: rows [row0, row0 + n) of K and V, as they come (bf16, fp16 or fp32; any head and row
// strides), become E2M1 codes and scale bytes in the same rows of the cache. Reader: the same rows as
// numbers. Both are one pass over the data, bound by HBM: 16 threads take a row, 8 channels each.
#include <type_traits>

#include "mxfp4.cuh"
#include "rope.cuh"

namespace ea {
namespace mx {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = kThreads / 16;

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

// grid (row blocks, kv heads, layers); thread = 8 channels of a K row and of a V row
template <class T>
__global__ void __launch_bounds__(mx::kThreads) mxfp4_write_kernel(const __grid_constant__ MxRowsParams p) {
  const int c = threadIdx.x & 15;
  const int r = blockIdx.x * mx::kRowsPerCta + (threadIdx.x >> 4);
  const int g = blockIdx.y;
  const MxRowsLayer& L = p.layer[blockIdx.z];
  pdl_wait_primary();
  pdl_launch_dependents();
  // a row's 16 threads are half a warp: the shuffles below stay inside it
  const bool live = r < p.n_rows;
  const size_t row = static_cast<size_t>(g) * p.Smax + p.row0 + (live ? r : 0);
  const long long src = g * p.head_stride + (live ? r : 0) * p.row_stride + 8 * c;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[8];
    mx::load8(static_cast<const T*>(kv ? L.v : L.k) + src, x);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = mx_exponent(amax);
    const uint32_t codes = mx_pack8(x, mx_pow2(-e));
    if (live) {
      *reinterpret_cast<uint32_t*>((kv ? L.vc : L.kc) + row * kMxRowBytes + 4 * c) = codes;
      if ((c & 3) == 0) (kv ? L.vs : L.ks)[row * kMxRowScales + (c >> 2)] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <class T>
__global__ void __launch_bounds__(mx::kThreads) mxfp4_read_kernel(const __grid_constant__ MxRowsParams p) {
  const int c = threadIdx.x & 15;
  const int r = blockIdx.x * mx::kRowsPerCta + (threadIdx.x >> 4);
  const int g = blockIdx.y;
  const MxRowsLayer& L = p.layer[blockIdx.z];
  pdl_wait_primary();
  pdl_launch_dependents();
  if (r >= p.n_rows) return;
  const size_t row = static_cast<size_t>(g) * p.Smax + p.row0 + r;
  const long long dst = g * p.head_stride + r * p.row_stride + 8 * c;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>((kv ? L.vc : L.kc) + row * kMxRowBytes + 4 * c);
    const uint32_t b = (kv ? L.vs : L.ks)[row * kMxRowScales + (c >> 2)];
    float x[8];
    mx_values8(w, mx_scale(b), x);
    mx::store8(static_cast<T*>(kv ? L.v : L.k) + dst, x);
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

// ------------------------------------------------------------------------------ attention
// Prologue: q rows normed and roped into the workspace (fp32), the new k rows normed, roped and
// encoded and the new v rows encoded into the cache. One octet of threads per row; grid
// (row blocks of 32, kv heads, layers); rows [0, rq) of a unit are its q rows, then tok k rows, then
// tok v rows.
__global__ void __launch_bounds__(256) mxfp4_prologue_kernel(const __grid_constant__ MxAttnParams p) {
  const int g = blockIdx.y, l = blockIdx.z, i = threadIdx.x & 7;
  const int rq = p.rep * p.tok;
  const int row0 = blockIdx.x * 32 + (threadIdx.x >> 3), rows = rq + 2 * p.tok;
  const bool live = row0 < rows;  // octets past the end repeat the last row and store nothing
  const int row = live ? row0 : rows - 1;
  pdl_wait_primary();
  const int kind = row < rq ? 0 : row < rq + p.tok ? 1 : 2;
  const int rr = kind == 0 ? row : kind == 1 ? row - rq : row - rq - p.tok;
  const int t = rr % p.tok;
  const MxAttnLayer& L = p.layer[l];
  const __nv_bfloat16* src = kind == 0 ? L.q_raw + (static_cast<size_t>(g) * rq + rr) * kD
                                       : (kind == 1 ? L.k_raw : L.v_raw) + (static_cast<size_t>(g) * p.tok + rr) * kD;
  const __nv_bfloat16* gam = kind == 0 ? L.q_gamma : L.k_gamma;
  const int dl = 8 * i, dh = 64 + 8 * i;
  float xl[8], xh[8], gl[8], gh[8], yl[8], yh[8];
  unpack_bf16x8(*reinterpret_cast<const uint4*>(src + dl), xl);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(src + dh), xh);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(gam + dl), gl);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(gam + dh), gh);
  Pair cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 a = p.rot_a[t >> 3][dl + e], b = p.rot_b[t & 7][dl + e];
    const Pair ca = {a.x, a.y}, sa = {a.z, a.w}, cb = {b.x, b.y}, sb = {b.z, b.w};
    cs[e] = ca * cb + -(sa * sb);
    sn[e] = sa * cb + ca * sb;
  }
  if (kind == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      yl[e] = xl[e];
      yh[e] = xh[e];
    }
  }
  float zl[8], zh[8];
  pair_norm_rope(xl, xh, gl, gh, cs, sn, zl, zh);
  if (kind != 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      yl[e] = zl[e];
      yh[e] = zh[e];
    }
  }
  uint32_t cl, ch, sc;
  int el, eh;
  mx_encode_octet(yl, yh, cl, ch, sc, el, eh);
  if (!live) return;
  if (kind == 0) {
    float* dst = p.q_ws + ((static_cast<size_t>(l) * kHkv + g) * rq + rr) * kD;
    mx::store8(dst + dl, yl);
    mx::store8(dst + dh, yh);
  } else {
    const size_t crow = static_cast<size_t>(g) * p.Smax + p.new_row0 + rr;
    uint8_t* codes = (kind == 1 ? L.kc : L.vc) + crow * kMxRowBytes;
    *reinterpret_cast<uint32_t*>(codes + 4 * i) = cl;
    *reinterpret_cast<uint32_t*>(codes + 32 + 4 * i) = ch;
    if (i == 0) *reinterpret_cast<uint32_t*>((kind == 1 ? L.ks : L.vs) + crow * kMxRowScales) = sc;
    __nv_bfloat16* val = kind == 1 ? L.k_new : L.v_new;
    if (val != nullptr) {
      val += (static_cast<size_t>(g) * p.tok + rr) * kD;
      mx_values8(cl, mx_pow2(el), xl);
      mx_values8(ch, mx_pow2(eh), xh);
      mx::store8(val + dl, xl);
      mx::store8(val + dh, xh);
    }
  }
}

// One warp per query row: lane l holds channels [4l, 4l + 4); online softmax over the keys one by one.
__global__ void __launch_bounds__(256) mxfp4_attention_kernel(const __grid_constant__ MxAttnParams p) {
  const int g = blockIdx.y, l = blockIdx.z, lane = threadIdx.x & 31;
  const int rq = p.rep * p.tok, row = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait_primary();
  const MxAttnLayer& L = p.layer[l];
  const size_t unit = static_cast<size_t>(l) * kHkv + g;
  const float4 q = *reinterpret_cast<const float4*>(p.q_ws + (unit * rq + row) * kD + 4 * lane);
  float m = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int n = p.first + p.tok;
  for (int j = 0; j < n; ++j) {
    const size_t r = static_cast<size_t>(g) * p.Smax + (j < p.first ? j : p.new_row0 + (j - p.first));
    auto four = [&](const uint8_t* codes, const uint8_t* scales, float (&x)[4]) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(codes + r * kMxRowBytes + 2 * lane);
      const float s = mx_scale(scales[r * kMxRowScales + (lane >> 3)]);
      float y[8];
      mx_values8(w, s, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = y[e];
    };
    float k[4], v[4];
    four(L.kc, L.ks, k);
    four(L.vc, L.vs, v);
    float s = q.x * k[0] + q.y * k[1] + q.z * k[2] + q.w * k[3];
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    sum = sum * a + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * a + w * v[e];
  }
  const float inv = 1.0f / sum;
  *reinterpret_cast<uint2*>(L.out + (static_cast<size_t>(g) * rq + row) * kD + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

cudaError_t launch_mxfp4_attention(const MxAttnParams& p, int n_layers, cudaLaunchConfig_t cfg) {
  const int rq = p.rep * p.tok;
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3((rq + 2 * p.tok + 31) / 32, kHkv, n_layers);
  cudaError_t e = cudaLaunchKernelEx(&cfg, mxfp4_prologue_kernel, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(rq / 8, kHkv, n_layers);
  return cudaLaunchKernelEx(&cfg, mxfp4_attention_kernel, p);
}

}  // namespace ea
