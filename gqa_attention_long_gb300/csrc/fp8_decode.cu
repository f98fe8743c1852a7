// fp8_decode.cu — the text model's decode step over an 8-bit cache: a simple form. One CTA per (layer, kv head) appends
// the new row, then walks the keys 128 at a time with the running maximum and sum of a softmax per head; a second walk, with the final ones, gives the
// weights.
#include "fp8.cuh"

namespace ea {
namespace f8d {

constexpr int kThreads = 256;

// Appends a row held by warp 0 (x, see f8_load_row) to the block at `codes`, `before` rows in: all threads.
__device__ __forceinline__ void append(uint8_t* codes, float* scale, int before, const float (&x)[4], float* red, __nv_bfloat16* val) {
  const int tid = threadIdx.x, lane = tid & 31;
  const float s = before > 0 ? *scale : f8_pow2(kF8FirstExp);
  if (tid < 32) {
    const float amax = f8_row_max(x);
    if (tid == 0) red[0] = amax;
  }
  __syncthreads();
  const int k = f8_growth(red[0], s);
  const float s1 = f8_grown(s, k);
  if (k > 0)
    for (int c = tid; c < before * kD / 16; c += kThreads) {
      uint4* old = reinterpret_cast<uint4*>(codes) + c;
      *old = f8_rescale16(*old, f8_shrink(k));
    }
  if (tid < 32) {
    const F8Quotient q(s1);
    const uint32_t w = f8_pack4(q(x[0]), q(x[1]), q(x[2]), q(x[3]));
    *reinterpret_cast<uint16_t*>(codes + before * kD + 2 * lane) = static_cast<uint16_t>(w);
    *reinterpret_cast<uint16_t*>(codes + before * kD + 64 + 2 * lane) = static_cast<uint16_t>(w >> 16);
    if (val != nullptr) {
      float y[4];
      f8_unpack4(w, y);
      *reinterpret_cast<uint32_t*>(val + 2 * lane) = pack_bf16x2(y[0] * s1, y[1] * s1);
      *reinterpret_cast<uint32_t*>(val + 64 + 2 * lane) = pack_bf16x2(y[2] * s1, y[3] * s1);
    }
    if (tid == 0) *scale = s1;
  }
  __syncthreads();
}

}  // namespace f8d

template <int CAP>
__global__ void __launch_bounds__(f8d::kThreads) fp8_decode_kernel(const __grid_constant__ F8DecodeParams<CAP> p) {
  using namespace f8d;
  __shared__ float q[kRepText][kD], s[kRepText][kKeyTile], red[2], hm[kRepText], ha[kRepText], hl[kRepText];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, u = blockIdx.x, g = u % kHkv;
  const F8AttnLayer& L = p.layer[u / kHkv];
  const size_t head = static_cast<size_t>(g) * p.Smax * kD;
  float* ks = L.ks + g * (p.Smax / kScaleBlock + 1);
  float* vs = L.vs + g * (p.Smax / kScaleBlock + 1);
  pdl_wait_primary();
  float x[4], gm[4], y[4];
  f8_load_row(L.q_raw + (kRepText * g + warp) * kD, lane, x);
  f8_load_row(L.q_gamma, lane, gm);
  f8_norm_rope(x, gm, p.rot, lane, y);
  for (int e = 0; e < 2; ++e) {
    q[warp][2 * lane + e] = y[e] * p.scale_log2;
    q[warp][64 + 2 * lane + e] = y[2 + e] * p.scale_log2;
  }
  const int blk = p.pos / kScaleBlock, before = p.pos % kScaleBlock;
  f8_load_row(L.k_raw + g * kD, lane, x);
  f8_load_row(L.k_gamma, lane, gm);
  f8_norm_rope_pair(x, gm, p.rot, lane, y);
  append(L.kc + head + static_cast<size_t>(blk) * kScaleBlock * kD, ks + blk, before, y, red, L.k_new ? L.k_new + g * kD : nullptr);
  f8_load_row(L.v_raw + g * kD, lane, x);
  append(L.vc + head + static_cast<size_t>(blk) * kScaleBlock * kD, vs + blk, before, x, red, L.v_new ? L.v_new + g * kD : nullptr);
  const int r = tid & 127, half = tid >> 7;
  auto scores = [&](int j, float (&d)[4]) {
    const int key = j * kKeyTile + r;
    for (int h = 0; h < 4; ++h) d[h] = -INFINITY;
    if (key > p.pos) return;
    for (int h = 0; h < 4; ++h) d[h] = 0.f;
    const uint4* row = reinterpret_cast<const uint4*>(L.kc + head + static_cast<size_t>(key) * kD);
    for (int c = 0; c < kD / 16; ++c) {
      const uint4 w = row[c];
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      for (int i = 0; i < 4; ++i) {
        float v[4];
        f8_unpack4(ws[i], v);
        for (int e = 0; e < 4; ++e)
          for (int h = 0; h < 4; ++h) d[h] = fmaf(v[e], q[4 * half + h][16 * c + 4 * i + e], d[h]);
      }
    }
    for (int h = 0; h < 4; ++h) d[h] *= ks[j];
  };
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f}, d[4];  // m, l: warp's head
  for (int j = 0; j < p.T; ++j) {
    scores(j, d);
    for (int h = 0; h < 4; ++h) s[4 * half + h][r] = d[h];
    __syncthreads();
    float t = -INFINITY;
    for (int i = lane; i < kKeyTile; i += 32) t = fmaxf(t, s[warp][i]);
    for (int i = 16; i >= 1; i >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, i));
    const float mn = fmaxf(m, t), a = exp2f(m - mn);
    float sum = 0.f;
    for (int i = lane; i < kKeyTile; i += 32) {
      const float e = exp2f(s[warp][i] - mn);
      s[warp][i] = e;
      sum += e;
    }
    for (int i = 16; i >= 1; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    l = l * a + sum;
    m = mn;
    if (lane == 0) ha[warp] = a;
    __syncthreads();
    for (int h = 0; h < 4; ++h) acc[h] *= ha[4 * half + h];
    const int n = min(kKeyTile, p.pos + 1 - j * kKeyTile);
    const uint8_t* v = L.vc + head + static_cast<size_t>(j) * kKeyTile * kD + r;
    for (int i = 0; i < n; ++i) {
      float c[4];
      f8_unpack4(v[i * kD], c);
      for (int h = 0; h < 4; ++h) acc[h] = fmaf(s[4 * half + h][i] * vs[j], c[0], acc[h]);
    }
    __syncthreads();
  }
  if (lane == 0) {
    hm[warp] = m;
    hl[warp] = l;
  }
  __syncthreads();
  for (int h = 0; h < 4; ++h) L.out[(kRepText * g + 4 * half + h) * kD + r] = __float2bfloat16_rn(acc[h] / hl[4 * half + h]);
  if (L.w_out != nullptr)
    for (int j = 0; j < p.T; ++j) {
      scores(j, d);
      float w = 0.f;
      for (int h = 0; h < 4; ++h) w += exp2f(d[h] - hm[4 * half + h]) / hl[4 * half + h];
      s[half][r] = w;
      __syncthreads();
      const int key = j * kKeyTile + r;
      const size_t at = static_cast<size_t>(g) * p.Smax + key;
      if (half == 0 && key <= p.pos) L.w_out[at] = (key < p.pos && L.w_in != nullptr ? L.w_in[at] : 0.f) + (w + s[1][r]);
      __syncthreads();
    }
  pdl_launch_dependents();
}

cudaError_t fp8_decode_set_attributes() { return cudaSuccess; }

template <int CAP>
cudaError_t launch_fp8_decode(const F8DecodeParams<CAP>& p, cudaLaunchConfig_t cfg) {
  cfg.gridDim = dim3(p.n_layers * kHkv);
  cfg.blockDim = dim3(f8d::kThreads);
  return cudaLaunchKernelEx(&cfg, fp8_decode_kernel<CAP>, p);
}
template cudaError_t launch_fp8_decode<kSmallCap>(const F8DecodeParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode<kDecodeMaxLayers>(const F8DecodeParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);

}  // namespace ea
