// fp8_decode_small.cu — the text model's decode step over an 8-bit cache for little work: a few key tiles to an SM.
//
// The same step as fp8_decode.cu's, whose ring of tiles, tensor memory and five kinds of warps take longer to get going than such a call
// has work. Here a warp takes 32 keys of one unit, straight from global memory into registers, and multiplies by mma.sync
// (f16, which holds every e4m3 code): S = Q K^T with the eight heads' q as rows 0-7 and what f16 rounded off them, times 2^11, as rows 8-15; and
// O = P V with P split the same way, so that both hold 22 bits. A lane's codes are in the order that its fragments want, because a product's
// inner index may run through the channels (the keys) in any order that both operands share:
//   K: lane 4 g + t holds bytes [16 t, 16 t + 16) and [64 + 16 t, 80 + 16 t) of key g of each eight: word s of them is its part of step s.
//   V: it holds bytes [16 g, 16 g + 16) of keys 2t, 2t + 1, 2t + 8, 2t + 9 of each sixteen: byte i of two keys is a pair for columns of channel 16 g + i.
// Scores come out in P's own fragment layout. A CTA has eight warps and whole 128-row blocks of one unit; the block of the new row is moved to a
// larger scale in the registers of the four warps that hold it. Two to four parts of a unit are a cluster and meet in shared memory; more of
// them are merged by the last one to finish. Whole units and clusters form the weights that are asked for, too: their keys' scores wait in
// shared memory until the parts have told each other their log2-sum-exps; else they go to the workspace, for a second kernel.
//
// What bounds it: latencies one after the other (launch, the rows' and the codes' loads, the norm and rotation, the merge); 1 layer at pos 300
// 6.7 us, at pos 4700 (9.6 MB of cache) 9.2 us, 8 layers at pos 1000 9.5 us.
#include "cluster_exit.cuh"
#include "fp8.cuh"

namespace ea {
namespace f8s {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = 32;  // of a warp's chunk

struct Smem {
  float4 rot[kD / 2];
  alignas(16) __half q[2][kRepText][kD];  // high and low halves
  alignas(16) float qf[kRepText];         // what a head's scores are multiplied by, beside K's scale
  alignas(16) uint8_t fresh[2][kD];       // the new row's codes, K and V
  float scale[2];                         // its block's scale
  float shrink[2];                        // what the block's earlier codes are multiplied by (1: nothing)
  float2 ml[kWarps][kRepText];            // (reference, sum)
  uint32_t last;
  float2 part_ml[kRepText];               // this CTA's, read by its cluster
  alignas(16) float part_o[kRepText][kD];
  alignas(16) float lse[kRepText];        // of the unit, if weights are formed
  alignas(16) float o[kWarps][kRepText][kD];
};  // then, if weights are formed, the scores of this CTA's keys: [key][8 heads]
constexpr int kAhead = 4;  // sums before that a thread loads early

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, int half) {
  return cvt_f16x2_e4m3x2(static_cast<uint16_t>(half ? w >> 16 : w));
}
// Two numbers as f16, and 2^11 times what that leaves.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(a, b);
  const float2 f = unpack_f16x2(hi);
  lo = pack_f16x2((a - f.x) * 2048.0f, (b - f.y) * 2048.0f);
}

// The new K (kv = 0) or V row, one warp: what it is made from, and then its codes, its block's scale, and how the block's earlier rows
// move.
struct NewRow {
  float x[4], gm[4], old;
};
template <class P>
__device__ __forceinline__ void load_new_row(const P& p, const F8AttnLayer& L, int g, int kv, int lane, NewRow& r) {
  f8_load_row((kv ? L.v_raw : L.k_raw) + g * kD, lane, r.x);
  f8_load_row(L.k_gamma, lane, r.gm);
  r.old = p.pos % kScaleBlock > 0 ? (kv ? L.vs : L.ks)[g * (p.Smax / kScaleBlock + 1) + p.pos / kScaleBlock] : f8_pow2(kF8FirstExp);
}
template <class P>
__device__ __forceinline__ void new_row(const P& p, Smem& sm, const F8AttnLayer& L, int g, int kv, int lane, const NewRow& r) {
  const int blk = p.pos / kScaleBlock, before = p.pos % kScaleBlock;
  float* scale = (kv ? L.vs : L.ks) + g * (p.Smax / kScaleBlock + 1) + blk;
  const float old = r.old;
  float x[4] = {r.x[0], r.x[1], r.x[2], r.x[3]};
  if (kv == 0) {
    float y[4];
    f8_norm_rope_pair(x, r.gm, sm.rot, lane, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = y[e];
  }
  const int k = f8_growth(f8_row_max(x), old);
  const float now = f8_grown(old, k);
  const F8Quotient q(now);
  const uint32_t w = f8_pack4(q(x[0]), q(x[1]), q(x[2]), q(x[3]));
  *reinterpret_cast<uint16_t*>(&sm.fresh[kv][2 * lane]) = static_cast<uint16_t>(w);
  *reinterpret_cast<uint16_t*>(&sm.fresh[kv][64 + 2 * lane]) = static_cast<uint16_t>(w >> 16);
  __syncwarp();
  if (lane == 0) {
    sm.scale[kv] = now;
    sm.shrink[kv] = before > 0 ? f8_shrink(k) : 1.0f;
    *scale = now;
  }
  uint8_t* codes = (kv ? L.vc : L.kc) + (static_cast<size_t>(g) * p.Smax + p.pos) * kD;
  if (lane < kD / 16) reinterpret_cast<uint4*>(codes)[lane] = reinterpret_cast<const uint4*>(sm.fresh[kv])[lane];
  __nv_bfloat16* val = kv ? L.v_new : L.k_new;
  if (val != nullptr) {
    float y[4];
    f8_unpack4(w, y);
    *reinterpret_cast<uint32_t*>(val + g * kD + 2 * lane) = pack_bf16x2(y[0] * now, y[1] * now);
    *reinterpret_cast<uint32_t*>(val + g * kD + 64 + 2 * lane) = pack_bf16x2(y[2] * now, y[3] * now);
  }
}

// q row h as f16 halves, times the power of two that puts its largest magnitude in [1, 2).
template <class P>
__device__ __forceinline__ void query_row(const P& p, Smem& sm, const F8AttnLayer& L, int g, int h, int lane) {
  float x[4], gm[4], y[4];
  f8_load_row(L.q_gamma, lane, gm);
  f8_load_row(L.q_raw + (kRepText * g + h) * kD, lane, x);
  f8_norm_rope(x, gm, sm.rot, lane, y);
  const int e = f16_exponent(f8_row_max(y));
  const float down = f8_pow2(-e);
  uint32_t hi[2], lo[2];
  split_f16(y[0] * down, y[1] * down, hi[0], lo[0]);
  split_f16(y[2] * down, y[3] * down, hi[1], lo[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<uint32_t*>(&sm.q[0][h][64 * i + 2 * lane]) = hi[i];
    *reinterpret_cast<uint32_t*>(&sm.q[1][h][64 * i + 2 * lane]) = lo[i];
  }
  if (lane == 0) sm.qf[h] = p.scale_log2 * f8_pow2(e);
}

// A lane's codes of a chunk: K [eight keys][half], V [sixteen keys][key of the lane]; zeros for rows from `rows` on.
struct Codes {
  uint4 k[4][2], v[2][4];
};
__device__ __forceinline__ void load_codes(Codes& c, const uint8_t* kc, const uint8_t* vc, int rows, int g, int t) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c.k[j][i] = 8 * j + g < rows ? *reinterpret_cast<const uint4*>(kc + (8 * j + g) * kD + 64 * i + 16 * t) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * j + 2 * t + (i & 1) + 8 * (i >> 1);
      c.v[j][i] = r < rows ? *reinterpret_cast<const uint4*>(vc + r * kD + 16 * g) : make_uint4(0u, 0u, 0u, 0u);
    }
}
// A chunk of the new row's block, rows [first, first + 32): earlier codes moved to the block's scale (and put back), the new row put in.
__device__ __forceinline__ void last_codes(Codes& c, Smem& sm, uint8_t* kc, uint8_t* vc, int rows, int at, int g, int t) {
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float f = sm.shrink[kv];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int r = kv ? 16 * (n >> 2) + 2 * t + (n & 1) + 8 * ((n >> 1) & 1) : 8 * (n >> 1) + g;
      const int b = kv ? 16 * g : 64 * (n & 1) + 16 * t;
      uint4& w = kv ? c.v[n >> 2][n & 3] : c.k[n >> 1][n & 1];
      if (f != 1.0f && r < rows) {
        w = f8_rescale16(w, f);
        *reinterpret_cast<uint4*>((kv ? vc : kc) + r * kD + b) = w;
      }
      if (r == at) w = *reinterpret_cast<const uint4*>(&sm.fresh[kv][b]);
    }
  }
}

}  // namespace f8s

template <int CAP, bool kForm>
__global__ void __launch_bounds__(f8s::kThreads, 1) fp8_decode_small_kernel(const __grid_constant__ F8SmallParams<CAP> p) {
  using namespace f8s;
  extern __shared__ __align__(16) uint8_t f8s_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(f8s_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gk = lane >> 2, t = lane & 3;
  const int u = blockIdx.x / p.parts, part = blockIdx.x % p.parts, g = u % kHkv;
  const F8AttnLayer& L = p.layer[u / kHkv];
  const int j0 = part * p.T / p.parts, j1 = (part + 1) * p.T / p.parts;  // tiles
  const int c1 = min(j1 * (kKeyTile / kKeys), p.pos / kKeys + 1);          // chunks
  const size_t head = static_cast<size_t>(g) * p.Smax * kD;
  if (tid < kD / 2) sm.rot[tid] = p.rot[tid];
  __syncthreads();
  pdl_wait_primary();
  int c = j0 * (kKeyTile / kKeys) + warp;
  Codes codes;
  auto chunk = [&](int i, const uint8_t* base) { return base + head + static_cast<size_t>(i) * kKeys * kD; };
  if (c < c1) load_codes(codes, chunk(c, L.kc), chunk(c, L.vc), p.pos - c * kKeys, gk, t);
  const float* ksc = L.ks + g * (p.Smax / kScaleBlock + 1);
  const float* vsc = L.vs + g * (p.Smax / kScaleBlock + 1);
  const int blk0 = c / (kKeyTile / kKeys);
  float ks = c < c1 && blk0 < p.T - 1 ? ksc[blk0] : 0.f, vs = c < c1 && blk0 < p.T - 1 ? vsc[blk0] : 0.f;
  const bool appends = j1 == p.T && warp >= kWarps - 2;  // (the last two warps: K's new row, and V's)
  NewRow fresh;
  if (appends) load_new_row(p, L, g, warp - (kWarps - 2), lane, fresh);
  const bool form = kForm && L.w_out != nullptr;
  float* xs = reinterpret_cast<float*>(f8s_smem + sizeof(Smem));
  const int first = j0 * kKeyTile, keys = min(j1 * kKeyTile, p.pos + 1) - first;  // this CTA's
  const float* w_in = form && L.w_in != nullptr ? L.w_in + static_cast<size_t>(g) * p.Smax + first : nullptr;
  auto sum_before = [&](int k) { return w_in != nullptr && k < keys && first + k < p.pos ? w_in[k] : 0.f; };
  float before[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) before[i] = sum_before(tid + kThreads * i);
  query_row(p, sm, L, g, warp, lane);
  if (appends) new_row(p, sm, L, g, warp - (kWarps - 2), lane, fresh);
  __syncthreads();
  pdl_launch_dependents();
  // A fragments of step s: q's channels of this lane's word s, high (rows 0-7) and low (8-15)
  uint32_t qa[8][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 channels, in two pieces of 8 halves
      const uint4 a = *reinterpret_cast<const uint4*>(&sm.q[0][gk][64 * i + 16 * t + 8 * h]);
      const uint4 b = *reinterpret_cast<const uint4*>(&sm.q[1][gk][64 * i + 16 * t + 8 * h]);
      const int s = 4 * i + 2 * h;
      qa[s][0] = a.x; qa[s][2] = a.y; qa[s + 1][0] = a.z; qa[s + 1][2] = a.w;
      qa[s][1] = b.x; qa[s][3] = b.y; qa[s + 1][1] = b.z; qa[s + 1][3] = b.w;
    }
  const float qf = sm.qf[gk];
  float m_run = -INFINITY, lsum = 0.f;  // head gk
  float down = 1.0f;                    // see f8_lower
  float o[16][2];                       // head gk, channels 16 (2t) + i and 16 (2t + 1) + i
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = 0.f;
  float x[4][2];  // the chunk's scores in log2 units: keys 8 j + 2 t, + 1
#pragma unroll 1
  for (; c < c1; c += kWarps) {
    const int j = c / (kKeyTile / kKeys), key0 = c * kKeys;
    if (j == p.T - 1) {
      const int rows = p.pos - key0;
      last_codes(codes, sm, const_cast<uint8_t*>(chunk(c, L.kc)), const_cast<uint8_t*>(chunk(c, L.vc)), rows, rows, gk, t);
      ks = sm.scale[0];
      vs = sm.scale[1];
    }
    float m = -INFINITY;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {codes.k[n][i].x, codes.k[n][i].y, codes.k[n][i].z, codes.k[n][i].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) mma(d, qa[4 * i + s], codes_f16(w[s], 0), codes_f16(w[s], 1));
      }
      const float f = qf * ks;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[n][e] = key0 + 8 * n + 2 * t + e <= p.pos ? fmaf(d[2 + e], 0x1p-11f, d[e]) * f : -INFINITY;
        m = fmaxf(m, x[n][e]);
      }
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (form) {
      float* to = xs + (key0 - first + 2 * t) * kRepText + gk;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) to[(8 * n + e) * kRepText] = x[n][e];
    } else if (p.scores != nullptr && L.w_out != nullptr) {
      float* to = p.scores + (static_cast<size_t>(2 * u + (gk >> 2)) * p.T * kKeyTile + key0 + 2 * t) * 4 + (gk & 3);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) to[(8 * n + e) * 4] = x[n][e];
    }
    const float top = fmaxf(m_run, m), fa = ex2_approx(m_run - top), fb = ex2_approx(m - top);
    m_run = top;
    // weights relative to the chunk's largest: A fragments of sixteen keys each
    float sum = 0.f;
    uint32_t pa[2][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const bool l0 = key0 + 8 * n + 2 * t <= p.pos, l1 = key0 + 8 * n + 2 * t + 1 <= p.pos;
      const float e0 = l0 ? ex2_approx(x[n][0] - m) : 0.f, e1 = l1 ? ex2_approx(x[n][1] - m) : 0.f;
      sum += e0 + e1;
      split_f16(e0, e1, pa[n >> 1][2 * (n & 1)], pa[n >> 1][2 * (n & 1) + 1]);
    }
    lsum = fmaf(lsum, fa, sum * fb);
    if (__builtin_expect(vs * down > kF8TopSum, 0)) {
      const float less = f8_lower(vs * down);
      down *= less;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i][0] *= less;
        o[i][1] *= less;
      }
    }
    const float fv = fb * (vs * down);
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // channels 16 g + 4 w .. + 3
      float d[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) d[e][k] = 0.f;
#pragma unroll
      for (int j2 = 0; j2 < 2; ++j2) {
        auto word = [&](int i) {
          const uint4& v = codes.v[j2][i];
          return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
        };
        const uint32_t a01 = __byte_perm(word(0), word(1), 0x5140), a23 = __byte_perm(word(0), word(1), 0x7362);
        const uint32_t b01 = __byte_perm(word(2), word(3), 0x5140), b23 = __byte_perm(word(2), word(3), 0x7362);
        mma(d[0], pa[j2], codes_f16(a01, 0), codes_f16(b01, 0));
        mma(d[1], pa[j2], codes_f16(a01, 1), codes_f16(b01, 1));
        mma(d[2], pa[j2], codes_f16(a23, 0), codes_f16(b23, 0));
        mma(d[3], pa[j2], codes_f16(a23, 1), codes_f16(b23, 1));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[4 * w + e][0] = fmaf(o[4 * w + e][0], fa, fmaf(d[e][2], 0x1p-11f, d[e][0]) * fv);
        o[4 * w + e][1] = fmaf(o[4 * w + e][1], fa, fmaf(d[e][3], 0x1p-11f, d[e][1]) * fv);
      }
    }
    if (c + kWarps < c1) {
      const int cn = c + kWarps, b = cn / (kKeyTile / kKeys);
      load_codes(codes, chunk(cn, L.kc), chunk(cn, L.vc), p.pos - cn * kKeys, gk, t);
      ks = b < p.T - 1 ? ksc[b] : 0.f;
      vs = b < p.T - 1 ? vsc[b] : 0.f;
    }
  }
  // ---- the CTA's eight warps into one
  lsum += __shfl_xor_sync(0xffffffffu, lsum, 1);
  lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
  if (t == 0) sm.ml[warp][gk] = f8_lowered(make_float2(m_run, lsum), down);
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    *reinterpret_cast<float4*>(&sm.o[warp][gk][32 * t + i]) = make_float4(o[i][0], o[i + 1][0], o[i + 2][0], o[i + 3][0]);
    *reinterpret_cast<float4*>(&sm.o[warp][gk][32 * t + 16 + i]) = make_float4(o[i][1], o[i + 1][1], o[i + 2][1], o[i + 3][1]);
  }
  __syncthreads();
  // thread: head warp, channels 4 lane .. + 3. (A warp without a chunk has reference -inf and adds nothing; every CTA has a key.)
  const int h = warp;
  float M = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm.ml[k][h].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float2 ml = sm.ml[k][h];
    if (ml.x == -INFINITY && ml.y == 0.f) continue;
    const float f = ex2_approx(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(&sm.o[k][h][4 * lane]);
    sum = fmaf(ml.y, f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  if (p.cluster) {
    // a unit's parts are a cluster: their partials stay in shared memory, and the first one combines them
    *reinterpret_cast<float4*>(&sm.part_o[h][4 * lane]) = acc;
    if (lane == 0) sm.part_ml[h] = make_float2(M, sum);
    cluster_sync();
    if (part == 0 || form) {
      float4 v[kF8SmallCluster];
      float2 ml[kF8SmallCluster];
#pragma unroll
      for (int k = 0; k < kF8SmallCluster; ++k)
        if (k < p.parts) {
          v[k] = part == 0 ? ld_shared_cluster_v4(mapa_shared(smem_u32(&sm.part_o[h][4 * lane]), k)) : make_float4(0.f, 0.f, 0.f, 0.f);
          ml[k] = ld_shared_cluster_v2(mapa_shared(smem_u32(&sm.part_ml[h]), k));
        }
#pragma unroll
      for (int k = 0; k < kF8SmallCluster; ++k)
        if (k < p.parts) M = fmaxf(M, ml[k].x);
      sum = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kF8SmallCluster; ++k)
        if (k < p.parts) {
          const float f = ex2_approx(ml[k].x - M);
          sum = fmaf(ml[k].y, f, sum);
          acc.x = fmaf(v[k].x, f, acc.x);
          acc.y = fmaf(v[k].y, f, acc.y);
          acc.z = fmaf(v[k].z, f, acc.z);
          acc.w = fmaf(v[k].w, f, acc.w);
        }
      // (a store that needs every load's value)
      *reinterpret_cast<volatile float*>(&sm.o[0][h][lane]) = ((acc.x + acc.y) + (acc.z + acc.w)) + sum;
    }
    cluster_sync_exit();  // no CTA leaves while another one reads its shared memory
    if (part != 0 && !form) return;
  } else if (p.parts > 1) {
    const size_t ps = static_cast<size_t>(blockIdx.x) * kRepText + h;
    __stcg(reinterpret_cast<float4*>(p.part_o + ps * kD) + lane, acc);
    if (lane == 0) __stcg(reinterpret_cast<float2*>(p.part_ml) + ps, make_float2(M, sum));
    __syncthreads();
    if (tid == 0) sm.last = atom_add_acq_rel_gpu(p.unit_cnt + u, 1u) == static_cast<uint32_t>(p.parts - 1) ? 1u : 0u;
    __syncthreads();
    if (!sm.last) return;
    // every part of head h: a lane weighs one
    const size_t first = static_cast<size_t>(u) * p.parts;
    const float2 ml = lane < p.parts ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (first + lane) * kRepText + h) : make_float2(-INFINITY, 0.f);
    float4 v[kF8SmallParts / 2];  // half of the parts under way at a time
    M = ml.x;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    const float f = lane < p.parts ? ex2_approx(ml.x - M) : 0.f;
    sum = lane < p.parts ? ml.y * f : 0.f;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < p.parts; k0 += kF8SmallParts / 2) {
#pragma unroll
      for (int k = 0; k < kF8SmallParts / 2; ++k)
        if (k0 + k < p.parts) v[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((first + k0 + k) * kRepText + h) * kD) + lane);
#pragma unroll
      for (int k = 0; k < kF8SmallParts / 2; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
        if (k0 + k < p.parts) {
          acc.x = fmaf(v[k].x, w, acc.x);
          acc.y = fmaf(v[k].y, w, acc.y);
          acc.z = fmaf(v[k].z, w, acc.z);
          acc.w = fmaf(v[k].w, w, acc.w);
        }
      }
    }
    if (tid == 0) p.unit_cnt[u] = 0u;  // ready for the next call
  }
  if (form) {
    if (lane == 0) sm.lse[h] = M + log2f(sum);
    __syncthreads();
    const float4 la = *reinterpret_cast<const float4*>(sm.lse), lb = *reinterpret_cast<const float4*>(sm.lse + 4);
    float* w_out = L.w_out + static_cast<size_t>(g) * p.Smax + first;
    auto put = [&](int k, float w) {
      const float4 a = *reinterpret_cast<const float4*>(xs + k * kRepText), b = *reinterpret_cast<const float4*>(xs + k * kRepText + 4);
      w_out[k] = w + f8_weight(a, b, la, lb);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (tid + kThreads * i < keys) put(tid + kThreads * i, before[i]);
    for (int k = tid + kThreads * kAhead; k < keys; k += kThreads) put(k, sum_before(k));
    if (p.cluster && part != 0) return;
  }
  const float inv = 1.0f / sum;
  *reinterpret_cast<uint2*>(L.out + (kRepText * g + h) * kD + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (!form && p.scores != nullptr && lane == 0) p.lse[u * kRepText + h] = M + log2f(sum);
}

cudaError_t fp8_decode_small_set_attributes() {
  const int bytes = static_cast<int>(sizeof(f8s::Smem)), kept = kF8SmallTiles * kKeyTile * kRepText * static_cast<int>(sizeof(float));
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel, int size) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, size);
  };
  set(fp8_decode_small_kernel<kSmallCap, false>, bytes);
  set(fp8_decode_small_kernel<kSmallCap, true>, bytes + kept);
  set(fp8_decode_small_kernel<kDecodeMaxLayers, false>, bytes);
  set(fp8_decode_small_kernel<kDecodeMaxLayers, true>, bytes + kept);
  return e;
}

template <int CAP>
cudaError_t launch_fp8_decode_small(const F8SmallParams<CAP>& p, cudaLaunchConfig_t cfg) {
  cudaLaunchAttribute attr[2] = {cfg.attrs[0]};
  if (p.cluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(p.parts), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  cfg.gridDim = dim3(p.n_layers * kHkv * p.parts);
  cfg.blockDim = dim3(f8s::kThreads);
  cfg.dynamicSmemBytes = sizeof(f8s::Smem);
  if (!p.form) return cudaLaunchKernelEx(&cfg, fp8_decode_small_kernel<CAP, false>, p);
  cfg.dynamicSmemBytes += static_cast<size_t>((p.T + p.parts - 1) / p.parts) * kKeyTile * kRepText * sizeof(float);
  return cudaLaunchKernelEx(&cfg, fp8_decode_small_kernel<CAP, true>, p);
}
template cudaError_t launch_fp8_decode_small<kSmallCap>(const F8SmallParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode_small<kDecodeMaxLayers>(const F8SmallParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);

}  // namespace ea
