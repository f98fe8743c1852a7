// mxfp4_attention.cu — the expert's attention over 4-bit caches on the tensor cores.
//
// Per (layer, kv head) unit: 128 folded query rows (2 heads x 64 tokens) against cache rows [0, S) and
// the 64 own rows, softmax(Q K^T / sqrt(128)) V over the stored values.
//
// A prologue kernel norms and ropes q and k, stages q as f16 tiles (times a power of two per row) and
// encodes the own rows into the cache; the attention kernel follows; units cut over several CTAs
// are joined by a merge kernel. The units' tiles of 128 keys (ceil(S / 128), then the own rows) are cut into
// one contiguous range per CTA, one CTA per SM.
//
// The codes are widened to f16 tiles in shared memory, where tcgen05.mma takes them (a fragment in
// registers, as the decode step has it, would have to be formed again for each of the 128 query rows'
// warps). A code times 2^(e - R + 8) is exact in f16 as long as its block's scale e is within 2^22 below R;
// R is a running reference per segment and tensor, the largest scale of a block that is not all zeros
// (raised when a tile exceeds it by 2^3). K's reference goes back into the scores, V's into the
// output, both in fp32.
//
// Warp roles (448 threads):
//   warps 0-3, 4-7  softmax of the even / odd tiles of the CTA: thread = query row = TMEM lane; own running
//              maximum (raised lazily), sum and TMEM accumulator, joined at the end of a segment
//   warps 8-11 converters: thread = key row of the tile; K's codes, then V's, into double-buffered f16 tiles
//   warp 12    loads: one thread, bulk copies of the packed rows into a three-stage ring
//   warp 13    MMA: one thread issues S = Q K^T, O += P V (P from TMEM) and the next segment's Q load
#include "merge.cuh"
#include "mxfp4.cuh"
#include "rope.cuh"

namespace ea {

// ------------------------------------------------------------------------------- prologue
// One octet of threads per row: a unit's 128 q rows, 64 k rows, 64 v rows; grid (8, kv heads, layers).
__global__ void __launch_bounds__(256) mxfp4_prologue_kernel(const __grid_constant__ MxPrologueParams p) {
  const int g = blockIdx.y, l = blockIdx.z, i = threadIdx.x & 7;
  const int row = blockIdx.x * 32 + (threadIdx.x >> 3);
  const int kind = row < kRows ? 0 : row < kRows + kTok ? 1 : 2;  // the same for a whole warp
  const int rr = kind == 0 ? row : (row - kRows) % kTok, t = rr % kTok;
  const int dl = 8 * i, dh = 64 + 8 * i;
  // the rotation tables are read by lane-dependent index: through a generic address, not the constant bank
  const float4 *ra = &p.rot_a[0][0], *rb = &p.rot_b[0][0];
  asm volatile("" : "+l"(ra), "+l"(rb));
  pdl_wait_primary();
  pdl_launch_dependents();
  const MxAttnLayer& L = p.layer[l];
  const size_t unit = static_cast<size_t>(l) * kHkv + g;
  const __nv_bfloat16* src = kind == 0 ? L.q_raw + (static_cast<size_t>(g) * kRows + rr) * kD
                                       : (kind == 1 ? L.k_raw : L.v_raw) + (static_cast<size_t>(g) * kTok + rr) * kD;
  const __nv_bfloat16* gam = kind == 0 ? L.q_gamma : L.k_gamma;
  float xl[8], xh[8], gl[8], gh[8], yl[8], yh[8];
  unpack_bf16x8(*reinterpret_cast<const uint4*>(src + dl), xl);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(src + dh), xh);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(gam + dl), gl);
  unpack_bf16x8(*reinterpret_cast<const uint4*>(gam + dh), gh);
  if (kind == 0) {
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 a = ra[(t >> 3) * (kD / 2) + dl + e], b = rb[(t & 7) * (kD / 2) + dl + e];
      cs[e] = a.x * b.x - a.z * b.z;
      sn[e] = a.z * b.x + a.x * b.z;
    }
    norm_rope(xl, xh, gl, gh, cs, sn, yl, yh);
    float factor;
    f16_row(yl, yh, p.scale_log2, factor);
    uint8_t* q = p.q_ws + unit * kQTileBytes;
    *reinterpret_cast<uint4*>(q + swz_off(rr, i, kQTileBytes / 2)) = pack8(yl, true);
    *reinterpret_cast<uint4*>(q + swz_off(rr, i + 8, kQTileBytes / 2)) = pack8(yh, true);
    if (i == 0) p.q_factor[unit * kRows + rr] = factor;
    return;
  }
  if (kind == 1) {
    Pair cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 a = ra[(t >> 3) * (kD / 2) + dl + e], b = rb[(t & 7) * (kD / 2) + dl + e];
      const Pair ca = {a.x, a.y}, sa = {a.z, a.w}, cb = {b.x, b.y}, sb = {b.z, b.w};
      cs[e] = ca * cb + -(sa * sb);
      sn[e] = sa * cb + ca * sb;
    }
    pair_norm_rope(xl, xh, gl, gh, cs, sn, yl, yh);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      xl[e] = yl[e];
      xh[e] = yh[e];
    }
  }
  uint32_t cl, ch, sc;
  int el, eh;
  mx_encode_octet(xl, xh, cl, ch, sc, el, eh);
  const size_t crow = static_cast<size_t>(g) * p.Smax + p.Smax - kTok + rr;
  uint8_t* codes = (kind == 1 ? L.kc : L.vc) + crow * kMxRowBytes;
  *reinterpret_cast<uint32_t*>(codes + 4 * i) = cl;
  *reinterpret_cast<uint32_t*>(codes + 32 + 4 * i) = ch;
  if (i == 0) *reinterpret_cast<uint32_t*>((kind == 1 ? L.ks : L.vs) + crow * kMxRowScales) = sc;
  __nv_bfloat16* val = kind == 1 ? L.k_new : L.v_new;
  if (val != nullptr) {
    val += (static_cast<size_t>(g) * kTok + rr) * kD;
    mx_values8(cl, mx_pow2(el), xl);
    mx_values8(ch, mx_pow2(eh), xh);
    *reinterpret_cast<uint4*>(val + dl) = pack8(xl, false);
    *reinterpret_cast<uint4*>(val + dh) = pack8(xh, false);
  }
}

namespace mxa {

constexpr int kThreads = 448;
constexpr int kSoftmax = 256, kConvert = 128;
constexpr int kRing = 3;
constexpr uint32_t kCodes = kKeyTile * kMxRowBytes, kScales = kKeyTile * kMxRowScales;
constexpr uint32_t kStageBytes = 2 * kCodes + 2 * kScales;  // K codes, V codes, K scales, V scales
constexpr uint32_t kAtom = 16384, kTile = 2 * kAtom;        // an f16 tile: two 64-channel halves
constexpr uint32_t SM_Q = 0, SM_K = SM_Q + kTile, SM_V = SM_K + 2 * kTile, SM_RING = SM_V + 2 * kTile;
constexpr uint32_t SM_X = SM_RING + kRing * kStageBytes;    // [segment parity][stream][row] (m, l, R, -)
constexpr uint32_t SM_REF = SM_X + 4 * kRows * 16;          // [4] (R of K, R of V) of tile n % 4
constexpr uint32_t SM_MAX = SM_REF + 4 * 8;                 // [4 warps] (K, V) of a reference's raise
constexpr uint32_t SM_BAR = SM_MAX + 4 * 8;
constexpr int B_FULL = 0, B_EMPTY = B_FULL + kRing, B_KRDY = B_EMPTY + kRing, B_VRDY = B_KRDY + 2, B_REF = B_VRDY + 2,
              B_SFULL = B_REF + 2, B_PFULL = B_SFULL + 2, B_ODONE = B_PFULL + 2, B_QFULL = B_ODONE + 2,
              B_OFREE = B_QFULL + 1, B_DRAIN = B_OFREE + 1, kNumBars = B_DRAIN + 1;
constexpr uint32_t SM_TMEM = SM_BAR + kNumBars * 8, SM_ABORT = SM_TMEM + 4;
constexpr uint32_t kSmemBytes = SM_ABORT + 4 + 1024;  // + slack to align the base
static_assert(kSmemBytes <= 232448 && SM_RING % 128 == 0 && SM_X % 16 == 0 && SM_BAR % 8 == 0, "shared memory of one sm_103 CTA");
constexpr uint32_t TM_S = 0, TM_O = 256, kTmemCols = 512;  // two score (then P) buffers, two accumulators
constexpr int kRefField = 23, kMaxField = 26;  // f16 exponent field of 2^(e - R + 8), and its cut (all-zero blocks)
constexpr float kLazy = 8.0f;
constexpr uint32_t kBarConvert = 1, kBarSoftmax = 2;

struct Seg {
  int u, j0, j1;
};
__device__ __forceinline__ bool next_seg(long long& t, long long end, int T, Seg& s) {
  if (t >= end) return false;
  const int ti = static_cast<int>(t);
  s.u = ti / T;
  s.j0 = ti - s.u * T;
  const long long j1 = s.j0 + (end - t);
  s.j1 = static_cast<int>(j1 < T ? j1 : T);
  t += s.j1 - s.j0;
  return true;
}

struct Ctx {
  uint8_t* smem;
  uint32_t sbase, tmem;
  volatile uint32_t* abort_flag;
  uint32_t* status;
  long long start, end;
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + SM_BAR + 8u * i; }
  __device__ __forceinline__ bool wait(int b, uint32_t parity, uint32_t err) const {
    return bounded_wait(bar(b), parity, abort_flag, status, err);
  }
};

// Tile j of a unit: its first cache row and how many of its 128 rows are keys.
__device__ __forceinline__ int tile_row0(const MxExpertParams& p, int j) { return j < p.n_main ? j * kKeyTile : p.Smax - kTok; }
__device__ __forceinline__ int tile_live(const MxExpertParams& p, int j) {
  return j < p.n_main ? min(kKeyTile, p.S - j * kKeyTile) : kTok;
}

// ---------------------------------------------------------------------------------- loads
__device__ __noinline__ void producer(const MxExpertParams& p, const Ctx cx) {
  const uint64_t pol = l2_policy_evict_first();
  uint32_t n = 0;
  bool ok = true;
  long long t = cx.start;
  Seg s;
  while (ok && next_seg(t, cx.end, p.T, s)) {
    const MxAttnLayer& L = p.layer[s.u / kHkv];
    const size_t head = static_cast<size_t>(s.u % kHkv) * p.Smax;
    for (int j = s.j0; j < s.j1; ++j) {
      const uint32_t slot = n % kRing, round = n / kRing;
      if (round > 0 && !cx.wait(B_EMPTY + slot, (round - 1) & 1, kErrProducerWait)) {
        ok = false;
        break;
      }
      const size_t row = head + tile_row0(p, j);
      const int live = tile_live(p, j);
      // scale words come in fours: up to three rows past the last key (still in the cache) come along
      const uint32_t codes = live * kMxRowBytes, scales = ((live + 3) & ~3) * kMxRowScales;
      const uint32_t fb = cx.bar(B_FULL + slot), dst = cx.sbase + SM_RING + slot * kStageBytes;
      mbar_expect_tx(fb, 2 * codes + 2 * scales);
      bulk_load(dst, L.kc + row * kMxRowBytes, codes, fb, pol);
      bulk_load(dst + 2 * kCodes, L.ks + row * kMxRowScales, scales, fb, pol);
      bulk_load(dst + kCodes, L.vc + row * kMxRowBytes, codes, fb, pol);
      bulk_load(dst + 2 * kCodes + kScales, L.vs + row * kMxRowScales, scales, fb, pol);
      ++n;
    }
  }
  pdl_launch_dependents();
  if (!ok)  // let every copy already issued land before the CTA gives its shared memory back
    for (uint32_t k = 0; k < static_cast<uint32_t>(kRing) && k < n; ++k) {
      const uint32_t q = n - 1 - k;
      if (!drain_wait(cx.bar(B_FULL + q % kRing), (q / kRing) & 1)) atomicOr(cx.status, kErrDrain);
    }
}

// ----------------------------------------------------------------------------- converters
// Row `row` of a packed tile, 16-byte blocks in an order that spreads the lanes over the banks.
__device__ __forceinline__ void load_row(uint32_t src, int row, uint4 (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = ld_shared_v4(src + row * kMxRowBytes + (((i + (row >> 1)) & 3) << 4));
}
// ... as f16 into a tile of the swizzled layout; block b's codes times 2^(scale - ref + 8) (0 for a dead row)
__device__ __forceinline__ void convert_row(uint32_t dst, int row, const uint4 (&c)[4], uint32_t scales, int ref, bool live) {
  const uint32_t d = dst + row * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = (i + (row >> 1)) & 3;
    const int field = static_cast<int>((scales >> (8 * b)) & 255u) - ref + kRefField;
    const uint32_t f = live ? static_cast<uint32_t>(max(min(field, kMaxField), 0)) * 0x04000400u : 0u;
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    const uint32_t at = d + (b >> 1) * kAtom;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h[4];
      mx_unpack8(w[k], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(f));
      st_shared_v4(at + (((4 * (b & 1) + k) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
    }
  }
}
__device__ __forceinline__ int top_byte(uint32_t w) {
  const uint32_t m = __vmaxu2(w & 0x00FF00FFu, (w >> 8) & 0x00FF00FFu);
  return static_cast<int>(max(m & 0xFFFFu, m >> 16));
}
// the largest scale of the row's blocks that hold a code other than zero
__device__ __forceinline__ uint32_t top_nonzero(const uint4 (&c)[4], uint32_t scales, int row) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((c[i].x | c[i].y | c[i].z | c[i].w) & 0x77777777u) != 0u) top = max(top, (scales >> (8 * ((i + (row >> 1)) & 3))) & 255u);
  return top;
}

__device__ __noinline__ void converter(const MxExpertParams& p, const Ctx cx) {
  const int row = threadIdx.x - kSoftmax, warp = row >> 5;
  int2* refs = reinterpret_cast<int2*>(cx.smem + SM_REF);
  volatile uint2* tops = reinterpret_cast<volatile uint2*>(cx.smem + SM_MAX);
  uint32_t n = 0;
  bool ok = true;  // on a wait that gave up: no more work, but every barrier of the warps is still passed
  long long t = cx.start;
  Seg s;
  while (next_seg(t, cx.end, p.T, s)) {
    int rk = 0, rv = 0;  // references as scale bytes
    for (int j = s.j0; j < s.j1; ++j, ++n) {
      const uint32_t slot = n % kRing, src = cx.sbase + SM_RING + slot * kStageBytes;
      const bool live = row < tile_live(p, j);
      ok = ok && cx.wait(B_FULL + slot, (n / kRing) & 1, kErrProducerWait);
      uint4 ck[4], cv[4];
      uint32_t sk = 0, sv = 0;
      bool high = false;
      if (ok) {
        load_row(src, row, ck);
        load_row(src + kCodes, row, cv);
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sk) : "r"(src + 2 * kCodes + 4 * row) : "memory");
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sv) : "r"(src + 2 * kCodes + kScales + 4 * row) : "memory");
        high = live && (top_byte(sk) > rk + (kMaxField - kRefField) || top_byte(sv) > rv + (kMaxField - kRefField));
      }
      if (!bar_sync_and(kBarConvert, kConvert, !high)) {
        const uint32_t tk = __reduce_max_sync(0xffffffffu, ok && live ? top_nonzero(ck, sk, row) : 0u);
        const uint32_t tv = __reduce_max_sync(0xffffffffu, ok && live ? top_nonzero(cv, sv, row) : 0u);
        if ((row & 31) == 0) {
          tops[warp].x = tk;
          tops[warp].y = tv;
        }
        bar_sync(kBarConvert, kConvert);
        int mk = 0, mv = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mk = max(mk, static_cast<int>(tops[w].x));
          mv = max(mv, static_cast<int>(tops[w].y));
        }
        bar_sync(kBarConvert, kConvert);  // read before the next raise writes
        if (mk > rk + (kMaxField - kRefField)) rk = mk;
        if (mv > rv + (kMaxField - kRefField)) rv = mv;
      }
      // tile n's f16 buffers held tile n - 2: K's is free once QK(n-2) is done, V's once PV(n-2) is
      if (row == 0) refs[n & 3] = make_int2(rk, rv);
      if (n >= 2) ok = ok && cx.wait(B_SFULL + (n & 1), ((n - 2) >> 1) & 1, kErrProducerWait);
      if (ok) {
        convert_row(cx.sbase + SM_K + (n & 1) * kTile, row, ck, sk, rk, live);
        fence_proxy_async_smem();
        mbar_arrive(cx.bar(B_KRDY + (n & 1)));
      }
      if (n >= 2) ok = ok && cx.wait(B_ODONE + (n & 1), ((n - 2) >> 1) & 1, kErrProducerWait);
      if (ok) {
        convert_row(cx.sbase + SM_V + (n & 1) * kTile, row, cv, sv, rv, live);
        fence_proxy_async_smem();
        mbar_arrive(cx.bar(B_VRDY + (n & 1)));
        mbar_arrive(cx.bar(B_EMPTY + slot));
      }
    }
  }
}

// ------------------------------------------------------------------------------------ MMA
// Tile n of the CTA belongs to stream n & 1. QK(n) writes the stream's score buffer, which holds P(n-2)
// until PV(n-2) is done; PV(n) adds to the stream's accumulator. Of QK(i) and PV(i-1), which belong to
// different streams, the one whose inputs arrive first is issued first. After a segment's last QK its Q
// buffer is refilled for the next segment.
__device__ __noinline__ void mma_issuer(const MxExpertParams& p, const Ctx cx) {
  constexpr uint32_t kIdescQK = umma_idesc_f16(128, 128, false, false, false);
  constexpr uint32_t kIdescPV = umma_idesc_f16(128, 128, false, false, true);
  const uint64_t pol = l2_policy_evict_first();
  uint32_t n = 0;  // tiles before the current segment
  int seg = 0;
  bool ok = true;
  long long t = cx.start;
  Seg s;
  auto load_q = [&](int u) {
    mbar_expect_tx(cx.bar(B_QFULL), kTile);
    bulk_load(cx.sbase + SM_Q, p.q_ws + static_cast<size_t>(u) * kQTileBytes, kTile, cx.bar(B_QFULL), pol);
  };
  int q_loads = 0;
  if (cx.start < cx.end) {
    load_q(static_cast<int>(cx.start) / p.T);
    ++q_loads;
  }
  while (ok && next_seg(t, cx.end, p.T, s)) {
    ok = cx.wait(B_QFULL, seg & 1, kErrMmaWait);
    if (!ok) break;
    tc_fence_after();
    const int nt = s.j1 - s.j0;
    const bool more = t < cx.end;
    auto qk_ready = [&](uint32_t m) -> bool {
      if (!mbar_test_wait(cx.bar(B_KRDY + (m & 1)), (m >> 1) & 1)) return false;
      return m < 2 || mbar_test_wait(cx.bar(B_ODONE + (m & 1)), ((m - 2) >> 1) & 1);
    };
    auto issue_qk = [&](uint32_t m) {
      mbar_arrive(cx.bar(B_REF + (m & 1)));  // the tile's references, seen with KRDY, are passed on to the softmax
      tc_fence_after();
      const uint32_t ka = cx.sbase + SM_K + (m & 1) * kTile, d = cx.tmem + TM_S + (m & 1) * 128;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
        umma_f16_ss(d, sw128_desc(cx.sbase + SM_Q + off, 16, 1024), sw128_desc(ka + off, 16, 1024), kIdescQK, kk > 0);
      }
      umma_commit(cx.bar(B_SFULL + (m & 1)));
    };
    auto pv_ready = [&](uint32_t m, int ii) -> bool {
      if (ii == 0 && seg > 0 && !mbar_test_wait(cx.bar(B_OFREE), (seg - 1) & 1)) return false;
      return mbar_test_wait(cx.bar(B_PFULL + (m & 1)), (m >> 1) & 1) &&
             mbar_test_wait(cx.bar(B_VRDY + (m & 1)), (m >> 1) & 1);
    };
    auto issue_pv = [&](uint32_t m, int ii) {
      tc_fence_after();
      const uint32_t va = cx.sbase + SM_V + (m & 1) * kTile, pc = cx.tmem + TM_S + (m & 1) * 128;
      const int nk = s.j0 + ii < p.n_main ? 8 : 4;  // the own tile has 64 keys
      for (int kk = 0; kk < nk; ++kk)
        umma_f16_ts(cx.tmem + TM_O + (m & 1) * 128, pc + kk * 8, sw128_desc(va + kk * 16 * 128, kAtom, 1024), kIdescPV,
                    (ii > 1 || kk > 0));
      umma_commit(cx.bar(B_ODONE + (m & 1)));
    };
    bool q_todo = more;
    for (int i = 0; i <= nt && ok; ++i) {
      bool qk_todo = i < nt, pv_todo = i > 0;
      uint64_t t0 = 0;
      for (uint32_t it = 0; qk_todo || pv_todo; ++it) {
        bool moved = false;
        if (qk_todo && qk_ready(n + i)) {
          issue_qk(n + i);
          qk_todo = false;
          moved = true;
        }
        if (pv_todo && pv_ready(n + i - 1, i - 1)) {
          issue_pv(n + i - 1, i - 1);
          pv_todo = false;
          moved = true;
        }
        if (q_todo && i == nt && mbar_test_wait(cx.bar(B_SFULL + ((n + nt - 1) & 1)), ((n + nt - 1) >> 1) & 1)) {
          load_q(s.u + 1);
          ++q_loads;
          q_todo = false;
        }
        if (moved) continue;
        // nothing to issue: suspend for a moment on the barrier that the next MMA most likely waits for
        if (pv_todo) mbar_try_wait_hint(cx.bar(B_PFULL + ((n + i - 1) & 1)), ((n + i - 1) >> 1) & 1, 300);
        else mbar_try_wait_hint(cx.bar(B_KRDY + ((n + i) & 1)), ((n + i) >> 1) & 1, 300);
        if ((it & 63u) == 0) {
          if (*cx.abort_flag) {
            ok = false;
            break;
          }
          const uint64_t now = globaltimer_ns();
          if (t0 == 0) t0 = now;
          if (now - t0 > kWaitLimitNs || it >= 0x7fffffc0u) {
            *cx.abort_flag = 1u;
            atomicOr(cx.status, kErrMmaWait);
            ok = false;
            break;
          }
        }
      }
    }
    n += nt;
    // (the last PV needs the last tile's P, so its QK is done: this does not wait in practice)
    if (ok && q_todo) {
      ok = cx.wait(B_SFULL + ((n - 1) & 1), ((n - 1) >> 1) & 1, kErrMmaWait);
      if (ok) {
        load_q(s.u + 1);
        ++q_loads;
      }
    }
    ++seg;
  }
  if (!ok && q_loads > 0 && !drain_wait(cx.bar(B_QFULL), (q_loads - 1) & 1)) atomicOr(cx.status, kErrDrain);
  umma_commit(cx.bar(B_DRAIN));  // every MMA issued is complete before TMEM is released
  if (!drain_wait(cx.bar(B_DRAIN), 0)) atomicOr(cx.status, kErrDrain);
}

// -------------------------------------------------------------------------------- softmax
__device__ __noinline__ void scale_tmem(uint32_t addr, float a, int cols) {
  for (int c = 0; c < cols; c += 32) {
    uint32_t o[32];
    tmem_ld32(addr + c, o);
    tmem_wait_ld();
    reg_fence32(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
    tmem_st32(addr + c, o);
  }
  tmem_wait_st();
}
__device__ __noinline__ void scale_p(uint32_t addr, float a) {  // 32 columns of f16 pairs
  uint32_t q[32];
  tmem_ld32(addr, q);
  tmem_wait_ld();
  reg_fence32(q);
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const float2 f = unpack_f16x2(q[e]);
    q[e] = pack_f16x2(f.x * a, f.y * a);
  }
  tmem_st32(addr, q);
  tmem_wait_st();
}

__device__ __noinline__ void softmax_warps(const MxExpertParams& p, const Ctx cx) {
  const int k = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane = static_cast<uint32_t>(r & ~31) << 16;
  const uint32_t sa = cx.tmem + lane + TM_S + k * 128, oa = cx.tmem + lane + TM_O + k * 128;
  const int2* refs = reinterpret_cast<const int2*>(cx.smem + SM_REF);
  uint32_t base = 0, seg = 0;
  bool ok = true;
  auto wait = [&](int b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, cx.wait(b, parity, kErrSoftmaxWait));
  };
  long long t = cx.start;
  Seg s;
  while (next_seg(t, cx.end, p.T, s)) {
    const int nt = s.j1 - s.j0;
    const float qf = p.q_factor[static_cast<size_t>(s.u) * kRows + r] * 0.00390625f;  // K's tiles carry 2^8
    float m = -INFINITY, lsum = 0.f;
    int ref = 0, last = -1;
    for (int i = (k - static_cast<int>(base)) & 1; ok && i < nt; i += 2) {
      const int n = static_cast<int>(base) + i, j = s.j0 + i;
      ok = wait(B_REF + k, (n >> 1) & 1) && wait(B_SFULL + k, (n >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const int2 rf = refs[n & 3];
      if (rf.y != ref) {  // V's reference was raised: the accumulator of earlier tiles moves to it
        if (last >= 0) scale_tmem(oa, ref - rf.y < -126 ? 0.f : mx_pow2(ref - rf.y), 128);
        ref = rf.y;
      }
      const float ct = qf * mx_scale(rf.x);
      const int live = tile_live(p, j);
      auto load_pair = [&](int pr, uint32_t (&v)[2][32]) {
        tmem_ld32(sa + 64 * pr, v[0]);
        tmem_ld32(sa + 64 * pr + 32, v[1]);
        tmem_wait_ld();
        reg_fence32(v[0]);
        reg_fence32(v[1]);
        if (64 * pr + 64 > live) {
#pragma unroll
          for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (64 * pr + 32 * ch + e >= live) v[ch][e] = __float_as_uint(-INFINITY);
        }
      };
      float2 ts[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) ts[q] = make_float2(0.f, 0.f);
      const float2 ct2 = make_float2(ct, ct);
      const int npair = j < p.n_main ? 2 : 1;
      // P goes over the scores' first columns: chunk pr's 32 columns of pairs hold scores of chunks <= pr
#pragma unroll 1
      for (int pr = 0; pr < npair; ++pr) {
        uint32_t v[2][32];
        load_pair(pr, v);
        float mx[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) mx[q] = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 7] = fmax3(mx[(e >> 1) & 7], __uint_as_float(v[ch][e]), __uint_as_float(v[ch][e + 1]));
        const float mc = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * ct;
        // chunk 0 always holds a key, so m is finite from there on
        if (__any_sync(0xffffffffu, m == -INFINITY || mc > m + kLazy)) {
          const float mn = fmaxf(m, mc), a = ex2_approx(m - mn);
          if (last >= 0 || pr > 0) {  // PV(n-2) is done (QK(n) waited for it): the accumulator is stable
            if (last >= 0) scale_tmem(oa, a, 128);
            if (pr > 0) scale_p(sa, a);
            load_pair(pr, v);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) ts[q] = make_float2(ts[q].x * a, ts[q].y * a);
          lsum *= a;
          m = mn;
        }
        const float2 neg = make_float2(-m, -m);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[ch][2 * e]), __uint_as_float(v[ch][2 * e + 1])), ct2, neg);
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            ts[e & 3] = __fadd2_rn(ts[e & 3], make_float2(p0, p1));
            pk[e] = pack_f16x2(p0, p1);
          }
          tmem_st16(sa + 32 * pr + 16 * ch, pk);
        }
      }
      lsum += ((ts[0].x + ts[0].y) + (ts[1].x + ts[1].y)) + ((ts[2].x + ts[2].y) + (ts[3].x + ts[3].y));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(cx.bar(B_PFULL + k));
      last = n;
    }
    // ---- the segment's end: both streams' last PV, then thread (k, r) joins columns [64 k, 64 k + 64)
    if (ok && last >= 0) ok = wait(B_ODONE + k, (last >> 1) & 1);
    // (by segment parity: a warpgroup without a tile in a segment may be here while the other still reads
    // the segment before; it cannot pass this segment's barrier before that)
    float4* xch = reinterpret_cast<float4*>(cx.smem + SM_X) + (seg & 1) * 2 * kRows;
    xch[k * kRows + r] = make_float4(m, lsum, static_cast<float>(ref), 0.f);
    ok = bar_sync_and(kBarSoftmax, kSoftmax, ok);
    if (ok) {
      tc_fence_after();
      const float4 x0 = xch[r], x1 = xch[kRows + r];
      const float M = fmaxf(x0.x, x1.x), a0 = ex2_approx(x0.x - M), a1 = ex2_approx(x1.x - M);
      const float L = a0 * x0.y + a1 * x1.y;
      // O is in units of 2^(R - 127 - 8)
      const float R = fmaxf(x0.z, x1.z), inv = 1.0f / L;
      const float c0 = a0 * inv * ex2_approx(x0.z - R), c1 = a1 * inv * ex2_approx(x1.z - R);
      const float two_r = mx_scale(static_cast<uint32_t>(R));
      // a segment of one tile leaves the other stream's accumulator as it was: not read
      const bool has0 = nt > static_cast<int>(base & 1), has1 = nt > static_cast<int>((base + 1) & 1);
      const int l = s.u / kHkv, g = s.u % kHkv;
      const bool full = s.j0 == 0 && s.j1 == p.T;
      float o[64];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t col = cx.tmem + lane + TM_O + 64 * k + 32 * h;
        uint32_t v[32];
        if (has0) {
          tmem_ld32(col, v);
          tmem_wait_ld();
          reg_fence32(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[32 * h + e] = __uint_as_float(v[e]) * c0;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[32 * h + e] = 0.f;
        }
        if (has1) {
          tmem_ld32(col + 128, v);
          tmem_wait_ld();
          reg_fence32(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[32 * h + e] = fmaf(__uint_as_float(v[e]), c1, o[32 * h + e]);
        }
      }
      tc_fence_before();
      mbar_arrive(cx.bar(B_OFREE));  // the accumulators are read
#pragma unroll
      for (int e = 0; e < 64; ++e) o[e] = o[e] * 0.00390625f * two_r;
      if (full) {
        __nv_bfloat16* dst = p.layer[l].out + (static_cast<size_t>(g) * kRows + r) * kD + 64 * k;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(dst + 8 * c) =
              make_uint4(pack_bf16x2(o[8 * c], o[8 * c + 1]), pack_bf16x2(o[8 * c + 2], o[8 * c + 3]),
                         pack_bf16x2(o[8 * c + 4], o[8 * c + 5]), pack_bf16x2(o[8 * c + 6], o[8 * c + 7]));
      } else {
        // a part: f16, the half row times the power of two that puts its largest magnitude in [2^14, 2^15)
        const size_t sl = static_cast<size_t>(blockIdx.x) * 2 + (base == 0 ? 0 : 1);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 64; ++e) amax = fmaxf(amax, fabsf(o[e]));
        const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -126), 112);
        const float up = mx_pow2(-ex);
        uint4* po = p.part_o + (sl * kPartChunks + 8 * k) * kRows + r;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          po[c * kRows] = make_uint4(pack_f16x2(o[8 * c] * up, o[8 * c + 1] * up), pack_f16x2(o[8 * c + 2] * up, o[8 * c + 3] * up),
                                     pack_f16x2(o[8 * c + 4] * up, o[8 * c + 5] * up), pack_f16x2(o[8 * c + 6] * up, o[8 * c + 7] * up));
        p.part_lse[(sl * 3 + 1 + k) * kRows + r] = mx_pow2(ex);
        if (k == 0) p.part_lse[sl * 3 * kRows + r] = M + log2f(L);
      }
    }
    base += nt;
    ++seg;
  }
}

}  // namespace mxa

__global__ void __launch_bounds__(mxa::kThreads, 1) mxfp4_attention_kernel(const __grid_constant__ MxExpertParams p) {
  using namespace mxa;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctx cx;
  cx.smem = smem;
  cx.sbase = smem_u32(smem);
  cx.abort_flag = reinterpret_cast<volatile uint32_t*>(smem + SM_ABORT);
  cx.status = p.status;
  cx.start = cta_tile_start(blockIdx.x, p.W, gridDim.x);
  cx.end = cta_tile_start(blockIdx.x + 1, p.W, gridDim.x);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kNumBars; ++b) {
      const bool conv = (b >= B_EMPTY && b < B_REF), sm = b >= B_PFULL && b < B_ODONE;
      mbar_init(cx.bar(b), conv ? kConvert : sm ? 128 : b == B_OFREE ? kSoftmax : 1);
    }
    *cx.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(cx.sbase + SM_TMEM, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cx.tmem = *reinterpret_cast<volatile uint32_t*>(smem + SM_TMEM);
  pdl_wait_primary();
  if (warp < 8) {
    softmax_warps(p, cx);
  } else if (warp < 12) {
    converter(p, cx);
  } else if (warp == 12 && (threadIdx.x & 31) == 0) {
    producer(p, cx);
  } else if (warp == 13 && (threadIdx.x & 31) == 0) {
    mma_issuer(p, cx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(cx.tmem, kTmemCols);
}

// The units that the CTA ranges cut: grid (units, 8), thread = one row's 8 columns.
__global__ void __launch_bounds__(256) mxfp4_merge_kernel(const __grid_constant__ MxExpertParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const SplitUnit su = p.split[blockIdx.x];
  merge_row_chunk<8>(p.part_o, p.part_lse, su, blockIdx.y * 2 + (threadIdx.x >> 7), threadIdx.x & 127,
                     p.layer[su.u / kHkv].out);
}

cudaError_t mxfp4_attention_set_attributes() {
  return cudaFuncSetAttribute(mxfp4_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(mxa::kSmemBytes));
}

cudaError_t launch_mxfp4_prologue(const MxPrologueParams& p, int n_layers, cudaLaunchConfig_t cfg) {
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3(8, kHkv, n_layers);
  return cudaLaunchKernelEx(&cfg, mxfp4_prologue_kernel, p);
}

cudaError_t launch_mxfp4_attention(const MxExpertParams& p, cudaLaunchConfig_t cfg) {
  cudaLaunchConfig_t c = cfg;
  c.blockDim = dim3(mxa::kThreads);
  c.dynamicSmemBytes = mxa::kSmemBytes;
  cudaError_t e = cudaLaunchKernelEx(&c, mxfp4_attention_kernel, p);
  if (e != cudaSuccess || p.n_split == 0) return e;
  cfg.gridDim = dim3(p.n_split, 8);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, mxfp4_merge_kernel, p);
}

}  // namespace ea
