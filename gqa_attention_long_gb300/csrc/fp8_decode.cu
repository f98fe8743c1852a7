// fp8_decode.cu — the text model's decode step over an 8-bit cache, on the tensor cores (tcgen05, e4m3 operands).
//
// Per layer and kv head (a unit): 8 query rows against rows [0, pos], the new row appended first. A unit's keys are cut into
// tiles of 128, which are the cache's blocks, so that a tile has one scale for K and one for V; the tiles of all units are cut into
// one contiguous range per CTA. HBM bounds it (16 flop a byte), if what is done to a tile stays well under the 0.73 us in which an
// SM's share of the bandwidth brings one.
//
// The codes go to the tensor cores as they are, K's as the rows of one product and V's as the columns of the next, and no value is
// ever widened. What they meet has more bits than a code: it comes in pieces. A number y, |y| <= 256, is c0 + c1 / 32 + c2 / 1024 + ..,
// each c the e4m3 number next to 32 times what the pieces before left: a code is off by at most half of its last place,
// 2^-5 of a number's power of two, so that four pieces hold a q row to 2^-20 of its largest channel (scores that weights come from:
// fp32 would be 2^-24), three hold a softmax weight to 2^-15 of itself down to 2^-13 of the tile's largest, and to 2^-28 of that below. Products of codes are exact, sums are in fp32, and
// pieces are columns that the MMA has to spare: 8 heads in 4 pieces are N = 32.
//   S^T  = K Q^T    M = 128 keys, N = 32 (piece, head), K = 128 channels; A = the K tile (K-major)
//   O^T  = V^T P^T  M = 128 channels, N = 32 (3 pieces and zeros), K = 128 keys; A = the V tile (MN-major)
// Each tile's weights are taken relative to its own largest score, and its O^T is read out and added, times its share and V's scale, in
// fp32: whatever scales and maxima the other tiles have, none of it is rounded away.
//
// Warp roles (512 threads): warps 0-3 and 4-7 softmax, of even and of odd tiles (thread = key = TMEM lane); warps 8-11 output
// (thread = channel = TMEM lane): sums of O^T, a segment's end, the merge; warp 12 loads tiles by TMA into a ring; warp 13 issues the MMAs;
// warps 14 and 15 prepare: the next segment's Q, and the new K and V row, which they append. S has four buffers, Q, P and O have two. A unit cut
// over several CTAs is merged by the part that finishes last.
// For layers whose weights are asked for, the scores go to the workspace (32 bytes a key) and a second kernel forms the weights
// from them and the units' log2-sum-exps.
#include "fp8.cuh"

namespace ea {
namespace f8d {

constexpr int kThreads = 512;
constexpr int kGroup = 128;  // threads of either set of softmax warps, and of the output warps
constexpr int kStages = 6;
constexpr uint32_t kTileBytes = kKeyTile * kD;      // a K or a V tile: 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr int kCols = 32;                           // N of both products
constexpr uint32_t kOpBytes = kCols * 128;          // Q or P: 32 rows of 128 bytes
constexpr int kMaxParts = 160;                      // parts of one unit (at most one per CTA)
constexpr int kMergeBatch = 6;
constexpr int kTails = 72;                          // units of one CTA, at most
// Shared memory (offsets from the 1024-byte-aligned base)
constexpr uint32_t SM_RING = 0;
constexpr uint32_t SM_QT = SM_RING + kStages * kStageBytes;      // 2 buffers
constexpr uint32_t SM_PT = SM_QT + 2 * kOpBytes;                 // 2 buffers
constexpr uint32_t SM_ROT = SM_PT + 2 * kOpBytes;                // float4 [64]
constexpr uint32_t SM_RED = SM_ROT + (kD / 2) * 16;              // [2 sets][2][4 warps][8 heads]
constexpr uint32_t SM_FAC = SM_RED + 2 * 2 * 4 * kRepText * 4;   // [4][8 heads]: (what the set's sums before are multiplied by, the tile's share)
constexpr uint32_t SM_FIN = SM_FAC + 4 * kRepText * 8;           // [8 segments][2 sets][8 heads]: (reference, sum)
constexpr uint32_t SM_QF = SM_FIN + 8 * 2 * kRepText * 8;        // [8 segments][8]: what a head's S columns are multiplied by (read up to four tiles after the last QK)
constexpr uint32_t SM_LRED = SM_QF + 8 * kRepText * 4;           // [2 sets][4 warps][8 heads]
constexpr uint32_t SM_TAILS = SM_LRED + 2 * 4 * kRepText * 4;    // [K, V][kTails]: the appended block's scale
constexpr uint32_t SM_SW = SM_TAILS + 2 * kTails * 4;            // merge weights [part][head]
constexpr uint32_t SM_BAR = (SM_SW + kMaxParts * kRepText * 4 + 7) & ~7u;
// PFULL, ODONE, OFREE: one barrier per parity of the tile count; SDONE: per S buffer; QFULL, QFREE: per Q buffer. The softmax warps
// can be two tiles, and so three segments, ahead of the output warps: what those wait for from them has as many barriers (FAC by
// tile, FIN by segment) as it takes for none to complete twice unseen.
constexpr int B_FULL = 0, B_EMPTY = kStages, B_SDONE = 2 * kStages, B_PFULL = B_SDONE + 4, B_ODONE = B_PFULL + 2,
              B_OFREE = B_ODONE + 2, B_QFULL = B_OFREE + 2, B_QFREE = B_QFULL + 2, B_FAC = B_QFREE + 2, B_FIN = B_FAC + 4,
              B_DRAIN = B_FIN + 8, kNumBars = B_DRAIN + 1;
constexpr uint32_t SM_TMEM = SM_BAR + kNumBars * 8;
constexpr uint32_t SM_ABORT = SM_TMEM + 4;
constexpr uint32_t SM_MERGE = SM_ABORT + 4;
constexpr uint32_t SM_TAILN = SM_MERGE + 4;  // [K, V]: units whose new row is in place
constexpr uint32_t kSmemBytes = SM_TAILN + 8 + 1024;  // + base alignment
static_assert(kSmemBytes <= 232448, "shared memory budget of one sm_103 CTA");
constexpr uint32_t kTmemCols = 256, TM_S = 0, TM_O = 128;  // 4 and 2 buffers of 32 columns

struct Seg {
  int u, j0, j1;  // unit and its key-tile range [j0, j1)
};
// Next segment of a CTA's tile range [t, end).
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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
// The largest of a warp's numbers (NaN passed over).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t atom_add_acq_rel_gpu(uint32_t* a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(a), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void st_shared_u8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire_shared(uint32_t a) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_release_shared(uint32_t a, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Two numbers' next piece: the pair of codes, and 32 times what it leaves.
__device__ __forceinline__ uint32_t take_piece(float& a, float& b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(a), "f"(b));
  const float2 f = unpack_f16x2(cvt_f16x2_e4m3x2(c));
  a = (a - f.x) * 32.0f;
  b = (b - f.y) * 32.0f;
  return c;
}

// ------------------------------------------------------------------------------- tail warps
// Waits until `n` units' new rows (of K: kv = 0; of V: 1) are in place.
template <class P>
__device__ __forceinline__ bool wait_tail(const P& p, uint32_t sbase, int kv, uint32_t n, volatile uint32_t* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0; it < 0x80000000u; ++it) {
    if (ld_acquire_shared(sbase + SM_TAILN + 4 * kv) >= n) return true;
    if ((it & 63u) == 63u) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
  }
  *abort_flag = 1u;
  atomicOr(p.status, kErrF8DecodeWait);
  return false;
}

// q rows h0 .. h0 + N - 1 of segment seg's unit, as pieces, into its Q buffer: one warp.
template <int N, int CAP>
__device__ __forceinline__ void prepare_q(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, int u, int h0, uint32_t seg, int lane) {
  const F8AttnLayer& L = p.layer[u / kHkv];
  const float4* rot = reinterpret_cast<const float4*>(smem + SM_ROT);
  float x[N][4], gm[4];
  f8_load_row(L.q_gamma, lane, gm);
#pragma unroll
  for (int k = 0; k < N; ++k) f8_load_row(L.q_raw + (kRepText * (u % kHkv) + h0 + k) * kD, lane, x[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int h = h0 + k;
    float y[4];
    f8_norm_rope(x[k], gm, rot, lane, y);
    const int e = f16_exponent(f8_row_max(y));  // the row's largest magnitude is in [2^e, 2^(e + 1)): put it in [128, 256)
    const float up = f8_pow2(min(7 - e, 126));
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= up;
    if (lane == 0) reinterpret_cast<float*>(smem + SM_QF)[(seg & 7) * kRepText + h] = __fdiv_rn(p.scale_log2, up);
#pragma unroll
    for (int piece = 0; piece < 4; ++piece) {
      const uint32_t lo = take_piece(y[0], y[1]), hi = take_piece(y[2], y[3]);
      const uint32_t row = sbase + SM_QT + (seg & 1) * kOpBytes + (piece * kRepText + h) * 128;  // 16-byte chunk c of row r at chunk c ^ (r % 8)
      st_shared_u16(row + (((lane >> 3) ^ h) << 4) + ((2 * lane) & 15), static_cast<uint16_t>(lo));
      st_shared_u16(row + ((((lane >> 3) + 4) ^ h) << 4) + ((2 * lane) & 15), static_cast<uint16_t>(hi));
    }
  }
  fence_proxy_async_smem();  // read by the tensor core
}

// One warp for K (kv = 0), one for V: half of every later segment's Q (the softmax warps prepare the first one), and the new row of every unit
// whose last tile this CTA has.
template <int CAP>
__device__ __noinline__ void prepare(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, int kv, long long start, long long end,
                                     volatile uint32_t* abort_flag) {
  const int lane = threadIdx.x & 31;
  const float4* rot = reinterpret_cast<const float4*>(smem + SM_ROT);
  const int blk = p.pos / kScaleBlock, before = p.pos % kScaleBlock;
  uint32_t n = 0, seg = 0;
  Seg s;
  for (long long t = start; next_seg(t, end, p.T, s); ++seg) {
    if (seg > 0) {
      const uint32_t bar0 = sbase + SM_BAR, buf = seg & 1;
      bool ok = true;
      if (seg > 1) ok = bounded_wait(bar0 + 8 * (B_QFREE + buf), ((seg - 2) >> 1) & 1, abort_flag, p.status, kErrF8DecodeWait);
      if (!__all_sync(0xffffffffu, ok)) return;
      prepare_q<4>(p, sbase, smem, s.u, 4 * kv, seg, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar0 + 8 * (B_QFULL + buf));
    }
    if (s.j1 != p.T) continue;
    const int g = s.u % kHkv;
    const F8AttnLayer& L = p.layer[s.u / kHkv];
    float* scale = (kv ? L.vs : L.ks) + g * (p.Smax / kScaleBlock + 1) + blk;
    uint8_t* codes = (kv ? L.vc : L.kc) + (static_cast<size_t>(g) * p.Smax + static_cast<size_t>(blk) * kScaleBlock) * kD;
    const float old = before > 0 ? *scale : f8_pow2(kF8FirstExp);
    float x[4];
    f8_load_row((kv ? L.v_raw : L.k_raw) + g * kD, lane, x);
    if (kv == 0) {
      float gm[4], y[4];
      f8_load_row(L.k_gamma, lane, gm);
      f8_norm_rope_pair(x, gm, rot, lane, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = y[e];
    }
    const int k = f8_growth(f8_row_max(x), old);
    const float now = f8_grown(old, k);
    if (k > 0 && before > 0) {
      const float f = f8_shrink(k);
      uint4* c = reinterpret_cast<uint4*>(codes) + lane;
      const int pieces = before * (kD / 16);
      for (int i = 0; i < pieces; i += 8 * 32) {
        uint4 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + 32 * e + lane < pieces) w[e] = c[i + 32 * e];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + 32 * e + lane < pieces) c[i + 32 * e] = f8_rescale16(w[e], f);
      }
    }
    const F8Quotient q(now);
    const uint32_t w = f8_pack4(q(x[0]), q(x[1]), q(x[2]), q(x[3]));
    *reinterpret_cast<uint16_t*>(codes + before * kD + 2 * lane) = static_cast<uint16_t>(w);
    *reinterpret_cast<uint16_t*>(codes + before * kD + 64 + 2 * lane) = static_cast<uint16_t>(w >> 16);
    fence_proxy_async_global();  // the rows are read back by TMA
    if (lane == 0) reinterpret_cast<float*>(smem + SM_TAILS)[kv * kTails + n] = now;
    __syncwarp();
    ++n;
    if (lane == 0) {
      st_release_shared(sbase + SM_TAILN + 4 * kv, n);
      *scale = now;
    }
    __nv_bfloat16* val = kv ? L.v_new : L.k_new;
    if (val != nullptr) {
      float y[4];
      f8_unpack4(w, y);
      *reinterpret_cast<uint32_t*>(val + g * kD + 2 * lane) = pack_bf16x2(y[0] * now, y[1] * now);
      *reinterpret_cast<uint32_t*>(val + g * kD + 64 + 2 * lane) = pack_bf16x2(y[2] * now, y[3] * now);
    }
  }
}

// --------------------------------------------------------------------------------- producer
template <int CAP>
__device__ __noinline__ void producer(const F8DecodeParams<CAP>& p, uint32_t sbase, long long start, long long end,
                                      volatile uint32_t* abort_flag) {
  const uint64_t pol = l2_policy_evict_first();  // every cache tile is read once
  const uint32_t bar0 = sbase + SM_BAR;
  uint32_t n = 0, tails = 0;
  bool ok = true;
  Seg s;
  for (long long t = start; ok && next_seg(t, end, p.T, s);) {
    const int l = s.u / kHkv, g = s.u % kHkv;
    for (int j = s.j0; j < s.j1; ++j) {
      if (j == p.T - 1) {  // the block of the new row
        ++tails;
        ok = wait_tail(p, sbase, 0, tails, abort_flag) && wait_tail(p, sbase, 1, tails, abort_flag);
        if (!ok) break;
        fence_proxy_async_global();
      }
      const uint32_t slot = n % kStages, round = n / kStages;
      if (round > 0) {
        ok = bounded_wait(bar0 + 8 * (B_EMPTY + slot), (round - 1) & 1, abort_flag, p.status, kErrF8DecodeWait);
        if (!ok) break;
      }
      const uint32_t fb = bar0 + 8 * (B_FULL + slot), dst = sbase + SM_RING + slot * kStageBytes;
      mbar_expect_tx(fb, kStageBytes);
      tma_load_3d(dst, &p.kmap[l], fb, 0, j * kKeyTile, g, pol);
      tma_load_3d(dst + kTileBytes, &p.vmap[l], fb, 0, j * kKeyTile, g, pol);
      ++n;
    }
  }
  pdl_launch_dependents();
  if (!ok) {  // let every copy already issued land before the CTA gives its shared memory back
    for (uint32_t k = 0; k < static_cast<uint32_t>(kStages) && k < n; ++k) {
      const uint32_t q = n - 1 - k;
      if (!drain_wait(bar0 + 8 * (B_FULL + q % kStages), (q / kStages) & 1)) atomicOr(p.status, kErrDrain);
    }
  }
}

// ------------------------------------------------------------------------------- MMA issuer
// QK(i) needs its tile, its segment's Q, and score buffer i % 4 read by the softmax of tile i - 4 (whose P, and so PV(i - 4), comes
// after that); PV(i) needs P(i) and O buffer i % 2 read out by the output warps (OFREE of tile i - 2).
template <int CAP>
__device__ __noinline__ void mma_issuer(const F8DecodeParams<CAP>& p, uint32_t sbase, uint32_t tmem, long long start, long long end,
                                        volatile uint32_t* abort_flag) {
  const uint32_t bar0 = sbase + SM_BAR;
  // e4m3 is format code 0; S^T: A and B K-major; O^T: A = V MN-major, B = P K-major
  constexpr uint32_t kIdescS = umma_idesc_f16(128, kCols, false, false, false);
  constexpr uint32_t kIdescO = umma_idesc_f16(128, kCols, false, true, false);
  auto bar = [&](int b) { return bar0 + 8 * b; };
  const int total = static_cast<int>(end - start);
  int qk = 0, pv = 0, left = 0, seg = -1;  // tiles issued; QKs of the current segment to come; its number
  long long t = start;
  Seg s;
  uint64_t t0 = 0;
  for (uint32_t it = 0; pv < total;) {
    bool moved = false;
    if (qk < total && qk < pv + 4) {
      if (left == 0) {
        next_seg(t, end, p.T, s);
        left = s.j1 - s.j0;
        ++seg;
      }
      if (mbar_test_wait(bar(B_FULL + qk % kStages), (qk / kStages) & 1) && mbar_test_wait(bar(B_QFULL + (seg & 1)), (seg >> 1) & 1)) {
        const uint32_t ka = sbase + SM_RING + (qk % kStages) * kStageBytes, qt = sbase + SM_QT + (seg & 1) * kOpBytes;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 channels per step
          umma_f8_ss(tmem + TM_S + (qk & 3) * kCols, sw128_desc(ka + kk * 32, 16, 1024), sw128_desc(qt + kk * 32, 16, 1024), kIdescS, kk > 0);
        umma_commit(bar(B_SDONE + (qk & 3)));
        ++qk;
        if (--left == 0) umma_commit(bar(B_QFREE + (seg & 1)));
        moved = true;
      }
    }
    if (pv < qk && mbar_test_wait(bar(B_PFULL + (pv & 1)), (pv >> 1) & 1) &&
        (pv < 2 || mbar_test_wait(bar(B_OFREE + (pv & 1)), ((pv - 2) >> 1) & 1))) {
      const uint32_t va = sbase + SM_RING + (pv % kStages) * kStageBytes + kTileBytes, pt = sbase + SM_PT + (pv & 1) * kOpBytes;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)  // 32 keys per step
        umma_f8_ss(tmem + TM_O + (pv & 1) * kCols, sw128_desc(va + kk * 32 * 128, kTileBytes, 1024), sw128_desc(pt + kk * 32, 16, 1024), kIdescO,
                   kk > 0);
      umma_commit(bar(B_ODONE + (pv & 1)));
      umma_commit(bar(B_EMPTY + pv % kStages));  // K and V of this stage are consumed
      ++pv;
      moved = true;
    }
    if (moved) {
      it = 0;
      t0 = 0;
      continue;
    }
    // bounded like every other wait: the CTA's abort flag, a time limit and a poll limit
    if ((it++ & 63u) == 0) {
      if (*abort_flag) break;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs || it >= 0x7fffffc0u) {
        *abort_flag = 1u;
        atomicOr(p.status, kErrF8DecodeWait);
        break;
      }
    }
  }
  // every MMA issued must be complete before TMEM is released
  umma_commit(bar(B_DRAIN));
  if (!drain_wait(bar(B_DRAIN), 0)) atomicOr(p.status, kErrDrain);
}

// ---------------------------------------------------------------------------- softmax warps
// One set of warps: tiles of this CTA whose number has parity `set`.
template <int CAP>
__device__ __noinline__ void softmax(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, uint32_t tmem, int set, long long start,
                                     long long end, volatile uint32_t* abort_flag) {
  const int tid = threadIdx.x & (kGroup - 1), warp = tid >> 5, lane = tid & 31;  // key of a tile = TMEM lane
  const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16, bar0 = sbase + SM_BAR, id = 1 + set;
  float* red = reinterpret_cast<float*>(smem + SM_RED) + set * 64;
  auto wait = [&](int b, uint32_t parity) { return bounded_wait(bar0 + 8 * b, parity, abort_flag, p.status, kErrF8DecodeWait); };
  uint32_t base = 0, seg = 0, tails = 0;  // this CTA's tiles before the segment, its segments, and appended rows
  Seg s;
  for (long long t = start; next_seg(t, end, p.T, s); ++seg) {
    const int l = s.u / kHkv, g = s.u % kHkv, nt = s.j1 - s.j0;
    const F8AttnLayer& L = p.layer[l];
    const float* ks = L.ks + g * (p.Smax / kScaleBlock + 1) + s.j0;
    float4* scores = p.scores != nullptr && L.w_out != nullptr
                         ? reinterpret_cast<float4*>(p.scores) + (static_cast<size_t>(s.u) * p.T * kKeyTile + static_cast<size_t>(s.j0) * kKeyTile + tid) * 2
                         : nullptr;
    const int last = s.j1 == p.T ? nt - 1 : nt;  // the tile whose scale the appending warp hands over
    tails += s.j1 == p.T ? 1 : 0;
    int i = static_cast<int>((base + set) & 1u);  // (the set's first tile of this segment)
    float k_next = i < last ? ks[i] : 0.f;
    if (seg == 0) {
      prepare_q<1>(p, sbase, smem, s.u, 4 * set + warp, seg, lane);
      bar_sync(id, kGroup);
      if (tid == 0) mbar_arrive(bar0 + 8 * B_QFULL);
    }
    float lsum[kRepText];
#pragma unroll
    for (int h = 0; h < kRepText; ++h) lsum[h] = 0.f;
    float m_run = -INFINITY;  // thread h < 8: head h's reference
    for (; i < nt; i += 2) {
      const uint32_t n = base + i;
      // S(n) is there; the set's P buffer is free, PV(n - 2) being complete
      bool okt = wait(B_SDONE + (n & 3), (n >> 2) & 1);
      if (n >= 2) okt = okt && wait(B_ODONE + set, ((n - 2) >> 1) & 1);
      float k_scale = k_next;
      if (i + 2 < last) k_next = ks[i + 2];
      if (i == last) {
        okt = okt && wait_tail(p, sbase, 0, tails, abort_flag);
        k_scale = reinterpret_cast<const float*>(smem + SM_TAILS)[tails - 1];
      }
      okt = __all_sync(0xffffffffu, okt);
      const bool live = (s.j0 + i) * kKeyTile + tid <= p.pos;
      float x[kRepText];
      if (okt) {
        tc_fence_after();
        uint32_t d[32];
        tmem_ld32(tmem + lane_addr + TM_S + (n & 3) * kCols, d);
        const float4* q4 = reinterpret_cast<const float4*>(smem + SM_QF) + (seg & 7) * 2;
        const float4 qa = q4[0], qb = q4[1];
        const float qf[kRepText] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
        tmem_wait_ld();
        reg_fence32(d);
#pragma unroll
        for (int h = 0; h < kRepText; ++h) {
          const float a = fmaf(__uint_as_float(d[24 + h]), 0x1p-15f, __uint_as_float(d[16 + h]) * 0x1p-10f);
          const float b = fmaf(__uint_as_float(d[8 + h]), 0x1p-5f, a) + __uint_as_float(d[h]);
          x[h] = live ? b * (qf[h] * k_scale) : -INFINITY;
        }
        if (scores != nullptr && live) {
          float4* to = scores + static_cast<size_t>(i) * kKeyTile * 2;
          to[0] = make_float4(x[0], x[1], x[2], x[3]);
          to[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
        float mine = 0.f;
#pragma unroll
        for (int h = 0; h < kRepText; ++h) {
          const float mx = warp_max(x[h]);
          mine = lane == h ? mx : mine;
        }
        if (lane < kRepText) red[(n & 2) * 16 + warp * kRepText + lane] = mine;
        if (!live) {  // a row behind the last one (or past Smax): its V row counts as zero
          const uint32_t v = sbase + SM_RING + (n % kStages) * kStageBytes + kTileBytes + tid * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) st_shared_v4(v + 16 * c, 0u, 0u, 0u, 0u);
        }
      }
      if (!bar_sync_and(id, kGroup, okt)) return;
      float m[kRepText], y[kRepText];
      const float4* r4 = reinterpret_cast<const float4*>(red + (n & 2) * 16);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 a = r4[q], b = r4[2 + q], c = r4[4 + q], d = r4[6 + q];
        m[4 * q] = fmaxf(fmaxf(a.x, b.x), fmaxf(c.x, d.x));
        m[4 * q + 1] = fmaxf(fmaxf(a.y, b.y), fmaxf(c.y, d.y));
        m[4 * q + 2] = fmaxf(fmaxf(a.z, b.z), fmaxf(c.z, d.z));
        m[4 * q + 3] = fmaxf(fmaxf(a.w, b.w), fmaxf(c.w, d.w));
      }
      // weights relative to the tile's largest, times 256, in three pieces
#pragma unroll
      for (int h = 0; h < kRepText; ++h) {
        x[h] = live ? ex2_approx(x[h] - m[h]) : 0.f;
        y[h] = x[h] * 256.0f;
      }
      const uint32_t at = sbase + SM_PT + set * kOpBytes + (tid & 15);
#pragma unroll
      for (int piece = 0; piece < 3; ++piece)
#pragma unroll
        for (int h = 0; h < kRepText; h += 2) {
          const uint32_t c = take_piece(y[h], y[h + 1]);
          st_shared_u8(at + (piece * kRepText + h) * 128 + (((tid >> 4) ^ h) << 4), c);
          st_shared_u8(at + (piece * kRepText + h + 1) * 128 + (((tid >> 4) ^ (h + 1)) << 4), c >> 8);
        }
      float2* fac = reinterpret_cast<float2*>(smem + SM_FAC) + (n & 3) * kRepText;
      if (tid < kRepText) {
        float mt = m[0];
#pragma unroll
        for (int h = 1; h < kRepText; ++h) mt = tid == h ? m[h] : mt;
        const float top = fmaxf(m_run, mt);
        fac[tid] = make_float2(ex2_approx(m_run - top), ex2_approx(mt - top));
        m_run = top;
      }
      fence_proxy_async_smem();  // P, and zeroed V rows, are read by the tensor core
      tc_fence_before();
      bar_sync(id, kGroup);
      if (tid == 0) {
        mbar_arrive(bar0 + 8 * (B_PFULL + set));  // P(n) is out, S(n) read
        mbar_arrive(bar0 + 8 * (B_FAC + (n & 3)));
      }
#pragma unroll
      for (int h = 0; h < kRepText; ++h) {
        const float2 f = fac[h];
        lsum[h] = fmaf(lsum[h], f.x, x[h] * f.y);
      }
    }
    base += nt;
    float* lred = reinterpret_cast<float*>(smem + SM_LRED) + set * 32;
#pragma unroll
    for (int h = 0; h < kRepText; ++h) {
      const float v = warp_sum(lsum[h]);
      if (lane == 0) lred[warp * kRepText + h] = v;
    }
    bar_sync(id, kGroup);
    if (warp == 0) {
      if (lane < kRepText)
        reinterpret_cast<float2*>(smem + SM_FIN)[((seg & 7) * 2 + set) * kRepText + lane] =
            make_float2(m_run, (lred[lane] + lred[kRepText + lane]) + (lred[2 * kRepText + lane] + lred[3 * kRepText + lane]));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar0 + 8 * (B_FIN + (seg & 7)));
    }
    // (lred is written again after a barrier that warp 0 reaches after this read: the next segment's, or that segment's end's)
    bar_sync(id, kGroup);
  }
}

// ----------------------------------------------------------------------------- output warps
template <int CAP>
__device__ __noinline__ void output(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, uint32_t tmem, long long start,
                                    long long end, volatile uint32_t* abort_flag) {
  const int tid = threadIdx.x - 2 * kGroup, warp = tid >> 5;  // channel = TMEM lane
  const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16, bar0 = sbase + SM_BAR;
  volatile uint32_t* merge_flag = reinterpret_cast<volatile uint32_t*>(smem + SM_MERGE);
  auto wait = [&](int b, uint32_t parity) { return bounded_wait(bar0 + 8 * b, parity, abort_flag, p.status, kErrF8DecodeWait); };
  uint32_t n = 0, seg = 0, tails = 0;
  Seg s;
  for (long long t = start; next_seg(t, end, p.T, s); ++seg) {
    const int l = s.u / kHkv, g = s.u % kHkv;
    const F8AttnLayer& L = p.layer[l];
    const float* vs = L.vs + g * (p.Smax / kScaleBlock + 1);
    const int last = s.j1 == p.T ? p.T - 1 : s.j1;  // the tile whose scale the appending warp hands over
    tails += s.j1 == p.T ? 1 : 0;
    float v_next = s.j0 < last ? vs[s.j0] : 0.f;
    float sums[2][kRepText];  // each softmax set's tiles, relative to its own reference
#pragma unroll
    for (int h = 0; h < kRepText; ++h) sums[0][h] = sums[1][h] = 0.f;
    for (int j = s.j0; j < s.j1; ++j, ++n) {
      bool okt = wait(B_FAC + (n & 3), (n >> 2) & 1);  // the tile's factors are there,
      okt = okt && wait(B_ODONE + (n & 1), (n >> 1) & 1);  // and its O
      float v_scale = v_next;
      if (j + 1 < last) v_next = vs[j + 1];
      if (j == last) {
        okt = okt && wait_tail(p, sbase, 1, tails, abort_flag);
        v_scale = reinterpret_cast<const float*>(smem + SM_TAILS)[kTails + tails - 1];
      }
      okt = __all_sync(0xffffffffu, okt);
      if (okt) {
        tc_fence_after();
        uint32_t d[32];
        tmem_ld32(tmem + lane_addr + TM_O + (n & 1) * kCols, d);
        tmem_wait_ld();
        reg_fence32(d);
        const float4* fac = reinterpret_cast<const float4*>(smem + SM_FAC) + (n & 3) * (kRepText / 2);
        const float vf = v_scale * 0x1p-8f;
        auto add = [&](float (&a)[kRepText]) {
#pragma unroll
          for (int h = 0; h < kRepText; h += 2) {
            const float4 f = fac[h / 2];
            const float o0 = fmaf(__uint_as_float(d[16 + h]), 0x1p-10f, __uint_as_float(d[8 + h]) * 0x1p-5f) + __uint_as_float(d[h]);
            const float o1 = fmaf(__uint_as_float(d[17 + h]), 0x1p-10f, __uint_as_float(d[9 + h]) * 0x1p-5f) + __uint_as_float(d[h + 1]);
            a[h] = fmaf(a[h], f.x, o0 * (f.y * vf));
            a[h + 1] = fmaf(a[h + 1], f.z, o1 * (f.w * vf));
          }
        };
        if (n & 1) add(sums[1]);
        else add(sums[0]);
        tc_fence_before();
      }
      if (!bar_sync_and(3, kGroup, okt)) return;
      if (tid == 0) mbar_arrive(bar0 + 8 * (B_OFREE + (n & 1)));
    }
    // ---- the segment's end: its sums, then its output or its part of one
    if (!bar_sync_and(3, kGroup, wait(B_FIN + (seg & 7), (seg >> 3) & 1))) return;
    const float2* fin = reinterpret_cast<const float2*>(smem + SM_FIN) + (seg & 7) * 2 * kRepText;
    float acc[kRepText];
    float2 mine = make_float2(0.f, 1.f);  // thread h < 8: head h's reference and sum
#pragma unroll
    for (int h = 0; h < kRepText; ++h) {
      const float2 a = fin[h], b = fin[kRepText + h];
      const float top = fmaxf(a.x, b.x), fa = ex2_approx(a.x - top), fb = ex2_approx(b.x - top);
      acc[h] = fmaf(sums[0][h], fa, sums[1][h] * fb);
      if (tid == h) mine = make_float2(top, fmaf(a.y, fa, b.y * fb));
    }
    if (s.j0 == 0 && s.j1 == p.T) {
      float* inv = reinterpret_cast<float*>(smem + SM_SW);
      if (tid < kRepText) {
        inv[tid] = 1.0f / mine.y;
        if (p.scores != nullptr) p.lse[s.u * kRepText + tid] = mine.x + log2f(mine.y);
      }
      bar_sync(3, kGroup);
      __nv_bfloat16* o = L.out + static_cast<size_t>(kRepText * g) * kD + tid;
#pragma unroll
      for (int h = 0; h < kRepText; ++h) o[h * kD] = __float2bfloat16_rn(acc[h] * inv[h]);
      bar_sync(3, kGroup);  // read before they are written again
      continue;
    }
    // Part index: 2 c + slot (a part is its CTA's first segment or its last). Layout [part][channel][8 heads].
    const int slot = seg == 0 ? 0 : 1;
    const size_t ps = static_cast<size_t>(blockIdx.x) * 2 + slot;
    float4* po = reinterpret_cast<float4*>(p.part_o + ps * kRepText * kD) + 2 * tid;
    po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (tid < kRepText) *reinterpret_cast<float2*>(p.part_ml + (ps * kRepText + tid) * 2) = mine;
    bar_sync(3, kGroup);
    const long long u0 = static_cast<long long>(s.u) * p.T;
    const int c0 = cta_of_tile(u0, p.W, gridDim.x), c1 = cta_of_tile(u0 + p.T - 1, p.W, gridDim.x);
    // the count's release publishes this part, and the last part's acquire orders the others' before its reads
    if (tid == 0) *merge_flag = atom_add_acq_rel_gpu(p.unit_cnt + s.u, 1u) == static_cast<uint32_t>(c1 - c0) ? 1u : 0u;
    bar_sync(3, kGroup);
    if (*merge_flag) {
      const int np = c1 - c0 + 1;
      const int slot0 = cta_tile_start(c0, p.W, gridDim.x) >= u0 ? 0 : 1;  // the first part may be its CTA's last segment
      auto part_index = [&](int k) -> size_t { return static_cast<size_t>(c0 + k) * 2 + (k == 0 ? slot0 : 0); };
      // weights 2^(m_k - M) / L of the parts, 16 threads a head
      float* sw = reinterpret_cast<float*>(smem + SM_SW);  // [part][head]
      {
        constexpr int kPer = kMaxParts / 16;
        const int h = tid >> 4, i = tid & 15;
        float2 ml[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int k = i + 16 * e;
          ml[e] = k < np ? __ldcg(reinterpret_cast<const float2*>(p.part_ml + (part_index(k) * kRepText + h) * 2)) : make_float2(-INFINITY, 0.f);
        }
        float M = -INFINITY;
#pragma unroll
        for (int e = 0; e < kPer; ++e) M = fmaxf(M, ml[e].x);
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          ml[e].x = i + 16 * e < np ? ex2_approx(ml[e].x - M) : 0.f;
          sum = fmaf(ml[e].y, ml[e].x, sum);
        }
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float inv = 1.0f / sum;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (i + 16 * e < np) sw[(i + 16 * e) * kRepText + h] = ml[e].x * inv;
        if (p.scores != nullptr && i == 0) p.lse[s.u * kRepText + h] = M + log2f(sum);
      }
      bar_sync(3, kGroup);
#pragma unroll
      for (int h = 0; h < kRepText; ++h) acc[h] = 0.f;
      const float4* sw4 = reinterpret_cast<const float4*>(sw);
      // from L2, kMergeBatch parts per round of independent 16-byte loads
      for (int cb = 0; cb < np; cb += kMergeBatch) {
        float4 v[kMergeBatch][2];
#pragma unroll
        for (int b = 0; b < kMergeBatch; ++b) {
          const int k = min(cb + b, np - 1);  // past the last part: a repeat, unused
          const float4* src = reinterpret_cast<const float4*>(p.part_o + part_index(k) * kRepText * kD) + 2 * tid;
          v[b][0] = __ldcg(src);
          v[b][1] = __ldcg(src + 1);
        }
#pragma unroll
        for (int b = 0; b < kMergeBatch; ++b)
          if (cb + b < np) {
            const float4 w0 = sw4[2 * (cb + b)], w1 = sw4[2 * (cb + b) + 1];
            acc[0] = fmaf(w0.x, v[b][0].x, acc[0]);
            acc[1] = fmaf(w0.y, v[b][0].y, acc[1]);
            acc[2] = fmaf(w0.z, v[b][0].z, acc[2]);
            acc[3] = fmaf(w0.w, v[b][0].w, acc[3]);
            acc[4] = fmaf(w1.x, v[b][1].x, acc[4]);
            acc[5] = fmaf(w1.y, v[b][1].y, acc[5]);
            acc[6] = fmaf(w1.z, v[b][1].z, acc[6]);
            acc[7] = fmaf(w1.w, v[b][1].w, acc[7]);
          }
      }
#pragma unroll
      for (int h = 0; h < kRepText; ++h) L.out[static_cast<size_t>(kRepText * g + h) * kD + tid] = __float2bfloat16_rn(acc[h]);
      if (tid == 0) p.unit_cnt[s.u] = 0u;  // every part has arrived: ready for the next call
    }
    bar_sync(3, kGroup);  // the flag is read before the next segment overwrites it
  }
}

}  // namespace f8d

template <int CAP>
__global__ void __launch_bounds__(f8d::kThreads, 1) fp8_decode_kernel(const __grid_constant__ F8DecodeParams<CAP> p) {
  using namespace f8d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + SM_BAR;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + SM_ABORT);
  const long long start = cta_tile_start(blockIdx.x, p.W, gridDim.x), end = cta_tile_start(blockIdx.x + 1, p.W, gridDim.x);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    // (Q comes from two warps, or two sets; a segment's end from both sets)
    for (int b = 0; b < kNumBars; ++b)
      mbar_init(bar0 + 8 * b, (b >= B_QFULL && b < B_QFULL + 2) || (b >= B_FIN && b < B_FIN + 8) ? 2 : 1);
    *abort_flag = 0u;
    reinterpret_cast<uint32_t*>(smem + SM_TAILN)[0] = 0u;
    reinterpret_cast<uint32_t*>(smem + SM_TAILN)[1] = 0u;
    fence_mbar_init();
  }
  if (threadIdx.x < kD / 2) reinterpret_cast<float4*>(smem + SM_ROT)[threadIdx.x] = p.rot[threadIdx.x];
  // rows 24-31 of both P operands are the padding of N = 32
  if (threadIdx.x >= 128 && threadIdx.x < 256) {
    const uint32_t i = threadIdx.x - 128;
    st_shared_v4(sbase + SM_PT + (i >> 6) * kOpBytes + 24 * 128 + (i & 63) * 16, 0u, 0u, 0u, 0u);
  }
  if (warp == 0) {
    tmem_alloc(sbase + SM_TMEM, kTmemCols);
    tmem_relinquish();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + SM_TMEM);
  if (warp == 13 && (threadIdx.x & 31) == 0) {
    // hints, while the kernel before finishes (what it still writes wins): the maps, and the first tiles into L2
    if (start < end) {
      const int l = static_cast<int>(start / p.T) / kHkv;
      prefetch_tensormap(&p.kmap[l]);
      prefetch_tensormap(&p.vmap[l]);
    }
    for (long long x = start; x < end && x < start + kStages; ++x) {
      const int u = static_cast<int>(x / p.T), j = static_cast<int>(x - static_cast<long long>(u) * p.T);
      const size_t off = (static_cast<size_t>(u % kHkv) * p.Smax + static_cast<size_t>(j) * kKeyTile) * kD;
      prefetch_l2_bulk(p.layer[u / kHkv].kc + off, kTileBytes);
      prefetch_l2_bulk(p.layer[u / kHkv].vc + off, kTileBytes);
    }
  }
  // everything below reads what earlier kernels in the stream wrote
  pdl_wait_primary();
  if (warp < 8) {
    softmax(p, sbase, smem, tmem, warp >> 2, start, end, abort_flag);
  } else if (warp < 12) {
    output(p, sbase, smem, tmem, start, end, abort_flag);
  } else if (warp == 12) {
    if ((threadIdx.x & 31) == 0) producer(p, sbase, start, end, abort_flag);
  } else if (warp == 13) {
    if ((threadIdx.x & 31) == 0) mma_issuer(p, sbase, tmem, start, end, abort_flag);
  } else {
    prepare(p, sbase, smem, warp - 14, start, end, abort_flag);
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Weights from the scores: thread = key of one unit. grid (key blocks, units)
template <int CAP>
__global__ void __launch_bounds__(256) fp8_weights_kernel(const __grid_constant__ F8DecodeParams<CAP> p) {
  const int u = blockIdx.y, key = blockIdx.x * 256 + threadIdx.x;
  const F8AttnLayer& L = p.layer[u / kHkv];
  pdl_wait_primary();
  pdl_launch_dependents();
  if (L.w_out == nullptr || key > p.pos) return;
  const float4* x = reinterpret_cast<const float4*>(p.scores) + (static_cast<size_t>(u) * p.T * kKeyTile + key) * 2;
  const float4* lse = reinterpret_cast<const float4*>(p.lse + u * kRepText);
  const float4 a = __ldcs(x), b = __ldcs(x + 1), c = lse[0], d = lse[1];
  const size_t at = static_cast<size_t>(u % kHkv) * p.Smax + key;
  const float w = key < p.pos && L.w_in != nullptr ? L.w_in[at] : 0.f;
  const float sum = ((ex2_approx(a.x - c.x) + ex2_approx(a.y - c.y)) + (ex2_approx(a.z - c.z) + ex2_approx(a.w - c.w))) +
                    ((ex2_approx(b.x - d.x) + ex2_approx(b.y - d.y)) + (ex2_approx(b.z - d.z) + ex2_approx(b.w - d.w)));
  L.w_out[at] = w + sum;
}

cudaError_t fp8_decode_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(fp8_decode_kernel<kSmallCap>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(f8d::kSmemBytes));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fp8_decode_kernel<kDecodeMaxLayers>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(f8d::kSmemBytes));
  return e;
}

template <int CAP>
cudaError_t launch_fp8_decode(const F8DecodeParams<CAP>& p, cudaLaunchConfig_t cfg) {
  if (p.n_layers * kHkv / static_cast<int>(cfg.gridDim.x) + 2 > f8d::kTails) return cudaErrorInvalidConfiguration;  // (a GPU of 7 SMs)
  cfg.blockDim = dim3(f8d::kThreads);
  cfg.dynamicSmemBytes = f8d::kSmemBytes;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_decode_kernel<CAP>, p);
  if (e != cudaSuccess || p.scores == nullptr) return e;
  cfg.gridDim = dim3(p.pos / 256 + 1, p.n_layers * kHkv);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fp8_weights_kernel<CAP>, p);
}
template cudaError_t launch_fp8_decode<kSmallCap>(const F8DecodeParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode<kDecodeMaxLayers>(const F8DecodeParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);

}  // namespace ea
