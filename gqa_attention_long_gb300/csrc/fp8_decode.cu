// fp8_decode.cu — the text model's decode step over an 8-bit cache, on the tensor cores (tcgen05, e4m3 operands).
//
// Per layer and kv head (a unit): 8 query rows against rows [0, pos], the new row appended first. A unit's keys are cut into
// tiles of 128, which are the cache's blocks, so that a tile has one scale for K and one for V; the tiles of all units are cut into
// one contiguous range per CTA. HBM bounds it (16 flop a byte), if what is done to a tile stays well under the 0.73 us in which an
// SM's share of the bandwidth brings one.
//
// The codes go to the tensor cores as they are, K's as the rows of one product and V's as the columns of the next, and no value is
// ever widened. What they meet has more bits than a code: it comes in pieces. A number y, |y| <= 256, is c0 + c1 / 32 + c2 / 1024 + ..,
// each c the e4m3 number next to 32 times what the pieces before left. A code has four bits: what it leaves of a y in [2^e, 2^(e+1)) is at
// most 2^(e-4), so that four pieces hold a q row to 2^-19 of its largest channel (scores that weights come from: fp32 would be
// 2^-24). A softmax weight has three, c0 + (c1 + c2) / 32, the last of which is the e4m3 number next to what c1 leaves as it is: a weight is held
// to 2^-14 of itself down to 2^-9 of the tile's largest, and to 2^-23 of that below. (With two, 2^-9 of itself, the
// bf16 output's error was 1.71e-3 of it, not 1.66e-3, and outputs that cancel were off by up to 2^-10 of what they come from.) Products of
// codes are exact, sums are in fp32, and pieces are columns that the MMA has to spare: 8 heads in 4 pieces are N = 32 (up to 64
// columns an MMA takes the same 46 cycles).
//   S^T  = K Q^T    M = 128 keys, N = 32 (half of the heads, piece, head), K = 128 channels; A = the K tile (K-major)
//   O^T  = V^T P^T  M = 128 channels, N = 32 (c0, c1, zeros, c2 by head), K = 128 keys; A = the V tile (MN-major). Where weights
//                   are formed (below), which takes the columns, N = 16: c0 and c1, then zeros and c2 into the same ones (a second set of
//                   MMAs, 2 us of 123 for 64 layers at pos 4700)
// Each tile's weights are taken relative to its own largest score, and its O^T is read out and added, times its share and V's scale, in
// fp32: whatever scales and maxima the other tiles have, none of it is rounded away.
//
// Warp roles (512 threads): warps 0-3 and 4-7 softmax, of heads 0-3 and 4-7 (thread = key = TMEM lane); warps 8-11 output
// (thread = channel = TMEM lane): sums of O^T, a segment's end, the merge; warp 12 loads tiles by TMA, K's into a ring of 4, V's, which
// are held longer, into one of 8; warps 13 and 14 issue the MMAs, one product each; warp 15 prepares what later segments need: their Q, and
// the new K and V rows, which it appends (the first segment's Q comes from the softmax warps, its new rows and the second segment's Q from
// output warps, which have nothing else to do yet). S has four buffers, Q, P and O have two. Five loops run side by side on one scheduler's instruction cache, and fetching
// was what they waited for most (2.8 of 10 warp cycles an instruction): they are short, and what is rare is out of their way.
// A unit cut over several CTAs is merged by the part that finishes last; a part that is not its CTA's last segment is counted by warp
// 15, and merged at the CTA's end should it be the last after all, so that the output warps need not wait. A CTA's last part of a unit of
// two whose other part has come adds that to its registers' sums (64 layers at pos 4700: 1.6 us less than through global memory).
// Weights that are asked for need a unit's scores once more when its log2-sum-exps are known: 32 bytes a key. They go to the workspace, and
// a second kernel forms the weights; or, where most units are whole ones of one CTA, these stay in tensor memory, whose columns hold 44 tiles'
// scores beside the accumulators, and the output warps form their weights between the next unit's tiles (64 layers at pos 4700: 122.5 us, not
// 133.6); the cut ones' are formed by the CTA that merges them. What that takes is the loads' latency (sums before come through
// prefetches and asynchronous copies: 10 us less) rather than the arithmetic.
// Figures (64 layers at pos 4700; 4 layers at pos 131070): 100.0 and 163 us, 91 % and 97 % of the copy's rate; the former's 125 tiles
// a CTA bear a start and an end of about 6 us. A unit has a chain of its own (its Q from one warp, its first scores, its end) of about 5 us, which
// the tiles of short units do not hide: 64 layers at pos 1000 40.1 us, at pos 380 28.1, two and three and a half times their bytes' time.
#include "fp8.cuh"

namespace ea {
namespace f8d {

constexpr int kThreads = 512;
constexpr int kGroup = 128;  // threads of either set of softmax warps, and of the output warps
constexpr int kOutWarp = 8;  // the first of the output warps
constexpr int kKRing = 4, kVRing = 8;
constexpr uint32_t kTileBytes = kKeyTile * kD;      // a K or a V tile: 128 rows of 128 bytes, 128-byte swizzle
constexpr int kCols = 32;                           // N of the first product
constexpr uint32_t kOpBytes = kCols * 128;          // Q: 32 rows of 128 bytes
constexpr uint32_t kPiece = kRepText * 128;         // a piece of P: a row for each head
constexpr uint32_t kPBytes = 4 * kPiece;            // P: c0, c1, zeros, c2
constexpr int kMaxParts = 160;                      // parts of one unit (at most one per CTA)
constexpr int kMergeBatch = 4;
constexpr int kWeigh = 4;  // tiles whose weights the output warps form at a time
constexpr int kTails = 72;                          // units of one CTA, at most
// Shared memory (offsets from the 1024-byte-aligned base)
constexpr uint32_t SM_K = 0;
constexpr uint32_t SM_V = SM_K + kKRing * kTileBytes;
constexpr uint32_t SM_QT = SM_V + kVRing * kTileBytes;           // 2 buffers
constexpr uint32_t SM_PT = SM_QT + 2 * kOpBytes;                 // 2 buffers
constexpr uint32_t SM_ROT = SM_PT + 2 * kPBytes;                // float4 [64]
constexpr uint32_t SM_RED = SM_ROT + (kD / 2) * 16;              // [2][8 warps][4 heads]
constexpr uint32_t SM_FAC = SM_RED + 2 * 8 * 4 * 4;              // [4][8 heads]: (what the sums before are multiplied by, the tile's share)
constexpr uint32_t SM_FIN = SM_FAC + 4 * kRepText * 8;           // [8 segments][8 heads]: (reference, sum)
constexpr uint32_t SM_QF = SM_FIN + 8 * kRepText * 8;            // [8 segments][8]: what a head's S columns are multiplied by (read up to four tiles after the last QK)
constexpr uint32_t SM_LRED = SM_QF + 8 * kRepText * 4;           // [8 warps][4 heads]
constexpr uint32_t SM_TAILS = SM_LRED + 8 * 4 * 4;    // [K, V][kTails]: the appended block's scale
constexpr uint32_t SM_SW = SM_TAILS + 2 * kTails * 4;            // merge weights [part][head]
constexpr uint32_t SM_UNIT = SM_SW + kMaxParts * kRepText * 4;   // WeighUnit
constexpr uint32_t SM_SUMS = SM_UNIT + 48;                       // sums before: [kWeigh][128]
constexpr uint32_t SM_BAR = SM_SUMS + kWeigh * kKeyTile * 4;
// PFULL, ODONE, OFREE: one barrier per parity of the tile count; SDONE: per S buffer; QFULL, QFREE: per Q buffer. The softmax warps
// can be two tiles, and so three segments, ahead of the output warps: what those wait for from them has as many barriers (FAC by
// tile, FIN by segment) as it takes for none to complete twice unseen. FAC also tells that a tile's S buffer has been read.
constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + kKRing, B_VFULL = B_KEMPTY + kKRing, B_VEMPTY = B_VFULL + kVRing, B_SDONE = B_VEMPTY + kVRing, B_PFULL = B_SDONE + 4, B_ODONE = B_PFULL + 2,
              B_OFREE = B_ODONE + 2, B_QFULL = B_OFREE + 2, B_QFREE = B_QFULL + 2, B_FAC = B_QFREE + 2, B_FIN = B_FAC + 4,
              B_DRAIN = B_FIN + 8, B_PART = B_DRAIN + 2, B_LATE = B_PART + 1, B_TAIL = B_LATE + 1, kNumBars = B_TAIL + 2 * kTails;  // TAIL: [K, V][unit], whose new row is in place
constexpr uint32_t SM_TMEM = SM_BAR + kNumBars * 8;
constexpr uint32_t SM_MERGE = SM_TMEM + 4;
constexpr uint32_t SM_TODO = SM_MERGE + 4;  // [2]: merged units whose weights are still to be formed (or -1)
constexpr uint32_t SM_LASTPART = SM_TODO + 8;  // whether the other part of the unit that the last segment begins is there already
constexpr uint32_t kSmemBytes = SM_LASTPART + 4 + 1024;  // + base alignment
static_assert(kSmemBytes <= 232448, "shared memory budget of one sm_103 CTA");
// 4 and 2 buffers of 32 columns (O: 16 in kForm); there, then, the scores of kKept tiles, 8 columns each
constexpr uint32_t kTmemCols = 512, TM_S = 0, TM_O = 128, TM_X = 160, kKept = (kTmemCols - TM_X) / 8;
// (kForm) Tile n's scores take the place of tile n - kKept's. Who writes them knows that output warps have read out O of tile n - 4, and have so
// formed the weights that go with tile n - 5's. They form those of tiles 4 k .. 4 k + 3 of a unit of T tiles beside tile T + k, both counted from
// its first: T + k <= 4 k + kKept - 5 for every k.
static_assert(kF8KeptTiles + 5 <= static_cast<int>(kKept), "scores are read before others take their place");

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

// What becomes of the weights: none is asked for; scores go to the workspace, for a second kernel; or this one forms them, of whole units
// from scores that it keeps in tensor memory.
constexpr int kNoWeights = 0, kScores = 1, kForm = 2;
constexpr int out_cols(int mode) { return mode == kForm ? 16 : 32; }  // N of the second product
// Whether the CTA whose segment s is keeps its unit's scores (kForm).
template <class P>
__device__ __forceinline__ bool kept_unit(const P& p, const Seg& s) {
  return s.j0 == 0 && s.j1 == p.T;
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
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t* a) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// The waits of this file are a whole warp's and take little code: one look here, and the further ones (counted_wait, which gives up after a
// number of them) out of the loops' way: 64 layers at pos 4700 107 -> 100 us. Who gives up notes it and leaves, and then so does, the
// same number of looks later, who waits for it.
__device__ __noinline__ bool long_wait(uint32_t bar, uint32_t parity) { return counted_wait(bar, parity); }
__device__ __forceinline__ bool short_wait(uint32_t bar, uint32_t parity) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
  return long_wait(bar, parity);
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float (&x)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(__float_as_uint(x[0])),
               "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3]))
               : "memory");
}
// 16 consecutive TMEM columns of this warp's 32 lanes -> 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// tcgen05.wait::ld, after which (and not before) the registers of the loads are used.
__device__ __forceinline__ void tmem_landed16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Two numbers' next piece: the pair of codes, and what it leaves, times `finer`.
__device__ __forceinline__ uint32_t take_piece(float& a, float& b, float finer = 32.0f) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(a), "f"(b));
  const float2 f = unpack_f16x2(cvt_f16x2_e4m3x2(c));
  a = (a - f.x) * finer;
  b = (b - f.y) * finer;
  return c;
}

// ------------------------------------------------------------------------ preparing segments
// One warp appends unit u's new K (kv = 0) or V row: the CTA's idx-th.
template <int CAP>
__device__ __noinline__ void append_row(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, int kv, int u, uint32_t idx) {
  const int lane = threadIdx.x & 31, g = u % kHkv;
  const float4* rot = reinterpret_cast<const float4*>(smem + SM_ROT);
  const int blk = p.pos / kScaleBlock, before = p.pos % kScaleBlock;
  const F8AttnLayer& L = p.layer[u / kHkv];
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
  if (lane == 0) reinterpret_cast<float*>(smem + SM_TAILS)[kv * kTails + idx] = now;
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(sbase + SM_BAR + 8 * (B_TAIL + kv * kTails + idx));
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

// q rows [h, h1) of segment seg's unit, as pieces, into its Q buffer: one warp, which loads a row ahead (64 layers at pos 1000, whose units are
// eight tiles: 42.3 -> 39.6 us).
template <int CAP>
__device__ __noinline__ void prepare_q(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, int u, int h, int h1, uint32_t seg) {
  const int lane = threadIdx.x & 31;
  const F8AttnLayer& L = p.layer[u / kHkv];
  const __nv_bfloat16* q = L.q_raw + kRepText * (u % kHkv) * kD;
  float next[4], gm[4];
  f8_load_row(L.q_gamma, lane, gm);
  f8_load_row(q + h * kD, lane, next);
#pragma unroll 1
  for (; h < h1; ++h) {
    float x[4] = {next[0], next[1], next[2], next[3]}, y[4];
    if (h + 1 < h1) f8_load_row(q + (h + 1) * kD, lane, next);
    f8_norm_rope(x, gm, reinterpret_cast<const float4*>(smem + SM_ROT), lane, y);
    const int e = f16_exponent(f8_row_max(y));  // the row's largest magnitude is in [2^e, 2^(e + 1)): put it in [128, 256)
    const float up = f8_pow2(min(7 - e, 126));
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fmaf(y[i], up, y[i] * 0.0f);  // (an infinity is NaN: as codes it would saturate)
    if (lane == 0) reinterpret_cast<float*>(smem + SM_QF)[(seg & 7) * kRepText + h] = p.scale_log2 * f8_pow2(max(e - 7, -126));  // over up
    // 16-byte chunk c of row r at chunk c ^ (r % 8)
    const uint32_t r0 = (h >> 2) * 16 + (h & 3), c = lane >> 3;
    uint32_t row = sbase + SM_QT + (seg & 1) * kOpBytes + r0 * 128 + ((2 * lane) & 15);
#pragma unroll
    for (int piece = 0; piece < 4; ++piece, row += 4 * 128) {
      const uint32_t r = (r0 + 4 * piece) & 7, lo = take_piece(y[0], y[1]), hi = take_piece(y[2], y[3]);
      st_shared_u16(row + ((c ^ r) << 4), static_cast<uint16_t>(lo));
      st_shared_u16(row + (((c + 4) ^ r) << 4), static_cast<uint16_t>(hi));
    }
  }
  fence_proxy_async_smem();  // read by the tensor core
}

// Counts a part of unit u whose partial the calling thread has seen written; whether it was the last one. (The count's release
// publishes the partial, its acquire orders the others' before what follows.)
template <class P>
__device__ __forceinline__ bool count_part(const P& p, int u) {
  const long long u0 = static_cast<long long>(u) * p.T;
  const int parts = cta_of_tile(u0 + p.T - 1, p.W, gridDim.x) - cta_of_tile(u0, p.W, gridDim.x) + 1;
  return atom_add_acq_rel_gpu(p.unit_cnt + u, 1u) == static_cast<uint32_t>(parts - 1);
}

// Whether segment s, after which t is the next tile, is the first of a unit's two parts and the CTA's last segment, with a Q that warp 15
// prepares: it then looks whether the other part, which its CTA began with, has arrived. If so nobody else will merge the unit, and this CTA
// need not write its part, count it and read it again.
template <class P>
__device__ __forceinline__ bool last_part(const P& p, const Seg& s, uint32_t seg, long long t, long long end) {
  return seg > 1 && t >= end && s.j0 == 0 && s.j1 < p.T &&
         cta_tile_start(blockIdx.x + 2, p.W, gridDim.x) >= static_cast<long long>(s.u + 1) * p.T;
}

// One warp: the Q and the new rows of every segment but the first.
template <int CAP>
__device__ __forceinline__ bool prepare(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, long long start, long long end) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar0 = sbase + SM_BAR;
  uint32_t idx = 0, seg = 0;
  int first = -1;  // the first segment's unit, if that is a part, and not the last segment: its partial is counted here
  Seg s;
#pragma unroll 1
  for (long long t = start;; ++seg) {
    const bool more = next_seg(t, end, p.T, s);
    if (first >= 0 && (seg > 2 || !more)) {  // (the third segment's Q was prepared when the first one's products were done)
      const bool ok = counted_wait(bar0 + 8 * B_PART, 0);
      if (lane == 0) {
        *reinterpret_cast<volatile uint32_t*>(smem + SM_MERGE) = ok && count_part(p, first) ? 1u : 0u;
        mbar_arrive(bar0 + 8 * B_LATE);
      }
      if (!ok) return false;
      first = -1;
    }
    if (!more) return true;
    if (seg == 0 && t < end && !(s.j0 == 0 && s.j1 == p.T)) first = s.u;
    if (seg > 0) {
      if (seg > 1) {  // (output warps have the second one's Q)
        const uint32_t buf = seg & 1;
        if (!counted_wait(bar0 + 8 * (B_QFREE + buf), ((seg - 2) >> 1) & 1)) return false;
        prepare_q(p, sbase, smem, s.u, 0, kRepText, seg);
        if (lane == 0 && last_part(p, s, seg, t, end))
          *reinterpret_cast<volatile uint32_t*>(smem + SM_LASTPART) = ld_acquire_gpu(p.unit_cnt + s.u);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar0 + 8 * (B_QFULL + buf));
      }
      if (s.j1 == p.T) {
        append_row(p, sbase, smem, 0, s.u, idx);
        append_row(p, sbase, smem, 1, s.u, idx);
      }
    }
    idx += s.j1 == p.T ? 1 : 0;
  }
}

// ---------------------------------------------------------------- producer and MMA issuers
// Each is a whole warp of which one elected lane issues, so that operands sit in the warp's uniform registers, which these instructions
// take (from a lone lane's registers each is moved over first: an MMA then takes 130 cycles to issue, and one warp that
// issued both products took 1,700 cycles a tile).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <int CAP>
__device__ __forceinline__ bool producer(const F8DecodeParams<CAP>& p, uint32_t sbase, long long start, long long end) {
  const uint64_t pol = l2_policy_evict_first();  // every cache tile is read once
  const uint32_t bar0 = sbase + SM_BAR;
  auto wait = [&](int b, uint32_t parity) { return short_wait(bar0 + 8 * b, parity); };
  uint32_t nk = 0, nv = 0, tails = 0;  // tiles of K and of V on their way
  bool ok = true;
  Seg s;
  for (long long t = start; ok && next_seg(t, end, p.T, s);) {
    const int l = s.u / kHkv, g = s.u % kHkv;
    for (int j = s.j0; j < s.j1; ++j) {
      const bool tail = j == p.T - 1;  // the block of the new row
      if (tail) ok = wait(B_TAIL + tails, 0);
      if (nk >= kKRing) ok = ok && wait(B_KEMPTY + nk % kKRing, (nk / kKRing - 1) & 1);
      if (!ok) break;
      if (tail) fence_proxy_async_global();
      if (elect_one()) {
        const uint32_t fb = bar0 + 8 * (B_KFULL + nk % kKRing);
        mbar_expect_tx(fb, kTileBytes);
        tma_load_3d(sbase + SM_K + nk % kKRing * kTileBytes, &p.kmap[l], fb, 0, j * kKeyTile, g, pol);
      }
      __syncwarp();
      ++nk;
      if (tail) ok = wait(B_TAIL + kTails + tails, 0);
      if (nv >= kVRing) ok = ok && wait(B_VEMPTY + nv % kVRing, (nv / kVRing - 1) & 1);
      if (!ok) break;
      if (tail) fence_proxy_async_global();
      if (elect_one()) {
        const uint32_t fb = bar0 + 8 * (B_VFULL + nv % kVRing);
        mbar_expect_tx(fb, kTileBytes);
        tma_load_3d(sbase + SM_V + nv % kVRing * kTileBytes, &p.vmap[l], fb, 0, j * kKeyTile, g, pol);
      }
      __syncwarp();
      ++nv;
      tails += tail ? 1 : 0;
    }
  }
  pdl_launch_dependents();
  if (!ok && elect_one()) {  // let every copy already issued land before the CTA gives its shared memory back
    for (uint32_t k = 1; k <= static_cast<uint32_t>(kKRing) && k <= nk; ++k)
      if (!drain_wait(bar0 + 8 * (B_KFULL + (nk - k) % kKRing), ((nk - k) / kKRing) & 1)) atomicOr(p.status, kErrDrain);
    for (uint32_t k = 1; k <= static_cast<uint32_t>(kVRing) && k <= nv; ++k)
      if (!drain_wait(bar0 + 8 * (B_VFULL + (nv - k) % kVRing), ((nv - k) / kVRing) & 1)) atomicOr(p.status, kErrDrain);
  }
  __syncwarp();
  return ok;
}

// QK(n) needs its tile, its segment's Q, and score buffer n % 4 read by the softmax of tile n - 4.
template <int CAP>
__device__ __forceinline__ bool qk_issuer(const F8DecodeParams<CAP>& p, uint32_t sbase, uint32_t tmem, long long start, long long end) {
  constexpr uint32_t kIdesc = umma_idesc_f16(128, kCols, false, false, false);  // (e4m3 is format code 0); A and B K-major
  const uint32_t bar0 = sbase + SM_BAR;
  const uint64_t kd = sw128_desc(sbase + SM_K, 16, 1024), qd = sw128_desc(sbase + SM_QT, 16, 1024);
  auto wait = [&](int b, uint32_t parity) { return short_wait(bar0 + 8 * b, parity); };
  uint32_t n = 0, seg = 0;
  bool ok = true;
  Seg s;
  for (long long t = start; ok && next_seg(t, end, p.T, s); ++seg) {
    ok = wait(B_QFULL + (seg & 1), (seg >> 1) & 1);
#pragma unroll 1
    for (int i = s.j1 - s.j0; ok && i > 0; --i, ++n) {
      ok = wait(B_KFULL + n % kKRing, (n / kKRing) & 1) && (n < 4 || wait(B_FAC + (n & 3), ((n - 4) >> 2) & 1));
      if (!ok) break;
      tc_fence_after();
      const uint64_t k0 = kd + n % kKRing * (kTileBytes >> 4), q0 = qd + (seg & 1) * (kOpBytes >> 4);
      const uint32_t d = tmem + TM_S + (n & 3) * kCols;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f8_ss(d, k0 + 2 * kk, q0 + 2 * kk, kIdesc, kk > 0);  // 32 channels per step
        umma_commit(bar0 + 8 * (B_SDONE + (n & 3)));
        umma_commit(bar0 + 8 * (B_KEMPTY + n % kKRing));
        if (i == 1) umma_commit(bar0 + 8 * (B_QFREE + (seg & 1)));
      }
      __syncwarp();
    }
  }
  if (elect_one()) {  // every MMA issued must be complete before TMEM is released
    umma_commit(bar0 + 8 * B_DRAIN);
    if (!drain_wait(bar0 + 8 * B_DRAIN, 0)) atomicOr(p.status, kErrDrain);
  }
  __syncwarp();
  return ok;
}

// PV(n) needs its tile, P(n), and O buffer n % 2 read out by the output warps.
template <int kMode, int CAP>
__device__ __forceinline__ bool pv_issuer(const F8DecodeParams<CAP>& p, uint32_t sbase, uint32_t tmem, uint32_t total) {
  constexpr int kOutCols = out_cols(kMode), kSteps = 4 * 32 / kOutCols;
  constexpr uint32_t kIdesc = umma_idesc_f16(128, kOutCols, false, true, false);  // A = V MN-major, B = P K-major
  const uint32_t bar0 = sbase + SM_BAR;
  const uint64_t vd = sw128_desc(sbase + SM_V, kTileBytes, 1024), pd = sw128_desc(sbase + SM_PT, 16, 1024);
  auto wait = [&](int b, uint32_t parity) { return short_wait(bar0 + 8 * b, parity); };
  uint32_t n = 0;
#pragma unroll 1
  for (; n < total; ++n) {
    if (!(wait(B_VFULL + n % kVRing, (n / kVRing) & 1) && wait(B_PFULL + (n & 1), (n >> 1) & 1) &&
          (n < 2 || wait(B_OFREE + (n & 1), ((n - 2) >> 1) & 1))))
      break;
    tc_fence_after();
    const uint64_t v0 = vd + n % kVRing * (kTileBytes >> 4), p0 = pd + (n & 1) * (kPBytes >> 4);
    const uint32_t d = tmem + TM_O + (n & 1) * kOutCols;
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < kSteps; ++kk)  // 32 keys per step
        umma_f8_ss(d, v0 + (kk & 3) * (32 * 128 >> 4), p0 + (kk >> 2) * (2 * kPiece >> 4) + 2 * (kk & 3), kIdesc, kk > 0);
      umma_commit(bar0 + 8 * (B_ODONE + (n & 1)));
      umma_commit(bar0 + 8 * (B_VEMPTY + n % kVRing));
    }
    __syncwarp();
  }
  if (elect_one()) {
    umma_commit(bar0 + 8 * (B_DRAIN + 1));
    if (!drain_wait(bar0 + 8 * (B_DRAIN + 1), 0)) atomicOr(p.status, kErrDrain);
  }
  __syncwarp();
  return n == total;
}

// ---------------------------------------------------------------------------- softmax warps
// A unit's last tile: once its new K row is in place, the tile's scale; and its V rows behind the last key (which stand for nothing and
// may hold anything) become zeros, once the tile is there.
template <int CAP>
__device__ __noinline__ float last_tile(const F8DecodeParams<CAP>& p, uint32_t sbase, const uint8_t* smem, uint32_t n, uint32_t tail, bool live, bool& ok) {
  const uint32_t bar0 = sbase + SM_BAR;
  ok = ok && counted_wait(bar0 + 8 * (B_TAIL + tail), 0);
  if (threadIdx.x < kGroup && p.pos % kKeyTile != kKeyTile - 1) {
    ok = ok && counted_wait(bar0 + 8 * (B_VFULL + n % kVRing), (n / kVRing) & 1);
    if (ok && !live) {
      const uint32_t v = sbase + SM_V + n % kVRing * kTileBytes + (threadIdx.x & (kGroup - 1)) * 128;
#pragma unroll
      for (int c = 0; c < 8; ++c) st_shared_v4(v + 16 * c, 0u, 0u, 0u, 0u);
    }
  }
  return reinterpret_cast<const float*>(smem + SM_TAILS)[tail];
}

// One set of warps: heads 4 set .. 4 set + 3 of every tile.
template <int kMode, int CAP>
__device__ __forceinline__ bool softmax(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, uint32_t tmem, int set, long long start,
                                     long long end) {
  constexpr int H = kRepText / 2;
  const int tid = threadIdx.x & (kGroup - 1), warp = tid >> 5, lane = tid & 31;  // key of a tile = TMEM lane
  const uint32_t bar0 = sbase + SM_BAR, id = 1 + set;
  const uint32_t s_cols = tmem + (static_cast<uint32_t>(warp * 32) << 16) + TM_S + set * 16;
  float* red = reinterpret_cast<float*>(smem + SM_RED) + set * 4 * H;  // [2][8 warps][4]
  // P^T row 8 piece + head (c2: 24 + head), column tid: 16-byte chunk c of row r at chunk c ^ (r % 8)
  uint32_t at[H];
#pragma unroll
  for (int h = 0; h < H; ++h) at[h] = sbase + SM_PT + (4 * set + h) * 128 + (((tid >> 4) ^ (4 * set + h)) << 4) + (tid & 15);
  auto wait = [&](int b, uint32_t parity) { return short_wait(bar0 + 8 * b, parity); };
  uint32_t n = 0, seg = 0, tails = 0;  // this CTA's tiles, its segments, and appended rows
  Seg s;
  for (long long t = start; next_seg(t, end, p.T, s); ++seg) {
    const int l = s.u / kHkv, g = s.u % kHkv;
    const F8AttnLayer& L = p.layer[l];
    const float* ks = L.ks + g * (p.Smax / kScaleBlock + 1);
    // where scores go: tensor memory (keep), or the workspace
    const bool weights = kMode != kNoWeights && L.w_out != nullptr, keep = kMode == kForm && weights && kept_unit(p, s);
    float4* scores = weights && !keep ? reinterpret_cast<float4*>(p.scores) + static_cast<size_t>(2 * s.u + set) * p.T * kKeyTile + tid
                                      : nullptr;
    const int last = s.j1 == p.T ? p.T - 1 : s.j1;  // the tile whose scale the appending warp hands over
    float k_next = s.j0 < last ? ks[s.j0] : 0.f;
    if (seg == 0) {
      prepare_q(p, sbase, smem, s.u, 4 * set + warp, 4 * set + warp + 1, seg);
      bar_sync(4, 2 * kGroup);
      if (threadIdx.x == 0) mbar_arrive(bar0 + 8 * B_QFULL);
    }
    float lsum[H], m_run[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      lsum[h] = 0.f;
      m_run[h] = -INFINITY;
    }
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j, ++n) {
      bool ok = wait(B_SDONE + (n & 3), (n >> 2) & 1);
      const bool live = j * kKeyTile + tid <= p.pos;
      float k_scale = k_next;
      if (j + 1 < last) k_next = ks[j + 1];
      if (__builtin_expect(j == last, 0)) k_scale = last_tile(p, sbase, smem, n, tails, live, ok);
      tc_fence_after();
      uint32_t d[16];
      tmem_ld16(s_cols + (n & 3) * kCols, d);
      const float4 qf = reinterpret_cast<const float4*>(smem + SM_QF)[(seg & 7) * 2 + set];
      const float f[H] = {qf.x * k_scale, qf.y * k_scale, qf.z * k_scale, qf.w * k_scale};
      // P buffer n % 2 is free, PV(n - 2) being complete
      if (n >= 2) ok = ok && wait(B_ODONE + (n & 1), ((n - 2) >> 1) & 1);
      tmem_landed16(d);
      float x[H], mine = 0.f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float a = fmaf(__uint_as_float(d[12 + h]), 0x1p-15f, __uint_as_float(d[8 + h]) * 0x1p-10f);
        const float b = fmaf(__uint_as_float(d[4 + h]), 0x1p-5f, a) + __uint_as_float(d[h]);
        x[h] = live ? b * f[h] : -INFINITY;
        const float mx = warp_max(x[h]);
        mine = lane == h ? mx : mine;
      }
      if (lane < H) red[(n & 1) * 32 + warp * H + lane] = mine;
      if (kMode != kNoWeights && scores != nullptr && live) scores[static_cast<size_t>(j) * kKeyTile] = make_float4(x[0], x[1], x[2], x[3]);
      if (keep) {
        tc_fence_after();
        tmem_st4(s_cols + TM_X - TM_S - set * 12 + n % kKept * 8, x);
      }
      if (__builtin_expect(!bar_sync_and(id, kGroup, ok), 0)) return false;
      const float4* r4 = reinterpret_cast<const float4*>(red + (n & 1) * 32);
      const float4 ra = r4[0], rb = r4[1], rc = r4[2], rd = r4[3];
      const float m[H] = {fmaxf(fmaxf(ra.x, rb.x), fmaxf(rc.x, rd.x)), fmaxf(fmaxf(ra.y, rb.y), fmaxf(rc.y, rd.y)),
                          fmaxf(fmaxf(ra.z, rb.z), fmaxf(rc.z, rd.z)), fmaxf(fmaxf(ra.w, rb.w), fmaxf(rc.w, rd.w))};
      // weights relative to the tile's largest, times 256, in three pieces
      const uint32_t buf = (n & 1) * kPBytes;
      float y[H];
      float2 fac[H];  // (what the sums before are multiplied by, the tile's share)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        x[h] = live ? ex2_approx(x[h] - m[h]) : 0.f;
        y[h] = x[h] * 256.0f;
        const float top = fmaxf(m_run[h], m[h]);
        fac[h] = make_float2(ex2_approx(m_run[h] - top), ex2_approx(m[h] - top));
        m_run[h] = top;
        lsum[h] = fmaf(lsum[h], fac[h].x, x[h] * fac[h].y);
      }
#pragma unroll
      for (int piece = 0; piece < 3; ++piece)
#pragma unroll
        for (int h = 0; h < H; h += 2) {
          const uint32_t c = take_piece(y[h], y[h + 1], piece == 0 ? 32.0f : 1.0f), to = buf + (piece < 2 ? piece : 3) * kPiece;
          st_shared_u8(at[h] + to, c);
          st_shared_u8(at[h + 1] + to, c >> 8);
        }
      if (tid == 0) {
        float4* to = reinterpret_cast<float4*>(smem + SM_FAC) + ((n & 3) * kRepText + set * H) / 2;
        to[0] = make_float4(fac[0].x, fac[0].y, fac[1].x, fac[1].y);
        to[1] = make_float4(fac[2].x, fac[2].y, fac[3].x, fac[3].y);
      }
      fence_proxy_async_smem();  // P, and zeroed V rows, are read by the tensor core
      if (keep) tmem_wait_st();
      tc_fence_before();
      bar_sync(id, kGroup);
      if (tid == 0) {
        mbar_arrive(bar0 + 8 * (B_PFULL + (n & 1)));  // P(n) is out
        mbar_arrive(bar0 + 8 * (B_FAC + (n & 3)));
      }
    }
    tails += s.j1 == p.T ? 1 : 0;
    float* lred = reinterpret_cast<float*>(smem + SM_LRED) + set * 4 * H;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float v = warp_sum(lsum[h]);
      if (lane == 0) lred[warp * H + h] = v;
    }
    bar_sync(id, kGroup);
    if (tid == 0) {
      float2* fin = reinterpret_cast<float2*>(smem + SM_FIN) + (seg & 7) * kRepText + set * H;
#pragma unroll
      for (int h = 0; h < H; ++h) fin[h] = make_float2(m_run[h], (lred[h] + lred[H + h]) + (lred[2 * H + h] + lred[3 * H + h]));
      mbar_arrive(bar0 + 8 * (B_FIN + (seg & 7)));
    }
    // (lred is written again after the next segment's barriers, which thread 0 reaches after this read)
  }
  return true;
}

// ----------------------------------------------------------------------------- output warps
// Merges unit u from its parts' partials: output thread = channel. The nth that this CTA merges, whose weights it forms, too.
template <int CAP>
__device__ __noinline__ void merge(const F8DecodeParams<CAP>& p, uint8_t* smem, int u, int nth) {
  const int tid = threadIdx.x - kOutWarp * 32, g = u % kHkv;
  const long long u0 = static_cast<long long>(u) * p.T;
  const int c0 = cta_of_tile(u0, p.W, gridDim.x), np = cta_of_tile(u0 + p.T - 1, p.W, gridDim.x) - c0 + 1;
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
    if (p.scores != nullptr && i == 0) p.lse[u * kRepText + h] = M + log2f(sum);
  }
  bar_sync(3, kGroup);
  float acc[kRepText];
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
  __nv_bfloat16* o = p.layer[u / kHkv].out + static_cast<size_t>(kRepText * g) * kD + tid;
#pragma unroll
  for (int h = 0; h < kRepText; ++h) o[h * kD] = __float2bfloat16_rn(acc[h]);
  if (tid == 0) {
    p.unit_cnt[u] = 0u;  // every part has arrived: ready for the next call
    if (p.layer[u / kHkv].w_out != nullptr) reinterpret_cast<int*>(smem + SM_TODO)[nth] = u;  // (read in kForm)
  }
}

// The same for a unit whose second part is there, the first being the calling thread's sums, `fin` and `down`. (The roundings are merge()'s, so that
// results do not depend on when the other part came.)
template <int CAP>
__device__ __noinline__ void merge_two(const F8DecodeParams<CAP>& p, uint8_t* smem, int u, const float2* fin, float down, float a0, float a1, float a2, float a3, float a4,
                                       float a5, float a6, float a7) {
  const int tid = threadIdx.x - kOutWarp * 32;
  const size_t ps = static_cast<size_t>(blockIdx.x + 1) * 2;
  const float4* po = reinterpret_cast<const float4*>(p.part_o + ps * kRepText * kD) + 2 * tid;
  const float4* pm = reinterpret_cast<const float4*>(p.part_ml + ps * kRepText * 2);
  const float4 o0 = __ldcg(po), o1 = __ldcg(po + 1), m[4] = {__ldcg(pm), __ldcg(pm + 1), __ldcg(pm + 2), __ldcg(pm + 3)};
  const float acc[kRepText] = {a0, a1, a2, a3, a4, a5, a6, a7}, other[kRepText] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
  const F8AttnLayer& L = p.layer[u / kHkv];
  __nv_bfloat16* out = L.out + static_cast<size_t>(kRepText * (u % kHkv)) * kD + tid;
#pragma unroll
  for (int h = 0; h < kRepText; ++h) {
    const float2 a = f8_lowered(fin[h], down), b = h & 1 ? make_float2(m[h / 2].z, m[h / 2].w) : make_float2(m[h / 2].x, m[h / 2].y);
    const float M = fmaxf(a.x, b.x), wa = ex2_approx(a.x - M), wb = ex2_approx(b.x - M);
    const float sum = __fadd_rn(__fmul_rn(a.y, wa), __fmul_rn(b.y, wb)), inv = 1.0f / sum;
    out[h * kD] = __float2bfloat16_rn(fmaf(wb * inv, other[h], __fmul_rn(wa * inv, acc[h])));
    if (p.scores != nullptr && tid == h) p.lse[u * kRepText + h] = M + log2f(sum);
  }
  if (tid == 0) {
    p.unit_cnt[u] = 0u;
    if (L.w_out != nullptr) reinterpret_cast<int*>(smem + SM_TODO)[1] = u;  // (read in kForm)
  }
}

// What the output warps do before there is any output: the first segment's new rows, and the second segment's Q (its unit is the next one).
template <int CAP>
__device__ __noinline__ void early(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, int u, bool tail, bool more, int warp) {
  if (tail && warp < 2) append_row(p, sbase, smem, warp, u, 0);
  if (!more) return;
  prepare_q(p, sbase, smem, u + 1, 2 * warp, 2 * warp + 2, 1);
  bar_sync(3, kGroup);
  if (threadIdx.x == kOutWarp * 32) mbar_arrive(sbase + SM_BAR + 8 * (B_QFULL + 1));
}

__device__ __forceinline__ float4 as_float4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return make_float4(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c), __uint_as_float(d));
}
// What the weights of a unit are formed with (the kernel's parameters are too far away to be looked up at every step).
struct WeighUnit {
  float lse[kRepText];
  const float* w_in;
  float* w_out;
};
// Its next tile's place in tensor memory, and that tile's first key.
struct Weighing {
  uint32_t slot;
  int key;
};
// A key's sums so far, of the kWeigh tiles from its own on (0 for the new row's, and behind it), on their way to the thread's words of
// shared memory: no register waits for them, which a call's return would do.
__device__ __forceinline__ void fetch_sums(const float* w_in, uint32_t sums, int key, int pos) {
#pragma unroll
  for (int i = 0; i < kWeigh; ++i) {
    const int k = key + i * kKeyTile;
    if (w_in == nullptr || k >= pos) {
      st_shared_f32(sums + i * kKeyTile * 4, 0.f);
    } else {
      cp_async4(sums + i * kKeyTile * 4, w_in + k);
    }
  }
}
// Weights of kWeigh tiles: cols is where tensor memory holds scores (what lies behind the last tile is not used), key the calling
// thread's.
__device__ __noinline__ void weigh(const uint8_t* smem, uint32_t cols, uint32_t slot, uint32_t sums, int key, int pos) {
  const WeighUnit& unit = *reinterpret_cast<const WeighUnit*>(smem + SM_UNIT);
  uint32_t x[kWeigh][8];
#pragma unroll
  for (int i = 0; i < kWeigh; ++i) {
    tmem_ld8(cols + 8 * slot, x[i]);
    slot = slot + 1 == kKept ? 0u : slot + 1;
  }
  const float4 la = *reinterpret_cast<const float4*>(unit.lse), lb = *reinterpret_cast<const float4*>(unit.lse + 4);
  const float* w_in = unit.w_in;
  float* w_out = unit.w_out;
  asm volatile("cp.async.wait_all;" ::: "memory");
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < kWeigh; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) asm volatile("" : "+r"(x[i][e])::"memory");  // (not before the wait)
    const int k = key + i * kKeyTile;
    if (k <= pos)
      w_out[k] = ld_shared_f32(sums + i * kKeyTile * 4) +
                 f8_weight(as_float4(x[i][0], x[i][1], x[i][2], x[i][3]), as_float4(x[i][4], x[i][5], x[i][6], x[i][7]), la, lb);
  }
  fetch_sums(w_in, sums, key + kWeigh * kKeyTile, pos);
}
__device__ __forceinline__ void weigh_on(Weighing& w, const uint8_t* smem, uint32_t cols, uint32_t sbase, int tid, int pos) {
  weigh(smem, cols, w.slot, sbase + SM_SUMS + 4 * tid, w.key + tid, pos);
  w.key += kWeigh * kKeyTile;
  w.slot = w.slot + kWeigh >= kKept ? w.slot + kWeigh - kKept : w.slot + kWeigh;
}

template <int kMode, int CAP>
__device__ __forceinline__ bool output_segments(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, uint32_t tmem, long long start, long long end,
                                                Weighing& weighing) {
  const int tid = threadIdx.x - kOutWarp * 32, warp = tid >> 5;  // channel = TMEM lane
  const uint32_t o_cols = tmem + (static_cast<uint32_t>(warp * 32) << 16) + TM_O, bar0 = sbase + SM_BAR;
  volatile uint32_t* merge_flag = reinterpret_cast<volatile uint32_t*>(smem + SM_MERGE);
  auto wait = [&](int b, uint32_t parity) { return short_wait(bar0 + 8 * b, parity); };
  uint32_t n = 0, seg = 0, tails = 0;
  int late = -1;  // a unit whose part warp 15 counts
  Seg s;
  for (long long t = start; next_seg(t, end, p.T, s); ++seg) {
    const int l = s.u / kHkv, g = s.u % kHkv;
    const F8AttnLayer& L = p.layer[l];
    const float* vs = L.vs + g * (p.Smax / kScaleBlock + 1);
    if (seg == 0) early(p, sbase, smem, s.u, s.j1 == p.T, t < end, warp);
    const int last = s.j1 == p.T ? p.T - 1 : s.j1;  // the tile whose scale the appending warp hands over
    float v_next = s.j0 < last ? vs[s.j0] : 0.f;
    if (kMode == kForm && tid == 0 && s.j0 == 0 && L.w_out != nullptr && L.w_in != nullptr)  // they are needed soon
      prefetch_l2_bulk(L.w_in + static_cast<size_t>(g) * p.Smax, p.T * kKeyTile * 4);
    float acc[kRepText], down = 1.0f;  // (down: see f8_lower)
#pragma unroll
    for (int h = 0; h < kRepText; ++h) acc[h] = 0.f;
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j, ++n) {
      bool ok = wait(B_FAC + (n & 3), (n >> 2) & 1) && wait(B_ODONE + (n & 1), (n >> 1) & 1);  // the tile's factors, and its O
      float v_scale = v_next;
      if (j + 1 < last) v_next = vs[j + 1];
      if (__builtin_expect(j == last, 0)) {
        ok = ok && wait(B_TAIL + kTails + tails, 0);
        v_scale = reinterpret_cast<const float*>(smem + SM_TAILS)[kTails + tails];
      }
      tc_fence_after();
      uint32_t d[16], d2[8];  // O^T row = channel tid, columns (piece, head)
      tmem_ld16(o_cols + (n & 1) * out_cols(kMode), d);
      if (kMode != kForm) tmem_ld8(o_cols + (n & 1) * out_cols(kMode) + 24, d2);
      const float4* fac = reinterpret_cast<const float4*>(smem + SM_FAC) + (n & 3) * (kRepText / 2);
      const float4 f[4] = {fac[0], fac[1], fac[2], fac[3]};
      if (__builtin_expect(v_scale * down > kF8TopSum, 0)) {
        const float less = f8_lower(v_scale * down);
        down *= less;
#pragma unroll
        for (int h = 0; h < kRepText; ++h) acc[h] *= less;
      }
      const float vf = v_scale * down * 0x1p-8f;
      tmem_landed16(d);
      if (kMode != kForm)
#pragma unroll
        for (int h = 0; h < kRepText; ++h) {
          asm volatile("" : "+r"(d2[h])::"memory");  // (not before the wait)
          d[8 + h] = __float_as_uint(__uint_as_float(d[8 + h]) + __uint_as_float(d2[h]));
        }
      tc_fence_before();
      if (__builtin_expect(!bar_sync_and(3, kGroup, ok), 0)) return false;
      if (tid == 0) mbar_arrive(bar0 + 8 * (B_OFREE + (n & 1)));
#pragma unroll
      for (int h = 0; h < kRepText; h += 2) {
        acc[h] = fmaf(acc[h], f[h / 2].x, fmaf(__uint_as_float(d[8 + h]), 0x1p-5f, __uint_as_float(d[h])) * (f[h / 2].y * vf));
        acc[h + 1] = fmaf(acc[h + 1], f[h / 2].z, fmaf(__uint_as_float(d[9 + h]), 0x1p-5f, __uint_as_float(d[h + 1])) * (f[h / 2].w * vf));
      }
      if (kMode == kForm && weighing.key <= p.pos) weigh_on(weighing, smem, o_cols + TM_X - TM_O, sbase, tid, p.pos);
    }
    tails += s.j1 == p.T ? 1 : 0;
    // ---- the segment's end: its sums, then its output or its part of one
    if (!bar_sync_and(3, kGroup, wait(B_FIN + (seg & 7), (seg >> 3) & 1))) return false;
    const float2* fin = reinterpret_cast<const float2*>(smem + SM_FIN) + (seg & 7) * kRepText;
    if (s.j0 == 0 && s.j1 == p.T) {
      __nv_bfloat16* o = L.out + static_cast<size_t>(kRepText * g) * kD + tid;
#pragma unroll
      for (int h = 0; h < kRepText; ++h) o[h * kD] = __float2bfloat16_rn(__fdividef(acc[h], fin[h].y * down));
      if (kMode != kNoWeights && L.w_out != nullptr) {
        if (kMode == kScores) {
          if (tid < kRepText) p.lse[s.u * kRepText + tid] = fin[tid].x + log2f(fin[tid].y);
        } else {  // (the unit before's are all formed: it had no more tiles than this one)
          WeighUnit& unit = *reinterpret_cast<WeighUnit*>(smem + SM_UNIT);
          const float* w_in = L.w_in != nullptr ? L.w_in + static_cast<size_t>(g) * p.Smax : nullptr;
          if (tid < kRepText) unit.lse[tid] = fin[tid].x + log2f(fin[tid].y);
          if (tid == 0) {
            unit.w_in = w_in;
            unit.w_out = L.w_out + static_cast<size_t>(g) * p.Smax;
          }
          weighing.slot = (n - p.T) % kKept;
          weighing.key = 0;
          fetch_sums(w_in, sbase + SM_SUMS + 4 * tid, tid, p.pos);
          tc_fence_after();
        }
      }
      continue;
    }
    if (last_part(p, s, seg, t, end) && wait(B_QFULL + (seg & 1), (seg >> 1) & 1) &&
        *reinterpret_cast<volatile uint32_t*>(smem + SM_LASTPART) == 1u) {
      merge_two(p, smem, s.u, fin, down, acc[0], acc[1], acc[2], acc[3], acc[4], acc[5], acc[6], acc[7]);
      if (late < 0) return true;
      s.u = late;  // (nothing more to count)
      break;
    }
    // Part index: 2 c + slot (a part is its CTA's first segment or its last). Layout [part][channel][8 heads].
    const size_t ps = static_cast<size_t>(blockIdx.x) * 2 + (seg == 0 ? 0 : 1);
    float4* po = reinterpret_cast<float4*>(p.part_o + ps * kRepText * kD) + 2 * tid;
    po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    if (tid < kRepText) *reinterpret_cast<float2*>(p.part_ml + (ps * kRepText + tid) * 2) = f8_lowered(fin[tid], down);
    bar_sync(3, kGroup);
    if (t < end) {  // (the first segment)
      late = s.u;
      if (tid == 0) mbar_arrive(bar0 + 8 * B_PART);
      continue;
    }
    if (late >= 0) break;  // (SM_MERGE is the other part's until it has been read)
    if (tid == 0) *merge_flag = count_part(p, s.u) ? 1u : 0u;
    bar_sync(3, kGroup);
    if (*merge_flag) merge(p, smem, s.u, 0);
    return true;
  }
  if (late < 0) return true;
  if (!bar_sync_and(3, kGroup, wait(B_LATE, 0))) return false;
  if (*merge_flag) merge(p, smem, late, 0);
  if (s.j1 == p.T || s.u == late) return true;  // (a CTA's last segment is a part unless it ends its unit)
  bar_sync(3, kGroup);
  if (tid == 0) *merge_flag = count_part(p, s.u) ? 1u : 0u;
  bar_sync(3, kGroup);
  if (*merge_flag) merge(p, smem, s.u, 1);
  return true;
}
// The whole CTA: the weights of a unit that it has merged, from the parts' scores in the workspace.
template <int CAP>
__device__ __noinline__ void weigh_merged(const F8DecodeParams<CAP>& p, int u) {
  constexpr int kBatch = (kF8KeptTiles * kKeyTile + kThreads - 1) / kThreads;  // all keys' loads are under way together
  const F8AttnLayer& L = p.layer[u / kHkv];
  const size_t half = static_cast<size_t>(p.T) * kKeyTile, at = static_cast<size_t>(u % kHkv) * p.Smax;
  const float4* x = reinterpret_cast<const float4*>(p.scores) + 2 * u * half;
  const float4* lse = reinterpret_cast<const float4*>(p.lse + u * kRepText);
  const float4 la = __ldcg(lse), lb = __ldcg(lse + 1);
  float4 a[kBatch], b[kBatch];
  float w[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int k = threadIdx.x + i * kThreads;
    w[i] = 0.f;
    if (k <= p.pos) {
      a[i] = __ldcg(x + k);
      b[i] = __ldcg(x + half + k);
      if (k < p.pos && L.w_in != nullptr) w[i] = L.w_in[at + k];
    }
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int k = threadIdx.x + i * kThreads;
    if (k <= p.pos) L.w_out[at + k] = w[i] + f8_weight(a[i], b[i], la, lb);
  }
}
template <int kMode, int CAP>
__device__ __forceinline__ bool output(const F8DecodeParams<CAP>& p, uint32_t sbase, uint8_t* smem, uint32_t tmem, long long start, long long end) {
  const int tid = threadIdx.x - kOutWarp * 32;
  Weighing weighing;
  weighing.key = p.pos + 1;  // nothing yet
  if (!output_segments<kMode>(p, sbase, smem, tmem, start, end, weighing)) return false;
  if (kMode != kForm) return true;
  bar_sync(3, kGroup);  // (the log2-sum-exps are there)
  while (weighing.key <= p.pos) weigh_on(weighing, smem, tmem + (static_cast<uint32_t>((tid >> 5) * 32) << 16) + TM_X, sbase, tid, p.pos);
  return true;
}

}  // namespace f8d

template <int CAP, int kMode>
__global__ void __launch_bounds__(f8d::kThreads, 1) fp8_decode_kernel(const __grid_constant__ F8DecodeParams<CAP> p) {
  using namespace f8d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = sbase + SM_BAR;
  const long long start = cta_tile_start(blockIdx.x, p.W, gridDim.x), end = cta_tile_start(blockIdx.x + 1, p.W, gridDim.x);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x >= 256 && threadIdx.x < 256 + kNumBars) {
    const int b = threadIdx.x - 256;  // (what softmax warps tell comes from two sets)
    mbar_init(bar0 + 8 * b, (b >= B_PFULL && b < B_PFULL + 2) || (b >= B_FAC && b < B_FIN + 8) ? 2 : 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 3) reinterpret_cast<int*>(smem + SM_TODO)[threadIdx.x] = threadIdx.x < 2 ? -1 : 0;  // (and SM_LASTPART)
  if (threadIdx.x < kD / 2) reinterpret_cast<float4*>(smem + SM_ROT)[threadIdx.x] = p.rot[threadIdx.x];
  if (threadIdx.x < 128)  // P's rows of zeros, of both buffers
    reinterpret_cast<uint4*>(smem + SM_PT + (threadIdx.x >> 6) * kPBytes + 2 * kPiece)[threadIdx.x & 63] = make_uint4(0u, 0u, 0u, 0u);
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
    for (long long x = start; x < end && x < start + 6; ++x) {
      const int u = static_cast<int>(x / p.T), j = static_cast<int>(x - static_cast<long long>(u) * p.T);
      const size_t off = (static_cast<size_t>(u % kHkv) * p.Smax + static_cast<size_t>(j) * kKeyTile) * kD;
      prefetch_l2_bulk(p.layer[u / kHkv].kc + off, kTileBytes);
      prefetch_l2_bulk(p.layer[u / kHkv].vc + off, kTileBytes);
    }
  }
  // everything below reads what earlier kernels in the stream wrote
  pdl_wait_primary();
  // (the roles' order is the code's, and matters to the instruction caches: 64 layers at pos 4700 take up to 2 % longer in others)
  bool ok = true;
  if (warp == 15) {
    ok = prepare(p, sbase, smem, start, end);
  } else if (warp == 12) {
    ok = producer(p, sbase, start, end);
  } else if (warp == 13) {
    ok = qk_issuer(p, sbase, tmem, start, end);
  } else if (warp == 14) {
    ok = pv_issuer<kMode>(p, sbase, tmem, static_cast<uint32_t>(end - start));
  } else if (warp >= kOutWarp && warp < kOutWarp + 4) {
    ok = output<kMode>(p, sbase, smem, tmem, start, end);
  } else if (warp < kOutWarp) {
    ok = softmax<kMode>(p, sbase, smem, tmem, warp >> 2, start, end);
  }
  if (!ok && (threadIdx.x & 31) == 0) atomicOr(p.status, kErrF8DecodeWait);
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (kMode == kForm)
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int u = reinterpret_cast<const int*>(smem + SM_TODO)[i];
      if (u >= 0) weigh_merged(p, u);
    }
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Weights from the scores: a thread has kWKeys keys of one unit under way. grid (key blocks, units)
constexpr int kWThreads = 256, kWKeys = 2;
__global__ void __launch_bounds__(kWThreads) fp8_weights_kernel(const __grid_constant__ F8WeightsParams p) {
  const int u = blockIdx.y, key0 = blockIdx.x * (kWThreads * kWKeys) + threadIdx.x;
  const F8AttnLayer& L = p.layer[u / kHkv];
  const size_t at = static_cast<size_t>(u % kHkv) * p.Smax + key0;
  const size_t half = static_cast<size_t>(p.T) * kKeyTile;
  const float4* x = reinterpret_cast<const float4*>(p.scores) + 2 * u * half + key0;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (L.w_out == nullptr) return;
  float4 a[kWKeys], b[kWKeys];
  float w[kWKeys];
#pragma unroll
  for (int i = 0; i < kWKeys; ++i) {
    const int key = key0 + i * kWThreads;
    if (key <= p.pos) {
      a[i] = __ldcs(x + i * kWThreads);
      b[i] = __ldcs(x + half + i * kWThreads);
    }
    w[i] = key < p.pos && L.w_in != nullptr ? L.w_in[at + i * kWThreads] : 0.f;
  }
  const float4* lse = reinterpret_cast<const float4*>(p.lse + u * kRepText);
  const float4 c = lse[0], d = lse[1];
#pragma unroll
  for (int i = 0; i < kWKeys; ++i)
    if (key0 + i * kWThreads <= p.pos)
      L.w_out[at + i * kWThreads] = w[i] + f8_weight(a[i], b[i], c, d);
}

cudaError_t fp8_decode_set_attributes() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(f8d::kSmemBytes));
  };
  set(fp8_decode_kernel<kSmallCap, f8d::kNoWeights>);
  set(fp8_decode_kernel<kSmallCap, f8d::kScores>);
  set(fp8_decode_kernel<kDecodeMaxLayers, f8d::kNoWeights>);
  set(fp8_decode_kernel<kDecodeMaxLayers, f8d::kScores>);
  set(fp8_decode_kernel<kDecodeMaxLayers, f8d::kForm>);
  return e;
}

template <int CAP>
cudaError_t launch_fp8_decode(const F8DecodeParams<CAP>& p, cudaLaunchConfig_t cfg) {
  if (p.n_layers * kHkv / static_cast<int>(cfg.gridDim.x) + 2 > f8d::kTails) return cudaErrorInvalidConfiguration;  // (a GPU of 7 SMs)
  cfg.blockDim = dim3(f8d::kThreads);
  cfg.dynamicSmemBytes = f8d::kSmemBytes;
  if (p.scores == nullptr) return cudaLaunchKernelEx(&cfg, fp8_decode_kernel<CAP, f8d::kNoWeights>, p);
  if constexpr (CAP == kDecodeMaxLayers)
    if (p.form) return cudaLaunchKernelEx(&cfg, fp8_decode_kernel<CAP, f8d::kForm>, p);
  return cudaLaunchKernelEx(&cfg, fp8_decode_kernel<CAP, f8d::kScores>, p);
}
template cudaError_t launch_fp8_decode<kSmallCap>(const F8DecodeParams<kSmallCap>&, cudaLaunchConfig_t);
template cudaError_t launch_fp8_decode<kDecodeMaxLayers>(const F8DecodeParams<kDecodeMaxLayers>&, cudaLaunchConfig_t);

cudaError_t launch_fp8_weights(const F8WeightsParams& p, cudaLaunchConfig_t cfg) {
  cfg.gridDim = dim3(p.pos / (kWThreads * kWKeys) + 1, p.n_layers * kHkv);
  cfg.blockDim = dim3(kWThreads);
  return cudaLaunchKernelEx(&cfg, fp8_weights_kernel, p);
}

}  // namespace ea
