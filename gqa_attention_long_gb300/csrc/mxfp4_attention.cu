// mxfp4_attention.cu — the expert's attention over 4-bit caches on the tensor cores.
//
// Per (layer, kv head) unit: 128 folded query rows (2 heads x 64 tokens) against cache rows [0, S) and
// the 64 own rows, softmax(Q K^T / sqrt(128)) V over the stored values.
//
// A prologue kernel norms and ropes q and k, stages q as f16 tiles (times a power of two per row; 11 bits, of which a
// score of unit variance feels 2^-12, against 2^-9 of the bf16 output; the weights P are f16 for the same reason) and
// encodes the own rows into the cache; the attention kernel follows; units cut over several CTAs
// are joined by a merge kernel. The units' tiles of 128 keys (ceil(S / 128), then the own rows) are cut into
// one contiguous range per CTA, one CTA per SM.
//
// The codes are widened to f16 tiles in shared memory, where tcgen05.mma takes them (a fragment in
// registers, as the decode step has it, would have to be formed again for each of the 128 query rows'
// warps). A code times 2^(e - R + 8) is exact in f16 as long as its block's scale e is within 2^22 below R, a
// reference per segment and tensor: the largest scale of a block that is not all zeros, as of the last tile that had one
// 2^3 above it or 2^22 below. K's reference goes back into the scores, V's into the output, both in fp32. A tile whose own
// blocks lie more than 2^22 apart goes through the tensor cores without the blocks below, and the softmax adds what
// those give in fp32 (to the scores before they are used, to the accumulator before the tile's P V): a tile of 128 keys
// then takes tens of microseconds, but no block counts as zero down to 2^100 below the segment's largest.
//
// Warp roles (768 threads):
//   warps 0-3, 4-7, 8-11  softmax of the CTA's tiles in turn: thread = query row = TMEM lane
//   warps 12-15, 16-19  converters of K and of V: thread = key row of the tile; into double-buffered f16 tiles
//   warps 20, 21  load K's and V's packed rows (bulk copies into three-stage rings) and set the tiles' references
//   warps 22, 23  issue S = Q K^T (and load each segment's Q) and O += P V (P from TMEM)
// TMEM: three score buffers (P(n) goes over S(n)), one per softmax warpgroup, and one accumulator. A softmax warpgroup
// waits for PV(n) and QK(n + 3) while the other two work; with two warpgroups, each with an accumulator, they
// waited two thirds of the time. The price is a running maximum shared by the warpgroups: one works on tile n
// with the maximum that it last knew (raised when a chunk's weights pass it by far) and compares notes with
// tile n - 1's at the end, through shared memory: only where the two differ is P(n), or the accumulator, scaled.
//
// Measured: 64 layers at S = 4700 158 us (of these the prologue 15, the merge 2), 2 layers at S = 65537 66 us,
// 1 layer at S = 4700 16.8 us, at S = 256 11.8 us. A tile takes about 1,800 cycles, of which its MMAs are 1,025 (tensor pipe
// 50 % busy). No unit is full: a converter spends 1,100 cycles on a row and 700 on its waits and hand-overs, a
// softmax warpgroup 2,700 on a tile, of which three are in flight, and together they take 60 % of the issue slots.
// Tried and slower, at 64 layers: tiles of 96 keys with four score buffers (+13 %: a tile's fixed costs), two
// warpgroups to a converter (+9 %), two for the softmax (+2 %), waits that spin (+5 %), scores fetched a chunk ahead
// (+6 %). One layer is a chain: prologue 3.5 us, load and reference 2.3, two tiles 3.2, epilogue 1.5, merge 3.3.
//
// The instruction cache held earlier forms back: with the roles' loops unrolled, 68 % of the peak of
// instruction fetches went to the second level and every role crawled (3,600 cycles a tile). So the
// loops are small, K and V share their code, and what is rare is out of line.
#include "merge.cuh"
#include "mxfp4.cuh"
#include "rope.cuh"

namespace ea {

// ------------------------------------------------------------------------------- prologue
// One octet of threads per token and kv head: the token's two q rows, its k row and its v row, whose angles are formed
// once (three CTAs to an SM); or, when there are too few of them to fill the GPU (kSplit), one of the four
// rows (with four rows or one, at S = 300: 1 layer 14.9 or 13.4 us, 4 layers 14.8 or 14.7, 8 layers 16.4 or 17.5). grid
// (2 or 8, kv heads, layers).
template <bool kSplit>
__global__ void __launch_bounds__(256, kSplit ? 1 : 3) mxfp4_prologue_kernel(const __grid_constant__ MxPrologueParams p) {
  const int g = blockIdx.y, l = blockIdx.z, i = threadIdx.x & 7;
  const int t = 32 * (blockIdx.x & 1) + (threadIdx.x >> 3);
  const int dl = 8 * i, dh = 64 + 8 * i;
  // The tables' rows that this half of the tokens needs, copied to shared memory while the preceding kernel ends (they
  // are read by lane-dependent index: through a generic address, not the constant bank). Frequency j at j + j / 8: an
  // octet's lanes, eight frequencies apart, fall in different banks.
  __shared__ float4 rot[4 + 8][kD / 2 + 8];
  {
    const float4 *pa = &p.rot_a[4 * (blockIdx.x & 1)][0], *pb = &p.rot_b[0][0];
    asm volatile("" : "+l"(pa), "+l"(pb));
    for (int k = threadIdx.x; k < 12 * (kD / 2); k += 256) {
      const int j = k % (kD / 2);
      rot[k / (kD / 2)][j + j / 8] = k < 4 * (kD / 2) ? pa[k] : pb[k - 4 * (kD / 2)];
    }
  }
  __syncthreads();
  const float4 *ra = &rot[(t >> 3) & 3][9 * i], *rb = &rot[4 + (t & 7)][9 * i];
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 a = ra[e], b = rb[e];
    cs[e] = fmaf(a.x, b.x, -a.z * b.z);
    sn[e] = fmaf(a.z, b.x, a.x * b.z);
  }
  auto angle = [&](int e, Pair& c, Pair& s) {
    const float4 a = ra[e], b = rb[e];
    const Pair ca = {a.x, a.y}, sa = {a.z, a.w}, cb = {b.x, b.y}, sb = {b.z, b.w};
    c = ca * cb + -(sa * sb);
    s = sa * cb + ca * sb;
  };
  pdl_wait_primary();
  pdl_launch_dependents();
  const MxAttnLayer& L = p.layer[l];
  const size_t unit = static_cast<size_t>(l) * kHkv + g;
  auto load = [&](const __nv_bfloat16* src, uint4 (&to)[2]) {
    to[0] = *reinterpret_cast<const uint4*>(src + dl);
    to[1] = *reinterpret_cast<const uint4*>(src + dh);
  };
  auto load_row = [&](int kind, uint4 (&to)[2]) {  // kind: q of the unit's two heads, k, v
    load(kind < 2 ? L.q_raw + (static_cast<size_t>(2 * g + kind) * kTok + t) * kD
                  : (kind == 2 ? L.k_raw : L.v_raw) + (static_cast<size_t>(g) * kTok + t) * kD, to);
  };
  auto q_row = [&](int kind, const uint4 (&raw)[2], const uint4 (&gain)[2]) {
    float xl[8], xh[8], gl[8], gh[8], yl[8], yh[8], factor;
    unpack_bf16x8(raw[0], xl);
    unpack_bf16x8(raw[1], xh);
    unpack_bf16x8(gain[0], gl);
    unpack_bf16x8(gain[1], gh);
    norm_rope(xl, xh, gl, gh, cs, sn, yl, yh);
    f16_row(yl, yh, p.scale_log2, factor);
    const int r = kind * kTok + t;
    uint8_t* q = p.q_ws + unit * kQTileBytes;
    *reinterpret_cast<uint4*>(q + swz_off(r, i, kQTileBytes / 2)) = pack8(yl, true);
    *reinterpret_cast<uint4*>(q + swz_off(r, i + 8, kQTileBytes / 2)) = pack8(yh, true);
    if (i == 0) p.q_factor[unit * kRows + r] = factor;
  };
  auto new_row = [&](bool v, const uint4 (&raw)[2], const uint4 (&gain)[2]) {
    float xl[8], xh[8], gl[8], gh[8];
    unpack_bf16x8(raw[0], xl);
    unpack_bf16x8(raw[1], xh);
    uint32_t cl, ch;
    int el, eh;
    if (v) {
      mx_encode_octet<true>(xl, xh, cl, ch, el, eh);
    } else {
      unpack_bf16x8(gain[0], gl);
      unpack_bf16x8(gain[1], gh);
      mx_encode_k_octet<true>(xl, xh, gl, gh, cs, sn, angle, cl, ch, el, eh);
    }
    __nv_bfloat16* val = v ? L.v_new : L.k_new;
    if (val != nullptr) val += (static_cast<size_t>(g) * kTok + t) * kD;
    mx_store_octet(cl, ch, el, eh, v ? L.vc : L.kc, v ? L.vs : L.ks, static_cast<size_t>(g) * p.Smax + p.Smax - kTok + t, i, val);
  };
  if constexpr (kSplit) {
    const int kind = blockIdx.x >> 1;
    uint4 raw[2], gain[2];
    load_row(kind, raw);
    load(kind < 2 ? L.q_gamma : L.k_gamma, gain);
    if (kind < 2) q_row(kind, raw, gain);
    else new_row(kind == 3, raw, gain);
  } else {
    uint4 raw[4][2], gq[2], gk[2];  // (every row's loads go out before the first is used)
#pragma unroll
    for (int kind = 0; kind < 4; ++kind) load_row(kind, raw[kind]);
    load(L.q_gamma, gq);
    load(L.k_gamma, gk);
    q_row(0, raw[0], gq);
    q_row(1, raw[1], gq);
    new_row(false, raw[2], gk);
    new_row(true, raw[3], gk);
  }
}

namespace mxa {

constexpr int kSoftWg = 3, kSoftmax = 128 * kSoftWg;  // softmax warpgroups, and their threads
constexpr int kConvert = 128;                         // threads of K's converters, and of V's
constexpr int kThreads = kSoftmax + 2 * kConvert + 128;
// registers per thread after the roles part (launched with kRegLaunch): the sum is the launch's at most
constexpr int kRegLaunch = 65536 / kThreads / 8 * 8;
constexpr int kRegSoftmax = 96, kRegConvert = 64, kRegIssue = 64;
static_assert(kSoftmax * kRegSoftmax + 2 * kConvert * kRegConvert + 128 * kRegIssue <= kThreads * kRegLaunch, "register split");
constexpr int kRing = 3;
constexpr uint32_t kCodes = kKeyTile * kMxRowBytes, kScales = kKeyTile * kMxRowScales;
constexpr uint32_t kStageBytes = kCodes + kScales;          // a tile's codes and scales, of K or of V
constexpr uint32_t kAtom = 16384, kTile = 2 * kAtom;        // an f16 tile: two 64-channel halves
constexpr uint32_t SM_Q = 0, SM_K = SM_Q + kTile, SM_V = SM_K + 2 * kTile, SM_RING = SM_V + 2 * kTile;
constexpr uint32_t SM_X = SM_RING + 2 * kRing * kStageBytes;   // [segment parity][warpgroup][row] (m, l)
constexpr uint32_t SM_M = SM_X + 2 * kSoftWg * kRows * 8;      // [row] running maximum (log2 units)
constexpr uint32_t SM_REF = SM_M + kRows * 4;               // [K, V][8]: R of tile n % 8, and kLow
constexpr uint32_t SM_BAR = SM_REF + 16 * 4;
// by tile n % 3: FULL and EMPTY (K's ring, V's ring), SFULL, MDONE, PFULL, ODONE; by n % 2: RDY (K's f16 tiles,
// V's); by n % 8: REF (K's, V's)
constexpr int B_FULL = 0, B_EMPTY = 6, B_SFULL = 12, B_MDONE = 15, B_PFULL = 18, B_ODONE = 21, B_RDY = 24, B_REF = 28,
              B_QFULL = 44, B_OFREE = 45, B_DRAIN = 46, kNumBars = 48;
static_assert(kRing == 3, "barrier indices");
__device__ __forceinline__ uint32_t bar_count(int b) {
  return b >= B_EMPTY && b < B_SFULL ? kConvert : b >= B_MDONE && b < B_ODONE ? 128 : b >= B_RDY && b < B_REF ? kConvert
         : b == B_OFREE ? 256 : 1;
}
constexpr uint32_t SM_TMEM = SM_BAR + kNumBars * 8, SM_FAILED = SM_TMEM + 4;
constexpr uint32_t kSmemBytes = SM_FAILED + 4 + 1024;  // + slack to align the base
static_assert(kSmemBytes <= 232448 && SM_RING % 128 == 0 && SM_X % 16 == 0 && SM_BAR % 8 == 0, "shared memory of one sm_103 CTA");
constexpr uint32_t TM_S = 0, TM_O = 384, kTmemCols = 512;  // three score (then P) buffers, the accumulator
constexpr int kRefField = 23, kMaxField = 26;  // f16 exponent field of 2^(e - R + 8), and its cut (all-zero blocks)
constexpr int kWindow = kRefField - 1;         // blocks from R - kWindow on are held
// V's reference follows a tile down to 2^-40 of the segment's highest: the accumulator, at most 2^52 (weights of 2^16, values
// of 2^14, 2^22 keys) in the highest one's units, stays within fp32.
constexpr int kFollow = 40;
constexpr int kLow = 256;                      // beside a tile's reference: the tile has blocks below the window
// A row's weights are 2^(s - m) with m set kLift below a maximum, so that f16 holds those down to 2^-32 of the largest
// (2^-24 of it would lose a key's weight where half a million of them still count).
constexpr float kLift = 8.f;
constexpr uint32_t kBarSoftmax = 1;

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A CTA's tiles as segments: the part [j0, j1) of unit u's tiles that its range holds.
struct Seg {
  int u, j0, j1, left;  // left: tiles of the range after this segment
};
__device__ __forceinline__ Seg first_seg(long long start, long long end, int T) {
  const int t = static_cast<int>(start), n = static_cast<int>(end - start);
  Seg s;
  s.u = t / T;
  s.j0 = t - s.u * T;
  s.j1 = min(T, s.j0 + n);
  s.left = n - (s.j1 - s.j0);
  return s;
}
__device__ __forceinline__ void next_seg(Seg& s, int T) {  // the range's later segments start at their unit's first tile
  ++s.u;
  s.j0 = 0;
  s.j1 = min(T, s.left);
  s.left -= s.j1;
}

// Tile n's place in a ring of three: b = n % 3, par = n / 3 & 1 (the parity of its barriers' phase).
struct Ring3 {
  uint32_t b = 0, par = 0;
  __device__ __forceinline__ void step(uint32_t by = 1) {  // by 1 to 3 tiles
    b += by;
    if (b >= 3) {
      b -= 3;
      par ^= 1;
    }
  }
  __device__ __forceinline__ Ring3 back(uint32_t by) const {  // the place of tile n - by, by 1 or 2
    Ring3 r;
    r.b = b >= by ? b - by : b + 3 - by;
    r.par = b >= by ? par : par ^ 1;
    return r;
  }
};

struct Ctx {
  uint8_t* smem;
  uint32_t sbase, tmem;
  volatile uint32_t* failed;
  uint32_t* status;
  long long start, end;
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + SM_BAR + 8u * i; }
  // (With bounded_wait's code in every role the 64 layers took 5 us more.) Whoever has to give up notes why; the other roles
  // then run out of looks themselves.
  __device__ __forceinline__ bool wait(int b, uint32_t parity, uint32_t err) const {
    if (counted_wait(bar(b), parity)) return true;
    *failed = err;  // (goes to the status word at the kernel's end)
    return false;
  }
  __device__ __forceinline__ bool wait3(int b, const Ring3& r, uint32_t err) const { return wait(b + r.b, r.par, err); }
  // tile n's phase of a barrier of three
  __device__ __forceinline__ bool wait3(int b, uint32_t n, uint32_t err) const { return wait(b + n % 3, (n / 3) & 1, err); }
};

// One lane of a warp that has converged, so that what it issues may take operands from the warp's uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Tile j of a unit: its first cache row and how many of its 128 rows are keys.
__device__ __forceinline__ int tile_row0(const MxExpertParams& p, int j) { return j < p.n_main ? j * kKeyTile : p.Smax - kTok; }
__device__ __forceinline__ int tile_live(const MxExpertParams& p, int j) {
  return j < p.n_main ? min(kKeyTile, p.S - j * kKeyTile) : kTok;
}

// ---------------------------------------------------------------------------------- loads
// The largest and the smallest scale of the blocks that hold a code other than zero, over the tile's live rows: 0 and 255 if
// there are none (the whole warp's result; lane: rows lane, lane + 32, .., each row's four blocks at once).
__device__ __noinline__ int2 nonzero_scales(uint32_t tile, int lane, int live) {
  uint32_t top = 0, low = 255;
#pragma unroll 1
  for (int r = lane; r < live; r += 32) {
    uint4 c[4];
    uint32_t sc;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sc) : "r"(tile + kCodes + 4 * r) : "memory");
#pragma unroll
    for (int b = 0; b < 4; ++b) c[b] = ld_shared_v4(tile + r * kMxRowBytes + (((b + (r >> 1)) & 3) << 4));
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool some = ((c[b].x | c[b].y | c[b].z | c[b].w) & 0x77777777u) != 0u;
      const uint32_t e = (sc >> (8 * ((b + (r >> 1)) & 3))) & 255u;
      top = max(top, some ? e : 0u);
      low = min(low, some ? e : 255u);
    }
  }
  return make_int2(static_cast<int>(__reduce_max_sync(0xffffffffu, top)), static_cast<int>(__reduce_min_sync(0xffffffffu, low)));
}

// One warp each for K (kv = 0) and V (kv = 1): loads the tiles, and one tile ahead of the converters looks
// at a tile's scales and publishes its reference. (Its own time a tile is what the rest waits for when it is long:
// the copies' operands are uniform over the warp, as the MMAs' are, and their sources step from tile to tile.)
template <int kv>
__device__ __forceinline__ void producer(const MxExpertParams& p, const Ctx cx) {
  const int lane = threadIdx.x & 31;
  constexpr int kFull = B_FULL + kRing * kv, kEmpty = B_EMPTY + kRing * kv;
  const uint32_t ring = cx.sbase + SM_RING + kv * kRing * kStageBytes;
  volatile int* refs = reinterpret_cast<volatile int*>(cx.smem + SM_REF) + 8 * kv;
  const int total = static_cast<int>(cx.end - cx.start);
  const uint64_t pol = l2_policy_evict_first();
  Seg l = first_seg(cx.start, cx.end, p.T), v = l;  // of the next tile to load, and of the next to look at
  int lj = l.j0, vj = v.j0, ref = 0, peak = 0, ln = 0;
  const uint8_t *codes = nullptr, *scales = nullptr;  // of the next tile to load
  bool jump = true;                                   // they are to be formed anew
  Ring3 at, look;                                     // the places of the two tiles
  bool ok = true;
#pragma unroll 1
  for (int vn = -1; vn < total; ++vn) {
    // tile vn + 1 is loaded once tile vn - 2, whose slot it takes, is converted; then tile vn is looked at
    if (vn + 1 < total) {
      if (jump) {
        const MxAttnLayer& L = p.layer[l.u / kHkv];
        const size_t row = static_cast<size_t>(l.u % kHkv) * p.Smax + tile_row0(p, lj);
        codes = (kv ? L.vc : L.kc) + row * kMxRowBytes;
        scales = (kv ? L.vs : L.ks) + row * kMxRowScales;
      }
      if (vn >= kRing - 1) ok = cx.wait(kEmpty + at.b, at.par ^ 1, kErrProducerWait);
      if (!ok) break;
      const int live = tile_live(p, lj);
      // scale words come in fours: up to three rows past the last key (still in the cache) come along
      const uint32_t cb = live * kMxRowBytes, sb = ((live + 3) & ~3) * kMxRowScales;
      const uint32_t fb = cx.bar(kFull + at.b), dst = ring + at.b * kStageBytes;
      if (elect_one()) {
        mbar_expect_tx(fb, cb + sb);
        bulk_load(dst, codes, cb, fb, pol);
        bulk_load(dst + kCodes, scales, sb, fb, pol);
      }
      __syncwarp();
      ++ln;
      at.step();
      codes += kCodes;
      scales += kScales;
      ++lj;
      jump = lj == l.j1 || lj == p.n_main;
      if (lj == l.j1) {
        next_seg(l, p.T);
        lj = 0;
      }
    }
    if (vn < 0) continue;
    ok = cx.wait(kFull + look.b, look.par, kErrProducerWait);
    if (!ok) break;
    if (vj == v.j0) ref = peak = 0;  // a segment starts: references of its own
    const int live = tile_live(p, vj);
    const uint32_t tile = ring + look.b * kStageBytes;
    const uint4 sc = ld_shared_v4(tile + kCodes + 16 * lane);  // of four rows
    const uint32_t e0 = sc.x & 0x00FF00FFu, e1 = sc.y & 0x00FF00FFu, e2 = sc.z & 0x00FF00FFu, e3 = sc.w & 0x00FF00FFu;
    const uint32_t f0 = (sc.x >> 8) & 0x00FF00FFu, f1 = (sc.y >> 8) & 0x00FF00FFu, f2 = (sc.z >> 8) & 0x00FF00FFu,
                   f3 = (sc.w >> 8) & 0x00FF00FFu;
    const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(e0, e1, e2), __vimax3_u16x2(e3, f0, f1), __vmaxu2(f2, f3));
    const uint32_t w = __vimin3_u16x2(__vimin3_u16x2(e0, e1, e2), __vimin3_u16x2(e3, f0, f1), __vminu2(f2, f3));
    const bool dead = 4 * lane >= live, ragged = 4 * lane + 3 >= live;  // (a ragged end is always looked at closely)
    const int high = dead ? 0 : ragged ? 255 : static_cast<int>(max(m & 0xFFFFu, m >> 16));
    const int deep = ragged ? 255 : static_cast<int>(min(w & 0xFFFFu, w >> 16));
    int low = 0;
    if (__any_sync(0xffffffffu, high > ref + (kMaxField - kRefField) || deep < ref - kWindow)) {
      const int2 t = nonzero_scales(tile, lane, live);
      if (t.x > ref + (kMaxField - kRefField)) ref = t.x;
      else if (t.y < ref - kWindow) ref = kv ? max(t.x, peak - kFollow) : t.x;
      peak = max(peak, ref);
      if (t.y < ref - kWindow) low = kLow;
    }
    if (lane == 0) {
      refs[vn & 7] = ref | low;
      mbar_arrive(cx.bar(B_REF + 8 * kv + (vn & 7)));
    }
    look.step();
    if (++vj == v.j1) {
      next_seg(v, p.T);
      vj = 0;
    }
  }
  __syncwarp();
  if (kv) pdl_launch_dependents();
  if (!ok && lane == 0)  // let every copy already issued land before the CTA gives its shared memory back
    for (int k = 1; k <= kRing && k <= ln; ++k)
      if (!drain_wait(cx.bar(kFull + (ln - k) % 3), ((ln - k) / 3) & 1)) atomicOr(cx.status, kErrDrain);
  __syncwarp();
}

// ----------------------------------------------------------------------------- converters
// One warpgroup each for K (kv = 0) and V (kv = 1): thread = row of a packed tile, whose codes it writes as f16 into a
// tile of the swizzled layout: block b's codes times 2^(scale - ref + 8), 0 for a dead row. A lane takes its row's
// blocks in an order that spreads the lanes over the banks; what follows from that order is formed once, so that a
// block costs 36 instructions for its codes and 7 more.
__device__ __forceinline__ void converter(const MxExpertParams& p, const Ctx cx, int kv) {
  const int row = threadIdx.x & 127;
  const int empty = B_EMPTY + kRing * kv, used = kv ? B_ODONE : B_SFULL, rdy = B_RDY + 2 * kv;
  const volatile int* refs = reinterpret_cast<const volatile int*>(cx.smem + SM_REF) + 8 * kv;
  uint32_t from[4], to[4], sel[4];  // the i-th block's place in the ring's first slot, in the first tile; its factor's selector
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = (i + (row >> 1)) & 3;
    from[i] = cx.sbase + SM_RING + kv * kRing * kStageBytes + row * kMxRowBytes + 16 * b;
    // word k of the block is chunk 4 (b % 2) + k of half b / 2; chunk c of a row sits at c ^ (row % 8)
    to[i] = cx.sbase + (kv ? SM_V : SM_K) + (b >> 1) * kAtom + row * 128 + (((4 * (b & 1)) ^ (row & 7)) << 4);
    sel[i] = b == 0 ? 0x1010 : b == 1 ? 0x5454 : b == 2 ? 0x3232 : 0x7676;
  }
  const uint32_t scale_at = cx.sbase + SM_RING + kv * kRing * kStageBytes + kCodes + 4 * row;
  uint32_t n = 0;
  Ring3 r;
  bool ok = true;
#pragma unroll 1
  for (Seg s = first_seg(cx.start, cx.end, p.T); ok && s.j1 > s.j0; next_seg(s, p.T)) {
#pragma unroll 1
    for (int j = s.j0; j < s.j1; ++j) {
      // (whoever published the reference had seen the tile arrive)
      ok = cx.wait(B_REF + 8 * kv + (n & 7), (n >> 3) & 1, kErrProducerWait);
      if (!ok) break;
      const uint32_t slot = r.b * kStageBytes, tile = (n & 1) * kTile;
      uint32_t sc;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sc) : "r"(scale_at + slot) : "memory");
      const uint32_t add = static_cast<uint32_t>((kRefField - (refs[n & 7] & 255)) & 0xFFFF) * 0x10001u;
      const uint32_t cut = row < tile_live(p, j) ? kMaxField * 0x10001u : 0u;
      const uint32_t f02 = __viaddmin_s16x2_relu(sc & 0x00FF00FFu, add, cut) << 10;         // blocks 0 and 2
      const uint32_t f13 = __viaddmin_s16x2_relu((sc >> 8) & 0x00FF00FFu, add, cut) << 10;  // blocks 1 and 3
      uint4 blk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) blk[i] = ld_shared_v4(from[i] + slot);
      // the f16 buffer held tile n - 2: K's is free once QK(n-2) is done, V's once PV(n-2) is
      ok = n < 2 || cx.wait3(used, r.back(2), kErrProducerWait);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 c = blk[i];
        const uint32_t f = __byte_perm(f02, f13, sel[i]);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const uint32_t at = to[i] + tile;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h[4];
          mx_unpack8(w[k], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(f));
          st_shared_v4(at ^ (16u * k), h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(cx.bar(rdy + (n & 1)));
      mbar_arrive(cx.bar(empty + r.b));
      ++n;
      r.step();
    }
  }
}

// ------------------------------------------------------------------------------------ MMA
// One warp issues S = Q K^T, another O += P V, each tile by tile as its inputs arrive: QK(n) needs K(n)'s tile, its
// segment's Q, and score buffer n % 3, which held P(n-3) until PV(n-3) was done; PV(n) needs P(n), V(n)'s tile and,
// for a segment's first, the accumulator read. (One warp that watched for both took 1,300 cycles a tile to look
// at its barriers, beside 1,370 to issue.) After a segment's last QK the Q buffer is refilled for the next.
//
// The whole warp runs the loop and one elected lane issues: so every operand is uniform over the warp and sits in
// the uniform registers that the instruction takes. From a lone lane's registers each of an MMA's operands
// was moved over first, about 130 cycles an MMA where the tensor core takes 64.
// Both operands' descriptors differ from tile to tile and step to step in their address field alone.
constexpr uint64_t kDescK = (1ull << 61 << 1) | (1ull << 46) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 16);
constexpr uint64_t kDescMN = (1ull << 61 << 1) | (1ull << 46) | (static_cast<uint64_t>(1024 >> 4) << 32) |
                             (static_cast<uint64_t>(kAtom >> 4) << 16);

__device__ __forceinline__ void qk_issuer(const MxExpertParams& p, const Ctx cx) {
  constexpr uint32_t kIdesc = umma_idesc_f16(128, 128, false, false, false);
  const uint64_t qd = kDescK | ((cx.sbase + SM_Q) >> 4), kd = kDescK | ((cx.sbase + SM_K) >> 4);
  auto wait = [&](int b, uint32_t parity) -> bool { return cx.wait(b, parity, kErrMmaWait); };
  uint32_t n = 0, b3 = 0, par = 0, loads = 0;  // b3 = n % 3, par = n / 3 & 1
  bool ok = true;
#pragma unroll 1
  for (Seg s = first_seg(cx.start, cx.end, p.T); ok && s.j1 > s.j0; next_seg(s, p.T)) {
    if (n > 0) ok = wait(B_SFULL + (b3 == 0 ? 2 : b3 - 1), b3 == 0 ? par ^ 1 : par);  // QK(n-1) has read the buffer
    if (!ok) break;
    if (elect_one()) {
      mbar_expect_tx(cx.bar(B_QFULL), kTile);
      bulk_load(cx.sbase + SM_Q, p.q_ws + static_cast<size_t>(s.u) * kQTileBytes, kTile, cx.bar(B_QFULL), l2_policy_evict_first());
    }
    __syncwarp();
    ++loads;
    ok = wait(B_QFULL, (loads - 1) & 1);
#pragma unroll 1
    for (int i = s.j1 - s.j0; ok && i > 0; --i) {
      ok = wait(B_RDY + (n & 1), (n >> 1) & 1) && (n < 3 || wait(B_ODONE + b3, par ^ 1));
      if (!ok) break;
      tc_fence_after();
      const uint64_t k0 = kd + (n & 1) * (kTile >> 4);
      const uint32_t d = TM_S + b3 * 128;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
          umma_f16_ss(d, qd + off, k0 + off, kIdesc, kk > 0);
        }
        umma_commit(cx.bar(B_SFULL + b3));
      }
      __syncwarp();
      ++n;
      if (++b3 == 3) {
        b3 = 0;
        par ^= 1;
      }
    }
  }
  // every load and MMA issued is complete before shared memory and TMEM are given back
  if (elect_one()) {
    if (loads > 0 && !drain_wait(cx.bar(B_QFULL), (loads - 1) & 1)) atomicOr(cx.status, kErrDrain);
    umma_commit(cx.bar(B_DRAIN));
    if (!drain_wait(cx.bar(B_DRAIN), 0)) atomicOr(cx.status, kErrDrain);
  }
  __syncwarp();
}

__device__ __forceinline__ void pv_issuer(const MxExpertParams& p, const Ctx cx) {
  constexpr uint32_t kIdesc = umma_idesc_f16(128, 128, false, false, true);
  const uint64_t vd = kDescMN | ((cx.sbase + SM_V) >> 4);
  auto wait = [&](int b, uint32_t parity) -> bool { return cx.wait(b, parity, kErrMmaWait); };
  const volatile int* refs = reinterpret_cast<const volatile int*>(cx.smem + SM_REF) + 8;
  uint32_t n = 0, b3 = 0, par = 0, seg = 0;
  bool ok = true;
#pragma unroll 1
  for (Seg s = first_seg(cx.start, cx.end, p.T); ok && s.j1 > s.j0; next_seg(s, p.T), ++seg) {
    if (seg > 0) ok = wait(B_OFREE, (seg - 1) & 1);
#pragma unroll 1
    for (int j = s.j0; ok && j < s.j1; ++j) {
      ok = wait(B_RDY + 2 + (n & 1), (n >> 1) & 1) && wait(B_PFULL + b3, par);
      if (!ok) break;
      tc_fence_after();
      const uint64_t v0 = vd + (n & 1) * (kTile >> 4);
      // (the accumulator of a segment's first tile may hold what its low blocks give)
      const uint32_t a = TM_S + b3 * 128, more = j > s.j0 || refs[n & 7] >= kLow;
      const bool own = j >= p.n_main;  // the own tile has 64 keys
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk < 4 || !own) umma_f16_ts(TM_O, a + kk * 8, v0 + kk * (16 * 128 >> 4), kIdesc, kk > 0 ? 1u : more);
        umma_commit(cx.bar(B_ODONE + b3));
      }
      __syncwarp();
      ++n;
      if (++b3 == 3) {
        b3 = 0;
        par ^= 1;
      }
    }
  }
  if (elect_one()) {
    umma_commit(cx.bar(B_DRAIN + 1));
    if (!drain_wait(cx.bar(B_DRAIN + 1), 0)) atomicOr(cx.status, kErrDrain);
  }
  __syncwarp();
}

// -------------------------------------------------------------------------------- softmax
__device__ __noinline__ void scale_accumulator(uint32_t addr, float a) {
  for (int c = 0; c < 128; c += 32) {
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

// P of a tile's first `chunks` 32-key chunks: 16 columns of f16 pairs each.
__device__ __noinline__ void scale_p(uint32_t addr, float a, int chunks) {
  for (int c = 0; c < 2 * chunks; ++c) {
    uint32_t q[8];
    tmem_wait_st();
    tmem_ld8(addr + 8 * c, q);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack_f16x2(q[e]);
      q[e] = pack_f16x2(f.x * a, f.y * a);
    }
    tmem_st8(addr + 8 * c, q);
  }
  tmem_wait_st();
}

// Scores of columns [live, cols) of a tile become -inf (a unit's last cache tile), before they are read.
__device__ __noinline__ void mask_scores(uint32_t addr, int live, int cols) {
  for (int c = live & ~31; c < cols; c += 32) {
    uint32_t v[32];
    tmem_ld32(addr + c, v);
    tmem_wait_ld();
    reg_fence32(v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (c + e >= live) v[e] = __float_as_uint(-INFINITY);
    tmem_st32(addr + c, v);
  }
  tmem_wait_st();
}

// One column, of this warp's 32 lanes.
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(addr) : "memory");
  tmem_wait_ld();
  asm volatile("" : "+r"(v) : : "memory");
  return v;
}
__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
// x 2^d for d <= 127, in two steps: the power alone may leave fp32's range
__device__ __forceinline__ float times_pow2(float x, int d) {
  return x * mx_pow2(max(d, -126)) * mx_pow2(max(min(d + 126, 0), -126));
}
// The rows of K (kv = 0) or V of a tile in the cache.
struct TileRows {
  const uint8_t *codes, *scales;
};
__device__ __forceinline__ TileRows tile_rows(const MxExpertParams& p, int kv, int u, int j) {
  const MxAttnLayer& L = p.layer[u / kHkv];
  const size_t row = static_cast<size_t>(u % kHkv) * p.Smax + tile_row0(p, j);
  return {(kv ? L.vc : L.kc) + row * kMxRowBytes, (kv ? L.vs : L.ks) + row * kMxRowScales};
}
// Block b of a tile's row, if it is below the window of reference ref and not all zeros: its scale, else -1 (the same for
// a whole warp).
__device__ __forceinline__ int low_block(const TileRows& t, int row, int b, int ref, uint4& c) {
  const int e = t.scales[row * kMxRowScales + b];
  if (e >= ref - kWindow) return -1;
  c = *reinterpret_cast<const uint4*>(t.codes + row * kMxRowBytes + 16 * b);
  return ((c.x | c.y | c.z | c.w) & 0x77777777u) != 0u ? e : -1;
}

// Adds to a tile's scores what its blocks of K below the window give, in the scores' unit 2^(ref - 8); r: this thread's row
// of the unit's q tile.
__device__ __noinline__ void low_scores(const MxExpertParams& p, uint32_t addr, int u, int j, int ref, int r) {
  const TileRows t = tile_rows(p, 0, u, j);
  const uint8_t* q = p.q_ws + static_cast<size_t>(u) * kQTileBytes;
  const int live = tile_live(p, j);
#pragma unroll 1
  for (int key = 0; key < live; ++key) {
    float add = 0.f;
    bool any = false;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      uint4 c;
      const int e = low_block(t, key, b, ref, c);
      if (e < 0) continue;
      any = true;
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x[8];
        mx_values8(w[k], 1.f, x);
        const uint4 v = *reinterpret_cast<const uint4*>(q + swz_off(r, 4 * b + k, kQTileBytes / 2));
        const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack_f16x2(h[i]);
          dot = fmaf(f.x, x[2 * i], fmaf(f.y, x[2 * i + 1], dot));
        }
      }
      add += times_pow2(dot, e - ref + kRefField - 15);
    }
    if (any) tmem_st1(addr + key, __float_as_uint(__uint_as_float(tmem_ld1(addr + key)) + add));
  }
  tmem_wait_st();
}

// Adds to the accumulator what a tile's blocks of V below the window give with its weights P, in the accumulator's unit
// 2^(ref - 8); fresh: to zero.
__device__ __noinline__ void low_values(const MxExpertParams& p, uint32_t oa, uint32_t pa, int u, int j, int ref, bool fresh) {
  const TileRows t = tile_rows(p, 1, u, j);
  const int live = tile_live(p, j);
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    float acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.f;
    bool any = fresh;
#pragma unroll 1
    for (int key = 0; key < live; ++key) {
      uint4 c;
      const int e = low_block(t, key, b, ref, c);
      if (e < 0) continue;
      any = true;
      const float2 pp = unpack_f16x2(tmem_ld1(pa + (key >> 1)));
      const float f = times_pow2(key & 1 ? pp.y : pp.x, e - ref + kRefField - 15);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x[8];
        mx_values8(w[k], 1.f, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[8 * k + i] = fmaf(f, x[i], acc[8 * k + i]);
      }
    }
    if (!any) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t o[8];
      if (!fresh) {
        tmem_ld8(oa + 32 * b + 8 * k, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+r"(o[i]) : : "memory");
        o[i] = __float_as_uint((fresh ? 0.f : __uint_as_float(o[i])) + acc[8 * k + i]);
      }
      tmem_st8(oa + 32 * b + 8 * k, o);
    }
  }
  tmem_wait_st();
}

__device__ __forceinline__ void softmax_warps(const MxExpertParams& p, const Ctx cx) {
  const int k = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane = static_cast<uint32_t>(r & ~31) << 16;
  const uint32_t oa = cx.tmem + lane + TM_O;
  const volatile int* refs = reinterpret_cast<const volatile int*>(cx.smem + SM_REF);
  volatile float* run = reinterpret_cast<volatile float*>(cx.smem + SM_M) + r;
  uint32_t base = 0, seg = 0;
  Ring3 rn;  // of this warpgroup's next tile
  rn.b = k;
  bool ok = true;
  auto wait3 = [&](int b, const Ring3& at) -> bool { return cx.wait3(b, at, kErrSoftmaxWait); };
#pragma unroll 1
  for (Seg s = first_seg(cx.start, cx.end, p.T); s.j1 > s.j0; next_seg(s, p.T)) {
    const int nt = s.j1 - s.j0;
    const float qf = p.q_factor[static_cast<size_t>(s.u) * kRows + r] * 0.00390625f;  // K's tiles carry 2^8
    float m = -INFINITY, lsum = 0.f;  // lsum: this warpgroup's keys, in units of 2^m
#pragma unroll 1
    for (int i = static_cast<int>((k + kSoftWg - base % kSoftWg) % kSoftWg); ok && i < nt; i += kSoftWg, rn.step(kSoftWg)) {
      const uint32_t n = base + i;
      const int j = s.j0 + i;
      // (K's reference was there before its tile was converted)
      ok = cx.wait(B_REF + 8 + (n & 7), (n >> 3) & 1, kErrSoftmaxWait) && wait3(B_SFULL, rn);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sa = cx.tmem + lane + TM_S + rn.b * 128;
      // (never 0, as the product of a small query's factor and a small reference can be: a masked score is -inf)
      const int kr = refs[n & 7];
      const float ct = fmaxf(qf * mx_scale(kr & 255), 0x1p-126f);
      // what V's reference, if it moved from the tile before (in the same segment) to this one, makes of the accumulator
      const int vr = refs[8 + (n & 7)];
      float scale = 1.f;
      if (i > 0) {
        const int d = (refs[8 + ((n - 1) & 7)] & 255) - (vr & 255);
        if (d != 0) scale = d < -126 ? 0.f : mx_pow2(d);
      }
      const int live = tile_live(p, j), chunks = j < p.n_main ? 4 : 2;
      if (kr >= kLow) low_scores(p, sa, s.u, j, kr & 255, r);
      if (live < 32 * chunks) mask_scores(sa, live, 32 * chunks);
      // (the other warpgroups' first tiles of a segment start from its first tile's maximum: their own would seldom do)
      if (i > 0 && i < kSoftWg) {
        ok = wait3(B_MDONE, rn.back(i));
        if (!ok) break;
        m = *run;
      }
      const float2 ct2 = make_float2(ct, ct);
      // P goes over the scores' first columns: chunk c's 16 columns of pairs hold scores of chunks <= c.
      // The maximum is not looked for: a chunk's sum that passes 2^15 tells that it has to rise (f16 holds
      // weights up to 2^16), and then, as in the segment's first chunk, the chunk is done once more.
      float tsum = 0.f;
      bool first = __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint32_t pk[16];
        float cs;
        bool rise = first, again = !first;
        first = false;
#pragma unroll 1
        for (;;) {
          uint32_t v[32];
          tmem_ld32(sa + 32 * c, v);
          tmem_wait_ld();
          reg_fence32(v);
          if (rise) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * ct - kLift), a = ex2_approx(m - mn);
            if (c > 0) scale_p(sa, a, c);  // the earlier chunks' P moves too
            tsum *= a;
            lsum *= a;
            m = mn;
          }
          const float2 neg = make_float2(-m, -m);
          float2 ts[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), ct2, neg);
            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            ts[e & 1] = __fadd2_rn(ts[e & 1], make_float2(p0, p1));
            pk[e] = pack_f16x2(p0, p1);
          }
          const float2 tt = __fadd2_rn(ts[0], ts[1]);
          cs = tt.x + tt.y;
          if (!again || !__any_sync(0xffffffffu, cs > 32768.f)) break;
          rise = true;
          again = false;
        }
        tsum += cs;
        tmem_st16(sa + 16 * c, pk);
      }
      lsum += tsum;
      tmem_wait_st();
      // the maximum that tile n - 1 left, nearly always this tile's too: else the larger one holds from here on
      if (i > 0) {
        ok = wait3(B_MDONE, rn.back(1));
        if (!ok) break;
        const float before = *run;
        if (__any_sync(0xffffffffu, before != m)) {
          const float mn = fmaxf(m, before), a = ex2_approx(m - mn);
          if (__any_sync(0xffffffffu, a != 1.f)) scale_p(sa, a, chunks);
          lsum *= a;
          m = mn;
          scale *= ex2_approx(before - mn);
          *run = m;
        }
      } else {
        *run = m;
      }
      mbar_arrive(cx.bar(B_MDONE + rn.b));
      const bool moves = __any_sync(0xffffffffu, scale != 1.f);
      if (moves || vr >= kLow) {  // the accumulator changes: stable once PV(n-1) is done, or the segment before is read
        if (i > 0) ok = wait3(B_ODONE, rn.back(1));
        else if (seg > 0) ok = cx.wait(B_OFREE, (seg - 1) & 1, kErrSoftmaxWait);
        if (!ok) break;
        tc_fence_after();
        if (moves) scale_accumulator(oa, scale);
        if (vr >= kLow) low_values(p, oa, sa, s.u, j, vr & 255, i == 0);
      }
      tc_fence_before();
      mbar_arrive(cx.bar(B_PFULL + rn.b));
    }
    // ---- the segment's end: the last PV, the warpgroups' sums; thread (k, r), k < 2, takes columns [64 k, 64 k + 64)
    const uint32_t last = base + nt - 1;
    if (ok) ok = cx.wait3(B_ODONE, last, kErrSoftmaxWait);
    // (by segment parity: a warpgroup may be here while the other still reads the segment before; it cannot
    // pass this segment's barrier before that)
    float2* xch = reinterpret_cast<float2*>(cx.smem + SM_X) + (seg & 1) * kSoftWg * kRows;
    xch[k * kRows + r] = make_float2(m, lsum);
    ok = bar_sync_and(kBarSoftmax, kSoftmax, ok);
    if (ok && k < 2) {
      tc_fence_after();
      float M = -INFINITY, L = 0.f;  // (the maximum never falls: the last tile's is the largest)
#pragma unroll
      for (int w = 0; w < kSoftWg; ++w) M = fmaxf(M, xch[w * kRows + r].x);
#pragma unroll
      for (int w = 0; w < kSoftWg; ++w) L += ex2_approx(xch[w * kRows + r].x - M) * xch[w * kRows + r].y;
      // O is in units of 2^(R - 127 - 8): a value is o * inv * f
      const float inv = 1.0f / L * 0.00390625f;
      const int rv = refs[8 + (last & 7)] & 255, l = s.u / kHkv, g = s.u % kHkv;
      const bool full = s.j0 == 0 && s.j1 == p.T;
      const uint32_t col = oa + 64 * k;
      const float f = mx_scale(rv);
      const size_t sl = static_cast<size_t>(blockIdx.x) * 2 + (base == 0 ? 0 : 1);
      uint4* dst = full ? reinterpret_cast<uint4*>(p.layer[l].out + (static_cast<size_t>(g) * kRows + r) * kD + 64 * k)
                        : p.part_o + (sl * kPartChunks + 8 * k) * kRows + r;
      const size_t step = full ? 1 : kRows;
      if (!full && k == 0) p.part_lse[sl * kMxPartRows * kRows + r] = M + log2f(L);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32], pk[16];
        tmem_ld32(col + 32 * h, v);
        tmem_wait_ld();
        reg_fence32(v);
        if (h == 1) {
          tc_fence_before();
          mbar_arrive(cx.bar(B_OFREE));  // the accumulator is read
        }
        float up = 1.f;
        if (!full) {
          // a part: f16 (11 bits: the bf16 output has 8), the 32 channels times the power of two that puts their largest
          // magnitude in [2^14, 2^15)
          float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], fabsf(__uint_as_float(v[e])), fabsf(__uint_as_float(v[e + 1])));
          const float amax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * inv * f;
          const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -126), 112);
          up = mx_pow2(-ex);
          p.part_lse[(sl * kMxPartRows + 1 + 2 * k + h) * kRows + r] = mx_pow2(ex);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = __uint_as_float(v[2 * e]) * inv * f * up, y = __uint_as_float(v[2 * e + 1]) * inv * f * up;
          pk[e] = full ? pack_bf16x2(x, y) : pack_f16x2(x, y);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) dst[(4 * h + c) * step] = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
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
  cx.failed = reinterpret_cast<volatile uint32_t*>(smem + SM_FAILED);
  cx.status = p.status;
  cx.start = cta_tile_start(blockIdx.x, p.W, gridDim.x);
  cx.end = cta_tile_start(blockIdx.x + 1, p.W, gridDim.x);
  const int warp = threadIdx.x >> 5;
  if (warp == 1) {
    for (int b = threadIdx.x & 31; b < kNumBars; b += 32) mbar_init(cx.bar(b), bar_count(b));
    if ((threadIdx.x & 31) == 0) *cx.failed = 0u;
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
  constexpr int kConv0 = kSoftmax / 32, kIssue0 = kConv0 + 2 * kConvert / 32;  // the roles' first warps
  if (warp < kConv0) {
    if constexpr (kRegSoftmax > kRegLaunch) regs_up<kRegSoftmax>();
    softmax_warps(p, cx);
  } else if (warp < kIssue0) {
    regs_down<kRegConvert>();
    converter(p, cx, warp >= kConv0 + kConvert / 32);
  } else {
    regs_down<kRegIssue>();
    if (warp == kIssue0) producer<0>(p, cx);
    if (warp == kIssue0 + 1) producer<1>(p, cx);
    if (warp == kIssue0 + 2) qk_issuer(p, cx);
    if (warp == kIssue0 + 3) pv_issuer(p, cx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(cx.tmem, kTmemCols);
  if (threadIdx.x == 0 && *cx.failed != 0u) atomicOr(p.status, *cx.failed);
}

// The units that the CTA ranges cut: grid (units, 16), thread = one row's 8 columns.
__global__ void __launch_bounds__(kRows) mxfp4_merge_kernel(const __grid_constant__ MxMergeParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const SplitUnit su = p.split[blockIdx.x];
  __nv_bfloat16* out = p.out[su.u / kHkv];
  if (su.nparts == 2) merge_row_chunk<2, kD / 32>(p.part_o, p.part_lse, su, blockIdx.y, threadIdx.x, out);
  else merge_row_chunk<20, kD / 32>(p.part_o, p.part_lse, su, blockIdx.y, threadIdx.x, out);
}

cudaError_t mxfp4_attention_set_attributes() {
  return cudaFuncSetAttribute(mxfp4_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(mxa::kSmemBytes));
}

cudaError_t launch_mxfp4_prologue(const MxPrologueParams& p, int n_layers, cudaLaunchConfig_t cfg) {
  cfg.blockDim = dim3(256);
  const bool split = n_layers <= 4;
  cfg.gridDim = dim3(split ? 8 : 2, kHkv, n_layers);
  return cudaLaunchKernelEx(&cfg, split ? mxfp4_prologue_kernel<true> : mxfp4_prologue_kernel<false>, p);
}

cudaError_t launch_mxfp4_attention(const MxExpertParams& p, cudaLaunchConfig_t cfg) {
  cfg.blockDim = dim3(mxa::kThreads);
  cfg.dynamicSmemBytes = mxa::kSmemBytes;
  return cudaLaunchKernelEx(&cfg, mxfp4_attention_kernel, p);
}

cudaError_t launch_mxfp4_merge(const MxMergeParams& p, int n_split, cudaLaunchConfig_t cfg) {
  cfg.gridDim = dim3(n_split, kPartChunks);
  cfg.blockDim = dim3(kRows);
  return cudaLaunchKernelEx(&cfg, mxfp4_merge_kernel, p);
}

}  // namespace ea
