// mxfp4_decode.cu — one token's attention over 4-bit caches.
//
// Per (layer, kv head) unit, with the 8 query heads q_h of the GQA group (normed and roped):
//   the new k (normed, roped) and v rows encoded into cache row pos;
//   s[key][h] = sum_b 2^ek[key][b] (codes of block b . q_h)    over the four 32-channel blocks b
//   out[h][d] = sum_key P[key][h] 2^ev[key][b(d)] code[key][d] / sum_key P[key][h],  P = 2^(s - m)
//
// What bounds it: HBM, 136 bytes a key and head for 4 x 8 x 128 flops. The codes have to be widened on the
// way to the tensor core, and through shared memory they would cost more than the read itself: 16-bit
// tiles are 64 KB written and 64 KB read per 128 keys (1,000 cycles at 128 bytes a cycle) where HBM
// takes 700. So the operands are formed in registers (mma.sync fragments straight from the packed
// codes), shared memory holds codes only, and every warp runs by itself: its own ring, its own keys, its
// own running maximum, no barrier until a unit ends.
//   K: a 16-byte block of a row is one matrix row of ldmatrix; a thread's word holds eight codes of one
//      key, cvt turns each byte into an f16 pair, and one accumulator per block b takes the two
//      k = 16 steps of its 32 channels (A = 16 keys, B = the 8 heads). The blocks' scales multiply the
//      four sums in fp32, so that K is exact at any scale.
//   V: ldmatrix.trans gives a thread four codes of key 2t (low half) and of key 2t + 1 (high half);
//      exchanging nibbles pairs the two keys in a byte, and cvt gives the f16 pair along the keys
//      that V^T (A = 16 channels, K = 16 keys) needs. V's scales go into P instead, once per block of
//      channels: 8 products of f16 pairs a step in place of 32.
// P 2^(ev - R) is held in f16, as the product of two f16 numbers. m stands 2^8 below a warp's maximum and is raised when a
// score passes that by 2^4 (so the largest P is 2^8 to 2^12); R is a running reference of the warp, the largest scale of a
// block that is not all zeros, as of the last time it was exceeded by 2^1, put at 2^2. So a weight keeps 11 bits down to
// 2^-22 of the largest, its product with a scale down to 2^-24, and a weight that is lost below is at most 2^-33 of the
// largest (with m at the maximum itself weights below 2^-25 counted as zero: of 350,000 keys, a warp's share of the
// longest cache, 1 % of the largest). A block more than 2^10 below R is not multiplied so: a chunk that holds such
// blocks goes over them again, at a reference of their own, and adds what they give in fp32 (it takes about three times
// as long).
//
// Work decomposition: the units' keys in chunks of 32, unit-major, one contiguous range per CTA; a CTA's
// twelve compute warps take its chunks in turn (64 layers at pos 4700: 79 us with eight). Where a unit ends a
// warp leaves its partial in shared memory and goes on with the next: four further warps join the
// partials, after they have prepared the next units' q rows and encoded the new rows. (When all warps met at a
// unit's end, each lost up to a chunk's time there: 64 layers 72.7 us, 65.7 without.) A unit cut over several CTAs
// is merged by the part that finishes last.
//
// Measured: 64 layers at pos 4700 65.3 us (5.1 TB/s, 74 % of a plain copy), 4 layers at pos 131070 100 us (5.7 TB/s,
// 84 %); 1 layer at pos 4700 8.3 us, at pos 300 5.0 us. What holds it below the copy: the conversions share the ALU
// pipe (60 % busy) and the issue slots (55 %) with the softmax; at one layer the latencies of the launch, one
// chunk's load, the parts' arrival and the merge.
#include "mxfp4.cuh"
#include "rope.cuh"

namespace ea {
namespace mxd {

constexpr int kWarps = kMxDecodeWarps;       // compute warps (at least 8: a unit's merge takes one per head)
constexpr int kCompute = 32 * kWarps;
constexpr int kPrep = 128;                   // two warps for the 8 q rows, one each for the k row and the v row
constexpr int kThreads = kCompute + kPrep;
constexpr int kKeys = 32;                    // keys per chunk
constexpr int kStages = 3;
constexpr uint32_t kCodes = kKeys * kMxRowBytes, kScales = kKeys * kMxRowScales;
constexpr uint32_t kStageBytes = 2 * kCodes + 2 * kScales;  // K codes, V codes, K scales, V scales
constexpr uint32_t SM_RING = 0;
constexpr uint32_t kFactorBytes = kKeys * 16 + kKeys * 8;  // a chunk's scales as factors: K's fp32, V's f16
constexpr uint32_t SM_FACT = SM_RING + kWarps * kStages * kStageBytes;
constexpr uint32_t SM_PART = SM_FACT + kWarps * kFactorBytes;  // [warp][head][132] fp32
constexpr uint32_t kPartRow = 132;           // 128 channels + 4 words: heads 2 apart fall in other banks
constexpr uint32_t SM_ML = SM_PART + kWarps * kRepText * kPartRow * 4;  // [warp][head] (m, l)
constexpr uint32_t SM_R = SM_ML + kWarps * kRepText * 8;                // [warp] reference scale byte
constexpr uint32_t SM_Q = (SM_R + kWarps * 4 + 15) & ~15u;              // 2 x [8 heads][128] f16
constexpr uint32_t SM_QF = SM_Q + 2 * kRepText * kD * 2;                // 2 x [8 heads] score factor
constexpr uint32_t kNewBytes = 2 * kMxRowBytes + 8;
constexpr uint32_t SM_NEW = SM_QF + 2 * kRepText * 4;                   // 2 x (K codes, V codes, scale words)
constexpr uint32_t SM_FLAG = SM_NEW + 2 * 144;
constexpr uint32_t SM_BAR = SM_FLAG + 16;
// by segment: a unit's q (and new rows) are there (in the buffer of its parity); its partials are; they are read
constexpr uint32_t B_QRDY = 0, B_PART = 2, B_READ = 3, kNumBars = 4;
constexpr uint32_t kSmemBytes = SM_BAR + 8 * kNumBars;
constexpr uint32_t kBarPrep = 1, kBarLast = 2, kBarEnd = 3;  // named barriers: the preparing warps; with four compute warps, at the end
static_assert(kNewBytes <= 144 && kSmemBytes <= 232448, "shared memory budget of one sm_103 CTA");
static_assert(kStageBytes % 128 == 0 && SM_FACT % 16 == 0 && SM_PART % 16 == 0 && SM_ML % 8 == 0 && SM_Q % 16 == 0 &&
                  SM_QF % 8 == 0 && SM_NEW % 16 == 0 && SM_BAR % 8 == 0,
              "alignment of the vector accesses");

// P 2^(ev - R): P <= 2^(kLift + kLazy); a block at the reference has the factor 2^(kRefField - 15) (f16 exponent fields);
// fields above kMaxField only occur for all-zero blocks and are cut there.
constexpr float kLift = 8.0f, kLazy = 4.0f;
constexpr int kRefField = 17, kMaxField = 18;
constexpr int kWindow = 10;  // blocks from R - kWindow on are multiplied in f16
static_assert(kLift + kLazy + kMaxField - 15 <= 15 && kRefField - kWindow >= 1, "products within f16");

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same onto a zero accumulator
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
  return x;
}
// x << 4 as a product: the multipliers are idle here, the logic pipe is what bounds the warps
__device__ __forceinline__ uint32_t times16(uint32_t x) {
  uint32_t r;
  asm("mul.lo.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(16u));
  return r;
}
// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// CTA c's first chunk: parts > 0: the unit's chunks in that many ranges; else all chunks in ranges whose
// lengths differ by at most one.
__device__ __forceinline__ uint32_t cta_start(const MxDecodeParams& p, uint32_t c) {
  if (p.parts > 0) return c / p.parts * p.T + c % p.parts * p.T / p.parts;
  return c * p.per_cta + min(c, p.extra);
}
__device__ __forceinline__ uint32_t cta_of(const MxDecodeParams& p, uint32_t x) {
  if (p.parts > 0) {  // x is a unit's first or last chunk
    return x / p.T * p.parts + (x % p.T == 0 ? 0 : p.parts - 1);
  }
  const uint32_t split = p.extra * (p.per_cta + 1);
  return x < split ? x / (p.per_cta + 1) : p.extra + (x - split) / p.per_cta;
}

// ------------------------------------------------------------------------------ chunk loads
// A warp's next chunk to load: chunk j of unit u, and where this lane's pieces of it start.
struct Cursor {
  uint32_t u, j;
  const uint8_t *k, *v;  // codes, at this lane's 16 bytes
  const uint8_t* s;      // scales: K's (lanes 0-7) or V's (lanes 8-15), at this lane's 16 bytes
};
__device__ __forceinline__ void cursor_unit(const MxDecodeParams& p, Cursor& c, int lane) {
  const MxAttnLayer& L = p.layer[c.u / kHkv];
  const size_t row = static_cast<size_t>(c.u % kHkv) * p.Smax + static_cast<size_t>(c.j) * kKeys;
  c.k = L.kc + row * kMxRowBytes + 16 * lane;
  c.v = L.vc + row * kMxRowBytes + 16 * lane;
  c.s = (lane < 8 ? L.ks : L.vs) + row * kMxRowScales + 16 * (lane & 7);
}
// The same warp's next chunk, kWarps further on.
__device__ __forceinline__ void cursor_next(const MxDecodeParams& p, Cursor& c, int lane) {
  c.j += kWarps;
  c.k += kWarps * kCodes;
  c.v += kWarps * kCodes;
  c.s += kWarps * kScales;
  if (c.j >= p.T) {
    c.u += c.j / p.T;
    c.j %= p.T;
    cursor_unit(p, c, lane);
  }
}
// Loads the rows of the cursor's chunk that lie before pos (the others arrive as zeros; row pos is put in
// by the warp itself). A chunk's codes are contiguous: lane i takes 16-byte pieces i, i + 32, ..; block b
// of row r goes to 16-byte slot b ^ (r / 2 % 4) of its row, so that the eight rows of an ldmatrix phase
// fall in different banks. `loff` is the lane's first piece's place.
__device__ __forceinline__ void load_chunk(const MxDecodeParams& p, const Cursor& c, uint32_t dst, uint32_t loff, int lane) {
  const int valid = p.pos - static_cast<int>(c.j) * kKeys;
  const uint32_t to = dst + loff;
  if (valid >= kKeys) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cp16(to + 512 * q, c.k + 512 * q, 16);
      cp16(to + kCodes + 512 * q, c.v + 512 * q, 16);
    }
    if (lane < 16) cp16(dst + 2 * kCodes + 16 * lane, c.s, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool live = 8 * q + (lane >> 2) < valid;  // a row that is not read is named by the chunk's first
      cp16(to + 512 * q, live ? c.k + 512 * q : c.k - 16 * lane, live ? 16 : 0);
      cp16(to + kCodes + 512 * q, live ? c.v + 512 * q : c.v - 16 * lane, live ? 16 : 0);
    }
    if (lane < 16) {
      const int bytes = max(0, min(16, 4 * valid - 16 * (lane & 7)));
      cp16(dst + 2 * kCodes + 16 * lane, bytes > 0 ? c.s : c.s - 16 * (lane & 7), bytes);
    }
  }
}

// ------------------------------------------------------------------------------ preparation
// Unit u's q rows (octets 0-7: normed, roped, f16 times a power of two that puts the row's largest magnitude in
// [1, 2)), and, when the segment holds the unit's last chunk, the new k row (octet 8) and v row (octet 12): into
// shared memory for this CTA, into the cache, and their values to the caller.
__device__ __forceinline__ void prepare(const MxDecodeParams& p, uint8_t* smem, uint32_t u, bool last, int buf, int tid) {
  const int l = u / kHkv, g = u % kHkv, oct = tid >> 3, i = tid & 7, dl = 8 * i, dh = 64 + 8 * i;
  const int kind = tid < 64 ? 0 : tid < 96 ? 1 : 2;  // (the same for a warp; octets 8-11 all hold the k row)
  if (kind > 0 && !last) return;
  const MxAttnLayer& L = p.layer[l];
  const __nv_bfloat16* src = kind == 0 ? L.q_raw + (static_cast<size_t>(g) * kRepText + oct) * kD
                                       : (kind == 1 ? L.k_raw : L.v_raw) + static_cast<size_t>(g) * kD;
  const __nv_bfloat16* gam = kind == 0 ? L.q_gamma : L.k_gamma;
  const uint4 r0 = *reinterpret_cast<const uint4*>(src + dl), r1 = *reinterpret_cast<const uint4*>(src + dh);
  const uint4 r2 = *reinterpret_cast<const uint4*>(gam + dl), r3 = *reinterpret_cast<const uint4*>(gam + dh);
  float xl[8], xh[8], gl[8], gh[8], cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = p.rot[dl + e].x;
    sn[e] = p.rot[dl + e].z;
  }
  unpack_bf16x8(r0, xl);
  unpack_bf16x8(r1, xh);
  unpack_bf16x8(r2, gl);
  unpack_bf16x8(r3, gh);
  if (kind == 0) {
    float yl[8], yh[8], factor;
    norm_rope(xl, xh, gl, gh, cs, sn, yl, yh);
    f16_row(yl, yh, p.scale_log2, factor);
    uint8_t* q = smem + SM_Q + (buf * kRepText + oct) * kD * 2;
    *reinterpret_cast<uint4*>(q + 2 * dl) = pack8(yl, true);
    *reinterpret_cast<uint4*>(q + 2 * dh) = pack8(yh, true);
    if (i == 0) reinterpret_cast<float*>(smem + SM_QF)[buf * kRepText + oct] = factor;
    return;
  }
  auto angle = [&](int e, Pair& c, Pair& s) {
    const float4 a = p.rot[dl + e];
    c = {a.x, a.y};
    s = {a.z, a.w};
  };
  uint32_t cl, ch;
  int el, eh;
  if (kind == 1) mx_encode_k_octet<false>(xl, xh, gl, gh, cs, sn, angle, cl, ch, el, eh);
  else mx_encode_octet<false>(xl, xh, cl, ch, el, eh);
  if ((oct & 3) != 0) return;
  const int v = kind - 1;
  uint8_t* nw = smem + SM_NEW + buf * 144;
  mx_store_octet(cl, ch, el, eh, nw + 64 * v, nw + 128 + 4 * v, 0, i, nullptr);
  __nv_bfloat16* val = v ? L.v_new : L.k_new;
  mx_store_octet(cl, ch, el, eh, v ? L.vc : L.kc, v ? L.vs : L.ks, static_cast<size_t>(g) * p.Smax + p.pos, i,
                 val == nullptr ? nullptr : val + static_cast<size_t>(g) * kD);
}

// --------------------------------------------------------------------------------- one chunk
struct Warp {
  float m[2], l[2];  // heads 2t, 2t + 1: reference maximum (log2 units); sum over this thread's keys
  float o[8][4];     // O^T: tile 2b + h of block b, rows = channels 32 b + 4 (lane/4) + 2 h + {0, 1}
  int ref;           // R as a scale byte
};

// Raises the reference maximum of both heads to 2^kLift below the chunk's (x: scores in log2 units).
__device__ __forceinline__ void raise_max(Warp& w, float x0, float x1) {
#pragma unroll
  for (int m = 4; m <= 16; m <<= 1) {
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, m));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, m));
  }
  const float n0 = fmaxf(w.m[0], x0 - kLift), n1 = fmaxf(w.m[1], x1 - kLift);
  const float a0 = ex2_approx(w.m[0] - n0), a1 = ex2_approx(w.m[1] - n1);
  w.m[0] = n0;
  w.m[1] = n1;
  w.l[0] *= a0;
  w.l[1] *= a1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w.o[i][0] *= a0;
    w.o[i][1] *= a1;
    w.o[i][2] *= a0;
    w.o[i][3] *= a1;
  }
}

// Words of ldmatrix.trans of V's codes: f16 pairs of channels 4g + {0, 2} (he) and {1, 3} (ho), keys (2t, 2t + 1), then
// (2t + 8, 2t + 9).
__device__ __forceinline__ void value_pairs(uint32_t r0, uint32_t r1, uint32_t (&he)[4], uint32_t (&ho)[4]) {
  const uint32_t lo = __byte_perm(r0, r1, 0x5410), hi = __byte_perm(r0, r1, 0x7632);
  mx_unpack8(select_bits(lo, times16(hi), 0x0F0F0F0Fu), he);
  mx_unpack8(select_bits(lo >> 4, hi, 0x0F0F0F0Fu), ho);
}

// The largest (kTop) or smallest scale of the chunk's V blocks that have a code other than zero, of those below `below`;
// -1, or 255, if there is none (lane = key; the whole warp's result).
template <bool kTop>
__device__ __forceinline__ int nonzero_scale(uint32_t st, int lane, int below) {
  const uint32_t sc = ld_shared_u32(st + 2 * kCodes + kScales + 4 * lane);
  int r = kTop ? -1 : 255;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint4 c = ld_shared_v4(st + kCodes + lane * kMxRowBytes + ((b ^ ((lane >> 1) & 3)) << 4));
    const int e = (sc >> (8 * b)) & 255;
    if (((c.x | c.y | c.z | c.w) & 0x77777777u) != 0u && e < below) r = kTop ? max(r, e) : min(r, e);
  }
  return kTop ? __reduce_max_sync(0xffffffffu, r) : __reduce_min_sync(0xffffffffu, r);
}

// Some scale of the chunk is far from the reference: raises the reference to the largest scale of a block that has a code
// other than zero, if that is far above it; whether such a block lies below the reference's window.
__device__ __forceinline__ bool look_at_scales(Warp& w, uint32_t st, int lane) {
  const int t = nonzero_scale<true>(st, lane, 256);
  if (t > w.ref + (kMaxField - kRefField)) {
    const float a = w.ref - t < -126 ? 0.f : mx_pow2(w.ref - t);
    w.ref = t;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) w.o[i][k] *= a;
  }
  return nonzero_scale<false>(st, lane, 256) < w.ref - kWindow;
}

// Writes the factors of the chunk's V blocks whose scale is below `below`, at a reference of their own: the largest such
// scale, which it returns (-1: there is none).
__device__ __forceinline__ int low_factors(uint32_t st, uint32_t fact, int lane, int below) {
  const int top = nonzero_scale<true>(st, lane, below);
  const uint32_t vs = ld_shared_u32(st + 2 * kCodes + kScales + 4 * lane);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int e = (vs >> (8 * b)) & 255, field = e < below && e >= top - kWindow ? min(e - top + kRefField, kMaxField) : 0;
    st_shared_u16(fact + 512 + 16 * (lane >> 1) + 4 * b + 2 * (lane & 1), static_cast<uint16_t>(field << 10));
  }
  __syncwarp();
  return top;
}

// The V blocks below the reference's window (their factors were 0), window by window, each from zero and added in fp32.
// pb: the weights of both 16-key steps; a0, a1: as in chunk(). (A function of its own, on a copy of the accumulators: in
// line it costs the chunks that do not need it 5 %.)
__device__ __noinline__ void low_values(float* o, int ref, uint4 pb, uint32_t st, uint32_t fact, uint32_t a0, uint32_t a1) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  int below = ref - kWindow;
#pragma unroll 1
  for (;;) {
    __syncwarp();
    const int top = low_factors(st, fact, lane, below);
    if (top < 0) return;
    const float down = top - ref < -126 ? 0.f : mx_pow2(top - ref);
#pragma unroll 1
    for (int a = 0; a < 2; ++a) {
      const uint4 ua = ld_shared_v4(fact + 512 + 16 * (8 * a + t)), ub = ld_shared_v4(fact + 512 + 16 * (8 * a + t + 4));
      const uint32_t fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w};
      uint32_t r[8];
      ldm4t(a0 + kCodes + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(r));
      ldm4t(a1 + kCodes + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(r + 4));
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t q0 = hmul2(a ? pb.z : pb.x, fa[b]), q1 = hmul2(a ? pb.w : pb.y, fb[b]);
        uint32_t he[4], ho[4];
        value_pairs(r[2 * b], r[2 * b + 1], he, ho);
        float d[2][4];
        mma16816_first(d[0], {he[0], ho[0], he[2], ho[2]}, q0, q1);
        mma16816_first(d[1], {he[1], ho[1], he[3], ho[3]}, q0, q1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[8 * b + 4 * h + k] = fmaf(down, d[h][k], o[8 * b + 4 * h + k]);
      }
    }
    below = top - kWindow;
  }
}

// `fact`: the warp's 768 bytes for the chunk's factors; `live`: the chunk's keys from here on are masked
__device__ __forceinline__ void chunk(Warp& w, const uint32_t (&q)[4][4], const float (&qf)[2], uint32_t st, uint32_t fact,
                                      int live, int lane) {
  const int g = lane >> 2, t = lane & 3;
  // ldmatrix: lane i names row (i & 7) + 8 ((i >> 3) & 1) of block (i >> 4) + {0, 2}
  const int lr = lane & 15;
  const uint32_t lrow = st + lr * kMxRowBytes;
  const uint32_t sw = (lr >> 1) & 3, b0 = lane >> 4;
  const uint32_t a0 = lrow + ((b0 ^ sw) << 4), a1 = lrow + (((b0 + 2) ^ sw) << 4);
  uint32_t rk[2][8];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    ldm4(a0 + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(rk[a]));
    ldm4(a1 + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(rk[a] + 4));
  }
  // The scales become factors once per key (lane = key), not once per thread that needs them:
  // K's four as fp32, at fact + 16 key; V's four as f16 2^(ev - R + 2), the pair of keys 2i and 2i + 1 of
  // block b at fact + 512 + 16 i + 4 b. (With K's codes read before, and V's factors formed between the products: 64
  // layers at pos 4700 65.8 -> 63.7 us, 4 layers at pos 131070 104 -> 98.)
  {
    const uint32_t ks = ld_shared_u32(st + 2 * kCodes + 4 * lane);
    // (a K scale byte of 0, 2^-127, is taken as 0: such a block adds nothing to a score)
    st_shared_v4(fact + 16 * lane, (ks << 23) & 0x7F800000u, (ks << 15) & 0x7F800000u, (ks << 7) & 0x7F800000u,
                 (ks >> 1) & 0x7F800000u);
    __syncwarp();
  }
  bool low = false;
  float x[2][4];  // [16 keys][key g: heads 2t, 2t+1; key g + 8: the same]
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const uint32_t(&r)[8] = rk[a];
    const uint4 u0 = ld_shared_v4(fact + 16 * (16 * a + g)), u1 = ld_shared_v4(fact + 16 * (16 * a + g + 8));
    const uint32_t f0[4] = {u0.x, u0.y, u0.z, u0.w}, f1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t h0[4], h1[4];  // f16 pairs of the eight codes of keys g and g + 8
      mx_unpack8(r[2 * b], h0);
      mx_unpack8(r[2 * b + 1], h1);
      float d[4];
      mma16816_first(d, {h0[0], h1[0], h0[1], h1[1]}, q[b][0], q[b][1]);
      mma16816(d, {h0[2], h1[2], h0[3], h1[3]}, q[b][2], q[b][3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __uint_as_float(k < 2 ? f0[b] : f1[b]);
        x[a][k] = b == 0 ? f * d[k] : fmaf(f, d[k], x[a][k]);
      }
    }
    if (a == 0) {  // (here, while the products run)
      const uint32_t vs = ld_shared_u32(st + 2 * kCodes + kScales + 4 * lane);
      uint32_t v02 = vs & 0x00FF00FFu, v13 = (vs >> 8) & 0x00FF00FFu;
      const uint32_t top = __vmaxu2(v02, v13), end = __vminu2(v02, v13);
      if (__any_sync(0xffffffffu, static_cast<int>(max(top & 0xFFFFu, top >> 16)) > w.ref + (kMaxField - kRefField) ||
                                      static_cast<int>(min(end & 0xFFFFu, end >> 16)) < w.ref - kWindow)) {
        low = look_at_scales(w, st, lane);
        if (low) {  // the blocks below the window have their turn later: no factor here
          const uint32_t from = static_cast<uint32_t>((w.ref - kWindow) & 0xFFFF) * 0x10001u;
          v02 = select_bits(v02, 0xC000C000u, __vcmpges2(v02, from));
          v13 = select_bits(v13, 0xC000C000u, __vcmpges2(v13, from));
        }
      }
      const uint32_t add = static_cast<uint32_t>((kRefField - w.ref) & 0xFFFF) * 0x10001u;
      const uint32_t f02 = __viaddmin_s16x2_relu(v02, add, kMaxField * 0x10001u) << 10;
      const uint32_t f13 = __viaddmin_s16x2_relu(v13, add, kMaxField * 0x10001u) << 10;
      const uint32_t at = fact + 512 + 16 * (lane >> 1) + 2 * (lane & 1);
      st_shared_u16(at, static_cast<uint16_t>(f02));
      st_shared_u16(at + 4, static_cast<uint16_t>(f13));
      st_shared_u16(at + 8, static_cast<uint16_t>(f02 >> 16));
      st_shared_u16(at + 12, static_cast<uint16_t>(f13 >> 16));
      __syncwarp();
    }
  }
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[a][k] *= qf[k & 1];
  if (live < kKeys) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (16 * a + g + 4 * (k & 2) >= live) x[a][k] = -INFINITY;
  }
  const float mx0 = fmax3(fmaxf(x[0][0], x[0][2]), x[1][0], x[1][2]);
  const float mx1 = fmax3(fmaxf(x[0][1], x[0][3]), x[1][1], x[1][3]);
  if (__any_sync(0xffffffffu, mx0 > w.m[0] + (kLift + kLazy) || mx1 > w.m[1] + (kLift + kLazy))) raise_max(w, mx0, mx1);
  uint32_t pb[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float p0 = ex2_approx(x[a][2 * k] - w.m[0]), p1 = ex2_approx(x[a][2 * k + 1] - w.m[1]);
      w.l[0] += p0;
      w.l[1] += p1;
      pb[a][k] = transpose8x8(pack_f16x2(p0, p1));  // -> head lane / 4, keys 2t, 2t + 1
    }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    // V's factors of keys 2t, 2t + 1 and 2t + 8, 2t + 9 of this 16-key step
    const uint4 ua = ld_shared_v4(fact + 512 + 16 * (8 * a + t)), ub = ld_shared_v4(fact + 512 + 16 * (8 * a + t + 4));
    const uint32_t fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w};
    uint32_t r[8];
    ldm4t(a0 + kCodes + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(r));
    ldm4t(a1 + kCodes + a * 16 * kMxRowBytes, *reinterpret_cast<uint32_t(*)[4]>(r + 4));
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t q0 = hmul2(pb[a][0], fa[b]), q1 = hmul2(pb[a][1], fb[b]);
      uint32_t he[4], ho[4];
      value_pairs(r[2 * b], r[2 * b + 1], he, ho);
      mma16816(w.o[2 * b], {he[0], ho[0], he[2], ho[2]}, q0, q1);
      mma16816(w.o[2 * b + 1], {he[1], ho[1], he[3], ho[3]}, q0, q1);
    }
  }
  if (low) {
    float o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = w.o[i >> 2][i & 3];
    low_values(o, w.ref, make_uint4(pb[0][0], pb[0][1], pb[1][0], pb[1][1]), st, fact, a0, a1);
#pragma unroll
    for (int i = 0; i < 32; ++i) w.o[i >> 2][i & 3] = o[i];
  }
}

// ------------------------------------------------------------------------------- a unit's end
// The warps' partials of unit u (in units of 2^(M + Rmax - 2)) joined by nw warps, this one the w-th: a warp per head,
// lane = channels [4 c, 4 c + 4). whole: the unit is this CTA's alone; else it is a part, and the part that comes last
// merges them all. The nw warps come here together.
__device__ __forceinline__ void join(const MxDecodeParams& p, uint8_t* smem, uint32_t u, uint32_t seg, bool whole, int w, int nw) {
  const int c = threadIdx.x & 31, l = u / kHkv, g = u % kHkv;
  const float2* ml = reinterpret_cast<const float2*>(smem + SM_ML);
  const int* rf = reinterpret_cast<const int*>(smem + SM_R);
  __nv_bfloat16* out = p.layer[l].out + static_cast<size_t>(g) * kRepText * kD + 4 * c;
  // slot 2 c + 1 if this CTA came to the unit from an earlier one, else 2 c
  const size_t ps = static_cast<size_t>(blockIdx.x) * 2 + (seg == 0 ? 0 : 1);
#pragma unroll 1
  for (int h = w; h < kRepText; h += nw) {
    float M = -INFINITY, Lsum = 0.f;
    int R = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      M = fmaxf(M, ml[k * kRepText + h].x);
      R = max(R, rf[k]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 v = ml[k * kRepText + h];
      const float a = ex2_approx(v.x - M);  // 0 for a warp without keys
      Lsum = fmaf(v.y, a, Lsum);
      const float s = ex2_approx(v.x - M + static_cast<float>(rf[k] - R));
      const float4 o = *reinterpret_cast<const float4*>(smem + SM_PART + ((k * kRepText + h) * kPartRow + 4 * c) * 4);
      acc.x = fmaf(s, o.x, acc.x);
      acc.y = fmaf(s, o.y, acc.y);
      acc.z = fmaf(s, o.z, acc.z);
      acc.w = fmaf(s, o.w, acc.w);
    }
    // 2^(R - 127 - 2) / L, in two steps: the power alone may leave fp32's range
    const float inv = 1.0f / Lsum, two_r = mx_scale(R), down = 1.0f / (1 << (kRefField - 15));
    acc.x = acc.x * inv * down * two_r;
    acc.y = acc.y * inv * down * two_r;
    acc.z = acc.z * inv * down * two_r;
    acc.w = acc.w * inv * down * two_r;
    if (whole) {
      *reinterpret_cast<uint2*>(out + h * kD) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    } else {
      *reinterpret_cast<float4*>(p.part_o + (ps * kRepText + h) * kD + 4 * c) = acc;
      if (c == 0) p.part_lse[ps * kRepText + h] = M + log2f(Lsum);
    }
  }
  if (whole) return;
  auto together = [&] {
    if (nw == kPrep / 32) bar_sync(kBarPrep, kPrep);
    else bar_sync(kBarLast, 2 * kPrep);
  };
  const uint32_t u0 = u * p.T, c0 = cta_of(p, u0), c1 = p.T == 1 ? c0 : cta_of(p, u0 + p.T - 1);
  volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(smem + SM_FLAG);
  together();
  if (w == 0 && c == 0) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p.unit_cnt + u) : "memory");
    *flag = old == c1 - c0 ? 1u : 0u;
  }
  together();
  if (*flag == 0u) return;
  // the last part: merges them all, in their order
  const uint32_t np = c1 - c0 + 1;
  const size_t first = static_cast<size_t>(c0) * 2 + (cta_start(p, c0) >= u0 ? 0 : 1);
  auto slot = [&](uint32_t k) -> size_t { return k == 0 ? first : static_cast<size_t>(c0 + k) * 2; };
#pragma unroll 1
  for (int h = w; h < kRepText; h += nw) {
    // lane k: part k's weight (np <= 32: kMxMaxParts); the first parts' loads go out together with the weights' (1
    // layer at pos 4700, 13 parts: 9.2 -> 8.2 us)
    constexpr uint32_t kAhead = 16;
    const float lse = c < np ? __ldcg(p.part_lse + slot(c) * kRepText + h) : -INFINITY;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + h * kD + 4 * c);
    float4 ahead[kAhead];
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k) ahead[k] = k < np ? __ldcg(src + slot(k) * (kRepText * kD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float wt = ex2_approx(lse - warp_max(lse));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    float ws = 0.f;
    auto add = [&](uint32_t k, const float4& o) {
      const float wk = __shfl_sync(0xffffffffu, wt, k);
      ws += wk;
      s.x = fmaf(wk, o.x, s.x);
      s.y = fmaf(wk, o.y, s.y);
      s.z = fmaf(wk, o.z, s.z);
      s.w = fmaf(wk, o.w, s.w);
    };
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k)
      if (k < np) add(k, ahead[k]);
#pragma unroll 4
    for (uint32_t k = kAhead; k < np; ++k) add(k, __ldcg(src + slot(k) * (kRepText * kD / 4)));
    const float iw = 1.0f / ws;
    *reinterpret_cast<uint2*>(out + h * kD) = make_uint2(pack_bf16x2(s.x * iw, s.y * iw), pack_bf16x2(s.z * iw, s.w * iw));
  }
  if (w == 0 && c == 0) p.unit_cnt[u] = 0u;  // every part has arrived: ready for the next call
}

}  // namespace mxd

__global__ void __launch_bounds__(mxd::kThreads, 1) mxfp4_decode_kernel(const __grid_constant__ MxDecodeParams p) {
  using namespace mxd;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t start = cta_start(p, blockIdx.x), end = cta_start(p, blockIdx.x + 1);
  auto bar = [&](uint32_t b) { return sbase + SM_BAR + 8 * b; };
  if (tid == 0) {
    mbar_init(bar(B_QRDY), kPrep / 32);
    mbar_init(bar(B_QRDY + 1), kPrep / 32);
    mbar_init(bar(B_PART), kWarps);
    mbar_init(bar(B_READ), kPrep / 32);
    fence_mbar_init();
  }
  pdl_wait_primary();
  auto wait = [&](uint32_t b, uint32_t parity) -> bool { return counted_wait(bar(b), parity); };
  auto arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  // The CTA's segments: what its range holds of unit u1 + seg's chunks [u0, u0 + T).
  const uint32_t u1 = start / p.T;
  int seg = 0;
  bool ok = true;
  if (warp < kWarps) {
    // a warp's chunks are start + warp + kWarps i; chunk i sits in slot i % kStages of its ring
    const uint32_t ring = sbase + SM_RING + warp * kStages * kStageBytes, fact = sbase + SM_FACT + warp * kFactorBytes;
    const uint32_t loff = 64 * (lane >> 2) + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    uint32_t f = start + warp, fl = f, slot = 0, lslot = 0;  // next chunk to use and to load, and their slots' offsets
    Cursor cur;
    auto load = [&] {
      if (fl < end) {
        load_chunk(p, cur, ring + lslot, loff, lane);
        fl += kWarps;
        if (fl < end) cursor_next(p, cur, lane);
      }
      cp_commit();
      lslot = lslot + kStageBytes == kStages * kStageBytes ? 0 : lslot + kStageBytes;
    };
    cur.u = f / p.T;
    cur.j = f - cur.u * p.T;
    if (f < end) cursor_unit(p, cur, lane);
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s) load();
    __syncthreads();  // the first unit's q is ready, and the barriers are
#pragma unroll 1
    for (;; ++seg) {
      const uint32_t u0 = (u1 + seg) * p.T, f1 = min(end, u0 + p.T);
      const int buf = seg & 1;
      if (seg > 0) ok = wait(B_QRDY + buf, ((seg - 1) >> 1) & 1);
      if (!ok) break;
      uint32_t q[4][4];
      float qf[2];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint4 v = ld_shared_v4(sbase + SM_Q + ((buf * kRepText + (lane >> 2)) * kD + 32 * b + 8 * (lane & 3)) * 2);
        q[b][0] = v.x; q[b][1] = v.y; q[b][2] = v.z; q[b][3] = v.w;
      }
      const float2 fv = reinterpret_cast<const float2*>(smem + SM_QF)[(buf * kRepText >> 1) + (lane & 3)];
      qf[0] = fv.x;
      qf[1] = fv.y;
      Warp w;
      w.m[0] = w.m[1] = -INFINITY;
      w.l[0] = w.l[1] = 0.f;
      w.ref = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) w.o[i][k] = 0.f;
#pragma unroll 1
      for (; f < f1; f += kWarps) {
        const uint32_t st = ring + slot;
        slot = slot + kStageBytes == kStages * kStageBytes ? 0 : slot + kStageBytes;
        cp_wait<kStages - 2>();
        __syncwarp();  // the chunk has landed for every lane, and every lane has left the slot that is refilled
        load();
        const int rr = p.pos - static_cast<int>(f - u0) * kKeys;  // the new row's place in this chunk
        if (rr < kKeys) {
          const uint8_t* nw = smem + SM_NEW + buf * 144;
          if (lane < 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(nw + 16 * lane);
            st_shared_v4(st + (lane >> 2) * kCodes + rr * kMxRowBytes + (((lane & 3) ^ ((rr >> 1) & 3)) << 4), v.x, v.y, v.z, v.w);
          } else if (lane < 10) {
            *reinterpret_cast<uint32_t*>(smem + (st - sbase) + 2 * kCodes + (lane - 8) * kScales + 4 * rr) =
                *reinterpret_cast<const uint32_t*>(nw + 128 + 4 * (lane - 8));
          }
          __syncwarp();
        }
        chunk(w, q, qf, st, fact, rr + 1, lane);
      }
      // this warp's partial: O in units of 2^(m + R - 2), m, l, R
#pragma unroll
      for (int m = 4; m <= 16; m <<= 1) {
        w.l[0] += __shfl_xor_sync(0xffffffffu, w.l[0], m);
        w.l[1] += __shfl_xor_sync(0xffffffffu, w.l[1], m);
      }
      if (seg > 0) ok = wait(B_READ, (seg - 1) & 1);  // the segment before's partials are read
      if (!ok) break;
      float* part = reinterpret_cast<float*>(smem + SM_PART) + warp * kRepText * kPartRow;
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float4*>(part + (2 * t + h) * kPartRow + 32 * b + 4 * g) =
              make_float4(w.o[2 * b][h], w.o[2 * b][2 + h], w.o[2 * b + 1][h], w.o[2 * b + 1][2 + h]);
      if (g < 2) {
        float2* ml = reinterpret_cast<float2*>(smem + SM_ML) + warp * kRepText;
        ml[2 * t + g] = g ? make_float2(w.m[1], w.l[1]) : make_float2(w.m[0], w.l[0]);
      }
      if (lane == 0) reinterpret_cast<int*>(smem + SM_R)[warp] = w.ref;
      if (f1 == end) break;
      arrive(B_PART);
    }
    cp_wait<0>();
    ok = bar_sync_and(kBarEnd, kThreads, ok);
    if (!ok && tid == 0) atomicOr(p.status, kErrDecodeWait);
    if (!ok || warp >= kPrep / 32) return;
  }
  // The preparing warps: unit 0, unit 1, then, segment by segment, the end of its unit and the unit after the next. At
  // the last segment four compute warps join half of the heads (from here on, too: one copy of the code).
  const bool prep = warp >= kWarps;
#pragma unroll 1
  for (int s = prep ? -2 : seg;; ++s) {
    const uint32_t us = u1 + s, un = us + 2;
    if (s >= 0) {
      const uint32_t u0 = us * p.T, f1 = min(end, u0 + p.T);
      const bool fin = f1 == end;
      if (prep) {
        if (fin) pdl_launch_dependents();
        else ok = bar_sync_and(kBarPrep, kPrep, wait(B_PART, s & 1));
        if (fin || !ok) ok = bar_sync_and(kBarEnd, kThreads, ok);  // (the compute warps come there in any case)
        if (!ok) break;
      }
      join(p, smem, us, s, start <= u0 && f1 == u0 + p.T, prep ? warp - kWarps : kPrep / 32 + warp, fin ? kPrep / 16 : kPrep / 32);
      if (fin) break;
      arrive(B_READ);
    }
    if (un * p.T < end) {
      prepare(p, smem, un, end >= (un + 1) * p.T, s & 1, tid - kCompute);
      if (s > -2) arrive(B_QRDY + (s & 1));
    }
    if (s == -2) __syncthreads();
  }
}

cudaError_t mxfp4_decode_set_attributes() {
  return cudaFuncSetAttribute(mxfp4_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(mxd::kSmemBytes));
}

cudaError_t launch_mxfp4_decode(const MxDecodeParams& p, cudaLaunchConfig_t cfg) {
  cfg.blockDim = dim3(mxd::kThreads);
  cfg.dynamicSmemBytes = mxd::kSmemBytes;
  return cudaLaunchKernelEx(&cfg, mxfp4_decode_kernel, p);
}

}  // namespace ea
