// fp8_evict.cu — eviction from an 8-bit cache by accumulated attention weight.
//
// Of a head's n_rows rows the first n_first and the last n_recent stay, and of the others those of the largest
// weights, n_keep rows in all; equal weights go to the lowest row. The kept rows' codes (of K and of V) and weights move up to rows
// [0, n_keep) in their order, in place or into another cache. Rows of several blocks meet in one: its scale becomes the
// largest of theirs, and a code of a row with a smaller one, s', is rounded again, code (s' / s).
//
// Two kernels. The selector (one CTA per (layer, kv head)) finds the weight of the last row that stays by its bits, from
// the top ones down, and writes the kept rows' numbers. The mover takes one destination block of K or of V of one head at a time:
// 128 rows are read, all of them, before one is written. In place, a block may be written once the rows that were in it have been read: those
// that stay go to at most two destination blocks, which the selector's counts name, with lower numbers or the same; work is
// handed out in order, so whoever waits waits for work that is already under way. (Bytes: the weights, and a kept row's 256 twice.)
#include "fp8.cuh"

namespace ea {
namespace ev {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kPieces = kScaleBlock * kD / 16 / kMoveThreads;  // 16-byte pieces of a block that a thread moves

// Order-preserving bits: NaN above infinity, the zeros equal.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  return w != w ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

}  // namespace ev

__global__ void __launch_bounds__(ev::kSelThreads) fp8_evict_select_kernel(const __grid_constant__ F8EvictParams p) {
  using namespace ev;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sums[2][32];
  __shared__ uint32_t found[2];
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const F8EvictLayer& L = p.layer[u / kHkv];
  const float* w = L.w + static_cast<size_t>(u % kHkv) * p.Smax;
  int* kept = L.kept + static_cast<size_t>(u % kHkv) * p.n_keep;
  uint32_t* before = p.before + static_cast<size_t>(u) * (p.blocks + 1);
  const int lo = p.n_first, hi = p.n_rows - p.n_recent;  // rows that are chosen among
  pdl_wait_primary();
  for (int i = tid; i < 2 * p.blocks; i += kSelThreads) p.loaded[static_cast<size_t>(u) * 2 * p.blocks + i] = 0u;
  if (u == 0 && tid == 0) *p.ticket = 0u;
  // the bits of the least weight that stays: `top` of them are known, `need` rows stay among those that share them
  uint32_t need = p.n_keep - p.n_first - p.n_recent, bits = 0u;
  for (int top = 0; top < 32; top += 8) {
    const int shift = 24 - top;
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = key_of(w[i]);
      if (top == 0 || (k >> (shift + 8)) == (bits >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t n = 0, d = 255;
      for (;; --d) {
        if (n + hist[d] >= need || d == 0) break;
        n += hist[d];
      }
      found[0] = d;
      found[1] = n;
    }
    __syncthreads();
    bits |= found[0] << shift;
    need -= found[1];
    __syncthreads();
  }
  // need > 0 rows of weight `bits` stay, the lowest ones (0 if no row is chosen at all)
  uint32_t above = 0, equal = 0;  // among the rows before
  for (int base = 0; base < p.n_rows; base += kSelThreads) {
    const int i = base + tid;
    bool gt = false, eq = false;
    if (i < p.n_rows) {
      if (i < lo || i >= hi) {
        gt = true;
      } else {
        const uint32_t k = key_of(w[i]);
        gt = k > bits;
        eq = k == bits;
      }
    }
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq), below = (1u << lane) - 1u;
    if (lane == 0) {
      sums[0][warp] = __popc(mg);
      sums[1][warp] = __popc(me);
    }
    __syncthreads();
    uint32_t a = above + __popc(mg & below), e = equal + __popc(me & below);
    for (int k = 0; k < kSelThreads / 32; ++k) {
      if (k < warp) {
        a += sums[0][k];
        e += sums[1][k];
      }
      above += sums[0][k];
      equal += sums[1][k];
    }
    const uint32_t at = a + min(e, need);
    if (i < p.n_rows) {
      if (gt || (eq && e < need)) kept[at] = i;
      if (i % kScaleBlock == 0) before[i / kScaleBlock] = at;
    }
    __syncthreads();
  }
  for (int b = (p.n_rows - 1) / kScaleBlock + 1 + tid; b <= p.blocks; b += kSelThreads) before[b] = p.n_keep;
  pdl_launch_dependents();
}

__global__ void __launch_bounds__(ev::kMoveThreads) fp8_evict_move_kernel(const __grid_constant__ F8EvictParams p) {
  using namespace ev;
  __shared__ float red[kMoveThreads / 32];
  __shared__ float factor[kScaleBlock];
  __shared__ int rows[kScaleBlock];
  __shared__ uint32_t next;
  __shared__ volatile uint32_t abort_flag;
  const int tid = threadIdx.x;
  const uint32_t chunks = (p.n_keep - 1) / kScaleBlock + 1, items = 2 * kHkv * p.n_layers;
  if (tid == 0) abort_flag = 0u;
  pdl_wait_primary();
  pdl_launch_dependents();
  for (;;) {
    __syncthreads();
    if (tid == 0) next = atomicAdd(p.ticket, 1u);
    __syncthreads();
    const uint32_t t = next;
    if (t >= chunks * items) return;
    const int c = t / items, item = t % items, kv = item & 1, u = item >> 1, g = u % kHkv;
    const F8EvictLayer& L = p.layer[u / kHkv];
    const uint8_t* src = (kv ? L.vc : L.kc) + static_cast<size_t>(g) * p.Smax * kD;
    uint8_t* dst = (kv ? L.vd : L.kd) + static_cast<size_t>(g) * p.Smax * kD;
    const float* ss = (kv ? L.vs : L.ks) + g * (p.blocks + 1);
    float* sd = (kv ? L.vsd : L.ksd) + g * (p.blocks + 1);
    uint32_t* loaded = p.loaded + static_cast<size_t>(item) * p.blocks;
    const bool in_place = src == dst;
    const int n = min(kScaleBlock, p.n_keep - c * kScaleBlock);
    // the rows and their scales
    float s = 0.f, wgt = 0.f;
    if (tid < n) {
      const int r = L.kept[static_cast<size_t>(g) * p.n_keep + c * kScaleBlock + tid];
      rows[tid] = r;
      s = ss[r / kScaleBlock];
      if (kv == 0) wgt = L.w[static_cast<size_t>(g) * p.Smax + r];
    }
    float top = s;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kScaleBlock / 32; ++k) top = fmaxf(top, red[k]);
    if (tid < n) factor[tid] = s == top ? 1.0f : __fdiv_rn(s, top);
    uint4 x[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int q = tid + kMoveThreads * i;
      if ((q >> 3) < n) x[i] = *reinterpret_cast<const uint4*>(src + static_cast<size_t>(rows[q >> 3]) * kD + 16 * (q & 7));
    }
    if (in_place) {
      asm volatile("" ::: "memory");
      __syncthreads();  // every thread's loads have returned what they read before any of the block's rows is written
      if (tid == 0) {
        st_release_gpu(loaded + c, 1u);
        // the destination blocks that read this block's rows
        const uint32_t* before = p.before + static_cast<size_t>(u) * (p.blocks + 1);
        const int a = before[c], b = before[c + 1];
        bool ok = true;
        for (int d = a / kScaleBlock; ok && d < c && d * kScaleBlock < b; ++d)
          ok = bounded_flag_wait(loaded + d, &abort_flag, p.status, kErrEvictWait);
      }
    }
    __syncthreads();
    if (abort_flag) return;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int q = tid + kMoveThreads * i;
      if ((q >> 3) < n) {
        const float f = factor[q >> 3];
        *reinterpret_cast<uint4*>(dst + (static_cast<size_t>(c) * kScaleBlock + (q >> 3)) * kD + 16 * (q & 7)) = f == 1.0f ? x[i] : f8_rescale16(x[i], f);
      }
    }
    if (tid < n && kv == 0) L.wd[static_cast<size_t>(g) * p.Smax + c * kScaleBlock + tid] = wgt;
    if (tid == 0) sd[c] = top;
  }
}

cudaError_t launch_fp8_evict(const F8EvictParams& p, int sm_count, cudaLaunchConfig_t cfg) {
  cfg.gridDim = dim3(p.n_layers * kHkv);
  cfg.blockDim = dim3(ev::kSelThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_evict_select_kernel, p);
  if (e != cudaSuccess) return e;
  const int work = ((p.n_keep - 1) / kScaleBlock + 1) * 2 * kHkv * p.n_layers, most = 6 * sm_count;
  cfg.gridDim = dim3(work < most ? work : most);
  cfg.blockDim = dim3(ev::kMoveThreads);
  return cudaLaunchKernelEx(&cfg, fp8_evict_move_kernel, p);
}

}  // namespace ea
