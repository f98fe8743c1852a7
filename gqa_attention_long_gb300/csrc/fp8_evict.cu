// fp8_evict.cu — eviction from an 8-bit cache by accumulated attention weight.
//
// Of a head's n_rows rows the first n_first and the last n_recent stay, and of the others those of the largest
// weights, n_keep rows in all; equal weights go to the lowest row. The kept rows' codes (of K and of V) and weights move up to rows
// [0, n_keep) in their order, in place or into another cache. Rows of several blocks meet in one: its scale becomes the
// largest of theirs, and a code of a row with a smaller one, s', is rounded again, code (s' / s).
//
// Two kernels. The selector takes a head's weights with one CTA, or, from kSlice rows on, a cluster of up to eight that share them: it
// finds the bits of the last weight that stays, eleven at a time from the top (a histogram of what shares the bits found so far, summed over the
// cluster's shared memory), then numbers the rows that stay. The mover takes one destination block of a head at a time, of K and V:
// 128 rows are read, all of them, before one is written. In place, a block may be written once the rows that were in it have been read: those
// that stay go to at most two destination blocks, which the selector's counts name, with lower numbers or the same; work is
// handed out in order, so whoever waits waits for work that is already under way. (Bytes: the weights, and a kept row's 256 twice.)
//
// 64 layers from 4700 rows to 4096: 182 us, of which the mover's 165 are the copy's rate, and the selector's 17 issue slots and barriers. 2 layers
// from 131001 to 32769: 69.3 us, 26 of them the selector's on 64 SMs. 1 layer from 4700 to 4096 9.7 us: latencies. In place, with the
// ticket and the waits, 64 layers take 12 % longer, the 2 long ones 11 %.
#include "cluster_exit.cuh"
#include "fp8.cuh"

namespace ea {
namespace ev {

constexpr int kSelWarps = 32;       // at most
constexpr int kBins = 2048;
constexpr int kSlice = 8192;        // rows of one CTA of a cluster, while so many suffice
constexpr int kCached = 32768;      // rows of a slice whose bits are kept in shared memory (else they are read again)
// A cluster's CTAs, at most, while their slices stay in shared memory: twice as many read as much of one another's histograms, and wait
// longer for as many free SMs beside one another (2 layers of 131001 rows: 69 us in fours, 84 in eights).
constexpr int kCluster = 4;
constexpr int kLoads = 2;           // loads of four weights that a thread has in flight
constexpr int kMoveThreads = 256;
constexpr int kPieces = kScaleBlock * kD / 16 / kMoveThreads;  // 16-byte pieces of a block that a thread moves

// Order-preserving bits of a weight: NaN above infinity, the zeros equal. No weight has kAlways or 0.
constexpr uint32_t kAlways = 0xFFFFFFFFu;  // a row that stays whatever its weight is (0: there is no such row)
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f), key = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
  return w != w ? kAlways - 1u : key;
}
// One more in a counter in shared memory, if v <= most (with a branch: 64 layers of 4700 rows 184.7 us, not 182.1).
__device__ __forceinline__ void count_up_to(uint32_t v, uint32_t most, uint32_t counter) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ls.u32 p, %0, %1;\n\t@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(v), "r"(most), "r"(counter) : "memory");
}
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

struct Sel {  // a CTA's shared memory; the slice's bits follow
  alignas(16) uint32_t hist[3][kBins];
  uint32_t warp[kSelWarps][2];  // rows above the threshold and at it, by warp
  uint32_t total[2];            // and of the slice
  uint32_t scan[kSelWarps];
  uint32_t found[2];
};

}  // namespace ev

// 512 threads, or 1024 for the slices of a cluster, which are longer: a warp has at most eight of a cached slice's blocks, whose marks it
// holds in 64 bits.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 2048 / kSelThreads) fp8_evict_select_kernel(const __grid_constant__ F8EvictParams p) {
  using namespace ev;
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ __align__(16) uint8_t ev_smem[];
  Sel& sm = *reinterpret_cast<Sel*>(ev_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + sizeof(Sel));
  const int cs = p.cluster, u = blockIdx.x / cs, rank = blockIdx.x % cs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const F8EvictLayer& L = p.layer[u / kHkv];
  const float* w = L.w + static_cast<size_t>(u % kHkv) * p.Smax;
  int* kept = L.kept + static_cast<size_t>(u % kHkv) * p.n_keep;
  uint32_t* before = p.before + static_cast<size_t>(u) * (p.blocks + 1);
  const int lo = p.n_first, hi = p.n_rows - p.n_recent;  // rows that are chosen among
  const int s0 = min(rank * p.slice, p.n_rows), s1 = min(s0 + p.slice, p.n_rows);  // this CTA's rows
  const int groups = (s1 - s0 + kScaleBlock - 1) / kScaleBlock, pad = groups * kScaleBlock;  // (Smax is in blocks, too)
  const bool cached = p.slice <= kCached;
  // bits of the four rows from row s0 + j on
  auto bits4 = [&](int j) {
    const float4 x = *reinterpret_cast<const float4*>(w + s0 + j);
    uint4 k = make_uint4(key_of(x.x), key_of(x.y), key_of(x.z), key_of(x.w));
    const int i = s0 + j;
    if (__builtin_expect(i < lo || i + 4 > hi, 0)) {
      auto mark = [&](int r, uint32_t v) { return r >= p.n_rows ? 0u : r < lo || r >= hi ? kAlways : v; };
      k = make_uint4(mark(i, k.x), mark(i + 1, k.y), mark(i + 2, k.z), mark(i + 3, k.w));
    }
    return k;
  };
  uint32_t need = p.n_keep, bits = 0u;
  for (int i = tid; i < 3 * kBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();
  if (rank == 0) {
    for (int i = tid; i < p.blocks; i += kSelThreads) p.loaded[static_cast<size_t>(u) * p.blocks + i] = 0u;
    if (u == 0 && tid == 0) *p.ticket = 0u;
  }
  // Of the least weight that stays: 11, then 11, then 10 bits. `need` rows stay among those that share the bits known so far.
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t most = pass == 0 ? 0xFFFFFFFFu : pass == 1 ? (1u << 21) - 1u : (1u << 10) - 1u;
    const uint32_t* hist = sm.hist[pass];
    const uint32_t bins = smem_u32(hist);
    const bool load = pass == 0 || !cached;
#pragma unroll 1
    for (int j0 = 4 * tid; j0 < pad; j0 += 4 * kLoads * kSelThreads) {
      uint4 k[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        const int j = j0 + 4 * kSelThreads * q;
        if (j < pad) k[q] = load ? bits4(j) : *reinterpret_cast<const uint4*>(keys + j);
      }
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        const int j = j0 + 4 * kSelThreads * q;
        if (j >= pad) break;
        if (pass == 0 && cached) *reinterpret_cast<uint4*>(keys + j) = k[q];
        const uint32_t v[4] = {k[q].x - bits, k[q].y - bits, k[q].z - bits, k[q].w - bits};
#pragma unroll
        for (int e = 0; e < 4; ++e) count_up_to(v[e], most, bins + 4 * (v[e] >> shift));
      }
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();
    // thread t: bins kBins - 4 - 4 t .. + 3, the cluster's; then how many rows lie above them
    const int b0 = kBins - 4 - 4 * tid;
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t at = smem_u32(hist + b0);
    if (tid >= kBins / 4) {
    } else if (cs == 1) {
      c = *reinterpret_cast<const uint4*>(hist + b0);
    } else {
#pragma unroll 1
      for (int r = 0; r < cs; r += 4) {  // four CTAs' loads in flight, the next CTA's first: not all of one CTA at a time
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int from = rank + r + q;
          v[q] = r + q < cs ? ld_cluster_v4(mapa_shared(at, from < cs ? from : from - cs)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          c.x += v[q].x;
          c.y += v[q].y;
          c.z += v[q].z;
          c.w += v[q].w;
        }
      }
    }
    const uint32_t mine = (c.x + c.y) + (c.z + c.w);
    uint32_t sum = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += v;
    }
    if (lane == 31) sm.scan[warp] = sum;
    __syncthreads();
    const uint32_t above0 = __reduce_add_sync(0xffffffffu, lane < min(warp, kBins / 128) ? sm.scan[lane] : 0u);
    uint32_t above = above0 + (sum - mine);
    if (above < need && need <= above + mine) {  // (one thread)
      uint32_t d = b0 + 3;
      if (above + c.w < need) { above += c.w; --d;
        if (above + c.z < need) { above += c.z; --d;
          if (above + c.y < need) { above += c.y; --d; } } }
      sm.found[0] = d;
      sm.found[1] = above;
    }
    __syncthreads();
    bits |= sm.found[0] << shift;
    need -= sm.found[1];
  }
  // Rows above the threshold and at it, by warp: a warp has 128-row blocks in a row, a lane four rows of each
  const int per = (groups + kSelWarps - 1) / kSelWarps;
  const int g0 = min(warp * per, groups), g1 = min(g0 + per, groups);
  // bit e: whether row s0 + 128 grp + 4 lane + e is above; bit 4 + e: at
  auto look = [&](int grp) {
    const int j = kScaleBlock * grp + 4 * lane;
    const uint4 k = cached ? *reinterpret_cast<const uint4*>(keys + j) : bits4(j);
    return (k.x > bits ? 1u : 0u) | (k.y > bits ? 2u : 0u) | (k.z > bits ? 4u : 0u) | (k.w > bits ? 8u : 0u) |
           (k.x == bits ? 16u : 0u) | (k.y == bits ? 32u : 0u) | (k.z == bits ? 64u : 0u) | (k.w == bits ? 128u : 0u);
  };
  static_assert(kCached / kScaleBlock / 32 <= 8 && kSlice / kScaleBlock / 16 <= 8, "eight blocks' bits in 64");
  uint64_t seen = 0;  // of a cached slice
  uint32_t a = 0, e = 0;
  for (int grp = g0; grp < g1; ++grp) {
    const uint32_t m = look(grp);
    if (cached) seen |= static_cast<uint64_t>(m) << (8 * (grp - g0));
    a += __popc(m & 15u);
    e += __popc(m >> 4);
  }
  a = __reduce_add_sync(0xffffffffu, a);
  e = __reduce_add_sync(0xffffffffu, e);
  if (lane == 0) {
    sm.warp[warp][0] = a;
    sm.warp[warp][1] = e;
  }
  __syncthreads();
  uint32_t above = 0, equal = 0;  // among the rows before the warp's
#pragma unroll 1
  for (int k = 0; k < warp; ++k) {
    above += sm.warp[k][0];
    equal += sm.warp[k][1];
  }
  if (cs > 1) {
    if (warp == kSelWarps - 1 && lane == 0) {
      sm.total[0] = above + a;
      sm.total[1] = equal + e;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const float2 t = ld_shared_cluster_v2(mapa_shared(smem_u32(sm.total), r));
      above += __float_as_uint(t.x);
      equal += __float_as_uint(t.y);
    }
    if (lane == 0) *const_cast<volatile uint32_t*>(&sm.scan[warp]) = above + equal;  // (a store that needs every load's value)
    cluster_sync_exit();  // no CTA leaves while another reads its shared memory
  }
  for (int grp = g0; grp < g1; ++grp) {
    const uint32_t m = cached ? static_cast<uint32_t>(seen >> (8 * (grp - g0))) & 255u : look(grp), c = __popc(m & 15u) | __popc(m >> 4) << 16;
    uint32_t sum = c;  // of the lanes up to this one: rows above, and (from bit 16) at the threshold
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    uint32_t a1 = above + ((sum - c) & 0xFFFFu), e1 = equal + ((sum - c) >> 16);
    const int i = s0 + kScaleBlock * grp + 4 * lane;
    if (lane == 0) before[i / kScaleBlock] = a1 + min(e1, need);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool gt = (m >> e) & 1u, eq = (m >> (4 + e)) & 1u;
      if (gt || (eq && e1 < need)) kept[a1 + min(e1, need)] = i + e;
      a1 += gt;
      e1 += eq;
    }
    sum = __shfl_sync(0xffffffffu, sum, 31);
    above += sum & 0xFFFFu;
    equal += sum >> 16;
  }
  if (rank == cs - 1)
    for (int b = (p.n_rows - 1) / kScaleBlock + 1 + tid; b <= p.blocks; b += kSelThreads) before[b] = p.n_keep;
}

__global__ void __launch_bounds__(ev::kMoveThreads, 4) fp8_evict_move_kernel(const __grid_constant__ F8EvictParams p) {
  using namespace ev;
  __shared__ float red[2][kMoveThreads / 32];
  __shared__ float factor[2][kScaleBlock];
  __shared__ uint32_t next;
  __shared__ volatile uint32_t abort_flag;
  const int tid = threadIdx.x;
  const uint32_t chunks = (p.n_keep - 1) / kScaleBlock + 1, units = kHkv * p.n_layers;
  if (tid == 0) abort_flag = 0u;
  pdl_wait_primary();
  pdl_launch_dependents();
  for (uint32_t t = blockIdx.x;; t += gridDim.x) {
    if (p.ordered) {  // some layer's rows move within its cache
      __syncthreads();
      if (tid == 0) next = atomicAdd(p.ticket, 1u);
      __syncthreads();
      t = next;
    }
    if (t >= chunks * units) return;
    const int c = t / units, u = t % units, g = u % kHkv;
    const F8EvictLayer& L = p.layer[u / kHkv];
    const size_t head = static_cast<size_t>(g) * p.Smax * kD;
    const int* kept = L.kept + static_cast<size_t>(g) * p.n_keep + c * kScaleBlock;
    const int n = min(kScaleBlock, p.n_keep - c * kScaleBlock);
    // a thread's pieces of rows tid / 8 + 32 i, of K and of V, and one row's scales and weight
    int r[kPieces], mine = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (tid / 8 + 32 * i < n) r[i] = kept[tid / 8 + 32 * i];
    if (tid < n) mine = kept[tid];
    uint4 x[2][kPieces];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (tid / 8 + 32 * i < n)
          x[kv][i] = *reinterpret_cast<const uint4*>((kv ? L.vc : L.kc) + head + static_cast<size_t>(r[i]) * kD + 16 * (tid & 7));
    float s[2] = {0.f, 0.f}, top[2], wgt = 0.f;
    if (tid < n) {
      const int b = g * (p.blocks + 1) + mine / kScaleBlock;
      s[0] = L.ks[b];
      s[1] = L.vs[b];
      wgt = L.w[static_cast<size_t>(g) * p.Smax + mine];
    }
    __syncthreads();  // (the block before is done with red and factor)
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      top[kv] = s[kv];
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) top[kv] = fmaxf(top[kv], __shfl_xor_sync(0xffffffffu, top[kv], m));
      if ((tid & 31) == 0) red[kv][tid >> 5] = top[kv];
    }
    __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      top[kv] = fmaxf(fmaxf(red[kv][0], red[kv][1]), fmaxf(red[kv][2], red[kv][3]));  // (n <= 128: four warps have rows)
      if (tid < n) factor[kv][tid] = s[kv] == top[kv] ? 1.0f : __fdiv_rn(s[kv], top[kv]);
    }
    if (L.kc == L.kd) {
      __syncthreads();  // every thread's loads have returned what they read before any of the block's rows is written
      if (tid == 0) {
        uint32_t* loaded = p.loaded + static_cast<size_t>(u) * p.blocks;
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
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = tid / 8 + 32 * i;
        if (row < n) {
          const float f = factor[kv][row];
          *reinterpret_cast<uint4*>((kv ? L.vd : L.kd) + head + (static_cast<size_t>(c) * kScaleBlock + row) * kD + 16 * (tid & 7)) =
              f == 1.0f ? x[kv][i] : f8_rescale16(x[kv][i], f);
        }
      }
    if (tid < n) L.wd[static_cast<size_t>(g) * p.Smax + c * kScaleBlock + tid] = wgt;
    if (tid == 0) {
      L.ksd[g * (p.blocks + 1) + c] = top[0];
      L.vsd[g * (p.blocks + 1) + c] = top[1];
    }
  }
}

cudaError_t fp8_evict_set_attributes() {
  const int most = static_cast<int>(sizeof(ev::Sel) + ev::kCached * sizeof(uint32_t));
  const cudaError_t e = cudaFuncSetAttribute(fp8_evict_select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(fp8_evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

cudaError_t launch_fp8_evict(F8EvictParams& p, int sm_count, cudaLaunchConfig_t cfg) {
  // slices of whole 128-row blocks
  p.cluster = (p.n_rows + ev::kSlice - 1) / ev::kSlice;
  if (p.cluster > ev::kCluster) p.cluster = p.n_rows <= ev::kCluster * ev::kCached ? ev::kCluster : 2 * ev::kCluster;
  p.slice = ((p.n_rows + p.cluster - 1) / p.cluster + kScaleBlock - 1) / kScaleBlock * kScaleBlock;
  cudaLaunchConfig_t sel = cfg;
  cudaLaunchAttribute attr[2];
  attr[0] = cfg.attrs[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
  sel.attrs = attr;
  sel.numAttrs = p.cluster > 1 ? 2 : 1;
  sel.gridDim = dim3(p.n_layers * kHkv * p.cluster);
  sel.blockDim = dim3(p.cluster > 1 ? 1024 : 512);
  sel.dynamicSmemBytes = sizeof(ev::Sel) + (p.slice <= ev::kCached ? p.slice * sizeof(uint32_t) : 0);
  // So much shared memory that no SM takes more CTAs than its share: started while the kernel before ends, they would crowd onto the SMs that
  // are free first (4 layers of 8000 rows to half, call after call: 21.9 us, and 30.4 without). Clusters of three and four do not fill every SM.
  const int sms = p.cluster > 2 ? sm_count / 8 * 7 : sm_count;
  const size_t share = (sel.gridDim.x + sms - 1) / sms, alone = 227 * 1024 / (share + 1) + 128;
  if (share < 4 && sel.dynamicSmemBytes < alone) sel.dynamicSmemBytes = alone / 128 * 128;
  const cudaError_t e = cudaLaunchKernelEx(&sel, p.cluster > 1 ? fp8_evict_select_kernel<1024> : fp8_evict_select_kernel<512>, p);
  if (e != cudaSuccess) return e;
  const int work = ((p.n_keep - 1) / kScaleBlock + 1) * kHkv * p.n_layers, most = 4 * sm_count;
  cfg.gridDim = dim3(work < most ? work : most);
  cfg.blockDim = dim3(ev::kMoveThreads);
  return cudaLaunchKernelEx(&cfg, fp8_evict_move_kernel, p);
}

}  // namespace ea
