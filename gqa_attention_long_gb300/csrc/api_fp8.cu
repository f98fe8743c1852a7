// api_fp8.cu — host side of the 8-bit cache's writer, reader, decode step and eviction: argument checks, launch planning and
// the launches per chunk of 64 layers. See include/expert_attn.h for the contract.
#include <array>
#include <cstring>
#include <mutex>

#include "expert_attn.h"
#include "host.cuh"
#include "internal.cuh"

namespace ea {
cudaError_t launch_fp8_rows(const F8RowsParams& p, int n_layers, int dtype, bool write, cudaLaunchConfig_t cfg);
cudaError_t fp8_decode_set_attributes();
template <int CAP>
cudaError_t launch_fp8_decode(const F8DecodeParams<CAP>& p, cudaLaunchConfig_t cfg);
cudaError_t fp8_decode_small_set_attributes();
template <int CAP>
cudaError_t launch_fp8_decode_small(const F8SmallParams<CAP>& p, cudaLaunchConfig_t cfg);
cudaError_t launch_fp8_weights(const F8WeightsParams& p, cudaLaunchConfig_t cfg);
cudaError_t fp8_evict_set_attributes();
cudaError_t launch_fp8_evict(F8EvictParams& p, int sm_count, cudaLaunchConfig_t cfg);
}  // namespace ea

namespace {

using namespace ea;

bool smax_ok(int Smax) { return Smax >= kScaleBlock && Smax % kScaleBlock == 0 && Smax <= (1 << 22); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Pointers that have to be there, 16-byte aligned codes and rows and 4-byte aligned numbers.
template <int N, int M>
int check_pointers(const void* const (&wide)[N], const void* const (&narrow)[M]) {
  for (const void* p : wide)
    if (p == nullptr) return EA_ERR_INVALID_ARG;
  for (const void* p : narrow)
    if (p == nullptr) return EA_ERR_INVALID_ARG;
  for (const void* p : wide)
    if (!aligned16(p)) return EA_ERR_MISALIGNED;
  for (const void* p : narrow)
    if (!aligned4(p)) return EA_ERR_MISALIGNED;
  return EA_OK;
}

int run_rows(const ea_fp8_rows* a, int n_layers, int row0, int n_rows, int Smax, int dtype, int64_t head_stride,
             int64_t row_stride, bool write, ea_stream_t stream) {
  if (a == nullptr || n_layers < 1) return EA_ERR_INVALID_ARG;
  if (!smax_ok(Smax) || row0 < 0 || n_rows < 0 || n_rows > Smax - row0) return EA_ERR_INVALID_ARG;
  if (dtype != EA_ROWS_BF16 && dtype != EA_ROWS_FP16 && dtype != EA_ROWS_FP32) return EA_ERR_INVALID_ARG;
  constexpr int64_t kMaxStride = 1LL << 40;
  if (head_stride < 0 || row_stride < 0 || head_stride > kMaxStride || row_stride > kMaxStride) return EA_ERR_INVALID_ARG;
  const int64_t esz = dtype == EA_ROWS_FP32 ? 4 : 2;
  if (head_stride * esz % 16 != 0 || (n_rows > 1 && row_stride * esz % 16 != 0)) return EA_ERR_MISALIGNED;
  // rows that are written must not overlap
  if (!write && (head_stride < kD || (n_rows > 1 && (row_stride < kD || (head_stride < (n_rows - 1) * row_stride + kD &&
                                                                        row_stride < (kHkv - 1) * head_stride + kD)))))
    return EA_ERR_INVALID_ARG;
  for (int l = 0; l < n_layers; ++l) {
    const ea_fp8_rows& x = a[l];
    const int rc = check_pointers<4, 2>({x.k, x.v, x.k_cache, x.v_cache}, {x.k_scale, x.v_scale});
    if (rc != EA_OK) return rc;
  }
  if (!(write ? mx_distinct<4>(a, n_layers, [](const ea_fp8_rows& x) {
          return std::array<const void*, 4>{x.k_cache, x.v_cache, x.k_scale, x.v_scale};
        })
              : mx_distinct<2>(a, n_layers, [](const ea_fp8_rows& x) { return std::array<const void*, 2>{x.k, x.v}; })))
    return EA_ERR_INVALID_ARG;
  int dev;
  DeviceInfo di;
  if (!device_info(&dev, &di)) return EA_ERR_UNSUPPORTED;
  if (n_rows == 0) return EA_OK;
  F8RowsParams p;
  std::memset(&p, 0, sizeof(p));
  p.head_stride = head_stride;
  p.row_stride = n_rows > 1 ? row_stride : 0;
  p.row0 = row0;
  p.n_rows = n_rows;
  p.Smax = Smax;
  cudaLaunchAttribute attr[1];
  for (int l0 = 0; l0 < n_layers; l0 += kMaxLayersPerLaunch) {
    const int n = n_layers - l0 < kMaxLayersPerLaunch ? n_layers - l0 : kMaxLayersPerLaunch;
    for (int l = 0; l < n; ++l) {
      const ea_fp8_rows& x = a[l0 + l];
      p.layer[l] = {x.k, x.v, static_cast<uint8_t*>(x.k_cache), static_cast<uint8_t*>(x.v_cache), x.k_scale, x.v_scale};
    }
    if (launch_fp8_rows(p, n, dtype, write, launch_config(static_cast<cudaStream_t>(stream), attr, true)) != cudaSuccess) {
      cudaGetLastError();
      return EA_ERR_CUDA;
    }
  }
  return EA_OK;
}

bool decode_attrs_ready(int dev) {
  static OncePerDevice once;
  return once(dev, [] {
    const bool ok = fp8_decode_set_attributes() == cudaSuccess && fp8_decode_small_set_attributes() == cudaSuccess;
    cudaGetLastError();
    return ok;
  });
}

bool evict_attrs_ready(int dev) {
  static OncePerDevice once;
  return once(dev, [] {
    const bool ok = fp8_evict_set_attributes() == cudaSuccess;
    cudaGetLastError();
    return ok;
  });
}

int validate_decode(const ea_decode_fp8_args* a, int n_layers, int pos, int Smax, long long p0, const void* ws) {
  if (a == nullptr || n_layers < 1 || ws == nullptr) return EA_ERR_INVALID_ARG;
  if (!smax_ok(Smax) || pos < 0 || pos >= Smax) return EA_ERR_INVALID_ARG;
  if (p0 <= -(1LL << 24) || p0 >= (1LL << 24)) return EA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return EA_ERR_MISALIGNED;
  for (int l = 0; l < n_layers; ++l) {
    const ea_decode_fp8_args& x = a[l];
    const int rc = check_pointers<8, 2>({x.q_raw, x.k_raw, x.v_raw, x.q_gamma, x.k_gamma, x.k_cache, x.v_cache, x.out},
                                        {x.k_scale, x.v_scale});
    if (rc != EA_OK) return rc;
    if (x.weight_out == nullptr && x.weight_in != nullptr) return EA_ERR_INVALID_ARG;
    if (!aligned16(x.k_new) || !aligned16(x.v_new) || !aligned16(x.weight_in) || !aligned16(x.weight_out))  // (null is aligned)
      return EA_ERR_MISALIGNED;
  }
  // what is written stands once; sums that are read from elsewhere are not written
  return mx_distinct<9>(a, n_layers, [](const ea_decode_fp8_args& x) {
           return std::array<const void*, 9>{x.k_cache, x.v_cache, x.k_scale, x.v_scale, x.out, x.k_new, x.v_new, x.weight_out,
                                             x.weight_in == x.weight_out ? nullptr : x.weight_in};
         })
             ? EA_OK
             : EA_ERR_INVALID_ARG;
}

bool any_weights(const ea_decode_fp8_args* a, int n) {
  for (int l = 0; l < n; ++l)
    if (a[l].weight_out != nullptr) return true;
  return false;
}

F8AttnLayer attn_layer(const ea_decode_fp8_args& x) {
  auto bf = [](const void* q) { return static_cast<const __nv_bfloat16*>(q); };
  return {bf(x.q_raw), bf(x.k_raw), bf(x.v_raw), bf(x.q_gamma), bf(x.k_gamma), static_cast<uint8_t*>(x.k_cache),
          static_cast<uint8_t*>(x.v_cache), x.k_scale, x.v_scale, static_cast<__nv_bfloat16*>(x.out),
          static_cast<__nv_bfloat16*>(x.k_new), static_cast<__nv_bfloat16*>(x.v_new), x.weight_in, x.weight_out};
}

// fp8_decode_kernel's CTAs, at most: one to an SM.
int decode_ctas(int sm_count) { return sm_count < kMaxGridCtas ? sm_count : kMaxGridCtas; }

// Whether fp8_decode_kernel forms the weights itself: units of at most kF8KeptTiles tiles, and one and a half of them to a CTA, so
// that most are whole ones. us a call:
//   layers x pos (units to a CTA)   second kernel   without it
//   64 x 4700 (3.4)                 133.6           122.5
//   64 x 2500 (3.4)                  79.8            74.8
//   32 x 4900 (1.7)                  78.6            76.0
//   29 x 4000 (1.5)                  63.3            61.6
//   24 x 4700 (1.3)                  60.0            60.0
//   16 x 4700 (0.8)                  45.3            47.3
bool forms_weights(int n, int pos, int sm_count) {
  return n > kSmallCap && pos / kKeyTile + 1 <= kF8KeptTiles && 2 * n * kHkv >= 3 * decode_ctas(sm_count);
}

// Parameter blocks are large (24 KB at full capacity): kept off the stack, one per capacity, with a mutex of its own.
template <int CAP>
struct DecodeBlock {
  F8DecodeParams<CAP> p;
  std::mutex mu;
};

template <int CAP>
int launch_decode_t(const ea_decode_fp8_args* a, int n, int pos, int Smax, long long p0, bool weights, uint8_t* ws,
                    const F8DecodeWs& wl, int sm_count, cudaStream_t st) {
  static DecodeBlock<CAP> block;
  std::lock_guard<std::mutex> lk(block.mu);
  F8DecodeParams<CAP>& p = block.p;
  for (int l = 0; l < n; ++l) {
    const ea_decode_fp8_args& x = a[l];
    if (!cache_map(x.k_cache, 0, Smax, true, &p.kmap[l]) || !cache_map(x.v_cache, 0, Smax, true, &p.vmap[l])) return EA_ERR_CUDA;
    p.layer[l] = attn_layer(x);
  }
  for (int j = 0; j < kD / 2; ++j) p.rot[j] = MxRotations::split(MxRotations::get().at(p0, j));
  p.part_o = reinterpret_cast<float*>(ws + wl.part_o_off);
  p.part_ml = reinterpret_cast<float*>(ws + wl.part_ml_off);
  p.unit_cnt = reinterpret_cast<uint32_t*>(ws + wl.cnt_off);
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.scores = weights ? reinterpret_cast<float*>(ws + wl.scores_off) : nullptr;
  p.lse = reinterpret_cast<float*>(ws + wl.lse_off);
  p.form = forms_weights(n, pos, sm_count);
  p.T = pos / kKeyTile + 1;
  p.W = static_cast<long long>(n) * kHkv * p.T;
  p.pos = pos;
  p.Smax = Smax;
  p.n_layers = n;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kD)));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = launch_config(st, attr, true);
  const int most = decode_ctas(sm_count);
  cfg.gridDim = dim3(most < p.W ? most : static_cast<int>(p.W));
  if (launch_fp8_decode<CAP>(p, cfg) != cudaSuccess) {
    cudaGetLastError();
    return EA_ERR_CUDA;
  }
  return EA_OK;
}

// Little work (see fp8_decode_small.cu): its kernel's CTAs, of `tiles` key tiles each, come in `waves` of one to an SM, and the start and
// the end of one are about four tiles' time: waves x (kSmallEnds + tiles) <= kSmallWork + waves / 2 (more units take the other
// kernel longer, too). us a call:
//   layers x pos (waves x (4 + tiles))   its kernel   the other one
//    1 x  300 (1 x  6)                    6.8         10.5
//    1 x 4700 (1 x  6)                    9.2         13.6
//   16 x 1000 (1 x 12)                   13.2         18.2
//   16 x 1500 (1 x 16)                   18.0         19.2
//    5 x 4700 (1 x 17)                   20.4         20.1
//   12 x 2000 (1 x 20)                   21.5         19.1
//   32 x  600 (2 x  9)                   21.7         23.4
//   32 x  800 (2 x 11)                   25.2         24.0
//   64 x  100 (4 x  5)                   21.8         22.9
//   64 x  380 (4 x  7)                   33.7         28.3
// Up to kOnePart tiles a unit is one CTA's (4 layers at pos 300, three tiles: 7.6 us whole, 7.0 in two parts). Up to kF8SmallCluster
// parts are a cluster (1 layer at pos 1000: 7.6 us, 7.9 through global memory; in clusters of eight 2 layers at pos 2000 wait for as
// many free SMs beside one another: 14.9 us, and 8.1). Clusters of three and four do not fill every SM: 6 layers at pos 600 in 48
// clusters of three took 13.4 us, and 9.1 in pairs; from seven eighths of the SMs on they are pairs.
constexpr int kSmallEnds = 4, kSmallWork = 18, kOnePart = 2;
static_assert(kSmallWork - kSmallEnds <= kF8SmallTiles, "a CTA's tiles: as many in one wave, fewer in more");

// Whether fp8_decode_small_kernel forms the weights itself: where a unit's CTAs can tell each other its log2-sum-exps. With a second
// kernel and without: 1 layer at pos 1000 9.1 and 8.1 us, 4 layers at pos 4700 19.9 and 17.9, 8 layers at pos 1000 11.8 and 10.3, 32 layers
// at pos 500 21.7 and 19.2.
bool small_forms(int parts) { return parts <= kF8SmallCluster; }

template <int CAP>
int launch_small(const ea_decode_fp8_args* a, int n, int pos, int Smax, long long p0, bool weights, uint8_t* ws, const F8DecodeWs& wl,
                 int parts, cudaStream_t st) {
  F8SmallParams<CAP> p;
  for (int l = 0; l < n; ++l) p.layer[l] = attn_layer(a[l]);
  for (int j = 0; j < kD / 2; ++j) p.rot[j] = MxRotations::split(MxRotations::get().at(p0, j));
  p.part_o = reinterpret_cast<float*>(ws + wl.part_o_off);
  p.part_ml = reinterpret_cast<float*>(ws + wl.part_ml_off);
  p.unit_cnt = reinterpret_cast<uint32_t*>(ws + wl.cnt_off);
  p.scores = weights ? reinterpret_cast<float*>(ws + wl.scores_off) : nullptr;
  p.lse = reinterpret_cast<float*>(ws + wl.lse_off);
  p.T = pos / kKeyTile + 1;
  p.parts = parts;
  p.cluster = parts > 1 && parts <= kF8SmallCluster;
  p.form = weights && small_forms(parts);
  p.pos = pos;
  p.Smax = Smax;
  p.n_layers = n;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kD)));
  cudaLaunchAttribute attr[1];
  if (launch_fp8_decode_small(p, launch_config(st, attr, true)) != cudaSuccess) {
    cudaGetLastError();
    return EA_ERR_CUDA;
  }
  return EA_OK;
}

int launch_weights(const ea_decode_fp8_args* a, int n, int pos, int Smax, uint8_t* ws, const F8DecodeWs& wl, cudaStream_t st) {
  F8WeightsParams p;
  for (int l = 0; l < n; ++l) p.layer[l] = attn_layer(a[l]);
  p.scores = reinterpret_cast<float*>(ws + wl.scores_off);
  p.lse = reinterpret_cast<float*>(ws + wl.lse_off);
  p.T = pos / kKeyTile + 1;
  p.pos = pos;
  p.Smax = Smax;
  p.n_layers = n;
  cudaLaunchAttribute attr[1];
  if (launch_fp8_weights(p, launch_config(st, attr, true)) != cudaSuccess) {
    cudaGetLastError();
    return EA_ERR_CUDA;
  }
  return EA_OK;
}

// The CTAs to a unit for a call of little work, 0 for another. A unit of up to kOnePart tiles is one
// CTA's.
int small_parts(int n, int pos, int sm_count) {
  const int T = pos / kKeyTile + 1, units = n * kHkv;
  int parts = sm_count / units;
  if (parts > (T + 1) / 2) parts = (T + 1) / 2;  // (two tiles keep a CTA's eight warps busy)
  if (parts > kF8SmallParts) parts = kF8SmallParts;
  if (parts > 2 && parts <= kF8SmallCluster && units * parts > sm_count / 8 * 7) parts = 2;
  if (parts < 1 || T <= kOnePart) parts = 1;
  const int waves = (units * parts + sm_count - 1) / sm_count, tiles = (T + parts - 1) / parts;
  return static_cast<long long>(waves) * (kSmallEnds + tiles) <= kSmallWork + waves / 2 ? parts : 0;
}

// Whether [a, a + n) and [b, b + n) share bytes without being the same.
bool partly(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && (x > y ? x - y : y - x) < n;
}

int validate_evict(const ea_evict_fp8_args* a, int n_layers, int n_rows, int n_keep, int n_first, int n_recent, int Smax,
                   const void* ws) {
  if (a == nullptr || n_layers < 1 || ws == nullptr || !smax_ok(Smax)) return EA_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > Smax || n_keep < 0 || n_keep > n_rows || n_first < 0 || n_recent < 0 || n_first > n_keep ||
      n_recent > n_keep - n_first)
    return EA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return EA_ERR_MISALIGNED;
  const size_t codes = static_cast<size_t>(kHkv) * Smax * kD, sums = static_cast<size_t>(kHkv) * Smax * sizeof(float),
               scales = static_cast<size_t>(kHkv) * (Smax / kScaleBlock + 1) * sizeof(float);
  for (int l = 0; l < n_layers; ++l) {
    const ea_evict_fp8_args& x = a[l];
    const int rc = check_pointers<6, 5>({x.k_cache, x.v_cache, x.k_dst, x.v_dst, x.weight, x.weight_dst},
                                        {x.k_scale, x.v_scale, x.k_scale_dst, x.v_scale_dst, x.kept});
    if (rc != EA_OK) return rc;
    const int same = (x.k_cache == x.k_dst) + (x.v_cache == x.v_dst) + (x.k_scale == x.k_scale_dst) + (x.v_scale == x.v_scale_dst) +
                     (x.weight == x.weight_dst);
    if (same != 0 && same != 5) return EA_ERR_INVALID_ARG;  // in place, or into other arrays
    if (partly(x.k_cache, x.k_dst, codes) || partly(x.v_cache, x.v_dst, codes) || partly(x.k_scale, x.k_scale_dst, scales) ||
        partly(x.v_scale, x.v_scale_dst, scales) || partly(x.weight, x.weight_dst, sums))
      return EA_ERR_INVALID_ARG;
  }
  return mx_distinct<6>(
             a, n_layers,
             [](const ea_evict_fp8_args& x) {
               return std::array<const void*, 6>{x.k_dst, x.v_dst, x.k_scale_dst, x.v_scale_dst, x.weight_dst, x.kept};
             },
             [](const ea_evict_fp8_args& x) {  // (in place they are what is written)
               const bool other = x.k_cache != x.k_dst;
               auto src = [&](const void* q) { return other ? q : nullptr; };
               return std::array<const void*, 5>{src(x.k_cache), src(x.v_cache), src(x.k_scale), src(x.v_scale), src(x.weight)};
             })
             ? EA_OK
             : EA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int expert_attn_write_fp8(const ea_fp8_rows* layers, int n_layers, int row0, int n_rows, int Smax, int dtype,
                          int64_t head_stride, int64_t row_stride, ea_stream_t stream) {
  return run_rows(layers, n_layers, row0, n_rows, Smax, dtype, head_stride, row_stride, true, stream);
}

int expert_attn_read_fp8(const ea_fp8_rows* layers, int n_layers, int row0, int n_rows, int Smax, int dtype,
                         int64_t head_stride, int64_t row_stride, ea_stream_t stream) {
  return run_rows(layers, n_layers, row0, n_rows, Smax, dtype, head_stride, row_stride, false, stream);
}

size_t text_decode_fp8_workspace_size(int n_layers, int Smax, int weights) {
  int dev;
  DeviceInfo di;
  if (n_layers < 1 || !smax_ok(Smax) || !device_info(&dev, &di)) return 0;
  return f8_decode_ws(di.sm_count, n_layers, Smax, weights != 0).total;
}

int text_decode_attention_fp8(const ea_decode_fp8_args* layers, int n_layers, int pos, int Smax, int rope_delta,
                              void* workspace, size_t ws_bytes, ea_stream_t stream) {
  const long long p0 = static_cast<long long>(pos) + rope_delta;
  int rc = validate_decode(layers, n_layers, pos, Smax, p0, workspace);
  if (rc != EA_OK) return rc;
  int dev;
  DeviceInfo di;
  if (!device_info(&dev, &di) || !decode_attrs_ready(dev)) return EA_ERR_UNSUPPORTED;
  const int per = n_layers < kDecodeMaxLayers ? n_layers : kDecodeMaxLayers;
  const F8DecodeWs wl = f8_decode_ws(di.sm_count, n_layers, Smax, any_weights(layers, n_layers));
  if (ws_bytes < wl.total) return EA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  for (int l0 = 0; l0 < n_layers; l0 += per) {
    const int n = n_layers - l0 < per ? n_layers - l0 : per;
    const bool weights = any_weights(layers + l0, n);
    const int parts = small_parts(n, pos, di.sm_count);
    rc = parts > 0 && n <= kSmallCap ? launch_small<kSmallCap>(layers + l0, n, pos, Smax, p0, weights, ws, wl, parts, st)
         : parts > 0 ? launch_small<kDecodeMaxLayers>(layers + l0, n, pos, Smax, p0, weights, ws, wl, parts, st)
         : n <= kSmallCap ? launch_decode_t<kSmallCap>(layers + l0, n, pos, Smax, p0, weights, ws, wl, di.sm_count, st)
                          : launch_decode_t<kDecodeMaxLayers>(layers + l0, n, pos, Smax, p0, weights, ws, wl, di.sm_count, st);
    const bool formed = parts > 0 ? small_forms(parts) : forms_weights(n, pos, di.sm_count);
    if (rc == EA_OK && weights && !formed) rc = launch_weights(layers + l0, n, pos, Smax, ws, wl, st);
    if (rc != EA_OK) return rc;
  }
  return EA_OK;
}

size_t expert_attn_evict_fp8_workspace_size(int n_layers, int Smax) {
  int dev;
  DeviceInfo di;
  if (n_layers < 1 || !smax_ok(Smax) || !device_info(&dev, &di)) return 0;
  return f8_evict_ws(n_layers, Smax).total;
}

int expert_attn_evict_fp8(const ea_evict_fp8_args* layers, int n_layers, int n_rows, int n_keep, int n_first, int n_recent,
                          int Smax, void* workspace, size_t ws_bytes, ea_stream_t stream) {
  const int rc = validate_evict(layers, n_layers, n_rows, n_keep, n_first, n_recent, Smax, workspace);
  if (rc != EA_OK) return rc;
  int dev;
  DeviceInfo di;
  if (!device_info(&dev, &di) || !evict_attrs_ready(dev)) return EA_ERR_UNSUPPORTED;
  const F8EvictWs wl = f8_evict_ws(n_layers, Smax);
  if (ws_bytes < wl.total) return EA_ERR_WORKSPACE;
  if (n_keep == 0) return EA_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  F8EvictParams p;
  std::memset(&p, 0, sizeof(p));
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.ticket = reinterpret_cast<uint32_t*>(ws + wl.ticket_off);
  p.before = reinterpret_cast<uint32_t*>(ws + wl.before_off);
  p.loaded = reinterpret_cast<uint32_t*>(ws + wl.loaded_off);
  p.n_rows = n_rows;
  p.n_keep = n_keep;
  p.n_first = n_first;
  p.n_recent = n_recent;
  p.Smax = Smax;
  p.blocks = Smax / kScaleBlock;
  cudaLaunchAttribute attr[1];
  for (int l0 = 0; l0 < n_layers; l0 += kMaxLayersPerLaunch) {
    p.n_layers = n_layers - l0 < kMaxLayersPerLaunch ? n_layers - l0 : kMaxLayersPerLaunch;
    p.ordered = 0;
    for (int l = 0; l < p.n_layers; ++l) {
      const ea_evict_fp8_args& x = layers[l0 + l];
      p.ordered |= x.k_cache == x.k_dst;
      p.layer[l] = {static_cast<const uint8_t*>(x.k_cache), static_cast<const uint8_t*>(x.v_cache), x.k_scale, x.v_scale, x.weight,
                    static_cast<uint8_t*>(x.k_dst), static_cast<uint8_t*>(x.v_dst), x.k_scale_dst, x.v_scale_dst, x.weight_dst, x.kept};
    }
    if (launch_fp8_evict(p, di.sm_count, launch_config(static_cast<cudaStream_t>(stream), attr, true)) != cudaSuccess) {
      cudaGetLastError();
      return EA_ERR_CUDA;
    }
  }
  return EA_OK;
}

}  // extern "C"
