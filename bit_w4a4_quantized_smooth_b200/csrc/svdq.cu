// C ABI of the SVDQuant W4A4 linear layer (include/svdq.h): argument
// validation, TMA tensor maps and kernel launches.  Host code only launches
// the kernels of the headers below; no step of the layer runs on the host.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "../../include/svdq.h"
#include "calib.cuh"
#include "fp8.cuh"
#include "linear.cuh"
#include "linear_fp8.cuh"
#include "linear_fp8_splitk.cuh"
#include "linear_splitk.cuh"
#include "lora.cuh"
#include "pack_residual.cuh"
#include "quantize_act.cuh"

namespace {

// ------------------------------------------------------------- limits --
// Rows (M, N) up to 2^22 and K up to 2^20 keep every grid dimension, tile
// count and 32-bit index product of the kernels in range.
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxK = int64_t(1) << 20;
// svdq_rmsnorm keeps a row in one CTA's registers: 16 warps x 4 x 512 values.
constexpr int64_t kMaxNormK = 32768;

// Which linear kernel svdq_linear launches: 0 picks by shape, 1 forces the
// large-M kernel, 2 the small-M kernel (svdq_set_linear_path).
std::atomic<int> g_linear_path{0};

// The same for svdq_linear_fp8 and svdq_linear_fp8_gelu (svdq_set_linear_fp8_path).
std::atomic<int> g_linear8_path{0};

// CTAs that share a tile of the few-rows kernel: 0 by estimate (svdq_set_linear_fp8_splits).
std::atomic<int> g_linear8_splits{0};

// Whether the layer's launches carry the programmatic stream-serialisation
// attribute (svdq_set_launch_overlap; default on).  With it a layer kernel
// may be scheduled while the kernel ahead of it in the stream finishes; it
// sets up (barriers, tensor memory, L2 prefetch of weights) and then waits
// in-kernel for that kernel before it touches anything it could share with it.
std::atomic<int> g_overlap{1};

// Appends the overlap attribute to attrs[n] when the setting is on.
unsigned add_overlap_attr(cudaLaunchAttribute* attrs, unsigned n) {
  if (!g_overlap.load(std::memory_order_relaxed)) return n;
  attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[n].val.programmaticStreamSerializationAllowed = 1;
  return n + 1;
}

// -------------------------------------------------------- wait timeout --
std::atomic<uint64_t> g_timeout_ns{0};

uint64_t wait_timeout_ns() {
  uint64_t t = g_timeout_ns.load(std::memory_order_relaxed);
  if (t == 0) {
    uint64_t ms = 2000;
    if (const char* e = std::getenv("SVDQ_WAIT_TIMEOUT_MS")) {
      long long v = std::atoll(e);
      if (v > 0) ms = static_cast<uint64_t>(v);
    }
    t = ms * 1000000ull;
    uint64_t expected = 0;
    if (!g_timeout_ns.compare_exchange_strong(expected, t)) t = expected;
  }
  return t;
}

// --------------------------------------------------------- tensor maps --
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// A tensor map is a pure function of its encoding parameters (the global
// address among them), so encoded maps are kept in a small cache keyed by
// all of them: a call whose buffers and shapes repeat an earlier call's
// reuses the earlier encoding instead of encoding again.
struct MapKey {
  uint64_t words[12];
  bool operator==(const MapKey& o) const { return std::memcmp(words, o.words, sizeof(words)) == 0; }
};
struct MapKeyHash {
  size_t operator()(const MapKey& k) const {
    uint64_t h = 1469598103934665603ull;
    for (uint64_t w : k.words) {
      h ^= w;
      h *= 1099511628211ull;
    }
    return static_cast<size_t>(h);
  }
};
constexpr size_t kMapCacheCap = 4096;
std::mutex g_map_mu;
std::unordered_map<MapKey, CUtensorMap, MapKeyHash> g_maps;

// 2D/3D tiled tensor map; dims/strides innermost first, strides in bytes.
svdq_status make_tmap(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t rank, const void* base,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swizzle) {
  MapKey key;
  std::memset(&key, 0, sizeof(key));
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SVDQ_ERR_CUDA;
  key.words[0] = static_cast<uint64_t>(dtype) | (static_cast<uint64_t>(rank) << 8) |
                 (static_cast<uint64_t>(swizzle) << 16) | (static_cast<uint64_t>(dev) << 32);
  key.words[1] = reinterpret_cast<uintptr_t>(base);
  for (uint32_t i = 0; i < rank; ++i) {
    key.words[2 + i] = dims[i];
    key.words[5 + i] = box[i];
    if (i + 1 < rank) key.words[8 + i] = strides[i];
  }
  {
    std::lock_guard<std::mutex> lock(g_map_mu);
    auto it = g_maps.find(key);
    if (it != g_maps.end()) {
      *map = it->second;
      return SVDQ_OK;
    }
  }
  auto enc = encode_fn();
  if (!enc) return SVDQ_ERR_CUDA;
  uint32_t estr[3] = {1, 1, 1};
  CUresult rc = enc(map, dtype, rank, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (rc != CUDA_SUCCESS) return SVDQ_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_map_mu);
  if (g_maps.size() >= kMapCacheCap) g_maps.clear();
  g_maps.emplace(key, *map);
  return SVDQ_OK;
}

// ---------------------------------------------------- device properties --
constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];

int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  return dev;
}

int sm_count(int dev) {
  int n = g_sm_count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    g_sm_count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// The largest dynamic shared memory size set so far, per (kernel, device):
// cudaFuncSetAttribute runs once per kernel and device unless a launch needs
// more than any earlier one.
std::mutex g_attr_mu;
std::unordered_map<uint64_t, int> g_smem_set;

svdq_status ensure_smem(const void* kern, int dev, size_t bytes) {
  const uint64_t key = (reinterpret_cast<uintptr_t>(kern) << 8) ^ static_cast<uint64_t>(dev);
  std::lock_guard<std::mutex> lock(g_attr_mu);
  auto it = g_smem_set.find(key);
  if (it != g_smem_set.end() && static_cast<size_t>(it->second) >= bytes) return SVDQ_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) !=
      cudaSuccess)
    return SVDQ_ERR_CUDA;
  g_smem_set[key] = static_cast<int>(bytes);
  return SVDQ_OK;
}

// Dynamic shared memory per CTA such that CTAs that each allocate
// `tmem_cols` tensor-memory columns never oversubscribe the SM's 512: the
// request is raised until shared memory alone admits no more CTAs per SM
// than the tensor memory does.  (A CTA blocked in tcgen05.alloc behind a CTA
// of its own cluster would wait for it forever.)
size_t smem_for_tmem(int dev, size_t smem, uint32_t tmem_cols) {
  if (tmem_cols == 0) return smem;
  int per_sm = 0, reserved = 0;
  if (cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
    return 0;
  const size_t allowed = 512 / tmem_cols;
  const size_t floor_bytes = static_cast<size_t>(per_sm) / (allowed + 1) + 1;  // > per_sm / (allowed + 1)
  if (smem + static_cast<size_t>(reserved) < floor_bytes) smem = floor_bytes - static_cast<size_t>(reserved);
  return smem;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

bool valid_rank(int64_t r) { return r >= 0 && r <= 128 && r % 16 == 0; }

// Every entry that reaches the CUDA runtime runs in here.  A launch is judged
// by its own return value, not by cudaGetLastError(), which may hold an error
// of the caller's; a call that fails takes its own error off that slot again,
// where the next check of the program (torch shares the runtime) would find it.
// The caches of maps, plans and limits allocate: no exception leaves a C call.
template <typename F>
svdq_status guarded(F&& f) {
  svdq_status rc = SVDQ_ERR_CUDA;
  try {
    rc = f();
  } catch (...) {
  }
  if (rc == SVDQ_ERR_CUDA) cudaGetLastError();
  return rc;
}

svdq_status launched(cudaError_t e) { return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA; }

// A plain launch: one block shape, no dynamic shared memory, no attributes.
template <typename... P, typename... A>
svdq_status launch_plain(void (*kern)(P...), dim3 grid, unsigned threads, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return launched(cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...));
}

uint32_t pow2_at_least(uint32_t x) {
  uint32_t p = 32;
  while (p < x) p <<= 1;
  return p;
}

// Work split of the activation step: 128-row tiles; when they are fewer
// than the SMs, the 64-column atoms of K are split over up to 16 CTAs per
// tile (no CTA without atoms).
struct QaPlan {
  int64_t row_tiles;
  int splits, apc;
};

QaPlan qa_plan(int64_t M, int64_t K, int sms) {
  QaPlan pl;
  pl.row_tiles = (M + svdq::kQaRows - 1) / svdq::kQaRows;
  const int atoms = static_cast<int>(K / 64);
  int splits = 1;
  if (pl.row_tiles < sms) {
    splits = static_cast<int>(sms / pl.row_tiles);
    if (splits > svdq::kQaMaxSplits) splits = svdq::kQaMaxSplits;
    if (splits > atoms) splits = atoms;
    if (splits < 1) splits = 1;
  }
  pl.apc = (atoms + splits - 1) / splits;
  pl.splits = (atoms + pl.apc - 1) / pl.apc;
  return pl;
}

// Small-M linear: 128 x 128 tiles, K stages split over a cluster.  The
// split minimises the stages the busiest SM runs (tiles x splits CTAs over
// the SMs, each CTA ceil(stages / splits) stages, plus one for the cluster's
// reduction), the smaller split on ties.
svdq_status launch_linear_splitk(const CUtensorMap& tm_xc, const CUtensorMap& tm_rc, const CUtensorMap& tm_xs,
                                 const CUtensorMap& tm_rs, const CUtensorMap& tm_t, const CUtensorMap& tm_l2,
                                 const void* bias, void* Y, int64_t M, int64_t K, int64_t N, int64_t r, float alpha,
                                 int dev, int sms, void* stream) {
  const int64_t tiles_m = (M + svdq::kLsBM - 1) / svdq::kLsBM;
  const int64_t tiles_n = (N + svdq::kLsBN - 1) / svdq::kLsBN;
  const int64_t tiles = tiles_m * tiles_n;
  const int n_k = static_cast<int>((K + svdq::kLsBK - 1) / svdq::kLsBK);
  const int n_lr = static_cast<int>((r + 63) / 64);
  int best_s = 1;
  int64_t best_cost = -1;
  for (int s = 1; s <= svdq::kLsMaxSplits && s <= n_k; ++s) {
    const int spc = (n_k + s - 1) / s;
    const int se = (n_k + spc - 1) / spc;
    if (se != s) continue;
    const int64_t cost = ((tiles * se + sms - 1) / sms) * (spc + n_lr) + (se > 1 ? 1 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best_s = s;
    }
  }
  const int splits = best_s;
  const int spc = (n_k + splits - 1) / splits;
  int stages = spc + n_lr;
  if (stages > svdq::kLsMaxStages) stages = svdq::kLsMaxStages;
  uint32_t ring = static_cast<uint32_t>(stages) * svdq::kLsStageBytes;
  if (splits > 1 && ring < svdq::kLsPartBytes) ring = svdq::kLsPartBytes;
  const size_t smem = smem_for_tmem(dev, 1024 + svdq::kLsHeadBytes + ring, svdq::kLsTmemCols);
  if (smem == 0 || smem > 232448) return SVDQ_ERR_CUDA;
  const void* kern = reinterpret_cast<const void*>(svdq::linear_splitk_kernel);
  if (svdq_status rc = ensure_smem(kern, dev, smem)) return rc;

  svdq::LsParams p;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.alpha = alpha;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.r = static_cast<int>(r);
  p.splits = splits;
  p.spc = spc;
  p.stages = stages;
  p.timeout_ns = wait_timeout_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(tiles_n), static_cast<unsigned>(tiles_m));
  cfg.blockDim = dim3(svdq::kLsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (splits > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    na = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = add_overlap_attr(attr, na);
  return launched(cudaLaunchKernelEx(&cfg, svdq::linear_splitk_kernel, tm_xc, tm_rc, tm_xs, tm_rs, tm_t, tm_l2, p));
}

// ------------------------------------------------------------ 8-bit layer --
// Launches `kern` with the layer's launch-overlap setting.
template <typename... P, typename... A>
svdq_status launch(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, void* stream,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (cluster > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    na = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = add_overlap_attr(attr, na);
  return launched(cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...));
}

// Codes [rows][K] as boxes of 128 columns x `box_rows` rows, 128-byte swizzle.
svdq_status fp8_codes_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(K)};
  const uint32_t box[2] = {128, box_rows};
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles of 512 bytes, viewed as [tiles][2][256]: one tile a box.
svdq_status fp8_scales_map(CUtensorMap* map, const void* scales, int64_t rows, int64_t K) {
  const uint64_t dims[3] = {256, 2,
                            static_cast<uint64_t>((rows + 127) / 128) * static_cast<uint64_t>(svdq::fp8_band_tiles(K))};
  const uint64_t strides[2] = {256, 512};
  const uint32_t box[3] = {256, 2, 1};
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, scales, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Few rows: 128-channel tiles, K split over a cluster; `bm` tokens a tile (M
// padded to 16, at most 128).  us: the estimate below, compared with the
// large-M kernel's.
struct S8Plan {
  int bm, splits, spc, stages;
  uint32_t tmem_cols;
  size_t smem;
  double us;
};

// CTAs of the kernel that the device holds at once, as clusters of `splits`:
// the occupancy of an empty kernel with the same block and shared memory,
// because the runtime answers one CTA per SM for any kernel that allocates
// tensor memory (smem_for_tmem has made shared memory the tighter limit).
int s8_active(int splits, size_t smem, int sms) {
  const void* kern = reinterpret_cast<const void*>(svdq::linear_fp8_splitk_occupancy_kernel);
  if (splits == 1) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, svdq::kS8Threads, smem) != cudaSuccess) {
      cudaGetLastError();  // this split is passed over; no error of the call
      return 0;
    }
    return per_sm * sms;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits * sms));
  cfg.blockDim = dim3(svdq::kS8Threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n * splits;
}

// The split of K and the ring depth with the least estimated time.  The
// estimate was fitted on B200 to the times of every split from 1 to 8 and
// depth from 2 to 8, and of the large-M kernel, at 140 sizes (M 1 to 2048, K
// 256 to 12288, N 512 to 12288; weights from HBM, launches back to back), for
// the choice rather than for the time itself: with x = bm / 128 and `occ` CTAs
// on an SM,
//   2.0 + 0.97 x us            launch, start, epilogue
//   + 1.9 with a cluster, + 0.37 per 100 CTAs (cluster launch and exchange)
//   + waves spc max(0.21, 0.71 (1 + 1.3 x) / depth, (0.097 + 0.13 x) occ)
//                              a stage: its issue; the latency of a load over
//                              the ring's depth; the SM's share of its loads
//   + 6.0 (waves - 1)          clusters that do not fit at once
//   + 0.25 passes              with GELU: six warps take a token each at a time
// Against the best of all measured, its choice (of the kernel as well) costs
// 0.5 % on average and 8 % at the worst.  At 110 other sizes (M 1 to 1024),
// against this choice with 2 and 4 us a wave and the large-M kernel: 0.3 % on
// average, 2 % at the worst for bf16 and 6 % with GELU (2 us a wave lost 41 %
// at 512 x 12288 x 3072; a choice that does not count the GELU 8 % on average
// and 62 % at the worst).  The deeper ring on ties.
// With `forced` splits only that many are considered, or the next smaller
// number that leaves no CTA without stages.
svdq_status s8_plan(S8Plan* out, bool gelu, int forced, int64_t M, int64_t K, int64_t N, int dev, int sms) {
  S8Plan best = {};
  const int bm = M >= svdq::kS8MaxBM ? svdq::kS8MaxBM : static_cast<int>((M + 15) / 16 * 16);
  const double x = bm / 128.0;
  const int64_t tiles = (N + svdq::kS8BN - 1) / svdq::kS8BN * ((M + svdq::kS8MaxBM - 1) / svdq::kS8MaxBM);
  const int k_stages = static_cast<int>((K + svdq::kS8BK - 1) / svdq::kS8BK);
  const uint32_t stage = svdq::s8_stage_bytes(bm);
  const uint32_t tmem_cols = pow2_at_least(static_cast<uint32_t>(bm + 32));
  const void* model = reinterpret_cast<const void*>(svdq::linear_fp8_splitk_occupancy_kernel);
  if (svdq_status rc = ensure_smem(model, dev, svdq::kS8SmemLimit)) return rc;
  int first = 1, last = std::min(svdq::kS8MaxSplits, k_stages);
  if (forced > 0) {
    last = std::min(last, forced);
    while ((k_stages + (k_stages + last - 1) / last - 1) / ((k_stages + last - 1) / last) != last) --last;
    first = last;
  }
  for (int s = first; s <= last; ++s) {
    const int spc = (k_stages + s - 1) / s;
    const int passes = ((bm + s - 1) / s + 5) / 6;
    if ((k_stages + spc - 1) / spc != s) continue;  // no CTA without stages
    for (int depth = std::min(spc, 3); depth <= std::min(spc, 8); ++depth) {
      const uint32_t ring = std::max<uint32_t>(depth * stage, static_cast<uint32_t>(bm) * svdq::kS8BN * 4);
      const size_t smem = smem_for_tmem(dev, 1024 + svdq::kS8HeadBytes + ring, tmem_cols);
      if (smem == 0 || smem > svdq::kS8SmemLimit) continue;
      const int active = s8_active(s, smem, sms);
      if (active <= 0) continue;
      const double ctas = static_cast<double>(tiles) * s;
      const double waves = std::ceil(ctas / active);
      const double occ = std::max(1.0, std::min<double>(ctas, active) / sms);
      const double per = std::max({0.21, 0.71 * (1.0 + 1.3 * x) / depth, (0.097 + 0.13 * x) * occ});
      const double us = 2.0 + 0.97 * x + (s > 1 ? 1.9 : 0.0) + 0.0037 * ctas + waves * spc * per + 6.0 * (waves - 1) -
                        0.02 * depth + (gelu ? 0.25 * passes : 0.0);
      if (best.splits == 0 || us < best.us) best = {bm, s, spc, depth, tmem_cols, smem, us};
    }
  }
  if (best.splits == 0) return SVDQ_ERR_CUDA;
  *out = best;
  return SVDQ_OK;
}

// The plan is a pure function of the sizes and the device, so chosen ones are
// kept (the occupancy calls take tens of microseconds).
struct S8Key {
  uint64_t words[3];
  bool operator==(const S8Key& o) const { return std::memcmp(words, o.words, sizeof(words)) == 0; }
};
struct S8KeyHash {
  size_t operator()(const S8Key& k) const {
    uint64_t h = 1469598103934665603ull;
    for (uint64_t w : k.words) h = (h ^ w) * 1099511628211ull;
    return static_cast<size_t>(h);
  }
};
std::mutex g_s8_mu;
std::unordered_map<S8Key, S8Plan, S8KeyHash> g_s8_plans;

svdq_status s8_plan_kept(S8Plan* out, bool gelu, int64_t M, int64_t K, int64_t N, int dev, int sms) {
  // M only through its tile count and padded tile
  const uint64_t m_class = M >= svdq::kS8MaxBM ? static_cast<uint64_t>((M + 127) / 128) << 8
                                               : static_cast<uint64_t>((M + 15) / 16);
  const int forced = g_linear8_splits.load(std::memory_order_relaxed);
  const S8Key key = {{m_class | static_cast<uint64_t>(forced) << 40 | static_cast<uint64_t>(gelu) << 47 |
                          static_cast<uint64_t>(dev) << 48,
                      static_cast<uint64_t>(K), static_cast<uint64_t>(N)}};
  {
    std::lock_guard<std::mutex> lock(g_s8_mu);
    auto it = g_s8_plans.find(key);
    if (it != g_s8_plans.end()) {
      *out = it->second;
      return SVDQ_OK;
    }
  }
  if (svdq_status rc = s8_plan(out, gelu, forced, M, K, N, dev, sms)) return rc;
  std::lock_guard<std::mutex> lock(g_s8_mu);
  if (g_s8_plans.size() >= kMapCacheCap) g_s8_plans.clear();
  g_s8_plans.emplace(key, *out);
  return SVDQ_OK;
}

template <bool FP8_OUT>
svdq_status launch_s8(const S8Plan& pl, int dev, const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                      const uint8_t* w_scales, const void* bias, int64_t M, int64_t K, int64_t N, void* Y,
                      uint8_t* y_scales, void* stream) {
  CUtensorMap tm_x, tm_w;
  if (svdq_status rc = fp8_codes_map(&tm_x, x_codes, M, K, static_cast<uint32_t>(pl.bm))) return rc;
  if (svdq_status rc = fp8_codes_map(&tm_w, w_codes, N, K, svdq::kS8BN)) return rc;
  const bool many = pl.bm > 64 && pl.splits >= 2 && pl.splits <= 4;
  auto kern = many ? svdq::linear_fp8_splitk_kernel<FP8_OUT, true> : svdq::linear_fp8_splitk_kernel<FP8_OUT, false>;
  if (svdq_status rc = ensure_smem(reinterpret_cast<const void*>(kern), dev, svdq::kS8SmemLimit)) return rc;
  svdq::S8Params p;
  p.x_scales = x_scales;
  p.w_scales = w_scales;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.Y = Y;
  p.y_scales = y_scales;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.bm = pl.bm;
  p.splits = pl.splits;
  p.spc = pl.spc;
  p.stages = pl.stages;
  p.tmem_cols = pl.tmem_cols;
  p.timeout_ns = wait_timeout_ns();
  const dim3 grid(static_cast<unsigned>(pl.splits), static_cast<unsigned>((N + svdq::kS8BN - 1) / svdq::kS8BN),
                  static_cast<unsigned>((M + svdq::kS8MaxBM - 1) / svdq::kS8MaxBM));
  return launch(kern, grid, svdq::kS8Threads, pl.smem, static_cast<unsigned>(pl.splits), stream, tm_x, tm_w, p);
}

// Rows of 256-row tiles per group of the large-M kernel's visiting order.  The
// pairs work on about 74 neighbouring tiles at once; whatever they come back
// to later should still be in L2, which keeps about half of its 126 MB of data
// that both dies read.  All rows, where the x codes fit beside the streamed w
// (8192 x 4096 x 14336 on B200: 378 us against 400 with 2 rows); otherwise two
// rows, where w fits and x is streamed (4608 x 12288 x 3072: 137 us against 145
// with all, 16384 x 12288 x 3072: 485 against 644); otherwise about 32 MB of x
// (8192 x 8192 x 8192: 417 us against 428 with 2 rows and 480 with all; 8192 x
// 14336 x 4096: 375, 385, 415).  All times are of calls in a row.
int l8_group(int64_t M, int64_t K, int64_t N, int m_tiles) {
  constexpr int64_t kX = 40000000, kW = 48000000, kPart = 33600000;
  if (M * K <= kX) return m_tiles;
  const int64_t g = N * K <= kW ? 2 : std::max<int64_t>(1, kPart / (svdq::kL8BM * K));
  return static_cast<int>(std::min<int64_t>(g, m_tiles));
}

// The product's entry: Y bf16 [M][N] (y_scales null), or codes [M][N] with
// y_scales and the GELU epilogue.
svdq_status linear_fp8_impl(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                            const uint8_t* w_scales, const void* bias, int64_t M, int64_t K, int64_t N, void* Y,
                            uint8_t* y_scales, bool fp8_out, void* stream) {
  if (!x_codes || !x_scales || !w_codes || !w_scales || !Y || (fp8_out && !y_scales) || M <= 0 || K <= 0 || N <= 0)
    return SVDQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % (fp8_out ? 16 : 8) != 0 || M > kMaxRows || N > kMaxRows || K > kMaxK ||
      (fp8_out && N > kMaxK))
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y) ||
      (bias && !aligned16(bias)) || (y_scales && !aligned16(y_scales)))
    return SVDQ_ERR_MISALIGNED;
  const int dev = current_device();
  if (dev < 0) return SVDQ_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms < 2) return SVDQ_ERR_CUDA;
  // The few-rows kernel where its estimate is below the large-M kernel's, 4.5
  // us (6.1 with GELU) + (0.30 a stage of 128 columns + 0.75) for every wave of CTA pairs
  // (measured on B200: 12.0 us against 7.8 at 128 x 3072 x 3072, 33.5 against
  // 17.3 at 256 x 12288 x 3072 and 29.4 at 512, but 14.3 against 15.3 at 256 x
  // 3072 x 12288 and 14.1 against 15.5 at 512 x 3072 x 9216).
  const int64_t pair_tiles = ((M + svdq::kL8BM - 1) / svdq::kL8BM) * ((N + svdq::kL8BN - 1) / svdq::kL8BN);
  const int64_t pair_waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  const int path = g_linear8_path.load(std::memory_order_relaxed);
  if (path == 2 || (path == 0 && M <= 2048)) {
    S8Plan pl;
    if (svdq_status rc = s8_plan_kept(&pl, fp8_out, M, K, N, dev, sms)) return rc;
    const double stages = static_cast<double>((K + svdq::kL8BK - 1) / svdq::kL8BK);
    if (path == 2 || pl.us < (fp8_out ? 6.1 : 4.5) + static_cast<double>(pair_waves) * (0.30 * stages + 0.75))
      return fp8_out ? launch_s8<true>(pl, dev, x_codes, x_scales, w_codes, w_scales, bias, M, K, N, Y, y_scales, stream)
                     : launch_s8<false>(pl, dev, x_codes, x_scales, w_codes, w_scales, bias, M, K, N, Y, nullptr, stream);
  }

  CUtensorMap tm_x, tm_w, tm_xs, tm_ws, tm_y;
  if (svdq_status rc = fp8_codes_map(&tm_x, x_codes, M, K, 128)) return rc;
  if (svdq_status rc = fp8_codes_map(&tm_w, w_codes, N, K, 128)) return rc;
  if (svdq_status rc = fp8_scales_map(&tm_xs, x_scales, M, K)) return rc;
  if (svdq_status rc = fp8_scales_map(&tm_ws, w_scales, N, K)) return rc;
  if (fp8_out) {
    if (svdq_status rc = fp8_codes_map(&tm_y, Y, M, N, 32)) return rc;  // one epilogue warp's 32 x 128 block
  } else {
    const uint64_t dims[2] = {static_cast<uint64_t>(N), static_cast<uint64_t>(M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(N) * 2};
    const uint32_t box[2] = {64, 32};  // one epilogue warp's 32 x 64 block
    if (svdq_status rc = make_tmap(&tm_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, dims, strides, box,
                                   CU_TENSOR_MAP_SWIZZLE_128B))
      return rc;
  }
  svdq::L8Params p;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.y_scales = y_scales;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.one = 1;
  p.m_tiles = static_cast<int>((M + svdq::kL8BM - 1) / svdq::kL8BM);
  const int n_tiles = static_cast<int>((N + svdq::kL8BN - 1) / svdq::kL8BN);
  p.tiles = p.m_tiles * n_tiles;
  p.group = l8_group(M, K, N, p.m_tiles);
  p.group_tiles = p.group * n_tiles;
  p.timeout_ns = wait_timeout_ns();
  const size_t smem = 1024 + svdq::kL8BarOffset + (svdq::kL8NumBars + 4) * 8;
  auto kern = fp8_out ? svdq::linear_fp8_kernel<true> : svdq::linear_fp8_kernel<false>;
  if (svdq_status rc = ensure_smem(reinterpret_cast<const void*>(kern), dev, smem)) return rc;
  const int pairs = p.tiles < sms / 2 ? p.tiles : sms / 2;
  return launch(kern, dim3(static_cast<unsigned>(2 * pairs)), fp8_out ? svdq::kL8ThreadsFp8 : svdq::kL8Threads, smem, 2, stream, tm_x, tm_w, tm_xs,
                tm_ws, tm_y, p);
}

template <typename RES>
svdq_status launch_rmsnorm(const void* X, int64_t ldx, const void* residual, const void* gamma, float eps, int64_t M,
                           int64_t K, void* residual_out, void* Y, uint8_t* x_codes, uint8_t* x_scales, void* stream) {
  // One segment of 512 columns a warp as far as 16 warps reach; two where
  // there are rows enough to fill the SMs several times.  Measured on B200 at
  // K = 4096 with a bf16 residual and FP8 output, one against two, by segments
  // an SM: 5.9 and 6.6 us at 40, 11.6 and 11.8 at 100, 14.1 and 14.0 at 130,
  // 16.5 and 16.2 at 160, 28.3 and 27.2 at 300, 86.8 and 79.6 at 1000 (K = 1024
  // and 3072 within 5 % of that; K = 8192, 16 warps a row, gains from two at 64
  // already, 9.3 and 8.2).  With an fp32 residual one stays better, 28.9 and 30.0
  // at 200, 64.5 and 65.4 at 500.  A row of one warp: four a CTA.
  const int dev = current_device();
  if (dev < 0) return SVDQ_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return SVDQ_ERR_CUDA;
  const int segs = static_cast<int>(svdq::fp8_band_tiles(K));
  const bool many = sizeof(RES) == 2 && M * segs >= 160 * static_cast<int64_t>(sms) && segs > 1;
  const int s = std::max((segs + 15) / 16, many ? 2 : 1);
  const int wpr = (segs + s - 1) / s;
  const int rpc = wpr == 1 ? 4 : 1;
  const bool wide = aligned32(X) && ldx % 16 == 0 && aligned32(residual) && aligned32(residual_out) &&
                    aligned32(gamma) && aligned32(Y);  // K is a multiple of 16
  auto kern = s == 1   ? svdq::rmsnorm_kernel<1, RES>
              : s == 2 ? svdq::rmsnorm_kernel<2, RES>
              : s == 3 ? svdq::rmsnorm_kernel<3, RES>
                       : svdq::rmsnorm_kernel<4, RES>;
  return launch(kern, dim3(static_cast<unsigned>((M + rpc - 1) / rpc + 1)), static_cast<unsigned>(32 * wpr * rpc), 0, 1,
                stream, static_cast<const __nv_bfloat16*>(X), ldx, static_cast<const RES*>(residual),
                static_cast<const __nv_bfloat16*>(gamma), eps, static_cast<int>(M), static_cast<int>(K), wpr, wide,
                static_cast<RES*>(residual_out), static_cast<__nv_bfloat16*>(Y), x_codes, x_scales);
}
}  // namespace

extern "C" {

const char* svdq_status_string(int status) {
  switch (status) {
    case SVDQ_OK: return "SVDQ_OK";
    case SVDQ_ERR_INVALID_ARG: return "SVDQ_ERR_INVALID_ARG";
    case SVDQ_ERR_UNSUPPORTED_SHAPE: return "SVDQ_ERR_UNSUPPORTED_SHAPE";
    case SVDQ_ERR_MISALIGNED: return "SVDQ_ERR_MISALIGNED";
    case SVDQ_ERR_CUDA: return "SVDQ_ERR_CUDA";
    case SVDQ_ERR_TIMEOUT: return "SVDQ_ERR_TIMEOUT";
    default: return "SVDQ_UNKNOWN_STATUS";
  }
}

svdq_status svdq_packed_sizes(int64_t rows, int64_t K, size_t* codes_bytes, size_t* scales_bytes) {
  if (rows < 0 || K <= 0 || !codes_bytes || !scales_bytes) return SVDQ_ERR_INVALID_ARG;
  if (K % 64 != 0 || K > kMaxK || rows > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  *codes_bytes = static_cast<size_t>(rows) * static_cast<size_t>(K / 2);
  *scales_bytes = static_cast<size_t>((rows + 127) / 128) * 128 * static_cast<size_t>(K / 16);
  return SVDQ_OK;
}

svdq_status svdq_pack_residual(const float* R, int64_t K, int64_t N, uint8_t* r_codes, uint8_t* r_scales,
                               void* stream) {
  if (!R || !r_codes || !r_scales || K <= 0 || N <= 0) return SVDQ_ERR_INVALID_ARG;
  if (K % 64 != 0 || N % 16 != 0 || K > kMaxK || N > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(R) || !aligned16(r_codes) || !aligned16(r_scales)) return SVDQ_ERR_MISALIGNED;
  dim3 grid(static_cast<unsigned>((N + 127) / 128), static_cast<unsigned>(K / 64));
  return guarded([&] {
    return launch_plain(svdq::pack_residual_kernel, grid, svdq::kPackThreads, stream, R, static_cast<int>(K),
                        static_cast<int>(N), r_codes, r_scales);
  });
}

svdq_status svdq_quantize_act_workspace(int64_t M, int64_t K, int64_t r, size_t* bytes) {
  if (!bytes || M <= 0 || K <= 0) return SVDQ_ERR_INVALID_ARG;
  if (K % 64 != 0 || !valid_rank(r) || M > kMaxRows || K > kMaxK) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  return guarded([&] {
    const int dev = current_device();
    if (dev < 0) return SVDQ_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SVDQ_ERR_CUDA;
    const QaPlan pl = qa_plan(M, K, sms);
    *bytes = svdq::qa_workspace_bytes(pl.row_tiles, pl.splits, static_cast<int>(r));
    return SVDQ_OK;
  });
}

namespace {
svdq_status quantize_act_impl(const void* X, const float* inv_lambda, const void* L1, int64_t M, int64_t K,
                              int64_t r, uint8_t* x_codes, uint8_t* x_scales, void* T, void* workspace,
                              size_t workspace_bytes, void* stream, bool gelu);
}  // namespace

svdq_status svdq_quantize_act(const void* X, const float* inv_lambda, const void* L1, int64_t M, int64_t K,
                              int64_t r, uint8_t* x_codes, uint8_t* x_scales, void* T, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return quantize_act_impl(X, inv_lambda, L1, M, K, r, x_codes, x_scales, T, workspace, workspace_bytes, stream,
                             false);
  });
}

svdq_status svdq_quantize_act_gelu(const void* X, const float* inv_lambda, const void* L1, int64_t M, int64_t K,
                                   int64_t r, uint8_t* x_codes, uint8_t* x_scales, void* T, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&] {
    return quantize_act_impl(X, inv_lambda, L1, M, K, r, x_codes, x_scales, T, workspace, workspace_bytes, stream,
                             true);
  });
}

namespace {
svdq_status quantize_act_impl(const void* X, const float* inv_lambda, const void* L1, int64_t M, int64_t K,
                              int64_t r, uint8_t* x_codes, uint8_t* x_scales, void* T, void* workspace,
                              size_t workspace_bytes, void* stream, bool gelu) {
  if (!X || !inv_lambda || !x_codes || !x_scales || M <= 0 || K <= 0) return SVDQ_ERR_INVALID_ARG;
  if (r > 0 && (!L1 || !T)) return SVDQ_ERR_INVALID_ARG;
  if (K % 64 != 0 || !valid_rank(r) || M > kMaxRows || K > kMaxK) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(X) || !aligned16(inv_lambda) || !aligned16(x_codes) || !aligned16(x_scales) ||
      (r > 0 && (!aligned16(L1) || !aligned16(T))) || (workspace && !aligned16(workspace)))
    return SVDQ_ERR_MISALIGNED;
  const int dev = current_device();
  if (dev < 0) return SVDQ_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return SVDQ_ERR_CUDA;

  const QaPlan pl = qa_plan(M, K, sms);
  const int ri = static_cast<int>(r);
  const size_t ws_need = svdq::qa_workspace_bytes(pl.row_tiles, pl.splits, ri);
  if (ws_need > 0 && (!workspace || workspace_bytes < ws_need)) return SVDQ_ERR_INVALID_ARG;
  const int n_l1 = r == 0 ? 0 : (r <= 64 ? 1 : 2);
  const uint32_t stage_bytes = svdq::qa_stage_bytes(n_l1);
  const uint32_t fixed = 1024 + svdq::kQaHeadBytes;
  int stages = static_cast<int>((svdq::kQaSmemLimit - fixed) / stage_bytes);
  if (stages > svdq::kQaMaxStages) stages = svdq::kQaMaxStages;
  if (stages > pl.apc) stages = pl.apc;
  if (stages < 1) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  // tensor-memory accumulators of at least 8 atoms (512 columns of K) each,
  // within the SM's 512 columns
  const int n_acc_cols = 64 * n_l1;
  int fold = pl.apc;
  uint32_t tmem_cols = 0;
  if (r > 0) {
    const int max_acc = 512 / n_acc_cols;
    fold = 8;
    if ((pl.apc + fold - 1) / fold > max_acc) fold = (pl.apc + max_acc - 1) / max_acc;
    tmem_cols = pow2_at_least(static_cast<uint32_t>(((pl.apc + fold - 1) / fold) * n_acc_cols));
  }
  const size_t smem = smem_for_tmem(dev, fixed + static_cast<size_t>(stages) * stage_bytes, tmem_cols);
  if (smem == 0 || smem > svdq::kQaSmemLimit) return SVDQ_ERR_CUDA;
  auto kfn = gelu ? svdq::quantize_act_kernel<true> : svdq::quantize_act_kernel<false>;
  const void* kern = reinterpret_cast<const void*>(kfn);
  if (svdq_status rc = ensure_smem(kern, dev, smem)) return rc;

  CUtensorMap tm_x, tm_l1, tm_xc;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(svdq::kQaRows)};
    svdq_status rc = make_tmap(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, X, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    // codes [M][K/2]: one store box per atom, 32 bytes x 128 rows (rows past M clipped)
    const uint64_t dims[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K / 2)};
    const uint32_t box[2] = {32, static_cast<uint32_t>(svdq::kQaRows)};
    svdq_status rc = make_tmap(&tm_xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x_codes, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  if (r > 0) {
    // L1 [K][r]: boxes of 64 k-rows x 64 ranks, 128-byte swizzle; ranks past
    // r arrive as zeros
    const uint64_t dims[2] = {static_cast<uint64_t>(r), static_cast<uint64_t>(K)};
    const uint64_t strides[1] = {static_cast<uint64_t>(r) * 2};
    const uint32_t box[2] = {64, 64};
    svdq_status rc = make_tmap(&tm_l1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, L1, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  } else {
    std::memset(&tm_l1, 0, sizeof(tm_l1));
  }

  svdq::QaParams p;
  p.inv_lambda = inv_lambda;
  p.x_codes = x_codes;
  p.x_scales = x_scales;
  p.T = static_cast<__nv_bfloat16*>(T);
  p.counters = ws_need ? static_cast<unsigned int*>(workspace) : nullptr;
  p.partials = ws_need ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                  svdq::kQaCounterBytes *
                                                      ((static_cast<size_t>(pl.row_tiles) * 4 +
                                                        svdq::kQaCounterBytes - 1) /
                                                       svdq::kQaCounterBytes))
                       : nullptr;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.r = ri;
  p.splits = pl.splits;
  p.apc = pl.apc;
  p.stages = stages;
  p.n_l1 = n_l1;
  p.fold = fold;
  p.stage_bytes = stage_bytes;
  p.tmem_cols = tmem_cols;
  p.timeout_ns = wait_timeout_ns();

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.splits), static_cast<unsigned>(pl.row_tiles));
  cfg.blockDim = dim3(svdq::kQaThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = add_overlap_attr(attr, 0);
  return launched(cudaLaunchKernelEx(&cfg, kfn, tm_x, tm_l1, tm_xc, p));
}
}  // namespace

svdq_status svdq_linear(const uint8_t* x_codes, const uint8_t* x_scales, const void* T, const uint8_t* r_codes,
                        const uint8_t* r_scales, const void* L2, const void* bias, int64_t M, int64_t K, int64_t N,
                        int64_t r, void* Y, void* stream) {
  return svdq_linear_scaled(x_codes, x_scales, T, r_codes, r_scales, L2, bias, M, K, N, r, 1.0f, Y, stream);
}

namespace {
svdq_status linear_impl(const uint8_t* x_codes, const uint8_t* x_scales, const void* T, const uint8_t* r_codes,
                        const uint8_t* r_scales, const void* L2, const void* bias, int64_t M, int64_t K, int64_t N,
                        int64_t r, float alpha, void* Y, void* stream) {
  // alpha: a power of two in [2^-100, 2^100] (the product acc * alpha is then exact)
  int alpha_exp = 0;
  if (!(alpha > 0.0f) || !std::isfinite(alpha) || std::frexp(alpha, &alpha_exp) != 0.5f || alpha_exp < -99 ||
      alpha_exp > 101)
    return SVDQ_ERR_INVALID_ARG;
  if (!x_codes || !x_scales || !r_codes || !r_scales || !Y || M <= 0 || K <= 0 || N <= 0)
    return SVDQ_ERR_INVALID_ARG;
  if (r > 0 && (!T || !L2)) return SVDQ_ERR_INVALID_ARG;
  if (K % 64 != 0 || N % 16 != 0 || !valid_rank(r) || M > kMaxRows || N > kMaxRows || K > kMaxK)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(r_codes) || !aligned16(r_scales) ||
      !aligned16(Y) || (bias && !aligned16(bias)) || (r > 0 && (!aligned16(T) || !aligned16(L2))))
    return SVDQ_ERR_MISALIGNED;
  const int dev = current_device();
  if (dev < 0) return SVDQ_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms < 2) return SVDQ_ERR_CUDA;

  CUtensorMap tm_xc, tm_rc, tm_t, tm_l2;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K / 2)};
    const uint32_t box[2] = {128, 128};
    svdq_status rc = make_tmap(&tm_xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x_codes, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(K / 2), static_cast<uint64_t>(N)};
    const uint64_t strides[1] = {static_cast<uint64_t>(K / 2)};
    const uint32_t box[2] = {128, 128};  // each CTA of a pair loads 128 R rows
    svdq_status rc = make_tmap(&tm_rc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, r_codes, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  // scale tiles viewed as [tiles][2][256] bytes: a box of 4 tiles is the
  // 2 KB of scales of one 256-wide K stage of a 128-row band
  CUtensorMap tm_xs, tm_rs;
  {
    const uint64_t dims[3] = {256, 2, static_cast<uint64_t>((M + 127) / 128) * static_cast<uint64_t>(K / 64)};
    const uint64_t strides[2] = {256, 512};
    const uint32_t box[3] = {256, 2, 4};
    svdq_status rc = make_tmap(&tm_xs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, x_scales, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  {
    const uint64_t dims[3] = {256, 2, static_cast<uint64_t>((N + 127) / 128) * static_cast<uint64_t>(K / 64)};
    const uint64_t strides[2] = {256, 512};
    const uint32_t box[3] = {256, 2, 4};
    svdq_status rc = make_tmap(&tm_rs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, r_scales, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc) return rc;
  }
  if (r > 0) {
    const uint64_t dt[2] = {static_cast<uint64_t>(r), static_cast<uint64_t>(M)};
    const uint64_t st[1] = {static_cast<uint64_t>(r) * 2};
    const uint32_t bt[2] = {64, 128};
    svdq_status rc = make_tmap(&tm_t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, T, dt, st, bt, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    const uint64_t dl[2] = {static_cast<uint64_t>(N), static_cast<uint64_t>(r)};
    const uint64_t sl[1] = {static_cast<uint64_t>(N) * 2};
    const uint32_t bl[2] = {64, 64};
    rc = make_tmap(&tm_l2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, L2, dl, sl, bl, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  } else {
    std::memset(&tm_t, 0, sizeof(tm_t));
    std::memset(&tm_l2, 0, sizeof(tm_l2));
  }

  CUtensorMap tm_y;
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(N), static_cast<uint64_t>(M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(N) * 2};
    const uint32_t box[2] = {64, 32};  // one epilogue warp's 32 x 64 block
    svdq_status rc = make_tmap(&tm_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, dims, strides, box,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }

  // At most 128 rows with tiles for under a quarter of the SMs: the large-M
  // kernel would leave most SMs idle, each busy pair walking all of K; the
  // small-M kernel splits K over a cluster instead.  Measured on B200
  // (K, N in {3072, 12288}): the small-M kernel is faster only there; from
  // 256 rows, or with N = 12288 at any M, the large-M kernel is.
  const int64_t pair_tiles = ((M + svdq::kLinBM - 1) / svdq::kLinBM) * ((N + svdq::kLinBN - 1) / svdq::kLinBN);
  const int path = g_linear_path.load(std::memory_order_relaxed);
  if (path == 2 || (path == 0 && M <= 128 && 4 * pair_tiles < sms))
    return launch_linear_splitk(tm_xc, tm_rc, tm_xs, tm_rs, tm_t, tm_l2, bias, Y, M, K, N, r, alpha, dev, sms,
                                stream);

  svdq::LinParams p;
  p.alpha = alpha;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.r = static_cast<int>(r);
  p.timeout_ns = wait_timeout_ns();
  p.m_tiles = static_cast<int>((M + svdq::kLinBM - 1) / svdq::kLinBM);
  p.tiles = p.m_tiles * static_cast<int>((N + svdq::kLinBN - 1) / svdq::kLinBN);

  const size_t smem = 1024 + svdq::kLinBarOffset + (svdq::kLinNumBars + 4) * 8;
  const bool full_k = (K % svdq::kLinBK) == 0;
  auto kern = full_k ? svdq::linear_kernel<true> : svdq::linear_kernel<false>;
  if (svdq_status rc = ensure_smem(reinterpret_cast<const void*>(kern), dev, smem)) return rc;
  const int pairs = p.tiles < sms / 2 ? p.tiles : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(svdq::kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = add_overlap_attr(attr, 1);
  return launched(cudaLaunchKernelEx(&cfg, kern, tm_xc, tm_rc, tm_xs, tm_rs, tm_t, tm_l2, tm_y, p));
}
}  // namespace

svdq_status svdq_linear_scaled(const uint8_t* x_codes, const uint8_t* x_scales, const void* T,
                               const uint8_t* r_codes, const uint8_t* r_scales, const void* L2, const void* bias,
                               int64_t M, int64_t K, int64_t N, int64_t r, float alpha, void* Y, void* stream) {
  return guarded([&] {
    return linear_impl(x_codes, x_scales, T, r_codes, r_scales, L2, bias, M, K, N, r, alpha, Y, stream);
  });
}

// ------------------------------------------------------------- 8-bit layer --

svdq_status svdq_fp8_sizes(int64_t rows, int64_t K, size_t* codes_bytes, size_t* scales_bytes) {
  if (rows < 0 || K <= 0 || !codes_bytes || !scales_bytes) return SVDQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kMaxK || rows > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  *codes_bytes = static_cast<size_t>(rows) * static_cast<size_t>(K);
  *scales_bytes = static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>(svdq::fp8_band_tiles(K)) * 512;
  return SVDQ_OK;
}

svdq_status svdq_pack_weight_fp8(const void* W, int w_dtype, int64_t K, int64_t N, uint8_t* w_codes,
                                 uint8_t* w_scales, void* stream) {
  if (!W || !w_codes || !w_scales || K <= 0 || N <= 0 || (w_dtype != SVDQ_BF16 && w_dtype != SVDQ_F32))
    return SVDQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0 || K > kMaxK || N > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(W) || !aligned16(w_codes) || !aligned16(w_scales)) return SVDQ_ERR_MISALIGNED;
  const dim3 grid(static_cast<unsigned>((N + 127) / 128 * (128 / svdq::kPw8N)),
                  static_cast<unsigned>(4 * svdq::fp8_band_tiles(K)));
  return guarded([&] {
    if (w_dtype == SVDQ_BF16)
      return launch(svdq::pack_weight_fp8_kernel<__nv_bfloat16>, grid, svdq::kPw8Threads, 0, 1, stream,
                    static_cast<const __nv_bfloat16*>(W), static_cast<int>(K), static_cast<int>(N), w_codes, w_scales);
    return launch(svdq::pack_weight_fp8_kernel<float>, grid, svdq::kPw8Threads, 0, 1, stream,
                  static_cast<const float*>(W), static_cast<int>(K), static_cast<int>(N), w_codes, w_scales);
  });
}

svdq_status svdq_quantize_fp8(const void* X, int64_t ldx, int64_t M, int64_t K, int gelu, uint8_t* x_codes,
                              uint8_t* x_scales, void* stream) {
  if (!X || !x_codes || !x_scales || M <= 0 || K <= 0 || ldx < K || (gelu != 0 && gelu != 1))
    return SVDQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || ldx % 8 != 0 || M > kMaxRows || K > kMaxK) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(X) || !aligned16(x_codes) || !aligned16(x_scales)) return SVDQ_ERR_MISALIGNED;
  return guarded([&] {
    // Rows a warp: one while that gives at most 128 warps an SM, else 4.  On
    // B200 at K = 3072, one row against four, by warps an SM with one row: 4.2
    // and 4.9 us at 64 (with GELU 5.7 and 7.7), 5.4 and 5.6 at 96 (7.8 and 8.3),
    // 6.7 and 6.6 at 128 (10.1 and 11.1; 10.1 and 9.8 at K = 512), 11.5 and 10.5
    // at 256 (17.9 and 16.5), 21.2 and 19.1 at 512 (33.9 and 29.3).
    const int dev = current_device();
    if (dev < 0) return SVDQ_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SVDQ_ERR_CUDA;
    const int64_t segs = svdq::fp8_band_tiles(K);
    const int rows = M * segs <= 128 * static_cast<int64_t>(sms) ? 1 : 4;
    const int64_t warps = (M + rows - 1) / rows * segs;
    const dim3 grid(static_cast<unsigned>((warps + svdq::kQ8Threads / 32 - 1) / (svdq::kQ8Threads / 32) + 1));
    auto kern = rows == 1 ? (gelu ? svdq::quantize_fp8_kernel<1, true> : svdq::quantize_fp8_kernel<1, false>)
                          : (gelu ? svdq::quantize_fp8_kernel<4, true> : svdq::quantize_fp8_kernel<4, false>);
    return launch(kern, grid, svdq::kQ8Threads, 0, 1, stream, static_cast<const __nv_bfloat16*>(X), ldx,
                  static_cast<int>(M), static_cast<int>(K), aligned32(X) && ldx % 16 == 0, x_codes, x_scales);
  });
}

svdq_status svdq_rmsnorm(const void* X, int64_t ldx, const void* residual, int residual_dtype, const void* gamma,
                         float eps, int64_t M, int64_t K, void* residual_out, void* Y, uint8_t* x_codes,
                         uint8_t* x_scales, void* stream) {
  if (!X || M <= 0 || K <= 0 || ldx < K || !(eps >= 0.0f) || !std::isfinite(eps) ||
      (residual_dtype != SVDQ_BF16 && residual_dtype != SVDQ_F32))
    return SVDQ_ERR_INVALID_ARG;
  if (!residual != !residual_out || !x_codes != !x_scales || (!Y && !x_codes)) return SVDQ_ERR_INVALID_ARG;
  if (K % 16 != 0 || ldx % 8 != 0 || M > kMaxRows || K > kMaxNormK) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  for (const void* q : {X, residual, gamma, static_cast<const void*>(residual_out), static_cast<const void*>(Y),
                        static_cast<const void*>(x_codes), static_cast<const void*>(x_scales)})
    if (!aligned16(q)) return SVDQ_ERR_MISALIGNED;
  return guarded([&] {
    return residual_dtype == SVDQ_F32
               ? launch_rmsnorm<float>(X, ldx, residual, gamma, eps, M, K, residual_out, Y, x_codes, x_scales, stream)
               : launch_rmsnorm<__nv_bfloat16>(X, ldx, residual, gamma, eps, M, K, residual_out, Y, x_codes, x_scales,
                                               stream);
  });
}

svdq_status svdq_linear_fp8(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                            const uint8_t* w_scales, const void* bias, int64_t M, int64_t K, int64_t N, void* Y,
                            void* stream) {
  return guarded([&] {
    return linear_fp8_impl(x_codes, x_scales, w_codes, w_scales, bias, M, K, N, Y, nullptr, false, stream);
  });
}

svdq_status svdq_linear_fp8_gelu(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                                 const uint8_t* w_scales, const void* bias, int64_t M, int64_t K, int64_t N,
                                 uint8_t* y_codes, uint8_t* y_scales, void* stream) {
  return guarded([&] {
    return linear_fp8_impl(x_codes, x_scales, w_codes, w_scales, bias, M, K, N, y_codes, y_scales, true, stream);
  });
}

svdq_status svdq_attach_lora(const void* L1, const void* L2, const float* lambda, const void* A, const void* B,
                             int64_t K, int64_t N, int64_t r, int64_t ra, void* L1_out, void* L2_out, void* stream) {
  if (!lambda || !A || !B || !L1_out || !L2_out || K <= 0 || N <= 0 || r < 0 || ra <= 0)
    return SVDQ_ERR_INVALID_ARG;
  if (r > 0 && (!L1 || !L2)) return SVDQ_ERR_INVALID_ARG;
  if (r % 16 != 0 || ra % 16 != 0 || r + ra > 128 || N % 16 != 0 || K > kMaxK || N > kMaxRows)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if ((r > 0 && (!aligned16(L1) || !aligned16(L2))) || !aligned16(lambda) || !aligned16(A) || !aligned16(B) ||
      !aligned16(L1_out) || !aligned16(L2_out))
    return SVDQ_ERR_MISALIGNED;
  return guarded([&] {
    const int dev = current_device();
    if (dev < 0) return SVDQ_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SVDQ_ERR_CUDA;
    const int64_t chunks = K * ((r + ra) / 8) + (r + ra) * N / 8;
    int64_t blocks = (chunks + svdq::kLoraThreads - 1) / svdq::kLoraThreads;
    if (blocks > 8 * sms) blocks = 8 * sms;
    return launch_plain(svdq::attach_lora_kernel, dim3(static_cast<unsigned>(blocks)), svdq::kLoraThreads, stream,
                        static_cast<const __nv_bfloat16*>(L1), static_cast<const __nv_bfloat16*>(L2), lambda,
                        static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B),
                        static_cast<int>(K), static_cast<int>(N), static_cast<int>(r), static_cast<int>(ra),
                        static_cast<__nv_bfloat16*>(L1_out), static_cast<__nv_bfloat16*>(L2_out));
  });
}

svdq_status svdq_channel_absmax(const void* X, int64_t M, int64_t K, float* amax, void* stream) {
  if (!X || !amax || M <= 0 || K <= 0) return SVDQ_ERR_INVALID_ARG;
  if (K % 8 != 0 || K > kMaxK || M > kMaxRows) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(X) || !aligned16(amax)) return SVDQ_ERR_MISALIGNED;
  return guarded([&] {
    const int dev = current_device();
    if (dev < 0) return SVDQ_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SVDQ_ERR_CUDA;
    // enough row ranges for about four blocks per SM, at least 32 rows each
    const int64_t col_blocks = (K / 8 + svdq::kAbsmaxThreads - 1) / svdq::kAbsmaxThreads;
    int64_t row_blocks = (4 * static_cast<int64_t>(sms) + col_blocks - 1) / col_blocks;
    if (row_blocks > (M + 31) / 32) row_blocks = (M + 31) / 32;
    if (row_blocks > 65535) row_blocks = 65535;
    const int64_t rows_per_block = (M + row_blocks - 1) / row_blocks;
    row_blocks = (M + rows_per_block - 1) / rows_per_block;
    const dim3 grid(static_cast<unsigned>(col_blocks), static_cast<unsigned>(row_blocks));
    return launch_plain(svdq::channel_absmax_kernel, grid, svdq::kAbsmaxThreads, stream,
                        static_cast<const __nv_bfloat16*>(X), static_cast<int>(M), static_cast<int>(K),
                        static_cast<int>(rows_per_block), reinterpret_cast<unsigned int*>(amax));
  });
}

svdq_status svdq_sync_status(void* stream, int* where) {
  if (where) *where = 0;
  return guarded([&] {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SVDQ_ERR_CUDA;
    unsigned int code = 0, w = 0;
    if (cudaMemcpyFromSymbol(&code, svdq::g_status_code, sizeof(code)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&w, svdq::g_status_where, sizeof(w)) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    if (code != 0) {
      const unsigned int zero = 0;
      if (cudaMemcpyToSymbol(svdq::g_status_code, &zero, sizeof(zero)) != cudaSuccess ||
          cudaMemcpyToSymbol(svdq::g_status_where, &zero, sizeof(zero)) != cudaSuccess)
        return SVDQ_ERR_CUDA;
      if (where) *where = static_cast<int>(w);
      return static_cast<svdq_status>(code);
    }
    return SVDQ_OK;
  });
}

svdq_status svdq_set_wait_timeout(uint64_t timeout_ns) {
  if (timeout_ns == 0 || timeout_ns > 60000000000ull) return SVDQ_ERR_INVALID_ARG;
  g_timeout_ns.store(timeout_ns, std::memory_order_relaxed);
  return SVDQ_OK;
}

svdq_status svdq_set_linear_path(int path) {
  if (path < 0 || path > 2) return SVDQ_ERR_INVALID_ARG;
  g_linear_path.store(path, std::memory_order_relaxed);
  return SVDQ_OK;
}

svdq_status svdq_set_linear_fp8_path(int path) {
  if (path < 0 || path > 2) return SVDQ_ERR_INVALID_ARG;
  g_linear8_path.store(path, std::memory_order_relaxed);
  return SVDQ_OK;
}

svdq_status svdq_set_linear_fp8_splits(int splits) {
  if (splits < 0 || splits > svdq::kS8MaxSplits) return SVDQ_ERR_INVALID_ARG;
  g_linear8_splits.store(splits, std::memory_order_relaxed);
  return SVDQ_OK;
}

svdq_status svdq_set_launch_overlap(int enable) {
  if (enable != 0 && enable != 1) return SVDQ_ERR_INVALID_ARG;
  g_overlap.store(enable, std::memory_order_relaxed);
  return SVDQ_OK;
}

svdq_status svdq_selftest_wait_timeout(uint64_t timeout_ns, void* stream) {
  if (timeout_ns == 0 || timeout_ns > 10000000000ull) return SVDQ_ERR_INVALID_ARG;
  return guarded([&] { return launch_plain(svdq::wait_timeout_selftest_kernel, dim3(1), 32, stream, timeout_ns); });
}

// ------------------------------------------------ allocation-free variant --
// svdq_quantize_act with its scratch in a fixed array of this library instead
// of a caller's buffer, for callers that can neither allocate device memory
// nor pass scratch (see include/svdq.h).  Every device that loads the library
// holds the array until the process exits.
}  // extern "C"

namespace {

constexpr size_t kNoAllocScratchBytes = size_t(8) << 20;  // 8 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

std::mutex g_noalloc_mu;
void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the scratch array on `dev` (the current device), set up
// on the first call there: the array's host-side name is only a stand-in, so
// the address comes from cudaGetSymbolAddress with the device current, and the
// array is zero-filled once (the counters of the partial-sum exchange must
// start at zero; every call leaves them at zero again).
svdq_status noalloc_scratch(int dev, void** ptr) {
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return SVDQ_ERR_CUDA;
    if (cudaMemset(p, 0, kNoAllocScratchBytes) != cudaSuccess) return SVDQ_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *ptr = g_noalloc_ptr[dev];
  return SVDQ_OK;
}

}  // namespace

extern "C" {

svdq_status svdq_quantize_act_noalloc(const void* X, const float* inv_lambda, const void* L1, int64_t M, int64_t K,
                                      int64_t r, uint8_t* x_codes, uint8_t* x_scales, void* T, void* stream) {
  size_t need = 0;
  if (svdq_status rc = svdq_quantize_act_workspace(M, K, r, &need)) return rc;
  if (need > kNoAllocScratchBytes) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  void* scratch = nullptr;
  if (need > 0) {
    const svdq_status rc = guarded([&] {
      const int dev = current_device();
      return dev < 0 ? SVDQ_ERR_CUDA : noalloc_scratch(dev, &scratch);
    });
    if (rc) return rc;
  }
  return svdq_quantize_act(X, inv_lambda, L1, M, K, r, x_codes, x_scales, T, scratch, need ? kNoAllocScratchBytes : 0,
                           stream);
}

}  // extern "C"
