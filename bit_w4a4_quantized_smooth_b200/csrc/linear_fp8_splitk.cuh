// 8-bit linear in the FP8 block-128 format for sm_100a, few-rows path: the
// weights' bytes bound it, so every SM streams its share of them.
//
// The roles of the operands are swapped: the weight tile (128 output channels)
// is the MMA's M = 128 side and the tokens, padded to a multiple of 16 and at
// most 128, its N side, so one token costs an N = 16 MMA and 2 KB of shared
// memory a stage instead of a padded 128-row tile.  A CTA computes one 128 x
// Mt tile over a contiguous range of the 128-column K stages; the `splits`
// CTAs of a tile form a cluster along K.  192 threads: warp 0 TMA producer,
// warp 1 tensor-memory owner and MMA issuer, warps 2-5 epilogue.
// Partials meet in distributed shared memory: CTA j adds the tokens j, j +
// splits, ... of every CTA's partial in rank order, adds the bias and stores
// (bf16, or GELU and the FP8 block of the token's 128 channels, which is
// exactly one warp's row).  No global scratch, and the sum's order is fixed.
// On B200, weights from HBM: 1 x 3072 x 9216 takes 7.1 us in a stream of calls
// (28.3 MB, 4.0 TB/s) and 7.5 in a graph; in a graph 1 x 3072 x 3072 4.7, 16 x
// 3072 x 12288 with GELU 9.2, 128 x 3072 x 3072 7.9.
// About 3 us of each are launch, first loads, exchange and stores, during which
// the weights do not stream; a plain kernel that only loads 37.7 MB takes 8.5.
#pragma once

#include "fp8.cuh"

namespace svdq {

constexpr int kS8Threads = 192;
constexpr int kS8BN = 128;       // output channels per tile (MMA M)
constexpr int kS8MaxBM = 128;    // tokens per tile at most (MMA N)
constexpr int kS8BK = 128;
constexpr uint32_t kS8WBytes = 16384;
constexpr uint32_t kS8SfBytes = 1024;   // w and x scale tiles of 512 columns
constexpr int kS8MaxSplits = 8;
constexpr uint32_t kS8HeadBytes = 1024;
constexpr uint32_t kS8SmemLimit = 232448;  // 227 KB opt-in dynamic shared memory

__host__ __device__ constexpr uint32_t s8_stage_bytes(int bm) {
  return kS8WBytes + static_cast<uint32_t>(bm) * kS8BK + kS8SfBytes;
}

struct S8Params {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const __nv_bfloat16* bias;
  void* Y;             // bf16 [M][N], or codes [M][N]
  uint8_t* y_scales;
  int M, K, N;
  int bm;              // tokens per tile, a multiple of 16
  int splits;          // CTAs per tile (cluster size along K)
  int spc;             // stages per CTA
  int stages;          // ring depth
  uint32_t tmem_cols;  // accumulator [0, bm), scale regions in the last 32 columns
  uint64_t timeout_ns;
};

// Never launched: the host asks for this kernel's occupancy.
__global__ void __launch_bounds__(kS8Threads) linear_fp8_splitk_occupancy_kernel() {}

template <int n>
struct Int {
  static constexpr int value = n;
};

// MANY (2 to 4 splits, more than 64 tokens a tile): the sum takes two or four
// tokens at a time, so that eight remote loads of 16 bytes are in flight a
// lane whatever the number of partials (256 x 3072 x 3072 with GELU 13.0 ->
// 11.8 us on B200, 96 x 3072 x 9216 10.1 -> 9.6; at 48 tokens 9.1 -> 9.3).  A
// kernel of its own: with both loops in one, one token took 0.2 us more.
template <bool FP8_OUT, bool MANY>
__global__ void __launch_bounds__(kS8Threads)
    linear_fp8_splitk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                             const S8Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int S = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // [S] stage landed
  uint64_t* empty = full + S;                          // [S] the stage's MMAs and copies are done
  uint64_t* fin = empty + S;                           // every MMA of the CTA complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* ring = smem + kS8HeadBytes;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int split = blockIdx.x;
  const int n0 = blockIdx.y * kS8BN;
  const int m0 = blockIdx.z * kS8MaxBM;
  const int k_stages = (p.K + kS8BK - 1) / kS8BK;
  const int ks0 = split * p.spc;
  const int total = min(p.spc, k_stages - ks0);  // stages of this CTA (>= 1)
  const int64_t band_tiles = fp8_band_tiles(p.K);
  const uint32_t stage_bytes = s8_stage_bytes(p.bm);
  const uint32_t x_bytes = static_cast<uint32_t>(p.bm) * kS8BK;

  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(fin), 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();  // with the tensor memory held (see ptx.cuh)
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = smem_u32(ring);

  if (warp == 0) {
    // ---------------------------------------------------------- producer --
    // While the kernel ahead finishes: the w codes of the ring's first stages into L2.
    for (int it = 0; it < min(total, S); ++it) e_tma_prefetch_2d(&tm_w, (ks0 + it) * kS8BK, n0);
    const uint8_t* w_sf = p.w_scales + static_cast<size_t>(n0 >> 7) * band_tiles * 512;
    const uint8_t* x_sf = p.x_scales + static_cast<size_t>(m0 >> 7) * band_tiles * 512;
    griddep_wait();
    // The loops of both issuing warps are as short as they get: slot, phase and
    // addresses carried along, one election and one vote a stage.  With a
    // division by the ring depth, a look at the abort flag and an election for
    // each instruction, a 16 KB stage took 0.38 us on B200 whatever the depth
    // and whatever its bytes.
    int issued = 0;
    uint32_t s = 0, ph = 1, fb = smem_u32(full), eb = smem_u32(empty), w_s = sbase;
    bool ok = true;
    for (int ks = ks0; ks < ks0 + total; ++ks) {
      if (issued >= S && !warp_wait_ready(eb, ph, p.timeout_ns, 80)) {
        ok = false;
        break;
      }
      const bool sf = issued == 0 || (ks & 3) == 0;  // the scale tiles of a new group of 512 columns
      e_stage_load(fb, kS8WBytes + x_bytes + (sf ? kS8SfBytes : 0u), w_s, &tm_w, n0, w_s + kS8WBytes, &tm_x, m0,
                   ks * kS8BK);
      if (sf) {
        const uint32_t sf_s = w_s + kS8WBytes + x_bytes;
        e_bulk_load(sf_s, w_sf + static_cast<size_t>(ks >> 2) * 512, 512u, fb);
        e_bulk_load(sf_s + 512, x_sf + static_cast<size_t>(ks >> 2) * 512, 512u, fb);
      }
      ++issued;
      ++s;
      fb += 8;
      eb += 8;
      w_s += stage_bytes;
      if (s == static_cast<uint32_t>(S)) {
        s = 0;
        ph ^= 1u;
        fb = smem_u32(full);
        eb = smem_u32(empty);
        w_s = sbase;
        if (warp_flag(abort_flag)) break;
      }
    }
    if (!ok) *abort_flag = 1;
    // after an abort: this CTA's own copies land before it may exit
    if (warp_flag(abort_flag))
      for (int c = issued > S ? issued - S : 0; c < issued; ++c)
        warp_wait(smem_u32(&full[c % S]), (c / S) & 1, p.timeout_ns, 81);
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    griddep_wait();  // bounded waits start once the kernel ahead is done
    const uint32_t idesc =
        (1u << 23) | ((static_cast<uint32_t>(p.bm) >> 3) << 17) | (static_cast<uint32_t>(kS8BN >> 4) << 24);
    const uint32_t sf_col = tmem + p.tmem_cols - 32;
    const uint64_t w_d0 = make_sdesc(sbase, 16, 1024, 2);
    const uint64_t x_d0 = make_sdesc(sbase + kS8WBytes, 16, 1024, 2);
    const uint64_t sf_d0 = make_sdesc(sbase + kS8WBytes + x_bytes, 0, 128, 0);
    const uint32_t step = stage_bytes >> 4;  // descriptor units
    uint32_t s = 0, ph = 0, fb = smem_u32(full), eb = smem_u32(empty), at = 0;
    uint32_t sft = sf_col + 16;
    uint32_t more = 0;  // the first MMA starts the accumulator
    bool ok = true;
    for (int ks = ks0; ks < ks0 + total; ++ks) {
      ok = warp_wait_ready(fb, ph, p.timeout_ns, 82);
      if (!ok) break;
      tc_fence_after();
      const uint32_t j = static_cast<uint32_t>(ks) & 3u;
      if (ks == ks0 || j == 0) {
        sft ^= (sf_col ^ (sf_col + 16));
        e_tmem_cp_32x128b_warpx4(sft, sf_d0 + at);
        e_tmem_cp_32x128b_warpx4(sft + 8, sf_d0 + at + 32);
      }
      const uint32_t id = idesc | (j << 4) | (j << 29);
      e_stage_mxf8(tmem, w_d0 + at, x_d0 + at, id, sft, sft + 8, more, eb);
      more = 1;
      ++s;
      fb += 8;
      eb += 8;
      at += step;
      if (s == static_cast<uint32_t>(S)) {
        s = 0;
        ph ^= 1u;
        fb = smem_u32(full);
        eb = smem_u32(empty);
        at = 0;
        if (warp_flag(abort_flag)) break;
      }
    }
    if (!ok) *abort_flag = 1;
    // every MMA (also after an abort) completes before the accumulator is
    // read or the tensor memory released
    e_commit(smem_u32(fin));
    if (!warp_wait(smem_u32(fin), 0, p.timeout_ns, 83)) *abort_flag = 1;
  }

  // --------------------------------------------------------- epilogue --
  griddep_wait();   // the bias and Y may belong to the kernel ahead
  const int n = n0 + 4 * lane;
  uint2 bw = make_uint2(0, 0);  // this lane's four channels, long before they are needed
  if (p.bias && n < p.N) bw = *reinterpret_cast<const uint2*>(p.bias + n);  // N is a multiple of 8
  // [bm][128], over the ring: once the MMAs are complete every stage that was
  // loaded has been read.  (After an abort a copy may still land in it.  This
  // CTA then stores nothing; the others of its cluster, which learn nothing of
  // it, store sums with that part in them: outputs of a launch that records a
  // timeout are undefined.)
  float* part = reinterpret_cast<float*>(ring);
  const int vrows = min(p.bm, p.M - m0);  // tokens of this tile
  if (warp >= 2 && !warp_wait(smem_u32(fin), 0, p.timeout_ns, 84)) {
    *abort_flag = 1;
  } else if (warp >= 2) {
    tc_fence_after();
    const int q = warp & 3;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float* dst = part + 32 * q + lane;
    for (int cb = 0; cb < vrows; cb += 32) {  // bm is a multiple of 16
      uint32_t v[32];
      if (cb + 16 < p.bm) tmem_ld_32x32b_x32(src + cb, v);
      else tmem_ld_32x32b_x16(src + cb, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e) dst[(cb + e) * kS8BN] = __uint_as_float(v[e]);
      if (cb + 16 < p.bm) {
#pragma unroll
        for (int e = 16; e < 32; ++e) dst[(cb + e) * kS8BN] = __uint_as_float(v[e]);
      }
    }
  }
  // The tensor memory goes back before the CTAs meet.  Launches of other sizes
  // (other column counts) on another stream may share the SMs; a CTA that held
  // its columns while it waited for a CTA of its cluster, which in turn waited
  // for columns elsewhere, could close a circle.  Warp 1 frees them between its
  // arrival and its wait (all before the arrival: 0.1 to 0.4 us a call).
  tc_fence_before();
  if (p.splits > 1) {
    cluster_arrive();
    if (warp >= 2) named_bar_arrive(1, 160);  // this warp has read its lanes
    if (warp == 1) {
      named_bar_sync(1, 160);
      tc_fence_after();
      tmem_dealloc(tmem, p.tmem_cols);
    }
    cluster_wait();  // every CTA's partial is in its shared memory
  } else {
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
  }
  const bool aborted = *abort_flag != 0;
  const uint32_t part_u = smem_u32(part);
  // one token of the tile: its 128 channels, four a lane
  auto store = [&](int r, const float4& acc) {
    float v[4] = {acc.x + bf16_lo(bw.x), acc.y + bf16_hi(bw.x), acc.z + bf16_lo(bw.y), acc.w + bf16_hi(bw.y)};
    const int64_t m = m0 + r;
    if constexpr (FP8_OUT) {
      if (!aborted) store_gelu_fp8(v, static_cast<uint8_t*>(p.Y), p.y_scales, m, n, p.N, lane);
    } else if (!aborted && n < p.N) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.Y) + m * p.N + n) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  };
  if (!MANY && p.splits == 1) {
#pragma unroll 4
    for (int r = warp; r < vrows; r += kS8Threads / 32)
      store(r, *reinterpret_cast<const float4*>(part + r * kS8BN + 4 * lane));
  } else {
    if constexpr (!MANY) {
      for (int r = split + p.splits * warp; r < vrows; r += p.splits * (kS8Threads / 32)) {
        const uint32_t off = part_u + static_cast<uint32_t>((r * kS8BN + 4 * lane) * 4);
        float4 o[kS8MaxSplits];  // all loads in flight before the first addition
#pragma unroll
        for (int src = 0; src < kS8MaxSplits; ++src)
          o[src] = src < p.splits ? ld_dsmem_f32x4(map_shared_rank(off, static_cast<uint32_t>(src)))
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int src = 1; src < kS8MaxSplits; ++src) {  // rank order; + 0 behind the last rank
          o[0].x = __fadd_rn(o[0].x, o[src].x);
          o[0].y = __fadd_rn(o[0].y, o[src].y);
          o[0].z = __fadd_rn(o[0].z, o[src].z);
          o[0].w = __fadd_rn(o[0].w, o[src].w);
        }
        store(r, o[0]);
      }
    } else {
      auto sum = [&](auto tokens) {
        constexpr int T = decltype(tokens)::value, P = kS8MaxSplits / T;
        const int step = p.splits * (kS8Threads / 32);
        for (int r = split + p.splits * warp; r < vrows; r += T * step) {
          float4 o[T][P];
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const uint32_t off = part_u + static_cast<uint32_t>(((r + t * step) * kS8BN + 4 * lane) * 4);
#pragma unroll
            for (int src = 0; src < P; ++src)
              o[t][src] = src < p.splits && r + t * step < vrows
                              ? ld_dsmem_f32x4(map_shared_rank(off, static_cast<uint32_t>(src)))
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
#pragma unroll
          for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int src = 1; src < P; ++src) {  // rank order; + 0 behind the last rank
              o[t][0].x = __fadd_rn(o[t][0].x, o[t][src].x);
              o[t][0].y = __fadd_rn(o[t][0].y, o[t][src].y);
              o[t][0].z = __fadd_rn(o[t][0].z, o[t][src].z);
              o[t][0].w = __fadd_rn(o[t][0].w, o[t][src].w);
            }
            if (r + t * step < vrows) store(r + t * step, o[t][0]);
          }
        }
      };
      if (p.splits <= 2) sum(Int<4>{});
      else sum(Int<2>{});
    }
  }
  if constexpr (FP8_OUT) {
    if (split == 0 && !aborted) zero_tile_scales(p.y_scales, vrows, m0, n0, p.N, tid, kS8Threads);
  }
  if (p.splits > 1) cluster_sync();  // no CTA leaves while another still reads its partial
}

}  // namespace svdq
