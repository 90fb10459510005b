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
#pragma once

#include "fp8.cuh"

namespace svdq {

constexpr int kS8Threads = 192;
constexpr int kS8BN = 128;       // output channels per tile (MMA M)
constexpr int kS8MaxBM = 128;    // tokens per tile at most (MMA N)
constexpr int kS8BK = 128;
constexpr uint32_t kS8WBytes = 16384;
constexpr uint32_t kS8SfBytes = 1024;   // w and x scale tiles of 512 columns
constexpr int kS8MaxStages = 12;
constexpr int kS8MaxSplits = 8;
constexpr uint32_t kS8HeadBytes = 1024;

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

template <bool FP8_OUT>
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
    griddep_wait();
    int issued = 0;
    for (int it = 0; it < total; ++it) {
      const int s = it % S;
      if (it >= S && !warp_wait(smem_u32(&empty[s]), ((it / S) - 1) & 1, p.timeout_ns, 80)) {
        *abort_flag = 1;
        break;
      }
      if (warp_flag(abort_flag)) break;
      const uint32_t fb = smem_u32(&full[s]);
      const uint32_t w_s = sbase + s * stage_bytes;
      const int ks = ks0 + it;
      const bool sf = it == 0 || (ks & 3) == 0;  // the scale tiles of a new group of 512 columns
      e_arrive_expect_tx(fb, kS8WBytes + x_bytes + (sf ? kS8SfBytes : 0u));
      e_tma_load_2d(w_s, &tm_w, fb, ks * kS8BK, n0);
      e_tma_load_2d(w_s + kS8WBytes, &tm_x, fb, ks * kS8BK, m0);
      if (sf) {
        const uint32_t sf_s = w_s + kS8WBytes + x_bytes;
        e_bulk_load(sf_s, p.w_scales + (static_cast<size_t>(n0 >> 7) * band_tiles + (ks >> 2)) * 512, 512u, fb);
        e_bulk_load(sf_s + 512, p.x_scales + (static_cast<size_t>(m0 >> 7) * band_tiles + (ks >> 2)) * 512, 512u, fb);
      }
      ++issued;
    }
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
    uint32_t sg = 0;  // scale groups copied
    for (int it = 0; it < total; ++it) {
      const int s = it % S;
      const bool ok = !warp_flag(abort_flag) && warp_wait(smem_u32(&full[s]), (it / S) & 1, p.timeout_ns, 82);
      if (!ok) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t w_s = sbase + s * stage_bytes;
      const uint32_t x_s = w_s + kS8WBytes;
      const uint32_t j = static_cast<uint32_t>(ks0 + it) & 3u;
      if (it == 0 || j == 0) {
        const uint32_t sft = sf_col + 16 * (sg & 1);
        e_tmem_cp_32x128b_warpx4(sft, make_sdesc(x_s + x_bytes, 0, 128, 0));
        e_tmem_cp_32x128b_warpx4(sft + 8, make_sdesc(x_s + x_bytes + 512, 0, 128, 0));
        ++sg;
      }
      const uint32_t sft = sf_col + 16 * ((sg - 1) & 1);
      const uint32_t id = idesc | (j << 4) | (j << 29);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        e_mma_mxf8(tmem, make_sdesc(w_s + kk * 32, 16, 1024, 2), make_sdesc(x_s + kk * 32, 16, 1024, 2), id, sft,
                   sft + 8, (it > 0 || kk > 0) ? 1u : 0u);
      e_commit(smem_u32(&empty[s]));
    }
    // every MMA (also after an abort) completes before the accumulator is
    // read or the tensor memory released
    e_commit(smem_u32(fin));
    if (!warp_wait(smem_u32(fin), 0, p.timeout_ns, 83)) *abort_flag = 1;
  }

  // --------------------------------------------------------- epilogue --
  griddep_wait();   // the bias and Y may belong to the kernel ahead
  __syncthreads();  // every role is done: the ring is idle, the MMAs complete
  const bool aborted = *abort_flag != 0;
  float* part = reinterpret_cast<float*>(ring);  // [bm][128], over the idle ring
  const int vrows = min(p.bm, p.M - m0);         // tokens of this tile
  if (warp >= 2 && !aborted && warp_wait(smem_u32(fin), 0, p.timeout_ns, 84)) {
    tc_fence_after();
    const int q = warp & 3;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float* dst = part + 32 * q + lane;
    for (int cb = 0; cb < vrows; cb += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(src + cb, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e) dst[(cb + e) * kS8BN] = __uint_as_float(v[e]);
    }
  }
  if (p.splits > 1) cluster_sync();  // every CTA's partial is in its shared memory
  else __syncthreads();
  const uint32_t part_u = smem_u32(part);
  const int n = n0 + 4 * lane;
  float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.bias && n < p.N) {  // N is a multiple of 8
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = __bfloat162float(p.bias[n + e]);
  }
  for (int r = split + p.splits * warp; r < vrows; r += p.splits * (kS8Threads / 32)) {
    const uint32_t off = part_u + static_cast<uint32_t>((r * kS8BN + 4 * lane) * 4);
    float4 acc;
    if (p.splits == 1) {
      acc = *reinterpret_cast<const float4*>(part + r * kS8BN + 4 * lane);
    } else {
      acc = ld_dsmem_f32x4(map_shared_rank(off, 0));
      for (int src = 1; src < p.splits; ++src) {  // rank order
        const float4 o = ld_dsmem_f32x4(map_shared_rank(off, static_cast<uint32_t>(src)));
        acc.x = __fadd_rn(acc.x, o.x);
        acc.y = __fadd_rn(acc.y, o.y);
        acc.z = __fadd_rn(acc.z, o.z);
        acc.w = __fadd_rn(acc.w, o.w);
      }
    }
    float v[4] = {acc.x + b[0], acc.y + b[1], acc.z + b[2], acc.w + b[3]};
    const int64_t m = m0 + r;
    if constexpr (FP8_OUT) {
      gelu_n<4>(v);
      if (n >= p.N) v[0] = v[1] = v[2] = v[3] = 0.0f;
      float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t sb = fp8_scale_byte(a);
      const float inv = fp8_inv_scale(sb);
      if (!aborted) {
        if (n < p.N)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.Y) + m * p.N + n) =
              cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        if (lane == 0) p.y_scales[fp8_scale_offset(m, n0 >> 7, fp8_band_tiles(p.N))] = static_cast<uint8_t>(sb);
      }
    } else if (!aborted && n < p.N) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.Y) + m * p.N + n) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
  if constexpr (FP8_OUT) {
    // zero scales: this tile's block of the band's padding rows, and behind
    // the row's last block the rest of its word, for every row of the band
    if (split == 0 && !aborted) {
      const int64_t y_tiles = fp8_band_tiles(p.N);
      const int blk = n0 >> 7;
      for (int r = vrows + tid; r < 128; r += kS8Threads) p.y_scales[fp8_scale_offset(m0 + r, blk, y_tiles)] = 0;
      if (n0 + kS8BN >= p.N) {
        for (int z = blk + 1; z < 4 * y_tiles; ++z)
          for (int r = tid; r < 128; r += kS8Threads) p.y_scales[fp8_scale_offset(m0 + r, z, y_tiles)] = 0;
      }
    }
  }
  if (p.splits > 1) cluster_sync();  // no CTA leaves while another still reads its partial
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

}  // namespace svdq
