// 8-bit linear in the FP8 block-128 format for sm_100a, large-M path:
// Y = deq(x) deq(w)^T + bias as bf16, or GELU of it quantised to the next
// layer's FP8 input.  The tensor cores apply both power-of-two scales
// themselves (kind::mxf8f6f4, one UE8M0 scale per 32 along K: the byte of a
// 128-block serves its four 32-blocks), so a tile accumulates over all of K in
// tensor memory.
#pragma once

#include "fp8.cuh"

namespace svdq {

// Persistent CTA pairs (clusters of 2): grid = 2 x min(pair tiles, SMs / 2),
// 192 threads per CTA (320 with the FP8 output): warp 0 TMA producer, warp 1
// TMEM owner and (even CTA) MMA issuer, the others epilogue; the roles, the
// hand-offs and the abort drain are those of the 4-bit kernel (linear.cuh).
// Tensor-bound: 348 GFLOP at 4608 x 3072 x 12288 take 123 us on B200 in a short
// run of calls (2.82 PFLOP/s, 85 % of twice the measured bf16 rate; 131 with GELU
// and FP8 output) and 152 with GELU in a long one, where the power limit holds
// the clock near 1.5 GHz; 4608 x 12288 x 3072 119 and 137.
// A tile is 24 stages of 11.4 thousand cycles together; the change to the next
// (its last MMAs, one 64- or 128-column read of tensor memory, one arrival)
// adds 1.9 thousand, the epilogue's arithmetic hides under the next tile.
// A pair computes 256 x 256 output tiles; CTA c holds 128 of the tile's x rows
// and 128 of its w rows, the even CTA issues 2-SM MMAs (M = 256, N = 256, K =
// 32).  The tiles are visited in groups of `group` rows of tiles, M-fastest
// within a group, so that one operand stays in L2 (l8_group in svdq.cu).
// Ring: 5 stages of 128 columns of K per CTA (x codes and w codes, 128 rows x
// 128 bytes each, 128-byte swizzle; a sixth changed nothing: 125.9 against
// 125.0 us at 4608 x 3072 x 12288).  Every fourth stage of a tile also brings
// the scale tiles of its 512 columns (this CTA's x rows; all 256 w rows), and
// the MMA warp copies them into one of two scale regions of tensor memory
// with three tcgen05.cp per 512 columns; stage j of the four selects byte j of
// each scale word through the instruction descriptor.  (At one scale per 16
// the 4-bit kernel needs twelve copies per 256 columns, the largest single
// cost of its tensor pipe.)  The tensor pipe runs a thread's copies and MMAs
// in order, so the regions alternate without a barrier.
// Accumulators: two 128 x 256 fp32 tiles overlap in each CTA's TMEM as in the
// 4-bit kernel: columns [0, 256) and [192, 448), scales in [448, 480).
constexpr int kL8Threads = 192, kL8ThreadsFp8 = 320;
constexpr int kL8Stages = 5;
constexpr int kL8BM = 256, kL8BN = 256, kL8BK = 128;
constexpr uint32_t kL8ABytes = 16384, kL8BBytes = 16384;
constexpr uint32_t kL8StageBytes = kL8ABytes + kL8BBytes;
constexpr uint32_t kL8SfBytes = 512 + 1024;           // a stage's scale tiles
constexpr uint32_t kL8SfOffset = kL8Stages * kL8StageBytes;
constexpr uint32_t kL8BiasOffset = kL8SfOffset + kL8Stages * kL8SfBytes;
constexpr uint32_t kL8OutOffset = (kL8BiasOffset + 2048 + 1023) / 1024 * 1024;
constexpr uint32_t kL8OutBytes = 4096;                // 32 rows x 128 bytes of output
constexpr uint32_t kL8BarOffset = kL8OutOffset + 8 * kL8OutBytes;
constexpr int kL8NumBars = 2 * kL8Stages + 2 + 2 + 1 + 1 + 1;
constexpr uint32_t kL8TmemCols = 512;
constexpr uint32_t kL8Acc1Col = 192;
constexpr uint32_t kL8SfCol = 448;                    // region p: x scales at +16 p, w scales at +16 p + 8

struct L8Params {
  const __nv_bfloat16* bias;
  uint8_t* y_scales;   // FP8 output: scale tiles of the output rows
  int M, K, N;
  int m_tiles, tiles;  // pair tiles: ceil(M / 256) x ceil(N / 256)
  int group;           // rows of tiles per group of the visiting order
  int group_tiles;     // group x ceil(N / 256)
  int one;             // 1 (see the FP8 epilogue)
  uint64_t timeout_ns;
};

// FP8_OUT: GELU and FP8 block-128 output.  Two warpgroups of epilogue warps
// take one 128-column block of the tile each; a thread holds one row's whole
// block, so the block's scale needs no exchange.  Otherwise bf16, one
// warpgroup.  Both leave through staging blocks and TMA stores (16-byte stores
// straight from the registers cost 13 us of 161 at 4608 x 3072 x 12288 with
// FP8 output).  The bias of the next tile is loaded while this one is worked on.
template <bool FP8_OUT>
__global__ void __launch_bounds__(FP8_OUT ? kL8ThreadsFp8 : kL8Threads, 1)
    linear_fp8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
                      const __grid_constant__ CUtensorMap tm_y, const L8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  float* bias_s = reinterpret_cast<float*>(smem + kL8BiasOffset);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kL8BarOffset);
  uint64_t* full = bars;                          // [S] even CTA: both CTAs' stage landed
  uint64_t* empty = full + kL8Stages;             // [S] the stage's MMAs and copies are done
  uint64_t* acc_full = empty + kL8Stages;         // [2] tile accumulated (both CTAs)
  uint64_t* acc_empty = acc_full + 2;             // [2] even CTA: both CTAs' epilogue warps drained it
  uint64_t* ovl_free = acc_empty + 2;             // even CTA: shared columns drained
  uint64_t* fin = ovl_free + 1;                   // even CTA: every MMA complete
  uint64_t* odd_done = fin + 1;                   // even CTA: the odd producer published its count
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kL8NumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* odd_issued = tmem_slot + 2;  // even CTA: stages the odd producer issued

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();  // 0 = even CTA (MMA issuer)
  const int pair = blockIdx.x >> 1;
  const int pairs = gridDim.x >> 1;
  const int N = p.N;
  const int total = (p.K + kL8BK - 1) / kL8BK;    // stages per tile
  const int band_tiles = (p.K + 511) >> 9;        // scale tiles per 128-row band

  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kL8TmemCols);
    tmem_relinquish_pair();
  }
  if (tid == 0) {
    for (int s = 0; s < kL8Stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), FP8_OUT ? 16 : 8);
    }
    mbar_init(smem_u32(ovl_free), 8);
    mbar_init(smem_u32(fin), 1);
    mbar_init(smem_u32(odd_done), 1);
    *odd_issued = 0;
    *abort_flag = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the even CTA's barriers exist before anyone signals them
  tc_fence_after();
  griddep_launch_dependents();  // with the tensor memory held (see ptx.cuh)
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  auto lead = [&](const uint64_t* bar) { return map_shared_rank(smem_u32(bar), 0); };
  // first row and column of tile t < p.tiles
  auto tile_at = [&](int t, int& m, int& n) {
    const int g = t / p.group_tiles, in = t - g * p.group_tiles;
    const int rows = min(p.group, p.m_tiles - g * p.group);
    const int col = in / rows;
    m = (g * p.group + in - col * rows) * kL8BM;
    n = col * kL8BN;
  };
  // bytes one CTA loads for stage `it` of a tile
  auto stage_tx = [](int it) { return kL8StageBytes + ((it & 3) == 0 ? kL8SfBytes : 0u); };

  if (warp == 0) {
    // ------------------------------------------------------- producer --
    if (lane == 0) {
      prefetch_tmap(&tm_x);
      prefetch_tmap(&tm_w);
      prefetch_tmap(&tm_xs);
      prefetch_tmap(&tm_ws);
    }
    __syncwarp();
    // While the kernel ahead finishes: the w codes of the ring's first stages into L2.
    if (pair < p.tiles) {
      int m, n;
      tile_at(pair, m, n);
      const int nb = n + 128 * static_cast<int>(rank);
      for (int it = 0; it < min(total, kL8Stages); ++it) e_tma_prefetch_2d(&tm_w, it * kL8BK, nb);
    }
    const uint32_t lead_full = lead(full);
    griddep_wait();
    // Both issue loops carry slot, phase and addresses along: they share their
    // schedulers with the epilogue's warps, and a stage is 515 cycles of MMAs.
    uint32_t g = 0, s = 0, ph = 1;
    bool ok = true;
    for (int t = pair; t < p.tiles && ok && !warp_flag(abort_flag); t += pairs) {
      int m, n0;
      tile_at(t, m, n0);
      const int band = (m >> 7) + static_cast<int>(rank);  // this CTA's 128 rows
      const int nb = n0 + 128 * static_cast<int>(rank);
      const int x_st = band * band_tiles, w_st = (n0 >> 7) * band_tiles;
      for (int it = 0; it < total; ++it) {
        ok = warp_wait_ready(smem_u32(empty) + 8 * s, ph, p.timeout_ns, 60);
        if (!ok) {
          *abort_flag = 1;
          break;
        }
        const uint32_t fb = lead_full + 8 * s;
        const uint32_t a_s = sbase + s * kL8StageBytes;
        e_stage_load_pair(fb, rank ^ 1u, smem_u32(full) + 8 * s, 2 * stage_tx(it), a_s, &tm_x, band * 128,
                          a_s + kL8ABytes, &tm_w, nb, it * kL8BK);
        if ((it & 3) == 0) {
          // bands past the end of a tensor read zeros; their rows are never stored
          const uint32_t sf = sbase + kL8SfOffset + s * kL8SfBytes;
          const int st = it >> 2;
          e_tma_load_3d_pair(sf, &tm_xs, fb, 0, 0, x_st + st);
          e_tma_load_3d_pair(sf + 512, &tm_ws, fb, 0, 0, w_st + st);
          e_tma_load_3d_pair(sf + 1024, &tm_ws, fb, 0, 0, w_st + band_tiles + st);
        }
        ++g;
        if (++s == kL8Stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // After an abort: both producers' copies complete on the even CTA's full[]
    // barriers, which only the even producer arms; it makes every phase either
    // CTA may still have in flight completable and waits for it (linear.cuh).
    if (rank == 1) {
      if (lane == 0) {
        st_dsmem_u32(map_shared_rank(smem_u32(const_cast<uint32_t*>(odd_issued)), 0), g);
        mbar_arrive_cluster(lead(odd_done));
      }
      __syncwarp();
    } else if (warp_flag(abort_flag)) {
      const bool have = warp_wait_cluster(smem_u32(odd_done), 0, 2 * p.timeout_ns + 100000000ull, 67);
      const uint32_t g_odd = have ? __shfl_sync(0xffffffffu, *odd_issued, 0) : g;
      const uint32_t hi = g > g_odd ? g : g_odd;
      for (uint32_t j = hi > kL8Stages ? hi - kL8Stages : 0; j < hi; ++j) {
        const uint32_t s = j % kL8Stages;
        const uint32_t per_cta = stage_tx(static_cast<int>(j % static_cast<uint32_t>(total)));
        if (j >= g) e_arrive_expect_tx(smem_u32(&full[s]), per_cta);           // only the odd CTA issued it
        else if (j >= g_odd) e_mbar_complete_tx(smem_u32(&full[s]), per_cta);  // only this CTA issued it
        warp_wait(smem_u32(&full[s]), (j / kL8Stages) & 1, p.timeout_ns, 66);
      }
    }
  } else if (warp == 1) {
    griddep_wait();  // bounded waits start once the kernel ahead is done
    if (rank == 0) {
      // -------------------------------------------------- MMA issuer --
      // E4M3 x E4M3, UE8M0 scales; bits 4-5 and 29-30 select the scale bytes
      const uint32_t idesc = (1u << 23) | ((kL8BN >> 3) << 17) | ((kL8BM >> 4) << 24);
      const uint64_t a_d0 = make_sdesc(sbase, 16, 1024, 2);
      const uint64_t b_d0 = make_sdesc(sbase + kL8ABytes, 16, 1024, 2);
      const uint64_t sf_d0 = make_sdesc(sbase + kL8SfOffset, 0, 128, 0);
      uint32_t s = 0, ph = 0;
      uint32_t sft = tmem + kL8SfCol + 16;
      int i = 0;
      bool ok = true;
      for (int t = pair; t < p.tiles && ok && !warp_flag(abort_flag); t += pairs, ++i) {
        const int b = i & 1;
        const uint32_t acc = tmem + (b ? kL8Acc1Col : 0u);
        if (i >= 2) ok = warp_wait_cluster(smem_u32(&acc_empty[b]), ((i >> 1) - 1) & 1, p.timeout_ns, 61);
        if (ok && i >= 1) ok = warp_wait_cluster(smem_u32(ovl_free), (i - 1) & 1, p.timeout_ns, 62);
        if (!ok) break;
        tc_fence_after();
        uint32_t more = 0;  // the tile's first MMA starts the accumulator
        for (int it = 0; it < total; ++it) {
          ok = warp_wait_ready(smem_u32(full) + 8 * s, ph, p.timeout_ns, 63);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a_d = a_d0 + s * (kL8StageBytes >> 4);
          const uint64_t b_d = b_d0 + s * (kL8StageBytes >> 4);
          const uint32_t j = static_cast<uint32_t>(it) & 3u;
          if (j == 0) {
            const uint64_t sf_d = sf_d0 + s * (kL8SfBytes >> 4);
            sft ^= (tmem + kL8SfCol) ^ (tmem + kL8SfCol + 16);
            e_tmem_cp_pair_32x128b_warpx4(sft, sf_d);
            e_tmem_cp_pair_32x128b_warpx4(sft + 8, sf_d + 32);
            e_tmem_cp_pair_32x128b_warpx4(sft + 12, sf_d + 64);
          }
          const uint32_t id = idesc | (j << 4) | (j << 29);
          e_stage_mxf8_pair(acc, a_d, b_d, id, sft, sft + 8, more, smem_u32(empty) + 8 * s);
          more = 1;
          if (++s == kL8Stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        e_commit_pair_both(smem_u32(&acc_full[b]));
      }
      if (!ok) *abort_flag = 1;
      // own MMAs (which write both CTAs' tensor memory) complete before the
      // pair may release it
      e_commit_pair_both(smem_u32(fin));
      if (!warp_wait(smem_u32(fin), 0, p.timeout_ns, 65)) *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------- epilogue --
    griddep_wait();            // the bias and Y may belong to the kernel ahead
    const int wg = FP8_OUT ? (warp - 2) >> 2 : 0;  // FP8 output: the warpgroup's block of the tile
    const int q = warp & 3;    // TMEM lane quadrant this warp may access
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint8_t* out_s = smem + kL8OutOffset + (FP8_OUT ? warp - 2 : 2 * (warp - 2)) * kL8OutBytes;
    // bias columns of this thread: c0 (and c0 + 128 with one warpgroup)
    const int c0 = 128 * wg + ((tid - 64) & 127);
    auto bias_of = [&](int t, int c) {
      if (!p.bias || t >= p.tiles) return 0.0f;
      int m, n;
      tile_at(t, m, n);
      return n + c < N ? __bfloat162float(p.bias[n + c]) : 0.0f;
    };
    bias_s[c0] = bias_of(pair, c0);
    if constexpr (!FP8_OUT) bias_s[c0 + 128] = bias_of(pair, c0 + 128);
    int i = 0;
    for (int t = pair; t < p.tiles; t += pairs, ++i) {
      const int b = i & 1;
      int m0, n0;
      tile_at(t, m0, n0);
      m0 += 128 * static_cast<int>(rank);
      named_bar_sync(1 + wg, 128);  // this tile's bias is there, the one before is done with
      const float* bias_t = bias_s + kL8BN * b;
      const float next0 = bias_of(t + pairs, c0);
      const float next1 = FP8_OUT ? 0.0f : bias_of(t + pairs, c0 + 128);
      // no early exit: the warps of a group must keep meeting its named barrier
      const bool ok = !warp_flag(abort_flag) && warp_wait(smem_u32(&acc_full[b]), (i >> 1) & 1, p.timeout_ns, 70);
      if (!ok) {
        *abort_flag = 1;
        continue;
      }
      bias_s[kL8BN * (b ^ 1) + c0] = next0;
      if constexpr (!FP8_OUT) bias_s[kL8BN * (b ^ 1) + c0 + 128] = next1;
      tc_fence_after();
      const uint32_t acc_col = b ? kL8Acc1Col : 0u;
      if constexpr (FP8_OUT) {
        const uint32_t src = tmem + lane_base + acc_col + 128 * wg;
        float v[128];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld_32x32b_x32(src + 32 * j, reinterpret_cast<uint32_t*>(v) + 32 * j);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (wg != b) mbar_arrive_remote(lead(ovl_free));  // this block holds the 64 shared columns
          mbar_arrive_remote(lead(&acc_empty[b]));
        }
        const float* bs = bias_t + 128 * wg;
        const int nb = n0 + 128 * wg;
        const int valid = N - nb;  // columns of the block below N; the others have zero weights and bias, GELU(0) = 0
        const int m = m0 + 32 * q + lane;
        // Always taken, but the compiler does not know: in one straight line it
        // moves the arithmetic ahead of the arrivals above, and the next
        // tile's MMAs wait for it (157 against 135 us at 4608 x 3072 x 12288 on
        // B200).
        if (p.one) {
#pragma unroll
          for (int j = 0; j < 128; j += 4) {
            const float4 c = *reinterpret_cast<const float4*>(bs + j);
            add2_rn(v[j], v[j + 1], v[j], v[j + 1], c.x, c.y);
            add2_rn(v[j + 2], v[j + 3], v[j + 2], v[j + 3], c.z, c.w);
          }
          // a row without an x above 0.3 needs more care (fp8.cuh)
          const float hi = max_n<128>(v);
          const bool careful = m < p.M && !(hi > kGeluPos);
          float top[2] = {hi, 0.0f};
          gelu_fast<2, false>(top);
          float amax = top[0];
          if (!__any_sync(0xffffffffu, careful)) {
#pragma unroll
            for (int j = 0; j < 128; j += 16) gelu_fast<16, false>(v + j);
          } else {
#pragma unroll
            for (int j = 0; j < 128; j += 16) {
              float x[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = v[j + e];
              gelu_fast<16, false>(v + j);
              if (careful) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (x[e] < -kGeluFast) v[j + e] = gelu_tail(x[e]);
              }
            }
            if (careful) amax = amax_n<128>(v);
          }
          const uint32_t sb = fp8_scale_byte(amax);
          const float inv = fp8_inv_scale(sb);
          if (lane == 0) bulk_wait_group_read<0>();  // this warp's previous store has read the block
          __syncwarp();
          uint8_t* rowp = out_s + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 16-byte chunk j = columns 16 j .. 16 j + 15
            *reinterpret_cast<uint4*>(rowp + ((j ^ (lane & 7)) << 4)) = codes16(v + 16 * j, inv);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && valid > 0 && m0 + 32 * q < p.M) {
            tma_store_2d(&tm_y, smem_u32(out_s), nb, m0 + 32 * q);
            bulk_commit_group();
          }
          // the block's scale byte; the last tile's second block also writes the
          // rest of the row's last word.  Padding rows of the last 128-row band
          // get zeros.
          if (m0 < p.M) {
            uint8_t* dst = p.y_scales + fp8_scale_offset(m, nb >> 7, fp8_band_tiles(N));
            *dst = m < p.M ? static_cast<uint8_t>(sb) : uint8_t{0};
            if (wg == 1 && ((n0 >> 8) & 1) == 0 && n0 + kL8BN >= N) *reinterpret_cast<uint16_t*>(dst + 1) = 0;
          }
        }
      } else {
#pragma unroll 1
        for (int gi = 0; gi < 4; ++gi) {
          // 64-column groups; the 64 shared columns ([192, 256)) come first
          const int g0 = b ? 2 * gi : ((6 + 2 * gi) & 7);  // first 32-column chunk
          uint32_t v[64];
          tmem_ld_32x32b_x32(tmem + lane_base + acc_col + 32 * g0, v);
          tmem_ld_32x32b_x32(tmem + lane_base + acc_col + 32 * g0 + 32, v + 32);
          tmem_ld_wait();
          if (gi == 0 || gi == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(lead(gi == 0 ? ovl_free : &acc_empty[b]));
          }
          // the staging block (alternating per group) must no longer be read
          // by this warp's last store but one
          uint8_t* blk = out_s + (gi & 1) * kL8OutBytes;
          uint8_t* rowp = blk + lane * 128;
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
          const float* bs = bias_t + 32 * g0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // 16-byte chunk j = columns 8 j .. 8 j + 7
            auto y = [&](int e) { return __uint_as_float(v[8 * j + e]) + bs[8 * j + e]; };
            *reinterpret_cast<uint4*>(rowp + ((j ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(y(0), y(1)), pack_bf16x2(y(2), y(3)), pack_bf16x2(y(4), y(5)),
                           pack_bf16x2(y(6), y(7)));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (n0 + 32 * g0 < N && m0 + 32 * q < p.M) tma_store_2d(&tm_y, smem_u32(blk), n0 + 32 * g0, m0 + 32 * q);
            bulk_commit_group();  // an empty one too: the wait above counts one per 64 columns
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();  // stores complete before the CTA exits
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs are complete before either CTA frees TMEM
  if (warp == 1) tmem_dealloc_pair(tmem, kL8TmemCols);
}

}  // namespace svdq
