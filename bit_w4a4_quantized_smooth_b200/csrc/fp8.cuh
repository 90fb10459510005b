// The 8-bit format beside the 4-bit layer ("FP8 block-128"): E4M3 codes with
// one power-of-two scale (E8M0, byte b = 2^(b - 127)) per 128 consecutive
// elements along K, and the pieces its kernels share.
//
// A block of values v with amax = max |v_i| takes the smallest scale 2^e,
// e >= -127, with amax <= 448 2^e, and the codes E4M3_RNE(v_i 2^-e).  A power
// of two costs no precision (the scaling is exact, and E4M3's own exponent
// absorbs up to one bit of headroom), never saturates, and is what the tensor
// cores multiply in by themselves: with an fp32 scale per block every 128 of K
// would have to leave tensor memory to be scaled on the CUDA cores.
#pragma once

#include "common.cuh"
#include "ptx_fp8.cuh"

namespace svdq {

constexpr int kFp8Block = 128;

// 512-byte scale tiles (128 rows x 4 blocks) per 128-row band.
__host__ __device__ __forceinline__ int64_t fp8_band_tiles(int64_t K) { return (K + 511) >> 9; }

// Byte offset of the scale of (row, block) in the tile layout; the four
// blocks 4 j .. 4 j + 3 of a row are consecutive.
__device__ __forceinline__ size_t fp8_scale_offset(int64_t row, int blk, int64_t band_tiles) {
  return (static_cast<size_t>(row >> 7) * static_cast<size_t>(band_tiles) + (blk >> 2)) * 512 +
         (static_cast<size_t>(row) & 31) * 16 + ((static_cast<size_t>(row) & 127) >> 5) * 4 + (blk & 3);
}

// The scale byte of a block.  amax = 2^(E - 127) (1 + f) needs
// e = E - 127 - 8 (448 = 1.75 2^8), one more when f > 0.75: adding 2^21 - 1 to
// the bits carries into the exponent exactly then.  Zero and tiny blocks clamp
// at b = 0; infinity gives b = 247.
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
  const int b = static_cast<int>((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(max(b, 0));
}

// 2^-e for a scale byte in [0, 247]: always a normal fp32 number.
__device__ __forceinline__ float fp8_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Four fp32 values -> four E4M3 codes, element i in byte i (round to nearest
// even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}

// Packed fp32 pairs (one instruction for both halves).
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Results below 2^-126 become 0: three instructions fewer.
__device__ __forceinline__ float ex2_approx_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------- GELU ----
// GELU(x) = x Phi(x) = max(x, 0) - |x| Phi(-|x|), which has no cancellation
// for negative x: within 2^-18 relative, also where the result is small (each
// value keeps its own E4M3 exponent, so an error against the block's largest
// value would not do).
//
// The fast form, |x| <= 5.5: Phi(-z) = 2^g(z) with g = log2 Phi(-z) as a
// polynomial of degree 10 in -z: one exponential an element, no division (a
// form with a reciprocal and a degree-7 polynomial needs two of the 16-lane
// special-function operations an element: 25 us of them alone at 4608 x
// 12288).  The coefficients are this project's own fit: minimax in g
// (reweighted least squares on Chebyshev nodes, |error| 1.3e-7 in ln Phi),
// rounded to fp32.
// Beyond 5.5 it clamps z.  For x > 5.5 that is right to the last bit; with
// TIES (inputs that are bf16, and so often E4M3 ties themselves) the last step
// rounds toward zero, because the exact result lies below x by less than half
// an ulp and rounding up to x would turn the tie the wrong way.  For x < -5.5
// it gives -1.05e-7 for a result between that and 0: in a block whose largest
// result is 0.1 or more both get the code -0 (half the smallest step is 2^-10
// 2^-12 = 2.4e-7), so gelu_tail is needed only in a block without any x above
// 0.3 (GELU(0.3) = 0.185).  Where there is one, it also has the block's
// largest magnitude: negative results end at -0.17.
constexpr float kGeluFast = 5.5f;
constexpr float kGeluPos = 0.3f, kGeluPosResult = 0.18f;  // GELU(0.3) = 0.1854

__device__ __forceinline__ uint64_t fma_rz_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// n values (n even), coefficient by coefficient: the n / 2 chains of packed
// operations are independent, and a coefficient's register pair is set once
// for all of them.
template <int n, bool TIES>
__device__ __forceinline__ void gelu_fast(float* x) {
  constexpr float c[11] = {-0.9999998211860657f,    1.1511125564575195f,    -0.4591609537601471f,
                           0.05260409042239189f,    0.007166661322116852f,  0.00016647009761072695f,
                           -0.0002045672881649807f, -5.589646752923727e-05f, -7.6225755947234575e-06f,
                           -5.619402827505837e-07f, -1.7772931570902983e-08f};
  uint64_t nz[n / 2], g[n / 2];
#pragma unroll
  for (int i = 0; i < n / 2; ++i)
    nz[i] = pack_f32x2(max_nan(-fabsf(x[2 * i]), -kGeluFast), max_nan(-fabsf(x[2 * i + 1]), -kGeluFast));
  {
    const uint64_t a = pack_f32x2(c[10], c[10]), b = pack_f32x2(c[9], c[9]);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) g[i] = fma_f32x2(a, nz[i], b);
  }
#pragma unroll
  for (int k = 8; k >= 0; --k) {
    const uint64_t b = pack_f32x2(c[k], c[k]);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) g[i] = fma_f32x2(g[i], nz[i], b);
  }
#pragma unroll
  for (int i = 0; i < n / 2; ++i) {
    float g0, g1;
    unpack_f32x2(g[i], g0, g1);
    const uint64_t phi = pack_f32x2(ex2_approx_ftz(g0), ex2_approx_ftz(g1));
    const uint64_t pos = pack_f32x2(fmaxf(x[2 * i], 0.0f), fmaxf(x[2 * i + 1], 0.0f));
    unpack_f32x2(TIES ? fma_rz_f32x2(nz[i], phi, pos) : fma_f32x2(nz[i], phi, pos), x[2 * i], x[2 * i + 1]);
  }
}

// x < -5.5: Phi(-z) = 2^(-z^2 log2(e) / 2) t P(t), t = 1 / (1 + 0.3 z), P of
// degree 7 fitted the same way to 0.5 erfcx(z / sqrt 2) / t with relative
// error 1.3e-7 up to z = 13.5; beyond, the result leaves fp32's normal range.
// The exponent reaches 131, where one rounding is worth 2.6e-6 of the result,
// so it is carried as a sum of two parts.
__device__ __forceinline__ float gelu_tail(float x) {
  constexpr float c_hi = 0.72134751081466675f, c_lo = 9.6298140e-9f;  // log2(e) / 2
  const float z = fminf(-x, 30.0f);
  const float sq = __fmul_rn(z, z);
  const float e = __fmul_rn(sq, c_hi);
  const float lo = __fmaf_rn(sq, c_hi, -e) + __fmaf_rn(__fmaf_rn(z, z, -sq), c_hi, sq * c_lo);
  const float t = rcp_approx(__fmaf_rn(z, 0.3f, 1.0f));
  float q = 0.03593172878026962f;
  q = __fmaf_rn(q, t, -0.15827596187591553f);
  q = __fmaf_rn(q, t, 0.20820654928684235f);
  q = __fmaf_rn(q, t, -0.055393803864717484f);
  q = __fmaf_rn(q, t, 0.12946918606758118f);
  q = __fmaf_rn(q, t, 0.09963750094175339f);
  q = __fmaf_rn(q, t, 0.12079835683107376f);
  q = __fmaf_rn(q, t, 0.11962638795375824f);
  q = __fmul_rn(q, __fmaf_rn(t, -0.69314718f * lo, t));  // 2^-lo to first order
  return __fmul_rz(-z, __fmul_rn(q, ex2_approx(-e)));
}

template <int n>
__device__ __forceinline__ float amax_n(const float* v) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < n; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}

// The largest of n values (n even), NaN ignored.
template <int n>
__device__ __forceinline__ float max_n(const float* v) {
  float a = fmaxf(v[0], v[1]);
#pragma unroll
  for (int i = 2; i < n; i += 2) a = max3(a, v[i], v[i + 1]);
  return a;
}

// GELU of this lane's n values (n even) of a block spread over `lanes`
// neighbouring lanes, and the block's largest magnitude.  All lanes call it.
template <int n, int lanes, bool TIES>
__device__ __forceinline__ float gelu_block(float* v) {
  float x[n];
#pragma unroll
  for (int i = 0; i < n; ++i) x[i] = v[i];
  gelu_fast<n, TIES>(v);
  float a = max_n<n>(v);
#pragma unroll
  for (int o = lanes / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const bool careful = !(a > kGeluPosResult);
  if (__any_sync(0xffffffffu, careful)) {
    if (careful) {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (x[i] < -kGeluFast) v[i] = gelu_tail(x[i]);
    }
    a = amax_n<n>(v);
#pragma unroll
    for (int o = lanes / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  }
  return a;
}

// ------------------------------------------------------------- elements ----
// 32 bytes of one thread: one access where the address allows it (`wide`, the
// same for the whole launch), else two of 16.
__device__ __forceinline__ void load32(const void* p, uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
// The same for data that is read once: not kept in L1, first to leave L2.
__device__ __forceinline__ void load32_stream(const void* p, uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    load32(p, w, false);
  }
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Eight consecutive elements of a row.
__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  v[0] = bf16_lo(w.x);
  v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y);
  v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z);
  v[5] = bf16_hi(w.z);
  v[6] = bf16_lo(w.w);
  v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x;
  v[1] = a.y;
  v[2] = a.z;
  v[3] = a.w;
  v[4] = b.x;
  v[5] = b.y;
  v[6] = b.z;
  v[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  float a, b, c, d;
  mul2_rn(a, b, v[0], v[1], inv, inv);
  mul2_rn(c, d, v[2], v[3], inv, inv);
  return cvt_e4m3x4(a, b, c, d);
}
__device__ __forceinline__ uint2 codes8(const float* v, float inv) {
  return make_uint2(codes4(v, inv), codes4(v + 4, inv));
}
__device__ __forceinline__ uint4 codes16(const float* v, float inv) {
  return make_uint4(codes4(v, inv), codes4(v + 4, inv), codes4(v + 8, inv), codes4(v + 12, inv));
}
// Zero scales of the padding rows [M, ceil(M / 128) 128): a word of four
// blocks at a time, by `threads` threads.
__device__ __forceinline__ void zero_pad_scales(uint8_t* scales, int64_t M, int64_t band_tiles, int tid, int threads) {
  const int64_t pad = ((M + 127) & ~int64_t(127)) - M;
  for (int64_t i = tid; i < pad * band_tiles; i += threads)
    *reinterpret_cast<uint32_t*>(scales + fp8_scale_offset(M + i / band_tiles, static_cast<int>(i % band_tiles) * 4,
                                                           band_tiles)) = 0;
}

// GELU of a token's 128 channels, four per lane of a warp (channel n = this
// lane's first), as one FP8 block; channels past N count as zeros and are not
// written.
__device__ __forceinline__ void store_gelu_fp8(float* v, uint8_t* codes, uint8_t* scales, int64_t m, int n, int N,
                                               int lane) {
  if (n >= N) v[0] = v[1] = v[2] = v[3] = 0.0f;  // GELU(0) = 0
  const float a = gelu_block<4, 32, false>(v);
  const uint32_t b = fp8_scale_byte(a);
  const float inv = fp8_inv_scale(b);
  if (n < N)
    *reinterpret_cast<uint32_t*>(codes + m * N + n) = codes4(v, inv);
  if (lane == 0) scales[fp8_scale_offset(m, n >> 7, fp8_band_tiles(N))] = static_cast<uint8_t>(b);
}

// Zero scales that the tile of channels [n0, n0 + 128) of the band's rows [m0,
// m0 + 128) owns: its block of the rows from `rows` on (padding), and, for the
// last tile, the blocks behind it in the band's last words.
__device__ __forceinline__ void zero_tile_scales(uint8_t* scales, int rows, int64_t m0, int n0, int N, int tid,
                                                 int threads) {
  const int64_t tiles = fp8_band_tiles(N);
  const int blk = n0 >> 7;
  for (int r = rows + tid; r < 128; r += threads) scales[fp8_scale_offset(m0 + r, blk, tiles)] = 0;
  if (n0 + 128 >= N)
    for (int z = blk + 1; z < 4 * tiles; ++z)
      for (int r = tid; r < 128; r += threads) scales[fp8_scale_offset(m0 + r, z, tiles)] = 0;
}

// ============================================================ quantiser ====
// x codes and scales of X (or GELU(X)), bf16 [M][K] with row stride ldx.
// HBM-bound: 2 + 1 bytes an element.  A warp takes 512 columns (one scale
// tile's four blocks) of R consecutive rows: a lane holds 16 columns of each
// row (32 bytes a row, all R rows' in flight before the first is used: 128
// bytes a thread at R = 4), 8 lanes a block; a row's four scale
// bytes leave as one word.  On B200 4608 x 12288 of 21504 columns take 23.3 us
// (170 MB, of which the codes largely stay in L2), with GELU 40.3: there a
// warp's loads and its polynomial alternate (arithmetic pipes 57 and 54 % busy,
// issue 67 %).  64 x 15360 take 4.3 us a call, which is the host's pace (3.0 in
// a graph).  (A first version with 8
// columns a lane, 4 rows and single scale bytes took 43.1 us, 59.4 with GELU:
// half the loads in flight, and 2.7 us for the byte stores.)
// The grid's last block zeroes the padding rows' scales.
constexpr int kQ8Threads = 128;

template <int R, bool GELU>
__global__ void __launch_bounds__(kQ8Threads)
    quantize_fp8_kernel(const __nv_bfloat16* __restrict__ X, int64_t ldx, int M, int K, bool wide,
                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int band_tiles = static_cast<int>(fp8_band_tiles(K));
  if (blockIdx.x == gridDim.x - 1) {
    zero_pad_scales(scales, M, band_tiles, threadIdx.x, kQ8Threads);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * (kQ8Threads / 32) + (threadIdx.x >> 5);  // 512-column segment, fastest along the row
  const int seg = w % band_tiles;
  const int row0 = (w / band_tiles) * R;
  if (row0 >= M) return;  // whole warps
  const int col = 512 * seg + 16 * lane;
  const bool in = col < K;  // K is a multiple of 16
  uint32_t raw[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (in && row0 + i < M) {
      load32_stream(X + (row0 + i) * ldx + col, raw[i], wide);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) raw[i][e] = 0;
    }
  }
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[2 * e] = bf16_lo(raw[i][e]);
      v[2 * e + 1] = bf16_hi(raw[i][e]);
    }
    float a;
    if constexpr (GELU) {
      a = gelu_block<16, 8, true>(v);
    } else {
      a = amax_n<16>(v);
#pragma unroll
      for (int o = 4; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    const uint32_t b = fp8_scale_byte(a);
    if (in && row0 + i < M)
      *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(row0 + i) * K + col) = codes16(v, fp8_inv_scale(b));
    uint32_t t = b << (lane & 24);  // the row's four bytes, in every lane
    t |= __shfl_xor_sync(0xffffffffu, t, 8);
    t |= __shfl_xor_sync(0xffffffffu, t, 16);
    if (lane == i) word = t;
  }
  if (lane < R && row0 + lane < M)
    *reinterpret_cast<uint32_t*>(scales + fp8_scale_offset(row0 + lane, 4 * seg, band_tiles)) = word;
}

// ============================================================ RMS norm ====
// h = X + residual (stored back), y = h / sqrt(mean(h^2) + eps) * gamma,
// written as FP8 block-128 and / or as bf16, from one read of X and the
// residual.  The norm is taken of the stored h (rounded to the residual's
// type), so the result is the same whether or not the addition is fused.
// HBM-bound: 7 bytes an element with a bf16 residual and FP8 output.
//
// A warp takes 512 columns (16 a lane, 8 lanes a block) of one row at a time,
// S such segments in registers (h as packed bf16 where that is its type);
// `wpr` warps share a row.  On B200 4608 x 3072 take 19.4 us (99 MB: 5.1 TB/s,
// 78 % of a copy; issue 62 %, and a row's outputs wait for all of its inputs),
// 333 x 8208 with an fp32 residual 7.5 us, one row 2.2 us of the GPU and 4.5 a
// call, which is the host's pace.  (A first version, one CTA a row and 8 columns
// a thread, spent 37 instructions an element, mostly on reductions: 23.5 us at
// 4608 x 3072.)
//
// Rounding.  1 / sqrt(...) is carried as a sum of two fp32 numbers, h gamma is
// exact (two 8-bit significands; with an fp32 residual its error is carried
// along), and y = h gamma (r_hi + r_lo) is one fused operation rounded toward
// zero with its last bit set to mark what was cut off.  Given r, the product is
// then rounded once, to E4M3 or bf16: an fp32 product rounded to nearest would
// land on an E4M3 tie for one value in a million and turn half of those the
// wrong way.  r itself carries half the relative error of the fp32 sum of
// squares (tens of 2^-24 at the most); its second word keeps the root and the
// division from adding to that.
constexpr int kNormMaxThreads = 512;

// 1 / sqrt(sum / K + eps) as hi + lo.  lo is 0 where hi^2 leaves fp32's range:
// below 2.9e-39 (s has 22 bits or fewer there), at zero and at infinity.
__device__ __forceinline__ void norm_rstd(float sum, float K, float eps, float& hi, float& lo) {
  const float q = __fdiv_rn(sum, K);
  const float q_lo = __fmaf_rn(-q, K, sum) * rcp_approx(K);
  const float s = __fadd_rn(q, eps);
  const float bb = __fsub_rn(s, q);
  const float s_lo = __fadd_rn(__fadd_rn(__fsub_rn(q, __fsub_rn(s, bb)), __fsub_rn(eps, bb)), q_lo);
  hi = __frsqrt_rn(s);
  const float p = __fmul_rn(hi, hi);
  float e = __fmaf_rn(-s, p, 1.0f);
  e = __fmaf_rn(-s, __fmaf_rn(hi, hi, -p), e);
  e = __fmaf_rn(-s_lo, p, e);
  lo = p > 0.0f && p <= 3.402823466e38f ? __fmul_rn(__fmul_rn(0.5f, hi), e) : 0.0f;
}

template <int S, typename RES>
__global__ void __launch_bounds__(kNormMaxThreads)
    rmsnorm_kernel(const __nv_bfloat16* X, int64_t ldx, const RES* residual, const __nv_bfloat16* __restrict__ gamma,
                   float eps, int M, int K, int wpr, bool wide, RES* residual_out, __nv_bfloat16* Y, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales) {
  constexpr bool kBf16 = sizeof(RES) == 2;
  __shared__ float part[kNormMaxThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int band_tiles = static_cast<int>(fp8_band_tiles(K));
  if (blockIdx.x == gridDim.x - 1) {
    if (scales) zero_pad_scales(scales, M, band_tiles, threadIdx.x, blockDim.x);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpc = (blockDim.x >> 5) / wpr;  // rows per CTA: more than one only with one warp a row
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rpc + warp / wpr;
  const int seg0 = warp % wpr;
  if (row >= M) return;  // whole warps, and whole CTAs where they meet at a barrier

  // h: packed bf16 pairs, or fp32
  uint32_t hb[kBf16 ? S : 1][8];
  float hf[kBf16 ? 1 : S][16];
  {
    uint32_t x[S][8], r[S][kBf16 ? 8 : 16];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int col = 512 * (seg0 + j * wpr) + 16 * lane;
      if (col < K) {
        load32(X + row * ldx + col, x[j], wide);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = 0;
      }
      if (col < K && residual) {
        load32(residual + row * K + col, r[j], wide);
        if constexpr (!kBf16) load32(residual + row * K + col + 8, r[j] + 8, wide);
      } else {
#pragma unroll
        for (int i = 0; i < (kBf16 ? 8 : 16); ++i) r[j][i] = 0;
      }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int col = 512 * (seg0 + j * wpr) + 16 * lane;
      const bool store = col < K && residual;
      if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          hb[j][i] = residual ? pack_bf16x2(bf16_lo(x[j][i]) + bf16_lo(r[j][i]), bf16_hi(x[j][i]) + bf16_hi(r[j][i]))
                              : x[j][i];
        if (store) store32(residual_out + row * K + col, hb[j], wide);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          hf[j][2 * i] = bf16_lo(x[j][i]) + __uint_as_float(r[j][2 * i]);
          hf[j][2 * i + 1] = bf16_hi(x[j][i]) + __uint_as_float(r[j][2 * i + 1]);
        }
        if (store) {
          store32(residual_out + row * K + col, reinterpret_cast<const uint32_t*>(hf[j]), wide);
          store32(residual_out + row * K + col + 8, reinterpret_cast<const uint32_t*>(hf[j]) + 8, wide);
        }
      }
    }
  }
  auto value = [&](int j, int i, float& a, float& b) {  // elements 2 i, 2 i + 1 of segment j
    if constexpr (kBf16) {
      a = bf16_lo(hb[j][i]);
      b = bf16_hi(hb[j][i]);
    } else {
      a = hf[j][2 * i];
      b = hf[j][2 * i + 1];
    }
  };
  uint64_t ss[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      value(j, i, a, b);
      const uint64_t h2 = pack_f32x2(a, b);
      ss[i & 1] = fma_f32x2(h2, h2, ss[i & 1]);
    }
  float s0, s1, s2, s3;
  unpack_f32x2(ss[0], s0, s1);
  unpack_f32x2(ss[1], s2, s3);
  float sum = (s0 + s1) + (s2 + s3);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (wpr > 1) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = lane < wpr ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  float r_hi, r_lo;
  norm_rstd(sum, static_cast<float>(K), eps, r_hi, r_lo);
  // a product of h gamma and a short r_hi alone is exact and must stay so
  const uint32_t cut = (r_lo != 0.0f || (__float_as_uint(r_hi) & 0xFFFFu) != 0) ? 1u : 0u;
  const uint64_t rh2 = pack_f32x2(r_hi, r_hi), rl2 = pack_f32x2(r_lo, r_lo);

  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int seg = seg0 + j * wpr;
    const int col = 512 * seg + 16 * lane;
    const bool in = col < K;
    uint32_t gw[8];
    if (gamma && in) {
      load32(gamma + col, gw, wide);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) gw[i] = 0x3F803F80u;  // ones
    }
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b, ta, tb;
      value(j, i, a, b);
      const float ga = bf16_lo(gw[i]), gb = bf16_hi(gw[i]);
      mul2_rn(ta, tb, a, b, ga, gb);
      const uint64_t t = pack_f32x2(ta, tb);
      uint64_t u = 0;
      if constexpr (!kBf16) u = fma_f32x2(pack_f32x2(__fmaf_rn(a, ga, -ta), __fmaf_rn(b, gb, -tb)), rh2, u);
      u = fma_f32x2(t, rl2, u);
      float ya, yb;
      unpack_f32x2(fma_rz_f32x2(t, rh2, u), ya, yb);
      y[2 * i] = __uint_as_float(__float_as_uint(ya) | cut);
      y[2 * i + 1] = __uint_as_float(__float_as_uint(yb) | cut);
    }
    if (Y && in) {
      uint32_t yw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) yw[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
      store32(Y + row * K + col, yw, wide);
    }
    if (codes) {
      float a = in ? amax_n<16>(y) : 0.0f;
#pragma unroll
      for (int o = 4; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t b = fp8_scale_byte(a);
      if (in) *reinterpret_cast<uint4*>(codes + row * K + col) = codes16(y, fp8_inv_scale(b));
      uint32_t t = b << (lane & 24);  // the segment's four scale bytes, in every lane
      t |= __shfl_xor_sync(0xffffffffu, t, 8);
      t |= __shfl_xor_sync(0xffffffffu, t, 16);
      if (lane == j) word = t;
    }
  }
  if (codes && lane < S && seg0 + lane * wpr < band_tiles)
    *reinterpret_cast<uint32_t*>(scales + fp8_scale_offset(row, 4 * (seg0 + lane * wpr), band_tiles)) = word;
}

// ======================================================== weight packer ====
// W [K][N] (row-major, as the layer's residual) -> codes [N][K] and scales:
// one row per output channel, blocks along K.  HBM-bound: sizeof(T) + 1 bytes an
// element, once per weight.
// A CTA takes one block of 128 rows of K and 64 channels.  A thread holds 8
// rows x 8 channels in registers: the channels' maxima meet by shuffles and
// then in shared memory, one per warp; every thread then encodes its values,
// eight codes along K a channel, and only the codes (one byte an element, not
// four) are transposed through shared memory, in 16-byte chunks permuted so
// that neither side has bank conflicts.  On B200 3072 x 12288 take 25.1 us from
// bf16 (113 MB, 69 % of a copy's rate) and 31.7 from fp32 (189 MB, 91 %).  (A
// first version transposed fp32 values: 43.7 us from bf16.)
constexpr int kPw8Threads = 128;
constexpr int kPw8N = 64;

template <typename T>
__global__ void __launch_bounds__(kPw8Threads)
    pack_weight_fp8_kernel(const T* __restrict__ W, int K, int N, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t tile[kPw8N * kFp8Block];
  __shared__ __align__(16) float top[kPw8Threads / 32][kPw8N];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  // thread (kq, nc): rows 8 kq .. 8 kq + 7 of the block, channels 8 nc .. 8 nc + 7;
  // a warp holds four kq and all eight nc
  const int kq = (tid >> 5) * 4 + (tid & 3), nc = (tid >> 2) & 7;
  const int n0 = blockIdx.x * kPw8N + 8 * nc;
  const int blk = blockIdx.y;  // up to the last block of the last scale tile: those past K are zero scales
  const int k0 = blk * kFp8Block + 8 * kq;  // K and N are multiples of 8: all of the 8 x 8 or none
  const int64_t band_tiles = fp8_band_tiles(K);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k0 < K && n0 < N) {
      load8(W + static_cast<int64_t>(k0 + i) * N + n0, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    }
  }
  float amax[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i][e]));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    amax[e] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
  }
  if ((tid & 3) == 0) store8(&top[tid >> 5][8 * nc], amax);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPw8Threads / 32; ++i) {
    float o[8];
    load8(&top[i][8 * nc], o);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax[e] = fmaxf(amax[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = amax[e];
    const uint32_t b = fp8_scale_byte(a);
    const float inv = fp8_inv_scale(b);
    const float c[8] = {v[0][e], v[1][e], v[2][e], v[3][e], v[4][e], v[5][e], v[6][e], v[7][e]};
    // channel 8 nc + e: chunk kq / 2 of its 128 bytes, permuted by nc
    *reinterpret_cast<uint2*>(tile + (8 * nc + e) * kFp8Block + (((kq >> 1) ^ (2 * nc & 7)) << 4) + 8 * (kq & 1)) =
        codes8(c, inv);
    // rows past N are zeros here: their scale byte is 0
    if (kq == e && n0 + e < ((static_cast<int64_t>(N) + 127) & ~int64_t(127)))
      scales[fp8_scale_offset(n0 + e, blk, band_tiles)] = static_cast<uint8_t>(b);
  }
  __syncthreads();
  for (int i = tid; i < kPw8N * 8; i += kPw8Threads) {
    const int n = i >> 3, c = i & 7;
    const int64_t row = blockIdx.x * kPw8N + n;
    const int k = blk * kFp8Block + 16 * c;  // K is a multiple of 16
    if (row < N && k < K)
      *reinterpret_cast<uint4*>(codes + row * K + k) =
          *reinterpret_cast<const uint4*>(tile + n * kFp8Block + ((c ^ (2 * (n >> 3) & 7)) << 4));
  }
}

}  // namespace svdq
