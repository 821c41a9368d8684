// Microscaled 4-bit matrices: quantisation, dequantisation, the tiled layout of their block
// scales, and bf16 activations as 4-bit limbs.
//
// "BitDelta Guide", "3. Quantized Base Model Compatibility (BitDelta + GPTQ / QuIP#)": the
// 1-bit delta goes on top of quantized base weights; "Per-Axis Weight Deltas for Frequent
// Model Updates", Future Directions: INT4/FP8 co-design.
#include "bd_fp4.cuh"

namespace bd {

// 16 consecutive values of a row
template <int DT>
__device__ __forceinline__ void load16(const void* row, int64_t k, float* v) {
  if (DT == BD_F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = p[j];
      v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + k);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 u = p[j];
      const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == BD_BF16) {
          v[8 * j + 2 * i] = bf16lo(a[i]);
          v[8 * j + 2 * i + 1] = bf16hi(a[i]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
          v[8 * j + 2 * i] = f.x;
          v[8 * j + 2 * i + 1] = f.y;
        }
      }
    }
  }
}

// 16 values to bf16 or fp32 memory
template <int DT>
__device__ __forceinline__ void store16(void* row, int64_t k, const float* v) {
  if (DT == BD_F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(row) + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint32_t a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = f2bf_bits(v[2 * j]) | (f2bf_bits(v[2 * j + 1]) << 16);
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(row) + k);
    p[0] = make_uint4(a[0], a[1], a[2], a[3]);
    p[1] = make_uint4(a[4], a[5], a[6], a[7]);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t block_umax(uint32_t m, uint32_t* red) {
  m = __reduce_max_sync(0xffffffffu, m);
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = m;
  __syncthreads();
  uint32_t r = 0;
  for (int i = 0; i < nw; ++i) r = max(r, red[i]);
  __syncthreads();
  return r;
}

// the least k with amax <= 2688 * 2^k (2688 = 6 * 448 = 1.3125 * 2^11), kept in [-126, 126];
// 0 for a row of zeros. amax is given by its bits.
__device__ __forceinline__ int row_exponent(uint32_t bits) {
  if (bits == 0) return 0;
  const int e = (int)(bits >> 23);  // a subnormal amax is below 2688 * 2^-126 anyway
  const int k = e - 127 - 11 + ((bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return k < -126 ? -126 : (k > 126 ? 126 : k);
}

// ------------------------------------------------------------------------------------
// quantise: one CTA per row; NV first takes the row's largest finite magnitude
// ------------------------------------------------------------------------------------
template <int FMT, int DT, int HAT>  // HAT: dtype of x_hat, or -1
__global__ void __launch_bounds__(256) k_fp4_quantize(const void* __restrict__ x, int64_t rows, int64_t cols,
                                                      int64_t ld, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, float* __restrict__ row_scales,
                                                      void* __restrict__ hat) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  __shared__ uint32_t red[8];
  const int64_t tiles_k = fp4_tiles_k(cols, FMT);
  const int64_t padded = (rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
  constexpr int kBlock = fp4_block(FMT);
  constexpr int kEs = DT == BD_F32 ? 4 : 2;
  for (int64_t row = blockIdx.x; row < padded; row += gridDim.x) {
    uint8_t* sr = scales + fp4_scale_row(row, tiles_k);
    const int64_t nb = row < rows ? cols / kBlock : 0;
    // padding scales (past the row's last block, or of a padding row) are zero
    for (int64_t b = nb + threadIdx.x; b < 4 * tiles_k; b += 256) sr[(b >> 2) * kFp4TileBytes + (b & 3)] = 0;
    if (row >= rows) continue;
    const uint8_t* xr = reinterpret_cast<const uint8_t*>(x) + row * ld * kEs;
    int k = 0;
    if (FMT == BD_FP4_NV) {
      uint32_t m = 0;
      for (int64_t c = (int64_t)threadIdx.x * 16; c < cols; c += 256 * 16) {
        float v[16];
        load16<DT>(xr, c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t a = abs_bits(v[j]);
          if (a < kInfBits) m = max(m, a);
        }
      }
      k = row_exponent(block_umax(m, red));
      if (threadIdx.x == 0) row_scales[row] = pow2f(k);
    }
    const float down = pow2f(-k);
    // every warp runs whole iterations: two neighbouring threads share an MX block
    for (int64_t c0 = (int64_t)(threadIdx.x & ~31) * 16; c0 < cols; c0 += 256 * 16) {
      const int64_t c = c0 + (threadIdx.x & 31) * 16;
      const bool in = c < cols;
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
      if (in) load16<DT>(xr, c, v);
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[j]));
      if (FMT == BD_FP4_MX) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const bool bad = m >= kInfBits;
      uint32_t code;
      float s, q[16];
      if (FMT == BD_FP4_NV) {
        code = bad ? 0x7Fu : ue4m3_code((__uint_as_float(m) * down) / 6.0f);
        s = ue4m3_value(code);
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = !bad && s > 0.f ? (v[j] * down) / s : 0.f;
      } else {
        // floor(log2 amax) - 2; a zero or subnormal amax ends at the lowest scale
        int e = (int)(m >> 23) - 127 - 2;
        if (e < -127) e = -127;
        code = bad ? 0xFFu : (uint32_t)(e + 127);
        s = bad ? __uint_as_float(0x7FFFFFFFu) : pow2f(e);
        const float up = pow2f(bad ? 0 : -e);
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = bad ? 0.f : v[j] * up;
      }
      if (!in) continue;
      __half2 h[8];
      uint2 p;
      if (HAT >= 0)
        p = make_uint2(e2m1_round8(q, h), e2m1_round8(q + 8, h + 4));
      else
        p = make_uint2(e2m1_pack8(q), e2m1_pack8(q + 8));
      *reinterpret_cast<uint2*>(codes + row * (cols >> 1) + (c >> 1)) = p;
      const int64_t b = c / kBlock;
      if (FMT == BD_FP4_NV || (threadIdx.x & 1) == 0) sr[(b >> 2) * kFp4TileBytes + (b & 3)] = (uint8_t)code;
      if (HAT >= 0) {
        const float r = pow2f(k);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = __half22float2(h[j]);
          v[2 * j] = f.x * s * r;
          v[2 * j + 1] = f.y * s * r;
        }
        store16<HAT == BD_F32 ? BD_F32 : BD_BF16>(
            reinterpret_cast<uint8_t*>(hat) + row * cols * (HAT == BD_F32 ? 4 : 2), c, v);
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// dequantise
// ------------------------------------------------------------------------------------
template <int FMT, int OUT>
__global__ void __launch_bounds__(256) k_fp4_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        const float* __restrict__ row_scales, int64_t rows,
                                                        int64_t cols, void* __restrict__ out) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  const int64_t tiles_k = fp4_tiles_k(cols, FMT);
  constexpr int kBlock = fp4_block(FMT);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const uint8_t* sr = scales + fp4_scale_row(row, tiles_k);
    const float r = row_scales ? row_scales[row] : 1.f;
    for (int64_t c = (int64_t)threadIdx.x * 16; c < cols; c += 256 * 16) {
      const uint2 p = *reinterpret_cast<const uint2*>(codes + row * (cols >> 1) + (c >> 1));
      const int64_t b = c / kBlock;
      const float s = fp4_scale_value<FMT>(sr[(b >> 2) * kFp4TileBytes + (b & 3)]);
      __half2 h[8];
      e2m1_unpack8(p.x, h);
      e2m1_unpack8(p.y, h + 4);
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = __half22float2(h[j]);
        v[2 * j] = f.x * s * r;
        v[2 * j + 1] = f.y * s * r;
      }
      store16<OUT>(reinterpret_cast<uint8_t*>(out) + row * cols * (OUT == BD_F32 ? 4 : 2), c, v);
    }
  }
}

// ------------------------------------------------------------------------------------
// row-major block scales [rows][nb] -> tiles, one thread per 4-scale word
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_fp4_tile_scales(const uint8_t* __restrict__ in, int64_t rows, int64_t nb,
                                                         int64_t tiles_k, uint32_t* __restrict__ out, int64_t words) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    // word i of the output: tile, then row % 32, then row / 32
    const int64_t tile = i >> 7;
    const int w = (int)(i & 127);
    const int64_t row = (tile / tiles_k) * kFp4TileRows + (w & 3) * 32 + (w >> 2);
    const int64_t b = (tile % tiles_k) * 4;
    uint32_t v = 0;
    if (row < rows)
      for (int j = 0; j < 4; ++j)
        if (b + j < nb) v |= (uint32_t)in[row * nb + b + j] << (8 * j);
    out[i] = v;
  }
}

// ------------------------------------------------------------------------------------
// activations -> limbs: x_t = 2^k_t * sum_l s_l * e2m1_l per block, s_0 the least power of
// two with max|block| <= 6 s_0, s_1 = s_0 / 4, and each further one an eighth of the one
// before: limb 0 leaves a remainder of at most s_0 = 4 s_1 (half a step between 4 and 6),
// limb l at most s_l / 2 = 4 s_{l+1}. A bf16 value has 8 significant bits, so with L limbs it
// is exact when its lowest bit is s_{L-1} or more (from s_0 / 2 of its block up with 4
// limbs, from s_0 / 128 with 6); smaller values end within s_{L-1} / 2 (s_0 / 512, s_0 / 32768).
// NV scales are E4M3, which holds powers of two from 2^-9 to 2^8 only: k_t puts the token's
// largest block at s_0 = 2^8, and limbs below 2^-9 are dropped (an error of at most 2^-8,
// below 2^-17 of the token's maximum, which is above 3 * 2^8). MX scales hold every power used, and k_t = 0.
// ------------------------------------------------------------------------------------
// One CTA per (token, 4096 columns), one thread per 16 columns; in NV every CTA of a token
// takes the maximum of the whole row (a few loads per thread, all in flight).
constexpr int kLimbThreads = 256;
constexpr int kLimbChunk = kLimbThreads * 16;

__device__ __forceinline__ uint32_t finite_max16(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t a = abs_bits(v[j]);
    if (a < kInfBits) m = max(m, a);
  }
  return m;
}

template <int FMT, int L>
__global__ void __launch_bounds__(kLimbThreads) k_fp4_limbs(const uint16_t* __restrict__ x, int64_t d_in, int h,
                                                            int n_stride, uint8_t* __restrict__ xc,
                                                            uint8_t* __restrict__ xs, float* __restrict__ xmul,
                                                            uint32_t* __restrict__ reset_status) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  constexpr int kBlock = fp4_block(FMT);
  constexpr int kLow = FMT == BD_FP4_NV ? -9 : -127;  // lowest scale
  __shared__ uint32_t red[kLimbThreads / 32];
  const int t = blockIdx.x;
  if (reset_status && t == 0 && blockIdx.y == 0 && threadIdx.x == 0) *reset_status = 0;  // reports this call
  const int64_t tiles_k = fp4_tiles_k(d_in, FMT);
  const uint16_t* xr = x + (int64_t)t * d_in;
  const int64_t row0 = (int64_t)(t / h) * n_stride + (t % h) / 8 * (8 * L) + t % 8;
  const int64_t c = (int64_t)blockIdx.y * kLimbChunk + threadIdx.x * 16;
  const bool in = c < d_in;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 0.f;
  if (in) load16<BD_BF16>(xr, c, v);
  int k = 0;
  if (FMT == BD_FP4_NV) {
    // the token's exponent: its largest finite |x| <= 6 * 2^8 * 2^k (1536 = 1.5 * 2^10)
    uint32_t m = finite_max16(v);
#pragma unroll 4
    for (int64_t o = threadIdx.x * 16; o < d_in; o += kLimbChunk)
      if (o != c) {
        float u[16];
        load16<BD_BF16>(xr, o, u);
        m = max(m, finite_max16(u));
      }
    m = block_umax(m, red);
    if (m > 0) {
      k = (int)(m >> 23) - 127 - 10 + ((m & 0x7FFFFFu) > 0x400000u ? 1 : 0);
      k = k < -126 ? -126 : k;
    }
  }
  if (threadIdx.x == 0 && blockIdx.y == 0) xmul[t] = pow2f(k);
  // padding scales past the row's last block are zero: at most 3 of them
  const int64_t nb = d_in / kBlock;
  if (blockIdx.y == 0 && threadIdx.x < 4 * L) {
    const int64_t b = nb + threadIdx.x / L;
    if (b < 4 * tiles_k)
      xs[fp4_scale_row(row0 + (threadIdx.x % L) * 8, tiles_k) + (b >> 2) * kFp4TileBytes + (b & 3)] = 0;
  }
  uint32_t bm = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) bm = max(bm, abs_bits(v[j]));
  if (FMT == BD_FP4_MX) bm = max(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
  if (!in) return;  // (two threads of an MX block go together)
  const bool bad = bm >= kInfBits;
  const float down = pow2f(-k);
  // s_0 = 2^e: least e with max|v| <= 6 * 2^e = 1.5 * 2^(e + 2)
  const uint32_t am = bad ? 0u : abs_bits(__uint_as_float(bm) * down);
  int e = (int)(am >> 23) - 127 - 2 + ((am & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  if (e < kLow) e = kLow;
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = bad ? 0.f : v[j] * down;
  const int64_t b = c / kBlock;
#pragma unroll
  for (int l = 0; l < L; ++l) {
    const int el = e - (l == 0 ? 0 : 3 * l - 1);
    const bool live = el >= kLow;
    const float up = live ? pow2f(-el) : 0.f, s = live ? pow2f(el) : 0.f;
    float q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = v[j] * up;
    __half2 hh[8];
    const uint2 p = make_uint2(e2m1_round8(q, hh), e2m1_round8(q + 8, hh + 4));
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // the remainder is exact: a multiple of v's lowest bit
      const float2 f = __half22float2(hh[j]);
      v[2 * j] = fmaf(-f.x, s, v[2 * j]);
      v[2 * j + 1] = fmaf(-f.y, s, v[2 * j + 1]);
    }
    const int64_t row = row0 + 8 * l;
    *reinterpret_cast<uint2*>(xc + row * (d_in >> 1) + (c >> 1)) = p;
    uint32_t code;
    if (FMT == BD_FP4_NV)  // E4M3: 2^el is a normal code from 2^-6 on, then 4, 2, 1
      code = bad ? 0x7Fu : (!live ? 0u : (el >= -6 ? (uint32_t)(el + 7) << 3 : 1u << (el + 9)));
    else
      code = bad ? 0xFFu : (!live ? 0u : (uint32_t)(el + 127));
    if (FMT == BD_FP4_NV || (threadIdx.x & 1) == 0)
      xs[fp4_scale_row(row, tiles_k) + (b >> 2) * kFp4TileBytes + (b & 3)] = (uint8_t)code;
  }
}

bd_status launch_fp4_limbs(const Fp4Plan& p, int fmt, const void* x, int64_t d_in, int64_t tokens, uint8_t* xc,
                           uint8_t* xs, float* xmul, uint32_t* reset_status, cudaStream_t s) {
  auto* fn = fmt == BD_FP4_NV ? (p.limbs == kFp4LimbsBf16 ? k_fp4_limbs<BD_FP4_NV, kFp4LimbsBf16>
                                                          : k_fp4_limbs<BD_FP4_NV, kFp4LimbsF32>)
                              : (p.limbs == kFp4LimbsBf16 ? k_fp4_limbs<BD_FP4_MX, kFp4LimbsBf16>
                                                          : k_fp4_limbs<BD_FP4_MX, kFp4LimbsF32>);
  const int64_t chunks = (d_in + kLimbChunk - 1) / kLimbChunk;  // at most 4096
  launch_begin(K_FP4_LIMBS, s);
  BD_CUDA_TRY(launch_pdl(fn, dim3((unsigned)tokens, (unsigned)chunks), dim3(kLimbThreads), 0, s,
                         static_cast<const uint16_t*>(x), d_in, p.h, p.n_stride, xc, xs, xmul, reset_status));
  launch_end(K_FP4_LIMBS, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

namespace {
bool fp4_fmt_ok(int32_t fmt) { return fmt == BD_FP4_NV || fmt == BD_FP4_MX; }
bool fp4_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 1 && rows <= kFp4MaxDim && cols >= 32 && cols <= kFp4MaxDim && (cols % 32) == 0;
}
int grid_rows(int64_t rows) {
  const int64_t cap = (int64_t)sm_count() * 8;  // resident CTAs of 256 threads
  return (int)(rows < cap ? rows : cap);
}

template <int FMT, int DT>
cudaError_t launch_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                            float* row_scales, void* hat, int32_t hat_dtype, cudaStream_t s) {
  const int64_t padded = (rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
  auto* fn = !hat ? k_fp4_quantize<FMT, DT, -1>
                  : (hat_dtype == BD_F32 ? k_fp4_quantize<FMT, DT, BD_F32> : k_fp4_quantize<FMT, DT, BD_BF16>);
  return launch_pdl(fn, dim3((unsigned)grid_rows(padded)), dim3(256), 0, s, x, rows, cols, ld, codes, scales,
                    row_scales, hat);
}
}  // namespace

}  // namespace bd

extern "C" size_t bd_fp4_scales_bytes(int64_t rows, int64_t cols, int32_t fmt) {
  using namespace bd;
  if (!fp4_fmt_ok(fmt) || !fp4_shape_ok(rows, cols)) return 0;
  return (size_t)fp4_scale_bytes(rows, cols, fmt);
}

extern "C" bd_status bd_prepare_fp4_scales(const uint8_t* scales, int32_t fmt, int64_t rows, int64_t cols,
                                           uint8_t* out, void* stream) {
  using namespace bd;
  if (!fp4_fmt_ok(fmt)) return BD_ERR_CONFIG;
  if (!fp4_shape_ok(rows, cols)) return BD_ERR_SHAPE;
  if (!scales || !out) return BD_ERR_NULL;
  if (!aligned16(out)) return BD_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t words = fp4_scale_bytes(rows, cols, fmt) / 4;
  const int64_t blocks = (words + 255) / 256;
  launch_begin(K_FP4_TILE_SCALES, s);
  BD_CUDA_TRY(launch_pdl(k_fp4_tile_scales, dim3((unsigned)grid_rows(blocks)), dim3(256), 0, s, scales, rows,
                         cols / fp4_block(fmt), fp4_tiles_k(cols, fmt), reinterpret_cast<uint32_t*>(out), words));
  launch_end(K_FP4_TILE_SCALES, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

extern "C" bd_status bd_quantize_fp4(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                     int32_t fmt, uint8_t* codes, uint8_t* scales, float* row_scales, void* x_hat,
                                     int32_t hat_dtype, void* stream) {
  using namespace bd;
  if (dtype != BD_F32 && dtype != BD_BF16 && dtype != BD_F16) return BD_ERR_DTYPE;
  if (x_hat && hat_dtype != BD_F32 && hat_dtype != BD_BF16) return BD_ERR_DTYPE;
  if (!fp4_fmt_ok(fmt)) return BD_ERR_CONFIG;
  const int es = dtype == BD_F32 ? 4 : 2;
  if (!fp4_shape_ok(rows, cols) || ld < cols || ld > kFp4MaxLd) return BD_ERR_SHAPE;
  if (!x || !codes || !scales || (fmt == BD_FP4_NV && !row_scales)) return BD_ERR_NULL;
  if (!aligned16(x) || (rows > 1 && (ld * es) % 16 != 0) || !aligned16(codes) || !aligned16(scales) ||
      (x_hat && !aligned16(x_hat)) || (reinterpret_cast<uintptr_t>(row_scales) & 3u))
    return BD_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_begin(K_FP4_QUANT, s);
  cudaError_t e;
#define BD_Q(F, D) launch_quantize<F, D>(x, rows, cols, ld, codes, scales, row_scales, x_hat, hat_dtype, s)
  if (fmt == BD_FP4_NV)
    e = dtype == BD_F32 ? BD_Q(BD_FP4_NV, BD_F32) : dtype == BD_BF16 ? BD_Q(BD_FP4_NV, BD_BF16) : BD_Q(BD_FP4_NV, BD_F16);
  else
    e = dtype == BD_F32 ? BD_Q(BD_FP4_MX, BD_F32) : dtype == BD_BF16 ? BD_Q(BD_FP4_MX, BD_BF16) : BD_Q(BD_FP4_MX, BD_F16);
#undef BD_Q
  BD_CUDA_TRY(e);
  launch_end(K_FP4_QUANT, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

extern "C" bd_status bd_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales,
                                       int32_t fmt, int64_t rows, int64_t cols, void* out, int32_t out_dtype,
                                       void* stream) {
  using namespace bd;
  if (out_dtype != BD_F32 && out_dtype != BD_BF16) return BD_ERR_DTYPE;
  if (!fp4_fmt_ok(fmt)) return BD_ERR_CONFIG;
  if (!fp4_shape_ok(rows, cols)) return BD_ERR_SHAPE;
  if (!codes || !scales || !out) return BD_ERR_NULL;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out) || (reinterpret_cast<uintptr_t>(row_scales) & 3u))
    return BD_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto* fn = fmt == BD_FP4_NV
                 ? (out_dtype == BD_F32 ? k_fp4_dequantize<BD_FP4_NV, BD_F32> : k_fp4_dequantize<BD_FP4_NV, BD_BF16>)
                 : (out_dtype == BD_F32 ? k_fp4_dequantize<BD_FP4_MX, BD_F32> : k_fp4_dequantize<BD_FP4_MX, BD_BF16>);
  launch_begin(K_FP4_DEQUANT, s);
  BD_CUDA_TRY(launch_pdl(fn, dim3((unsigned)grid_rows(rows)), dim3(256), 0, s, codes, scales, row_scales, rows, cols,
                         out));
  launch_end(K_FP4_DEQUANT, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}
