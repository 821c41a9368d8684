// Microscaled 4-bit matrices: quantisation, dequantisation, the tiled layout of their block
// scales, and bf16 activations as 4-bit limbs.
//
// "BitDelta Guide", "3. Quantized Base Model Compatibility (BitDelta + GPTQ / QuIP#)": the
// 1-bit delta goes on top of quantized base weights; "Per-Axis Weight Deltas for Frequent
// Model Updates", Future Directions: INT4/FP8 co-design.
//
// All of these move bytes: they are bound by HBM from a few MB on, and by their launch below
// that. Times quoted here and below are of one B200 whose device-to-device copy runs at 6550
// GB/s, inputs not in L2.
#include "bd_fp4.cuh"

namespace bd {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// 32 bytes per thread and instruction, read once / written once
__device__ __forceinline__ void ldg32(const void* p, uint32_t* r) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void stg32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 consecutive values of a row as they are stored: 8 words of pairs, or 16 floats
template <int DT>
struct Raw16 {
  static constexpr int kWords = DT == BD_F32 ? 16 : 8;
  uint32_t w[kWords];
};
// WIDE: 32-byte aligned
template <int DT, bool WIDE>
__device__ __forceinline__ void load_raw(const void* row, int64_t k, Raw16<DT>& r) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(row) + k * (DT == BD_F32 ? 4 : 2);
#pragma unroll
  for (int j = 0; j < Raw16<DT>::kWords; j += 8) {
    if (WIDE) {
      ldg32(p + 4 * j, r.w + j);
    } else {
      const uint4 a = ldg_stream(p + 4 * j), b = ldg_stream(p + 4 * j + 16);
      r.w[j] = a.x; r.w[j + 1] = a.y; r.w[j + 2] = a.z; r.w[j + 3] = a.w;
      r.w[j + 4] = b.x; r.w[j + 5] = b.y; r.w[j + 6] = b.z; r.w[j + 7] = b.w;
    }
  }
}
template <int DT>
__device__ __forceinline__ void widen(const Raw16<DT>& r, float* v) {
#pragma unroll
  for (int j = 0; j < Raw16<DT>::kWords; ++j) {
    if (DT == BD_F32) {
      v[j] = __uint_as_float(r.w[j]);
    } else if (DT == BD_BF16) {
      v[2 * j] = bf16lo(r.w[j]);
      v[2 * j + 1] = bf16hi(r.w[j]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ void load16(const void* row, int64_t k, float* v) {
  Raw16<DT> r;
  load_raw<DT, false>(row, k, r);
  widen<DT>(r, v);
}

// 16 values to bf16 or fp32 memory (16-byte aligned; WIDE: 32)
template <int DT, bool WIDE>
__device__ __forceinline__ void store16(void* row, int64_t k, const float* v) {
  uint8_t* p = reinterpret_cast<uint8_t*>(row) + k * (DT == BD_F32 ? 4 : 2);
  constexpr int kWords = DT == BD_F32 ? 16 : 8;
  uint32_t a[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    if (DT == BD_F32)
      a[j] = __float_as_uint(v[j]);
    else
      a[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
  }
#pragma unroll
  for (int j = 0; j < kWords; j += 8) {
    if (WIDE) {
      stg32(p + 4 * j, a + j);
    } else {
      reinterpret_cast<uint4*>(p + 4 * j)[0] = make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]);
      reinterpret_cast<uint4*>(p + 4 * j)[1] = make_uint4(a[j + 4], a[j + 5], a[j + 6], a[j + 7]);
    }
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

__device__ __forceinline__ uint32_t finite_max16(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t a = abs_bits(v[j]);
    if (a < kInfBits) m = max(m, a);
  }
  return m;
}

// largest magnitude of 16 values; an infinity or a NaN among them shows as one
__device__ __forceinline__ float max16(const float* v) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < 16; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[j])));
  return m;
}
__device__ __forceinline__ bool finite(float m) { return abs_bits(m) < kInfBits; }

// The codes of 16 values of a block, and x_hat. q = v / s is taken as Markstein's corrected
// product: with y = 1 / s, q0 = v y, q = q0 - (q0 s - v) y, whose remainder is exact. Near a
// border b of E2M1, v = b s is an fp32 number, so q = b exactly there, and a v beside it
// differs by a whole unit in its last place, more than q's rounding can undo.
template <int HAT, bool WIDE>
__device__ __forceinline__ uint2 encode16(const float* v, bool none, float down, float s, float y, float r, void* hat_row,
                                          int64_t c) {
  float q[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = v[j] * down, q0 = a * y;
    q[j] = fmaf(-fmaf(q0, s, -a), y, q0);  // (this way round a zero keeps its sign)
  }
  if (none) {
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = 0.f;
  }
  if (HAT < 0) return make_uint2(e2m1_pack8(q), e2m1_pack8(q + 8));
  __half2 h[8];
  const uint2 p = make_uint2(e2m1_round8(q, h), e2m1_round8(q + 8, h + 4));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = __half22float2(h[j]);
    q[2 * j] = f.x * s * r;
    q[2 * j + 1] = f.y * s * r;
  }
  store16<HAT == BD_F32 ? BD_F32 : BD_BF16, WIDE>(hat_row, c, q);
  return p;
}

// the same for a block whose scale is a power of two, 1 / s = up
template <int HAT, bool WIDE>
__device__ __forceinline__ uint2 encode16_pow2(const float* v, bool bad, float up, float s, void* hat_row, int64_t c) {
  float q[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) q[j] = bad ? 0.f : v[j] * up;
  if (HAT < 0) return make_uint2(e2m1_pack8(q), e2m1_pack8(q + 8));
  __half2 h[8];
  const uint2 p = make_uint2(e2m1_round8(q, h), e2m1_round8(q + 8, h + 4));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = __half22float2(h[j]);
    q[2 * j] = f.x * s;
    q[2 * j + 1] = f.y * s;
  }
  store16<HAT == BD_F32 ? BD_F32 : BD_BF16, WIDE>(hat_row, c, q);
  return p;
}

// ------------------------------------------------------------------------------------
// quantise, BD_FP4_NV: one CTA per row. A thread holds NB blocks of the row as stored between
// the row's maximum and the codes, so the row is read once (from memory again in the loop
// when it has more than 8 blocks per thread). The two reads of a row cannot be closer than the
// row's maximum; a CTA per row keeps them a barrier apart, and up to 16 rows per SM hide it.
// Bound by HBM: 28672 x 4096 bf16 with x_hat, 536 MB, in 86-96 us (a plain read of the row
// twice, one warp per row, took 179).
// ------------------------------------------------------------------------------------
constexpr int kQuantThreads = 128;

template <int DT, int HAT, int NB, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads) k_fp4_quantize_nv(const void* __restrict__ x, int64_t rows,
                                                                   int64_t cols, int64_t ld,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales,
                                                                   float* __restrict__ row_scales,
                                                                   void* __restrict__ hat) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  __shared__ uint32_t red[kQuantThreads / 32];
  const int64_t tiles_k = fp4_tiles_k(cols, BD_FP4_NV);
  const int64_t row = blockIdx.x;
  uint8_t* sr = scales + fp4_scale_row(row, tiles_k);
  if (row >= rows) {  // a padding row of the scale tiles
    for (int64_t t = threadIdx.x; t < tiles_k; t += kQuantThreads) *reinterpret_cast<uint32_t*>(sr + t * kFp4TileBytes) = 0;
    return;
  }
  const uint8_t* xr = reinterpret_cast<const uint8_t*>(x) + row * ld * (DT == BD_F32 ? 4 : 2);
  uint8_t* hr = reinterpret_cast<uint8_t*>(hat) + row * cols * (HAT == BD_F32 ? 4 : 2);
  constexpr int kPass = kQuantThreads * 16;
  Raw16<DT> raw[NB];
  float bm[NB];
  uint32_t top = 0;
  auto row_max = [&](const float* v, float m) {
    if (finite(m)) {
      top = max(top, abs_bits(m));
    } else {
      top = max(top, finite_max16(v));
    }
  };
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t c = (int64_t)i * kPass + threadIdx.x * 16;
    if (c < cols) load_raw<DT, WIDE>(xr, c, raw[i]);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t c = (int64_t)i * kPass + threadIdx.x * 16;
    bm[i] = 0.f;
    if (c < cols) {
      float v[16];
      widen<DT>(raw[i], v);
      bm[i] = max16(v);
      row_max(v, bm[i]);
    }
  }
  for (int64_t c = (int64_t)NB * kPass + threadIdx.x * 16; c < cols; c += kPass) {
    float v[16];
    load16<DT>(xr, c, v);
    row_max(v, max16(v));
  }
  const int k = row_exponent(block_umax(top, red));
  if (threadIdx.x == 0) row_scales[row] = pow2f(k);
  const float down = pow2f(-k), r = pow2f(k);
  // every thread of a warp takes part, so that four neighbours' scale bytes go out as a word
  auto block = [&](const Raw16<DT>& w, float m, int64_t c) {
    const bool in = c < cols, bad = !finite(m);
    const uint32_t code = bad ? 0x7Fu : ue4m3_code((m * down) / 6.0f);
    const float s = ue4m3_value(code);
    uint32_t word = (in ? code : 0u) << (8 * (threadIdx.x & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const int64_t t = c >> 6;
    if ((threadIdx.x & 3) == 0 && t < tiles_k) *reinterpret_cast<uint32_t*>(sr + t * kFp4TileBytes) = word;
    if (in) {
      float v[16];
      widen<DT>(w, v);
      const bool none = !(s > 0.f);  // a scale of 0 or NaN: the codes are 0, without the values' signs
      const uint2 p = encode16<HAT, WIDE>(v, none, down, s, none ? 0.f : 1.0f / s, r, hr, c);
      *reinterpret_cast<uint2*>(codes + row * (cols >> 1) + (c >> 1)) = p;
    }
  };
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t c = (int64_t)i * kPass + threadIdx.x * 16;
    if ((int64_t)i * kPass < cols) block(raw[i], bm[i], c);
  }
  for (int64_t c0 = (int64_t)NB * kPass; c0 < cols; c0 += kPass) {
    const int64_t c = c0 + threadIdx.x * 16;
    Raw16<DT> w = {};
    float m = 0.f;
    if (c < cols) {
      load_raw<DT, WIDE>(xr, c, w);
      float v[16];
      widen<DT>(w, v);
      m = max16(v);
    }
    block(w, m, c);
  }
}

// ------------------------------------------------------------------------------------
// quantise, BD_FP4_MX: one thread per block of 32 columns, four blocks of scales per 4 lanes.
// Bound by HBM and, at a few MB, the ramp of the loads: 512 x 14336 fp32 with x_hat, 62 MB, in
// 15.7 us (floor 9.6).
// ------------------------------------------------------------------------------------
template <int DT, int HAT, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads) k_fp4_quantize_mx(const void* __restrict__ x, int64_t rows, int64_t cols,
                                                         int64_t ld, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales, void* __restrict__ hat) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  const uint32_t tiles_k = (uint32_t)fp4_tiles_k(cols, BD_FP4_MX);
  const int64_t padded = (rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
  // a row's blocks are padded to whole words of four; a unit is one block, real or padding
  const int64_t units = padded * tiles_k * 4;
  for (int64_t u0 = (int64_t)blockIdx.x * kQuantThreads; u0 < units; u0 += (int64_t)gridDim.x * kQuantThreads) {
    const int64_t u = u0 + threadIdx.x;  // (units is a multiple of 512: whole warps)
    const int64_t row = units < (1ll << 32) ? (int64_t)((uint32_t)u / (tiles_k * 4)) : u / (tiles_k * 4);
    const int64_t b = u - row * (tiles_k * 4), c = b * 32;
    const bool in = row < rows && c < cols;
    uint32_t code = 0;
    if (in) {
      const uint8_t* xr = reinterpret_cast<const uint8_t*>(x) + row * ld * (DT == BD_F32 ? 4 : 2);
      Raw16<DT> w[2];
      load_raw<DT, WIDE>(xr, c, w[0]);
      load_raw<DT, WIDE>(xr, c + 16, w[1]);
      float v[32];
      widen<DT>(w[0], v);
      widen<DT>(w[1], v + 16);
      float m = max16(v);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(max16(v + 16)));
      const bool bad = !finite(m);
      // floor(log2 max) - 2; a zero or subnormal maximum ends at the lowest scale
      int e = (int)(abs_bits(m) >> 23) - 127 - 2;
      if (e < -127) e = -127;
      code = bad ? 0xFFu : (uint32_t)(e + 127);
      const float s = bad ? __uint_as_float(0x7FFFFFFFu) : pow2f(e), up = pow2f(bad ? 0 : -e);
      uint8_t* hr = reinterpret_cast<uint8_t*>(hat) + row * cols * (HAT == BD_F32 ? 4 : 2);
      uint2 p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) p[h] = encode16_pow2<HAT, WIDE>(v + 16 * h, bad, up, s, hr, c + 16 * h);
      *reinterpret_cast<uint4*>(codes + row * (cols >> 1) + (c >> 1)) = make_uint4(p[0].x, p[0].y, p[1].x, p[1].y);
    }
    uint32_t word = code << (8 * (threadIdx.x & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if ((threadIdx.x & 3) == 0)
      *reinterpret_cast<uint32_t*>(scales + fp4_scale_row(row, tiles_k) + (b >> 2) * kFp4TileBytes) = word;
  }
}

// ------------------------------------------------------------------------------------
// dequantise: one thread per 32 columns, four such units in flight (one in flight: 38.8 us where
// this takes 26.7: 14336 x 4096 to bf16, 150 MB, floor 23.0). Bound by HBM's writes.
// ------------------------------------------------------------------------------------
template <int FMT, int OUT, bool WIDE>
__global__ void __launch_bounds__(256) k_fp4_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        const float* __restrict__ row_scales, int64_t rows,
                                                        int64_t cols, void* __restrict__ out) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  constexpr int kUnroll = 4;
  const int64_t tiles_k = fp4_tiles_k(cols, FMT);
  const int64_t per_row = cols / 32, units = rows * per_row;
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t u0 = (int64_t)blockIdx.x * 256 + threadIdx.x; u0 < units; u0 += kUnroll * stride) {
    uint4 p[kUnroll];
    uint32_t sc[kUnroll];
    float r[kUnroll];
    int64_t at[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t u = u0 + i * stride;
      if (u < units) {
        const int64_t row = u < (1ll << 32) ? (int64_t)((uint32_t)u / (uint32_t)per_row) : u / per_row;
        const int64_t c = (u - row * per_row) * 32, b = c / fp4_block(FMT);
        at[i] = row * cols + c;
        p[i] = ldg_stream(codes + at[i] / 2);
        const uint8_t* s = scales + fp4_scale_row(row, tiles_k) + (b >> 2) * kFp4TileBytes + (b & 3);
        sc[i] = FMT == BD_FP4_NV ? *reinterpret_cast<const uint16_t*>(s) : *s;
        r[i] = row_scales ? row_scales[row] : 1.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (u0 + i * stride >= units) break;
      const uint32_t w[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = fp4_scale_value<FMT>(FMT == BD_FP4_NV ? (sc[i] >> (8 * h)) & 0xFFu : sc[i]);
        __half2 e[8];
        e2m1_unpack8(w[2 * h], e);
        e2m1_unpack8(w[2 * h + 1], e + 4);
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = __half22float2(e[j]);
          v[2 * j] = f.x * s * r[i];
          v[2 * j + 1] = f.y * s * r[i];
        }
        store16<OUT, WIDE>(out, at[i] + 16 * h, v);
      }
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
// activations -> limbs: x_t = 2^k_t * sum_l s_l * e2m1_l per block, s_l the least power of two
// with max|what limbs 0 .. l-1 left| <= 6 s_l. Limb 0 leaves at most s_0 (half a step between 4 and
// 6), which is within 4 of s_0 / 4; a limb that is given at most 4 s_l leaves at most s_l / 2, within
// 4 of s_l / 8: so s_1 <= s_0 / 4, s_{l+1} <= s_l / 8 from there (a smaller scale has a finer
// grid wherever it reaches, so it leaves no more), and the smallest limb leaves at most half of
// s_{L-1} <= s_0 / 2^limb_shift(L-1): s_0 / 512 with 4 limbs, s_0 / 32768 with 6. A bf16 value has 8
// significant bits, so with L limbs it is exact from s_0 / 2 of its block up with 4 limbs, from
// s_0 / 128 with 6. Scales that follow what is left, instead of falling by 4, 8, 8, ... whatever
// is left, cost a maximum per limb and gain most where it counts: behind an outlier that the
// first limbs hold exactly the others start again from the block's own size (relative error of a
// product, K = 4096, NV: Gaussian tokens 3e-5 instead of 1.1e-4 with 4 limbs, 2e-8 instead of 2e-7
// with 6; one value of 4e4 at weights of zero 7e-3 instead of 6e-2, 5e-5 instead of 2e-2).
// NV scales are E4M3, which holds powers of two from 2^-9 to 2^8 only: k_t puts the token's
// largest block at s_0 <= 2^8, and limb l's scale is stored 2^limb_shift(l) larger than it is (the
// product's epilogue takes that off again), so that every limb has the whole range. What a block
// loses to the lowest scale is at most half of 2^-9 / 2^limb_shift(L-1), which is 2^-27 (4 limbs) or
// 2^-33 (6) of the token's maximum, above 3 * 2^8. MX scales hold every power used, and k_t = 0.
// ------------------------------------------------------------------------------------
// One CTA per (token, 4096 columns), one thread per 16 columns; in NV every CTA of a token
// takes the maximum of the whole row (a few loads per thread, all in flight). Bound by its
// launch up to a few tokens (about 2 us); 512 tokens of 4096 take 5.4 us.
constexpr int kLimbThreads = 256;
constexpr int kLimbChunk = kLimbThreads * 16;

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
  const uint32_t pair = __ballot_sync(0xffffffffu, in);  // (the two threads of an MX block go together)
  if (!in) return;
  const bool bad = bm >= kInfBits;
  const float down = pow2f(-k);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = bad ? 0.f : v[j] * down;
  const int64_t b = c / kBlock;
#pragma unroll
  for (int l = 0; l < L; ++l) {
    const int shift = FMT == BD_FP4_NV ? limb_shift(l) : 0;
    float m = abs_max<16>(v);
    if (FMT == BD_FP4_MX) m = fmaxf(m, __shfl_xor_sync(pair, m, 1));
    const int e = max(limb_exponent(__float_as_uint(m)), kLow - shift);
    const float up = pow2f(-e), s = pow2f(e);
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
    if (FMT == BD_FP4_NV)  // E4M3: 2^es is a normal code from 2^-6 on, then 4, 2, 1
      code = bad ? 0x7Fu : (e + shift >= -6 ? (uint32_t)(e + shift + 7) << 3 : 1u << (e + shift + 9));
    else
      code = bad ? 0xFFu : (uint32_t)(e + 127);
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

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  uint8_t *codes, *scales;
  float* row_scales;
  void* hat;
  int32_t hat_dtype;
  cudaStream_t s;
};
template <int DT, int HAT, int NB, bool WIDE>
cudaError_t quantize_nv(const QuantArgs& a) {
  const int64_t padded = (a.rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
  return launch_pdl(k_fp4_quantize_nv<DT, HAT, NB, WIDE>, dim3((unsigned)padded), dim3(kQuantThreads), 0, a.s, a.x,
                    a.rows, a.cols, a.ld, a.codes, a.scales, a.row_scales, a.hat);
}
template <int DT, int HAT, bool WIDE>
cudaError_t quantize(const QuantArgs& a, int fmt) {
  if (fmt == BD_FP4_MX) {
    const int64_t padded = (a.rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
    const int64_t blocks = padded * fp4_tiles_k(a.cols, BD_FP4_MX) * 4 / kQuantThreads;
    const int64_t cap = 1 << 30;
    return launch_pdl(k_fp4_quantize_mx<DT, HAT, WIDE>, dim3((unsigned)(blocks < cap ? blocks : cap)),
                      dim3(kQuantThreads), 0, a.s, a.x, a.rows, a.cols, a.ld, a.codes, a.scales, a.hat);
  }
  // blocks of a row per thread
  const int64_t nb = (a.cols + kQuantThreads * 16 - 1) / (kQuantThreads * 16);
  if (nb <= 1) return quantize_nv<DT, HAT, 1, WIDE>(a);
  if (nb <= 2) return quantize_nv<DT, HAT, 2, WIDE>(a);
  if (nb <= 4) return quantize_nv<DT, HAT, 4, WIDE>(a);
  return quantize_nv<DT, HAT, 8, WIDE>(a);
}
template <int DT>
cudaError_t quantize_dt(const QuantArgs& a, int fmt) {
  // 32-byte accesses where every row of x and x_hat starts on 32 bytes (cols % 32 == 0 sees to
  // x_hat's), else 16-byte ones
  const bool wide = aligned32(a.x) && (a.rows == 1 || a.ld * (DT == BD_F32 ? 4 : 2) % 32 == 0) && aligned32(a.hat);
  if (!a.hat) return wide ? quantize<DT, -1, true>(a, fmt) : quantize<DT, -1, false>(a, fmt);
  if (a.hat_dtype == BD_F32) return wide ? quantize<DT, BD_F32, true>(a, fmt) : quantize<DT, BD_F32, false>(a, fmt);
  return wide ? quantize<DT, BD_BF16, true>(a, fmt) : quantize<DT, BD_BF16, false>(a, fmt);
}
template <int FMT, int OUT>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int64_t rows,
                       int64_t cols, void* out, cudaStream_t s) {
  const int64_t blocks = (rows * (cols / 32) + 1023) / 1024;
  const int64_t cap = (int64_t)sm_count() * 8;
  auto* fn = aligned32(out) ? k_fp4_dequantize<FMT, OUT, true> : k_fp4_dequantize<FMT, OUT, false>;
  return launch_pdl(fn, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, s, codes, scales, row_scales, rows,
                    cols, out);
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
  const QuantArgs a{x, rows, cols, ld, codes, scales, row_scales, x_hat, hat_dtype, s};
  launch_begin(K_FP4_QUANT, s);
  BD_CUDA_TRY(dtype == BD_F32    ? quantize_dt<BD_F32>(a, fmt)
              : dtype == BD_BF16 ? quantize_dt<BD_BF16>(a, fmt)
                                 : quantize_dt<BD_F16>(a, fmt));
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
  launch_begin(K_FP4_DEQUANT, s);
  cudaError_t e;
  if (fmt == BD_FP4_NV)
    e = out_dtype == BD_F32 ? dequantize<BD_FP4_NV, BD_F32>(codes, scales, row_scales, rows, cols, out, s)
                            : dequantize<BD_FP4_NV, BD_BF16>(codes, scales, row_scales, rows, cols, out, s);
  else
    e = out_dtype == BD_F32 ? dequantize<BD_FP4_MX, BD_F32>(codes, scales, row_scales, rows, cols, out, s)
                            : dequantize<BD_FP4_MX, BD_BF16>(codes, scales, row_scales, rows, cols, out, s);
  BD_CUDA_TRY(e);
  launch_end(K_FP4_DEQUANT, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}
