// Microscaled 4-bit format: element and scale codes, the tiled scale layout, and the plan
// of the 4-bit products (see include/bitdelta.h for the format itself).
#pragma once

#include <cuda_fp8.h>

#include "bd_internal.cuh"

namespace bd {

// kernel kinds of the 4-bit operators, numbered after those of bd_internal.cuh
enum Fp4KernelKind : int32_t {
  K_FP4_QUANT = K_KIND_COUNT,  // microscaled 4-bit quantization
  K_FP4_DEQUANT,               // ... and back
  K_FP4_TILE_SCALES,           // row-major block scales -> the tiled layout
  K_FP4_LIMBS,                 // activations -> 4-bit limbs with power-of-two block scales
  K_FP4_MM,                    // tcgen05 block-scaled 4-bit product
  K_FP4_SEG_LIMBS,             // limbs of the delta segments' tokens
  K_DELTA_FP4,                 // the tenants' deltas as a 4-bit product + combine
  K_FP4_GEMV,                  // product with a few bf16 tokens on the CUDA cores
  kKindCount                   // all kinds
};

constexpr int kFp4KStage = 256;   // columns per shared-memory stage of a product: one 128-byte swizzle row
constexpr int kFp4TileRows = 128;  // rows of a scale tile
constexpr int kFp4TileBytes = 512;
constexpr int64_t kFp4MaxDim = 1 << 24;      // rows, columns
constexpr int64_t kFp4MaxTokens = 65536;     // X rows of a product
constexpr int64_t kFp4MaxLd = 1ll << 31;     // row stride of a quantiser's input, elements

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == BD_FP4_NV ? 16 : 32; }
// scale tiles along a row (each holds 4 scales of 128 rows)
__host__ __device__ inline int64_t fp4_tiles_k(int64_t cols, int fmt) {
  const int64_t per = 4 * fp4_block(fmt);
  return (cols + per - 1) / per;
}
__host__ __device__ inline int64_t fp4_scale_bytes(int64_t rows, int64_t cols, int fmt) {
  return (rows + kFp4TileRows - 1) / kFp4TileRows * fp4_tiles_k(cols, fmt) * kFp4TileBytes;
}
// byte of scale column 0 of row `row` in its tile 0
__host__ __device__ inline int64_t fp4_scale_row(int64_t row, int64_t tiles_k) {
  return (row >> 7) * tiles_k * kFp4TileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// 2^e for -127 <= e <= 127 (the lowest is a subnormal float)
__host__ __device__ __forceinline__ uint32_t pow2_bits(int e) {
  return e < -126 ? 0x00400000u : (uint32_t)(e + 127) << 23;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(pow2_bits(e)); }

// 8 values -> 8 E2M1 codes, value 0 in the lowest nibble (nearest, ties to even, saturating)
__device__ __forceinline__ uint32_t e2m1_pack8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// ... and the codes' values as 4 fp16 pairs. (One block: unpacking a word that e2m1_pack8 has
// just packed lost its upper bytes when ptxas 12.9 joined the two.)
__device__ __forceinline__ uint32_t e2m1_round8(const float* v, __half2* h) {
  uint32_t r, u[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %8, %7;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %10, %9;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %12, %11;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %4, d;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=&r"(r), "=&r"(u[0]), "=&r"(u[1]), "=&r"(u[2]), "=&r"(u[3])
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = *reinterpret_cast<const __half2*>(&u[j]);
  return r;
}
// 8 codes -> 4 fp16 pairs (exact)
__device__ __forceinline__ void e2m1_unpack8(uint32_t c, __half2* h) {
  uint32_t a, b, d, e;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "mov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(a), "=r"(b), "=r"(d), "=r"(e)
      : "r"(c));
  const uint32_t u[4] = {a, b, d, e};
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = *reinterpret_cast<const __half2*>(&u[j]);
}
__device__ __forceinline__ float ue4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ uint32_t ue4m3_code(float v) {
  return (uint32_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
// value of a block scale; 0xFF is E8M0's NaN
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t code) {
  if (FMT == BD_FP4_NV) return ue4m3_value(code);
  return code == 0xFFu ? __uint_as_float(0x7FFFFFFFu) : pow2f((int)code - 127);
}

// Limbs of a block of activations (bd_fp4.cu, bd_delta_fp4.cu): limb l has scale 2^e with the
// least e for which 6 * 2^e holds the largest magnitude of what the limbs before it left. `bits`
// are that magnitude's (6 = 1.5 * 2^2); what fp32 holds as a subnormal gives less than -127.
__device__ __forceinline__ int limb_exponent(uint32_t bits) {
  return (int)(bits >> 23) - 127 - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
}
// largest of N magnitudes, as a tree (the limbs' maxima are on their kernels' longest chain)
template <int N>
__device__ __forceinline__ float abs_max(const float* v) {
  if (N == 2) return fmaxf(fabsf(v[0]), fabsf(v[1]));
  return fmaxf(abs_max<(N > 2 ? N / 2 : 2)>(v), abs_max<(N > 2 ? N / 2 : 2)>(v + N / 2));
}
// limb l > 0 is at least 2^limb_shift(l) smaller than limb 0: the limb before leaves at most half a
// step, which is s_0 = 6 (s_0 / 4) / 1.5 after limb 0 and 4 s_{l+1} = s_l / 2 after a further one
__host__ __device__ constexpr int limb_shift(int l) { return l == 0 ? 0 : 3 * l - 1; }

// Launch plan of a 4-bit product D[W rows][X rows]. X rows are tokens, or `limbs` rows per
// token: N tile j holds h tokens from row j * n_stride, limb l of its token t in row
// (t / 8) * 8 * limbs + 8 * l + t % 8.
struct Fp4Plan {
  int pair;                     // the kernel for many X rows
  int limbs, h;                 // limb rows per token; tokens of an N tile
  int n_tile, n_stride;         // X rows of a tile (MMA N), distance of the tiles' first rows
  int tiles_n, tiles_m, kblocks, split, stages;
  int64_t ctas;
  size_t smem;
  int64_t x_rows;               // rows of the X operand (limb rows padded to whole tiles)
  size_t xc_bytes, xs_bytes;    // limb codes and scales in the workspace (0 without limbs)
};
struct Fp4Mat {                 // a packed operand: codes, tiled block scales, row scales or nullptr
  const uint8_t* codes;
  const uint8_t* scales;
  const float* row;
};
// The deltas over a 4-bit base (bd_delta_fp4.cu): segments of up to fp4_seg_tokens() tokens of
// one tenant, from the plan in the apply workspace; xc [max_tc][kFp4SegRows][d_in / 2] codes and
// xs [max_tc][scale tiles] scales of their activations' limbs.
constexpr int kFp4SegRows = 32;
__host__ __device__ constexpr int fp4_seg_tokens(int limbs) { return kFp4SegRows / limbs; }  // 8, or 5
struct DeltaFp4Args {
  const bd_tenant* tc_rec;
  const int32_t* seg;
  int max_groups, max_tc;
  const void* x;
  int64_t d_out, d_in;
  uint8_t *xc, *xs;
  const float* y_part;
  void* y;
  bool y_bf16;
  uint32_t* status;
  int64_t batch;
};
bd_status launch_delta_fp4(const DeltaFp4Args& a, int limbs, cudaStream_t s);
constexpr int kFp4LimbsBf16 = 4, kFp4LimbsF32 = 6;
Fp4Plan plan_fp4(int64_t d_out, int64_t d_in, int64_t tokens, int limbs, int fmt, bool y_bf16);
bd_status launch_fp4_limbs(const Fp4Plan& p, int fmt, const void* x, int64_t d_in, int64_t tokens, uint8_t* xc,
                           uint8_t* xs, float* xmul, uint32_t* reset_status, cudaStream_t s);
// The few-token kernel is bound by its unpacking, so its time grows with tokens * d_out * d_in;
// the limbs and tensor-core kernels cost two launches. Measured on the device, weights not in L2
// (us, few-token kernel / the others):
//                                NV            MX
//   1024 x 4096   1 token     3.0 / 6.2     2.9 / 5.8
//                 4 tokens    5.3 / 6.5     5.5 / 5.8
//   2048 x 4096   4 tokens    8.3 / 7.5     8.6 / 6.6
//   4096 x 4096   1 token     6.0 / 8.0     6.0 / 7.0
//                 2 tokens    7.4 / 8.1     7.5 / 7.1
//                 4 tokens   12.8 / 8.1    13.3 / 7.2
//   4096 x 14336  1 token    16.2 / 14.4   16.9 / 12.8
//   28672 x 4096  1 token    28.9 / 16.7   29.1 / 15.6
// The border is 2^25 for both: what it loses next to it on the device is less than the second
// launch costs the host, and the products are exact.
constexpr int64_t kFp4GemvTokens = 4;
inline bool fp4_use_gemv(int64_t d_out, int64_t d_in, int64_t tokens) {
  return tokens <= kFp4GemvTokens && tokens * d_out * d_in <= (1 << 25);
}
bd_status launch_fp4_gemv(int fmt, const Fp4Mat& w, const void* x, int64_t d_out, int64_t d_in, int64_t tokens,
                          void* y, int32_t y_dtype, uint32_t* reset_status, cudaStream_t s);
bd_status launch_fp4_mm(const Fp4Plan& p, int fmt, const Fp4Mat& w, const Fp4Mat& x, int64_t d_out, int64_t d_in,
                        int64_t tokens, void* y, int32_t y_dtype, uint32_t* status, cudaStream_t s);
// y = x W^T with bf16 x: the few-token kernel, or limbs (xc, xs, xmul: the plan's) and launch_fp4_mm
bd_status launch_fp4_linear(const Fp4Plan& p, int fmt, const Fp4Mat& w, const void* x, int64_t d_out, int64_t d_in,
                            int64_t tokens, uint8_t* xc, uint8_t* xs, float* xmul, void* y, int32_t y_dtype,
                            uint32_t* reset_status, uint32_t* status, cudaStream_t s);

}  // namespace bd
