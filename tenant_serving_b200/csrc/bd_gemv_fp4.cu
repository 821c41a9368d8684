// y[t] = W_hat x[t] for a few bf16 tokens, W microscaled 4-bit, on the CUDA cores.
//
// With so few tokens the product is one pass over W: unpack, multiply in fp32 (a code times a
// bf16 value is exact there), add. It needs no limbs, so one launch instead of two, and no
// rounding but that of the fp32 sums.
//
// One CTA per four rows r, r + 32, r + 64, r + 96 of a 128-row tile, whose scales of four
// blocks are 16 neighbouring bytes of the tiled layout; four warps take 256-column steps in
// turn, a lane 8 columns of each row, and add their sums in warp order. Loads of several steps
// are in flight before the first is used. Bound by the unpacking (about 8 issue slots per 32
// weights, half of them E2M1 -> fp16 conversions), so it is for small products only, see
// fp4_use_gemv(): one token on 4096 x 4096 takes 5.3-6.1 us on the device (its bytes 1.4) and
// 9.2 per call from Python, where the limbs and tensor-core kernels take 7.6 and 11.5.
#include "bd_fp4.cuh"

namespace bd {

constexpr int kGvThreads = 128, kGvWarps = kGvThreads / 32, kGvStep = 256;

__device__ __forceinline__ uint32_t ldg_stream32(const void* p) {
  uint32_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

template <int FMT, int T>
__global__ void __launch_bounds__(kGvThreads) k_fp4_gemv(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         const float* __restrict__ w_row,
                                                         const uint16_t* __restrict__ x, int64_t d_out, int64_t d_in,
                                                         void* __restrict__ y, bool y_bf16,
                                                         uint32_t* __restrict__ reset_status) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  if (reset_status && blockIdx.x == 0 && threadIdx.x == 0) *reset_status = 0;  // reports this call
  constexpr int U = T <= 2 ? 4 : 2;  // steps in flight
  constexpr int kBlock = fp4_block(FMT);
  __shared__ float red[kGvWarps][5 * T];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x >> 5, row0 = tile * kFp4TileRows + (blockIdx.x & 31);
  if (row0 >= d_out) return;
  const uint8_t* sr = scales + tile * fp4_tiles_k(d_in, FMT) * kFp4TileBytes + (blockIdx.x & 31) * 16;
  const uint8_t* wr[4];  // (a row past the last one reads the first again)
#pragma unroll
  for (int i = 0; i < 4; ++i) wr[i] = codes + (row0 + 32 * i < d_out ? row0 + 32 * i : row0) * (d_in >> 1);
  // The sums of a token near fp32's largest number can pass it before the row's scale brings them
  // back: a CTA that ends with some that are not finite takes those from a second pass with the
  // tokens 2^64 smaller.
  const int oi = threadIdx.x / T, ot = threadIdx.x % T;  // threads below 4 T: an output each
  float v = 0.f, bad = 0.f, post = 1.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float acc[4][T], nan[T];  // nan: 0, or NaN once a value of the token is not finite
#pragma unroll
    for (int t = 0; t < T; ++t) {
      nan[t] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][t] = 0.f;
    }
    for (int64_t c0 = warp * kGvStep + lane * 8; c0 < d_in; c0 += U * kGvWarps * kGvStep) {
      uint32_t w[U][4];
      uint4 s[U], xv[U][T];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * kGvWarps * kGvStep;
        s[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[u][i] = 0u;
#pragma unroll
        for (int t = 0; t < T; ++t) xv[u][t] = make_uint4(0u, 0u, 0u, 0u);
        if (c < d_in) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[u][i] = ldg_stream32(wr[i] + (c >> 1));
          s[u] = __ldg(reinterpret_cast<const uint4*>(sr + c / (4 * kBlock) * kFp4TileBytes));
#pragma unroll
          for (int t = 0; t < T; ++t) xv[u][t] = __ldg(reinterpret_cast<const uint4*>(x + t * d_in + c));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int shift = (int)((c0 + u * kGvWarps * kGvStep) / kBlock & 3) * 8;
        float xf[T][8];
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const uint32_t a[4] = {xv[u][t].x, xv[u][t].y, xv[u][t].z, xv[u][t].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xf[t][2 * j] = bf16lo(a[j]);
            xf[t][2 * j + 1] = bf16hi(a[j]);
            nan[t] = fmaf(xf[t][2 * j], 0.f, nan[t]);
            nan[t] = fmaf(xf[t][2 * j + 1], 0.f, nan[t]);
          }
        }
        if (pass > 0) {
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) xf[t][j] *= 0x1p-64f;
        }
        const uint32_t sw[4] = {s[u].x, s[u].y, s[u].z, s[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __half2 h[4];
          e2m1_unpack8(w[u][i], h);
          float e[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            e[2 * j] = f.x;
            e[2 * j + 1] = f.y;
          }
          const float sc = fp4_scale_value<FMT>((sw[i] >> shift) & 0xFFu);
#pragma unroll
          for (int t = 0; t < T; ++t) {
            float d = e[0] * xf[t][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) d = fmaf(e[j], xf[t][j], d);
            acc[i][t] = fmaf(sc, d, acc[i][t]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = warp_sum_f(acc[i][t]);
        if (lane == 0) red[warp][i * T + t] = v;
      }
      const float v = warp_sum_f(nan[t]);
      if (lane == 0) red[warp][4 * T + t] = v;
    }
    __syncthreads();
    const auto finite = [](float f) { return (__float_as_uint(f) & 0x7FFFFFFFu) < 0x7F800000u; };
    if (threadIdx.x < 4 * T && (pass == 0 || !finite(v))) {
      v = bad = 0.f;
#pragma unroll
      for (int k = 0; k < kGvWarps; ++k) {
        v += red[k][oi * T + ot];
        bad += red[k][4 * T + ot];
      }
      if (pass > 0) post = 0x1p64f;
    }
    if (!__syncthreads_or(!finite(v))) break;
  }
  const int64_t row = row0 + 32 * oi;
  if (threadIdx.x < 4 * T && row < d_out) {
    if (w_row) v *= w_row[row];
    v = v * post + bad;
    if (y_bf16)
      reinterpret_cast<uint16_t*>(y)[ot * d_out + row] = (uint16_t)f2bf_bits(v);
    else
      reinterpret_cast<float*>(y)[ot * d_out + row] = v;
  }
}

template <int FMT>
static cudaError_t launch_gemv(const Fp4Mat& w, const void* x, int64_t d_out, int64_t d_in, int64_t tokens, void* y,
                               bool y_bf16, uint32_t* reset_status, cudaStream_t s) {
  auto* fn = tokens == 1 ? k_fp4_gemv<FMT, 1>
           : tokens == 2 ? k_fp4_gemv<FMT, 2>
           : tokens == 3 ? k_fp4_gemv<FMT, 3>
                         : k_fp4_gemv<FMT, 4>;
  static_assert(kFp4GemvTokens == 4, "");
  const int64_t tiles = (d_out + kFp4TileRows - 1) / kFp4TileRows;
  return launch_pdl(fn, dim3((unsigned)(tiles * 32)), dim3(kGvThreads), 0, s, w.codes, w.scales, w.row,
                    static_cast<const uint16_t*>(x), d_out, d_in, y, y_bf16, reset_status);
}

bd_status launch_fp4_gemv(int fmt, const Fp4Mat& w, const void* x, int64_t d_out, int64_t d_in, int64_t tokens,
                          void* y, int32_t y_dtype, uint32_t* reset_status, cudaStream_t s) {
  launch_begin(K_FP4_GEMV, s);
  BD_CUDA_TRY(fmt == BD_FP4_NV ? launch_gemv<BD_FP4_NV>(w, x, d_out, d_in, tokens, y, y_dtype == BD_BF16, reset_status, s)
                               : launch_gemv<BD_FP4_MX>(w, x, d_out, d_in, tokens, y, y_dtype == BD_BF16, reset_status, s));
  launch_end(K_FP4_GEMV, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

}  // namespace bd
