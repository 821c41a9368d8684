// Products of microscaled 4-bit matrices on the tensor cores: D = W_hat X_hat^T with
// tcgen05.mma kind::mxf4nvf4 (block 16, UE4M3 scales) or kind::mxf4 (block 32, E8M0 scales),
// fp32 accumulation in tensor memory.
//
// One CTA owns a 128-row block of W and n_tile rows of X and a range of K; the CTAs of a
// cluster split K. Warp 0 issues the loads of a 256-column stage (codes by TMA with the
// 128-byte swizzle, their block scales by plain bulk copies: the tiled layout keeps a
// stage's scales of 128 rows contiguous), warp 1 copies the scales to tensor memory
// (tcgen05.cp) and issues the four K = 64 MMAs. The epilogue adds the limbs of a token; with
// a split, each CTA leaves its fp32 sums in its own shared memory and the CTAs of the cluster
// add them in rank order over distributed shared memory, so results do not depend on timing.
#include "bd_fp4.cuh"
#include "bd_tc.cuh"

namespace bd {

constexpr int kMmThreads = 128;
constexpr uint32_t kMmABytes = 128 * 128;  // W codes of a stage

// D[tmem] (+)= (A * SFA) (B * SFB), 4-bit operands with block scales in tensor memory
template <int FMT>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (FMT == BD_FP4_NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// one 512-byte scale tile (32 rows of 16 bytes) -> 4 columns of tensor memory, repeated in
// all four 32-lane quarters; ordered before the MMAs that this thread issues next
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// shared-memory descriptor of a scale tile: no swizzle, 8-row core matrices 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  return d;
}

// Instruction descriptor of the block-scaled 4-bit kinds: A and B E2M1, K-major; scale ids
// select the byte pair of a scale word (block 32: two K steps share a word).
__host__ __device__ constexpr uint32_t umma_idesc_fp4(int m, int n, bool e8m0, int sf_id) {
  return ((uint32_t)sf_id << 4)           // B scale id
         | (1u << 7)                      // A format: E2M1
         | (1u << 10)                     // B format: E2M1
         | ((uint32_t)(n >> 3) << 17)     // N / 8
         | ((e8m0 ? 1u : 0u) << 23)       // scale format
         | ((uint32_t)(m >> 4) << 24)     // M / 16
         | ((uint32_t)sf_id << 29);       // A scale id
}

// 32 lanes x 8 consecutive 32-bit columns of tensor memory
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* r) {
  uint32_t u[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __uint_as_float(u[j]);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

struct MmArgs {
  const uint8_t *w_scales, *x_scales;
  const float *w_row, *x_row;
  void* y;
  uint32_t* status;
  int64_t d_out, tokens;
  int tiles_kw;                        // scale tiles along K
  int limbs, h, n_tile, n_stride, kblocks, k_steps, split, stages, y_bf16;
  int x_row_tiles;                     // scale tiles along the rows of X
};

template <int FMT>
__global__ void __launch_bounds__(kMmThreads) k_fp4_mm(const __grid_constant__ CUtensorMap tm_w,
                                                       const __grid_constant__ CUtensorMap tm_x, const MmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kTilesPerStage = FMT == BD_FP4_NV ? 4 : 2;   // scale tiles of a stage, per 128 rows
  constexpr uint32_t kSfBytes = kTilesPerStage * kFp4TileBytes;
  const int sfb_tiles = (p.n_tile + 127) / 128;              // 128-row scale tiles of the X rows
  const uint32_t b_bytes = (uint32_t)p.n_tile * 128u;
  const int stages = p.stages;
  uint8_t* sa = smem;
  uint8_t* sb = sa + (size_t)stages * kMmABytes;
  uint8_t* ssa = sb + (size_t)stages * b_bytes;
  uint8_t* ssb = ssa + (size_t)stages * kSfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ssb + (size_t)stages * sfb_tiles * kSfBytes);
  uint64_t* empty = full + stages;
  uint64_t* done = empty + stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued_out = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int64_t item = blockIdx.x / split;
  const int tiles_n = (int)((p.tokens + p.h - 1) / p.h);
  const int n_blk = (int)(item % tiles_n);
  const int64_t m_blk = item / tiles_n;
  const int kb0 = (int)((int64_t)p.kblocks * rank / split), kb1 = (int)((int64_t)p.kblocks * (rank + 1) / split);
  const int nkb = kb1 - kb0;  // >= 1: split <= kblocks

  // tensor memory: D, then two buffers of the scales of a stage
  const uint32_t d_cols = (uint32_t)(p.n_tile + 31) & ~31u;
  constexpr uint32_t kSfaCols = kTilesPerStage * 4;
  const uint32_t sf_cols = kSfaCols * (1 + sfb_tiles);
  uint32_t tcols = 32;
  while (tcols < d_cols + 2 * sf_cols) tcols <<= 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    *issued_out = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, tcols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  pdl_wait();  // the set-up above overlaps the previous kernel on the stream
  pdl_trigger();

  bool timed_out = false;
  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      const int64_t x_row0 = (int64_t)n_blk * p.n_stride;
      for (int i = 0; i < nkb; ++i) {
        const int s = i % stages;
        const uint32_t ph = (uint32_t)(i / stages) & 1u;
        if (i >= stages && !mbar_wait(&empty[s], ph ^ 1u, abort_flag)) {
          timed_out = true;
          *abort_flag = 1;
          break;
        }
        const int kb = kb0 + i;
        const int t0 = kb * kTilesPerStage;
        const uint32_t sf = (uint32_t)min(kTilesPerStage, p.tiles_kw - t0) * kFp4TileBytes;
        const int xt0 = (int)(x_row0 >> 7);
        const int xt = min(sfb_tiles, p.x_row_tiles - xt0);
        mbar_arrive_expect_tx(&full[s], kMmABytes + b_bytes + sf * (1 + xt));
        tma_load_2d(sa + (size_t)s * kMmABytes, &tm_w, &full[s], kb * 128, (int)(m_blk * 128));
        bulk_load(ssa + (size_t)s * kSfBytes, p.w_scales + ((int64_t)m_blk * p.tiles_kw + t0) * kFp4TileBytes, sf,
                  &full[s]);
        tma_load_2d(sb + (size_t)s * b_bytes, &tm_x, &full[s], kb * 128, (int)x_row0);
        for (int j = 0; j < xt; ++j)
          bulk_load(ssb + ((size_t)s * sfb_tiles + j) * kSfBytes,
                    p.x_scales + ((int64_t)(xt0 + j) * p.tiles_kw + t0) * kFp4TileBytes, sf, &full[s]);
        ++issued;
      }
      *issued_out = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id0 = umma_idesc_fp4(128, p.n_tile, FMT == BD_FP4_MX, 0);
      const uint32_t id1 = umma_idesc_fp4(128, p.n_tile, FMT == BD_FP4_MX, 2);
      for (int i = 0; i < nkb; ++i) {
        const int s = i % stages;
        const uint32_t ph = (uint32_t)(i / stages) & 1u;
        if (!mbar_wait(&full[s], ph, abort_flag)) {
          timed_out = true;
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        // scales: SFA tile of a step in 4 columns, SFB likewise per 128 rows, steps apart
        const uint32_t sfa = tmem_d + d_cols + (uint32_t)(i & 1) * sf_cols;
        const uint32_t sfb = sfa + kSfaCols;
        const int steps = min(4, p.k_steps - (kb0 + i) * 4);
        const int sf_tiles = FMT == BD_FP4_NV ? steps : (steps + 1) / 2;
        for (int t = 0; t < sf_tiles; ++t) {
          tmem_cp_scales(sfa + 4 * t, scale_desc(smem_u32(ssa + (size_t)s * kSfBytes + t * kFp4TileBytes)));
          for (int j = 0; j < sfb_tiles; ++j)
            tmem_cp_scales(sfb + 4 * (t * sfb_tiles + j),
                           scale_desc(smem_u32(ssb + ((size_t)s * sfb_tiles + j) * kSfBytes + t * kFp4TileBytes)));
        }
        const uint64_t ad = umma_desc_sw128(smem_u32(sa + (size_t)s * kMmABytes));
        const uint64_t bdsc = umma_desc_sw128(smem_u32(sb + (size_t)s * b_bytes));
        for (int k = 0; k < steps; ++k) {
          // 64 columns: 32 bytes further inside the swizzled 128-byte row
          const int t = FMT == BD_FP4_NV ? k : k >> 1;
          umma_fp4<FMT>(tmem_d, ad + (uint64_t)(2 * k), bdsc + (uint64_t)(2 * k),
                        FMT == BD_FP4_MX && (k & 1) ? id1 : id0, sfa + 4 * t, sfb + 4 * (t * sfb_tiles),
                        (i > 0 || k > 0) ? 1u : 0u);
        }
        umma_commit(&empty[s]);
      }
      umma_commit(done);
    }
    __syncwarp();
  }

  const bool ok = mbar_wait(done, 0, nullptr);
  tc_fence_after();
  if (!ok) timed_out = true;
  if (timed_out) *abort_flag = 1;
  __syncthreads();
  const bool aborted = *abort_flag != 0;
  if (aborted && threadIdx.x == 0) {
    atomicOr(p.status, BD_DEV_TIMEOUT);
    // every load this CTA issued lands before its shared memory is used again or goes away
    const int issued = *issued_out;
    for (int i = max(0, issued - stages); i < issued; ++i)
      mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u, nullptr);
  }

  const int64_t t0 = (int64_t)n_blk * p.h;
  const int n_tok = (int)min((int64_t)p.h, p.tokens - t0);
  const uint32_t lane_addr = tmem_d + ((uint32_t)(warp * 32) << 16);
  if (split == 1) {
    const int64_t row = m_blk * 128 + threadIdx.x;
    const bool in = row < p.d_out && !aborted;
    const float rs = in && p.w_row ? p.w_row[row] : 1.f;
    for (int c0 = 0; c0 < n_tok; c0 += 8) {
      float v[8];
      for (int l = 0; l < p.limbs; ++l) {
        float u[8];
        tmem_ld8(lane_addr + (uint32_t)(l * p.h + c0), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = l == 0 ? u[j] : v[j] + u[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (in && c0 + j < n_tok) {
          const int64_t t = t0 + c0 + j;
          const float o = v[j] * rs * (p.x_row ? p.x_row[t] : 1.f);
          if (p.y_bf16)
            reinterpret_cast<uint16_t*>(p.y)[t * p.d_out + row] = (uint16_t)f2bf_bits(o);
          else
            reinterpret_cast<float*>(p.y)[t * p.d_out + row] = o;
        }
      }
    }
  } else {
    // sums [token][128 rows] in the (now unused) stage buffers
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
    for (int c0 = 0; c0 < n_tok; c0 += 8) {
      float v[8];
      for (int l = 0; l < p.limbs; ++l) {
        float u[8];
        tmem_ld8(lane_addr + (uint32_t)(l * p.h + c0), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = l == 0 ? u[j] : v[j] + u[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < n_tok) part[(c0 + j) * 128 + threadIdx.x] = v[j];
    }
    // tensor memory goes back before the CTAs wait for one another: a CTA that held it while
    // waiting could keep one of another cluster's CTAs, and so that cluster, from starting
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem_d, tcols);
    cluster_sync_all();
    const int64_t row = m_blk * 128 + threadIdx.x;
    const bool in = row < p.d_out && !aborted;
    const float rs = in && p.w_row ? p.w_row[row] : 1.f;
    for (int j = rank; j < n_tok; j += split) {
      const uint32_t at = smem_u32(part + j * 128 + threadIdx.x);
      float v = 0.f;
      for (int r = 0; r < split; ++r) v += ld_cluster_f32(at, (uint32_t)r);
      if (in) {
        const int64_t t = t0 + j;
        const float o = v * rs * (p.x_row ? p.x_row[t] : 1.f);
        if (p.y_bf16)
          reinterpret_cast<uint16_t*>(p.y)[t * p.d_out + row] = (uint16_t)f2bf_bits(o);
        else
          reinterpret_cast<float*>(p.y)[t * p.d_out + row] = o;
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
  }
  if (split == 1) {
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem_d, tcols);
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
static bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows) {
  TensorMapEncodeFn enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Fp4Plan plan_fp4(int64_t d_out, int64_t d_in, int64_t tokens, int limbs, int fmt) {
  Fp4Plan p;
  p.limbs = limbs;
  // tokens of an N tile: as many as fit 256 X rows, in steps of 8 (16 without limbs), all
  // tokens in one tile when they fit
  const int step = limbs > 1 ? 8 : 16;
  const int most = limbs > 1 ? 256 / limbs / 8 * 8 : 256;
  p.h = (int)((tokens + step - 1) / step * step);
  if (p.h > most) p.h = most;
  if (limbs == 1 && p.h > 128) p.h = 256;  // X rows of a tile start at a scale tile
  p.n_tile = p.h * limbs;
  p.n_stride = limbs > 1 ? (p.n_tile + 127) / 128 * 128 : p.n_tile;
  p.tiles_n = (int)((tokens + p.h - 1) / p.h);
  p.tiles_m = (int)((d_out + 127) / 128);
  p.kblocks = (int)((d_in + kFp4KStage - 1) / kFp4KStage);
  p.x_rows = limbs > 1 ? (int64_t)p.tiles_n * p.n_stride : tokens;
  p.xc_bytes = limbs > 1 ? align_up((size_t)p.x_rows * (size_t)(d_in / 2), 256) : 0;
  p.xs_bytes = limbs > 1 ? (size_t)fp4_scale_bytes(p.x_rows, d_in, fmt) : 0;
  const int64_t tiles = (int64_t)p.tiles_n * p.tiles_m;
  p.split = 1;
  while (p.split < 8 && p.split * 2 <= p.kblocks && tiles * p.split < sm_count()) p.split *= 2;
  const int sf = (fmt == BD_FP4_NV ? 4 : 2) * kFp4TileBytes;
  const size_t stage = kMmABytes + (size_t)p.n_tile * 128 + (size_t)sf * (1 + (p.n_tile + 127) / 128);
  int st = (int)((200 * 1024) / stage);
  const int need = (p.kblocks + p.split - 1) / p.split;
  if (st > need) st = need;
  if (st > 8) st = 8;
  p.stages = st;
  size_t bytes = (size_t)st * stage;
  if (p.split > 1 && bytes < (size_t)p.h * 512) bytes = (size_t)p.h * 512;
  p.smem = 1024 + bytes + (2 * st + 1) * 8 + 16;
  return p;
}

bd_status launch_fp4_mm(const Fp4Plan& p, int fmt, const Fp4Mat& w, const Fp4Mat& x, int64_t d_out, int64_t d_in,
                        int64_t tokens, void* y, int32_t y_dtype, uint32_t* status, cudaStream_t s) {
  CUtensorMap tw, tx;
  if (!encode_codes(&tw, w.codes, d_out, d_in / 2, 128)) return BD_ERR_CUDA;
  if (!encode_codes(&tx, x.codes, p.x_rows, d_in / 2, p.n_tile)) return BD_ERR_CUDA;
  static std::atomic<uint64_t> attr_nv{0}, attr_mx{0};
  auto* fn = fmt == BD_FP4_NV ? k_fp4_mm<BD_FP4_NV> : k_fp4_mm<BD_FP4_MX>;
  if (!ensure_dyn_smem(fn, 227 * 1024, fmt == BD_FP4_NV ? attr_nv : attr_mx)) return BD_ERR_CUDA;
  MmArgs a;
  a.w_scales = w.scales;
  a.x_scales = x.scales;
  a.w_row = w.row;
  a.x_row = x.row;
  a.y = y;
  a.status = status;
  a.d_out = d_out;
  a.tokens = tokens;
  a.tiles_kw = (int)fp4_tiles_k(d_in, fmt);
  a.limbs = p.limbs;
  a.h = p.h;
  a.n_tile = p.n_tile;
  a.n_stride = p.n_stride;
  a.kblocks = p.kblocks;
  a.k_steps = (int)((d_in + 63) / 64);
  a.split = p.split;
  a.stages = p.stages;
  a.y_bf16 = y_dtype == BD_BF16;
  a.x_row_tiles = (int)((p.x_rows + 127) / 128);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.tiles_m * p.tiles_n * p.split));
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  launch_begin(K_FP4_MM, s);
  BD_CUDA_TRY(cudaLaunchKernelEx(&cfg, fn, tw, tx, a));
  launch_end(K_FP4_MM, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

namespace {
// arguments of both products; BD_OK and *nothing = true for an empty batch
bd_status check_mm(const Fp4Mat& w, int32_t fmt, int64_t d_out, int64_t d_in, int64_t tokens, const void* x,
                   const void* y, int32_t y_dtype, const void* workspace, size_t ws_bytes, size_t need) {
  if (y_dtype != BD_BF16 && y_dtype != BD_F32) return BD_ERR_DTYPE;
  if (fmt != BD_FP4_NV && fmt != BD_FP4_MX) return BD_ERR_CONFIG;
  if (d_out < 1 || d_out > kFp4MaxDim || d_in < 32 || d_in > kFp4MaxDim || (d_in % 32) != 0) return BD_ERR_SHAPE;
  if (tokens < 0 || tokens > kFp4MaxTokens) return BD_ERR_SHAPE;
  if (tokens == 0) return BD_OK;
  if (!w.codes || !w.scales || !x || !y) return BD_ERR_NULL;
  if (!aligned16(w.codes) || !aligned16(w.scales) || !aligned16(x) || !aligned16(y) ||
      (reinterpret_cast<uintptr_t>(w.row) & 3u))
    return BD_ERR_ALIGN;
  if (!workspace || ws_bytes < need) return BD_ERR_WORKSPACE;
  if (!aligned16(workspace)) return BD_ERR_ALIGN;
  return BD_OK;
}
struct LinearLayout {
  Fp4Plan p;
  size_t off_c, off_s, off_mul, total;
};
LinearLayout layout_linear(int64_t d_out, int64_t d_in, int64_t tokens, int32_t y_dtype, int fmt) {
  LinearLayout L;
  L.p = plan_fp4(d_out, d_in, tokens, y_dtype == BD_F32 ? kFp4LimbsF32 : kFp4LimbsBf16, fmt);
  L.off_c = kStatusBytes;
  L.off_s = L.off_c + L.p.xc_bytes;
  L.off_mul = L.off_s + L.p.xs_bytes;
  L.total = align_up(L.off_mul + (size_t)tokens * 4, 256);
  return L;
}
}  // namespace

}  // namespace bd

extern "C" size_t bd_matmul_fp4_workspace_size(int64_t d_out, int64_t d_in, int64_t tokens) {
  using namespace bd;
  if (d_out < 1 || d_in < 32 || tokens < 0) return 0;
  return kStatusBytes;
}

extern "C" bd_status bd_matmul_fp4(const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scales,
                                   const uint8_t* x_codes, const uint8_t* x_scales, const float* x_row_scales,
                                   int32_t fmt, int64_t d_out, int64_t d_in, int64_t tokens, void* y,
                                   int32_t y_dtype, void* workspace, size_t ws_bytes, void* stream) {
  using namespace bd;
  const Fp4Mat w{w_codes, w_scales, w_row_scales}, x{x_codes, x_scales, x_row_scales};
  const bd_status st = check_mm(w, fmt, d_out, d_in, tokens, x_codes, y, y_dtype, workspace, ws_bytes, kStatusBytes);
  if (st != BD_OK || tokens == 0) return st;
  if (!x_scales) return BD_ERR_NULL;
  if (!aligned16(x_scales) || (reinterpret_cast<uintptr_t>(x_row_scales) & 3u)) return BD_ERR_ALIGN;
  return launch_fp4_mm(plan_fp4(d_out, d_in, tokens, 1, fmt), fmt, w, x, d_out, d_in, tokens, y, y_dtype,
                       static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(stream));
}

extern "C" size_t bd_linear_fp4_workspace_size(int64_t d_out, int64_t d_in, int64_t tokens) {
  using namespace bd;
  if (d_out < 1 || d_out > kFp4MaxDim || d_in < 32 || d_in > kFp4MaxDim || (d_in % 32) != 0 || tokens < 0 ||
      tokens > kFp4MaxTokens)
    return 0;
  if (tokens == 0) return kStatusBytes;
  size_t most = 0;
  for (int fmt = BD_FP4_NV; fmt <= BD_FP4_MX; ++fmt)
    for (int dt = BD_F32; dt <= BD_BF16; ++dt) {
      const size_t n = layout_linear(d_out, d_in, tokens, dt, fmt).total;
      if (n > most) most = n;
    }
  return most;
}

extern "C" bd_status bd_linear_fp4(const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scales,
                                   int32_t fmt, int64_t d_out, int64_t d_in, const void* x, int64_t tokens, void* y,
                                   int32_t y_dtype, void* workspace, size_t ws_bytes, void* stream) {
  using namespace bd;
  const Fp4Mat w{w_codes, w_scales, w_row_scales};
  // (a shape that check_mm refuses has no layout)
  const bool plannable = d_out >= 1 && d_out <= kFp4MaxDim && d_in >= 32 && d_in <= kFp4MaxDim && tokens > 0 &&
                         tokens <= kFp4MaxTokens && (fmt == BD_FP4_NV || fmt == BD_FP4_MX);
  LinearLayout L = {};
  if (plannable) L = layout_linear(d_out, d_in, tokens, y_dtype, fmt);
  const bd_status st = check_mm(w, fmt, d_out, d_in, tokens, x, y, y_dtype, workspace, ws_bytes, L.total);
  if (st != BD_OK || tokens == 0) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  float* xmul = reinterpret_cast<float*>(ws + L.off_mul);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bd_status r = launch_fp4_limbs(L.p, fmt, x, d_in, tokens, ws + L.off_c, ws + L.off_s, xmul, status, s);
  if (r != BD_OK) return r;
  return launch_fp4_mm(L.p, fmt, w, Fp4Mat{ws + L.off_c, ws + L.off_s, xmul}, d_out, d_in, tokens, y, y_dtype,
                       status, s);
}
