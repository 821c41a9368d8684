// Products of microscaled 4-bit matrices on the tensor cores: D = W_hat X_hat^T with
// tcgen05.mma kind::mxf4nvf4 (block 16, UE4M3 scales) or kind::mxf4 (block 32, E8M0 scales),
// fp32 accumulation in tensor memory.
//
// Two kernels:
//   k_fp4_mm_rows  few X rows (one N tile of at most 256): bound by reading W. One CTA per
//                  (128-row block of W, N tile, K range); the CTAs of a cluster split K and
//                  add their fp32 sums in rank order in distributed shared memory.
//   k_fp4_mm_pair  many X rows: bound by the tensor cores' power and by what an SM can load.
//                  Persistent CTA pairs (cta_group::2), a 256 x 256 tile each.
// In both, warp 0 issues the loads of 256-column stages (codes with the 128-byte swizzle, and
// their block scales, which the tiled layout keeps contiguous) and warp 1 copies the scales to
// tensor memory (tcgen05.cp) and issues the four K = 64 MMAs of a stage. No sum depends on
// timing.
//
// X rows are tokens, or limbs of tokens in groups of 8: rows 8 L g + 8 l + j of a tile are
// limb l of its token 8 g + j, so a group's sums are 8 L neighbouring accumulator columns.
#include "bd_fp4.cuh"
#include "bd_fp4_mma.cuh"
#include "bd_tc.cuh"

namespace bd {

constexpr int kMmThreads = 256;
constexpr uint32_t kMmABytes = 128 * 128;  // W codes of a stage
constexpr int kMaxSplit = 8;               // CTAs of a cluster that split K (a power of two)

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

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t map_cluster(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}

// Accumulator columns come in groups that hold whole tokens: 32 tokens without limbs, else
// the 8 L columns of 8 tokens.
template <int L>
struct Group {
  static constexpr int kCols = L == 1 ? 32 : 8 * L;
  static constexpr int kTok = kCols / L;
};
// Sums of a group's tokens, the smallest limb first. In BD_FP4_NV limb l's columns are
// 2^limb_shift(l) too large: each step takes what lies between two limbs off.
template <int FMT, int L>
__device__ __forceinline__ void load_group(uint32_t taddr, float* v) {
  uint32_t r[Group<L>::kCols];
  tmem_load<32>(taddr, r);
  if (L == 6) tmem_load<16>(taddr + 32, r + 32);
  tmem_wait();
#pragma unroll
  for (int j = 0; j < Group<L>::kTok; ++j) {
    float a = __uint_as_float(r[8 * (L - 1) + j]);
#pragma unroll
    for (int l = L - 2; l >= 0; --l) {
      const float down = FMT == BD_FP4_NV ? 1.f / (float)(1 << (limb_shift(l + 1) - limb_shift(l))) : 1.f;
      a = fmaf(a, down, __uint_as_float(r[8 * l + j]));
    }
    v[j] = a;
  }
}

// v * a * b, the scales of a row and a token, without leaving fp32's range on the way to a result
// inside it: the scales' product first, or one after the other where that is no normal number. Then
// both are large, or one is below 2^-63 (or zero) and the other any number that cannot make up for
// it: the smaller one goes first where v is large or a scale is zero, else the larger one.
__device__ __forceinline__ float scaled(float v, float a, float b) {
  const float q = a * b, m = fabsf(q);
  if (m >= 0x1p-126f && m <= 0x1.fffffep127f) return v * q;
  const bool smaller = fabsf(v) >= 0x1p60f || a == 0.f || b == 0.f;
  return (fabsf(a) > fabsf(b)) != smaller ? v * a * b : v * b * a;
}
template <bool B>
struct Flag {
  static constexpr bool value = B;
};
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct MmArgs {
  const uint8_t *w_scales, *x_scales;
  const float *w_row, *x_row;
  void* y;
  uint32_t* status;
  int64_t d_out, tokens;
  int tiles_kw;     // scale tiles along K
  int x_row_tiles;  // scale tiles along the rows of X
  int h, n_tile, n_stride, tiles_n, kblocks, k_steps, split, stages, y_bf16;
  int w_early;      // nothing still running on the stream writes W or its scales
  int y_tma;        // y's rows are whole 16-byte units: tiles go out through tm_y
};

__device__ __forceinline__ void store_y(const MmArgs& p, int64_t t, int64_t row, float v) {
  if (p.y_bf16)
    reinterpret_cast<uint16_t*>(p.y)[t * p.d_out + row] = (uint16_t)f2bf_bits(v);
  else
    reinterpret_cast<float*>(p.y)[t * p.d_out + row] = v;
}

// four consecutive rows of a token
__device__ __forceinline__ void store_y4(const MmArgs& p, int64_t t, int64_t row, float4 v) {
  if ((p.d_out & 3) == 0) {
    if (row >= p.d_out) return;
    if (p.y_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.y) + t * p.d_out + row) =
          make_uint2(f2bf_bits(v.x) | (f2bf_bits(v.y) << 16), f2bf_bits(v.z) | (f2bf_bits(v.w) << 16));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.y) + t * p.d_out + row) = v;
    return;
  }
  const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (row + q < p.d_out) store_y(p, t, row + q, a[q]);
}

// ------------------------------------------------------------------------------------
// few X rows
// ------------------------------------------------------------------------------------
template <int FMT, int L>
__global__ void __launch_bounds__(kMmThreads) k_fp4_mm_rows(const __grid_constant__ CUtensorMap tm_w,
                                                            const __grid_constant__ CUtensorMap tm_x,
                                                            const MmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kTilesPerStage = FMT == BD_FP4_NV ? 4 : 2;   // scale tiles of a stage, per 128 rows
  constexpr uint32_t kSfBytes = kTilesPerStage * kFp4TileBytes;
  const int sfb_tiles = (p.n_tile + 127) / 128;              // 128-row scale tiles of the X rows
  const uint32_t b_bytes = (uint32_t)p.n_tile * 128u;
  const int stages = p.stages, split = p.split;
  uint8_t* sa = smem;
  uint8_t* sb = sa + (size_t)stages * kMmABytes;
  uint8_t* ssa = sb + (size_t)stages * b_bytes;
  uint8_t* ssb = ssa + (size_t)stages * kSfBytes;
  // with a split: this CTA's share of the tile's sums from every CTA, [rank][share][128 rows]
  float* gather = reinterpret_cast<float*>(ssb + (size_t)stages * sfb_tiles * kSfBytes);
  const int share = split > 1 ? (p.h + split - 1) / split : 0;  // tokens of a CTA
  float* xr = gather + (size_t)split * share * 128;             // the tile's token scales
  uint64_t* full = reinterpret_cast<uint64_t*>(xr + p.h);
  uint64_t* empty = full + stages;
  uint64_t* done = empty + stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued_out = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int64_t item = blockIdx.x / split;
  const int n_blk = (int)(item % p.tiles_n);
  const int64_t m_blk = item / p.tiles_n;
  const int kb0 = (int)((int64_t)p.kblocks * rank / split), kb1 = (int)((int64_t)p.kblocks * (rank + 1) / split);
  const int nkb = kb1 - kb0;  // >= 1: split <= kblocks

  // tensor memory: D, then two buffers of the scales of a stage
  const uint32_t d_cols = (uint32_t)(p.n_tile + 31) & ~31u;
  constexpr uint32_t kSfaCols = kTilesPerStage * 4;
  const uint32_t sf_cols = kSfaCols * (1 + sfb_tiles);
  uint32_t tcols = 32;
  while (tcols < d_cols + 2 * sf_cols) tcols <<= 1;

  if (split > 1) cluster_arrive();  // this CTA has started
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

  bool timed_out = false;
  if (warp == 0) {
    const int64_t x_row0 = (int64_t)n_blk * p.n_stride;
    const int xt0 = (int)(x_row0 >> 7);
    const int xt = min(sfb_tiles, p.x_row_tiles - xt0);
    auto sf_of = [&](int i) {
      return (uint32_t)min(kTilesPerStage, p.tiles_kw - (kb0 + i) * kTilesPerStage) * kFp4TileBytes;
    };
    auto load_w = [&](int i) {
      const int s = i % stages;
      const uint32_t sf = sf_of(i);
      mbar_arrive_expect_tx(&full[s], kMmABytes + b_bytes + sf * (1 + xt));
      tma_load_2d(sa + (size_t)s * kMmABytes, &tm_w, &full[s], (kb0 + i) * 128, (int)(m_blk * 128));
      bulk_load(ssa + (size_t)s * kSfBytes,
                p.w_scales + (m_blk * p.tiles_kw + (int64_t)(kb0 + i) * kTilesPerStage) * kFp4TileBytes, sf, &full[s]);
    };
    // the weights of the first stages are asked for before the kernel that writes X is over
    const int first = min(nkb, stages);
    int early = 0;
    if (p.w_early) {
      if (elect_one())
        for (int i = 0; i < first; ++i) load_w(i);
      __syncwarp();
      early = first;
    }
    pdl_wait();
    pdl_trigger();
    int issued = 0;
    for (int i = 0; i < nkb; ++i) {
      const int s = i % stages;
      const uint32_t ph = (uint32_t)(i / stages) & 1u;
      if (i >= stages && !warp_wait(&empty[s], ph ^ 1u, abort_flag)) {
        timed_out = true;
        *abort_flag = 1;
        break;
      }
      if (elect_one()) {
        if (i >= early) load_w(i);
        const uint32_t sf = sf_of(i);
        tma_load_2d(sb + (size_t)s * b_bytes, &tm_x, &full[s], (kb0 + i) * 128, (int)x_row0);
        for (int j = 0; j < xt; ++j)
          bulk_load(
              ssb + ((size_t)s * sfb_tiles + j) * kSfBytes,
              p.x_scales + ((int64_t)(xt0 + j) * p.tiles_kw + (int64_t)(kb0 + i) * kTilesPerStage) * kFp4TileBytes,
              sf, &full[s]);
      }
      __syncwarp();
      ++issued;
    }
    if (lane == 0) *issued_out = issued;
  } else if (warp == 1) {
    // Everything that a stage needs is a constant step from the stage before: the issuing
    // thread has 512 cycles of MMAs per stage to hide its own work behind.
    const uint32_t id0 = umma_idesc_fp4(128, p.n_tile, FMT == BD_FP4_MX, 0);
    const uint32_t id1 = umma_idesc_fp4(128, p.n_tile, FMT == BD_FP4_MX, 2);
    const uint64_t ad0 = umma_desc_sw128(smem_u32(sa)), bd0 = umma_desc_sw128(smem_u32(sb));
    const uint64_t sad0 = scale_desc(smem_u32(ssa)), sbd0 = scale_desc(smem_u32(ssb));
    const uint32_t b_step = b_bytes >> 4, sb_step = (uint32_t)sfb_tiles * (kSfBytes >> 4);
    const bool two = sfb_tiles == 2;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nkb; ++i) {
      if (!warp_wait(&full[s], ph, abort_flag)) {
        timed_out = true;
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sfa = tmem_d + d_cols + (uint32_t)(i & 1) * sf_cols;
        const uint32_t sfb = sfa + kSfaCols;
        const uint64_t ad = ad0 + (uint32_t)s * (kMmABytes >> 4), bdsc = bd0 + (uint32_t)s * b_step;
        const uint64_t sad = sad0 + (uint32_t)s * (kSfBytes >> 4), sbd = sbd0 + (uint32_t)s * sb_step;
        const int steps = p.k_steps - (kb0 + i) * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps) {
            // scales: SFA tile of a step in 4 columns, SFB likewise per 128 rows
            const int t = FMT == BD_FP4_NV ? k : k >> 1;
            const uint32_t sfb_t = sfb + (two ? 8 : 4) * t;
            if (FMT == BD_FP4_NV || (k & 1) == 0) {
              tmem_cp_scales(sfa + 4 * t, sad + t * (kFp4TileBytes >> 4));
              tmem_cp_scales(sfb_t, sbd + t * (kFp4TileBytes >> 4));
              if (two) tmem_cp_scales(sfb_t + 4, sbd + (kSfBytes >> 4) + t * (kFp4TileBytes >> 4));
            }
            // 64 columns: 32 bytes further inside the swizzled 128-byte row
            umma_fp4<FMT>(tmem_d, ad + 2 * k, bdsc + 2 * k, FMT == BD_FP4_MX && (k & 1) ? id1 : id0, sfa + 4 * t,
                          sfb_t, k > 0 ? 1u : (i > 0 ? 1u : 0u));
          }
        umma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (elect_one()) umma_commit(done);
    __syncwarp();
  } else {
    pdl_wait();
    const int64_t t0 = (int64_t)n_blk * p.h;
    for (int j = threadIdx.x - 64; j < p.h; j += kMmThreads - 64)
      xr[j] = p.x_row && t0 + j < p.tokens ? p.x_row[t0 + j] : 1.f;
  }

  const bool ok = mbar_wait(done, 0, nullptr);
  tc_fence_after();
  if (!ok) timed_out = true;
  if (timed_out) *abort_flag = 1;
  __syncthreads();
  const bool aborted = *abort_flag != 0;
  if (aborted && threadIdx.x == 0) {
    atomicOr(p.status, BD_DEV_TIMEOUT);
    // every load this CTA issued lands before its shared memory goes away
    const int issued = *issued_out;
    for (int i = max(0, issued - stages); i < issued; ++i)
      mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u, nullptr);
  }

  const int64_t t0 = (int64_t)n_blk * p.h;
  const int n_tok = (int)min((int64_t)p.h, p.tokens - t0);
  // eight warps: warps w and w + 4 read the same 32 lanes (rows) and take turns at the groups
  const int set = warp >> 2, r0 = (warp & 3) * 32 + lane;
  const uint32_t lane_addr = tmem_d + ((uint32_t)((warp & 3) * 32) << 16);
  constexpr int kTok = Group<L>::kTok;
  if (split == 1) {
    const int64_t row = m_blk * 128 + r0;
    const bool in = row < p.d_out && !aborted;
    const float rs = in && p.w_row ? p.w_row[row] : 1.f;
    for (int c0 = set * kTok; c0 < n_tok; c0 += 2 * kTok) {
      float v[kTok];
      load_group<FMT, L>(lane_addr + (uint32_t)(c0 * L), v);
#pragma unroll
      for (int j = 0; j < kTok; ++j)
        if (in && c0 + j < n_tok) store_y(p, t0 + c0 + j, row, scaled(v[j], rs, xr[c0 + j]));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem_d, tcols);
    return;
  }
  // Token j of the tile belongs to the CTA of rank j % split: each CTA writes its sums into
  // its owners' shared memory, and after a cluster barrier each adds what it was given in
  // rank order. The first barrier only says that every CTA has started: they arrive at it
  // before they ask for tensor memory, so that no CTA waits for another while holding some
  // (a CTA of this cluster could be waiting for what one of another cluster's holds, and
  // that one for this).
  cluster_wait();
  const int log2 = 31 - __clz(split);  // split is a power of two
  const uint32_t mine = smem_u32(gather + (size_t)rank * share * 128 + r0);
  for (int c0 = set * kTok; c0 < n_tok; c0 += 2 * kTok) {
    float v[kTok];
    load_group<FMT, L>(lane_addr + (uint32_t)(c0 * L), v);
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (c0 + j < n_tok) {
        const int t = c0 + j;
        st_cluster_f32(map_cluster(mine + (uint32_t)(t >> log2) * 512, (uint32_t)(t & (split - 1))), v[j]);
      }
  }
  tc_fence_before();  // tensor memory goes back before the barrier, for the same reason
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem_d, tcols);
  // four rows of a token per lane, a token per warp
  const int64_t row = m_blk * 128 + 4 * lane;
  float rs[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) rs[q] = p.w_row && row + q < p.d_out ? p.w_row[row + q] : 1.f;
  cluster_arrive();
  cluster_wait();
  for (int j = warp; rank + j * split < n_tok; j += kMmThreads / 32) {
    const float4* g = reinterpret_cast<const float4*>(gather + (size_t)j * 128) + lane;
    float4 u[kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
      if (r < split) u[r] = g[(size_t)r * share * 32];
    float4 v = u[0];
#pragma unroll
    for (int r = 1; r < kMaxSplit; ++r)
      if (r < split) {
        v.x += u[r].x;
        v.y += u[r].y;
        v.z += u[r].z;
        v.w += u[r].w;
      }
    const int t = rank + j * split;
    const float xs = xr[t];
    if (!aborted)
      store_y4(p, t0 + t, row,
               make_float4(scaled(v.x, rs[0], xs), scaled(v.y, rs[1], xs), scaled(v.z, rs[2], xs), scaled(v.w, rs[3], xs)));
  }
}

// ------------------------------------------------------------------------------------
// many X rows: persistent CTA pairs, a tile of 256 W rows x n_tile X rows at a time
// ------------------------------------------------------------------------------------
// Each CTA of a pair loads its 128 W rows and half of the X rows (and the scales of its W
// rows and of all X rows); the even CTA issues the cta_group::2 MMAs for both, and each holds
// the accumulator of its own W rows. Two accumulators overlap by what the scales take of
// tensor memory: [0, n_tile) and [n_tile - overlap, ...), so the next tile's MMAs start as
// soon as the epilogue has read the overlap (the columns that it reads first), and run beside
// the rest of it. At 256 x 256 a stage's loads (39 KB per CTA in BD_FP4_NV) take as long as 64
// bytes per cycle and SM allow, 610 cycles; its MMAs 512. Under load the clock falls to 1.25
// GHz (power): 8192 tokens on 28672 x 4096 run in 386-460 us on different boards, 4.2-5.0
// PFLOP/s (4 times the measured bf16 rate would be 6.7); 512 tokens in 4 limbs on the same W in
// 94-113 us, the tensor pipe active for 69% of the cycles at 1.6 GHz.
// With few tiles two pairs of a cluster share one (split == 2), half of K each: then each CTA
// sends the sums of half of its accumulator's groups to its counterpart of the other pair and
// adds what it is sent to the other half.
constexpr int kPairThreads = 384;       // warp 0 loads, warp 1 MMAs, warps 4-7 and 8-11 epilogue
constexpr uint32_t kPairSfCol = 448;    // scales in columns 448..511
constexpr uint32_t kPairOut = 2 * 64 * 128;  // outputs on their way out: 64 tokens x 128 rows of each set
constexpr int kPairGroupM = 8;          // tiles are walked in bands of this many row blocks

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
template <int FMT>
__device__ __forceinline__ void umma_fp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if (FMT == BD_FP4_NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// arrives on the barrier at this offset in both CTAs of a pair (mask: their ranks) when the MMAs
// issued so far are done
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}

// whether `v` holds in all 128 threads that meet at named barrier `id`
__device__ __forceinline__ bool bar_all(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred.aligned q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int FMT, int L>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_fp4_mm_pair(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                  const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs,
                  const __grid_constant__ CUtensorMap tm_y, const MmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kTilesPerStage = FMT == BD_FP4_NV ? 4 : 2;
  constexpr uint32_t kSfBytes = kTilesPerStage * kFp4TileBytes;
  constexpr uint32_t kNTile = 256 / (8 * L) * (8 * L);       // 256, or 240 with 6 limbs
  constexpr uint32_t kOverlap = 2 * kNTile - kPairSfCol;     // columns the accumulators share
  constexpr uint32_t kBBytes = kNTile / 2 * 128;
  constexpr uint32_t kStage = kMmABytes + kBBytes + 3 * kSfBytes;
  constexpr uint32_t kSfaCols = kTilesPerStage * 4;
  constexpr int kGroups = kNTile / Group<L>::kCols;
  static_assert(kOverlap <= 2 * Group<L>::kCols, "the sets' first groups hold the overlap");
  constexpr int kTok = Group<L>::kTok;
  constexpr int kOutBufs = 64 / kTok;                        // of a set: 2 groups of 32 tokens, or 8 of 8
  const int stages = p.stages;
  uint8_t* sa = smem;                                        // [stages] W codes, X codes, scales
  uint8_t* sb = sa + (size_t)stages * kMmABytes;
  uint8_t* ss = sb + (size_t)stages * kBBytes;
  uint8_t* sy = ss + (size_t)stages * 3 * kSfBytes;          // [2 sets][kOutBufs] groups of finished outputs
  const uint32_t out_bytes = p.y_bf16 ? kPairOut * 2 : kPairOut * 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(sy + out_bytes);
  uint64_t* empty = full + stages;
  uint64_t* acc_full = empty + stages;  // [2] an accumulator is complete (both CTAs)
  uint64_t* drained = acc_full + 2;     // the overlap of the current tile has been read (even CTA)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* x_range = tmem_slot + 2;    // bits of the tokens' least and largest scale

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), cta = rank & 1, lead = rank & ~1;
  const bool leader = cta == 0;
  const uint16_t mask = (uint16_t)(3u << lead);
  const int tiles_m = (int)((p.d_out + 255) / 256);
  const int64_t tiles = (int64_t)tiles_m * p.tiles_n;
  // with a split, cluster `pair` owns tile `pair` and there is no other
  const int pairs = (int)gridDim.x / (2 * p.split), pair = (int)blockIdx.x / (2 * p.split);
  const int kb_first = p.split == 2 ? p.kblocks * (rank >> 1) / 2 : 0;
  const int kb_end = p.split == 2 ? p.kblocks * ((rank >> 1) + 1) / 2 : p.kblocks;
  // tile i of the walk: bands of kPairGroupM row blocks, all N tiles of a band before the next
  auto tile_of = [&](int64_t i, int& m, int& n) {
    const int64_t band = i / ((int64_t)kPairGroupM * p.tiles_n);
    const int rows = min(kPairGroupM, tiles_m - (int)band * kPairGroupM);
    const int64_t r = i - band * kPairGroupM * p.tiles_n;
    m = (int)band * kPairGroupM + (int)(r % rows);
    n = (int)(r / rows);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full[0], 1);
    mbar_init(&acc_full[1], 1);
    mbar_init(drained, 16);  // eight epilogue warps of each CTA
    *abort_flag = 0;
    x_range[0] = 0x7F800000u;
    x_range[1] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_ws);
    tma_prefetch_desc(&tm_xs);
    if (p.y_tma) tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // the pair's barriers and tensor memory are ready
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  bool timed_out = false;
  if (warp == 0) {
    int it = 0, s = 0;  // stages used so far, stage of the ring
    uint32_t ph = 1;    // a fresh barrier's "previous" phase counts as complete
    const uint32_t full0 = map_cluster(smem_u32(full), lead);
    for (int64_t i = pair; i < tiles && !timed_out; i += pairs) {
      int m, n;
      tile_of(i, m, n);
      const int w_row0 = m * 256 + cta * 128;
      const int x_row0 = n * p.n_stride;
      const int w_tile0 = (w_row0 >> 7) * p.tiles_kw, x_tile0 = (x_row0 >> 7) * p.tiles_kw;
      for (int kb = kb_first; kb < kb_end; ++kb, ++it) {
        if (!warp_wait(&empty[s], ph, abort_flag)) {
          timed_out = true;
          break;
        }
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * kStage);
          const uint32_t bar = full0 + 8 * s;
          uint8_t* sf = ss + (size_t)s * 3 * kSfBytes;
          const int t0 = kb * kTilesPerStage;
          tma_load_2d_pair(sa + (size_t)s * kMmABytes, &tm_w, bar, kb * 128, w_row0);
          tma_load_2d_pair(sb + (size_t)s * kBBytes, &tm_x, bar, kb * 128, x_row0 + cta * (int)(kNTile / 2));
          tma_load_2d_pair(sf, &tm_ws, bar, 0, w_tile0 + t0);
          tma_load_2d_pair(sf + kSfBytes, &tm_xs, bar, 0, x_tile0 + t0);
          tma_load_2d_pair(sf + 2 * kSfBytes, &tm_xs, bar, 0, x_tile0 + p.tiles_kw + t0);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // all MMAs that read this CTA's shared memory are over before it leaves (bounded)
    for (int k = max(0, it - stages); k < it; ++k)
      if (!warp_wait(&empty[k % stages], (uint32_t)(k / stages) & 1u, abort_flag)) timed_out = true;
    if (timed_out) *abort_flag = 1;
  } else if (warp == 1 && leader) {
    const uint32_t id0 = umma_idesc_fp4(256, kNTile, FMT == BD_FP4_MX, 0);
    const uint32_t id1 = umma_idesc_fp4(256, kNTile, FMT == BD_FP4_MX, 2);
    const uint32_t sfa = tmem + kPairSfCol, sfb = sfa + kSfaCols;
    const uint64_t ad0 = umma_desc_sw128(smem_u32(sa)), bd0 = umma_desc_sw128(smem_u32(sb));
    const uint64_t sd0 = scale_desc(smem_u32(ss));
    int s = 0, j = 0;  // stage of the ring, tiles so far
    uint32_t ph = 0;
    for (int64_t i = pair; i < tiles && !timed_out; i += pairs, ++j) {
      if (j > 0) {
        if (!warp_wait(drained, (uint32_t)(j - 1) & 1u, abort_flag)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
      }
      const uint32_t d = tmem + (j & 1 ? kNTile - kOverlap : 0);
      for (int kb = kb_first; kb < kb_end; ++kb) {
        if (!warp_wait(&full[s], ph, abort_flag)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = ad0 + (uint32_t)s * (kMmABytes >> 4), bdsc = bd0 + (uint32_t)s * (kBBytes >> 4);
          const uint64_t sd = sd0 + (uint32_t)s * (3 * kSfBytes >> 4);
          const int steps = p.k_steps - kb * 4;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps) {
              const int t = FMT == BD_FP4_NV ? k : k >> 1;
              if (FMT == BD_FP4_NV || (k & 1) == 0) {
                tmem_cp_scales_pair(sfa + 4 * t, sd + t * (kFp4TileBytes >> 4));
                tmem_cp_scales_pair(sfb + 8 * t, sd + ((kSfBytes + t * kFp4TileBytes) >> 4));
                tmem_cp_scales_pair(sfb + 8 * t + 4, sd + ((2 * kSfBytes + t * kFp4TileBytes) >> 4));
              }
              umma_fp4_pair<FMT>(d, ad + 2 * k, bdsc + 2 * k, FMT == BD_FP4_MX && (k & 1) ? id1 : id0, sfa + 4 * t,
                                 sfb + 8 * t, k > 0 ? 1u : (kb > kb_first ? 1u : 0u));
            }
          umma_commit_pair(&empty[s], mask);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (elect_one()) umma_commit_pair(&acc_full[j & 1], mask);
      __syncwarp();
    }
    if (timed_out) *abort_flag = 1;
  }

  // ---------------- epilogue: two sets of four warps take turns at the groups of a tile ----------------
  const int w = warp & 3, set = warp >= 8 ? 1 : 0;
  const int r0 = w * 32 + lane;  // row of this CTA's half of a tile
  uint8_t* const bufs = sy + (size_t)set * (out_bytes / 2);
  int out = 0;                   // groups so far
  // lane k: the scale of token k of group g of the tile at token t0
  auto token_scale = [&](int64_t t0, int g) {
    const int64_t t = t0 + (int64_t)g * kTok + lane;
    return p.x_row && lane < kTok && t < p.tokens ? p.x_row[t] : 1.f;
  };
  // The tokens' scales lie between x_lo and x_hi. Where these and a warp's row scales cannot take
  // scaled() out of its first case, the outputs of a tile are v times the scales' product (looked
  // at per output it took 5% more where outputs dominate, 8192 tokens x 20000 x 256).
  float x_lo = 1.f, x_hi = 1.f;
  if (warp >= 4 && p.x_row) {
    uint32_t lo = 0x7F800000u, hi = 0;
#pragma unroll 8
    for (int64_t t = threadIdx.x - 128; t < p.tokens; t += kPairThreads - 128) {
      const uint32_t m = magnitude_bits(p.x_row[t]);
      lo = min(lo, m);
      hi = max(hi, m);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&x_range[0], lo);
      atomicMax(&x_range[1], hi);
    }
    asm volatile("bar.sync 3, %0;" ::"n"(kPairThreads - 128) : "memory");
    x_lo = __uint_as_float(x_range[0]);
    x_hi = __uint_as_float(x_range[1]);
  }
  auto in_range = [&](float rs) {
    const float lo = __uint_as_float(__reduce_min_sync(0xffffffffu, magnitude_bits(rs))) * x_lo;
    const float hi = __uint_as_float(__reduce_max_sync(0xffffffffu, magnitude_bits(rs))) * x_hi;
    return lo >= 0x1p-126f && hi <= 0x1.fffffep127f;
  };
  // outputs of group g: v times the row's scale rs and the tokens' xs
  auto emit = [&](auto plain, int64_t row0, int64_t t0, int g, float rs, float xs, float* v) {
    const int64_t tg = t0 + (int64_t)g * kTok;
#pragma unroll
    for (int c = 0; c < kTok; ++c) {
      const float x = __shfl_sync(0xffffffffu, xs, c);
      v[c] = plain.value ? v[c] * (rs * x) : scaled(v[c], rs, x);
    }
    if (p.y_tma) {
      // [token][128 rows] in shared memory, then one bulk store of the group; a buffer is
      // written again only after the store that read it (waited for before the barrier that
      // every writer passes)
      uint8_t* buf = bufs + (size_t)(out % kOutBufs) * (out_bytes / 2 / kOutBufs);
      if (p.y_bf16) {
#pragma unroll
        for (int c = 0; c < kTok; ++c) reinterpret_cast<uint16_t*>(buf)[c * 128 + r0] = (uint16_t)f2bf_bits(v[c]);
      } else {
#pragma unroll
        for (int c = 0; c < kTok; ++c) reinterpret_cast<float*>(buf)[c * 128 + r0] = v[c];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (w == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOutBufs - 2) : "memory");
      asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
      if (w == 0 && lane == 0) {
        if (row0 < p.d_out && tg < p.tokens) tma_store_2d(&tm_y, buf, (int)row0, (int)tg);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      ++out;
    } else {
      const int n_tok = (int)min((int64_t)kTok, p.tokens - tg);
#pragma unroll
      for (int c = 0; c < kTok; ++c)
        if (row0 + r0 < p.d_out && c < n_tok) store_y(p, tg + c, row0 + r0, v[c]);
    }
  };
  if (warp >= 4 && p.split == 1) {
    const uint32_t drained_bar = map_cluster(smem_u32(drained), lead);
    int j = 0;  // tiles so far
    for (int64_t i = pair; i < tiles; i += pairs, ++j) {
      int m, n;
      tile_of(i, m, n);
      const int64_t row0 = (int64_t)m * 256 + cta * 128, t0 = (int64_t)n * p.h;
      const float rs = p.w_row && row0 + r0 < p.d_out ? p.w_row[row0 + r0] : 1.f;
      // the overlap lies at the end of the even accumulator and at the start of the odd one:
      // the groups that hold it (one of each set) come first
      auto group_of = [&](int q) { return (j & 1) ? q : kGroups - 1 - q; };
      float xs = set < kGroups ? token_scale(t0, group_of(set)) : 1.f;
      // (all warps of a set leave together: emit() has a barrier for them)
      const bool come = mbar_wait(&acc_full[j & 1], (uint32_t)(j >> 1) & 1u, abort_flag);
      if (!bar_all(1 + set, come)) {
        timed_out = true;
        break;
      }
      tc_fence_after();
      const uint32_t at = tmem + (j & 1 ? kNTile - kOverlap : 0) + ((uint32_t)(w * 32) << 16);
      auto tile = [&](auto plain) {
        for (int q = set; q < kGroups; q += 2) {
          const int g = group_of(q);
          float v[kTok];
          load_group<FMT, L>(at + (uint32_t)(g * Group<L>::kCols), v);
          if (q == set) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(drained_bar);
          }
          const float xg = xs;
          if (q + 2 < kGroups) xs = token_scale(t0, group_of(q + 2));
          emit(plain, row0, t0, g, rs, xg, v);
        }
      };
      if (in_range(rs))
        tile(Flag<true>{});
      else
        tile(Flag<false>{});
    }
    if (timed_out) *abort_flag = 1;
  }
  if (p.split == 2) {
    int m, n;
    tile_of(pair, m, n);
    const int64_t row0 = (int64_t)m * 256 + cta * 128, t0 = (int64_t)n * p.h;
    constexpr int kHalf = (kGroups + 1) / 2;  // groups of the first pair; the others are the second's
    const int own0 = rank < 2 ? 0 : kHalf, own1 = rank < 2 ? kHalf : kGroups;
    const int far0 = rank < 2 ? kHalf : 0, far1 = rank < 2 ? kGroups : kHalf;
    const uint32_t at = tmem + ((uint32_t)(w * 32) << 16);
    float* sums = reinterpret_cast<float*>(smem);  // [token][128 rows], in the W stages
    if (warp >= 4 && !mbar_wait(&acc_full[0], 0, abort_flag)) *abort_flag = 1;
    tc_fence_after();
    __syncwarp();
    cluster_arrive();  // all MMAs and loads of the cluster are over: the stages are free
    cluster_wait();
    if (warp >= 4)
      for (int g = far0 + set; g < far1; g += 2) {
        float v[kTok];
        load_group<FMT, L>(at + (uint32_t)(g * Group<L>::kCols), v);
        const uint32_t to = map_cluster(smem_u32(sums + (g - far0) * kTok * 128 + r0), (uint32_t)(rank ^ 2));
#pragma unroll
        for (int c = 0; c < kTok; ++c) st_cluster_f32(to + c * 512, v[c]);
      }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp >= 4) {
      const float rs = p.w_row && row0 + r0 < p.d_out ? p.w_row[row0 + r0] : 1.f;
      auto tile = [&](auto plain) {
        for (int g = own0 + set; g < own1; g += 2) {
          const float xs = token_scale(t0, g);
          float v[kTok];
          load_group<FMT, L>(at + (uint32_t)(g * Group<L>::kCols), v);
#pragma unroll
          for (int c = 0; c < kTok; ++c) v[c] += sums[((g - own0) * kTok + c) * 128 + r0];
          emit(plain, row0, t0, g, rs, xs, v);
        }
      };
      if (in_range(rs))
        tile(Flag<true>{});
      else
        tile(Flag<false>{});
    }
  }
  if (warp >= 4 && p.y_tma && w == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) {
    atomicOr(p.status, BD_DEV_TIMEOUT);
    // copies in flight complete on barriers that nobody may wait for any more: they get a
    // millisecond to land before the shared memory goes away
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
  }
  __syncthreads();
  cluster_arrive();  // neither CTA leaves while the other's MMAs or barriers may reach it
  cluster_wait();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
// the tiled scales as rows of one tile (128 words), so that a stage's tiles are one box
static bool encode_scales(CUtensorMap* m, const void* base, int64_t tiles, int box_tiles) {
  TensorMapEncodeFn enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {128, (cuuint64_t)tiles};
  cuuint64_t strides[1] = {(cuuint64_t)kFp4TileBytes};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_tiles};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [tokens][d_out], boxes of 128 columns x box_tokens rows
static bool encode_out(CUtensorMap* m, const MmArgs& a, int box_tokens) {
  TensorMapEncodeFn enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)a.d_out, (cuuint64_t)a.tokens};
  cuuint64_t strides[1] = {(cuuint64_t)a.d_out * (a.y_bf16 ? 2 : 4)};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_tokens};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, a.y_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.y, dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K split and stages of k_fp4_mm_rows. For each split the time is estimated in SM cycles as
// the larger of what an SM has to load (60 bytes per cycle) and its longest chain: 1200 per
// CTA it starts, and for each set of resident CTAs 1500 until the first data, then per stage
// the instruction issue or the MMAs, and 1500 for a cluster's join; the best split is taken.
// Clusters of 4 and 8 do not fit every SM (132 and 120 at one CTA each, by the occupancy
// query). Stages take the shared memory that the resident CTAs of an SM leave each other.
// Measured (us, splits 1 / 2 / 4 / 8): 1 token on 4096 x 4096 9.4 / 7.8 / 6.4 / 8.5, 20 tokens
// fp32 on 4096 x 14336 25.8 / 16.8 / 13.2 / 13.8, 77 4-bit tokens on 1024 x 4096 10.5 / 8.0 /
// 6.2 / 5.4, 64 tokens on 14336 x 4096 (the product alone) 18.7 / 27.1 / 37.3 / 57.7: the rule
// takes 4, 4, 8 and 1.
static void plan_rows(Fp4Plan& p, int sf) {
  const int sms = sm_count();
  const int64_t tiles = (int64_t)p.tiles_n * p.tiles_m;
  const size_t stage = kMmABytes + (size_t)p.n_tile * 128 + (size_t)sf * (1 + (p.n_tile + 127) / 128);
  const int sf_cols = sf / kFp4TileBytes * 4 * (1 + (p.n_tile + 127) / 128);
  int tcols = 32;
  while (tcols < (p.n_tile + 31) / 32 * 32 + 2 * sf_cols) tcols *= 2;
  const double mma = 4.0 * (p.n_tile / 2 > 48 ? p.n_tile / 2 : 48);
  const double step = mma > 450 ? mma : 450;
  double best = 1e30;
  for (int split = 1; split <= kMaxSplit && split <= p.kblocks; split *= 2) {
    const size_t gather = split > 1 ? (size_t)split * ((p.h + split - 1) / split) * 512 : 0;
    const size_t fixed = 1024 + gather + (size_t)p.h * 4 + 17 * 8 + 16;
    const int need = (p.kblocks + split - 1) / split;
    const int usable = split <= 2 ? sms : (split == 4 ? sms * 132 / 148 : sms * 120 / 148);
    const int64_t per_sm = (tiles * split + usable - 1) / usable;
    // resident CTAs of an SM: all of its share if tensor and shared memory allow
    int res = (int)(per_sm < 512 / tcols ? per_sm : 512 / tcols);
    if (res > 6) res = 6;
    const int two = need < 2 ? need : 2;
    while (res > 1 && (size_t)res * (fixed + two * stage + 1024) > 227 * 1024) --res;
    int st = (int)((227 * 1024 / res - 1024 - fixed) / stage);
    if (st < 1) continue;
    if (st > need) st = need;
    if (st > 8) st = 8;
    const double waves = (double)((per_sm + res - 1) / res);
    const double load = (double)per_sm * need * stage / 60.0;
    const double chain = 1200.0 * per_sm + waves * (1500 + need * step + (split > 1 ? 1500 : 0));
    const double cost = load > chain ? load : chain;
    if (cost < best) {
      best = cost;
      p.split = split;
      p.stages = st;
      p.smem = fixed + st * stage;
      p.ctas = tiles * split;
    }
  }
}

Fp4Plan plan_fp4(int64_t d_out, int64_t d_in, int64_t tokens, int limbs, int fmt, bool y_bf16) {
  Fp4Plan p = {};
  p.limbs = limbs;
  p.kblocks = (int)((d_in + kFp4KStage - 1) / kFp4KStage);
  const int sf = (fmt == BD_FP4_NV ? 4 : 2) * kFp4TileBytes;
  // tokens of an N tile of at most 256 X rows: in steps of 8 with limbs, 16 without
  const int step = limbs > 1 ? 8 : 16;
  const int most = 256 / (8 * limbs) * 8;
  p.pair = tokens > most;
  if (p.pair) {
    p.h = most;
    p.n_tile = p.h * limbs;
    p.n_stride = 256;
    p.tiles_n = (int)((tokens + p.h - 1) / p.h);
    p.tiles_m = (int)((d_out + 255) / 256);
    const size_t stage = kMmABytes + (size_t)p.n_tile * 64 + 3 * (size_t)sf;
    const size_t out = (size_t)kPairOut * (y_bf16 ? 2 : 4);
    p.stages = (int)((226 * 1024 - 1024 - out) / stage);
    if (p.stages > 6) p.stages = 6;
    // two pairs per tile when all tiles then still run at once, unless K is short (512 tokens
    // on 4096 x 14336, 32 tiles: 25.6 us split, 33 without, on one board)
    const int64_t all = (int64_t)p.tiles_m * p.tiles_n;
    p.split = all * 4 <= sm_count() * 132 / 148 && p.kblocks >= 8 ? 2 : 1;
    p.smem = 1024 + p.stages * stage + out + (2 * p.stages + 3) * 8 + 16;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, pairs = sm_count() / 2;
    p.ctas = p.split == 2 ? 4 * tiles : 2 * (tiles < pairs ? tiles : pairs);
  } else {
    p.h = (int)((tokens + step - 1) / step * step);
    if (p.h > 128) p.h = 128;  // a cluster keeps h * 128 sums in each CTA's shared memory
    p.n_tile = p.h * limbs;
    p.n_stride = (p.n_tile + 127) / 128 * 128;
    p.tiles_n = (int)((tokens + p.h - 1) / p.h);
    p.tiles_m = (int)((d_out + 127) / 128);
    plan_rows(p, sf);
  }
  p.x_rows = limbs > 1 ? (int64_t)p.tiles_n * p.n_stride : tokens;
  p.xc_bytes = limbs > 1 ? align_up((size_t)p.x_rows * (size_t)(d_in / 2), 256) : 0;
  p.xs_bytes = limbs > 1 ? (size_t)fp4_scale_bytes(p.x_rows, d_in, fmt) : 0;
  return p;
}

namespace {
template <int FMT, int L>
bd_status launch_mm(const Fp4Plan& p, const Fp4Mat& w, const Fp4Mat& x, const MmArgs& a, int64_t d_in,
                    cudaStream_t s) {
  CUtensorMap tw, tx;
  if (!encode_codes(&tw, w.codes, a.d_out, d_in / 2, 128)) return BD_ERR_CUDA;
  if (!encode_codes(&tx, x.codes, p.x_rows, d_in / 2, p.pair ? p.n_tile / 2 : p.n_tile)) return BD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(p.pair ? kPairThreads : kMmThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)(p.pair ? 2 * p.split : p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static std::atomic<uint64_t> attr_rows{0}, attr_pair{0};
  if (p.pair) {
    CUtensorMap tws, txs;
    const int box = FMT == BD_FP4_NV ? 4 : 2;
    if (!encode_scales(&tws, w.scales, (a.d_out + 127) / 128 * a.tiles_kw, box) ||
        !encode_scales(&txs, x.scales, (int64_t)a.x_row_tiles * a.tiles_kw, box))
      return BD_ERR_CUDA;
    CUtensorMap ty = {};
    if (a.y_tma && !encode_out(&ty, a, Group<L>::kTok)) return BD_ERR_CUDA;
    if (!ensure_dyn_smem(k_fp4_mm_pair<FMT, L>, 227 * 1024, attr_pair)) return BD_ERR_CUDA;
    BD_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_fp4_mm_pair<FMT, L>, tw, tx, tws, txs, ty, a));
  } else {
    if (!ensure_dyn_smem(k_fp4_mm_rows<FMT, L>, 227 * 1024, attr_rows)) return BD_ERR_CUDA;
    BD_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_fp4_mm_rows<FMT, L>, tw, tx, a));
  }
  return BD_OK;
}
}  // namespace

bd_status launch_fp4_mm(const Fp4Plan& p, int fmt, const Fp4Mat& w, const Fp4Mat& x, int64_t d_out, int64_t d_in,
                        int64_t tokens, void* y, int32_t y_dtype, uint32_t* status, cudaStream_t s) {
  MmArgs a = {};
  a.w_scales = w.scales;
  a.x_scales = x.scales;
  a.w_row = w.row;
  a.x_row = x.row;
  a.y = y;
  a.status = status;
  a.d_out = d_out;
  a.tokens = tokens;
  a.tiles_kw = (int)fp4_tiles_k(d_in, fmt);
  a.x_row_tiles = (int)((p.x_rows + 127) / 128);
  a.h = p.h;
  a.n_tile = p.n_tile;
  a.n_stride = p.n_stride;
  a.tiles_n = p.tiles_n;
  a.kblocks = p.kblocks;
  a.k_steps = (int)((d_in + 63) / 64);
  a.split = p.split;
  a.stages = p.stages;
  a.y_bf16 = y_dtype == BD_BF16;
  // the limbs kernel goes before: its blocks start the next kernel after they have waited for
  // everything earlier on the stream, and it does not write W
  a.w_early = p.limbs > 1;
  a.y_tma = (d_out * (a.y_bf16 ? 2 : 4)) % 16 == 0;
  launch_begin(K_FP4_MM, s);
  bd_status r;
  if (fmt == BD_FP4_NV)
    r = p.limbs == 1   ? launch_mm<BD_FP4_NV, 1>(p, w, x, a, d_in, s)
        : p.limbs == 4 ? launch_mm<BD_FP4_NV, kFp4LimbsBf16>(p, w, x, a, d_in, s)
                       : launch_mm<BD_FP4_NV, kFp4LimbsF32>(p, w, x, a, d_in, s);
  else
    r = p.limbs == 1   ? launch_mm<BD_FP4_MX, 1>(p, w, x, a, d_in, s)
        : p.limbs == 4 ? launch_mm<BD_FP4_MX, kFp4LimbsBf16>(p, w, x, a, d_in, s)
                       : launch_mm<BD_FP4_MX, kFp4LimbsF32>(p, w, x, a, d_in, s);
  if (r != BD_OK) return r;
  launch_end(K_FP4_MM, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

bd_status launch_fp4_linear(const Fp4Plan& p, int fmt, const Fp4Mat& w, const void* x, int64_t d_out, int64_t d_in,
                            int64_t tokens, uint8_t* xc, uint8_t* xs, float* xmul, void* y, int32_t y_dtype,
                            uint32_t* reset_status, uint32_t* status, cudaStream_t s) {
  if (fp4_use_gemv(d_out, d_in, tokens))
    return launch_fp4_gemv(fmt, w, x, d_out, d_in, tokens, y, y_dtype, reset_status, s);
  const bd_status r = launch_fp4_limbs(p, fmt, x, d_in, tokens, xc, xs, xmul, reset_status, s);
  if (r != BD_OK) return r;
  return launch_fp4_mm(p, fmt, w, Fp4Mat{xc, xs, xmul}, d_out, d_in, tokens, y, y_dtype, status, s);
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
  L.p = plan_fp4(d_out, d_in, tokens, y_dtype == BD_F32 ? kFp4LimbsF32 : kFp4LimbsBf16, fmt, y_dtype == BD_BF16);
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
  return launch_fp4_mm(plan_fp4(d_out, d_in, tokens, 1, fmt, y_dtype == BD_BF16), fmt, w, x, d_out, d_in, tokens, y, y_dtype,
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
  return launch_fp4_linear(L.p, fmt, w, x, d_out, d_in, tokens, ws + L.off_c, ws + L.off_s, xmul, y, y_dtype, status,
                           status, s);
}
