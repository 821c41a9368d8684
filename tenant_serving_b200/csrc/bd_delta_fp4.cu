// The tenants' deltas over a 4-bit base, as a 4-bit product on the tensor cores.
//
// A sign is an E2M1 value: +1 is code 2, -1 code 10. So B_u x_t is a block-scaled 4-bit
// product (tcgen05.mma kind::mxf4) of the expanded signs with scale 1 and the activations'
// limbs (bd_fp4.cu), exact but for the limbs, and one MMA covers 128 rows x 64 columns of
// signs for 8 tokens. A warp's worth of expansion is two operations for eight signs, because
// the columns of every 32 are taken in another order: nibble i of output word j is bit
// 4 i + j of the sign word, and the limbs are written in that order.
//
// One item is (segment of up to 8 tokens of one tenant, 256 rows; 5 tokens with 6 limbs);
// persistent CTAs, one per SM, walk items in stages of 256 columns. Warp 0 copies a stage's
// signs (8 KB, with the group scales 1 KB more), warp 2 its limbs; warps 4-11 expand the signs
// into tensor memory (the A operands of two 128-row products), four of them a stage, a thread
// for rows r and r + 128; warp 1 issues the MMAs; warps 12-15 hold the sums; warp 3 fetches an item's
// tokens, base sums and row scales an item ahead. GROUP and BLOCK scales apply every 128
// columns or more: each 128-column chunk has accumulators of its own, which the epilogue
// scales and adds in fp32. ROW, TENSOR and COL deltas (COL scales are in the limbs) accumulate
// over the row.
//
// What bounds it: a stage takes about 830 cycles (GROUP) or 740 (ROW), shared between the
// expansion's instructions and the stage's chain of barriers; the MMAs themselves are cheap
// (issued twice over they add 2%), HBM is at 36%. 64 one-token tenants on 14336 x 4096 take
// 180 us where the lookup kernel takes 225 (528 MB of signs and scales: floor 81). A call with
// 32 ROW tenants and 256 tokens on 6144 x 4096 takes 95 us, with the lookup and fp16
// tensor-core kernels 228. An item has 256 rows because a stage's barriers are paid per item
// row block. A tenant's signs are expanded again for every 8 tokens, so its lead over the fp16
// tensor-core kernel of the other bases (64 tokens of a tenant at a time) shrinks with the tokens
// per tenant. 14336 x 4096, all of a call's delta kernels, this / fp16: 16 GROUP tenants with 16
// tokens each 139 / 246 us, with 32 237 / 272; 4 with 64 138 / 123, with 128 237 / 192; ROW 130 / 247,
// 214 / 273, 115 / 123, 194 / 192. Without effect or slower: a deeper ring of limbs, a stage's codes made before the
// wait for its slot, a second MMA warp, two sets of sum warps, four banks of half the columns,
// shifts on the multiplier.
#include "bd_fp4_mma.cuh"

namespace bd {

constexpr int kDfThreads = 512;
constexpr int kDfRows = 256;
constexpr int kDfStages = 3;                 // stages of A (tensor memory) and X (shared memory)
constexpr int kDfRaw = 10;                   // stages of packed signs in flight
constexpr int kDfSigns = kDfRows * 32, kDfScales = kDfRows * 4;  // bytes of a stage's signs, group scales
constexpr int kDfRawBytes = kDfSigns + kDfScales;
constexpr int kDfScaleSlots = 6;             // see the expander
struct DfItem {                              // an item as the epilogue needs it
  int32_t count, chunked;
  int32_t tok[8];
  float scale[kDfRows];
  float base[8][kDfRows];
};
constexpr uint32_t kDfN = kFp4SegRows;       // MMA N, and X rows of a segment's slot
constexpr uint32_t kDfSmallN = 16;           // MMA N of a segment of 1 or 2 tokens
constexpr uint32_t kDfXBytes = kDfN * 128;
constexpr uint32_t kDfXsBytes = 2 * kFp4TileBytes;
constexpr int kDfCopy = 2048;                // columns of y that a block copies at a time
// tensor memory: two banks of accumulators [2 products][2 chunks], the A ring, scales of one,
// scales of X
constexpr uint32_t kDfBank = 4 * kDfN;
constexpr uint32_t kDfA = 2 * kDfBank;
constexpr uint32_t kDfSfa = kDfA + 64 * kDfStages;
constexpr uint32_t kDfSfb = kDfSfa + 4;
static_assert(kDfSfb + 8 * kDfStages <= 512, "");

struct DfSegs {
  const int32_t *start, *count, *base_only, *perm;  // *base_only: tokens of the base alone, last in perm
};
__device__ __forceinline__ DfSegs df_segs(const int32_t* seg_base, int max_groups, int max_tc) {
  DfSegs g;
  const int32_t* tenant = seg_base + kSegHeader + 3 * max_groups;
  g.start = tenant + max_tc;
  g.count = g.start + max_tc;
  g.base_only = g.count + max_tc;
  g.perm = g.base_only + max_tc;
  return g;
}
// The CTA's items in turn: item blockIdx.x + i gridDim.x is (segment, row tile), stepped
// without a division.
struct DfWalk {
  int seg, mt, left, mtiles, seg_step, mt_step;
  __device__ __forceinline__ DfWalk(int segs, int tiles) {
    const int64_t items = (int64_t)segs * tiles;
    mtiles = tiles;
    left = items > blockIdx.x ? (int)((items - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
    seg = (int)blockIdx.x / tiles;
    mt = (int)blockIdx.x - seg * tiles;
    seg_step = (int)gridDim.x / tiles;
    mt_step = (int)gridDim.x - seg_step * tiles;
  }
  __device__ __forceinline__ void next() {
    --left;
    seg += seg_step;
    mt += mt_step;
    if (mt >= mtiles) {
      mt -= mtiles;
      ++seg;
    }
  }
};
__device__ __forceinline__ bool df_chunked(int32_t mode) { return mode == BD_SCALE_GROUP || mode == BD_SCALE_BLOCK; }

// ------------------------------------------------------------------------------------
// limbs of a segment's tokens, columns in the signs' order: position 8 j + i of every 32 is
// column 4 i + j. Limb l of token t of a segment is row l * gs + t of its slot of 32 rows, gs =
// 2 for a segment of 1 or 2 tokens, else the most tokens a segment has (8, or 5 with 6 limbs).
// The blocks behind the segments' write y for the tokens of the base alone.
// ------------------------------------------------------------------------------------
template <int L>
__global__ void __launch_bounds__(128) k_fp4_seg_limbs(const int32_t* __restrict__ seg_base, int max_groups,
                                                       int max_tc, const bd_tenant* __restrict__ tc_rec,
                                                       const uint16_t* __restrict__ x, int64_t d_in,
                                                       uint8_t* __restrict__ xc, uint8_t* __restrict__ xs,
                                                       const float* __restrict__ y_part, int64_t d_out, int batch,
                                                       void* __restrict__ y, bool y_bf16) {
  pdl_wait();  // inputs may come from the previous kernel on the stream
  pdl_trigger();
  constexpr int kTok = fp4_seg_tokens(L);
  const DfSegs sg = df_segs(seg_base, max_groups, max_tc);
  if ((int)blockIdx.x >= max_tc * kTok) {
    const int n = *sg.base_only, chunks = (int)((d_out + kDfCopy - 1) / kDfCopy);
    const int64_t units = (int64_t)n * chunks, stride = gridDim.x - max_tc * kTok;
    for (int64_t u = (int64_t)blockIdx.x - max_tc * kTok; u < units; u += stride) {
      const int64_t c0 = (u % chunks) * kDfCopy, t = sg.perm[batch - n + (int)(u / chunks)];
      const int64_t c1 = min(c0 + kDfCopy, d_out);
      const float* p = y_part + t * d_out;
      if (d_out % 4 == 0) {
        for (int64_t c = c0 + threadIdx.x * 4; c < c1; c += 512) {
          const float4 v = *reinterpret_cast<const float4*>(p + c);
          if (y_bf16)
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(y) + t * d_out + c) =
                make_uint2(f2bf_bits(v.x) | ((uint32_t)f2bf_bits(v.y) << 16),
                           f2bf_bits(v.z) | ((uint32_t)f2bf_bits(v.w) << 16));
          else
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + t * d_out + c) = v;
        }
      } else {
        for (int64_t c = c0 + threadIdx.x; c < c1; c += 128) {
          if (y_bf16)
            reinterpret_cast<uint16_t*>(y)[t * d_out + c] = (uint16_t)f2bf_bits(p[c]);
          else
            reinterpret_cast<float*>(y)[t * d_out + c] = p[c];
        }
      }
    }
    return;
  }
  const int seg = (int)blockIdx.x / kTok, j = (int)blockIdx.x - seg * kTok;
  if (seg >= seg_base[1]) return;
  const int count = sg.count[seg];
  if (j >= count) return;
  const int gs = count <= 2 ? 2 : fp4_seg_tokens(L);
  const int64_t t = sg.perm[sg.start[seg] + j];
  const bd_tenant T = tc_rec[seg];
  const __half* col = T.mode == BD_SCALE_COL ? static_cast<const __half*>(T.scales) : nullptr;
  const int64_t tiles_k = fp4_tiles_k(d_in, BD_FP4_MX);
  uint8_t* const srow = xs + (int64_t)seg * tiles_k * kFp4TileBytes;
  const int64_t nb = d_in / 32;
  for (int64_t b = threadIdx.x; b < 4 * tiles_k; b += 128) {
    uint8_t* const sb = srow + (b >> 2) * kFp4TileBytes + (b & 3);
    if (b >= nb) {  // padding scales are zero
      for (int l = 0; l < L; ++l) sb[(l * gs + j) * 16] = 0;
      continue;
    }
    float v[32];
    {
      const uint4* p = reinterpret_cast<const uint4*>(x + t * d_in + b * 32);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 u = p[q];
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * q + 2 * i] = bf16lo(a[i]);
          v[8 * q + 2 * i + 1] = bf16hi(a[i]);
        }
      }
    }
    if (col) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= __half2float(col[b * 32 + i]);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
    const bool bad = (__float_as_uint(m) & 0x7FFFFFFFu) >= 0x7F800000u;
    if (bad) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int e = max(limb_exponent(__float_as_uint(abs_max<32>(v))), -127);
      const float up = pow2f(-e), s = pow2f(e);
      uint32_t w[4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float q[8];
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = v[4 * i + jj] * up;
        w[jj] = e2m1_round8(q, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(h[i]);
          v[8 * i + jj] = fmaf(-f.x, s, v[8 * i + jj]);
          v[8 * i + 4 + jj] = fmaf(-f.y, s, v[8 * i + 4 + jj]);
        }
      }
      const int r = l * gs + j;
      *reinterpret_cast<uint4*>(xc + ((int64_t)seg * kFp4SegRows + r) * (d_in >> 1) + b * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
      sb[r * 16] = (uint8_t)(bad ? 0xFFu : (uint32_t)(e + 127));
    }
  }
}

// ------------------------------------------------------------------------------------
// delta + combine
// ------------------------------------------------------------------------------------
__device__ __forceinline__ void umma_mxf4_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], [%1], %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// acc[p][t] += s[p][c] * (sum of token t's limbs in chunk c of product p) for CHUNKS chunks; a
// chunk's columns are l * GS + t
template <int L, int GS, int CHUNKS, int TOK>
__device__ __forceinline__ void take_sums(uint32_t taddr, const float (*s)[2], float (*acc)[TOK]) {
  constexpr int kCols = GS * L <= 8 ? 8 : GS * L <= 16 ? 16 : 32;
  constexpr int kAtOnce = kCols < 32 ? 2 : 1;  // products read before one wait
#pragma unroll
  for (int p0 = 0; p0 < 2; p0 += kAtOnce) {
    uint32_t u[kAtOnce][CHUNKS][kCols];
#pragma unroll
    for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) tmem_load<kCols>(taddr + (2 * (p0 + p) + c) * kDfN, u[p][c]);
    tmem_wait();
#pragma unroll
    for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < GS; ++j) {
          float a = __uint_as_float(u[p][c][GS * (L - 1) + j]);
#pragma unroll
          for (int l = L - 2; l >= 0; --l) a += __uint_as_float(u[p][c][GS * l + j]);
          acc[p0 + p][j] = fmaf(s[p0 + p][c], a, acc[p0 + p][j]);
        }
  }
}

template <int L>
__global__ void __launch_bounds__(kDfThreads, 1)
    k_delta_fp4(const __grid_constant__ CUtensorMap tm_small, const __grid_constant__ CUtensorMap tm_x,
                const uint8_t* __restrict__ xs, const bd_tenant* __restrict__ tc_rec,
                const int32_t* __restrict__ seg_base, int max_groups, int max_tc, const float* __restrict__ y_part,
                int64_t d_out, int64_t d_in, void* __restrict__ y, bool y_bf16, uint32_t* __restrict__ status) {
  constexpr int kTok = fp4_seg_tokens(L);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = smem;                                              // [stages] limb codes
  uint8_t* sxs = sx + (size_t)kDfStages * kDfXBytes;               // [stages][2 scale tiles]
  uint8_t* raw = sxs + (size_t)kDfStages * kDfXsBytes;             // [raw] signs, then group scales
  uint8_t* ones = raw + (size_t)kDfRaw * kDfRawBytes;              // a scale tile of ones
  uint2* sc = reinterpret_cast<uint2*>(ones + kFp4TileBytes);      // [slots][128] two scales of rows r and r + 128
  // full: a stage's limbs have landed and its signs are expanded; done: its MMAs are over
  DfItem* items = reinterpret_cast<DfItem*>(sc + kDfScaleSlots * 128);  // [2]
  uint64_t* full = reinterpret_cast<uint64_t*>(items + 2);
  uint64_t* done = full + kDfStages;
  uint64_t* raw_full = done + kDfStages;
  uint64_t* raw_empty = raw_full + kDfRaw;
  uint64_t* bank_full = raw_empty + kDfRaw;  // [2]
  uint64_t* bank_empty = bank_full + 2;      // [2]
  uint64_t* item_full = bank_empty + 2;      // [2]
  uint64_t* item_empty = item_full + 2;      // [2]
  uint64_t* drain = item_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDfStages; ++i) {
      mbar_init(&full[i], 1 + 4);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < kDfRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bank_full[b], 1);
      mbar_init(&bank_empty[b], 4);
      mbar_init(&item_full[b], 1);
      mbar_init(&item_empty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_small);
    tma_prefetch_desc(&tm_x);
  }
  if (threadIdx.x >= 64 && threadIdx.x < 192) reinterpret_cast<uint32_t*>(ones)[threadIdx.x - 64] = 0x7F7F7F7Fu;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int mtiles = (int)((d_out + kDfRows - 1) / kDfRows);
  const DfSegs sg = df_segs(seg_base, max_groups, max_tc);
  const int nst = (int)((d_in + 255) / 256);
  const int tiles_k = (int)fp4_tiles_k(d_in, BD_FP4_MX);  // 128-column chunks of a row
  DfWalk it(seg_base[1], mtiles);
  bool ok = true;

  if (warp == 0) {
    // ---------------- signs and group scales, up to kDfRaw stages ahead ----------------
    int rs = 0;
    uint32_t rph = 1;
    int64_t n = 0;  // stages issued
    bd_tenant next_t = {};
    if (it.left > 0) next_t = tc_rec[it.seg];
    while (it.left > 0 && ok) {
      const int row0 = it.mt * kDfRows;
      const bd_tenant T = next_t;
      it.next();
      if (it.left > 0) next_t = tc_rec[it.seg];
      const bool with_scales = T.mode == BD_SCALE_GROUP && T.group_size == 128;
      // (the serving layout's tiles have 512 rows: the second half of one may be the next's start)
      const uint8_t* signs = reinterpret_cast<const uint8_t*>(T.signs) + (int64_t)(row0 / 512) * nst * 16384 + (row0 % 512) * 32;
      const uint8_t* scales = static_cast<const uint8_t*>(T.scales) + (int64_t)(row0 / 512) * nst * 2048 + (row0 % 512) * 4;
      for (int st = 0; st < nst; ++st) {
        if (!warp_wait(&raw_empty[rs], rph, abort_flag)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* dst = raw + rs * kDfRawBytes;
          mbar_arrive_expect_tx(&raw_full[rs], with_scales ? kDfRawBytes : kDfSigns);
          bulk_load(dst, signs, kDfSigns, &raw_full[rs]);
          if (with_scales) bulk_load(dst + kDfSigns, scales, kDfScales, &raw_full[rs]);
        }
        __syncwarp();
        signs += 16384;
        scales += 2048;
        ++n;
        if (++rs == kDfRaw) {
          rs = 0;
          rph ^= 1;
        }
      }
    }
    if (!ok) {  // every copy lands before the shared memory goes away
      *abort_flag = 1;
      for (int64_t i = n > kDfRaw ? n - kDfRaw : 0; i < n; ++i)
        warp_wait(&raw_full[i % kDfRaw], (uint32_t)(i / kDfRaw) & 1u, nullptr);
    }
  } else if (warp == 2) {
    // ---------------- limbs ----------------
    int s = 0;
    uint32_t ph = 1;
    int64_t n = 0;
    int32_t count = it.left > 0 ? sg.count[it.seg] : 0;
    while (it.left > 0 && ok) {
      const int x_row = it.seg * (int)kFp4SegRows;
      const uint8_t* xsr = xs + (int64_t)it.seg * tiles_k * kFp4TileBytes;
      const bool small = count <= 2;
      it.next();
      if (it.left > 0) count = sg.count[it.seg];
      for (int st = 0; st < nst; ++st) {
        if (!warp_wait(&done[s], ph, abort_flag)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sf = (uint32_t)min(2, tiles_k - 2 * st) * kFp4TileBytes;
          mbar_arrive_expect_tx(&full[s], (small ? kDfSmallN : kDfN) * 128 + sf);
          tma_load_2d(sx + s * kDfXBytes, small ? &tm_small : &tm_x, &full[s], st * 128, x_row);
          bulk_load(sxs + s * kDfXsBytes, xsr + st * (2 * kFp4TileBytes), sf, &full[s]);
        }
        __syncwarp();
        ++n;
        if (++s == kDfStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {
      // as above, but these copies complete on barriers that other warps may no longer arrive
      // at: they get the time instead
      *abort_flag = 1;
      for (int64_t i = n > kDfStages ? n - kDfStages : 0; i < n; ++i)
        warp_wait(&full[i % kDfStages], (uint32_t)(i / kDfStages) & 1u, nullptr, 2000000);
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    // (one thread walks the stages: it has no vote to take after each wait)
    if (elect_one()) {
      const uint32_t sfa = tmem + kDfSfa;
      tmem_cp_scales(sfa, scale_desc(smem_u32(ones)));
      const uint64_t bd0 = umma_desc_sw128(smem_u32(sx)), sd0 = scale_desc(smem_u32(sxs));
      const int k_steps = (int)((d_in + 63) / 64);
      int s = 0;
      uint32_t ph = 0, bn = 0;  // ring position; accumulator banks handed to the epilogue so far
      int32_t mode = 0, count = 0;
      if (it.left > 0) {
        mode = tc_rec[it.seg].mode;
        count = sg.count[it.seg];
      }
      while (it.left > 0 && ok) {
        const bool chunked = df_chunked(mode);
        const uint32_t nn = count <= 2 ? kDfSmallN : kDfN;
        it.next();
        if (it.left > 0) {
          mode = tc_rec[it.seg].mode;
          count = sg.count[it.seg];
        }
        const uint32_t id0 = umma_idesc_fp4(128, nn, true, 0), id1 = umma_idesc_fp4(128, nn, true, 2);
        const uint32_t step = chunked ? kDfN : 0;  // from a chunk's accumulator to the next one's
        const uint32_t on = chunked ? 0u : 1u;     // a second chunk adds to the first one's
        for (int st = 0; st < nst; ++st) {
          if ((chunked || st == 0) && bn >= 2 && !mbar_wait(&bank_empty[bn & 1], ((bn >> 1) & 1) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (!mbar_wait(&full[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool last = chunked || st == nst - 1;
          const uint32_t d = tmem + (bn & 1) * kDfBank, d2 = d + step;
          const uint32_t a = tmem + kDfA + 64 * s, sfb = tmem + kDfSfb + 8 * s;
          const uint64_t b = bd0 + (uint32_t)s * (kDfXBytes >> 4), sd = sd0 + (uint32_t)s * (kDfXsBytes >> 4);
          const int steps = k_steps - 4 * st;
          const uint32_t more = !chunked && st > 0 ? 1u : 0u;
          // products of rows r (A columns 0-31) and r + 128 (32-63)
          tmem_cp_scales(sfb, sd);
          umma_mxf4_ts(d, a, b, id0, sfa, sfb, more);
          umma_mxf4_ts(d + 2 * kDfN, a + 32, b, id0, sfa, sfb, more);
          if (steps > 1) {
            umma_mxf4_ts(d, a + 8, b + 2, id1, sfa, sfb, 1u);
            umma_mxf4_ts(d + 2 * kDfN, a + 40, b + 2, id1, sfa, sfb, 1u);
          }
          if (steps > 2) {
            tmem_cp_scales(sfb + 4, sd + (kFp4TileBytes >> 4));
            umma_mxf4_ts(d2, a + 16, b + 4, id0, sfa, sfb + 4, on);
            umma_mxf4_ts(d2 + 2 * kDfN, a + 48, b + 4, id0, sfa, sfb + 4, on);
          }
          if (steps > 3) {
            umma_mxf4_ts(d2, a + 24, b + 6, id1, sfa, sfb + 4, 1u);
            umma_mxf4_ts(d2 + 2 * kDfN, a + 56, b + 6, id1, sfa, sfb + 4, 1u);
          }
          umma_commit(&done[s]);
          if (last) {
            umma_commit(&bank_full[bn & 1]);
            ++bn;
          }
          if (++s == kDfStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) *abort_flag = 1;
      umma_commit(drain);
    }
    __syncwarp();
    warp_wait(drain, 0, nullptr);  // no MMA may be in flight when the CTA leaves
  } else if (warp >= 4 && warp < 12) {
    // ---------------- signs -> E2M1 in tensor memory, every other stage ----------------
    const int r = (warp & 3) * 32 + lane;
    const uint32_t a_lane = tmem + kDfA + ((uint32_t)((warp & 3) * 32) << 16);
    int rs = 0, s = 0, slot = 0;
    uint32_t rph = 0, ph = 1;
    bool turn = warp < 8;
    bd_tenant next_t = {};
    if (it.left > 0) next_t = tc_rec[it.seg];
    while (it.left > 0 && ok) {
      const int64_t row = (int64_t)it.mt * kDfRows + r;
      const bd_tenant T = next_t;
      it.next();
      if (it.left > 0) next_t = tc_rec[it.seg];
      const bool chunked = df_chunked(T.mode), tiled = T.mode == BD_SCALE_GROUP && T.group_size == 128;
      const int gshift = chunked ? __ffs(T.group_size) - 1 : 0;
      // scales that are not in the tiled layout: a row's two of a stage
      auto plain_pair = [&](int64_t o, int st) {
        if (o >= d_out) return 0u;
        const uint16_t* p =
            static_cast<const uint16_t*>(T.scales) + (T.mode == BD_SCALE_BLOCK ? o >> gshift : o) * (d_in >> gshift);
        const uint32_t lo = p[((int64_t)st * 256) >> gshift];
        const uint32_t hi = 2 * st + 1 < tiles_k ? p[((int64_t)st * 256 + 128) >> gshift] : 0u;
        return lo | (hi << 16);
      };
      for (int st = 0; st < nst; ++st, turn = !turn) {
        if (turn) {
          if (!warp_wait(&raw_full[rs], rph, abort_flag)) {
            ok = false;
            break;
          }
          const uint8_t* src = raw + rs * kDfRawBytes;
          uint4 w[4];
          uint32_t scl[2] = {0u, 0u};
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            w[2 * p] = *reinterpret_cast<const uint4*>(src + (p * 128 + r) * 32);
            w[2 * p + 1] = *reinterpret_cast<const uint4*>(src + (p * 128 + r) * 32 + 16);
            if (tiled)
              scl[p] = *reinterpret_cast<const uint32_t*>(src + kDfSigns + (p * 128 + r) * 4);
            else if (chunked)
              scl[p] = plain_pair(row + 128 * p, st);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[rs]);
          if (!warp_wait(&done[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t sw[8] = {w[2 * p].x,     w[2 * p].y,     w[2 * p].z,     w[2 * p].w,
                                    w[2 * p + 1].x, w[2 * p + 1].y, w[2 * p + 1].z, w[2 * p + 1].w};
            uint32_t e[32];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) e[4 * i + j] = (~(sw[i] << (3 - j)) & 0x88888888u) | 0x22222222u;
            tmem_store32(a_lane + 64 * s + 32 * p, e);
          }
          // Slots count the stages of chunked items. The epilogue reads a slot after its bank's
          // MMAs; it is written again 6 such stages later, once the A slot of 3 stages before
          // that is free: then the MMAs of (at least) 3 such stages after this one are done,
          // and they waited until the bank of the stage after this one had been read.
          if (chunked) {
            sc[slot * 128 + r] = make_uint2(scl[0], scl[1]);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
        if (chunked && ++slot == kDfScaleSlots) slot = 0;
        if (++rs == kDfRaw) {
          rs = 0;
          rph ^= 1;
        }
        if (++s == kDfStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == 3) {
    // ---------------- an item's tokens, row scales and base sums ----------------
    uint32_t n = 0;
    for (; it.left > 0 && ok; it.next(), ++n) {
      DfItem& I = items[n & 1];
      const int seg = it.seg;
      const int32_t mode = tc_rec[seg].mode, count = sg.count[seg], start = sg.start[seg];
      const int my_tok = lane < count ? sg.perm[start + lane] : 0;
      if (!warp_wait(&item_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        I.count = count;
        I.chunked = df_chunked(mode);
      }
      if (lane < count) I.tok[lane] = my_tok;
      const int64_t row0 = (int64_t)it.mt * kDfRows + lane;
      const __half* scales = static_cast<const __half*>(tc_rec[seg].scales);
#pragma unroll
      for (int q = 0; q < kDfRows / 32; ++q) {
        const int64_t row = row0 + 32 * q;
        float s = 1.f;
        if (row < d_out && mode == BD_SCALE_ROW) s = __half2float(scales[row]);
        if (mode == BD_SCALE_TENSOR) s = __half2float(scales[0]);
        I.scale[32 * q + lane] = s;
      }
      for (int j = 0; j < count; ++j) {
        const float* p = y_part + (int64_t)__shfl_sync(0xffffffffu, my_tok, j) * d_out + row0;
#pragma unroll
        for (int q = 0; q < kDfRows / 32; ++q)
          I.base[j][32 * q + lane] = row0 + 32 * q < d_out ? p[32 * q] : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_full[n & 1]);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 12) {
    // ---------------- sums and combine ----------------
    const int r = (warp & 3) * 32 + lane;
    const uint32_t d_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t bn = 0, n = 0;
    int slot = 0;
    for (; it.left > 0 && ok; it.next(), ++n) {
      const DfItem& I = items[n & 1];
      if (!warp_wait(&item_full[n & 1], (n >> 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      const int count = I.count;
      const bool small = count <= 2, chunked = I.chunked != 0;
      float acc[2][kTok];
#pragma unroll
      for (int j = 0; j < kTok; ++j) acc[0][j] = acc[1][j] = 0.f;
      const int banks = chunked ? nst : 1;
      for (int k = 0; k < banks; ++k, ++bn) {
        if (!warp_wait(&bank_full[bn & 1], (bn >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = d_lane + (bn & 1) * kDfBank;
        float s4[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
        if (chunked) {
          const uint2 p = sc[slot * 128 + r];
          if (++slot == kDfScaleSlots) slot = 0;
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&p.x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&p.y));
          s4[0][0] = lo.x;
          s4[0][1] = lo.y;
          s4[1][0] = hi.x;
          s4[1][1] = hi.y;
        }
        if (chunked && 2 * k + 1 < tiles_k) {
          if (small)
            take_sums<L, 2, 2, kTok>(d, s4, acc);
          else
            take_sums<L, kTok, 2, kTok>(d, s4, acc);
        } else {
          if (small)
            take_sums<L, 2, 1, kTok>(d, s4, acc);
          else
            take_sums<L, kTok, 1, kTok>(d, s4, acc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bank_empty[bn & 1]);
      }
      if (!ok) break;
      const int64_t row = (int64_t)it.mt * kDfRows + r;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (row + 128 * p >= d_out) break;
        const float s = I.scale[128 * p + r];
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
          if (j >= count) break;
          const float v = fmaf(s, acc[p][j], I.base[j][128 * p + r]);
          const int64_t at = (int64_t)I.tok[j] * d_out + row + 128 * p;
          if (y_bf16)
            reinterpret_cast<uint16_t*>(y)[at] = (uint16_t)f2bf_bits(v);
          else
            reinterpret_cast<float*>(y)[at] = v;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[n & 1]);
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(status, BD_DEV_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
template <int L>
static bd_status launch_delta(const DeltaFp4Args& a, cudaStream_t s) {
  const int64_t copies = a.batch * ((a.d_out + kDfCopy - 1) / kDfCopy), copy_cap = (int64_t)sm_count() * 4;
  const int64_t blocks = (int64_t)a.max_tc * fp4_seg_tokens(L) + (copies < copy_cap ? copies : copy_cap);
  launch_begin(K_FP4_SEG_LIMBS, s);
  BD_CUDA_TRY(launch_pdl(k_fp4_seg_limbs<L>, dim3((unsigned)blocks), dim3(128), 0, s, a.seg, a.max_groups, a.max_tc,
                         a.tc_rec, static_cast<const uint16_t*>(a.x), a.d_in, a.xc, a.xs, a.y_part, a.d_out,
                         (int)a.batch, a.y, a.y_bf16));
  launch_end(K_FP4_SEG_LIMBS, s);
  BD_LAUNCH_CHECK();
  CUtensorMap small, full;
  const int64_t rows = (int64_t)a.max_tc * kFp4SegRows;
  if (!encode_codes(&small, a.xc, rows, a.d_in / 2, kDfSmallN) || !encode_codes(&full, a.xc, rows, a.d_in / 2, kDfN))
    return BD_ERR_CUDA;
  const size_t smem = 1024 + (size_t)kDfStages * (kDfXBytes + kDfXsBytes) + (size_t)kDfRaw * kDfRawBytes +
                      kFp4TileBytes + (size_t)kDfScaleSlots * 1024 + 2 * sizeof(DfItem) +
                      (2 * kDfStages + 2 * kDfRaw + 9) * 8 + 16;
  static std::atomic<uint64_t> attr{0};
  if (!ensure_dyn_smem(k_delta_fp4<L>, 227 * 1024, attr)) return BD_ERR_CUDA;
  const int64_t most = (a.d_out + kDfRows - 1) / kDfRows * a.max_tc, grid = (int64_t)sm_count();
  launch_begin(K_DELTA_FP4, s);
  BD_CUDA_TRY(launch_pdl(k_delta_fp4<L>, dim3((unsigned)(grid < most ? grid : most)), dim3(kDfThreads),
                         smem < 120 * 1024 ? 120 * 1024 : smem,  // one CTA per SM: each takes all of tensor memory
                         s, small, full, (const uint8_t*)a.xs, a.tc_rec, a.seg, a.max_groups, a.max_tc, a.y_part,
                         a.d_out, a.d_in, a.y, a.y_bf16, a.status));
  launch_end(K_DELTA_FP4, s);
  BD_LAUNCH_CHECK();
  return BD_OK;
}

bd_status launch_delta_fp4(const DeltaFp4Args& a, int limbs, cudaStream_t s) {
  return limbs == kFp4LimbsBf16 ? launch_delta<kFp4LimbsBf16>(a, s) : launch_delta<kFp4LimbsF32>(a, s);
}

}  // namespace bd
