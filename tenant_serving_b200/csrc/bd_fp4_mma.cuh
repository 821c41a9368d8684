// Device building blocks of the block-scaled 4-bit tensor-core kernels: scales into tensor
// memory, instruction descriptors, issue by one elected lane, accumulator reads.
#pragma once

#include "bd_fp4.cuh"
#include "bd_tc.cuh"

namespace bd {

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

// One lane of a converged warp, the same one each time. Operands of the tensor-core and copy
// instructions live in uniform registers; behind a `lane == 0` branch the compiler cannot
// know that they are, and moves each operand there lane by lane (73 cycles per instruction
// measured, 1170 for the sixteen of a stage).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// A bounded wait of a whole warp: all lanes give up when one does, so that what the warp does
// together afterwards stays together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag,
                                          long long limit_cycles = kWaitCycles) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, limit_cycles));
}
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// N (8, 16 or 32) consecutive 32-bit columns of the thread's lane; tmem_wait() before use
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else if (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// tensor map of packed codes [rows][row_bytes], boxes of 128 bytes (256 columns) x box_rows
inline bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows) {
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

}  // namespace bd
