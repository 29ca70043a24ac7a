// Building blocks of the attention kernels: format conversions, the shared
// memory swizzle, TMEM rows of 32 columns, reductions over a warp's lanes, and
// the tensor maps of query and window rows.
#pragma once

#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "host_once.cuh"
#include "tc.cuh"

namespace csa2 {

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// what the rounding of (lo, hi) to the two bf16 of `w` left of them, as two bf16: together they
// hold 16 bits of each
__device__ __forceinline__ uint32_t bf16x2_rest(float lo, float hi, uint32_t w) {
  return pack_bf16x2(lo - __uint_as_float(w << 16), hi - __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// two bf16 (element 0 in the low half) -> two f16, round to nearest
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Eight E2M1 codes (element k in bits 4k .. 4k+3 of w) -> four f16x2 words
// (element 2i in the low half of word i): one hardware conversion per byte.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t o[4]) {
  asm("{ .reg .b8 t0, t1, t2, t3;\n mov.b32 {t0, t1, t2, t3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, t0;\n cvt.rn.f16x2.e2m1x2 %1, t1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, t2;\n cvt.rn.f16x2.e2m1x2 %3, t3; }"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}

// Two E4M3 bytes (element 0 in bits 0..7) -> one f16x2 word (element 0 in the
// low half).  Exact: every E4M3 value is an f16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t d;
  asm("{ .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(two));
  return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// byte offset of (row, byte) in a 1 KB-aligned SW128 region of 128-byte rows
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t byte) {
  return row * 128u + ((((byte >> 4) ^ (row & 7u)) << 4) | (byte & 15u));
}

// 2^x, approximate (the MUFU unit), subnormal results flushed to zero
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void named_sync(uint32_t id, uint32_t n) {
  asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(n) : "memory");
}

// 32 consecutive TMEM columns of this thread's lane -> r (waited)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  tc::tmem_ld_x32_nowait(taddr, r);
  tc::tmem_wait_ld_regs(r);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                  "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                  "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
                  "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
                  "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}

// transpose-reduction over the 32 lanes of a warp: afterwards lane l holds the
// reduction of column l (r[l] of every lane); r is destroyed
template <bool MAX>
__device__ __forceinline__ float lane_columns(float* r, int lane) {
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) {
    const bool upper = (lane & k) != 0;
#pragma unroll
    for (int i = 0; i < k; i++) {
      const float send = upper ? r[i] : r[i + k];
      const float keep = upper ? r[i + k] : r[i];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, send, k);
      r[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return r[0];
}

// ------------------------------------------------------------------ host side
// E4M3 matrix [rows][512] with unswizzled boxes of 64 bytes x box_rows rows.
inline bool encode_u8_rows512(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 matrix [rows][512] with SW128 boxes of 64 columns x box_rows rows.
inline bool encode_bf16_rows512(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, rows};
  cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace csa2
