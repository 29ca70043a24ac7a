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

// Sixteen int8 -> eight f16x2 words (element 2i in the low half of word i), exactly: the byte
// b + 128 in the low bits of f16 1024 is 1152 + b.
__device__ __forceinline__ void i8x16_to_f16(const uint4& c, uint32_t* o) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t u = w[i] ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * i]) : "r"(prmt(u, 0x64646464u, 0x4140u)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * i + 1]) : "r"(prmt(u, 0x64646464u, 0x4342u)), "r"(0x64806480u));
  }
}

// The same -> eight bf16x2 words, exactly: b is 128 + (b & 127) less 128, or less 256 when b is negative.
__device__ __forceinline__ void i8x16_to_bf16(const uint4& c, uint32_t* o) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t u = prmt(w[i >> 1], 0x43434343u, i & 1 ? 0x4342u : 0x4140u);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(u & 0xFF7FFF7Fu), "r"(u & 0xFF80FF80u));
  }
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

// Whether x holds in any of the n threads of named barrier `id`.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t n, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.or.pred b, %2, %3, a;\n"
               " selp.u32 %0, 1, 0, b;\n}\n" : "=r"(r) : "r"((uint32_t)x), "r"(id), "r"(n) : "memory");
  return r != 0;
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

// 16 consecutive TMEM columns of this thread's lane, without waiting: valid after tmem_wait_ld16
__device__ __forceinline__ void tmem_ld_x16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr) : "memory");
}

// Waits for this thread's TMEM loads; the registers pass through the same statement.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* r, uint32_t* s) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(s[0]), "+r"(s[1]), "+r"(s[2]), "+r"(s[3]), "+r"(s[4]), "+r"(s[5]), "+r"(s[6]), "+r"(s[7]),
                 "+r"(s[8]), "+r"(s[9]), "+r"(s[10]), "+r"(s[11]), "+r"(s[12]), "+r"(s[13]), "+r"(s[14]), "+r"(s[15])
               :: "memory");
}

// 8 consecutive TMEM columns of this thread's lane
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
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

// 8-bit matrix [rows][512] with SW128 boxes of 128 columns x box_rows rows.
inline bool encode_u8_rows512_sw128(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, rows};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

// Matrices [rows][512] as column chunks of 128 bytes: half of a row's dims in one SW128 copy, chunk after chunk
// (one copy a chunk: a thread issues them at 200 cycles each).  Coordinates: 0, row, first chunk.
inline bool encode_rows512_halves(CUtensorMap* map, CUtensorMapDataType type, int bytes, const void* base, uint64_t rows,
                                  uint32_t box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const uint32_t chunk = 128 / bytes, chunks = D / chunk;
  cuuint64_t dims[3] = {chunk, rows, chunks};
  cuuint64_t strides[2] = {(cuuint64_t)(D * bytes), 128};
  cuuint32_t box[3] = {chunk, box_rows, chunks / 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool encode_bf16_rows512_halves(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  return encode_rows512_halves(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, box_rows);
}
inline bool encode_u8_rows512_halves(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  return encode_rows512_halves(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, box_rows);
}

}  // namespace csa2
