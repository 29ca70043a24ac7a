// Queries and window keys: RMSNorm per head and the rotation of the last 64
// channels in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w        over the 512 channels of a head
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos)
//                                            pairs a = 448 + 2i, b = a + 1,
//                                            cos/sin from row pos of the table
//
// Everything between the bf16 load and the final rounding (bf16, or E4M3 for a
// window stored in 8 bits) is binary32: the squares, their sum and the
// reciprocal root lose nothing that the 8 significant bits of the result hold.
//
// Bound by HBM: a token reads and writes 64 KB of queries and 1 + 1 KB (or
// 512 B) of window row against 0.2 Mflop.  One warp takes one row (a head of a
// token, or a token's key row) or, in long calls, two heads of a token; lane l owns
// channels 8l .. 8l + 7 and 256 + 8l .. 256 + 8l + 7 of a row, so every load and store of
// a warp is 512 contiguous bytes.  The rotated tail lies in the second half of lanes
// 24..31 (four pairs a lane).
// Rows a warp and CTAs an SM, us for 16 / 300 / 777 / 1500 / 3000 / 8192 tokens: 1 and 12
// 2.0 / 7.6 / 18.0 / 32.1 / 61.5 / 164.7, 2 and 10 (48 registers, one of them spilled) 2.3 / 8.0 / 17.6 /
// 30.6 / 58.2 / 155.2 (7.0 TB/s), 2 and 12 (40 registers, more spills) 157.8 at 8192, 4 rows 158.7.
// Two rows keep more loads in flight; one fills a short call's only waves better.
#include "host_once.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int QK_THREADS = 128;
constexpr int qk_ctas(int rows) { return rows == 1 ? 12 : 10; }   // an SM: at most 40 and 48 registers
constexpr int64_t QK_LONG = 600;                    // tokens from which a warp takes two heads

__device__ __forceinline__ uint32_t qk_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// a in the low byte
__device__ __forceinline__ uint32_t qk_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void qk_unpack(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// 1 / sqrt(mean square + eps) of a row, from this lane's 16 channels of it
__device__ __forceinline__ float qk_inv_rms(const uint4& a, const uint4& b, float eps) {
  float f[16];
  qk_unpack(a, f);
  qk_unpack(b, f + 8);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) s = fmaf(f[i], f[i], s);
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
  return 1.0f / sqrtf(s * (1.0f / D) + eps);
}

// eight channels of the half `half` (0: 8l.., 1: 256 + 8l..) scaled, weighted and rotated
__device__ __forceinline__ void qk_finish(const uint4& v, float r, const float4* w, int half, int lane,
                                          const float4* cs, float* f) {
  qk_unpack(v, f);
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] *= r;
  if (w) {
    const float4 w0 = __ldca(w + 64 * half + 2 * lane), w1 = __ldca(w + 64 * half + 2 * lane + 1);
    const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] *= wv[i];
  }
  if (half == 1 && lane >= 24) {
    const float4 c0 = __ldca(cs + 2 * (lane - 24)), c1 = __ldca(cs + 2 * (lane - 24) + 1);   // cos, sin, cos, sin
    const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float y0 = f[2 * i], y1 = f[2 * i + 1];
      f[2 * i] = y0 * c[i] - y1 * s[i];
      f[2 * i + 1] = y0 * s[i] + y1 * c[i];
    }
  }
}

__device__ __forceinline__ uint4 qk_pack_bf16(const float* f) {
  return make_uint4(qk_bf16x2(f[0], f[1]), qk_bf16x2(f[2], f[3]), qk_bf16x2(f[4], f[5]), qk_bf16x2(f[6], f[7]));
}

// A token's row of the rotation table, or null when the token is padding (-1)
// or its position lies outside the table (reported).
__device__ __forceinline__ const float4* qk_table_row(const QkParams& p, int64_t pos, bool reports) {
  if (pos >= 0 && pos < p.rope_P) return reinterpret_cast<const float4*>(p.rope_cs + pos * D_ROPE);
  if (pos != -1 && reports) report(p.hdr, CSA2_ERR_BOUNDS, pos);
  return nullptr;
}

// QROWS: neighbouring heads of a token that a warp takes.
template <int QROWS>
__global__ void __launch_bounds__(QK_THREADS, qk_ctas(QROWS)) qk_norm_rope_kernel(QkParams p) {
  // (what the kernel before writes is not read-only for this one's life: no __ldg, and every load behind
  // the wait)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * (QK_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t nq = p.q ? p.T * (H / QROWS) : 0;
  const bool is_q = g < nq;
  const int64_t token = is_q ? g / (H / QROWS) : g - nq;
  if (!is_q && (!p.k || token >= p.T)) return;
  const int head = is_q ? (int)(g % (H / QROWS)) * QROWS : 0, rows = is_q ? QROWS : 1;
  const uint4* in = reinterpret_cast<const uint4*>(is_q ? p.q + token * p.q_stride + head * D : p.k + token * p.k_stride);
  uint4 v[QROWS][2] = {};
#pragma unroll
  for (int i = 0; i < QROWS; i++)
    if (i < rows) {
      v[i][0] = __ldcs(in + i * (D / 8) + lane);
      v[i][1] = __ldcs(in + i * (D / 8) + 32 + lane);
    }
  // the queries' warps report a bad position when there are queries
  const float4* cs = qk_table_row(p, p.pos[token], lane == 0 && (is_q ? head == 0 : !p.q));
  int64_t slot = is_q ? 0 : (p.k_slot ? p.k_slot[token] : token);
  if (!cs || slot == -1) return;
  if (!is_q && (slot < 0 || slot >= p.n_rows)) {
    if (lane == 0) report(p.hdr, CSA2_ERR_BOUNDS, slot);
    return;
  }
  const float4* w = reinterpret_cast<const float4*>(is_q ? p.q_weight : p.k_weight);
#pragma unroll
  for (int i = 0; i < QROWS; i++) {
    if (i >= rows) break;
    const float r = qk_inv_rms(v[i][0], v[i][1], p.eps);
#pragma unroll
    for (int half = 0; half < 2; half++) {
      float f[8];
      qk_finish(v[i][half], r, w, half, lane, cs, f);
      if (is_q) {
        __stcs(reinterpret_cast<uint4*>(p.q_out + (token * H + head + i) * D) + 32 * half + lane, qk_pack_bf16(f));
      } else if (p.rows_fp8) {
        reinterpret_cast<uint2*>(p.rows + slot * D)[32 * half + lane] =
            make_uint2(qk_e4m3x2(f[0], f[1]) | qk_e4m3x2(f[2], f[3]) << 16,
                       qk_e4m3x2(f[4], f[5]) | qk_e4m3x2(f[6], f[7]) << 16);
      } else {
        reinterpret_cast<uint4*>(p.rows + slot * D * 2)[32 * half + lane] = qk_pack_bf16(f);
      }
    }
  }
}

cudaError_t launch_qk_norm_rope(const QkParams& p, cudaStream_t stream) {
  const int qrows = p.T >= QK_LONG ? 2 : 1;
  const int64_t tasks = (p.q ? p.T * (H / qrows) : 0) + (p.k ? p.T : 0);
  if (tasks == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div(tasks, QK_THREADS / 32));
  cfg.blockDim = dim3(QK_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qrows == 2 ? qk_norm_rope_kernel<2> : qk_norm_rope_kernel<1>, p);
}

}  // namespace csa2
