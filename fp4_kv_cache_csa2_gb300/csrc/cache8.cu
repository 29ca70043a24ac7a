// Entries of the 8-bit cache: bf16 latents to int8 codes with one scale for each
// block of 8 entries.
//
//   s = max(max |x| / 127, 2^-60)   over the block's new entries; not below the old
//                                   scale when the block keeps entries
//   code = RNE(x / s),  a kept code becomes RNE(code * s_old / s)
//
// A warp takes a block: every lane 16 channels of each of its 8 rows, in registers, so that the
// largest magnitude costs one reduction and the scale no barrier.  The quotients are
// rounded as if they were exact: x times the reciprocal, in one fma, is off by 2^-17 at most (|code| <= 127),
// so only a quotient that close to a tie is looked at again, by its rest x - n s, which one
// fma gives exactly.  A sum with 1.5 2^23 rounds and leaves the code in its
// low byte.
//
// Moves 1024 bytes in and 512 out an entry.  A warp an entry (a CTA a block) was bound by its instructions, 71 %
// of the issue slots: 13.9 us for 4 x 8191 tokens, here 10.6 (in a graph 10.3; 8.1 without the look at ties, which 28 %
// of the warps' steps of 256 values take).  1,025 CTAs of which 760 fit at once.
#include <cuda_runtime.h>

#include "common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int C8_THREADS = 128, C8_WARPS = C8_THREADS / 32;
constexpr float C8_FLOOR = 0x1p-60f;                  // least scale
constexpr uint32_t C8_MAX = 0x7F7Fu;                  // largest finite bf16
constexpr float C8_TIE = 0.49999f;                    // quotients this far from their rounding are looked at again
constexpr float C8_ROUND = 12582912.f;                // 1.5 2^23: a sum with it is rounded to whole numbers

// the low bytes of four words
__device__ __forceinline__ uint32_t c8_pack(const uint32_t* w) {
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// n = rint of a quotient next to a tie, given rest = (dividend - n * s) exactly: the exactly rounded n.
template <class F>
__device__ __forceinline__ float c8_settle(float n, F rest, F s) {
  const F half = s / 2;
  const bool odd = (int)n & 1;
  if (rest > half || (rest == half && odd)) return n + 1.f;
  if (rest < -half || (rest == -half && odd)) return n - 1.f;
  return n;
}

// two bf16 without their infinities (the largest finite) and NaN (0)
__device__ __noinline__ uint32_t c8_finite(uint32_t w) {
  uint32_t out = 0;
  for (int k = 0; k < 32; k += 16) {
    const uint32_t h = w >> k & 0xFFFFu, a = h & 0x7FFFu;
    out |= (a > 0x7F80u ? 0u : a == 0x7F80u ? (h & 0x8000u) | C8_MAX : h) << k;
  }
  return out;
}

// Eight kept codes under the new scale.
__device__ __noinline__ uint2 c8_again(uint2 had, float s_old, float s, float ratio) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int code = (int)(int8_t)((i < 4 ? had.x : had.y) >> (8 * (i & 3)) & 0xFFu);
    const float t = (float)code * ratio;              // off by 2^-16 at most
    float n = rintf(t);
    // (31-bit products: the rest is exact in 64 bits)
    if (fabsf(t - n) > 0.49998f) n = c8_settle(n, fma(-(double)n, (double)s, (double)code * (double)s_old), (double)s);
    c[i] = (uint32_t)min(max((int)n, -128), 127);
  }
  return make_uint2(c8_pack(c), c8_pack(c + 4));
}

__global__ void __launch_bounds__(C8_THREADS, 5) cache8_write_kernel(C8WriteParams p, int blocks) {
  const int64_t item = (int64_t)blockIdx.x * C8_WARPS + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= (int64_t)p.B * blocks) return;
  const int b = (int)(item / blocks), nth = (int)(item % blocks);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t start = p.start[b];
  int count = p.n_new ? p.n_new[b] : p.T;
  if (nth == 0 && lane == 0) {
    if (count < 0 || count > p.T) report(p.hdr, CSA2_ERR_BOUNDS, count);
    const int c = min(max(count, 0), p.T);
    if (c > 0 && start < 0) report(p.hdr, CSA2_ERR_BOUNDS, start);
    else if (c > 0 && (start > p.cap || p.cap - start < c)) report(p.hdr, CSA2_ERR_BOUNDS, max(start, p.cap));
  }
  count = min(max(count, 0), p.T);
  if (start >= p.cap || start <= -(int64_t)count) return;
  const int64_t lo = max(start, (int64_t)0), hi = min(start + count, p.cap);   // entries written
  const int64_t block = lo / BLK + nth, e0 = block * BLK;
  if (e0 >= hi) return;
  // rows r0 .. r1 - 1 are written; those before r0, and from r1 on those below `there`, are kept
  const int r0 = (int)max(lo - e0, (int64_t)0), r1 = (int)min(hi - e0, (int64_t)BLK);
  const uint4* in = reinterpret_cast<const uint4*>(p.x + ((int64_t)b * p.T + (e0 - start)) * p.x_stride) + lane;
  uint4 v[BLK][2];
#pragma unroll
  for (int r = 0; r < BLK; r++)
#pragma unroll
    for (int g = 0; g < 2; g++)
      v[r][g] = r >= r0 && r < r1 ? __ldcs(in + r * (p.x_stride / 8) + 32 * g) : make_uint4(0u, 0u, 0u, 0u);
  float* scale_at = p.scales + (int64_t)b * (p.cap / BLK) + block;
  const int there = r1 < BLK ? (int)min(max(min((int64_t)p.n_entries[b], p.cap) - e0, (int64_t)0), (int64_t)BLK) : 0;
  const bool keeps = r0 > 0 || there > r1;
  const float s_old = keeps ? *scale_at : 0.f;
  uint2* out = reinterpret_cast<uint2*>(p.codes + ((int64_t)b * p.cap + e0) * D) + lane;
  uint32_t m2 = 0u;                                   // largest magnitudes of the even and odd channels, bf16 bits
#pragma unroll
  for (int r = 0; r < BLK; r++)
#pragma unroll
    for (int g = 0; g < 2; g++)
      m2 = __vmaxu2(__vmaxu2(__vmaxu2(m2, v[r][g].x & 0x7FFF7FFFu), __vmaxu2(v[r][g].y & 0x7FFF7FFFu, v[r][g].z & 0x7FFF7FFFu)),
                    v[r][g].w & 0x7FFF7FFFu);
  if (__any_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16) > C8_MAX)) {
    m2 = 0u;
#pragma unroll
    for (int r = 0; r < BLK; r++)
#pragma unroll
      for (int g = 0; g < 2; g++) {
        v[r][g] = make_uint4(c8_finite(v[r][g].x), c8_finite(v[r][g].y), c8_finite(v[r][g].z), c8_finite(v[r][g].w));
        m2 = __vmaxu2(__vmaxu2(__vmaxu2(m2, v[r][g].x & 0x7FFF7FFFu), __vmaxu2(v[r][g].y & 0x7FFF7FFFu, v[r][g].z & 0x7FFF7FFFu)),
                      v[r][g].w & 0x7FFF7FFFu);
      }
  }
  const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  float s = fmaxf(__fdiv_rn(bf16_bits_to_f32(most), 127.f), C8_FLOOR);
  if (keeps) s = fmaxf(s, s_old);
  __syncwarp();                                       // every lane has read the old scale
  if (lane == 0) *scale_at = s;
  const float inv = __fdiv_rn(1.f, s);
#pragma unroll
  for (int r = 0; r < BLK; r++) {
    if (r < r0 || r >= r1) continue;
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const uint32_t x[4] = {v[r][g].x, v[r][g].y, v[r][g].z, v[r][g].w};
      uint32_t c[8];
      float far = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float f = __uint_as_float(i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16), w = fmaf(f, inv, C8_ROUND);
        far = fmaxf(far, fabsf(fmaf(f, inv, C8_ROUND - w)));
        c[i] = __float_as_uint(w);
      }
      if (far > C8_TIE) {
        // (one value in 300, more often than by chance: quotients of 8-bit numbers, all of one scale.)  The rest
        // x - n s is exact; beyond half of s, or at it with an odd code, the code moves towards it.
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float f = __uint_as_float(i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
          const float rest = fmaf(C8_ROUND - __uint_as_float(c[i]), s, f);
          if (__float_as_uint(fabsf(rest)) + (c[i] & 1u) > __float_as_uint(0.5f * s)) c[i] += rest < 0.f ? ~0u : 1u;
        }
      }
      out[r * (D / 8) + 32 * g] = make_uint2(c8_pack(c), c8_pack(c + 4));
    }
  }
  if (!keeps || s == s_old) return;
  const float ratio = __fdiv_rn(s_old, s);
  uint2 had[BLK][2] = {};
#pragma unroll
  for (int r = 0; r < BLK; r++)
#pragma unroll
    for (int g = 0; g < 2; g++)
      if (r < r0 || (r >= r1 && r < there)) had[r][g] = out[r * (D / 8) + 32 * g];
#pragma unroll
  for (int r = 0; r < BLK; r++)
#pragma unroll
    for (int g = 0; g < 2; g++)
      if (r < r0 || (r >= r1 && r < there)) out[r * (D / 8) + 32 * g] = c8_again(had[r][g], s_old, s, ratio);
}

cudaError_t launch_cache8_write(const C8WriteParams& p, cudaStream_t stream) {
  const int blocks = (p.T + 2 * BLK - 2) / BLK;       // that a run of T entries can touch
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div((int64_t)p.B * blocks, C8_WARPS));
  cfg.blockDim = dim3(C8_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache8_write_kernel, p, blocks);
}

}  // namespace csa2
