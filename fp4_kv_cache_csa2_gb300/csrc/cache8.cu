// Entries of the 8-bit cache: bf16 latents to int8 codes with one scale for each
// block of 8 entries.
//
//   s = max(max |x| / 127, 2^-60)   over the block's new entries; not below the old
//                                   scale when the block keeps entries
//   code = RNE(x / s),  a kept code becomes RNE(code * s_old / s)
//
// A CTA takes a block, a warp an entry, a lane 16 of its channels.  The quotients are
// rounded as if they were exact: x times the reciprocal is off by 2^-15 at most (|code| <= 127),
// so only a quotient that close to a tie is looked at again, by the sign of
// x - (n + 1/2) s, which one fma gives exactly.
//
// Bound by HBM: 1024 bytes in and 512 out an entry.
#include <cuda_runtime.h>

#include "common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int C8_THREADS = 32 * BLK;
constexpr float C8_FLOOR = 0x1p-60f;                  // least scale
constexpr uint32_t C8_MAX = 0x7F7Fu;                  // largest finite bf16
constexpr float C8_TIE = 0.4999f;                     // quotients this far from their rounding are looked at again

// Eight codes -> 8 bytes, code 0 in the lowest.
__device__ __forceinline__ uint2 c8_pack(const int* c) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; i++)
    w[i] = (c[4 * i] & 0xFF) | (c[4 * i + 1] & 0xFF) << 8 | (c[4 * i + 2] & 0xFF) << 16 | (uint32_t)c[4 * i + 3] << 24;
  return make_uint2(w[0], w[1]);
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

__global__ void __launch_bounds__(C8_THREADS) cache8_write_kernel(C8WriteParams p, int blocks) {
  __shared__ uint32_t most_of[BLK];
  __shared__ int keeps[BLK];
  const int b = (int)(blockIdx.x / (uint32_t)blocks), nth = (int)(blockIdx.x % (uint32_t)blocks);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t start = p.start[b];
  int count = p.n_new ? p.n_new[b] : p.T;
  if (nth == 0 && threadIdx.x == 0) {
    if (count < 0 || count > p.T) report(p.hdr, CSA2_ERR_BOUNDS, count);
    const int c = min(max(count, 0), p.T);
    if (c > 0 && start < 0) report(p.hdr, CSA2_ERR_BOUNDS, start);
    else if (c > 0 && (start > p.cap || p.cap - start < c)) report(p.hdr, CSA2_ERR_BOUNDS, max(start, p.cap));
  }
  count = min(max(count, 0), p.T);
  if (start >= p.cap || start <= -(int64_t)count) return;
  const int64_t lo = max(start, (int64_t)0), hi = min(start + count, p.cap);   // entries written
  const int64_t block = lo / BLK + nth, e = block * BLK + w;
  if (block * BLK >= hi) return;
  const bool fresh = e >= lo && e < hi;
  const bool kept = !fresh && (e < lo || e < min((int64_t)p.n_entries[b], p.cap));
  uint4 v[2] = {};
  uint32_t m2 = 0u;                                   // largest magnitudes of the even and odd channels, bf16 bits
  if (fresh) {
    const uint4* in = reinterpret_cast<const uint4*>(p.x + ((int64_t)b * p.T + (e - start)) * p.x_stride);
    v[0] = __ldcs(in + lane);
    v[1] = __ldcs(in + 32 + lane);
  }
  uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int i = 0; i < 8; i++) m2 = __vmaxu2(m2, x[i] & 0x7FFF7FFFu);
  if (__any_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16) > C8_MAX)) {
    m2 = 0u;
    for (int i = 0; i < 8; i++) {
      x[i] = c8_finite(x[i]);
      m2 = __vmaxu2(m2, x[i] & 0x7FFF7FFFu);
    }
  }
  const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  float* scale_at = p.scales + (int64_t)b * (p.cap / BLK) + block;
  const float s_old = *scale_at;
  if (lane == 0) {
    most_of[w] = most;
    keeps[w] = kept;
  }
  __syncthreads();
  uint32_t a = 0u;
  int any_kept = 0;
#pragma unroll
  for (int i = 0; i < BLK; i++) {
    a = max(a, most_of[i]);
    any_kept |= keeps[i];
  }
  float s = fmaxf(__fdiv_rn(bf16_bits_to_f32(a), 127.f), C8_FLOOR);
  if (any_kept) s = fmaxf(s, s_old);
  if (threadIdx.x == 0) *scale_at = s;                // (every read of it lies before the barrier)
  uint2* out = reinterpret_cast<uint2*>(p.codes + ((int64_t)b * p.cap + e) * D);
  if (fresh) {
    const float inv = __fdiv_rn(1.f, s);
#pragma unroll
    for (int g = 0; g < 2; g++) {
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint32_t word = x[4 * g + i / 2];
        const float f = __uint_as_float(i & 1 ? word & 0xFFFF0000u : word << 16), t = f * inv;
        float n = rintf(t);
        if (fabsf(t - n) > C8_TIE) n = c8_settle(n, fmaf(-n, s, f), s);
        c[i] = (int)n;
      }
      out[32 * g + lane] = c8_pack(c);
    }
  } else if (kept && s != s_old) {
    const float ratio = __fdiv_rn(s_old, s);
#pragma unroll
    for (int g = 0; g < 2; g++) {
      const uint2 had = out[32 * g + lane];
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int code = (int)(int8_t)((i < 4 ? had.x : had.y) >> (8 * (i & 3)) & 0xFFu);
        const float t = (float)code * ratio;
        float n = rintf(t);
        // (31-bit products: the rest is exact in 64 bits)
        if (fabsf(t - n) > C8_TIE) n = c8_settle(n, fma(-(double)n, (double)s, (double)code * (double)s_old), (double)s);
        c[i] = min(max((int)n, -128), 127);
      }
      out[32 * g + lane] = c8_pack(c);
    }
  }
}

cudaError_t launch_cache8_write(const C8WriteParams& p, cudaStream_t stream) {
  const int blocks = (p.T + 2 * BLK - 2) / BLK;       // that a run of T entries can touch
  if (p.B == 0 || p.T == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.B * (unsigned)blocks);
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
