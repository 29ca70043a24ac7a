// Eviction: the units (1 or 8 entries) of a cache that gathered the least weight leave, the
// others move to the front in their order.
//
// evict_select_kernel: a cluster of EV_CLUSTER CTAs a sequence.  Units become 32-bit
// keys in the order of their weights (the largest of a unit's entries; forced units above
// all); three radix passes (11, 11, 10 bits) with histograms in shared memory, joined over
// the cluster, find the key of the last unit that stays and how many of its equals do; a last walk
// writes the numbers of the units that stay, ascending.  A CTA keeps its slice of the keys in
// shared memory when it fits.
//
// evict_move_kernel: a CTA moves a chunk of units: their bytes into shared memory, then to
// where they go, one contiguous piece an array.  In place a chunk may be written only when the
// chunks before it have been read (a unit never moves up, so a chunk's sources lie at or
// behind its own place, and what it writes are sources of the chunks before it or its own).  Chunks are
// taken by ticket, in order: all a CTA waits for (with a limit) are flags of CTAs that run
// already and wait for nothing before they set them.
//
// Bound by HBM: the bytes that stay, in and out.
#include <cuda_runtime.h>

#include "common.cuh"
#include "host_once.cuh"
#include "params.cuh"
#include "tc.cuh"

namespace csa2 {

constexpr int EV_CLUSTER = 8, EV_THREADS = 1024, EV_BINS = 2048;
constexpr int EV_KEYS = 48 * 1024;                        // of a slice that are kept in shared memory at most
constexpr uint32_t EV_FORCED = 0xFFFFFFFFu;
constexpr int EV_MOVE_THREADS = 256, EV_MOVE_BYTES = 96 * 1024;
constexpr int EV_ZEROS = 16384;                           // weights behind the last that a CTA clears

struct EvSelect {
  int hist[EV_BINS];
  int warp_sum[EV_THREADS / 32];
  int warp_eq[EV_THREADS / 32];
  int bin, above;                     // the pass's bin, keys of the sequence above it
  int gt, eq;                         // of this CTA: keys above the last key, equal to it
  uint32_t keys[1];                   // the slice, when it fits
};

__device__ __forceinline__ uint32_t ev_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void ev_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// the int at `p`'s place in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ int ev_remote(const int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t ev_key(float w) {
  if (w != w) return 0u;                              // NaN: below every number
  return float_key(w == 0.f ? 0.f : w);               // -0 is 0
}

// Key of unit u of a sequence with n entries.
template <int UNIT>
__device__ __forceinline__ uint32_t ev_unit_key(const EvParams& p, const float* w, int64_t u, int64_t n) {
  if (u < p.first || u >= (p.recent > 0 ? max(n - p.recent, (int64_t)0) / UNIT : INT64_MAX)) return EV_FORCED;
  if (UNIT == 1) return ev_key(__ldcg(w + u));
  uint32_t k = 0u;
  if (u * UNIT + UNIT <= n) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(w + u * UNIT)), c = __ldcg(reinterpret_cast<const float4*>(w + u * UNIT) + 1);
    k = max(max(max(ev_key(a.x), ev_key(a.y)), max(ev_key(a.z), ev_key(a.w))),
            max(max(ev_key(c.x), ev_key(c.y)), max(ev_key(c.z), ev_key(c.w))));
  } else {
    for (int64_t j = u * UNIT; j < n; j++) k = max(k, ev_key(__ldcg(w + j)));
  }
  return k;
}

template <int UNIT>
__global__ void __launch_bounds__(EV_THREADS, 1) evict_select_kernel(EvParams p, int slots) {
  extern __shared__ __align__(16) unsigned char smem[];
  EvSelect& sm = *reinterpret_cast<EvSelect*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = ev_cluster_rank();
  const int b = (int)(blockIdx.x / EV_CLUSTER);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t given = p.n_entries[b];
  const int64_t n = max((int64_t)0, min((int64_t)given, p.cap));
  if (given > p.cap && rank == 0 && tid == 0) report(p.hdr, CSA2_ERR_BOUNDS, given);
  const int64_t units = (n + UNIT - 1) / UNIT, K = p.units;
  const int count = (int)min(units, K);
  int32_t* kept = p.kept + (int64_t)b * K;
  // flags of the moves, and behind the last kept unit: -1
  for (int64_t i = rank * EV_THREADS + tid; i < p.chunks; i += EV_CLUSTER * EV_THREADS) p.flags[(int64_t)b * p.chunks + i] = 0;
  for (int64_t i = count + rank * EV_THREADS + tid; i < K; i += EV_CLUSTER * EV_THREADS) kept[i] = -1;
  if (rank == 0 && tid == 0) p.marks[b] = 0;
  if (b == 0 && rank == 0 && tid == 0) *p.ticket = 0u;
  if (units <= K) {                                   // all stay
    for (int64_t i = rank * EV_THREADS + tid; i < units; i += EV_CLUSTER * EV_THREADS) kept[i] = (int32_t)i;
    ev_cluster_sync();                                // every CTA has read n_entries
    if (rank == 0 && tid == 0) {
      p.n_new[b] = (int32_t)n;
      p.n_out[b] = (int32_t)n;
    }
    return;
  }
  const float* w = p.weights + (int64_t)b * p.cap;
  const int64_t per = (units + EV_CLUSTER - 1) / EV_CLUSTER, u0 = min(per * rank, units);
  const int mine = (int)(min(u0 + per, units) - u0);
  const bool cached = mine <= slots;
  auto key = [&](int i) { return cached ? sm.keys[i] : ev_unit_key<UNIT>(p, w, u0 + i, n); };
  if (cached)
    for (int i = tid; i < mine; i += EV_THREADS) sm.keys[i] = ev_unit_key<UNIT>(p, w, u0 + i, n);
  int64_t left = K;                                   // units still to be found at or below the prefix's bins
  uint32_t prefix = 0u;
  int gt = 0;                                         // keys of this CTA above the prefix so far
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < EV_BINS; i += EV_THREADS) sm.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < mine; i += EV_THREADS) {
      const uint32_t k = key(i);
      if (pass == 0 || (k ^ prefix) >> (shift + bits) == 0u) atomicAdd(&sm.hist[k >> shift & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    ev_cluster_sync();
    // thread t has bins 2 t', 2 t' + 1 from the top, t' = EV_THREADS - 1 - t
    const int lo = 2 * (EV_THREADS - 1 - tid);
    int own[2] = {sm.hist[lo], sm.hist[lo + 1]}, all[2] = {0, 0};
#pragma unroll
    for (uint32_t r = 0; r < EV_CLUSTER; r++) {
      all[0] += ev_remote(&sm.hist[lo], r);
      all[1] += ev_remote(&sm.hist[lo + 1], r);
    }
    // sums over the threads before this one (the bins above)
    int sum = all[0] + all[1], own_sum = own[0] + own[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d), y = __shfl_up_sync(0xFFFFFFFFu, own_sum, d);
      if (lane >= d) sum += x, own_sum += y;
    }
    if (lane == 31) sm.warp_sum[warp] = sum, sm.warp_eq[warp] = own_sum;
    __syncthreads();
    if (warp == 0) {
      int x = sm.warp_sum[lane], y = sm.warp_eq[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, x, d), c = __shfl_up_sync(0xFFFFFFFFu, y, d);
        if (lane >= d) x += a, y += c;
      }
      sm.warp_sum[lane] = x, sm.warp_eq[lane] = y;
    }
    __syncthreads();
    const int before = (warp ? sm.warp_sum[warp - 1] : 0) + sum - all[0] - all[1];
    const int own_before = (warp ? sm.warp_eq[warp - 1] : 0) + own_sum - own[0] - own[1];
    // the bin in which the `left`-th key from the top lies
    if (before < left && left <= (int64_t)before + all[1]) {
      sm.bin = lo + 1;
      sm.above = before;
      sm.gt = own_before;
      sm.eq = own[1];
    } else if (before + all[1] < left && left <= (int64_t)before + all[1] + all[0]) {
      sm.bin = lo;
      sm.above = before + all[1];
      sm.gt = own_before + own[1];
      sm.eq = own[0];
    }
    __syncthreads();
    prefix |= (uint32_t)sm.bin << shift;
    left -= sm.above;
    gt += sm.gt;
    ev_cluster_sync();                                // all have read this pass's histogram
  }
  const uint32_t last = prefix;                       // key of the last unit that stays; `left` of its equals do
  if (tid == 0) sm.gt = gt;
  ev_cluster_sync();
  if (rank == 0 && tid == 0) {
    // the last unit may be a part, which is not kept when another of its key comes first
    const int64_t tail = n - (units - 1) * UNIT;
    bool tail_stays = true;
    if (UNIT > 1 && tail < UNIT) {
      const uint32_t k = ev_unit_key<UNIT>(p, w, units - 1, n);
      int equal = 0;
      for (uint32_t r = 0; r < EV_CLUSTER; r++) equal += ev_remote(&sm.eq, r);
      tail_stays = k > last || (k == last && left == equal);
    }
    const int32_t out = (int32_t)(K * UNIT - (tail_stays ? UNIT - tail : 0));
    p.n_new[b] = out;
    p.n_out[b] = out;
  }
  int64_t gt_base = 0, eq_base = 0;                   // of the CTAs before this one
  for (uint32_t r = 0; r < rank; r++) {
    gt_base += ev_remote(&sm.gt, r);
    eq_base += ev_remote(&sm.eq, r);
  }
  ev_cluster_sync();                                  // (no CTA leaves while another reads its shared memory)
  constexpr int EACH = 8;                             // units of a thread in a row
  for (int i0 = 0; i0 < mine; i0 += EACH * EV_THREADS) {
    uint32_t k[EACH];
    int g = 0, e = 0;
#pragma unroll
    for (int x = 0; x < EACH; x++) {
      const int i = i0 + EACH * tid + x;
      k[x] = i < mine ? key(i) : 0u;
      if (i < mine) {
        g += k[x] > last;
        e += k[x] == last;
      }
    }
    int gs = g, es = e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, gs, d), y = __shfl_up_sync(0xFFFFFFFFu, es, d);
      if (lane >= d) gs += x, es += y;
    }
    __syncthreads();                                  // the sums of the turn before are read
    if (lane == 31) sm.warp_sum[warp] = gs, sm.warp_eq[warp] = es;
    __syncthreads();
    int64_t gp = gt_base + gs - g, ep = eq_base + es - e;
    int gt_all = 0, eq_all = 0;
    for (int x = 0; x < EV_THREADS / 32; x++) {
      const int a = sm.warp_sum[x], c = sm.warp_eq[x];
      if (x < warp) gp += a, ep += c;
      gt_all += a;
      eq_all += c;
    }
    gt_base += gt_all;
    eq_base += eq_all;
#pragma unroll
    for (int x = 0; x < EACH; x++) {
      const int i = i0 + EACH * tid + x;
      if (i >= mine) break;
      if (k[x] > last) {
        kept[gp + min(ep, left)] = (int32_t)(u0 + i);
        gp++;
      } else if (k[x] == last) {
        if (ep < left) kept[gp + ep] = (int32_t)(u0 + i);
        ep++;
      }
    }
  }
}

__device__ __forceinline__ void ev_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void ev_bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
               :: "l"(dst), "r"(tc::smem_u32(src)), "r"(bytes) : "memory");
}

// BITS of the cache's entries, UNIT entries that move together.
template <int BITS, int UNIT>
struct Ev {
  static constexpr int ROW = BITS == 8 ? D : MAIN_BYTES;            // bytes of an entry
  static constexpr int BYTES = UNIT * (ROW + 4) + (BITS == 8 ? 4 : UNIT * (IDX_CODE_BYTES + IDX_SCALE_BYTES));
  static constexpr int MOST = EV_MOVE_BYTES / BYTES;
  static constexpr int CHUNK = MOST < 256 ? MOST : 256;             // units
  static constexpr int SMEM = CHUNK * BYTES + 64;
};

template <int BITS, int UNIT>
__global__ void __launch_bounds__(EV_MOVE_THREADS) evict_move_kernel(EvParams p) {
  using C = Ev<BITS, UNIT>;
  constexpr int CU = C::CHUNK, CE = CU * UNIT;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* rows = smem;                         // entries, index codes, then 4-byte words
  unsigned char* idx = rows + CE * C::ROW;
  uint32_t* word = reinterpret_cast<uint32_t*>(idx + (BITS == 8 ? 0 : CE * IDX_CODE_BYTES));   // index scales, or a scale a unit
  float* weight = reinterpret_cast<float*>(word + (BITS == 8 ? CU : CE));
  __shared__ uint32_t ticket;
  __shared__ int from[CU];
  __shared__ int late;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) {
    ticket = atomicAdd(p.ticket, 1u);
    late = 0;
  }
  __syncthreads();
  const int b = (int)(ticket % (uint32_t)p.B);
  const int64_t c = ticket / (uint32_t)p.B;           // chunks first, then the clearing of weights
  const int64_t n = p.n_new[b], chunks = (n + CE - 1) / CE;
  int32_t* flags = p.flags + (int64_t)b * p.chunks;
  // the chunks before `before` have been read (those before the mark are known to have been)
  auto wait_for = [&](int64_t before) {
    bool there = true;
    int32_t mark;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(mark) : "l"(p.marks + b) : "memory");
    for (int64_t i = mark + tid; i < before && there; i += EV_MOVE_THREADS) {
      int32_t f = 0;
      for (uint32_t it = 0; it < 4000000u; it++) {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(f) : "l"(flags + i) : "memory");
        if (f) break;
        __nanosleep(64);
      }
      there = f != 0;
    }
    if (!there) {
      late = 1;
      report(p.hdr, CSA2_ERR_TIMEOUT, 70);
    }
    __syncthreads();
    if (tid == 0 && late == 0) {
      __threadfence();
      atomicMax(p.marks + b, (int32_t)before);
    }
    return late == 0;
  };
  if (c >= p.chunks) {                                // weights behind the last entry: zeros
    const int64_t lo = max((c - p.chunks) * EV_ZEROS, n), hi = min((c - p.chunks + 1) * EV_ZEROS, p.to_cap);
    if (lo >= hi || (p.in_place && !wait_for(chunks))) return;
    for (int64_t j = lo + tid; j < hi; j += EV_MOVE_THREADS) p.to_weights[b * p.to_cap + j] = 0.f;
    return;
  }
  if (c >= chunks) return;
  const int64_t d0 = c * CE;                          // entries d0 .. of the result
  const int ne = (int)min((int64_t)CE, n - d0), nu = (ne + UNIT - 1) / UNIT;
  for (int i = tid; i < nu; i += EV_MOVE_THREADS) from[i] = __ldcg(p.kept + b * p.units + c * CU + i);
  __syncthreads();
  // else all of it stays where it is
  const bool moves = !p.in_place || from[nu - 1] != c * CU + nu - 1 || (p.to_weights && p.to_weights != p.weights);
  const int64_t e0 = (int64_t)b * p.cap, t0 = (int64_t)b * p.to_cap + d0;
  if (moves) {
    constexpr int RP = C::ROW / 16, IP = IDX_CODE_BYTES / 16;
    for (int i = tid; i < ne * RP; i += EV_MOVE_THREADS) {
      const int e = i / RP, x = i - e * RP;
      ev_copy16(rows + (int64_t)i * 16, p.rows + (e0 + (int64_t)from[e / UNIT] * UNIT + e % UNIT) * C::ROW + x * 16);
    }
    if (BITS == 4 && p.idx_codes)
      for (int i = tid; i < ne * IP; i += EV_MOVE_THREADS) {
        const int e = i / IP, x = i - e * IP;
        ev_copy16(idx + i * 16, p.idx_codes + (e0 + (int64_t)from[e / UNIT] * UNIT + e % UNIT) * IDX_CODE_BYTES + x * 16);
      }
    if (BITS == 4 && p.idx_codes)
      for (int e = tid; e < ne; e += EV_MOVE_THREADS)
        word[e] = __ldcg(reinterpret_cast<const uint32_t*>(p.idx_scales) + e0 + (int64_t)from[e / UNIT] * UNIT + e % UNIT);
    if (BITS == 8)
      for (int u = tid; u < nu; u += EV_MOVE_THREADS)
        word[u] = __ldcg(reinterpret_cast<const uint32_t*>(p.scales) + e0 / UNIT + from[u]);
    if (p.to_weights)
      for (int e = tid; e < ne; e += EV_MOVE_THREADS)
        weight[e] = __ldcg(p.weights + e0 + (int64_t)from[e / UNIT] * UNIT + e % UNIT);
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc::fence_proxy_async_smem();                     // the stores below read it through the asynchronous proxy
  }
  __syncthreads();
  if (p.in_place) {
    if (tid == 0) asm volatile("st.release.gpu.global.s32 [%0], %1;" :: "l"(flags + c), "r"(1) : "memory");
    if (!moves || !wait_for(c)) return;
  }
  if (tid == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");
    ev_bulk_store(p.to_rows + t0 * C::ROW, rows, (uint32_t)(ne * C::ROW));
    if (BITS == 4 && p.idx_codes) ev_bulk_store(p.to_idx_codes + t0 * IDX_CODE_BYTES, idx, (uint32_t)(ne * IDX_CODE_BYTES));
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  if (BITS == 4 && p.idx_codes)
    for (int e = tid; e < ne; e += EV_MOVE_THREADS) reinterpret_cast<uint32_t*>(p.to_idx_scales)[t0 + e] = word[e];
  if (BITS == 8)
    for (int u = tid; u < nu; u += EV_MOVE_THREADS) reinterpret_cast<uint32_t*>(p.to_scales)[t0 / UNIT + u] = word[u];
  if (p.to_weights)
    for (int e = tid; e < ne; e += EV_MOVE_THREADS) p.to_weights[t0 + e] = weight[e];
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ host side
int64_t evict_chunks(int bits, int unit, int64_t units) {
  const int c = bits == 8 ? Ev<8, 8>::CHUNK : unit == 1 ? Ev<4, 1>::CHUNK : Ev<4, 8>::CHUNK;
  return ceil_div(units, c);
}

template <int UNIT>
static cudaError_t ev_select(const EvParams& p, cudaLaunchConfig_t cfg) {
  static PerDeviceOnce attrs;
  constexpr int most = (int)sizeof(EvSelect) + EV_KEYS * 4;
  cudaError_t e = attrs.ensure([](int) {
    return cudaFuncSetAttribute(evict_select_kernel<UNIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  const int64_t slice = ceil_div(ceil_div(p.cap, UNIT), EV_CLUSTER);
  const int slots = (int)(slice < EV_KEYS ? slice : EV_KEYS);
  cfg.gridDim = dim3((unsigned)p.B * EV_CLUSTER);
  cfg.blockDim = dim3(EV_THREADS);
  cfg.dynamicSmemBytes = sizeof(EvSelect) + (size_t)slots * 4;
  cudaLaunchAttribute attr[2];
  attr[0] = cfg.attrs[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = EV_CLUSTER;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<UNIT>, p, slots);
}

template <int BITS, int UNIT>
static cudaError_t ev_move(const EvParams& p, cudaLaunchConfig_t cfg) {
  using C = Ev<BITS, UNIT>;
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure([](int) {
    return cudaFuncSetAttribute(evict_move_kernel<BITS, UNIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  const int64_t zeros = p.to_weights ? ceil_div(p.to_cap, EV_ZEROS) : 0;
  cfg.gridDim = dim3((unsigned)(p.B * (p.chunks + zeros)));
  cfg.blockDim = dim3(EV_MOVE_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<BITS, UNIT>, p);
}

cudaError_t launch_evict(EvParams p, int bits, int unit, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  p.chunks = evict_chunks(bits, unit, p.units);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = unit == 1 ? ev_select<1>(p, cfg) : ev_select<8>(p, cfg);
  if (e != cudaSuccess) return e;
  return bits == 8 ? ev_move<8, 8>(p, cfg) : unit == 1 ? ev_move<4, 1>(p, cfg) : ev_move<4, 8>(p, cfg);
}

}  // namespace csa2
