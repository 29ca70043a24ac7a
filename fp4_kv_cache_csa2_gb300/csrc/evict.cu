// Eviction: the units (1 or 8 entries) of a cache that gathered the least weight leave, the
// others move to the front in their order.
//
// evict_select_kernel: a CTA or a cluster of them a sequence.  Units become 32-bit
// keys in the order of their weights (the largest of a unit's entries; forced units above
// all); three radix passes (11, 11, 10 bits) with histograms in shared memory find the
// key of the last unit that stays and how many of its equals do; a last walk
// writes the numbers of the units that stay, ascending.  A CTA keeps its slice of the keys in
// shared memory when it fits.  Of the other CTAs' histograms a CTA reads 32 sums and then the 64 bins
// under one of them: all 2048 bins of eight CTAs took 4.5 us a pass.
//
// evict_move_kernel: a CTA moves a chunk of units: their bytes into shared memory, then to
// where they go, one contiguous piece an array.  In place a chunk may be written only when those
// chunks before it have been read whose sources lie there (a unit never moves up, so they are before it);
// which they are a search over the kept numbers tells, while the chunk's own copies are on their way.
// Chunks are taken by ticket, in order: all a CTA waits for (with a limit) are flags of CTAs that
// run already and wait for nothing before they set them.  16 x 131,072 entries in place 173 us (151 into another
// cache), 1M in 8 bits 121 (107).  (Waiting for every chunk before it, with an earlier selection in both: 225 us
// instead of 213 and 280 instead of 153.)
//
// Bound by HBM: the bytes that stay, in and out.
#include <climits>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host_once.cuh"
#include "params.cuh"
#include "tc.cuh"

namespace csa2 {

constexpr int EV_BINS = 2048;
constexpr int EV_COARSE = 32, EV_FINE = EV_BINS / EV_COARSE;   // a pass finds its bin in two steps
constexpr int EV_KEYS = 48 * 1024;                        // of a slice that are kept in shared memory at most
constexpr uint32_t EV_FORCED = 0xFFFFFFFFu;
constexpr int EV_MOVE_THREADS = 256, EV_MOVE_BYTES = 24 * 1024;
constexpr int EV_ZEROS = 16384;                           // weights behind the last that a CTA clears

template <int CLUSTER, int THREADS>
struct EvSelect {
  int hist[2][EV_BINS];               // of a pass, in turn
  int coarse[2][EV_COARSE];           // its sums over EV_FINE bins
  int all_coarse[CLUSTER][EV_COARSE]; // of every CTA
  int all_fine[CLUSTER][EV_FINE];     // the bins of the chosen coarse one, of every CTA
  int warp_gt[THREADS / 32], warp_eq[THREADS / 32];
  int gt, eq;                         // of this CTA: keys above the last key, equal to it
  alignas(16) uint32_t keys[4];       // the slice, when it fits
};

__device__ __forceinline__ uint32_t ev_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of the cluster (of the CTA, when it is alone).
template <int CLUSTER>
__device__ __forceinline__ void ev_sync() {
  if (CLUSTER == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

// the int at `p`'s place in the shared memory of the cluster's CTA `rank`
template <int CLUSTER>
__device__ __forceinline__ int ev_remote(const int* p, uint32_t rank) {
  if (CLUSTER == 1) return *p;
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Sum of x over the lanes before this one.
__device__ __forceinline__ int ev_before(int x, int lane) {
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += y;
  }
  return s - x;
}

__device__ __forceinline__ uint32_t ev_key(float w) {
  if (w != w) return 0u;                              // NaN: below every number
  return float_key(w == 0.f ? 0.f : w);               // -0 is 0
}

// Keys of a sequence's units: the order of their weights, those that stay in any case above all.
template <int UNIT>
struct EvUnits {
  const float* w;                     // the sequence's weights
  int64_t n, first, recent;           // entries; units before `first` and from `recent` on are forced

  __device__ __forceinline__ uint32_t one(int64_t u) const {
    if (u < first || u >= recent) return EV_FORCED;
    uint32_t k = 0u;
    for (int64_t j = u * UNIT; j < min(u * UNIT + UNIT, n); j++) k = max(k, ev_key(__ldcg(w + j)));
    return k;
  }
  // units u .. u + 3 (u a multiple of 4; behind the last: anything)
  __device__ __forceinline__ uint4 four(int64_t u) const {
    uint32_t k[4];
    if ((u + 4) * UNIT <= n) {
      float4 v[UNIT];
#pragma unroll
      for (int i = 0; i < UNIT; i++) v[i] = __ldcg(reinterpret_cast<const float4*>(w + u * UNIT) + i);
      if (UNIT == 1) {
        k[0] = ev_key(v[0].x), k[1] = ev_key(v[0].y), k[2] = ev_key(v[0].z), k[3] = ev_key(v[0].w);
      } else {
#pragma unroll
        for (int x = 0; x < 4; x++) {
          k[x] = 0u;
#pragma unroll
          for (int i = x * UNIT / 4; i < (x + 1) * UNIT / 4; i++)
            k[x] = max(k[x], max(max(ev_key(v[i].x), ev_key(v[i].y)), max(ev_key(v[i].z), ev_key(v[i].w))));
        }
      }
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (u + x < first || u + x >= recent) k[x] = EV_FORCED;
    } else {
#pragma unroll
      for (int x = 0; x < 4; x++) k[x] = one(u + x);
    }
    return make_uint4(k[0], k[1], k[2], k[3]);
  }
};

template <int UNIT, int CLUSTER, int EV_THREADS>
__global__ void __launch_bounds__(EV_THREADS, 1024 / EV_THREADS) evict_select_kernel(EvParams p, int slots) {
  extern __shared__ __align__(128) unsigned char smem[];
  using S = EvSelect<CLUSTER, EV_THREADS>;
  constexpr int EV_WARPS = EV_THREADS / 32;
  S& sm = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = CLUSTER == 1 ? 0u : ev_cluster_rank();
  const int b = (int)(blockIdx.x / CLUSTER);
  for (int i = tid; i < 2 * EV_BINS; i += EV_THREADS) sm.hist[0][i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t given = p.n_entries[b];
  const int64_t n = max((int64_t)0, min((int64_t)given, p.cap));
  if (given > p.cap && rank == 0 && tid == 0) report(p.hdr, CSA2_ERR_BOUNDS, given);
  const int64_t units = (n + UNIT - 1) / UNIT, K = p.units;
  const int count = (int)min(units, K);
  int32_t* kept = p.kept + (int64_t)b * K;
  // flags of the moves, and behind the last kept unit: -1
  for (int64_t i = rank * EV_THREADS + tid; i < p.chunks; i += CLUSTER * EV_THREADS)
    p.flags[(int64_t)b * p.chunks + i] = 0;
  for (int64_t i = count + rank * EV_THREADS + tid; i < K; i += CLUSTER * EV_THREADS) kept[i] = -1;
  if (b == 0 && rank == 0 && tid == 0) *p.ticket = 0u;
  if (units <= K) {                                   // all stay
    for (int64_t i = rank * EV_THREADS + tid; i < units; i += CLUSTER * EV_THREADS) kept[i] = (int32_t)i;
    ev_sync<CLUSTER>();                               // every CTA has read n_entries
    if (rank == 0 && tid == 0) {
      p.n_new[b] = (int32_t)n;
      p.n_out[b] = (int32_t)n;
    }
    return;
  }
  const EvUnits<UNIT> all{p.weights + (int64_t)b * p.cap, n, p.first,
                          p.recent > 0 ? max(n - p.recent, (int64_t)0) / UNIT : INT64_MAX};
  const int64_t per = ((units + CLUSTER - 1) / CLUSTER + 3) / 4 * 4, u0 = min(per * rank, units);
  const int mine = (int)(min(u0 + per, units) - u0), quads = (mine + 3) / 4;
  const bool cached = 4 * quads <= slots;
  uint4* keys = reinterpret_cast<uint4*>(sm.keys);
  if (cached) {
    // Batches of loads, then their keys.  UNIT 8: a lane takes half a unit (a lane a unit would touch a line each),
    // neighbours join theirs.
    constexpr int BATCH = UNIT == 1 ? 4 : 8;
    const float4* w4 = reinterpret_cast<const float4*>(all.w + u0 * UNIT);
    const int fours = UNIT == 1 ? quads : (2 * mine + 31) / 32 * 32;
    // of them without a part behind the last entry
    const int whole = (int)min(max(n - u0 * UNIT, (int64_t)0) / 4, (int64_t)fours);
    const int f_lo = (int)min(max(all.first - u0, (int64_t)0), (int64_t)INT_MAX);
    const int f_hi = (int)min(max(all.recent - u0, (int64_t)0), (int64_t)INT_MAX);
    for (int i0 = tid; i0 < fours; i0 += BATCH * EV_THREADS) {
      float4 v[BATCH];
#pragma unroll
      for (int y = 0; y < BATCH; y++)
        if (i0 + y * EV_THREADS < whole) v[y] = __ldcg(w4 + i0 + y * EV_THREADS);
#pragma unroll
      for (int y = 0; y < BATCH; y++) {
        const int i = i0 + y * EV_THREADS;
        if (i >= fours) continue;                     // (of UNIT 8 whole warps)
        uint32_t k[4] = {};
        if (i < whole) {
          k[0] = ev_key(v[y].x), k[1] = ev_key(v[y].y), k[2] = ev_key(v[y].z), k[3] = ev_key(v[y].w);
        } else {
          for (int x = 0; x < 4; x++)
            if (u0 * UNIT + 4 * (int64_t)i + x < n) k[x] = ev_key(__ldcg(all.w + u0 * UNIT + 4 * (int64_t)i + x));
        }
        if (UNIT == 1) {
          if (4 * i < f_lo || 4 * i + 3 >= f_hi)
            for (int x = 0; x < 4; x++)
              if (4 * i + x < f_lo || 4 * i + x >= f_hi) k[x] = EV_FORCED;
          keys[i] = make_uint4(k[0], k[1], k[2], k[3]);
        } else {
          uint32_t most = max(max(k[0], k[1]), max(k[2], k[3]));
          most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
          if ((i & 1) == 0 && i / 2 < 4 * quads) sm.keys[i / 2] = i / 2 < f_lo || i / 2 >= f_hi ? EV_FORCED : most;
        }
      }
    }
  }
  auto four = [&](int i) { return cached ? keys[i] : all.four(u0 + 4 * (int64_t)i); };
  int left = (int)K;                                  // keys still to be found among those with the prefix
  uint32_t prefix = 0u;
  int gt = 0;                                         // keys of this CTA above the prefix
  int eq = 0;                                         // keys of this CTA with it
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    // (the first pass's buffer again in the third: between them lies a barrier that its readers have come to)
    int* hist = sm.hist[pass & 1];
    if (pass == 2)
      for (int i = tid; i < EV_BINS; i += EV_THREADS) hist[i] = 0;
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < quads; i += EV_THREADS) {
      const uint4 v = four(i);
      const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (4 * i + x < mine && (pass == 0 || (k[x] ^ prefix) >> (shift + bits) == 0u))
          atomicAdd(&hist[k[x] >> shift & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    for (int c = warp; c < EV_COARSE; c += EV_WARPS) {
      const int s = __reduce_add_sync(0xFFFFFFFFu, hist[EV_FINE * c + lane] + hist[EV_FINE * c + 32 + lane]);
      if (lane == 0) sm.coarse[pass & 1][c] = s;
    }
    ev_sync<CLUSTER>();
    if (warp < CLUSTER) sm.all_coarse[warp][lane] = ev_remote<CLUSTER>(&sm.coarse[pass & 1][lane], warp);
    __syncthreads();
    // Lane l has bin EV_COARSE - 1 - l; in every warp the same.
    int sum = 0;
#pragma unroll
    for (int r = 0; r < CLUSTER; r++) sum += sm.all_coarse[r][EV_COARSE - 1 - lane];
    int own = sm.all_coarse[rank][EV_COARSE - 1 - lane];
    int above = ev_before(sum, lane), own_above = ev_before(own, lane);
    int at = __ffs(__ballot_sync(0xFFFFFFFFu, above < left && left <= above + sum)) - 1;
    const int coarse = EV_COARSE - 1 - at;
    left -= __shfl_sync(0xFFFFFFFFu, above, at);
    gt += __shfl_sync(0xFFFFFFFFu, own_above, at);
    for (int c = warp; c < 2 * CLUSTER; c += EV_WARPS)
      sm.all_fine[c >> 1][32 * (c & 1) + lane] =
          ev_remote<CLUSTER>(&hist[EV_FINE * coarse + 32 * (c & 1) + lane], c >> 1);
    __syncthreads();
    // lane l has bins EV_FINE - 1 - 2 l and the one below
    int2 f = make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < CLUSTER; r++) {
      f.x += sm.all_fine[r][EV_FINE - 1 - 2 * lane];
      f.y += sm.all_fine[r][EV_FINE - 2 - 2 * lane];
    }
    const int ox = sm.all_fine[rank][EV_FINE - 1 - 2 * lane], oy = sm.all_fine[rank][EV_FINE - 2 - 2 * lane];
    above = ev_before(f.x + f.y, lane);
    own_above = ev_before(ox + oy, lane);
    at = __ffs(__ballot_sync(0xFFFFFFFFu, above < left && left <= above + f.x + f.y)) - 1;
    const bool second = left > above + f.x;           // (of lane `at`)
    const int bin = EV_FINE * coarse + EV_FINE - 1 - 2 * lane - (second ? 1 : 0);
    prefix |= (uint32_t)__shfl_sync(0xFFFFFFFFu, bin, at) << shift;
    eq = __shfl_sync(0xFFFFFFFFu, second ? oy : ox, at);
    gt += __shfl_sync(0xFFFFFFFFu, own_above + (second ? ox : 0), at);
    left -= __shfl_sync(0xFFFFFFFFu, above + (second ? f.x : 0), at);
  }
  const uint32_t last = prefix;                       // key of the last unit that stays; `left` of its equals do
  if (tid == 0) {
    sm.gt = gt;
    sm.eq = eq;
  }
  ev_sync<CLUSTER>();
  int gt_base, eq_base, eq_all;                       // of the CTAs before this one; of all
  {
    const int g = lane < CLUSTER ? ev_remote<CLUSTER>(&sm.gt, lane) : 0;
    const int e = lane < CLUSTER ? ev_remote<CLUSTER>(&sm.eq, lane) : 0;
    gt_base = __reduce_add_sync(0xFFFFFFFFu, lane < (int)rank ? g : 0);
    eq_base = __reduce_add_sync(0xFFFFFFFFu, lane < (int)rank ? e : 0);
    eq_all = __reduce_add_sync(0xFFFFFFFFu, e);
  }
  // (no CTA leaves while another reads its shared memory: waited for at the end)
  if (CLUSTER > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (rank == 0 && tid == 0) {
    // the last unit may be a part, which is not kept when others of its key come first
    const int64_t tail = n - (units - 1) * UNIT;
    bool tail_stays = true;
    if (UNIT > 1 && tail < UNIT) {
      const uint32_t k = all.one(units - 1);
      tail_stays = k > last || (k == last && left == eq_all);
    }
    const int32_t out = (int32_t)(K * UNIT - (tail_stays ? UNIT - tail : 0));
    p.n_new[b] = out;
    p.n_out[b] = out;
  }
  // A warp takes a run of fours: it counts them, and when it knows what lies before them writes where they go.
  const int run = ((quads + EV_WARPS - 1) / EV_WARPS + 31) / 32 * 32, q0 = run * warp, q1 = min(q0 + run, quads);
  int g = 0, e = 0;
#pragma unroll 2
  for (int q = q0 + lane; q < q1; q += 32) {
    const uint4 v = four(q);
    const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int x = 0; x < 4; x++)
      if (4 * q + x < mine) {
        g += k[x] > last;
        e += k[x] == last;
      }
  }
  g = __reduce_add_sync(0xFFFFFFFFu, g);
  e = __reduce_add_sync(0xFFFFFFFFu, e);
  if (lane == 0) {
    sm.warp_gt[warp] = g;
    sm.warp_eq[warp] = e;
  }
  __syncthreads();
  int gp = gt_base + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sm.warp_gt[lane] : 0);
  int ep = eq_base + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sm.warp_eq[lane] : 0);
  for (int qw = q0; qw < q1; qw += 32) {
    const int q = qw + lane;
    const uint4 v = q < q1 ? four(q) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t k[4] = {v.x, v.y, v.z, v.w};
    uint32_t above[4], equal = 0u;
#pragma unroll
    for (int x = 0; x < 4; x++) {
      const bool in = q < q1 && 4 * q + x < mine;
      above[x] = __ballot_sync(0xFFFFFFFFu, in && k[x] > last);
      equal |= in && k[x] == last;
    }
    if (!__any_sync(0xFFFFFFFFu, equal)) {            // nearly always
      const uint32_t lower = (1u << lane) - 1u;
      int32_t* to = kept + gp + min(ep, left);
      int at = __popc(above[0] & lower) + __popc(above[1] & lower) + __popc(above[2] & lower) + __popc(above[3] & lower);
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (above[x] >> lane & 1u) to[at++] = (int32_t)(u0 + 4 * q + x);
      gp += __popc(above[0]) + __popc(above[1]) + __popc(above[2]) + __popc(above[3]);
      continue;
    }
    uint32_t both = 0u;                               // keys above (low half) and equal (high half) in this lane's four
#pragma unroll
    for (int x = 0; x < 4; x++)
      if (q < q1 && 4 * q + x < mine) both += (k[x] > last) + ((uint32_t)(k[x] == last) << 16);
    const uint32_t sum = (uint32_t)ev_before((int)both, lane);
    int gl = gp + (int)(sum & 0xFFFFu), el = ep + (int)(sum >> 16);
#pragma unroll
    for (int x = 0; x < 4; x++)
      if (q < q1 && 4 * q + x < mine) {
        if (k[x] > last) {
          kept[gl + min(el, left)] = (int32_t)(u0 + 4 * q + x);
          gl++;
        } else if (k[x] == last) {
          if (el < left) kept[gl + el] = (int32_t)(u0 + 4 * q + x);
          el++;
        }
      }
    gp = __shfl_sync(0xFFFFFFFFu, gl, 31);
    ep = __shfl_sync(0xFFFFFFFFu, el, 31);
  }
  if (CLUSTER > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
  // index scales, or a scale a unit
  uint32_t* word = reinterpret_cast<uint32_t*>(idx + (BITS == 8 ? 0 : CE * IDX_CODE_BYTES));
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
  const int32_t* kept = p.kept + b * p.units;
  const int count = (int)((n + UNIT - 1) / UNIT);     // units that stay
  // How many of them lie before unit x (every thread of the CTA).
  auto before = [&](int64_t x) {
    int lo = 0, left = count;
    while (left > 0) {
      const int step = (left + EV_MOVE_THREADS - 1) / EV_MOVE_THREADS, i = tid * step;
      const int hits = __syncthreads_count(i < left && __ldcg(kept + lo + i) < x);
      if (hits == 0) break;
      const int next = (hits - 1) * step + 1;
      left = min(step - 1, left - next);
      lo += next;
    }
    return lo;
  };
  // The chunks before chunk `end` that have units i0 .. i1 - 1 of those that stay have been read.
  auto wait_for = [&](int i0, int i1, int64_t end) {
    const int64_t c0 = i0 / CU, c1 = i1 > i0 ? min((int64_t)(i1 - 1) / CU + 1, end) : c0;
    bool there = true;
    for (int64_t i = c0 + tid; i < c1 && there; i += EV_MOVE_THREADS) {
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
    return late == 0;
  };
  if (c >= p.chunks) {                                // weights behind the last entry: zeros
    const int64_t lo = max((c - p.chunks) * EV_ZEROS, n), hi = min((c - p.chunks + 1) * EV_ZEROS, p.to_cap);
    if (lo >= hi || (p.in_place && !wait_for(before(lo / UNIT), before((hi + UNIT - 1) / UNIT), chunks))) return;
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
  int i0 = 0, i1 = 0;                                 // units whose sources the chunk writes over
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
    if (p.in_place) {
      i0 = before(c * CU);
      static_assert(CU <= EV_MOVE_THREADS, "one probe a unit of the chunk");
      i1 = i0 + __syncthreads_count(tid < nu && i0 + tid < count && __ldcg(kept + i0 + tid) < c * CU + nu);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc::fence_proxy_async_smem();                     // the stores below read it through the asynchronous proxy
  }
  __syncthreads();
  if (p.in_place) {
    if (tid == 0) asm volatile("st.release.gpu.global.s32 [%0], %1;" :: "l"(flags + c), "r"(1) : "memory");
    if (!moves || !wait_for(i0, i1, c)) return;
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

template <int UNIT, int CLUSTER, int THREADS>
static cudaError_t ev_select(const EvParams& p, cudaLaunchConfig_t cfg) {
  using S = EvSelect<CLUSTER, THREADS>;
  static PerDeviceOnce attrs;
  constexpr int most = (int)sizeof(S) + EV_KEYS * 4;
  static_assert(most <= 227 * 1024, "shared memory per CTA");
  auto* kernel = evict_select_kernel<UNIT, CLUSTER, THREADS>;
  cudaError_t e = attrs.ensure([kernel](int) {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess && CLUSTER > 8) r = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int64_t slice = ceil_div(ceil_div(ceil_div(p.cap, UNIT), CLUSTER), 4) * 4;
  const int slots = slice <= EV_KEYS ? (int)slice : 0;
  cfg.gridDim = dim3((unsigned)p.B * CLUSTER);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sizeof(S) + (size_t)slots * 4;
  cudaLaunchAttribute attr[2];
  attr[0] = cfg.attrs[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CLUSTER;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, slots);
}

// CTAs of a sequence's selection.  A cluster of 8 CTAs of 1024 threads fits 15 times (one to an SM), so that 16
// sequences of 131,072 took two waves, 43 us; of 512 threads 32 (26 since loads go in batches and numbers by
// ballots).  A few long ones: 16 CTAs, then 32 us, now 28 (512 threads: 40) for 131,072 blocks.
template <int UNIT>
static cudaError_t ev_select_any(const EvParams& p, const cudaLaunchConfig_t& cfg) {
  const int64_t units = ceil_div(p.cap, UNIT);
  if (units <= 8192) return ev_select<UNIT, 1, 512>(p, cfg);
  return units <= 65536 || p.B > 6 ? ev_select<UNIT, 8, 512>(p, cfg) : ev_select<UNIT, 16, 1024>(p, cfg);
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
  cudaError_t e = unit == 1 ? ev_select_any<1>(p, cfg) : ev_select_any<8>(p, cfg);
  if (e != cudaSuccess) return e;
  return bits == 8 ? ev_move<8, 8>(p, cfg) : unit == 1 ? ev_move<4, 1>(p, cfg) : ev_move<4, 8>(p, cfg);
}

}  // namespace csa2
