// Attention over the 8-bit cache and a window for calls of several queries a sequence: two
// queries by a pair of CTAs, the 64 heads of each at the full rate of the tensor cores.
//
//   o_h = sum_i softmax_i(scale q_h . v_i) v_i,   lse_h = log sum_i exp(scale q_h . v_i)
//
// as in keys_attention.cu, whose chunks of 64 keys, softmax state, partial states and outputs these
// are.  There a product of 64 rows runs at half the rate, and each query's CTA widens every key for
// itself.  Here a product spans two CTAs (cta_group::2, M = 128: 64 rows in each).  Of such
// a product TMEM lanes 0 .. 63 of a CTA take the columns of B that lie in CTA 0's shared memory, lanes
// 64 .. 127 those in CTA 1's, each times the A of the lane itself: two products of 64 rows.  So CTA r
// keeps half r of the dims of every key, and
//   * S = Q K^T   A = the query's dims 0 .. 255 (lanes 0 ..), 256 .. 511 (lanes 64 ..), B = the
//     keys' dims of either CTA: 16 MMAs of N = 128; a head's score is the sum of its two lanes
//   * O += P V    A = P in both lanes of a head, B = 2 x 128 dims of either CTA: 8 MMAs of N = 256;
//     lanes 0 .. 63 hold O's dims 0 .. 255, the others 256 .. 511
// 1,079 cycles of MMAs a chunk for two queries on two SMs, against 2,074 for one on one; each CTA stages and
// widens half of a chunk (512 cycles of shared memory instead of 1024), and the products read half (512).
// The lanes of a head sit in different warps, which pass each other partial scores and weights through
// shared memory (384 cycles).
//
// Bound by shared memory: 1,900 cycles a chunk, 1,557 of them in use (by counters: 917 of the load/store
// unit, with waits and the above; 512 of products; 128 of copies), and what waits behind them: the softmax takes
// 1,600 from scores to weights.  2048 queries over 8192 entries 1.53 ms (a CTA a query 2.06),
// 3 x 37 over 10,007, 7006 and 4005 entries 105 us (134).  A pair costs 8 us beside its chunks.  Without the
// staging area, codes by 16-byte loads a chunk ahead: 0.09 ms more; two softmax groups, even and odd chunks: 0.37 more.
//
// Both queries share the keys, each with its own limits: what one of them does not see has weight 0
// for it.  So no key may hold an infinity or a NaN: codes cannot, and of window rows
// such values are written as 0 and every output of the queries that see the row becomes NaN.
//
// Roles of each CTA's warps: 0..7 move Q, then softmax (two a quarter of the lanes, a half of a lane's
// keys each: four alone take 2,200 cycles a chunk), then write the output; 8..15 fill; 16 issues the MMAs (in
// CTA 0); 17 the copies.
#include <cfloat>

#include "attn_common.cuh"
#include "keys_common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int PA_SOFT_WARPS = 8, PA_FILL_WARPS = 8;
constexpr int PA_FILL = 32 * PA_FILL_WARPS;
constexpr int PA_MMA_WARP = PA_SOFT_WARPS + PA_FILL_WARPS, PA_COPY_WARP = PA_MMA_WARP + 1;
constexpr int PA_THREADS = 32 * (PA_COPY_WARP + 1);
constexpr int PA_KEYS = KEYS_CHUNK;
constexpr int PA_COL = 64 * 128;                          // [64 rows][64 dims] 16-bit, SW128
constexpr int PA_BUF = 4 * PA_COL;                        // a chunk's 256 dims
constexpr int PA_BUFS = 4;                                // the last two take Q first
constexpr int PA_STAGE = 2 * PA_COL;                      // a chunk's 256 codes a key, SW128
constexpr int PA_STAGES = 2;
constexpr int PA_OFF_STAGE = PA_BUFS * PA_BUF;
constexpr int PA_OFF_S = PA_OFF_STAGE + PA_STAGES * PA_STAGE;   // scores for the other lane: [4][256 threads] float4
constexpr int PA_OFF_P = PA_OFF_S + 4 * 256 * 16;         // weights for the other lane: [2][256 threads] uint4
constexpr int PA_OFF_SMALL = PA_OFF_P + 2 * 256 * 16;
constexpr int PA_O_COL = 0, PA_Q_COL = 256, PA_S_COL = 384;
constexpr int PA_AHEAD = 6;                               // chunks of codes that are on their way to L2

struct PaSmall {
  uint64_t q_full, q_moved;           // TMA: Q; Q is in TMEM (both CTAs' softmax warps; CTA 0's counts)
  uint64_t stage_full[PA_STAGES], stage_free[PA_STAGES];   // TMA; a fill warp each
  uint64_t row_full[PA_BUFS];         // TMA: rows in K buffer i
  uint64_t full[PA_BUFS];             // K buffer i is filled (both CTAs' fill warps; CTA 0's counts)
  uint64_t free_[PA_BUFS];            // O of the chunk in K buffer i is done (told to both)
  uint64_t s_full[2], p_ready[2];     // S of every second chunk is done (told to both); its P is written (CTA 0's counts)
  uint64_t q_here;                    // this CTA's softmax warps have read Q
  float sum[4][H], top[4][H];         // of the softmax, a quarter of the keys each; maxima on their way to the others
  float ref[H];                       // the heads' references
  uint32_t tmem_base;
  int err, poison;                    // a row that is not finite lies before this CTA's query
};
constexpr int PA_SMEM = PA_OFF_SMALL + (int)sizeof(PaSmall);
static_assert(PA_SMEM <= 227 * 1024, "shared memory per CTA");

__device__ __noinline__ bool pa_timeout(int* err, WsHeader* hdr, int where) {
  if (atomicExch(err, 1) == 0) report(hdr, CSA2_ERR_TIMEOUT, where);
  return false;
}

// What one query sees: window rows row_lo .. row_hi - 1 of the buffer, entries 0 .. entries - 1 (each below 2^31).
struct PaQuery {
  int64_t t, lo;                      // position (below 0: none), first window position
  int row_lo, row_hi, entries;
};

__device__ __forceinline__ PaQuery pa_query(const KeysParams& p, int32_t n_entries, int64_t base, int64_t t) {
  PaQuery q{t, 0, 0, 0, 0};
  if (t < 0) return q;
  q.lo = p.W > 0 && q.t >= p.W ? q.t - p.W + 1 : 0;   // (W = 0: t + 1 need not exist)
  if (p.W > 0 && q.t >= base) {       // (unsigned differences: any two positions have one)
    const uint64_t s = (uint64_t)p.S, r0 = q.lo > base ? (uint64_t)q.lo - (uint64_t)base : 0;
    const uint64_t end = (uint64_t)q.t - (uint64_t)base, r1 = end < s ? end + 1 : s;
    if (r0 < r1) {
      q.row_lo = (int)r0;
      q.row_hi = (int)r1;
    }
  }
  const int64_t seen = (min(t, INT64_MAX - 1) + 1) >> (p.m - 1);   // (m is 1 or 2)
  q.entries = (int)max(min(seen, min((int64_t)n_entries, p.cap)), (int64_t)0);
  return q;
}

// The pair's keys: rows a0 .. (chunks before ca), rows b0 .. (before cb), entries; a CTA's run of their
// chunks is [c0, c0 + n).
struct PaRun {
  int a0, an, b0, bn, en;             // first row and number of rows of either part; entries
  int ca, cb, c0, n;
  __device__ __forceinline__ bool rows(int c) const { return c0 + c < cb; }
  // row or entry of the chunk's first key, keys of the chunk
  __device__ __forceinline__ int first(int c) const {
    const int k = c0 + c;
    return k >= cb ? PA_KEYS * (k - cb) : k < ca ? a0 + PA_KEYS * k : b0 + PA_KEYS * (k - ca);
  }
  __device__ __forceinline__ int keys(int c) const {
    const int k = c0 + c;
    return min(k >= cb ? en - PA_KEYS * (k - cb) : k < ca ? an - PA_KEYS * k : bn - PA_KEYS * (k - ca), PA_KEYS);
  }
};

__device__ __forceinline__ PaRun pa_run(const PaQuery* q, int sp, int split) {
  PaRun r{};
  const int n0 = q[0].row_hi - q[0].row_lo, n1 = q[1].row_hi - q[1].row_lo;
  r.a0 = q[0].row_lo;
  r.an = n0;
  r.b0 = q[1].row_lo;
  r.bn = n1;
  if (n0 > 0 && n1 > 0) {
    const int lo = min(q[0].row_lo, q[1].row_lo), hi = max(q[0].row_hi, q[1].row_hi);
    // windows that overlap or meet: one part.  (Else rows of one are none of the other's)
    if ((int64_t)hi - lo <= (int64_t)n0 + n1) {
      r.a0 = lo;
      r.an = hi - lo;
      r.bn = 0;
    }
  }
  r.en = max(q[0].entries, q[1].entries);
  r.ca = (int)ceil_div(r.an, PA_KEYS);
  r.cb = r.ca + (int)ceil_div(r.bn, PA_KEYS);
  const uint32_t nc = (uint32_t)r.cb + (uint32_t)ceil_div(r.en, PA_KEYS);
  const uint32_t each = nc / (uint32_t)split, more = nc % (uint32_t)split;
  r.c0 = sp * (int)each + min(sp, (int)more);
  r.n = (int)each + (sp < (int)more ? 1 : 0);
  return r;
}

__global__ void __launch_bounds__(PA_THREADS, 1)
pair_attn_kernel(KeysParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_rows,
                 const __grid_constant__ CUtensorMap map_codes) {
  extern __shared__ __align__(1024) unsigned char smem[];
  PaSmall& sm = *reinterpret_cast<PaSmall*>(smem + PA_OFF_SMALL);
  // the swizzled tiles need the declared alignment (the same in both CTAs)
  if (tc::smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) report(p.hdr, CSA2_ERR_CUDA, 5);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int rank = (int)tc::cluster_rank(), split = p.split;
  const uint32_t item = blockIdx.x / 2u, pairs = (uint32_t)(p.Q + 1) / 2u;
  const int sp = (int)(item % (uint32_t)split);
  const uint32_t pair = item / (uint32_t)split;
  const int b = (int)(pair / pairs), qi = 2 * (int)(pair % pairs);
  const bool there = qi + rank < p.Q;                 // the last pair of a sequence may have one query
  // (the loads that all else follows from are on their way while the pair sets itself up)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t base = p.W > 0 ? p.base_pos[b] : 0;
  const int64_t t0 = p.q_pos[(int64_t)b * p.Q + qi], t1 = qi + 1 < p.Q ? p.q_pos[(int64_t)b * p.Q + qi + 1] : -1;
  const int32_t n_entries = p.n_entries[b];
  const int64_t bq = (int64_t)b * p.Q + qi + rank;
  float* part = p.part + (bq * split + sp) * KA_PART_FLOATS;   // with split > 1

  if (warp == PA_MMA_WARP) tc::tmem_alloc_pair(&sm.tmem_base, 512);
  if (tid == 32 * PA_COPY_WARP) {
    tc::bar_init(&sm.q_full, 1);
    tc::bar_init_fence();
  }
  if (tid == 0) {
    tc::bar_init(&sm.q_moved, 2 * PA_SOFT_WARPS);
    tc::bar_init(&sm.q_here, PA_SOFT_WARPS);
    for (int i = 0; i < PA_STAGES; i++) {
      tc::bar_init(&sm.stage_full[i], 1);
      tc::bar_init(&sm.stage_free[i], PA_FILL_WARPS);
    }
    for (int i = 0; i < PA_BUFS; i++) {
      tc::bar_init(&sm.row_full[i], 1);
      tc::bar_init(&sm.full[i], 2 * PA_FILL_WARPS);
      tc::bar_init(&sm.free_[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.p_ready[i], 2 * PA_SOFT_WARPS);
    }
    sm.err = 0;
    sm.poison = 0;
    tc::bar_init_fence();
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_rows);
    tc::prefetch_tensormap(&map_codes);
  }
  tc::fence_before_sync();
  __syncwarp();
  tc::cluster_arrive();
  if (tid == 32 * PA_COPY_WARP && there) {            // Q into the last two K buffers
    tc::bar_arrive_expect_tx(&sm.q_full, 8u * PA_COL);
    for (int h = 0; h < 2; h++)
      tc::tma_load_3d(smem + (PA_BUFS - 2 + h) * PA_BUF, &map_q, 0, (int32_t)(bq * H), 4 * h, &sm.q_full);
  }

  const PaQuery qs[2] = {pa_query(p, n_entries, base, t0), pa_query(p, n_entries, base, t1)};
  const PaRun run = pa_run(qs, sp, split);
  __syncwarp();
  tc::cluster_wait();
  tc::fence_after_sync();
  if (sm.tmem_base != 0 && tid == 0) report(p.hdr, CSA2_ERR_CUDA, 6);
  const int n_ch = run.n;
  const PaQuery mine = rank ? qs[1] : qs[0];
  if (sp == 0 && tid == 0 && mine.t >= 0) {           // what the caller did not supply
    if (p.W > 0) {
      if (mine.lo < base) report(p.hdr, CSA2_ERR_BOUNDS, mine.lo);
      else if ((uint64_t)mine.t - (uint64_t)base >= (uint64_t)p.S) report(p.hdr, CSA2_ERR_BOUNDS, mine.t);
    }
    if (n_entries > p.cap) report(p.hdr, CSA2_ERR_BOUNDS, n_entries);
  }
  bool ok = true;                                     // a thread that has given up once waits no more
  auto wait = [&](uint64_t* bar, uint32_t use, int where) {
    if (ok) ok = tc::bar_wait(bar, use & 1u) || pa_timeout(&sm.err, p.hdr, where);
  };
  auto arrive_first = [&](uint64_t* bar) {            // on CTA 0's barrier
    if (rank) tc::bar_arrive_first(bar);
    else tc::bar_arrive(bar);
  };

  // With a window every thread comes to one more barrier of the cluster: behind it the softmax warps know whether a
  // fill warp of either CTA has met a row that is not finite.
  auto told = [&]() {
    if (p.W == 0) return;
    __syncwarp();
    tc::cluster_arrive();
    tc::cluster_wait();
  };

  if (warp == PA_MMA_WARP) {
    // ================= MMAs, in CTA 0 (the whole warp runs the loop, one lane issues)
    constexpr uint32_t idesc_s = tc::idesc_f16(128, 128, 0, 0), idesc_o = tc::idesc_f16(128, 256, 0, 1);
    const uint64_t k_d = tc::smem_desc(tc::smem_u32(smem), 16, 1024, tc::SW_128B);
    const uint64_t v_d = tc::smem_desc(tc::smem_u32(smem), PA_COL, 1024, tc::SW_128B);
    const uint32_t leader = tc::elect_one();
    const int n = rank == 0 ? (int)__reduce_or_sync(0xFFFFFFFFu, (uint32_t)n_ch) : 0;
    auto wait_mma = [&](uint64_t* bar, uint32_t use, int where) {
      if (ok) ok = tc::bar_wait_relaxed(bar, use & 1u) || pa_timeout(&sm.err, p.hdr, where);
      tc::fence_after_sync();
    };
    if (n > 0) wait_mma(&sm.q_moved, 0, 80);
    auto scores = [&](uint32_t c) {
      const uint32_t buf = c % PA_BUFS;
      wait_mma(&sm.full[buf], c / PA_BUFS, 81);
      tc::acquire_shared();
      const uint64_t ka = k_d + buf * (PA_BUF >> 4);
      const uint32_t s = PA_S_COL + 64 * (c & 1);
#pragma unroll
      for (int i = 0; i < 16; i++)
        tc::mma_f16_ts_pair(leader, s, PA_Q_COL + 8 * i, ka + ((uint32_t)((i >> 2) * PA_COL + (i & 3) * 32) >> 4), idesc_s,
                            i ? 1u : 0u);
      tc::commit_pair(leader, &sm.s_full[c & 1]);
    };
    if (n > 0) scores(0);
    for (uint32_t c = 0; c < (uint32_t)n; c++) {
      if (c + 1 < (uint32_t)n) scores(c + 1);
      wait_mma(&sm.p_ready[c & 1], c >> 1, 82);
      const uint32_t buf = c % PA_BUFS, s = PA_S_COL + 64 * (c & 1);
#pragma unroll
      for (int g = 0; g < 2; g++) {
        const uint64_t va = v_d + ((buf * PA_BUF + g * 2 * PA_COL) >> 4);
#pragma unroll
        for (int ks = 0; ks < PA_KEYS / 16; ks++)
          tc::mma_f16_ts_pair(leader, PA_O_COL + 128 * g, s + 8 * ks, va + (uint32_t)(ks * (2048 >> 4)), idesc_o,
                              (c || ks) ? 1u : 0u);
      }
      tc::commit_pair(leader, &sm.free_[buf]);
    }
    told();
  } else if (warp == PA_COPY_WARP) {
    // ================= copies: this CTA's half of the dims
    if (lane == 0 && n_ch > 0) {
      const uint8_t* kv = p.main_kv + (int64_t)b * p.cap * D;
      auto ahead = [&](int c) {                       // (each CTA sends for half of the keys, whole)
        if (c >= n_ch || run.rows(c)) return;
        const int keys = run.keys(c), k0 = rank ? keys / 2 : 0, k1 = rank ? keys : keys / 2;
        if (k1 > k0) tc::prefetch_l2(kv + (int64_t)(run.first(c) + k0) * D, (uint32_t)((k1 - k0) * D));
      };
      uint32_t staged = 0;
      for (int c = 0; c < n_ch; c++) {
        const int first = run.first(c);
        if (c == 1)                                   // (behind the first chunk's own copies)
          for (int i = 2; i < 1 + PA_AHEAD; i++) ahead(i);
        if (c > 0) ahead(c + PA_AHEAD);
        if (!run.rows(c)) {
          const uint32_t s = staged % PA_STAGES;
          if (staged >= PA_STAGES) wait(&sm.stage_free[s], staged / PA_STAGES - 1, 83);
          staged++;
          unsigned char* dst = smem + PA_OFF_STAGE + s * PA_STAGE;
          tc::bar_arrive_expect_tx(&sm.stage_full[s], PA_STAGE);
          tc::tma_load_3d(dst, &map_codes, 0, (int32_t)(b * p.cap + first), 2 * rank, &sm.stage_full[s]);
          continue;
        }
        const uint32_t buf = c % PA_BUFS, use = c / PA_BUFS;
        if (use > 0) wait(&sm.free_[buf], use - 1, 84);
        else if (buf >= PA_BUFS - 2 && there) wait(&sm.q_here, 0, 84);
        unsigned char* kt = smem + buf * PA_BUF;
        const int32_t row = (int32_t)((int64_t)b * p.S + first);
        tc::bar_arrive_expect_tx(&sm.row_full[buf], p.rows_fp8 ? PA_BUF / 2 : PA_BUF);
        if (p.rows_fp8) {                             // the second half of each column chunk
          for (int i = 0; i < 4; i++)
            tc::tma_load_2d(kt + PA_COL / 2 + i * PA_COL, &map_rows, 256 * rank + 64 * i, row, &sm.row_full[buf]);
        } else {
          tc::tma_load_3d(kt, &map_rows, 0, row, 4 * rank, &sm.row_full[buf]);
        }
      }
      // the last arrivals of CTA 0's products, of which the fill warps have not waited for all, before this CTA ends
      for (int i = 0; i < min(n_ch, PA_BUFS); i++) wait(&sm.free_[i], (n_ch - 1 - i) / PA_BUFS, 92);
    }
    __syncwarp();
    told();
  } else if (warp >= PA_SOFT_WARPS) {
    // ================= K buffers
    const int ft = tid - 32 * PA_SOFT_WARPS;
    // codes: lane = key, 64 dims a thread, so that both swizzles spread eight lanes over the banks
    const int key8 = 32 * (ft >> 5 & 1) + lane, part8 = ft >> 6;
    // rows in E4M3: thread = (key, part j: 32 of each 128 dims), as in keys_attention.cu
    const int k8 = (ft >> 2) & 7, j = ft & 3, key = ((ft >> 2) & ~7) + ((k8 & 4) | (k8 & 1) << 1 | (k8 >> 1 & 1));
    const bool odd = (j & 2) != 0;
    uint32_t staged = 0;
    for (int c = 0; c < n_ch; c++) {
      const uint32_t buf = c % PA_BUFS, use = c / PA_BUFS;
      unsigned char* kt = smem + buf * PA_BUF;
      if (use > 0) wait(&sm.free_[buf], use - 1, 85);
      else if (buf >= PA_BUFS - 2 && there) wait(&sm.q_here, 0, 85);
      tc::fence_after_sync();
      if (!run.rows(c)) {
        // (keys behind the last: whatever lies there, finite, with weights of 0)
        const uint32_t s = staged % PA_STAGES;
        wait(&sm.stage_full[s], staged / PA_STAGES, 86);
        staged++;
        const unsigned char* e = smem + PA_OFF_STAGE + s * PA_STAGE + (part8 >> 1) * PA_COL;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
          v[i] = *reinterpret_cast<const uint4*>(e + sw128((uint32_t)key8, 16u * (uint32_t)(4 * (part8 & 1) + i)));
        tc::fence_proxy_async_smem();                 // reads done before a copy writes there again
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sm.stage_free[s]);
        unsigned char* dst = kt + part8 * PA_COL;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          uint32_t o[8];
          i8x16_to_f16(v[i], o);
          *reinterpret_cast<uint4*>(dst + sw128((uint32_t)key8, 32u * i)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + sw128((uint32_t)key8, 32u * i + 16u)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
        const int first = run.first(c), keys = run.keys(c);
        wait(&sm.row_full[buf], use, 87);             // (rows come first: copy `use` of the buffer too)
        // values that are not finite: 0, and the queries that see their row are told
        auto bad = [](uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; };   // exponent of all ones
        auto finite = [&](uint32_t w, int row) -> uint32_t {
          const uint32_t is = bad(w);
          if (is == 0u) return w;
          for (int q = 0; q < 2; q++)
            if (first + row >= qs[q].row_lo && first + row < qs[q].row_hi) {
              if (q == rank) *(volatile int*)&sm.poison = 1;
              else tc::store_other(&sm.poison, 1, q);
            }
          return (is & 0x8000u ? 0u : w & 0xFFFFu) | (is & 0x80000000u ? 0u : w & 0xFFFF0000u);
        };
        if (p.rows_fp8) {
          uint32_t o[2][16];
#pragma unroll
          for (int y = 0; y < 2; y++) {
            const uint4* src = reinterpret_cast<const uint4*>(kt + 2 * y * PA_COL + (j >> 1) * PA_COL + PA_COL / 2 +
                                                              key * 64 + 32 * (j & 1));
            uint4 a = make_uint4(0u, 0u, 0u, 0u), e = a;
            if (key < keys) {
              a = src[odd ? 1 : 0];
              e = src[odd ? 0 : 1];
            }
            const uint32_t v[8] = {odd ? e.x : a.x, odd ? e.y : a.y, odd ? e.z : a.z, odd ? e.w : a.w,
                                   odd ? a.x : e.x, odd ? a.y : e.y, odd ? a.z : e.z, odd ? a.w : e.w};
#pragma unroll
            for (int x = 0; x < 8; x++) {
              o[y][2 * x] = e4m3x2_to_f16x2(v[x]);
              o[y][2 * x + 1] = e4m3x2_to_f16x2(v[x] >> 16);
            }
          }
          uint32_t any = 0u;
#pragma unroll
          for (int x = 0; x < 32; x++) any |= bad(o[x >> 4][x & 15]);
          if (any != 0u) {
#pragma unroll
            for (int x = 0; x < 32; x++) o[x >> 4][x & 15] = finite(o[x >> 4][x & 15], key);
          }
          named_sync(1, PA_FILL);                     // all are read before any is written
#pragma unroll
          for (int y = 0; y < 2; y++) {
            unsigned char* dst = kt + 2 * y * PA_COL + (j >> 1) * PA_COL + key * 128;
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const uint4 v = make_uint4(
                  odd ? o[y][4 * (g ^ 1)] : o[y][4 * g], odd ? o[y][4 * (g ^ 1) + 1] : o[y][4 * g + 1],
                  odd ? o[y][4 * (g ^ 1) + 2] : o[y][4 * g + 2], odd ? o[y][4 * (g ^ 1) + 3] : o[y][4 * g + 3]);
              const uint32_t unit = (uint32_t)(4 * (j & 1) + (odd ? g ^ 1 : g));
              *reinterpret_cast<uint4*>(dst + ((unit ^ (uint32_t)(key & 7)) << 4)) = v;
            }
          }
        } else {
          uint4* u = reinterpret_cast<uint4*>(kt) + ft;
          uint4 x[PA_BUF / 16 / PA_FILL] = {};
#pragma unroll
          for (int i = 0; i < PA_BUF / 16 / PA_FILL; i++) {
            const int row = ((ft + i * PA_FILL) >> 3) & (PA_KEYS - 1);
            if (row < keys) x[i] = u[i * PA_FILL];
          }
#pragma unroll
          for (int i = 0; i < PA_BUF / 16 / PA_FILL; i++) {
            uint4 o = make_uint4(bf16x2_to_f16x2(x[i].x), bf16x2_to_f16x2(x[i].y), bf16x2_to_f16x2(x[i].z),
                                 bf16x2_to_f16x2(x[i].w));
            if ((bad(o.x) | bad(o.y) | bad(o.z) | bad(o.w)) != 0u) {
              const int row = ((ft + i * PA_FILL) >> 3) & (PA_KEYS - 1);
              o = make_uint4(finite(o.x, row), finite(o.y, row), finite(o.z, row), finite(o.w, row));
            }
            u[i * PA_FILL] = o;
          }
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {                                // (for the warp, whose writes come before)
        if (rank) tc::bar_arrive_first_release(&sm.full[buf]);
        else tc::bar_arrive(&sm.full[buf]);
      }
    }
    told();
  } else {
    // ================= softmax: lane of TMEM l = 32 (warp % 4) + lane: head l % 64, half l / 64 (of Q's dims, of the
    // keys); of its 32 keys and its columns of Q and O the warp takes the half `sub`
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    const int half = warp >> 1 & 1, sub = warp >> 2, head = 32 * (warp & 1) + lane, other = tid ^ 64;
    const int two = 3 + (warp & 1) + 2 * sub;         // named barrier of the two warps with a head's lanes for the same keys
    const int four = 7 + (warp & 1);                  // of the four that have a head
    const int own = 2 * half + sub;                   // quarter of the keys
    float4* xs = reinterpret_cast<float4*>(smem + PA_OFF_S);
    uint4* xp = reinterpret_cast<uint4*>(smem + PA_OFF_P);
    float sc2 = p.scale * KA_LOG2E;                   // products to scores in powers of two
    float m_used = -INFINITY, l_sum = 0.f;
    if (there) wait(&sm.q_full, 0, 88);               // (without keys too: no copy may land behind the CTA's end)
    if (n_ch > 0) {                                   // Q: 128 dims of this lane's head to TMEM
      const unsigned char* qh = smem + (PA_BUFS - 2 + half) * PA_BUF;
      __half2 most = __half2half2(__ushort_as_half(0));
#pragma unroll 1
      for (int g = 2 * sub; g < 2 * sub + 2; g++) {
        uint32_t w[32] = {};
        if (there) {
#pragma unroll
          for (int u = 0; u < 8; u++) {
            const uint4 x = *reinterpret_cast<const uint4*>(qh + g * PA_COL + sw128((uint32_t)head, 16u * u));
            w[4 * u] = x.x;
            w[4 * u + 1] = x.y;
            w[4 * u + 2] = x.z;
            w[4 * u + 3] = x.w;
          }
#pragma unroll
          for (int x = 0; x < 32; x++) {
            w[x] = bf16x2_to_f16x2(w[x]);
            most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&w[x])));
          }
        }
        tmem_st32(quarter + PA_Q_COL + 32 * g, w);
      }
      const bool big = __hisinf(__hmax(__low2half(most), __high2half(most))) != 0;
      if (bar_any(four, 128, big)) {
        // heads with a |q| of 2^16 or more, out of f16's range: once more, times a power of two that puts the
        // largest into [2^15, 2^16), and their scale times its inverse.  (An infinity stays one.)
        uint32_t size = 0u;                           // largest |q|, bf16 bits
        if (there) {
#pragma unroll 1
          for (uint32_t x = 0; x < 64; x++) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(qh + (2 * sub + (x >> 5)) * PA_COL +
                                                                  sw128((uint32_t)head, 4u * (x & 31u)));
            size = max(size, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
          }
        }
        sm.top[own][head] = __uint_as_float(size);
        named_sync(four, 128);
#pragma unroll
        for (int i = 0; i < 4; i++) size = max(size, __float_as_uint(sm.top[i][head]));
        named_sync(four, 128);                        // (the maxima of a chunk go there next)
        const int e = max(min((int)(size >> 7), 254) - 142, 0);
        const float down = __int_as_float((127 - e) << 23);
        sc2 = fmaxf(fminf(sc2 * __int_as_float((127 + e) << 23), FLT_MAX), -FLT_MAX);
        tc::tmem_wait_st();
#pragma unroll 1
        for (int g = 2 * sub; g < 2 * sub + 2; g++) {
          uint32_t w[32] = {};
          if (there) {
#pragma unroll
            for (int x = 0; x < 32; x++) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(qh + g * PA_COL + sw128((uint32_t)head, 4u * x));
              w[x] = pack_f16x2(__uint_as_float(v << 16) * down, __uint_as_float(v & 0xFFFF0000u) * down);
            }
          }
          tmem_st32(quarter + PA_Q_COL + 32 * g, w);
        }
      }
      tc::tmem_wait_st();
      tc::fence_proxy_async_smem();                   // the buffers go to copies and stores of others
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::bar_arrive(&sm.q_here);
        arrive_first(&sm.q_moved);
      }
    }
    // the scales of this lane's two blocks of keys of chunk c (rows, and what the query does not see: 1)
    const float* scale_row = p.scales8 + (int64_t)b * (p.cap / BLK);
    const int k_own = 32 * half + 16 * sub;
    auto scales = [&](int c, float* s) {
      const int k0 = c < n_ch && !run.rows(c) ? run.first(c) + k_own : INT32_MAX - 16;
#pragma unroll
      for (int i = 0; i < 2; i++) s[i] = k0 + BLK * i < mine.entries ? __ldcg(scale_row + k0 / BLK + i) : 1.f;
    };
    float s8_next[2];
    scales(0, s8_next);
    for (int c = 0; c < n_ch; c++) {
      float s8[2], by[2], up[2];                      // scales, what turns products into scores, log2 of the scales
#pragma unroll
      for (int i = 0; i < 2; i++) {
        s8[i] = s8_next[i];
        by[i] = fmaxf(fminf(sc2 * s8[i], FLT_MAX), -FLT_MAX);   // finite: a product may be 0
        up[i] = __log2f(fmaxf(s8[i], KA_FLOOR8));     // (of the reference alone: any value near it would do)
      }
      // keys of this lane that the query sees: x_lo .. x_hi - 1 of 16.  (A part's chunk may end before rows that
      // the query sees in the other part)
      const bool rows = run.rows(c);
      const int k0 = run.first(c) + k_own;
      const int x_lo = rows ? mine.row_lo - k0 : 0;
      const int x_hi = min((rows ? mine.row_hi : mine.entries) - k0, run.keys(c) - k_own);
      const uint32_t s_addr = quarter + PA_S_COL + 64 * (c & 1);
      wait(&sm.s_full[c & 1], c >> 1, 89);
      tc::fence_after_sync();
      scales(c + 1, s8_next);
      float v[16];
      {
        // every lane has its half of the dims' part of each score: those of 16 keys go to the other lane
        uint32_t s0[16], s1[16];
        tmem_ld_x16_nowait(s_addr + 32 * (half ^ 1) + 16 * sub, s0);
        tmem_ld_x16_nowait(s_addr + k_own, s1);
        tmem_wait_ld16(s0, s1);
#pragma unroll
        for (int x = 0; x < 4; x++)
          xs[x * 256 + tid] = make_float4(__uint_as_float(s0[4 * x]), __uint_as_float(s0[4 * x + 1]),
                                          __uint_as_float(s0[4 * x + 2]), __uint_as_float(s0[4 * x + 3]));
        named_sync(two, 64);
#pragma unroll
        for (int x = 0; x < 4; x++) {
          const float4 f = xs[x * 256 + other];
          const float got[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int y = 0; y < 4; y++)                 // (not to be fused with the reference's subtraction)
            v[4 * x + y] = __fmul_rn(__uint_as_float(s1[4 * x + y]) + got[y], by[(4 * x + y) / BLK]);
        }
      }
      if (!__all_sync(0xFFFFFFFFu, x_lo <= 0 && x_hi >= 16)) {
#pragma unroll
        for (int x = 0; x < 16; x++) v[x] = x >= x_lo && x < x_hi ? v[x] : -INFINITY;
      }
      float cm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float m8 = v[8 * i];
#pragma unroll
        for (int x = 1; x < 8; x++) m8 = fmaxf(m8, v[8 * i + x]);
        cm = fmaxf(cm, m8 + up[i]);
      }
      // the reference moves when a score of the head lies far above it, or when it has none (rare, but for the
      // first chunk): then the four lanes of every head of these warps look at all maxima
      if (bar_any(four, 128, cm > -INFINITY && !(cm - m_used <= KA_MOST))) {
        sm.top[own][head] = cm;
        named_sync(four, 128);
#pragma unroll
        for (int i = 0; i < 4; i++) cm = fmaxf(cm, sm.top[i][head]);
        const float to = fabsf(cm) < 0x1p26f ? cm - KA_TOP : cm;
        float alpha = 1.f;
        if (m_used == -INFINITY) {
          m_used = to;                                // O holds nothing yet, or only zeros
        } else if (cm - m_used > KA_MOST) {
          alpha = ex2_ftz(m_used - to);
          m_used = to;
          l_sum *= alpha;
        }
        if (__any_sync(0xFFFFFFFFu, alpha != 1.f) && c > 0) {   // after the chunk before is in O
          wait(&sm.free_[(c - 1) % PA_BUFS], (c - 1) / PA_BUFS, 90);
          tc::fence_after_sync();
#pragma unroll 1
          for (int g = 128 * sub; g < 128 * sub + 128; g += 32) {
            uint32_t o[32];
            tmem_ld32(quarter + PA_O_COL + g, o);
#pragma unroll
            for (int x = 0; x < 32; x++) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            tmem_st32(quarter + PA_O_COL + g, o);
          }
        }
      }
      const float ref = m_used == -INFINITY ? 0.f : m_used;
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[8];
#pragma unroll
      for (int x = 0; x < 8; x++) {
        const float e0 = ex2_ftz(v[2 * x] - ref), e1 = ex2_ftz(v[2 * x + 1] - ref);
        l4[x & 3] += e0 + e1;
        pk[x] = pack_f16x2(e0 * s8[2 * x / BLK], e1 * s8[2 * x / BLK]);
      }
      l_sum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      xp[tid] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      xp[256 + tid] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      // P of the 16 keys in this lane and in the other, over S: columns of the keys' pairs.  (A column of S is
      // read by one of the two warps of a quarter and written by either: all four have read theirs)
      tmem_st8(s_addr + 8 * own, pk);
      named_sync(two, 64);
      {
        const uint4 a = xp[other], d = xp[256 + other];
        const uint32_t got[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
        tmem_st8(s_addr + 8 * (own ^ 2), got);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_first(&sm.p_ready[c & 1]);
    }
    sm.sum[own][head] = l_sum;
    if (own == 0) sm.ref[head] = m_used;              // (all lanes of a head have the same)

    // ================= output: 128 of a lane's 256 dims a warp
    if (p.W > 0) {
      __syncwarp();
      tc::cluster_arrive_relaxed();                   // (what these warps have written is not the other CTA's)
    }
    if (n_ch > 0) {
      const int last = n_ch - 1;
      if (*(volatile int*)&sm.err == 0) wait(&sm.free_[last % PA_BUFS], last / PA_BUFS, 91);
      tc::fence_after_sync();
    }
    if (p.W > 0) {
      __syncwarp();
      tc::cluster_wait();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    named_sync(2, 32 * PA_SOFT_WARPS);                // the sums
    const int head0 = 32 * (warp & 1), g0 = 128 * sub;
    const uint32_t o_addr = quarter + PA_O_COL + g0;
    float l = (sm.sum[0][head] + sm.sum[1][head]) + (sm.sum[2][head] + sm.sum[3][head]);
    if (*(volatile int*)&sm.poison != 0) l = __int_as_float(0x7FC00000);
    if (there && own == 0) {
      const float m = sm.ref[head];
      if (split > 1) {
        part[head] = m;
        part[H + head] = l;
      } else if (p.lse) {                             // l = 0: no visible key
        p.lse[bq * H + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * KA_LN2;
      }
    }
    if (!there) {
    } else if (split == 1) {
      const float inv = 1.0f / l;
      const bool none = l == 0.f;                     // no visible key: zeros
      unsigned char* rows8 = smem + warp * 8192;      // over the K buffers, whose last reader is done
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (n_ch > 0) tmem_ld32(o_addr + c, o);
#pragma unroll
        for (int x = 0; x < 4; x++) {
          float f[8];
#pragma unroll
          for (int y = 0; y < 8; y++) f[y] = none ? 0.f : __uint_as_float(o[8 * x + y]) * inv;
          *reinterpret_cast<uint4*>(rows8 + lane * 256 + ((((c >> 3) + x) ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
      }
      __syncwarp();
      uint4* out = reinterpret_cast<uint4*>(p.out + (bq * H + head0) * D) + (D / 16) * half + g0 / 8;
#pragma unroll 4
      for (int x = 0; x < 16; x++) {                  // two rows of 256 bytes an instruction
        const int row = 2 * x + (lane >> 4), u = lane & 15;
        out[row * (D / 8) + u] = *reinterpret_cast<const uint4*>(rows8 + row * 256 + ((u ^ (row & 7)) << 4));
      }
    } else if (n_ch > 0) {
      // a partial state: O as [dims / 4][head][4]
      float4* out = reinterpret_cast<float4*>(part + 2 * H) + ((D / 8) * half + g0 / 4) * H + head;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_addr + c, o);
#pragma unroll
        for (int x = 0; x < 8; x++)
          out[(c / 4 + x) * H] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                             __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  // after a timeout copies may be in flight that nobody waited for: time for them to land
  if (*(volatile int*)&sm.err != 0)
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  __syncwarp();
  tc::cluster_arrive_relaxed();                       // (each CTA has waited for all that the other sends it)
  tc::cluster_wait();
  if (warp == PA_MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(0u, 512);
  }
}

// mr8: map of E4M3 rows (boxes of 64 bytes, widened where they lie)
cudaError_t launch_pair_attention(const KeysParams& p, int B, const CUtensorMap& mr8, cudaStream_t stream) {
  CUtensorMap mq, mr = mr8, mc;
  const uint64_t rows = (uint64_t)((int64_t)B * p.S), entries = (uint64_t)(B * p.cap);
  if (!encode_bf16_rows512_halves(&mq, p.q, (uint64_t)((int64_t)B * p.Q * H), H)) return cudaErrorInvalidValue;
  if (!p.rows_fp8 && rows > 0 && !encode_bf16_rows512_halves(&mr, p.rows, rows, PA_KEYS)) return cudaErrorInvalidValue;
  if (entries > 0 && !encode_u8_rows512_halves(&mc, reinterpret_cast<const uint8_t*>(p.main_kv), entries, PA_KEYS))
    return cudaErrorInvalidValue;
  if (entries == 0) mc = mq;                          // (never read)
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure([](int) {
    return cudaFuncSetAttribute(pair_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PA_SMEM);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)B * ((p.Q + 1) / 2) * p.split * 2));
  cfg.blockDim = dim3(PA_THREADS);
  cfg.dynamicSmemBytes = PA_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pair_attn_kernel, p, mq, mr, mc);
}

}  // namespace csa2
