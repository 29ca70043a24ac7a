// The attention weight that every cache entry gathers from a call's queries:
//
//   w_j = decay prev_j + sum over queries and heads that see j of exp(scale q_h . k_j - lse_h)
//
// on the 5th-generation tensor cores: S^T = K Q^T with 128 entries as the rows of an
// M = 128 tile, so that a thread has all heads of one entry in its TMEM lane and the sum
// over heads and queries stays in its registers: no exchange between lanes, no
// atomics, the same result every time.
//
// Sums: the 64 weights of a query in binary32, in eight runs; compensated over a CTA's queries, and again over the
// CTAs that share them.
//
// A CTA takes a run of tiles of one sequence.  The tile's entries lie in TMEM as the A operand
// (256 columns of 16-bit pairs): with A in shared memory a product of N = 64 would take 48
// cycles instead of 32, and the widened tile 128 KB.  Two S accumulators.
// One query (N = 64): a CTA rounds it to f16 (a head that reaches 2^16 scaled into f16's range
// by a power of two) and keeps it in shared memory; the entries are exact in f16, the cheapest to
// widen to.  More: two CTAs make a pair (cta_group::2) that takes 256 entries, a half each, and a run
// of groups of two queries (N = 128); each CTA loads one query of a group through a ring of stages,
// and the pair's products read both.  Operands are bf16, in which q is as it came and entries are exact
// too (at most 8 significant bits).  With single CTAs of two queries every SM took 128 KB of queries
// from L2 for 2048 cycles of products and waited for them: 4180 cycles a group.
// An 8-bit entry's scale is a factor of the thread that has it.
//
// Warps 0..7: exponentials and sums (warps 4..7: the second query, or the second half of the heads);
// 8..15: entries to TMEM, a half of the dims each four; 16: MMAs; 17: every second tile's MMAs (one
// query: a warp issues one in about 40 cycles), or the lse of a group's heads; 18: copies of entries;
// 19: copies of queries.  All waits are bounded; a timeout reports CSA2_ERR_TIMEOUT.
#include <cfloat>

#include "attn_common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int AW_KEYS = 128;                              // entries of a tile
constexpr int AW_SUM_WARPS = 8, AW_FILL_WARPS = 8;
constexpr int AW_MMA_WARP = AW_SUM_WARPS + AW_FILL_WARPS, AW_MMA2_WARP = AW_MMA_WARP + 1;
constexpr int AW_KEY_WARP = AW_MMA2_WARP + 1, AW_Q_WARP = AW_KEY_WARP + 1;
constexpr int AW_THREADS = 32 * (AW_Q_WARP + 1);
constexpr int AW_PIECES = 8;                              // of 64 dims of a query
constexpr int AW_STAGE = 64 * 128;                        // [64 heads][64 dims] f16, SW128
constexpr int AW_GROUPS = 512;                            // query groups of a CTA at most
constexpr float AW_LOG2E = 1.4426950408889634f;
constexpr int AW_SMS = 152;

// PAIR: two CTAs, two queries a group; else one of each.  A buffers hold half of the dims of a tile.
template <bool E8, bool PAIR>
struct Aw {
  static constexpr int NQ = PAIR ? 2 : 1, N = 64 * NQ;
  static constexpr int STEP = NQ * AW_KEYS;               // entries of a step
  static constexpr int ENTRY = E8 ? D : MAIN_BYTES;
  static constexpr int TILE = AW_KEYS * ENTRY;            // bytes of a tile as stored
  static constexpr int TILES = PAIR ? 1 : E8 ? 2 : 4;     // staged tiles
  static constexpr int A_BUFS = PAIR ? 2 : 3;             // of 128 columns
  static constexpr int S_COL = 128 * A_BUFS;
  static constexpr int RING = PAIR ? 2 : 1;               // groups of query stages
  static constexpr int COLS = PAIR ? 4 : 1;               // groups' factors
  static constexpr int OFF_TILE = RING * AW_PIECES * AW_STAGE;
  static constexpr int OFF_SMALL = OFF_TILE + TILES * TILE;
  struct Small {
    // A head's factor and minus its lse in powers of two; of a pair, groups in turn, minus the lse and a mask of
    // its weights' bits (none for a head that saw nothing: its q may be NaN)
    float2 col[COLS][N];
    float joined[2][AW_KEYS];         // the second half's sums
    int vis[AW_GROUPS * NQ];          // entries each query sees
    uint64_t tile_full[TILES], tile_free[TILES];    // TMA; a fill warp each
    // Of a pair CTA 0's a_full, q_full and s_free count, for both; what MMAs complete is told to both.
    uint64_t a_full[A_BUFS], a_free[A_BUFS];        // four fill warps of a CTA; MMAs
    uint64_t q_full[RING][2], q_free[RING][2];      // half of a group's dims: TMA (one query: the sum warps); MMAs
    uint64_t s_full[2], s_free[2];                  // MMAs; sum warps
    uint64_t col_full[COLS], col_free[COLS];        // warp 17; sum warps
    uint32_t tmem_base;
    int most, err;
  };
  static constexpr int SMEM = OFF_SMALL + (int)sizeof(Small);
  static_assert(SMEM <= 227 * 1024 && S_COL + 2 * N <= 512 && TILE % 1024 == 0, "");
};

__device__ __noinline__ bool aw_timeout(int* err, WsHeader* hdr, int where) {
  if (atomicExch(err, 1) == 0) report(hdr, CSA2_ERR_TIMEOUT, where);
  return false;
}

// x, the same in every lane, in a uniform register.
__device__ __forceinline__ uint32_t aw_uniform(uint32_t x) { return __reduce_or_sync(0xFFFFFFFFu, x); }

// x's bits that the mask has
__device__ __forceinline__ float aw_masked(float x, float mask) {
  return __uint_as_float(__float_as_uint(x) & __float_as_uint(mask));
}

// acc += x, with what its rounding loses kept for the next sum.
__device__ __forceinline__ void aw_add(float& acc, float& lost, float x) {
  const float y = x - lost, z = acc + y;
  lost = fabsf(z) < INFINITY ? (z - acc) - y : 0.f;
  acc = z;
}

// entries of sequence b that the call deals with
__device__ __forceinline__ int aw_entries(const AwParams& p, int b) {
  return (int)max((int64_t)0, min((int64_t)p.n_entries[b], min(p.cap, p.max_n)));
}

// One head by a warp: q as f16 into its row of the stages, its factor and its lse in powers of two.
__device__ __forceinline__ float2 aw_head(const uint16_t* q, float lse, float scale, bool live, unsigned char* stages,
                                          int row, int lane) {
  uint4 v[2] = {};
  live = live && lse != -INFINITY;                    // else weights of 0, whatever q holds
  if (live) {
    v[0] = __ldcg(reinterpret_cast<const uint4*>(q) + lane);
    v[1] = __ldcg(reinterpret_cast<const uint4*>(q) + 32 + lane);
  }
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t most = 0u;
#pragma unroll
  for (int i = 0; i < 8; i++) most = __vmaxu2(most, w[i] & 0x7FFF7FFFu);
  most = __reduce_max_sync(0xFFFFFFFFu, max(most & 0xFFFFu, most >> 16));
  // |q| of 2^16 or more (bf16 bits 143 << 7): the largest goes to [2^15, 2^16)
  const int e = max(min((int)(most >> 7), 254) - 142, 0);
  const float down = __int_as_float((127 - e) << 23);
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; i++)
    o[i] = pack_f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xFFFF0000u) * down);
  // dims 8 lane .. and 256 + 8 lane ..
  unsigned char* dst = stages + (lane >> 3) * AW_STAGE + sw128((uint32_t)row, 16u * (lane & 7));
  *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(dst + 4 * AW_STAGE) = make_uint4(o[4], o[5], o[6], o[7]);
  if (!live) return make_float2(0.f, -INFINITY);
  const float by = scale * AW_LOG2E * __int_as_float((127 + e) << 23);
  return make_float2(fmaxf(fminf(by, FLT_MAX), -FLT_MAX), -lse * AW_LOG2E);   // finite: a product may be 0
}

// two f16 -> two bf16, exact for an entry's values
__device__ __forceinline__ uint32_t aw_f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x, f.y);
}

template <bool E8, bool PAIR>
__global__ void __launch_bounds__(AW_THREADS, 1)
attn_weights_kernel(AwParams p, const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_codes) {
  using C = Aw<E8, PAIR>;
  using Small = typename C::Small;
  constexpr int NQ = C::NQ;
  extern __shared__ __align__(1024) unsigned char smem[];
  Small& sm = *reinterpret_cast<Small*>(smem + C::OFF_SMALL);
  WsHeader* hdr = p.hdr;
  // the swizzled tiles need the declared alignment (the same in both CTAs)
  if (tc::smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) report(hdr, CSA2_ERR_CUDA, 3);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int rank = PAIR ? (int)tc::cluster_rank() : 0;
  // block = (query split, sequence, run of steps, CTA of the pair)
  const uint32_t item = blockIdx.x / (uint32_t)NQ;
  const int run = (int)(item % (uint32_t)p.runs), sb = (int)(item / (uint32_t)p.runs);
  const int b = sb % p.B, qs = sb / p.B;

  if (warp == AW_MMA_WARP) {
    if (PAIR) tc::tmem_alloc_pair(&sm.tmem_base, 512);
    else tc::tmem_alloc(&sm.tmem_base, 512);
  }
  if (tid == 0) {
    for (int i = 0; i < C::TILES; i++) {
      tc::bar_init(&sm.tile_full[i], 1);
      tc::bar_init(&sm.tile_free[i], AW_FILL_WARPS);
    }
    for (int i = 0; i < C::A_BUFS; i++) {
      tc::bar_init(&sm.a_full[i], NQ * AW_FILL_WARPS / 2);
      tc::bar_init(&sm.a_free[i], 1);
    }
    for (int i = 0; i < C::RING; i++)
      for (int k = 0; k < 2; k++) {
        tc::bar_init(&sm.q_full[i][k], PAIR ? 1 : AW_SUM_WARPS);
        tc::bar_init(&sm.q_free[i][k], 1);
      }
    for (int i = 0; i < 2; i++) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.s_free[i], NQ * AW_SUM_WARPS);
    }
    for (int i = 0; i < C::COLS; i++) {
      tc::bar_init(&sm.col_full[i], 1);
      tc::bar_init(&sm.col_free[i], AW_SUM_WARPS);
    }
    sm.most = 0;
    sm.err = 0;
    tc::bar_init_fence();
    if (PAIR) tc::prefetch_tensormap(&map_q);
    if (E8) tc::prefetch_tensormap(&map_codes);
  }
  tc::fence_before_sync();
  if (PAIR) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after_sync();
  if (sm.tmem_base != 0 && tid == 0) report(hdr, CSA2_ERR_CUDA, 4);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int n = aw_entries(p, b);
  if (item == (uint32_t)(b * p.runs) && rank == 0 && tid == 0 && p.n_entries[b] > min(p.cap, p.max_n))
    report(hdr, CSA2_ERR_BOUNDS, p.n_entries[b]);
  const int steps = (n + C::STEP - 1) / C::STEP;
  const int t_lo = (int)((int64_t)steps * run / p.runs), t_n = (int)((int64_t)steps * (run + 1) / p.runs) - t_lo;
  const int groups = (p.Q + NQ - 1) / NQ;
  const int g_lo = (int)((int64_t)groups * qs / p.splits), ng = (int)((int64_t)groups * (qs + 1) / p.splits) - g_lo;
  // what the run's queries see (AW_GROUPS groups at most); those behind the last query: nothing
  int most = 0;
  for (int i = tid; i < ng * NQ; i += AW_THREADS) {
    const int qi = g_lo * NQ + i;
    int v = 0;
    if (qi < p.Q) {
      const int64_t t = p.q_pos[(int64_t)b * p.Q + qi];
      if (t >= 0) v = (int)min((min(t, INT64_MAX - 1) + 1) >> (p.m - 1), (int64_t)n);   // (m is 1 or 2)
    }
    sm.vis[i] = v;
    most = max(most, v);
  }
  if (most > 0) atomicMax(&sm.most, most);
  __syncthreads();
  // the steps that some query sees come first
  const int live = min(max((sm.most + C::STEP - 1) / C::STEP - t_lo, 0), t_n);
  const bool resident = ng == 1;                      // the one group's dims stay in their stages
  auto next_group = [&](int g, int step) {            // the first group from g on that sees the step
    while (g < ng && max(sm.vis[NQ * g], sm.vis[NQ * g + NQ - 1]) <= step * C::STEP) g++;
    return g;
  };
  bool ok = true;                                     // a thread that has given up once waits no more
  auto wait = [&](uint64_t* bar, uint32_t use, int where) {
    if (ok) ok = tc::bar_wait(bar, use & 1u) || aw_timeout(&sm.err, hdr, where);
  };
  auto arrive_first = [&](uint64_t* bar) {            // on CTA 0's barrier
    if (PAIR && rank != 0) tc::bar_arrive_first(bar);
    else tc::bar_arrive(bar);
  };

  if (warp == AW_MMA_WARP || (!PAIR && warp == AW_MMA2_WARP)) {
    // ================= MMAs (the whole warp runs the loop, one lane issues; of a pair, in CTA 0)
    // An MMA takes its addresses from uniform registers: what the loops follow from goes through a
    // reduction over the warp, whose result is uniform (else an MMA takes 82 cycles to issue).
    constexpr uint32_t idesc =
        PAIR ? tc::idesc_bf16(NQ * AW_KEYS, C::N, 0, 0) : tc::idesc_f16(NQ * AW_KEYS, C::N, 0, 0);
    const uint64_t q_d = tc::smem_desc(tc::smem_u32(smem), 16, 1024, tc::SW_128B);
    const uint32_t leader = tc::elect_one();
    const int n_live = rank == 0 ? (int)aw_uniform((uint32_t)live) : 0, n_g = (int)aw_uniform((uint32_t)ng);
    auto wait_mma = [&](uint64_t* bar, uint32_t use, int where) {
      if (ok) ok = tc::bar_wait_relaxed(bar, use & 1u) || aw_timeout(&sm.err, hdr, where);
    };
    auto commit = [&](uint64_t* bar) {
      if (PAIR) tc::commit_pair(leader, bar);
      else tc::commit_warp(leader, bar);
    };
    // S number i += the half h of the dims, A buffer k times the queries of ring place `ring`
    auto products = [&](uint32_t i, int h, uint32_t k, uint32_t ring) {
      tc::fence_after_sync();
      const uint64_t qa = q_d + (uint32_t)((ring * AW_PIECES + 4 * h) * AW_STAGE >> 4);
      const uint32_t s = C::S_COL + C::N * i, a = 128 * k;
#pragma unroll
      for (int x = 0; x < 16; x++) {
        const uint64_t qx = qa + (uint32_t)(((x >> 2) * AW_STAGE + 32 * (x & 3)) >> 4);
        if (PAIR) tc::mma_f16_ts_pair(leader, s, a + 8 * x, qx, idesc, (h || x) ? 1u : 0u);
        else tc::mma_f16_ts_warp(leader, s, a + 8 * x, qx, idesc, (h || x) ? 1u : 0u);
      }
    };
    if (!PAIR) {
      // tiles in turn with the other warp
      const uint32_t mine = warp == AW_MMA2_WARP ? 1u : 0u;
      if (n_live > (int)mine)
        for (int h = 0; h < 2; h++) wait_mma(&sm.q_full[0][h], 0, 62);
      uint32_t ab = 2 * mine, ab_use = 0;             // A buffer and its use: 2 t % 3, 2 t / 3
      for (uint32_t t = mine; t < (uint32_t)n_live; t += 2) {
        if (t >= 2) wait_mma(&sm.s_free[mine], (t >> 1) - 1, 60);
#pragma unroll 1
        for (int h = 0; h < 2; h++) {
          wait_mma(&sm.a_full[ab], ab_use, 61);
          products(mine, h, ab, 0);
          commit(&sm.a_free[ab]);
          if (++ab == C::A_BUFS) ab = 0, ab_use++;
        }
        commit(&sm.s_full[mine]);
        ab += 2;                                      // the other warp's two
        if (ab >= C::A_BUFS) ab -= C::A_BUFS, ab_use++;
      }
    } else {
      uint32_t u = 0;                                 // group of the CTA
      for (int t = 0; t < n_live; t++) {              // A buffer = half of the dims
        int g = (int)aw_uniform((uint32_t)next_group(0, t_lo + t));
        bool first = true;
        while (g < n_g) {
          const int after = (int)aw_uniform((uint32_t)next_group(g + 1, t_lo + t));
          if (u >= 2) wait_mma(&sm.s_free[u & 1], (u >> 1) - 1, 60);
          const uint32_t ring = n_g > 1 ? u % C::RING : 0;   // (one group stays where it is)
#pragma unroll 1
          for (int h = 0; h < 2; h++) {
            if (first) wait_mma(&sm.a_full[h], t, 61);
            if (n_g > 1 || u == 0) wait_mma(&sm.q_full[ring][h], u / C::RING, 62);
            products(u & 1, h, h, ring);
            if (n_g > 1) commit(&sm.q_free[ring][h]);
            if (after >= n_g) commit(&sm.a_free[h]);
          }
          commit(&sm.s_full[u & 1]);
          u++;
          g = after;
          first = false;
        }
      }
      // CTA 1's last arrivals, before this CTA ends
      for (uint32_t x = u < 2 ? 0 : u - 2; x < u; x++) wait_mma(&sm.s_free[x & 1], x >> 1, 60);
    }
  } else if (PAIR && warp == AW_MMA2_WARP) {
    // ================= the lse of a group's heads
    uint32_t u = 0;
    for (int t = 0; t < (resident ? min(live, 1) : live); t++) {
      for (int g = next_group(0, t_lo + t); g < ng; g = next_group(g + 1, t_lo + t)) {
        float l[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {                 // (none behind the sequence's last query)
          const int64_t q = (int64_t)(g_lo + g) * NQ + (i >> 1);
          l[i] = q < p.Q ? __ldcg(p.lse + ((int64_t)b * p.Q + q) * H + 32 * (i & 1) + lane) : -INFINITY;
        }
        const uint32_t ci = u % C::COLS;
        if (u >= C::COLS) wait(&sm.col_free[ci], u / C::COLS - 1, 64);
#pragma unroll
        for (int i = 0; i < 4; i++)
          sm.col[ci][32 * i + lane] = make_float2(-l[i] * AW_LOG2E, __uint_as_float(l[i] == -INFINITY ? 0u : ~0u));
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sm.col_full[ci]);
        u++;
      }
    }
  } else if (warp == AW_KEY_WARP) {
    // ================= copies of entries
    if (lane == 0) {
      for (int t = 0; t < live; t++) {
        const uint32_t ts = t % C::TILES, use = t / C::TILES;
        const int64_t first = (int64_t)(t_lo + t) * C::STEP + AW_KEYS * rank;
        unsigned char* dst = smem + C::OFF_TILE + ts * C::TILE;
        if (use > 0) wait(&sm.tile_free[ts], use - 1, 63);
        if (E8) {                                     // four column chunks of 128 dims, SW128
          tc::bar_arrive_expect_tx(&sm.tile_full[ts], C::TILE);
          for (int i = 0; i < D / 128; i++)
            tc::tma_load_2d(dst + i * (AW_KEYS * 128), &map_codes, i * 128, (int32_t)(b * p.cap + first),
                            &sm.tile_full[ts]);
        } else {                                      // (none: the pair's second half may lie behind the cache)
          const uint32_t bytes = (uint32_t)max(min((int64_t)AW_KEYS, p.cap - first), (int64_t)0) * MAIN_BYTES;
          tc::bar_arrive_expect_tx(&sm.tile_full[ts], bytes);
          if (bytes > 0) tc::bulk_load(dst, p.kv + (b * p.cap + first) * MAIN_BYTES, bytes, &sm.tile_full[ts]);
        }
      }
    }
    __syncwarp();
  } else if (warp == AW_Q_WARP) {
    // ================= copies of queries: each CTA of a pair takes one query of a group
    if (PAIR && lane == 0) {
      uint32_t u = 0;
      for (int t = 0; t < (resident ? min(live, 1) : live); t++) {
        for (int g = next_group(0, t_lo + t); g < ng; g = next_group(g + 1, t_lo + t)) {
          const int64_t row = ((int64_t)b * p.Q + (int64_t)(g_lo + g) * NQ) * H;
          const uint32_t ring = u % C::RING;
          for (int h = 0; h < 2; h++) {
            unsigned char* dst = smem + (ring * AW_PIECES + 4 * h) * AW_STAGE;
            uint64_t* bar = &sm.q_full[ring][h];
            if (u >= C::RING) wait(&sm.q_free[ring][h], u / C::RING - 1, 65);
            if (rank == 0) tc::bar_arrive_expect_tx(bar, NQ * 4 * AW_STAGE);
            tc::tma_load_3d_pair(dst, &map_q, 0, (int32_t)row + H * rank, 4 * h, bar);
          }
          u++;
        }
      }
      // the last arrivals of CTA 0's products, before this CTA ends
      if (!resident)
        for (uint32_t x = u < C::RING ? 0 : u - C::RING; x < u; x++)
          for (int h = 0; h < 2; h++) wait(&sm.q_free[x % C::RING][h], x / C::RING, 65);
      for (int h = 0; h < 2 && live > 0; h++) wait(&sm.a_free[h], live - 1, 67);
    }
    __syncwarp();
  } else if (warp >= AW_SUM_WARPS) {
    // ================= entries to TMEM: lane = entry, four warps a half of the dims
    const int h = (warp - AW_SUM_WARPS) >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    for (int t = 0; t < live; t++) {
      const uint32_t k = 2 * t + h, ab = k % C::A_BUFS, use = k / C::A_BUFS, ts = t % C::TILES;
      const unsigned char* tile = smem + C::OFF_TILE + ts * C::TILE;
      wait(&sm.tile_full[ts], t / C::TILES, 66);
      if (use > 0) wait(&sm.a_free[ab], use - 1, 67);
      tc::fence_after_sync();
      uint4 sc = make_uint4(0u, 0u, 0u, 0u);
      if (!E8) sc = *reinterpret_cast<const uint4*>(tile + row * MAIN_BYTES + 256 + 16 * h);
      const uint32_t scw[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
      for (int i = 0; i < 4; i++) {                   // 64 dims: 32 columns
        uint32_t o[32];
        if (E8) {
#pragma unroll
          for (int x = 0; x < 4; x++) {
            const uint4 c = *reinterpret_cast<const uint4*>(tile + (2 * h + (i >> 1)) * (AW_KEYS * 128) +
                                                            sw128((uint32_t)row, 16u * (4 * (i & 1) + x)));
            if (PAIR) i8x16_to_bf16(c, o + 8 * x);
            else i8x16_to_f16(c, o + 8 * x);
          }
        } else {
          // rows are 18 units of 16 bytes: of the eight lanes of a phase four take their two units in the
          // other order, so that they lie in eight bank groups
          const uint4* src = reinterpret_cast<const uint4*>(tile + row * MAIN_BYTES + 128 * h + 32 * i);
          const int turn = lane >> 2 & 1;
          const uint4 a = src[turn], c = src[turn ^ 1];
          const uint32_t w[8] = {turn ? c.x : a.x, turn ? c.y : a.y, turn ? c.z : a.z, turn ? c.w : a.w,
                                 turn ? a.x : c.x, turn ? a.y : c.y, turn ? a.z : c.z, turn ? a.w : c.w};
#pragma unroll
          for (int x = 0; x < 8; x++) {
            e2m1x8_to_f16(w[x], o + 4 * x);
            const uint32_t s2 = e4m3x2_to_f16x2(prmt(scw[i], 0u, 0x1111u * (x >> 1)));
#pragma unroll
            for (int y = 0; y < 4; y++) {
              o[4 * x + y] = hmul2(o[4 * x + y], s2);
              if (PAIR) o[4 * x + y] = aw_f16x2_to_bf16x2(o[4 * x + y]);
            }
          }
        }
        tmem_st32(quarter + 128 * ab + 32 * i, o);
      }
      tc::fence_proxy_async_smem();                   // reads done before a copy writes there again
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::bar_arrive(&sm.tile_free[ts]);
        arrive_first(&sm.a_full[ab]);
      }
    }
  } else {
    // ================= weights: lane = entry, warps 4..7 the second half of the columns
    const int half = warp >> 2, row = 32 * (warp & 3) + lane;
    constexpr int COLS = C::N / 2;
    const uint32_t addr = ((uint32_t)(32 * (warp & 3)) << 16) + C::S_COL + COLS * half;
    if (!PAIR && live > 0) {                          // the query: eight heads a warp
      for (int i = 0; i < H / AW_SUM_WARPS; i++) {
        const int head = (H / AW_SUM_WARPS) * warp + i;
        const float2 c = aw_head(p.q + ((int64_t)b * H + head) * D, __ldcg(p.lse + (int64_t)b * H + head), p.scale,
                                 sm.vis[0] > 0, smem, head, lane);
        if (lane == 0) sm.col[0][head] = c;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int h = 0; h < 2; h++) tc::bar_arrive(&sm.q_full[0][h]);
      named_sync(1, 32 * AW_SUM_WARPS);               // the factors
    }
    const float by0 = p.scale * AW_LOG2E;
    uint32_t u = 0;
    for (int t = 0; t < t_n; t++) {
      const int j = (t_lo + t) * C::STEP + AW_KEYS * rank + row;
      float acc = 0.f, lost = 0.f;                    // compensated over the queries
      float had = 0.f;                                // loaded ahead of the products it waits for
      if (half == 0 && p.splits == 1 && p.prev && j < n) had = __ldcg(p.prev + (int64_t)b * p.cap + j);
      if (t < live) {
        float s8 = 1.f;
        if (E8) s8 = j < n ? __ldcg(p.scales8 + (int64_t)b * (p.cap / BLK) + j / BLK) : 0.f;
        const float by = by0 * s8;                    // (of a pair: one query's heads have their own)
        for (int g = next_group(0, t_lo + t); g < ng; g = next_group(g + 1, t_lo + t)) {
          const uint32_t i = u & 1;
          const uint32_t ci = resident ? 0 : u % C::COLS;
          const float4* col = reinterpret_cast<const float4*>(sm.col[ci] + COLS * half);
          if (PAIR && (!resident || u == 0)) wait(&sm.col_full[ci], u / C::COLS, 68);
          wait(&sm.s_full[i], u >> 1, 69);
          tc::fence_after_sync();
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < COLS; c += 32) {
            uint32_t r[32];
            tmem_ld32(addr + C::N * i + c, r);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float4 f = col[(c + x) / 2];
              const float v0 = __uint_as_float(r[x]), v1 = __uint_as_float(r[x + 1]);
              if (PAIR) {
                s4[x & 2] += aw_masked(ex2_ftz(fmaf(v0, by, f.x)), f.y);
                s4[(x & 2) + 1] += aw_masked(ex2_ftz(fmaf(v1, by, f.z)), f.w);
              } else {
                s4[x & 2] += ex2_ftz(fmaf(E8 ? v0 * s8 : v0, f.x, f.y));
                s4[(x & 2) + 1] += ex2_ftz(fmaf(E8 ? v1 * s8 : v1, f.z, f.w));
              }
            }
          }
          tc::fence_before_sync();
          tc::fence_proxy_async_smem();               // reads of the factors done before a copy writes there again
          __syncwarp();
          if (lane == 0) {
            arrive_first(&sm.s_free[i]);
            tc::bar_arrive(&sm.col_free[ci]);
          }
          if (j < sm.vis[NQ == 1 ? g : 2 * g + half]) {
            aw_add(acc, lost, (s4[0] + s4[1]) + (s4[2] + s4[3]));
          }
          u++;
        }
      }
      if (half == 1) sm.joined[t & 1][row] = acc;
      named_sync(1, 32 * AW_SUM_WARPS);
      if (half == 0 && j < n) {
        acc += sm.joined[t & 1][row];
        if (p.splits > 1) {
          p.part[((int64_t)qs * p.B + b) * p.pitch + j] = acc;
        } else {
          p.out[(int64_t)b * p.cap + j] = p.prev ? fmaf(p.decay, had, acc) : acc;
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  // after a timeout copies may be in flight that nobody waited for: time for them to land
  if (*(volatile int*)&sm.err != 0)
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  // (each CTA has waited for all that the other sends it)
  if (PAIR) {
    __syncwarp();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
  }
  if (warp == AW_MMA_WARP) {
    tc::fence_after_sync();
    if (PAIR) tc::tmem_dealloc_pair(0u, 512);
    else tc::tmem_dealloc(0u, 512);
  }
}

// The query splits' sums of an entry, in order, and what it had.  (No splits: the call launches nothing else, and
// this kernel reports.)
__global__ void __launch_bounds__(256) attn_weights_join_kernel(AwParams p, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = (int)(blockIdx.x / (uint32_t)blocks), n = aw_entries(p, b);
  const int64_t j = (int64_t)(blockIdx.x % (uint32_t)blocks) * 256 + threadIdx.x;
  if (p.splits == 0 && j == 0 && p.n_entries[b] > min(p.cap, p.max_n)) report(p.hdr, CSA2_ERR_BOUNDS, p.n_entries[b]);
  if (j >= n) return;
  float acc = 0.f, lost = 0.f;                        // compensated: there may be 16,384 splits
  for (int s = 0; s < p.splits; s++) aw_add(acc, lost, __ldcg(p.part + ((int64_t)s * p.B + b) * p.pitch + j));
  const int64_t at = (int64_t)b * p.cap + j;
  p.out[at] = p.prev ? fmaf(p.decay, p.prev[at], acc) : acc;
}

// ------------------------------------------------------------------ host side
// Runs of steps of a sequence and splits of its queries: the least time on 152 SMs with one CTA each.  In
// tenths of a us: a CTA costs 50, a step 8 with one query, else 10 and 11 a group; the join of splits 30.
AwPlan attn_weights_plan(int B, int Q, int64_t max_n) {
  AwPlan best{1, 1};
  const int ctas = Q == 1 ? AW_SMS : AW_SMS / 2;      // or pairs
  const int64_t steps = ceil_div(max_n, Q == 1 ? AW_KEYS : 2 * AW_KEYS), groups = Q == 1 ? 1 : ceil_div(Q, 2);
  if (B <= 0 || Q <= 0 || steps == 0) return best;
  int64_t best_cost = INT64_MAX;
  const int64_t least = ceil_div(groups, AW_GROUPS);
  for (int64_t s = least; s <= groups && s < least + 32; s++) {
    for (int waves = 1; waves <= 4; waves++) {
      int64_t runs = (int64_t)ctas * waves / (B * s);
      runs = runs < 1 ? 1 : runs > steps ? steps : runs;
      const int64_t per = ceil_div(steps, runs) * (Q == 1 ? 8 : 10 + 11 * ceil_div(groups, s));
      const int64_t cost = ceil_div(B * s * runs, ctas) * (50 + per) + (s > 1 ? 30 : 0);
      if (cost < best_cost) {
        best_cost = cost;
        best = {(int)runs, (int)s};
      }
    }
  }
  return best;
}

// floats of a sequence's partial sums
int64_t attn_weights_pitch(int64_t max_n) { return ceil_div(max_n, AW_KEYS) * AW_KEYS; }

template <bool E8, bool PAIR>
static cudaError_t aw_launch(const AwParams& p, const CUtensorMap& mq, const CUtensorMap& mc, cudaLaunchConfig_t cfg) {
  using C = Aw<E8, PAIR>;
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure([](int) {
    return cudaFuncSetAttribute(attn_weights_kernel<E8, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.runs * p.splits * C::NQ));
  cfg.blockDim = dim3(AW_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute attr[2];
  attr[0] = cfg.attrs[0];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::NQ;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_weights_kernel<E8, PAIR>, p, mq, mc);
}

cudaError_t launch_attn_weights(AwParams p, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  const int64_t most = min(p.max_n, p.cap);           // (0: a report is all that can come of it)
  const AwPlan plan = attn_weights_plan(p.B, p.Q, p.max_n);
  p.runs = plan.runs;
  p.splits = p.Q > 0 && most > 0 ? plan.splits : 0;
  p.pitch = attn_weights_pitch(p.max_n);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  if (p.splits > 0) {
    CUtensorMap mq = {}, mc = {};                     // (of what the kernel does not copy: unused)
    if (p.Q > 1 && !encode_bf16_rows512_halves(&mq, p.q, (uint64_t)p.B * p.Q * H, H)) return cudaErrorInvalidValue;
    if (p.scales8 && !encode_u8_rows512_sw128(&mc, p.kv, (uint64_t)p.B * p.cap, AW_KEYS)) return cudaErrorInvalidValue;
    if (p.scales8) e = p.Q == 1 ? aw_launch<true, false>(p, mq, mc, cfg) : aw_launch<true, true>(p, mq, mc, cfg);
    else e = p.Q == 1 ? aw_launch<false, false>(p, mq, mc, cfg) : aw_launch<false, true>(p, mq, mc, cfg);
    if (e != cudaSuccess || p.splits == 1) return e;
  }
  const int blocks = (int)max(ceil_div(most, 256), (int64_t)1);
  cfg.gridDim = dim3((unsigned)p.B * (unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_weights_join_kernel, p, blocks);
}

}  // namespace csa2
