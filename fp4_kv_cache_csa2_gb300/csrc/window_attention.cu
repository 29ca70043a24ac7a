// Attention of 64 query heads over a short window of the shared 512-d latent (K = V) and a
// few first rows, for many queries in a row (a prefill chunk of a window-only layer).
//
//   o_h = sum_i softmax_i(scale q_h . v_i) v_i,   lse_h = log sum_i exp(scale q_h . v_i)
//
// With 128 keys a query the work is bound by memory: 64 KB of q and 64 KB of output against
// 17 Mflop.  Two neighbouring queries of a sequence make the 128 rows of a tile (64 heads
// each); all keys that the two see, at most 160, lie in shared memory at once, so a tile needs
// one softmax and no running state.  Row r of the window buffer lies in slot n_sink + r mod R of
// a ring, sink p in slot p; the order of keys does not matter to the products, and which
// slots a query sees is a circular interval.  A CTA takes a run of neighbouring tiles, so that
// a tile loads the two rows that its queries see newly (the first one its window, by all warps but
// the copies'), and streams q in and the output out:
//   warps 0..3    softmax, one thread a row, from TMEM; P goes back over S as 16-bit A operands
//   warps 4..7    output: O by 64 dims to bf16 rows
//   warps 8..11   the ring: rows that the next tile's queries see newly
//   warp 12       S = Q K^T (M = 128, N = slots, K = 512), Q in 64-dim pieces through 3 stages
//   warp 13       O = P V by 64 dims (M = 128, N = 64, K = slots, P in two parts), V the ring read MN-major
//   warp 14       copies of Q
// S has two buffers of 160 columns of TMEM and O three of 64, so a tile's products run beside
// the softmax and the output of its neighbours.  Operands are bf16 (q and bf16 rows as they
// are, E4M3 rows exactly, P as two bf16 of 8 bits, its rounding and what that left, with the
// softmax's sum taken before either; the first alone makes the outputs' errors 1.3 times those
// of their own rounding).  8192 queries of 128 rows and 4 sinks: 205 us, 5.3 TB/s of q, rows and
// output (one part 183; the second product is most of the difference: a tile's S waits for the P V
// of the tile before the last).
//
// A slot that a query does not see has weight zero for it, and zero times an infinity or a NaN
// is a NaN.  A row goes to the ring while tiles are at work only if all of it is finite; when
// one is not, each query of the tile is taken alone, on a ring that holds what it sees and zeros.
// All waits are bounded; a timeout reports CSA2_ERR_TIMEOUT, a thread that gave up one waits no
// more, and every thread still takes every CTA barrier.
#include "attn_common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int WA_SLOTS = 160;                             // keys of a tile at most
constexpr int WA_ROWS = 2 * H;
constexpr int WA_OUT_WARP = 4, WA_RING_WARP = 8, WA_S_WARP = 12, WA_O_WARP = 13, WA_COPY_WARP = 14;
constexpr int WA_THREADS = 32 * 15;
constexpr int WA_RING = 128;                              // threads of the ring warps
constexpr int WA_KCOL = WA_SLOTS * 128;                   // column chunk of 64 dims: [slots][128 B], SW128
constexpr int WA_QCOL = WA_ROWS * 128;                    // [128 rows][64 dims], SW128
constexpr int WA_STAGES = 3;
constexpr int WA_OFF_Q = 8 * WA_KCOL;
constexpr int WA_OFF_OUT = WA_OFF_Q + WA_STAGES * WA_QCOL;   // [32 rows][64 dims] bf16 an output warp
constexpr int WA_OFF_SMALL = WA_OFF_OUT + 4 * 4096;
constexpr int WA_S_COL = 0, WA_O_COL = 2 * WA_SLOTS, WA_O_BUFS = 3;
constexpr int WA_JOBS = 4;
constexpr float WA_LOG2E = 1.4426950408889634f;
constexpr float WA_LN2 = 0.6931471805599453f;

// What one pass over the ring works on: the tile's queries that see slots, and those whose
// output it writes.
struct WaJob {
  uint32_t bq;                        // first query
  int write;                          // bit i: query i's output is written; -1: no more jobs
  int sn[2], s0[2], cnt[2];           // sinks [0, sn); window slots s0 .., cnt of them around the ring
};

// A wait for a phase by its parity needs that the barrier cannot have passed the phase after
// it: whatever completes that one waits for the waiter.
struct WaSmall {
  WaJob job[WA_JOBS];
  float2 state[2][WA_ROWS];           // 1 / sum and lse of each row, of every second job
  uint32_t next_bq[WA_JOBS];          // first query of a job to come, ~0: none, for the copies of Q
  uint64_t told[WA_JOBS];             // it is written
  uint64_t job_ready[WA_JOBS];        // the job is written and its slots are filled (a ring warp each)
  uint64_t job_free[WA_JOBS];         // every reader is done with it
  uint64_t q_full[WA_STAGES], q_free[WA_STAGES];
  uint64_t s_full[2], p_ready[2], state_ready[2], pv_done[2];   // of every second job
  uint64_t o_full[WA_O_BUFS], o_free[WA_O_BUFS];
  uint32_t tmem_base;
  int err;
};
constexpr int WA_SMEM = WA_OFF_SMALL + (int)sizeof(WaSmall);
constexpr int WA_READERS = 1 + 1 + 1 + 4 + 4;             // of a job: copy, S, O, softmax, output warps
static_assert(WA_SMEM <= 227 * 1024, "shared memory per CTA");
static_assert(WA_O_COL + 64 * WA_O_BUFS <= 512, "TMEM columns");

__device__ __noinline__ bool wa_timeout(int* err, WsHeader* hdr, int where) {
  if (atomicExch(err, 1) == 0) report(hdr, CSA2_ERR_TIMEOUT, where);
  return false;
}

__device__ __forceinline__ bool wa_wait(uint64_t* bar, uint32_t count, WaSmall& sm, WsHeader* hdr, int where) {
  return tc::bar_wait(bar, count & 1u) || wa_timeout(&sm.err, hdr, where);
}

// One query's rows of the window buffer and its sinks.
struct WaQuery {
  int r0, wn, sn;
};

__device__ __forceinline__ WaQuery wa_query(const KeysParams& p, int64_t t, int64_t base, bool reports) {
  WaQuery q{0, 0, 0};
  if (t < 0) return q;
  const int64_t lo = t >= p.W ? t - p.W + 1 : 0;
  q.sn = lo < p.n_sink ? (int)lo : p.n_sink;
  if (t >= base) {                    // unsigned differences: any two positions have one
    const uint64_t s = (uint64_t)p.S, r0 = lo > base ? (uint64_t)lo - (uint64_t)base : 0;
    const uint64_t end = (uint64_t)t - (uint64_t)base;
    const uint64_t r1 = end < s ? end + 1 : s;
    if (r0 < r1) {
      q.r0 = (int)r0;
      q.wn = (int)(r1 - r0);
    }
  }
  if (reports) {                      // what the caller did not supply
    if (lo < base) report(p.hdr, CSA2_ERR_BOUNDS, lo);
    else if ((uint64_t)t - (uint64_t)base >= (uint64_t)p.S) report(p.hdr, CSA2_ERR_BOUNDS, t);
  }
  return q;
}

// f16x2 -> bf16x2, for values that bf16 holds exactly
__device__ __forceinline__ uint32_t wa_f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ bool wa_not_finite(const uint4& v) {
  constexpr uint32_t E = 0x7F80u;
  return (v.x & E) == E || (v.x >> 16 & E) == E || (v.y & E) == E || (v.y >> 16 & E) == E || (v.z & E) == E ||
         (v.z >> 16 & E) == E || (v.w & E) == E || (v.w >> 16 & E) == E;
}

// Barrier ID of N threads that tells each of them whether any came with x set.  A flag in shared
// memory, read behind a plain barrier, could already be the next tile's: a warp that reads it late
// would part from the others.
template <int ID, int N>
__device__ __forceinline__ bool wa_any(bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.or.pred b, %2, %3, a;\n"
               " selp.u32 %0, 1, 0, b;\n}\n" : "=r"(r) : "r"((uint32_t)x), "n"(ID), "n"(N) : "memory");
  return r != 0;
}

// A row of the window buffer, 16 bytes of each half a lane (E4M3: 16 dims in the first).  From L2: the
// kernel before, beside whose end this one starts, may have written it.
__device__ __forceinline__ void wa_load_row(uint4* v, const uint8_t* row, int fp8, int lane) {
  const uint4* src = reinterpret_cast<const uint4*>(row);
  v[0] = __ldcg(src + lane);
  if (!fp8) v[1] = __ldcg(src + 32 + lane);
}

// to its slot, as bf16.  False: it is not finite, and stays out unless `any` row may go in
__device__ __forceinline__ bool wa_put_row(unsigned char* ring, int slot, const uint4* v, int fp8, bool any, int lane) {
  uint4 lo = v[0], hi = v[1];
  if (fp8) {
    const uint32_t e[4] = {lo.x, lo.y, lo.z, lo.w};
    uint32_t o[8];
#pragma unroll
    for (int y = 0; y < 4; y++) {
      o[2 * y] = wa_f16x2_to_bf16x2(e4m3x2_to_f16x2(e[y]));
      o[2 * y + 1] = wa_f16x2_to_bf16x2(e4m3x2_to_f16x2(e[y] >> 16));
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
  }
  if (!any && __any_sync(0xFFFFFFFFu, wa_not_finite(lo) || wa_not_finite(hi))) return false;
  const int u0 = fp8 ? 2 * lane : lane, u1 = fp8 ? 2 * lane + 1 : 32 + lane;   // 16-byte units
  unsigned char* dst = ring + slot * 128;
  *reinterpret_cast<uint4*>(dst + (u0 >> 3) * WA_KCOL + (((u0 ^ slot) & 7) << 4)) = lo;
  *reinterpret_cast<uint4*>(dst + (u1 >> 3) * WA_KCOL + (((u1 ^ slot) & 7) << 4)) = hi;
  return true;
}

// The rows that a tile's queries see: both queries at once when they together fit the ring.
struct WaTile {
  int lo, hi;                         // rows [lo, hi), if joint
  bool joint;
};

__device__ __forceinline__ WaTile wa_tile(const WaQuery& q0, const WaQuery& q1, int R) {
  WaTile t;
  t.lo = q0.wn == 0 ? q1.r0 : (q1.wn == 0 ? q0.r0 : min(q0.r0, q1.r0));
  t.hi = max(q0.wn ? q0.r0 + q0.wn : 0, q1.wn ? q1.r0 + q1.wn : 0);
  t.joint = q0.wn == 0 || q1.wn == 0 || t.hi - t.lo <= R;
  return t;
}

// bits [a, b) of the 32 from g on
__device__ __forceinline__ uint32_t wa_bits(int a, int b, int g) {
  a = max(a - g, 0);
  b = min(b - g, 32);
  return a < b ? (b == 32 ? ~0u : (1u << b) - 1u) & ~((1u << a) - 1u) : 0u;
}

__device__ __forceinline__ void wa_tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                  "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

__global__ void __launch_bounds__(WA_THREADS, 1)
window_attn_kernel(KeysParams p, int B, int slots, const __grid_constant__ CUtensorMap map_q) {
  extern __shared__ __align__(1024) unsigned char smem[];
  WaSmall& sm = *reinterpret_cast<WaSmall*>(smem + WA_OFF_SMALL);
  if (tc::smem_u32(smem) & 1023u) {                   // the swizzled tiles need the declared alignment
    if (threadIdx.x == 0) report(p.hdr, CSA2_ERR_CUDA, 1);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  // ---------------- set-up (reads no input: overlaps the previous kernel)
  if (warp == WA_S_WARP) tc::tmem_alloc(&sm.tmem_base, 512);
  if (tid == 0) {
    for (int i = 0; i < WA_JOBS; i++) {
      tc::bar_init(&sm.told[i], 1);
      tc::bar_init(&sm.job_ready[i], WA_RING / 32);
      tc::bar_init(&sm.job_free[i], WA_READERS);
    }
    for (int i = 0; i < WA_STAGES; i++) {
      tc::bar_init(&sm.q_full[i], 1);
      tc::bar_init(&sm.q_free[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.p_ready[i], 4);
      tc::bar_init(&sm.state_ready[i], 4);
      tc::bar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < WA_O_BUFS; i++) {
      tc::bar_init(&sm.o_full[i], 1);
      tc::bar_init(&sm.o_free[i], 4);
    }
    sm.err = 0;
    tc::bar_init_fence();
    tc::prefetch_tensormap(&map_q);
  }
  // slots that were never filled are read with weight zero: they must be finite
  for (int i = tid; i < 8 * WA_KCOL / 16; i += WA_THREADS) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns: an allocation of them begins at column 0
  if (sm.tmem_base != 0 && tid == 0) report(p.hdr, CSA2_ERR_CUDA, 2);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int pairs = (p.Q + 1) >> 1;
  const int64_t tiles = (int64_t)B * pairs;
  bool ok = true;
  const int64_t k_lo = tiles * blockIdx.x / gridDim.x, k_hi = tiles * (blockIdx.x + 1) / gridDim.x;
  const int R = slots - p.n_sink;                     // window slots
  const size_t row_bytes = p.rows_fp8 ? D : 2 * D;
  int held_b = -1, rl = 0, rh = 0, ns = 0;            // the ring: rows [rl, rh) and sinks [0, ns) of sequence held_b
  if (warp != WA_COPY_WARP) {
    // the first tile's window is loaded by every other warp (a call of one tile a CTA: 15 us, 19 with the
    // ring warps alone), its queries by that one meanwhile.  If a row is not finite, the ring
    // warps begin anew
    const int b = (int)(k_lo / pairs), i = 2 * (int)(k_lo - (int64_t)b * pairs);
    const int64_t at = (int64_t)b * p.Q + i;
    if (tid == 0) {
      sm.next_bq[0] = (uint32_t)at;
      tc::bar_arrive(&sm.told[0]);
    }
    const int64_t base = p.base_pos[b];
    const WaQuery q0 = wa_query(p, p.q_pos[at], base, false);
    const WaQuery q1 = wa_query(p, i + 1 < p.Q ? p.q_pos[at + 1] : -1, base, false);
    const WaTile t = wa_tile(q0, q1, R);
    const int n_row = t.joint ? max(t.hi - t.lo, 0) : 0, n_sink = t.joint ? max(q0.sn, q1.sn) : 0;
    const uint8_t* rows = p.rows + ((size_t)b * (size_t)p.S + (size_t)t.lo) * row_bytes;
    const uint8_t* sinks = p.sinks + (size_t)b * (size_t)p.n_sink * row_bytes;
    bool bad = !t.joint;
#pragma unroll 1
    for (int x0 = warp; x0 < n_row + n_sink; x0 += 4 * WA_COPY_WARP) {
      uint4 v[4][2];
#pragma unroll
      for (int y = 0; y < 4; y++) {
        const int x = x0 + y * WA_COPY_WARP;
        v[y][0] = v[y][1] = make_uint4(0u, 0u, 0u, 0u);
        if (x < n_row + n_sink)
          wa_load_row(v[y], x < n_row ? rows + (size_t)x * row_bytes : sinks + (size_t)(x - n_row) * row_bytes, p.rows_fp8, lane);
      }
#pragma unroll
      for (int y = 0; y < 4; y++) {
        const int x = x0 + y * WA_COPY_WARP;
        if (x >= n_row + n_sink) continue;
        int slot = p.n_sink + t.lo % R + x;
        if (slot >= slots) slot -= R;
        if (x >= n_row) slot = x - n_row;
        if (!wa_put_row(smem, slot, v[y], p.rows_fp8, false, lane)) bad = true;
      }
    }
    tc::fence_proxy_async_smem();
    if (!wa_any<2, 32 * WA_COPY_WARP>(bad)) {
      held_b = b;
      rl = t.lo;
      rh = t.lo + n_row;
      ns = n_sink;
    }
  }
  // the readers' view of the jobs
  auto next_job = [&](uint32_t j) -> WaJob {
    ok = ok && wa_wait(&sm.job_ready[j % WA_JOBS], j / WA_JOBS, sm, p.hdr, 60);
    WaJob job = sm.job[j % WA_JOBS];
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) job.write = -1;                          // given up: no more jobs
    return job;
  };
  auto done_job = [&](uint32_t j) {
    __syncwarp();
    if (lane == 0) tc::bar_arrive(&sm.job_free[j % WA_JOBS]);
  };

  if (warp == WA_S_WARP) {
    // ================= S = Q K^T
    const uint32_t idesc = tc::idesc_bf16(WA_ROWS, 0, 0, 0) | (uint32_t)(slots >> 3) << 17;
    const uint64_t q_d = tc::smem_desc(tc::smem_u32(smem + WA_OFF_Q), 16, 1024, tc::SW_128B);
    const uint64_t k_d = tc::smem_desc(tc::smem_u32(smem), 16, 1024, tc::SW_128B);
    const uint32_t leader = tc::elect_one();
    int stage = 0;
    uint32_t use = 0;
    for (uint32_t j = 0; next_job(j).write >= 0; j++) {
      if (j >= 2) ok = ok && wa_wait(&sm.pv_done[j & 1], (j >> 1) - 1, sm, p.hdr, 61);   // P of job j - 2 lay over this S
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < 8; c++) {
        ok = ok && wa_wait(&sm.q_full[stage], use, sm, p.hdr, 62);
        tc::fence_after_sync();
        const uint64_t qa = q_d + (uint32_t)(stage * (WA_QCOL >> 4)), ka = k_d + (uint32_t)(c * (WA_KCOL >> 4));
#pragma unroll
        for (int k = 0; k < 4; k++)
          tc::mma_f16_ss_warp(leader, WA_S_COL + WA_SLOTS * (j & 1), qa + 2 * k, ka + 2 * k, idesc, (c || k) ? 1u : 0u);
        tc::commit_warp(leader, &sm.q_free[stage]);
        if (++stage == WA_STAGES) stage = 0, use++;
      }
      tc::commit_warp(leader, &sm.s_full[j & 1]);
      done_job(j);
    }
  } else if (warp == WA_O_WARP) {
    // ================= O = P V, 64 dims at a time
    constexpr uint32_t idesc = tc::idesc_bf16(WA_ROWS, 64, 0, 1);
    const uint64_t v_d = tc::smem_desc(tc::smem_u32(smem), WA_KCOL, 1024, tc::SW_128B);
    const uint32_t leader = tc::elect_one();
    const int steps = slots >> 4;
    int buf = 0;
    uint32_t use = 0;
    for (uint32_t j = 0; next_job(j).write >= 0; j++) {
      ok = ok && wa_wait(&sm.p_ready[j & 1], j >> 1, sm, p.hdr, 63);
#pragma unroll 1
      for (int u = 0; u < 8; u++) {
        if (use > 0) ok = ok && wa_wait(&sm.o_free[buf], use - 1, sm, p.hdr, 64);
        tc::fence_after_sync();
        const uint64_t va = v_d + (uint32_t)(u * (WA_KCOL >> 4));
#pragma unroll 2
        for (int k = 0; k < steps; k++) {             // P of 16 keys, then what its rounding left of it
          const uint32_t pa = WA_S_COL + WA_SLOTS * (j & 1) + 32 * (k >> 1) + 8 * (k & 1);
          const uint64_t vk = va + (uint32_t)(k * (2048 >> 4));
          tc::mma_f16_ts_warp(leader, WA_O_COL + 64 * buf, pa, vk, idesc, k ? 1u : 0u);
          tc::mma_f16_ts_warp(leader, WA_O_COL + 64 * buf, pa + 16, vk, idesc, 1u);
        }
        tc::commit_warp(leader, &sm.o_full[buf]);
        if (++buf == WA_O_BUFS) buf = 0, use++;
      }
      tc::commit_warp(leader, &sm.pv_done[j & 1]);
      done_job(j);
    }
  } else if (warp == WA_COPY_WARP) {
    // ================= Q in 64-dim pieces
    int stage = 0;
    uint32_t use = 0;
    for (uint32_t j = 0;; j++) {
      // told before the job's slots are filled: Q is on its way while the ring's rows come
      ok = ok && wa_wait(&sm.told[j % WA_JOBS], j / WA_JOBS, sm, p.hdr, 59);
      ok = __all_sync(0xFFFFFFFFu, ok);
      const uint32_t bq = sm.next_bq[j % WA_JOBS];
      if (bq == ~0u || !ok) break;
      for (int c = 0; c < 8; c++) {
        if (use > 0) ok = ok && wa_wait(&sm.q_free[stage], use - 1, sm, p.hdr, 65);
        if (lane == 0) {
          tc::bar_arrive_expect_tx(&sm.q_full[stage], WA_QCOL);
          tc::tma_load_2d(smem + WA_OFF_Q + stage * WA_QCOL, &map_q, c * 64, (int32_t)(bq * H), &sm.q_full[stage]);
        }
        if (++stage == WA_STAGES) stage = 0, use++;
      }
      done_job(j);
    }
  } else if (warp >= WA_RING_WARP) {
    // ================= the ring
    const int rt = tid - 32 * WA_RING_WARP, rw = rt >> 5;
    uint32_t j = 0;                                   // jobs published, and (told ones) announced
    uint32_t announced = 1;
    auto pv_wait = [&](uint32_t job) { ok = ok && wa_wait(&sm.pv_done[job & 1], job >> 1, sm, p.hdr, 66); };
    // the first query of the next job, as soon as it is known
    auto announce = [&](uint32_t bq) {
      if (announced >= WA_JOBS)
        ok = ok && wa_wait(&sm.job_free[announced % WA_JOBS], announced / WA_JOBS - 1, sm, p.hdr, 67);
      if (rt == 0) {
        sm.next_bq[announced % WA_JOBS] = bq;
        tc::bar_arrive(&sm.told[announced % WA_JOBS]);
      }
      announced++;
    };
    auto publish = [&](uint32_t bq, int write, int sn0, int r0, int n0, int sn1, int r1, int n1) {
      tc::fence_proxy_async_smem();
      if (rt == 0) {                                  // the slot is free: announce waited for it
        WaJob& job = sm.job[j % WA_JOBS];
        job.bq = bq;
        job.write = write;
        job.sn[0] = sn0;
        job.s0[0] = p.n_sink + r0 % R;
        job.cnt[0] = n0;
        job.sn[1] = sn1;
        job.s0[1] = p.n_sink + r1 % R;
        job.cnt[1] = n1;
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.job_ready[j % WA_JOBS]);
      j++;
    };
    bool stale = false;                               // it may hold rows that are not finite
    int before = 0;                                   // first row that the job before sees
    int b = (int)(k_lo / pairs), i0 = 2 * (int)(k_lo - (int64_t)b * pairs);
    // positions of the next tile, loaded one tile ahead
    int64_t nt0 = -1, nt1 = -1, nbase = 0;
    auto fetch = [&](int fb, int fi) {
      const int64_t at = (int64_t)fb * p.Q + fi;
      nt0 = p.q_pos[at];
      nt1 = fi + 1 < p.Q ? p.q_pos[at + 1] : -1;
      nbase = p.base_pos[fb];
    };
    if (k_lo < k_hi) fetch(b, i0);
    for (int64_t k = k_lo; k < k_hi; k++) {
      const uint32_t bq = (uint32_t)b * (uint32_t)p.Q + (uint32_t)i0;
      const int have = i0 + 1 < p.Q ? 3 : 1;
      if (k > k_lo) announce(bq);
      const WaQuery q0 = wa_query(p, nt0, nbase, rt == 0), q1 = wa_query(p, nt1, nbase, rt == 0);
      const uint8_t* rows = p.rows + (size_t)b * (size_t)p.S * row_bytes;
      const uint8_t* sinks = p.sinks + (size_t)b * (size_t)p.n_sink * row_bytes;
      const int tile_b = b;
      i0 += 2;
      if (i0 >= p.Q) i0 = 0, b++;
      if (k + 1 < k_hi) fetch(b, i0);
      const WaTile tile = wa_tile(q0, q1, R);
      const int lo = tile.lo, hi = tile.hi;
      int todo = tile.joint ? 3 : 1 | 2 << 2;         // two bits a job: the queries it takes
      bool exact = false, first = true;               // exact: on zeros and what its query sees
      while (todo != 0) {
        const int mask = todo & 3;
        todo >>= 2;
        if (!first) announce(bq);
        first = false;
        const int L = mask == 3 ? lo : (mask == 2 ? q1.r0 : q0.r0);
        const int E = mask == 3 ? hi : L + (mask == 2 ? q1.wn : q0.wn);      // rows [L, E)
        const int NS = mask == 3 ? max(q0.sn, q1.sn) : (mask == 2 ? q1.sn : q0.sn);
        // what may be written when: after every tile at work, or after the last but one, or (a
        // new row takes a slot that the job before sees) after the one before
        bool all = false, last = false;
        if (exact || stale || tile_b != held_b) {
          all = true;
          held_b = exact ? -1 : tile_b;
          rl = rh = L;
          ns = 0;
        } else if (E > L && (L < rl || L > rh)) {
          all = true;
          rl = rh = L;
        } else {
          last = E > rh && E - R > before;
        }
        const bool zero = exact || stale;
        stale = exact;
        bool open = false;                            // whether that wait is over
        auto gate = [&]() {
          if (open) return;
          open = true;
          if (j >= 2) pv_wait(j - 2);
          if (j >= 1 && (all || last)) pv_wait(j - 1);
          if (zero) {
            for (int x = rt; x < 8 * WA_KCOL / 16; x += WA_RING) reinterpret_cast<uint4*>(smem)[x] = make_uint4(0u, 0u, 0u, 0u);
            named_sync(1, WA_RING);
          }
        };
        // new rows [rh, E) to their window slots, new sinks [ns, NS) to theirs.  A row that is not
        // finite is left out (and told) unless the job is exact
        bool dirty = false;
        const int n_row = max(E - rh, 0), n_all = n_row + max(NS - ns, 0);
        const int slot_r = p.n_sink + rh % R;
#pragma unroll 1
        for (int x0 = 0; x0 < n_all; x0 += 4 * (WA_RING / 32)) {
          uint4 v[4][2];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int x = x0 + 4 * i + rw;            // neighbouring rows in different warps
            v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (x < n_all)
              wa_load_row(v[i], x < n_row ? rows + (size_t)(rh + x) * row_bytes : sinks + (size_t)(ns + x - n_row) * row_bytes,
                          p.rows_fp8, lane);
          }
          gate();
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int x = x0 + 4 * i + rw;
            if (x >= n_all) continue;
            int slot = slot_r + x;
            if (slot >= slots) slot -= R;             // around the ring
            if (x >= n_row) slot = ns + x - n_row;
            if (!wa_put_row(smem, slot, v[i], p.rows_fp8, exact, lane)) dirty = true;
          }
        }
        gate();
        rh = max(rh, E);
        rl = max(rl, E - R);
        ns = max(ns, NS);
        if (wa_any<1, WA_RING>(dirty)) {              // each query of this job alone, with what it sees as it is
          const int singles = (mask & have) == 3 ? 1 | 2 << 2 : mask & have;
          todo = singles | todo << (singles > 3 ? 4 : 2);
          exact = true;
          first = true;                               // the announced job is the first of them
          continue;
        }
        before = L;
        const bool on0 = (mask & 1) != 0, on1 = (mask & 2) != 0;
        publish(bq, mask & have, on0 ? q0.sn : 0, q0.r0, on0 ? q0.wn : 0, on1 ? q1.sn : 0, q1.r0, on1 ? q1.wn : 0);
      }
    }
    announce(~0u);
    publish(0, -1, 0, 0, 0, 0, 0, 0);
  } else if (warp >= WA_OUT_WARP) {
    // ================= output: thread = row
    const int ow = warp - WA_OUT_WARP, i = ow >> 1;   // query
    const uint32_t lanes = (uint32_t)(ow * 32) << 16;
    unsigned char* mine = smem + WA_OFF_OUT + ow * 4096;
    int buf = 0;
    uint32_t use = 0;
    for (uint32_t j = 0;; j++) {
      const WaJob job = next_job(j);
      if (job.write < 0) break;
      const bool write = (job.write >> i & 1) != 0;
      const int64_t row = ((int64_t)job.bq + i) * H + (ow & 1) * 32;      // of lane 0
      ok = ok && wa_wait(&sm.state_ready[j & 1], j >> 1, sm, p.hdr, 68);
      const float2 st = sm.state[j & 1][32 * ow + lane];
      if (write && p.lse) p.lse[row + lane] = st.y;
#pragma unroll 1
      for (int u = 0; u < 8; u++) {
        ok = ok && wa_wait(&sm.o_full[buf], use, sm, p.hdr, 69);
        tc::fence_after_sync();
        uint32_t o[2][32];
        tc::tmem_ld_x32_nowait(lanes + WA_O_COL + 64 * buf, o[0]);
        tc::tmem_ld_x32_nowait(lanes + WA_O_COL + 64 * buf + 32, o[1]);
        tc::tmem_wait_ld_regs(o[0]);
        tc::tmem_wait_ld_regs(o[1]);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sm.o_free[buf]);
        if (++buf == WA_O_BUFS) buf = 0, use++;
        if (!write) continue;
        // through shared memory, so that an instruction stores 128 bytes of each of four rows
#pragma unroll
        for (int x = 0; x < 8; x++) {
          const uint32_t* w = &o[x >> 2][8 * (x & 3)];
          float f[8];
#pragma unroll
          for (int y = 0; y < 8; y++) f[y] = st.x == 0.f ? 0.f : __uint_as_float(w[y]) * st.x;   // no key: zeros
          *reinterpret_cast<uint4*>(mine + lane * 128 + ((x ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
        __syncwarp();
        uint4* out = reinterpret_cast<uint4*>(p.out + row * D + 64 * u);
#pragma unroll
        for (int x = 0; x < 8; x++) {
          const int r = 4 * x + (lane >> 3), c = lane & 7;
          __stcs(out + r * (D / 8) + c, *reinterpret_cast<const uint4*>(mine + r * 128 + ((c ^ (r & 7)) << 4)));
        }
        __syncwarp();
      }
      done_job(j);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else {
    // ================= softmax: thread = row
    const int i = warp >> 1;                          // query
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float sc2 = p.scale * WA_LOG2E;
    // rounded before the largest is subtracted: a fused multiply-add of the two would leave the largest
    // itself its rounding, 2^128 and more from scores of 2^32 on
    auto score = [&](uint32_t s) { return __fmul_rn(__uint_as_float(s), sc2); };
    for (uint32_t j = 0;; j++) {
      const WaJob job = next_job(j);
      if (job.write < 0) break;
      const int sn = i ? job.sn[1] : job.sn[0], s0 = i ? job.s0[1] : job.s0[0], cnt = i ? job.cnt[1] : job.cnt[0];
      const int wrap = max(s0 + cnt - slots, 0);      // slots n_sink .. n_sink + wrap - 1 continue the interval
      const uint32_t s_addr = lanes + WA_S_COL + WA_SLOTS * (j & 1);
      ok = ok && wa_wait(&sm.s_full[j & 1], j >> 1, sm, p.hdr, 70);
      tc::fence_after_sync();
      auto seen = [&](int g) {
        return wa_bits(0, sn, g) | wa_bits(s0, min(s0 + cnt, slots), g) | wa_bits(p.n_sink, p.n_sink + wrap, g);
      };
      float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int g = 0; g < slots; g += 32) {
        uint32_t s[32];
        tmem_ld32(s_addr + g, s);
        const uint32_t m = seen(g);
        if (m == ~0u) {
#pragma unroll
          for (int x = 0; x < 32; x++) c4[x & 3] = fmaxf(c4[x & 3], score(s[x]));
        } else {
#pragma unroll
          for (int x = 0; x < 32; x++) c4[x & 3] = fmaxf(c4[x & 3], (m >> x & 1) ? score(s[x]) : -INFINITY);
        }
      }
      const float mx = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
      const float ref = mx == -INFINITY ? 0.f : mx;
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int g = 0; g < slots; g += 32) {
        uint32_t s[32], pk[16], rest[16];
        tmem_ld32(s_addr + g, s);
        const uint32_t m = seen(g);
#pragma unroll
        for (int x = 0; x < 16; x++) {
          const float e0 = (m >> (2 * x) & 1) ? ex2_ftz(score(s[2 * x]) - ref) : 0.f;
          const float e1 = (m >> (2 * x + 1) & 1) ? ex2_ftz(score(s[2 * x + 1]) - ref) : 0.f;
          l4[x & 3] += e0 + e1;
          pk[x] = pack_bf16x2(e0, e1);
          rest[x] = bf16x2_rest(e0, e1, pk[x]);
        }
        wa_tmem_st16(s_addr + g, pk);                 // over these 32 columns of S: 16 bits a weight in two halves
        wa_tmem_st16(s_addr + g + 16, rest);
      }
      const float l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      sm.state[j & 1][32 * warp + lane] = make_float2(l == 0.f ? 0.f : 1.0f / l, l == 0.f ? -INFINITY : (mx + log2f(l)) * WA_LN2);
      __syncwarp();
      if (lane == 0) {
        tc::bar_arrive(&sm.p_ready[j & 1]);
        tc::bar_arrive(&sm.state_ready[j & 1]);
      }
      done_job(j);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  // after a timeout copies may be in flight that nobody waited for: time for them to land
  if (*(volatile int*)&sm.err != 0)
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  if (warp == WA_S_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(0u, 512);
  }
}

// ------------------------------------------------------------------ host side
// The ring holds the rows of two neighbouring queries and the sinks; two more rows let the
// next tile's come while this one is at work.
bool window_ring_fits(int64_t W, int n_sink) { return W + 1 + n_sink <= WA_SLOTS; }

cudaError_t launch_window_ring(const KeysParams& p, int B, cudaStream_t stream) {
  const int64_t tiles = (int64_t)B * ((p.Q + 1) / 2);
  if (tiles == 0) return cudaSuccess;
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure(
      [](int) { return cudaFuncSetAttribute(window_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WA_SMEM); });
  if (e != cudaSuccess) return e;
  int sms = 0;
  if ((e = device_sms(&sms)) != cudaSuccess) return e;
  CUtensorMap mq;
  if (!encode_bf16_rows512(&mq, p.q, (uint64_t)B * (uint64_t)p.Q * H, WA_ROWS)) return cudaErrorInvalidValue;
  const int want = (int)((p.W + 3 + p.n_sink + 15) & ~(int64_t)15);
  const int slots = want < WA_SLOTS ? want : WA_SLOTS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms));   // one CTA an SM
  cfg.blockDim = dim3(WA_THREADS);
  cfg.dynamicSmemBytes = WA_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set-up overlaps the previous kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_attn_kernel, p, B, slots, mq);
}

}  // namespace csa2
