// Attention of 64 query heads over every visible key of the shared 512-d latent
// (K = V), on the 5th-generation tensor cores: the window rows, a few first
// rows that stay visible (sinks), and the entries of the 4-bit or of the 8-bit cache.
//
//   o_h = sum_i softmax_i(scale q_h . v_i) v_i,   lse_h = log sum_i exp(scale q_h . v_i)
//
// A query's keys are numbered in chunks of 64: the window rows (positions
// max(0, t-W+1) .. t), then the sinks (those before the window), then the cache
// entries.  A CTA walks a run of one query's chunks with one running softmax
// state.  A call with too few queries to fill the GPU divides each query's chunks
// over `split` CTAs, and keys_combine_kernel joins their states.
//
// Per chunk, with the 64 heads as the rows of M = 64 tiles:
//   * S = Q K^T   N = keys, K = 512 in two halves of 256 dims (16 MMAs each)
//   * softmax, two lanes a head, straight from TMEM; P = 2^(S scale log2 e - m) goes back
//     to TMEM over S as the 16-bit A operand of the next product.  The reference m of a head
//     moves only when a chunk's scores exceed it by far (KA_TOP, KA_MOST, KA_TAU; then the head's
//     O and its sum are rescaled), and P stays inside f16
//   * O += P V    N = 2 x 256 dims, K = keys: V is the K tile read MN-major (twice with two-part P)
// An M = 64 tile takes 16 lanes of each of TMEM's four lane quarters, so two of them
// share columns: half h of the dims has its Q, its part of S and its O in lanes
// 16h .. 16h + 15 (256 columns of O, 128 of Q, twice 64 of S), P lies in both.  With Q and P
// in TMEM a product reads only the K tile from shared memory, 16 of its 32 cycles at
// N = 64 (with Q there too it takes all 32, and the fill's stores come on top: 3100 to 3300
// cycles a chunk, and 2300 to 2500 with Q and P in TMEM and the third buffer).
// Operands: F16 (calls with cache entries or E4M3 rows) keeps every dequantised FP4
// value (at most 6 significant bits, 2^-10 .. 2688) and every E4M3 value exactly and
// rounds q and bf16 window rows to f16, exact inside [2^-14, 65504], with P to 11
// bits (fewer below 2^-22 of the largest weight, see KA_TOP); a head of q that reaches 2^16 is
// scaled into f16's range by a power of two, so that q may be of any size, as with bf16
// operands.  With bf16 rows alone the operands are bf16: q and rows as they are, P as two bf16
// of 8 bits, its rounding and what that left (a second product with the same V): with the
// first alone the errors of the outputs are 1.3 times those of their own rounding, with both
// 1.00; 16 queries of 132 rows take 9.0 us instead of 7.7.  The sum of the softmax is taken
// before any rounding, in binary32.
//
// Shared memory: three K buffers of [64 keys][512 dims] (two halves of 32 KB, four SW128
// column chunks each; the third takes Q on its way to TMEM first) and a staging area
// for the next chunk's entries as stored (18 KB; of 8-bit codes 32).  Roles:
// warps 0..3 move Q, then softmax; warps 4..11 fill the K buffers (from the staged bytes
// through registers; bf16 rows are rounded in place if need be); warps 0..7 write the
// output; warp 12 issues the MMAs, S of chunk c + 1 before O of chunk c, so that the
// softmax of a chunk runs beside the products of its neighbours; warp 13 issues the copies.
// All waits are bounded; a timeout reports CSA2_ERR_TIMEOUT and every thread still takes
// every barrier.
//
// Bound by the tensor cores, on which an M = 64 tile takes as long as one of M = 128 (two queries a
// tile would need all of TMEM for O): 2048 cycles a chunk, 3072 with two-part P.  2048 queries over 8192
// entries 1.93 ms, 1.02 PFLOP/s, their pipe active in 86 % of the cycles; 16 queries over 131,072 entries
// 262 us, 0.99 PFLOP/s; 602 queries of 1000 E4M3 rows 114 us.  A CTA costs about 7 us beside its chunks: 16
// queries of 132 bf16 rows take 9.0 us.
// With 8-bit entries the shared memory binds too: 2048 cycles a chunk (products 1024, staged bytes in and
// out 512, widened codes 512) beside 2074 of MMAs.  16 queries over 131,072 entries 271 us; 2048 over 8192 would
// take 2.06 ms, pairs of CTAs (pair_attention.cu) 1.53.  (Codes to registers without staging, four lanes a key,
// the same; staged rows without a swizzle, two keys a phase with their pieces in turn, 2.65 ms.)
#include <cfloat>

#include "attn_common.cuh"
#include "keys_common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int KA_SOFT_WARPS = 4;                          // softmax: lane = (half of the dims or keys, head)
constexpr int KA_OUT_WARPS = 2 * KA_SOFT_WARPS;             // output: these and the first fill warps
constexpr int KA_FILL_WARPS = 8;                          // K buffers
constexpr int KA_FILL = 32 * KA_FILL_WARPS;
constexpr int KA_MMA_WARP = KA_SOFT_WARPS + KA_FILL_WARPS;
constexpr int KA_COPY_WARP = KA_MMA_WARP + 1;
constexpr int KA_THREADS = 32 * (KA_COPY_WARP + 1);
constexpr int KA_KEYS = KEYS_CHUNK;                       // keys per chunk
constexpr int KA_COL = 64 * 128;                          // [64 rows][64 dims] 16-bit, SW128
constexpr int KA_HALF = 4 * KA_COL;                       // half of a K buffer: 256 dims
constexpr int KA_BUFS = 3;                                // K buffers: chunk c in c % 3
constexpr int KA_OFF_STAGE = KA_BUFS * 2 * KA_HALF;
constexpr int KA_OFF_OUT = 0;                             // outputs: [32 rows][128 dims] bf16 an output warp, over the K buffers
template <bool E8> constexpr int KA_ENTRY = E8 ? D : MAIN_BYTES;          // bytes of an entry as stored
template <bool E8> constexpr int KA_OFF_SMALL = KA_OFF_STAGE + KA_KEYS * KA_ENTRY<E8>;
constexpr int KA_TMEM_COLS = 512;
constexpr int KA_O_COL = 0;                               // half h of the dims: lanes 16h .. of each quarter
constexpr int KA_Q_COL = 256;
constexpr int KA_S_COL = 384;                             // S, then P, of chunk c at 64 (c % 2)
constexpr uint32_t KA_HALF_LANES = 16u << 16;
constexpr int KA_AHEAD = 5;                               // chunks of entries that are on their way to L2

// A wait for a phase by its parity needs that the barrier cannot have passed the phase
// after it: whatever completes that one must itself wait for the waiter.  Where two
// phases in a row do not depend on the waiter, there are two barriers in turn.
struct KaSmall {
  uint64_t q_full, q_moved;           // TMA: Q; Q is in TMEM (a softmax warp each)
  uint64_t stage_full, stage_free;    // the staged bytes have come / were read (a fill warp each)
  uint64_t row_full[KA_BUFS][2];      // TMA: rows in half h of K buffer i
  uint64_t full[KA_BUFS][2];          // half h of K buffer i is filled (a fill warp each)
  uint64_t free_[KA_BUFS];            // O of the chunk in K buffer i is done
  uint64_t s_full[2];                 // S of every second chunk is done
  uint64_t p_ready[2];                // its P is written, O rescaled if needed (a softmax warp each)
  float sum[H];                       // of the softmax
  uint32_t tmem_base;
  int err;
};
template <bool E8> constexpr int KA_SMEM = KA_OFF_SMALL<E8> + (int)sizeof(KaSmall);
static_assert(KA_SMEM<true> <= 227 * 1024, "shared memory per CTA");

__device__ __noinline__ bool ka_timeout(int* err, WsHeader* hdr, int where) {
  if (atomicExch(err, 1) == 0) report(hdr, CSA2_ERR_TIMEOUT, where);
  return false;
}

// `ok = ok && ka_wait(..)`: a thread that has given up once waits no more.
__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t count, KaSmall& sm, WsHeader* hdr, int where) {
  return tc::bar_wait(bar, count & 1u) || ka_timeout(&sm.err, hdr, where);
}

// One query's keys, and a CTA's run of their chunks [c_lo, c_lo + n): window rows, then
// sinks, then cache entries.
struct KaRun {
  int64_t t, lo;                      // position, first window position
  int64_t r0;                         // buffer row of the run's first window key, were it chunk 0
  int64_t s0, e0;                     // the same for sinks and entries (negative: they start later)
  int n, cw, cr;                      // chunks; those before cw are of the window, before cr of rows
  uint32_t wl, sl, el;                // keys of each kind from chunk 0 on (chunk c has them less 64 c)
};

__device__ __forceinline__ KaRun ka_run(const KeysParams& p, int64_t t, int64_t base, int32_t n_entries, int sp,
                                        int split) {
  KaRun q;
  q.t = t;
  const bool live = q.t >= 0;
  // W = 0: no window, and no first position of one (t + 1 need not exist)
  q.lo = live && p.W > 0 && q.t >= p.W ? q.t - p.W + 1 : 0;
  // the window positions lo .. t that lie in rows 0 .. S - 1 (unsigned differences: any
  // two positions have one), so that the work is bounded by what was supplied
  int64_t row = 0, wn = 0, en = 0;
  if (live && p.W > 0 && q.t >= base) {
    const uint64_t s = (uint64_t)p.S, r0 = q.lo > base ? (uint64_t)q.lo - (uint64_t)base : 0;
    const uint64_t end = (uint64_t)q.t - (uint64_t)base;     // row of position t
    const uint64_t r1 = end < s ? end + 1 : s;
    if (r0 < r1) {
      row = (int64_t)r0;
      wn = (int64_t)(r1 - r0);
    }
  }
  const int64_t sn = live ? (q.lo < p.n_sink ? q.lo : (int64_t)p.n_sink) : 0;
  if (live && p.main_kv) {
    // (m is 1 or 2, and t + 1 has to exist)
    en = min((min(q.t, INT64_MAX - 1) + 1) >> (p.m - 1), (int64_t)n_entries);
    if (en > p.cap) en = p.cap;       // reported by the kernel
    if (en < 0) en = 0;
  }
  const int64_t cw = ceil_div(wn, KA_KEYS), cr = cw + ceil_div(sn, KA_KEYS), nc = cr + ceil_div(en, KA_KEYS);
  const uint32_t each = (uint32_t)nc / (uint32_t)split, more = (uint32_t)nc - each * (uint32_t)split;   // nc < 2^27
  const int64_t c_lo = (int64_t)sp * each + min((uint32_t)sp, more);
  q.n = (int)(each + ((uint32_t)sp < more ? 1u : 0u));
  q.cw = (int)max(cw - c_lo, (int64_t)0);
  q.cr = (int)max(cr - c_lo, (int64_t)0);
  q.r0 = row + KA_KEYS * c_lo;
  q.s0 = KA_KEYS * (c_lo - cw);
  q.e0 = KA_KEYS * (c_lo - cr);
  // every count is below 2^31 and so is 64 c: no wrap where a chunk has keys of the kind
  q.wl = (uint32_t)(wn - KA_KEYS * c_lo);
  q.sl = (uint32_t)(sn - q.s0);
  q.el = (uint32_t)(en - q.e0);
  return q;
}

// x, the same in every lane, in a uniform register.
__device__ __forceinline__ uint32_t ka_uniform(uint32_t x) { return __reduce_or_sync(0xFFFFFFFFu, x); }

// Keys of chunk c (1 .. 64).
__device__ __forceinline__ int ka_keys(const KaRun& q, int c) {
  const uint32_t left = (c < q.cw ? q.wl : c < q.cr ? q.sl : q.el) - (uint32_t)(KA_KEYS * c);
  return left < (uint32_t)KA_KEYS ? (int)left : KA_KEYS;
}

template <bool F16, bool E8>
__global__ void __launch_bounds__(KA_THREADS, 1)
keys_attn_kernel(KeysParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_rows,
                 const __grid_constant__ CUtensorMap map_sinks) {
  static_assert(F16 || !E8, "8-bit entries are widened to f16");
  constexpr int ENTRY = KA_ENTRY<E8>;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* stage = smem + KA_OFF_STAGE;
  KaSmall& sm = *reinterpret_cast<KaSmall*>(smem + KA_OFF_SMALL<E8>);

  if (tc::smem_u32(smem) & 1023u) {                   // the swizzled tiles need the declared alignment
    if (threadIdx.x == 0) report(p.hdr, CSA2_ERR_CUDA, 1);
    return;
  }
  const int split = p.split;
  const int64_t bq = blockIdx.x / (uint32_t)split;
  const int sp = (int)(blockIdx.x % (uint32_t)split);
  const int b = (int)((uint32_t)bq / (uint32_t)p.Q);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  float* part = p.part + (int64_t)blockIdx.x * KA_PART_FLOATS;   // with split > 1

  // ---------------- set-up (reads no input: overlaps the previous kernel)
  if (warp == KA_MMA_WARP) tc::tmem_alloc(&sm.tmem_base, KA_TMEM_COLS);
  if (tid == 0) {
    tc::bar_init(&sm.q_full, 1);
    tc::bar_init(&sm.q_moved, KA_SOFT_WARPS);
    tc::bar_init(&sm.stage_full, 1);
    tc::bar_init(&sm.stage_free, KA_FILL_WARPS);
    for (int i = 0; i < KA_BUFS; i++) {
      for (int h = 0; h < 2; h++) {
        tc::bar_init(&sm.row_full[i][h], 1);
        tc::bar_init(&sm.full[i][h], KA_FILL_WARPS);
      }
      tc::bar_init(&sm.free_[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::bar_init(&sm.s_full[i], 1);
      tc::bar_init(&sm.p_ready[i], KA_SOFT_WARPS);
    }
    sm.err = 0;
    tc::bar_init_fence();
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_rows);
    tc::prefetch_tensormap(&map_sinks);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns: an allocation of them begins at column 0
  if (sm.tmem_base != 0 && tid == 0) report(p.hdr, CSA2_ERR_CUDA, 2);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // (one latency for all three.  The copy of Q into the last K buffer begins with the position's: a padded query needs
  // none.  2048 window queries, all but a quarter of them padding: 77.0 us, 82.4 when each has its Q copied)
  const int64_t base = E8 && p.W == 0 ? 0 : p.base_pos[b], t = p.q_pos[bq];
  const int32_t n_entries = p.main_kv ? p.n_entries[b] : 0;
  if (tid == 32 * KA_COPY_WARP && t >= 0) {
    tc::bar_arrive_expect_tx(&sm.q_full, 8u * KA_COL);
    for (int h = 0; h < 2; h++)
      tc::tma_load_3d(smem + ((KA_BUFS - 1) * 2 + h) * KA_HALF, &map_q, 0, (int32_t)(bq * H), 4 * h, &sm.q_full);
  }
  const KaRun q = ka_run(p, t, base, n_entries, sp, split);
  const int n_ch = q.n;
  if (sp == 0 && tid == 0 && q.t >= 0) {              // what the caller did not supply
    if (E8 && p.W == 0) {                             // no window
    } else if (q.lo < base) report(p.hdr, CSA2_ERR_BOUNDS, q.lo);
    else if ((uint64_t)q.t - (uint64_t)base >= (uint64_t)p.S) report(p.hdr, CSA2_ERR_BOUNDS, q.t);
    if (n_entries > p.cap && p.main_kv) report(p.hdr, CSA2_ERR_BOUNDS, n_entries);
  }

  // Chunk c (counted from c_lo) uses K buffer c % 3; it is that buffer's use c / 3.
  if (warp == KA_MMA_WARP) {
    // ================= MMAs (the whole warp runs the loop, one lane issues)
    // An MMA takes its addresses and descriptors from uniform registers.  They stay there when
    // the compiler sees that every lane has the same: TMEM addresses are constants (the CTA has
    // all of TMEM, from column 0), and what the chunks follow from is read from memory, so it
    // goes through a reduction over the warp, whose result is uniform.
    constexpr uint32_t idesc_s = F16 ? tc::idesc_f16(H, 0, 0, 0) : tc::idesc_bf16(H, 0, 0, 0);       // + N
    constexpr uint32_t idesc_o = F16 ? tc::idesc_f16(H, 256, 0, 1) : tc::idesc_bf16(H, 256, 0, 1);
    const uint64_t k_d = tc::smem_desc(tc::smem_u32(smem), 16, 1024, tc::SW_128B);
    const uint64_t v_d = tc::smem_desc(tc::smem_u32(smem), KA_COL, 1024, tc::SW_128B);
    const uint32_t leader = tc::elect_one();
    KaRun run;                                        // q, uniform
    run.cw = (int)ka_uniform((uint32_t)q.cw);
    run.cr = (int)ka_uniform((uint32_t)q.cr);
    run.wl = ka_uniform(q.wl);
    run.sl = ka_uniform(q.sl);
    run.el = ka_uniform(q.el);
    const int n = (int)ka_uniform((uint32_t)n_ch);
    bool ok = n > 0 ? ka_wait(&sm.q_moved, 0, sm, p.hdr, 40) : true;
    int sb = 0, su = 0, ob = 0;                       // K buffer and use of the next S, K buffer of the next O
    auto scores = [&](int c) {
      const uint32_t idesc = idesc_s | (uint32_t)((ka_keys(run, c) + 15) >> 4 << 1) << 17;
      const uint32_t s = KA_S_COL + 64 * (c & 1);
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        ok = ok && ka_wait(&sm.full[sb][h], su, sm, p.hdr, 41);
        tc::fence_after_sync();
        const uint64_t ka = k_d + (uint32_t)((2 * sb + h) * (KA_HALF >> 4));
        const uint32_t lanes = h * KA_HALF_LANES;
#pragma unroll
        for (int i = 0; i < 16; i++)
          tc::mma_f16_ts_warp(leader, s + lanes, KA_Q_COL + lanes + 8 * i,
                              ka + ((uint32_t)((i >> 2) * KA_COL + (i & 3) * 32) >> 4), idesc, i ? 1u : 0u);
      }
      tc::commit_warp(leader, &sm.s_full[c & 1]);
      if (++sb == KA_BUFS) sb = 0, su++;
    };
    if (n > 0) scores(0);
    for (int c = 0; c < n; c++) {
      if (c + 1 < n) scores(c + 1);
      const int steps = (ka_keys(run, c) + 15) >> 4;
      ok = ok && ka_wait(&sm.p_ready[c & 1], c >> 1, sm, p.hdr, 42);
      tc::fence_after_sync();
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        const uint64_t va = v_d + (uint32_t)((2 * ob + h) * (KA_HALF >> 4));
        const uint32_t lanes = h * KA_HALF_LANES;
#pragma unroll
        for (int ks = 0; ks < KA_KEYS / 16; ks++)
          if (ks < steps)
#pragma unroll
            for (int part = 0; part < (F16 ? 1 : 2); part++)     // P, what its rounding left of it
              tc::mma_f16_ts_warp(leader, KA_O_COL + lanes, KA_S_COL + 64 * (c & 1) + lanes + 32 * part + 8 * ks,
                                  va + (uint32_t)(ks * (2048 >> 4)), idesc_o, (c || ks || part) ? 1u : 0u);
      }
      tc::commit_warp(leader, &sm.free_[ob]);
      if (++ob == KA_BUFS) ob = 0;
    }
  } else if (warp == KA_COPY_WARP) {
    // ================= copies
    if (lane == 0 && n_ch > 0) {
      bool ok = true;
      uint32_t staged = 0;                            // uses of the staging area
      auto next_stage = [&](uint32_t bytes) {
        if (staged > 0) ok = ok && ka_wait(&sm.stage_free, staged - 1, sm, p.hdr, 43);
        staged++;
        tc::bar_arrive_expect_tx(&sm.stage_full, bytes);
      };
      int kb = 0, use = 0;
      // entries ahead of the staging area into L2: a copy from there takes a third of the
      // time of one from memory, and there is room for one chunk only
      const uint8_t* kv = p.main_kv + ((int64_t)b * p.cap + q.e0) * ENTRY;   // entry 0 of chunk 0
      auto ahead = [&](int c) {
        if (c >= q.cr && c < n_ch) tc::prefetch_l2(kv + (int64_t)c * (KA_KEYS * ENTRY), ka_keys(q, c) * ENTRY);
      };
      for (int c = 0; c < n_ch; c++) {
        if (p.main_kv && c == 1)                      // (behind the first chunk's own copies)
          for (int i = 1; i < 1 + KA_AHEAD; i++) ahead(i);
        if (c >= q.cr) {                              // entries, contiguous
          const uint32_t bytes = (uint32_t)((E8 ? KA_KEYS : ka_keys(q, c)) * ENTRY);
          next_stage(bytes);
          if (E8) {                                   // four column chunks of 128 dims, SW128
            for (int i = 0; i < D / 128; i += 2)
              tc::tma_load_3d(stage + i * (KA_KEYS * 128), &map_sinks, 0,
                              (int32_t)((int64_t)b * p.cap + q.e0 + KA_KEYS * c), i, &sm.stage_full);
          } else {
            tc::bulk_load(stage, kv + (int64_t)c * (KA_KEYS * ENTRY), bytes, &sm.stage_full);
          }
          if (c > 0) ahead(c + KA_AHEAD);
          continue;
        }
        if (p.main_kv && c > 0) ahead(c + KA_AHEAD);
        const bool window = c < q.cw;
        const CUtensorMap* map = window ? &map_rows : &map_sinks;
        const int32_t y = (int32_t)(window ? (int64_t)b * p.S + q.r0 + KA_KEYS * c : (int64_t)b * p.n_sink + q.s0 + KA_KEYS * c);
        // the tensor cores (the softmax warps, of Q) have read the buffer, which is waited for here
        if (use > 0) ok = ok && ka_wait(&sm.free_[kb], use - 1, sm, p.hdr, 44);
        else if (kb == KA_BUFS - 1) ok = ok && ka_wait(&sm.q_moved, 0, sm, p.hdr, 44);
        for (int h = 0; h < 2; h++) {
          unsigned char* kt = smem + (2 * kb + h) * KA_HALF + (p.rows_fp8 ? KA_COL / 2 : 0);
          tc::bar_arrive_expect_tx(&sm.row_full[kb][h], p.rows_fp8 ? KA_HALF / 2 : KA_HALF);
          for (int i = 0; i < 4; i++) tc::tma_load_2d(kt + i * KA_COL, map, (4 * h + i) * 64, y, &sm.row_full[kb][h]);
        }
        if (++kb == KA_BUFS) kb = 0, use++;
      }
    }
    __syncwarp();
  } else if (warp >= KA_SOFT_WARPS) {
    // ================= K buffers
    const int ft = tid - 32 * KA_SOFT_WARPS;
    bool ok = true;
    // thread = (key, part j: 32 of each 128 dims).  The lanes of an eight-lane phase hold keys
    // k and k + 2: with 18 units of 16 bytes an entry, their reads lie in eight different bank
    // groups
    const int k8 = (ft >> 2) & 7, j = ft & 3;
    const int key = ((ft >> 2) & ~7) + ((k8 & 4) | (k8 & 1) << 1 | (k8 >> 1 & 1));
    const bool odd = (j & 2) != 0;
    // 16 bytes of codes (32 dims) times their two scales, the bytes of `w2`
    auto dequant = [&](const uint4& c, uint32_t w2, uint32_t* o) {
      const uint32_t sa = e4m3x2_to_f16x2(prmt(w2, 0u, 0x0000u)), sb = e4m3x2_to_f16x2(prmt(w2, 0u, 0x1111u));
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int g = 0; g < 4; g++) {
        e2m1x8_to_f16(cw[g], o + 4 * g);
#pragma unroll
        for (int x = 0; x < 4; x++) o[4 * g + x] = hmul2(o[4 * g + x], g < 2 ? sa : sb);
      }
    };
    // 32 dims of key `key` into a quarter (two column chunks): column chunk j / 2, units
    // 4 (j % 2) ..; lanes with j >= 2 walk them as g ^ 1, so that the eight lanes of a phase store
    // to eight different bank groups
    auto store = [&](unsigned char* kt, const uint32_t* o) {
      unsigned char* dst = kt + (j >> 1) * KA_COL + key * 128;
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const uint4 v = make_uint4(odd ? o[4 * (g ^ 1)] : o[4 * g], odd ? o[4 * (g ^ 1) + 1] : o[4 * g + 1],
                                   odd ? o[4 * (g ^ 1) + 2] : o[4 * g + 2], odd ? o[4 * (g ^ 1) + 3] : o[4 * g + 3]);
        const uint32_t unit = (uint32_t)(4 * (j & 1) + (odd ? g ^ 1 : g));
        *reinterpret_cast<uint4*>(dst + ((unit ^ (uint32_t)(key & 7)) << 4)) = v;
      }
    };
    // 32 E4M3 dims of row `key` from a quarter; rows behind the chunk's last: zeros.  Lanes with
    // j >= 2 take their two pieces in the other order (bank groups)
    auto widen = [&](const unsigned char* kt, uint32_t* o, int n) {
      const uint4* src = reinterpret_cast<const uint4*>(kt + (j >> 1) * KA_COL + KA_COL / 2 + key * 64 + 32 * (j & 1));
      uint4 a = make_uint4(0u, 0u, 0u, 0u), e = a;
      if (key < n) {
        a = src[odd ? 1 : 0];
        e = src[odd ? 0 : 1];
      }
      const uint32_t v[8] = {odd ? e.x : a.x, odd ? e.y : a.y, odd ? e.z : a.z, odd ? e.w : a.w,
                             odd ? a.x : e.x, odd ? a.y : e.y, odd ? a.z : e.z, odd ? a.w : e.w};
#pragma unroll
      for (int x = 0; x < 8; x++) {
        o[2 * x] = e4m3x2_to_f16x2(v[x]);
        o[2 * x + 1] = e4m3x2_to_f16x2(v[x] >> 16);
      }
    };
    uint32_t staged = 0;                              // uses of the staging area
    // the reads of the staged bytes are done, before a copy (the asynchronous proxy) writes there
    // again: without the fence the arrival may overtake reads whose values are not used yet
    auto stage_read = [&]() {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.stage_free);
    };
    int kb = 0, use = 0;
    for (int c = 0; c < n_ch; c++) {
      const int keys = ka_keys(q, c);
      const bool entries = c >= q.cr;
      if (use > 0) {
        ok = ok && ka_wait(&sm.free_[kb], use - 1, sm, p.hdr, 47);
        tc::fence_after_sync();
      } else if (kb == KA_BUFS - 1) {
        ok = ok && ka_wait(&sm.q_moved, 0, sm, p.hdr, 47);
      }
      uint4 cd[4] = {}, sc[2] = {};                   // entries: codes of the four quarters, scales of the two halves
      // 8-bit entries: a lane takes 64 dims of each half of one key, so that eight lanes of a phase have
      // eight rows and both swizzles spread them over the banks.  (Keys behind the last: whatever lies there;
      // codes are finite and their weights 0.)
      uint4 c8[E8 ? 8 : 1] = {};
      const int k8l = 32 * ((ft >> 5) & 1) + lane, part8 = ft >> 6;
      if (F16 && entries) {
        // all at once (263 us for 16 queries over 131,072 entries; a half at a time, which holds
        // the staging area longer, 310)
        ok = ok && ka_wait(&sm.stage_full, staged++, sm, p.hdr, 46);
        if (E8) {
          // dims 64 part8 .. of half h: units 4 (part8 % 2) .. of the 128-dim column chunk 2 h + part8 / 2
          const unsigned char* e = stage + (part8 >> 1) * (KA_KEYS * 128);
#pragma unroll
          for (int i = 0; i < (E8 ? 8 : 0); i++)
            c8[i] = *reinterpret_cast<const uint4*>(e + (i >> 2) * (2 * KA_KEYS * 128) +
                                                    sw128((uint32_t)k8l, 16u * (uint32_t)(4 * (part8 & 1) + (i & 3))));
        } else if (key < keys) {                      // keys behind the last: zeros
          const uint4* e = reinterpret_cast<const uint4*>(stage + key * ENTRY);
#pragma unroll
          for (int i = 0; i < 4; i++) cd[i] = e[4 * i + j];
          sc[0] = e[16];
          sc[1] = e[17];
        }
        stage_read();
      }
#pragma unroll
      for (int h = 0; h < 2; h++) {
        unsigned char* kt = smem + (2 * kb + h) * KA_HALF;
        if (E8 && entries) {
          unsigned char* dst = kt + part8 * KA_COL;
#pragma unroll
          for (int i = 0; i < (E8 ? 4 : 0); i++) {
            uint32_t o[8];
            i8x16_to_f16(c8[4 * h + i], o);
            *reinterpret_cast<uint4*>(dst + sw128((uint32_t)k8l, 32u * i)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + sw128((uint32_t)k8l, 32u * i + 16u)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        } else if (F16 && (entries || p.rows_fp8)) {
          uint32_t o[2][16];
          if (!E8 && entries) {
            // scale bytes 2j, 2j + 1 of each quarter
            dequant(cd[2 * h], (odd ? sc[h].y : sc[h].x) >> (16 * (j & 1)), o[0]);
            dequant(cd[2 * h + 1], (odd ? sc[h].w : sc[h].z) >> (16 * (j & 1)), o[1]);
          } else {
            // E4M3 rows, in the upper halves of the column chunks: all are read before any is written
            ok = ok && ka_wait(&sm.row_full[kb][h], use, sm, p.hdr, 48);
            widen(kt, o[0], keys);
            widen(kt + 2 * KA_COL, o[1], keys);
            named_sync(1, KA_FILL);
          }
          store(kt, o[0]);
          store(kt + 2 * KA_COL, o[1]);
        } else {
          // bf16 rows, where the copy has put them (rows come first: copy `use` of the buffer too):
          // rounded to f16 when the operands are f16, rows behind the chunk's last set to zero
          // (what is not seen may hold anything, infinities among it)
          ok = ok && ka_wait(&sm.row_full[kb][h], use, sm, p.hdr, 48);
          if (F16 || keys < KA_KEYS) {
            uint4* u = reinterpret_cast<uint4*>(kt) + ft;
            uint4 x[KA_HALF / 16 / KA_FILL] = {};
#pragma unroll
            for (int i = 0; i < KA_HALF / 16 / KA_FILL; i++)
              if (F16 && (((ft + i * KA_FILL) >> 3) & (KA_KEYS - 1)) < keys) x[i] = u[i * KA_FILL];
#pragma unroll
            for (int i = 0; i < KA_HALF / 16 / KA_FILL; i++)
              if (F16 || (((ft + i * KA_FILL) >> 3) & (KA_KEYS - 1)) >= keys)
                u[i * KA_FILL] = make_uint4(bf16x2_to_f16x2(x[i].x), bf16x2_to_f16x2(x[i].y), bf16x2_to_f16x2(x[i].z),
                                            bf16x2_to_f16x2(x[i].w));
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sm.full[kb][h]);
      }
      if (++kb == KA_BUFS) kb = 0, use++;
    }
  } else {
    // ================= softmax and output: lane = (half, head 16 warp + lane % 16)
    const uint32_t quarter = (uint32_t)(warp * 32) << 16;
    float sc2 = p.scale * KA_LOG2E;                   // products to scores in powers of two
    const int head = 16 * warp + (lane & 15), half = lane >> 4;
    float m_used = -INFINITY, l_sum = 0.f;            // the head's reference; its sum over this lane's keys
    bool ok = true;
    // (without keys too: no copy may land behind the CTA's end)
    if (q.t >= 0) ok = ok && ka_wait(&sm.q_full, 0, sm, p.hdr, 45);
    if (n_ch > 0) {                                   // Q: this lane's 256 dims of its head to TMEM
      const unsigned char* qh = smem + ((KA_BUFS - 1) * 2 + half) * KA_HALF;
      __half2 most = __half2half2(__ushort_as_half(0));   // F16: largest |q| of the lane's even and odd dims
#pragma unroll 1
      for (int g = 0; g < 4; g++) {                   // column chunk g of the half: 32 columns of TMEM
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 8; u++) {
          const uint4 x = *reinterpret_cast<const uint4*>(qh + g * KA_COL + sw128((uint32_t)head, 16u * u));
          w[4 * u] = x.x;
          w[4 * u + 1] = x.y;
          w[4 * u + 2] = x.z;
          w[4 * u + 3] = x.w;
        }
        if (F16) {
#pragma unroll
          for (int x = 0; x < 32; x++) {
            w[x] = bf16x2_to_f16x2(w[x]);
            most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&w[x])));
          }
        }
        tmem_st32(quarter + KA_Q_COL + 32 * g, w);
      }
      if (F16) {
        if (__any_sync(0xFFFFFFFFu, __hisinf(__hmax(__low2half(most), __high2half(most))) != 0)) {
          // heads with a |q| of 2^16 or more, out of f16's range: once more, times a power of two that
          // puts the largest into [2^15, 2^16), and their scale times its inverse.  (An infinity
          // stays one.)
          uint32_t size = 0u;                         // largest |q|, bf16 bits (2^16: 143 << 7)
#pragma unroll 1
          for (uint32_t x = 0; x < 128; x++) {
            const uint32_t b =
                *reinterpret_cast<const uint32_t*>(qh + (x >> 5) * KA_COL + sw128((uint32_t)head, 4u * (x & 31u)));
            size = max(size, max(b & 0x7FFFu, b >> 16 & 0x7FFFu));
          }
          size = max(size, __shfl_xor_sync(0xFFFFFFFFu, size, 16));
          const int e = max(min((int)(size >> 7), 254) - 142, 0);
          const float down = __int_as_float((127 - e) << 23);
          sc2 = fmaxf(fminf(sc2 * __int_as_float((127 + e) << 23), FLT_MAX), -FLT_MAX);   // finite: a product may be 0
          tc::tmem_wait_st();
#pragma unroll 1
          for (int g = 0; g < 4; g++) {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 32; x++) {
              const uint32_t b =
                  *reinterpret_cast<const uint32_t*>(qh + g * KA_COL + sw128((uint32_t)head, 4u * x));
              w[x] = pack_f16x2(__uint_as_float(b << 16) * down, __uint_as_float(b & 0xFFFF0000u) * down);
            }
            tmem_st32(quarter + KA_Q_COL + 32 * g, w);
          }
        }
      }
      tc::tmem_wait_st();
      tc::fence_proxy_async_smem();                   // the buffer goes to copies and stores of others
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.q_moved);
    }
    int ob = 0, ou = 0;                               // K buffer and use of the chunk before
    // 8-bit entries: the scales of this lane's four blocks of keys of chunk c (rows: 1)
    auto scales = [&](int c, float* s) {
      const int n = c < n_ch && c >= q.cr ? ka_keys(q, c) - 32 * half : 0;
      const float* at = p.scales8 + (int64_t)b * (p.cap / BLK) + (q.e0 + (int64_t)KA_KEYS * c) / BLK + 4 * half;
#pragma unroll
      for (int i = 0; i < 4; i++) s[i] = BLK * i < n ? __ldcg(at + i) : 1.f;
    };
    float s8_next[4] = {1.f, 1.f, 1.f, 1.f};
    if (E8) scales(0, s8_next);
    for (int c = 0; c < n_ch; c++) {
      float s8[4] = {1.f, 1.f, 1.f, 1.f}, by[4];      // scales, and what turns products into scores
      if (E8) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          s8[i] = s8_next[i];
          by[i] = fmaxf(fminf(sc2 * s8[i], FLT_MAX), -FLT_MAX);   // finite: a product may be 0
        }
        scales(c + 1, s8_next);
      }
      const int n = ka_keys(q, c) - 32 * half;   // this lane takes keys 32 half ..: n of them are there
      const uint32_t s_addr = quarter + KA_S_COL + 64 * (c & 1);
      ok = ok && ka_wait(&sm.s_full[c & 1], c >> 1, sm, p.hdr, 49);
      tc::fence_after_sync();
      float v[32];
      {
        // every lane holds its half of the dims' part of 64 keys: the two lanes of a head
        // swap 32 of them, so that each has the whole of its 32 keys
        uint32_t s0[32], s1[32];
        tc::tmem_ld_x32_nowait(s_addr, s0);
        tc::tmem_ld_x32_nowait(s_addr + 32, s1);
        tc::tmem_wait_ld_regs(s0);
        tc::tmem_wait_ld_regs(s1);
#pragma unroll
        for (int x = 0; x < 32; x++) {
          const float got = __uint_as_float(__shfl_xor_sync(0xFFFFFFFFu, half ? s0[x] : s1[x], 16));
          // (not to be fused with the reference's subtraction: the largest score minus itself is 0)
          v[x] = __fmul_rn(__uint_as_float(half ? s1[x] : s0[x]) + got, E8 ? by[x / BLK] : sc2);
        }
      }
      const bool whole = __all_sync(0xFFFFFFFFu, n >= 32);
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 32; x++) v[x] = x < n ? v[x] : -INFINITY;
      }
      float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 32; x++) c4[E8 ? x / BLK : x & 3] = fmaxf(c4[E8 ? x / BLK : x & 3], v[x]);
      if (E8) {
#pragma unroll
        for (int i = 0; i < 4; i++)                   // (of the reference alone: any value near it would do)
          c4[i] += __log2f(fmaxf(s8[i], KA_FLOOR8));
      }
      float cm = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
      cm = fmaxf(cm, __shfl_xor_sync(0xFFFFFFFFu, cm, 16));
      float alpha = 1.f;
      // where neighbouring scores lie 8 and more apart, a rounded cm - KA_TOP could lie too low
      const float to = F16 && fabsf(cm) < 0x1p26f ? cm - KA_TOP : cm;
      if (m_used == -INFINITY) {
        m_used = to;                                  // O holds nothing yet, or only zeros
      } else if (cm - m_used > (F16 ? KA_MOST : KA_TAU)) {   // (a sum m_used + .. could round up to the next score)
        alpha = ex2_ftz(m_used - to);
        m_used = to;
        l_sum *= alpha;
      }
      if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) {    // after the chunk before is in O
        ok = ok && ka_wait(&sm.free_[ob], ou, sm, p.hdr, 50);
        tc::fence_after_sync();
#pragma unroll 1
        for (int g = 0; g < D / 2; g += 32) {
          uint32_t o[32];
          tmem_ld32(quarter + KA_O_COL + g, o);
#pragma unroll
          for (int x = 0; x < 32; x++) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
          tmem_st32(quarter + KA_O_COL + g, o);
        }
      }
      if (c > 0 && ++ob == KA_BUFS) ob = 0, ou++;
      const float ref = m_used == -INFINITY ? 0.f : m_used;
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[16], rest[16];
#pragma unroll
      for (int x = 0; x < 16; x++) {
        float e0 = ex2_ftz(v[2 * x] - ref), e1 = ex2_ftz(v[2 * x + 1] - ref);
        l4[x & 3] += e0 + e1;
        pk[x] = E8    ? pack_f16x2(e0 * s8[2 * x / BLK], e1 * s8[2 * x / BLK])
                : F16 ? pack_f16x2(e0, e1)
                      : pack_bf16x2(e0, e1);
        if (!F16) rest[x] = bf16x2_rest(e0, e1, pk[x]);
      }
      l_sum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      // P of all 64 keys for this lane's half of the dims, over S
      auto put = [&](uint32_t taddr, const uint32_t* k) {
        uint32_t pw[32];
#pragma unroll
        for (int x = 0; x < 16; x++) {
          const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, k[x], 16);
          pw[x] = half ? got : k[x];
          pw[16 + x] = half ? k[x] : got;
        }
        tmem_st32(taddr, pw);
      };
      put(s_addr, pk);
      if (!F16) put(s_addr + 32, rest);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.p_ready[c & 1]);
    }

    const float l = l_sum + __shfl_xor_sync(0xFFFFFFFFu, l_sum, 16);
    if (half == 0) {
      sm.sum[head] = l;
      if (split > 1) {
        part[head] = m_used;
        part[H + head] = l;
      } else if (p.lse) {                             // l = 0: no visible key
        p.lse[bq * H + head] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * KA_LN2;
      }
    }
  }

  if (warp < KA_OUT_WARPS) {
    // ================= output: lane = (half of the dims, head), 128 of the half's dims a warp
    // (four warps alone take 3900 cycles, half of what the CTA needs beside its chunks)
    if (n_ch > 0) {
      const int last = n_ch - 1;
      if (*(volatile int*)&sm.err == 0) ka_wait(&sm.free_[last % KA_BUFS], last / KA_BUFS, sm, p.hdr, 51);
      tc::fence_after_sync();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    named_sync(2, 32 * KA_OUT_WARPS);                 // the sums
    const int qt = warp & 3, half = lane >> 4, head = 16 * qt + (lane & 15), g0 = 128 * (warp >> 2);
    const uint32_t o_addr = ((uint32_t)(qt * 32) << 16) + KA_O_COL + g0;
    if (split == 1) {
      const float l = sm.sum[head], inv = 1.0f / l;
      const bool none = l == 0.f;                     // no visible key: zeros
      // A lane holds 32 dims of its row at a time.  Stored from there, an instruction would touch
      // 32 rows of 1 KB with 16 bytes each (7000 cycles for 256 dims a lane); through shared memory (the K
      // buffers, whose last reader is done) it covers 256 bytes of two rows.
      unsigned char* mine = smem + KA_OFF_OUT + warp * 8192;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (n_ch > 0) tmem_ld32(o_addr + c, o);
#pragma unroll
        for (int x = 0; x < 4; x++) {
          float f[8];
#pragma unroll
          for (int y = 0; y < 8; y++) f[y] = none ? 0.f : __uint_as_float(o[8 * x + y]) * inv;
          *reinterpret_cast<uint4*>(mine + lane * 256 + ((((c >> 3) + x) ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
      }
      __syncwarp();
      uint4* out = reinterpret_cast<uint4*>(p.out + (bq * H + 16 * qt) * D);
#pragma unroll 4
      for (int x = 0; x < 16; x++) {                  // lane `row` of the warp: head 16 qt + row % 16, half row / 16
        const int row = 2 * x + half, u = lane & 15;
        out[(row & 15) * (D / 8) + (D / 16) * (row >> 4) + g0 / 8 + u] =
            *reinterpret_cast<const uint4*>(mine + row * 256 + ((u ^ (row & 7)) << 4));
      }
    } else if (n_ch > 0) {
      // a partial state: O as [dims / 4][head][4], so that the lanes of a half write 256 bytes
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
  if (warp == KA_MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(0u, KA_TMEM_COLS);
  }
}

// One query's output from its CTAs' partial states: with m = max_s m_s and
// w_s = 2^(m_s - m), O = sum_s w_s O_s / sum_s w_s l_s.  A CTA takes 16 GROUPS dims of all
// heads: thread = (slice of the states, head, 4 dims of each group), so that a warp reads pieces of
// 128 bytes of [dims / 4][head][4] and writes 32 bytes a head.  Bound by the latency of its reads (a
// state is 130 KB, in L2): a thread has BATCH states on their way while the CTA works out
// the weights.  It may start while the CTAs of the query still write their states, so these are not
// read-only for its life: no __restrict__, and every read of them is a load from L2 behind the wait.
template <int SLICES, int GROUPS, int BATCH, int MOST>
__global__ void __launch_bounds__(SLICES * H * 4)
keys_combine_kernel(const float* part, int split, uint16_t* out, float* lse) {
  constexpr int ROWS = SLICES * 4;                    // states whose references are read at once
  constexpr int CTAS = D / (16 * GROUPS);             // of a query
  __shared__ __align__(16) float weight[MOST][H];     // then the slices' sums
  __shared__ float red[ROWS][H], sum[H];
  static_assert(MOST >= (SLICES - 1) * 16 && (SLICES == 1 || GROUPS == 1), "the slices' sums lie over the weights");
  const int tid = threadIdx.x;
  const int64_t bq = blockIdx.x / CTAS;
  const int dims = (blockIdx.x % CTAS) * 16 * GROUPS;
  const int g = tid % 4, h = tid / 4 % H, z = tid / (4 * H);
  const float* pb = part + bq * split * KA_PART_FLOATS;
  const float4* o = reinterpret_cast<const float4*>(pb + 2 * H) + (dims / 4 + g) * H + h;
  float4 x[BATCH][GROUPS];                         // O of states s, s + SLICES ..
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < BATCH; i++)
      if (s + i * SLICES < split)
#pragma unroll
        for (int k = 0; k < GROUPS; k++) x[i][k] = __ldcg(o + (int64_t)(s + i * SLICES) * (KA_PART_FLOATS / 4) + k * 4 * H);
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  load(z);
  {
    const int hw = tid % H, r = tid / H;
    float mx = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int s = r; s < split; s += ROWS) mx = fmaxf(mx, __ldcg(pb + (int64_t)s * KA_PART_FLOATS + hw));
    red[r][hw] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; i++) mx = fmaxf(mx, red[i][hw]);
    __syncthreads();
#pragma unroll 4
    for (int s = r; s < split; s += ROWS) {
      const float* ps = pb + (int64_t)s * KA_PART_FLOATS + hw;
      const float l = __ldcg(ps + H), w = l != 0.f ? exp2f(__ldcg(ps) - mx) : 0.f;   // l = 0: a state without keys
      weight[s][hw] = w;
      L += w * l;
    }
    red[r][hw] = L;
    __syncthreads();
    if (r == 0) {
      L = 0.f;
#pragma unroll
      for (int i = 0; i < ROWS; i++) L += red[i][hw];
      sum[hw] = L;
      if (lse && dims == 0) lse[bq * H + hw] = L == 0.f ? -INFINITY : (mx + log2f(L)) * KA_LN2;
    }
    __syncthreads();
  }
  float4 a[GROUPS] = {};
  for (int s = z; s < split; s += BATCH * SLICES) {
    if (s > z) load(s);
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
      const float w = s + i * SLICES < split ? weight[s + i * SLICES][h] : 0.f;
      if (w != 0.f) {                                 // a state without keys holds no O
#pragma unroll
        for (int k = 0; k < GROUPS; k++) {
          a[k].x += w * x[i][k].x;
          a[k].y += w * x[i][k].y;
          a[k].z += w * x[i][k].z;
          a[k].w += w * x[i][k].w;
        }
      }
    }
  }
  if (SLICES > 1) {
    float4* slice = reinterpret_cast<float4*>(weight);
    __syncthreads();
    if (z > 0) slice[tid - 4 * H] = a[0];
    __syncthreads();
    if (z > 0) return;
#pragma unroll
    for (int i = 0; i < SLICES - 1; i++) {
      const float4 y = slice[tid + i * 4 * H];
      a[0].x += y.x;
      a[0].y += y.y;
      a[0].z += y.z;
      a[0].w += y.w;
    }
  }
  const float inv = sum[h] == 0.f ? 0.f : 1.0f / sum[h];   // no visible key: zeros
#pragma unroll
  for (int k = 0; k < GROUPS; k++)
    *reinterpret_cast<uint2*>(out + (bq * H + h) * D + dims + 16 * k + 4 * g) =
        make_uint2(pack_bf16x2(a[k].x * inv, a[k].y * inv), pack_bf16x2(a[k].z * inv, a[k].w * inv));
}

// ------------------------------------------------------------------ host side
// CTAs per query: the number whose time is least.  In chunks (1.2 us each) a CTA costs those it
// has and about KA_FIXED more (set-up, the first keys, the output), one to an SM; the join costs
// 2.5, 1/16 for each state of a query and 1/48 for each of the call.  At most KA_WAVES CTAs an SM, which
// bounds the partial states to 80 MB.  The GPU's 152 SMs are a constant here so that the workspace can be
// sized without a device.  One query, us (undivided / as chosen): 600 entries 19.7 / 11.6, 2000
// 44.2 / 13.8, 8000 149 / 17.3.
constexpr int KA_FIXED = 6, KA_WAVES = 4;
// Queries whose join takes CTAs of four slices: one slice / four, us a call over 600, 2000 and 8000 entries:
// 1 query 13.2 / 12.1, 15.0 / 14.3, 21.5 / 18.0; 4 queries 13.8 / 12.1, 16.5 / 14.4, 25.9 / 18.0; 5 queries
// 13.0 / 15.1, 17.5 / 17.3, 26.0 / 22.6; 8 queries 13.5 / 15.4, 17.7 / 17.5, 25.8 / 25.1; 12 queries
// 14.0 / 18.0, 18.4 / 20.8, 27.7 / 30.3.  (Five to eight long caches would gain too; the weights of one
// slice's CTA lie in shared memory for 608 / (KC_LATENT + 1) states.)
constexpr int KC_LATENT = 4;

static int keys_split(int64_t BQ, int64_t chunks, int64_t* cost_out = nullptr) {
  if (BQ <= 0) return 1;
  int best = 1;
  int64_t best_cost = 48 * ceil_div(BQ, KA_SMS) * (KA_FIXED + chunks);   // in 48ths
  for (int s = 2; s <= KA_SMS && s <= chunks && BQ * s <= KA_WAVES * KA_SMS; s++) {
    const int64_t cost = 48 * ceil_div(BQ * s, KA_SMS) * (KA_FIXED + ceil_div(chunks, s)) + 120 + 3 * s + BQ * s;
    if (cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  if (cost_out) *cost_out = best_cost;
  return best;
}

// A call over an 8-bit cache: pairs of CTAs with two queries each (pair_attention.cu), or a CTA a query as
// here, whichever takes less time by the same count.  A pair's chunk takes 0.85 us (1.2 here), and it costs
// PAIR_FIXED of them, 9 us, beside its own (7 here).  Us (pairs / single CTAs, each with its best split):
// 1 x 100 queries of 4000 entries 60 / 81, 1 x 4 of 131,072 64 / 80, 8 x 4 of 4000 28.6 / 32.6, 16 x 2 of 2000
// 21.2 / 23.0, 1 x 16 of 4000 21.8 / 23.2, 1 x 2 of 8000 17.6 / 17.4, 1 x 8 of 600 14.5 / 12.9, 1 x 32 of 1000
// 18.2 / 17.7.  (Of 15 sizes two are chosen wrongly: 4 x 3 of 30,000 65.5 / 63.3 and 2 x 8 of 2000 17.4 / 18.4.)
// The lengths of the sequences are on the device, and `chunks` is the longest's.  So a split counts for pairs with
// the mean of two times: of B lengths alike, and of B lengths spread evenly below the longest (B / B, .. 1 / B of
// it: (B + 1) / 2B on average), whose items fill the gaps in each other's waves.  Of 18 sizes (2 to 32 sequences, 4
// to 128 queries, 2000 to 30,000 entries) the split taken costs 1.04 times the best one's time when lengths are
// alike (1.19 at most: 7 x 16 of 5300, 103 us for 86), 1.03 when they are spread (1.16); a split for lengths alike
// 1.00 and 1.18 (1.68).
constexpr int PAIR_FIXED = 11;

Cache8Plan cache8_plan(int B, int Q, int64_t chunks) {
  int64_t single = 0;
  const Cache8Plan alone{false, keys_split((int64_t)B * Q, chunks, &single)};
  const int64_t pairs = (int64_t)B * ((Q + 1) / 2), slots = KA_SMS / 2;
  if (Q < 2 || B < 1) return alone;
  int split = 1;
  int64_t best = INT64_MAX, time = 0;
  for (int s = 1; s <= slots && s <= chunks && (s == 1 || pairs * s <= KA_WAVES * slots); s++) {
    const int64_t join = s > 1 ? 169 + 4 * s + 3 * pairs * s : 0, longest = 48 * (PAIR_FIXED + ceil_div(chunks, s));
    const int64_t alike = longest * ceil_div(pairs * s, slots) + join;
    const int64_t each = PAIR_FIXED + (B + 1) * ceil_div(chunks, s) / (2 * (int64_t)B);
    const int64_t spread = B > 1 ? max(longest, 48 * pairs * s * each / slots) + join : alike;
    if (alike + spread < best) {
      split = s;
      best = alike + spread;
      time = alike;
    }
  }
  return time == 0 || 85 * time >= 120 * single ? alone : Cache8Plan{true, split};   // (48ths of 0.85 and 1.2 us)
}

size_t cache8_part_bytes(int B, int Q, int64_t chunks) {
  const int s = cache8_plan(B, Q, chunks).split;
  return s > 1 ? (size_t)((int64_t)B * Q * s) * KA_PART_FLOATS * sizeof(float) : 0;
}

size_t keys_part_bytes(int64_t BQ, int64_t chunks) {
  const int s = keys_split(BQ, chunks);
  return s > 1 ? (size_t)(BQ * s) * KA_PART_FLOATS * sizeof(float) : 0;
}

template <bool F16, bool E8>
static cudaError_t keys_launch(const KeysParams& p, int64_t BQ, const CUtensorMap& mq, const CUtensorMap& mr,
                               const CUtensorMap& ms, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure([](int) {
    return cudaFuncSetAttribute(keys_attn_kernel<F16, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, KA_SMEM<E8>);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(BQ * p.split));
  cfg.blockDim = dim3(KA_THREADS);
  cfg.dynamicSmemBytes = KA_SMEM<E8>;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set-up overlaps the previous kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, keys_attn_kernel<F16, E8>, p, mq, mr, ms);
  return e != cudaSuccess || p.split == 1 ? e : launch_keys_join(p, BQ, stream);
}

cudaError_t launch_keys_join(const KeysParams& p, int64_t BQ, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cc = {};
  // Few queries: CTAs of many threads, one to an SM.  Else one slice; up to four states then
  // want the registers of half as many CTAs (4 states of 111 queries 132 us in all, 136 otherwise).
  const bool latent = BQ <= KC_LATENT, few = !latent && p.split <= 4;
  cc.gridDim = dim3((unsigned)(BQ * (few ? D / 32 : D / 16)));
  cc.blockDim = dim3((latent ? 4 : 1) * H * 4);
  cc.stream = stream;
  cc.attrs = attr;
  cc.numAttrs = 1;
  auto* kernel = latent ? keys_combine_kernel<4, 1, 8, KA_SMS>
                 : few ? keys_combine_kernel<1, 2, 4, 4> : keys_combine_kernel<1, 1, 8, KA_WAVES * KA_SMS / (KC_LATENT + 1)>;
  return cudaLaunchKernelEx(&cc, kernel, (const float*)p.part, p.split, p.out, p.lse);
}

// Calls that window_attention.cu takes: short windows, where its time is less.  In tenths of a us: this
// file's kernel takes 70 and 1/10 a key for each wave of queries; the ring's 60, 3/10 a key for a CTA's
// first window, and for its longest CTA 45 a tile (two queries) and 9/10 a key for each further sequence in
// its run (of 410 calls measured both ways none loses more than 2 % by it).  The SMs are KA_SMS here, for
// the kernel's launch the device's: with another number the rule would still be right, but not the best.
// Window 128, 4 sinks, bf16, us (here / the ring's): 1 x 153 queries 17.9 / 16.3, 1 x 304 19.4 / 17.3, 1 x 608
// 39.8 / 21.6, 1 x 2432 164 / 66, 100 x 4 28.1 / 34.2, 152 x 4 43.3 / 21.7, 60 x 5 19.4 / 34.1, 80 x 8 49.1 / 38.6,
// 608 x 1 48.8 / 85.8; window 32: 1 x 153 14.2 / 11.8, 100 x 4 22.7 / 20.6.
static bool keys_in_ring(const KeysParams& p, int B, int64_t BQ) {
  if (p.main_kv || !window_ring_fits(p.W, p.n_sink) || BQ <= KA_SMS) return false;
  const int64_t keys = p.W + p.n_sink, pairs = (p.Q + 1) / 2, tiles = B * pairs, ctas = min(tiles, (int64_t)KA_SMS);
  int64_t longest = 0;
  for (int64_t i = 0; i < ctas; i++) {
    const int64_t lo = tiles * i / ctas, hi = tiles * (i + 1) / ctas;
    longest = max(longest, 45 * (hi - lo) + ((hi - 1) / pairs - lo / pairs) * keys * 9 / 10);
  }
  return 60 + keys * 3 / 10 + longest < ceil_div(BQ, KA_SMS) * (70 + keys / 10);
}

cudaError_t launch_keys_attention(KeysParams p, int B, int64_t chunks, void* part, cudaStream_t stream) {
  const int64_t BQ = (int64_t)B * p.Q;
  if (BQ == 0) return cudaSuccess;
  if (keys_in_ring(p, B, BQ)) return launch_window_ring(p, B, stream);
  const Cache8Plan plan = p.scales8 ? cache8_plan(B, p.Q, chunks) : Cache8Plan{false, keys_split(BQ, chunks)};
  p.split = plan.split;
  p.part = reinterpret_cast<float*>(part);
  CUtensorMap mq, mr, ms;
  if (!encode_bf16_rows512_halves(&mq, p.q, (uint64_t)BQ * H, H)) return cudaErrorInvalidValue;
  auto rows = [&](CUtensorMap* map, const void* base, int64_t n) {
    return p.rows_fp8 ? encode_u8_rows512(map, base, (uint64_t)n, KA_KEYS)
                      : encode_bf16_rows512(map, base, (uint64_t)n, KA_KEYS);
  };
  const int64_t nr = (int64_t)B * p.S, nk = (int64_t)B * p.n_sink;
  // an empty buffer is never read: its map is a copy of one that exists
  if (nr > 0 && !rows(&mr, p.rows, nr)) return cudaErrorInvalidValue;
  if (nr == 0) mr = mq;
  if (nk > 0 && !rows(&ms, p.sinks, nk)) return cudaErrorInvalidValue;
  if (nk == 0) ms = mr;
  if (p.scales8) {                                    // no sinks: their map is the codes'
    if (plan.pairs) {
      const cudaError_t e = launch_pair_attention(p, B, mr, stream);
      return e != cudaSuccess || p.split == 1 ? e : launch_keys_join(p, BQ, stream);
    }
    if (p.cap > 0 && !encode_u8_rows512_halves(&ms, p.main_kv, (uint64_t)B * p.cap, KA_KEYS)) return cudaErrorInvalidValue;
    return keys_launch<true, true>(p, BQ, mq, mr, ms, stream);
  }
  return p.main_kv || p.rows_fp8 ? keys_launch<true, false>(p, BQ, mq, mr, ms, stream)
                                 : keys_launch<false, false>(p, BQ, mq, mr, ms, stream);
}

}  // namespace csa2
