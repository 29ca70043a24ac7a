// Attention of 64 query heads over every visible key of the shared 512-d latent
// (K = V), on the 5th-generation tensor cores: the window rows, a few first
// rows that stay visible (sinks), and the entries of the 4-bit cache.
//
//   o_h = sum_i softmax_i(scale q_h . v_i) v_i,   lse_h = log sum_i exp(scale q_h . v_i)
//
// A query's keys are numbered in chunks of 128: the window rows (positions
// max(0, t-W+1) .. t), then the sinks (those before the window), then the
// cache entries.  A CTA walks a run of a query's chunks with one running
// softmax state; a query's chunks are divided over `split` CTAs when the call
// has too few queries to fill the GPU, and keys_combine_kernel joins their
// states.
//
// Per chunk (one CTA, one query):
//   * S^T = K Q^T    M = 128 keys, N = 64 heads, K = 512   (32 MMAs, one accumulator)
//   * P^T = 2^(S^T scale log2 e - m)   16-bit, MN-major operand of the next product;
//     the reference m of a head moves only when a chunk exceeds it by more than
//     e^8 (then O^T and the sum are rescaled), so P stays inside f16
//   * O^T += V^T P^T 4 tiles of M = 128 dims, N = 64, K = 128 (32 MMAs)
// Operands: F16 (calls with cache entries) keeps every dequantised FP4 value
// exactly (at most 6 significant bits, 2^-10 .. 2688) and rounds q and bf16
// window rows to f16, exact inside [2^-14, 65504], with P to 11 bits.  Without
// cache entries the operands are bf16: q and bf16 rows as they are, E4M3 rows
// exactly, P to 8 bits (its rounding errors are independent and average out;
// the sum of the softmax is taken before that rounding, in binary32).
//
// Roles: warps 0..7 softmax and output, warps 8..15 bring a chunk into the key
// buffer (entries dequantised from registers that were loaded one chunk ahead,
// rows by TMA and then widened or rounded in place), one thread of warp 16
// issues all MMAs.  Tile t of the key buffer (dims 128t ..) is refilled as soon
// as the O^T tile t of the chunk before is done, and S^T's chain follows tile by
// tile.  All waits are bounded; a timeout reports CSA2_ERR_TIMEOUT and every
// thread still takes every barrier.
#include "attn_common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr int KA_MATH_WARPS = 8;                          // softmax, output
constexpr int KA_FILL_WARPS = 8;                          // key buffer
constexpr int KA_FILL = 32 * KA_FILL_WARPS;
constexpr int KA_MMA_WARP = KA_MATH_WARPS + KA_FILL_WARPS;
constexpr int KA_THREADS = 32 * (KA_MMA_WARP + 1);
constexpr int KA_KEYS = 128;                              // keys per chunk
constexpr int KA_KCOL = KA_KEYS * 128;                    // column chunk of 64 dims: [128 keys][128 B], SW128
constexpr int KA_QCOL = H * 128;                          // [64 heads][128 B], SW128
constexpr int KA_OFF_Q = 8 * KA_KCOL;
constexpr int KA_OFF_P = KA_OFF_Q + 8 * KA_QCOL;          // P^T [128 keys][64 heads], SW128
constexpr int KA_OFF_SMALL = KA_OFF_P + KA_KEYS * H * 2;
constexpr int KA_TMEM_COLS = 512;                         // S^T 64 + O^T 256, a power of two
constexpr int KA_S_COL = 0;
constexpr int KA_O_COL = 256;
constexpr float KA_LOG2E = 1.4426950408889634f;
constexpr float KA_LN2 = 0.6931471805599453f;
constexpr float KA_TAU = 8.0f * KA_LOG2E;
constexpr int KA_PART_FLOATS = 2 * H + H * D;             // one partial state: references, sums, O [head][dim]

struct KaSmall {
  float red[KA_MATH_WARPS][32];
  alignas(16) float mv[KA_MATH_WARPS][32];
  uint64_t q_full[4];                 // TMA: Q column chunks 2t, 2t + 1
  uint64_t row_full[4];               // TMA: a row chunk's column chunks 2t, 2t + 1
  uint64_t kready[4];                 // tile t of a chunk is in the key buffer (a fill warp each)
  uint64_t s_full;                    // S^T of a chunk is done
  uint64_t p_ready;                   // P^T is written, O^T rescaled if needed (a math warp each)
  uint64_t pv_done[4];                // O^T tile t of a chunk is done
  uint32_t tmem_base;
  int err;
};
constexpr int KA_SMEM = KA_OFF_SMALL + (int)sizeof(KaSmall) + 1024;
static_assert(KA_SMEM <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ bool ka_wait(uint64_t* bar, uint32_t parity, KaSmall& sm, WsHeader* hdr, int where) {
  if (tc::bar_wait(bar, parity)) return true;
  if (atomicExch(&sm.err, 1) == 0) report(hdr, CSA2_ERR_TIMEOUT, where);
  return false;
}

// One query's keys and how they lie in chunks.
struct KaQuery {
  int64_t t, lo;                      // position, first window position
  int64_t wn, sn, en;                 // window rows, sinks, cache entries it sees
  int64_t cw, cs, nc;                 // window chunks, sink chunks, all chunks
};

__device__ __forceinline__ KaQuery ka_query(const KeysParams& p, int64_t bq, int b) {
  KaQuery q;
  q.t = p.q_pos[bq];
  const bool live = q.t >= 0;
  q.lo = live && q.t >= p.W ? q.t - p.W + 1 : 0;
  q.wn = live ? q.t - q.lo + 1 : 0;
  q.sn = live ? (q.lo < p.n_sink ? q.lo : (int64_t)p.n_sink) : 0;
  q.en = 0;
  if (live && p.main_kv) {
    q.en = visible_entries(q.t, p.m, p.n_entries[b]);
    if (q.en > p.cap) q.en = p.cap;   // reported below
    if (q.en < 0) q.en = 0;
  }
  q.cw = ceil_div(q.wn, KA_KEYS);
  q.cs = ceil_div(q.sn, KA_KEYS);
  q.nc = q.cw + q.cs + ceil_div(q.en, KA_KEYS);
  return q;
}

// A chunk's rows: where they start in their buffer (row 0 = the sequence's
// first) and which of the 128 are visible and supplied, [ra, rb).
struct KaRows {
  int64_t first;
  int ra, rb;
};

__device__ __forceinline__ KaRows ka_rows(const KeysParams& p, const KaQuery& q, int64_t c, int64_t base) {
  KaRows r;
  if (c < q.cw) {
    r.first = q.lo + KA_KEYS * c - base;
    const int64_t n = q.wn - KA_KEYS * c;
    r.rb = n < KA_KEYS ? (int)n : KA_KEYS;
    if (r.first + r.rb > p.S) r.rb = r.first >= p.S ? 0 : (int)(p.S - r.first);
    r.ra = r.first >= 0 ? 0 : (r.first <= -KA_KEYS ? KA_KEYS : (int)-r.first);
  } else {
    r.first = KA_KEYS * (c - q.cw);
    const int64_t n = q.sn - r.first;
    r.rb = n < KA_KEYS ? (int)n : KA_KEYS;
    r.ra = 0;
  }
  if (r.ra >= r.rb) r.ra = r.rb = 0;
  return r;
}

// f16x2 -> bf16x2, for values that bf16 holds exactly
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x, f.y);
}

template <bool F16, bool SPLIT>
__global__ void __launch_bounds__(KA_THREADS, 1)
keys_attn_kernel(KeysParams p, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_rows,
                 const __grid_constant__ CUtensorMap map_sinks) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = tc::align_smem_1k(smem_raw);
  unsigned char* kbuf = smem;
  unsigned char* qbuf = smem + KA_OFF_Q;
  unsigned char* pbuf = smem + KA_OFF_P;
  KaSmall& sm = *reinterpret_cast<KaSmall*>(smem + KA_OFF_SMALL);

  const int split = SPLIT ? p.split : 1;
  const int64_t bq = blockIdx.x / split;
  const int sp = blockIdx.x % split;
  const int b = (int)(bq / p.Q);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  // ---------------- set-up (reads no input: overlaps the previous kernel)
  if (warp == KA_MMA_WARP) tc::tmem_alloc(&sm.tmem_base, KA_TMEM_COLS);
  if (tid == 0) {
    for (int t = 0; t < 4; t++) {
      tc::bar_init(&sm.q_full[t], 1);
      tc::bar_init(&sm.row_full[t], 1);
      tc::bar_init(&sm.kready[t], KA_FILL_WARPS);
      tc::bar_init(&sm.pv_done[t], 1);
    }
    tc::bar_init(&sm.s_full, 1);
    tc::bar_init(&sm.p_ready, KA_MATH_WARPS);
    sm.err = 0;
    tc::bar_init_fence();
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_rows);
    tc::prefetch_tensormap(&map_sinks);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const KaQuery q = ka_query(p, bq, b);
  const int64_t base = p.base_pos[b];
  const int64_t c_lo = q.nc * sp / split, c_hi = q.nc * (sp + 1) / split;
  if (sp == 0 && tid == 0 && q.t >= 0) {              // what the caller did not supply
    if (q.lo < base) report(p.hdr, CSA2_ERR_BOUNDS, q.lo);
    else if (q.t - base >= p.S) report(p.hdr, CSA2_ERR_BOUNDS, q.t);
    if (p.main_kv && p.n_entries[b] > p.cap) report(p.hdr, CSA2_ERR_BOUNDS, p.n_entries[b]);
  }

  if (warp == KA_MMA_WARP) {
    // ================= MMAs
    if (lane == 0 && c_lo < c_hi) {
      constexpr uint32_t idesc_s = F16 ? tc::idesc_f16(KA_KEYS, H, 0, 0) : tc::idesc_bf16(KA_KEYS, H, 0, 0);
      constexpr uint32_t idesc_o = F16 ? tc::idesc_f16(128, H, 1, 1) : tc::idesc_bf16(128, H, 1, 1);
      const uint64_t a_s = tc::smem_desc(tc::smem_u32(kbuf), 16, 1024, tc::SW_128B);
      const uint64_t b_s = tc::smem_desc(tc::smem_u32(qbuf), 16, 1024, tc::SW_128B);
      const uint64_t a_o = tc::smem_desc(tc::smem_u32(kbuf), KA_KCOL, 1024, tc::SW_128B);
      const uint64_t b_o = tc::smem_desc(tc::smem_u32(pbuf), 8192, 1024, tc::SW_128B);
      bool ok = true;
      uint32_t ph = 0;
      for (int64_t c = c_lo; c < c_hi; c++, ph ^= 1u) {
#pragma unroll
        for (int t = 0; t < 4; t++) {
          ok = ka_wait(&sm.kready[t], ph, sm, p.hdr, 41) && ok;
          tc::fence_after_sync();
          if (ok) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const uint32_t ka = (uint32_t)((2 * t + (i >> 2)) * KA_KCOL + (i & 3) * 32) >> 4;
              const uint32_t qa = (uint32_t)((2 * t + (i >> 2)) * KA_QCOL + (i & 3) * 32) >> 4;
              tc::mma_f16(tmem + KA_S_COL, a_s + ka, b_s + qa, idesc_s, (t || i) ? 1u : 0u);
            }
          }
        }
        tc::commit(&sm.s_full);
        ok = ka_wait(&sm.p_ready, ph, sm, p.hdr, 42) && ok;
        tc::fence_after_sync();
        const uint32_t add = c > c_lo ? 1u : 0u;
#pragma unroll
        for (int t = 0; t < 4; t++) {
          if (ok) {
#pragma unroll
            for (int ks = 0; ks < KA_KEYS / 16; ks++)
              tc::mma_f16(tmem + KA_O_COL + 64 * t, a_o + (uint32_t)((2 * t * KA_KCOL + ks * 2048) >> 4),
                          b_o + (uint32_t)(ks * 2048 >> 4), idesc_o, ks ? 1u : add);
          }
          tc::commit(&sm.pv_done[t]);
        }
      }
    }
    __syncwarp();
  } else if (warp >= KA_MATH_WARPS) {
    // ================= the key buffer
    const int ft = tid - 32 * KA_MATH_WARPS;
    const int key = ft >> 1, kh = ft & 1;             // entries: key row, 64-dim half of each tile
    const uint32_t xr = (uint32_t)key & 7u;
    const bool lead = ft == 0;
    bool ok = true;
    const int64_t c_rows = q.cw + q.cs;
    if (lead && c_lo < c_hi) {                        // Q, 8 column chunks of 64 heads
      for (int t = 0; t < 4; t++) {
        tc::bar_arrive_expect_tx(&sm.q_full[t], 2u * KA_QCOL);
        for (int c = 2 * t; c < 2 * t + 2; c++)
          tc::tma_load_2d(qbuf + c * KA_QCOL, &map_q, c * 64, (int32_t)(bq * H), &sm.q_full[t]);
      }
    }
    uint4 cd[8];                                      // FP4 codes of the next entry chunk: tile t in cd[2t], cd[2t+1]
    uint4 scv[2];                                     // its 32 scale bytes
    auto load_entries = [&](int64_t c) {
      const int64_t e = KA_KEYS * (c - c_rows) + key;
#pragma unroll
      for (int i = 0; i < 8; i++) cd[i] = make_uint4(0u, 0u, 0u, 0u);
      scv[0] = scv[1] = make_uint4(0u, 0u, 0u, 0u);
      if (e < q.en) {
        const uint4* s4 = reinterpret_cast<const uint4*>(p.main_kv + ((int64_t)b * p.cap + e) * MAIN_BYTES);
#pragma unroll
        for (int t = 0; t < 4; t++) {
          cd[2 * t] = __ldg(s4 + 4 * t + 2 * kh);
          cd[2 * t + 1] = __ldg(s4 + 4 * t + 2 * kh + 1);
        }
        scv[0] = __ldg(s4 + 16);
        scv[1] = __ldg(s4 + 17);
      }
    };
    auto dequant_tile = [&](int t) {
      const uint4 c0 = cd[2 * t], c1 = cd[2 * t + 1];
      const uint32_t cwd[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const uint4& sv = scv[t >> 1];
      const uint32_t sw = (t & 1) ? (kh ? sv.w : sv.z) : (kh ? sv.y : sv.x);
      unsigned char* dst = kbuf + (2 * t + kh) * KA_KCOL + key * 128;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        // the odd half walks its 16-channel groups as i ^ 2: the two threads of a key
        // then never store to the same 16-byte bank group in one instruction
        const int g = kh ? (i ^ 2) : i;
        const uint32_t wa = kh ? cwd[2 * (i ^ 2)] : cwd[2 * i];
        const uint32_t wb = kh ? cwd[2 * (i ^ 2) + 1] : cwd[2 * i + 1];
        const uint32_t sc2 = e4m3x2_to_f16x2(prmt(sw >> (8 * g), 0u, 0x0000u));
        uint32_t o[8];
        e2m1x8_to_f16(wa, o);
        e2m1x8_to_f16(wb, o + 4);
#pragma unroll
        for (int k = 0; k < 8; k++) o[k] = hmul2(o[k], sc2);
        *reinterpret_cast<uint4*>(dst + (((2u * g) ^ xr) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + (((2u * g + 1u) ^ xr) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    };
    // a tile of rows that the copy has brought: E4M3 widened, bf16 rounded to f16
    // when the operands are f16, rows outside [ra, rb) set to zero (a masked row
    // may hold anything, infinities among it)
    auto convert_rows = [&](int t, const KaRows& r) {
      unsigned char* kt = kbuf + 2 * t * KA_KCOL;
      if (p.rows_fp8) {
        const int row = ft >> 1, h = ft & 1;
        uint4 raw[2][2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const uint4* src = reinterpret_cast<const uint4*>(kt + i * KA_KCOL + KA_KCOL / 2 + row * 64 + h * 32);
          raw[i][0] = src[0];
          raw[i][1] = src[1];
        }
        named_sync(1, KA_FILL);
        const bool vis = row >= r.ra && row < r.rb;
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint4& w = raw[i][j >> 1];
            const uint32_t lo = (j & 1) ? w.z : w.x, hi = (j & 1) ? w.w : w.y;
            uint32_t o[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi),
                             e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
            for (int k = 0; k < 4; k++) o[k] = !vis ? 0u : (F16 ? o[k] : f16x2_to_bf16x2(o[k]));
            *reinterpret_cast<uint4*>(kt + i * KA_KCOL + sw128((uint32_t)row, (uint32_t)(64 * h + 16 * j))) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      } else if (F16 || r.ra > 0 || r.rb < KA_KEYS) {
#pragma unroll 4
        for (int i = ft; i < 2 * KA_KCOL / 16; i += KA_FILL) {
          uint4* u = reinterpret_cast<uint4*>(kt) + i;
          const int row = (i >> 3) & (KA_KEYS - 1);
          const bool vis = row >= r.ra && row < r.rb;
          if (!vis) *u = make_uint4(0u, 0u, 0u, 0u);
          else if (F16) {
            const uint4 x = *u;
            *u = make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
          }
        }
      }
    };
    if (F16 && c_lo < c_hi && c_lo >= c_rows) load_entries(c_lo);
    uint32_t ph = 0, rph = 0;
    for (int64_t c = c_lo; c < c_hi; c++, ph ^= 1u) {
      const bool rows = c < c_rows;
      KaRows r{0, 0, 0};
      if (rows) r = ka_rows(p, q, c, base);
      const bool fetch = rows && r.rb > r.ra;
#pragma unroll
      for (int t = 0; t < 4; t++) {
        if (c > c_lo) {
          ok = ka_wait(&sm.pv_done[t], ph ^ 1u, sm, p.hdr, 43) && ok;
          tc::fence_after_sync();
        }
        if (fetch && lead) {
          // the buffer was read by the tensor cores (their completion was waited for)
          // and written by ordinary stores before; the copy comes after both
          tc::fence_proxy_async_smem();
          const CUtensorMap* map = c < q.cw ? &map_rows : &map_sinks;
          const int64_t y = (int64_t)b * (c < q.cw ? (int64_t)p.S : (int64_t)p.n_sink) + r.first;
          tc::bar_arrive_expect_tx(&sm.row_full[t], p.rows_fp8 ? (uint32_t)KA_KCOL : 2u * KA_KCOL);
          for (int cc = 2 * t; cc < 2 * t + 2; cc++)
            tc::tma_load_2d(kbuf + cc * KA_KCOL + (p.rows_fp8 ? KA_KCOL / 2 : 0), map, cc * 64, (int32_t)y,
                            &sm.row_full[t]);
        }
        if (F16 && c == c_lo) {                       // Q's tile rounded to f16 in place
          ok = ka_wait(&sm.q_full[t], 0, sm, p.hdr, 44) && ok;
          uint4* qv = reinterpret_cast<uint4*>(qbuf + 2 * t * KA_QCOL);
#pragma unroll
          for (int i = ft; i < 2 * KA_QCOL / 16; i += KA_FILL) {
            const uint4 x = qv[i];
            qv[i] = make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
          }
        }
        if (!F16 && c == c_lo) ok = ka_wait(&sm.q_full[t], 0, sm, p.hdr, 44) && ok;
        if (!rows) {
          if (F16) dequant_tile(t);
        } else if (fetch) {
          ok = ka_wait(&sm.row_full[t], rph, sm, p.hdr, 45) && ok;
          convert_rows(t, r);
        } else {                                      // no row of the chunk was supplied
          for (int i = ft; i < 2 * KA_KCOL / 16; i += KA_FILL)
            reinterpret_cast<uint4*>(kbuf + 2 * t * KA_KCOL)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sm.kready[t]);
      }
      if (fetch) rph ^= 1u;
      if (F16 && c + 1 < c_hi && c + 1 >= c_rows) load_entries(c + 1);
    }
  } else {
    // ================= softmax and output
    const int q4 = warp & 3, hh = warp >> 2;          // TMEM lane quarter; head half (heads 32 hh ..)
    const int m = q4 * 32 + lane;                     // key row of a chunk / dim row of a tile
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float sc2 = p.scale * KA_LOG2E;
    float m_used = -INFINITY;                         // reference of head 32 hh + lane
    float l_part = 0.f;                               // sum of P over this warp's keys, head 32 hh + lane
    bool ok = true;
    uint32_t ph = 0;
    for (int64_t c = c_lo; c < c_hi; c++, ph ^= 1u) {
      bool valid;
      if (c < q.cw + q.cs) {
        const KaRows r = ka_rows(p, q, c, base);
        valid = m >= r.ra && m < r.rb;
      } else {
        valid = KA_KEYS * (c - q.cw - q.cs) + m < q.en;
      }
      ok = ka_wait(&sm.s_full, ph, sm, p.hdr, 46) && ok;
      tc::fence_after_sync();
      float v[32], r[32];
      {
        uint32_t s[32];
        tmem_ld32(tmem + lane_off + KA_S_COL + 32 * hh, s);
#pragma unroll
        for (int j = 0; j < 32; j++) r[j] = v[j] = valid ? __uint_as_float(s[j]) * sc2 : -INFINITY;
      }
      sm.red[warp][lane] = lane_columns<true>(r, lane);
      named_sync(2 + hh, 128);                        // the four warps of this head half
      const float cm = fmaxf(fmaxf(sm.red[4 * hh][lane], sm.red[4 * hh + 1][lane]),
                             fmaxf(sm.red[4 * hh + 2][lane], sm.red[4 * hh + 3][lane]));
      float alpha = 1.f;
      if (m_used == -INFINITY) {
        m_used = cm;                                  // O^T holds nothing yet, or only zeros
      } else if (cm > m_used + KA_TAU) {
        alpha = ex2_ftz(m_used - cm);
        m_used = cm;
        l_part *= alpha;
      }
      if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) {
        // the same decision in the four warps of the half; the chunk before is in
        // O^T entirely (this chunk's S^T needed its buffer)
        float al[32];
#pragma unroll
        for (int j = 0; j < 32; j++) al[j] = __shfl_sync(0xFFFFFFFFu, alpha, j);
#pragma unroll 1
        for (int u = 0; u < 4; u++) {
          uint32_t o[32];
          const uint32_t taddr = tmem + lane_off + KA_O_COL + 64 * u + 32 * hh;
          tmem_ld32(taddr, o);
#pragma unroll
          for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * al[j]);
          tmem_st32(taddr, o);
        }
        tc::tmem_wait_st();
      }
      sm.mv[warp][lane] = m_used;
      __syncwarp();
      uint32_t pk[16];
#pragma unroll
      for (int j4 = 0; j4 < 8; j4++) {
        const float4 m4 = *reinterpret_cast<const float4*>(&sm.mv[warp][4 * j4]);
        const float mj[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int j = 4 * j4 + e;
          r[j] = (v[j] == -INFINITY) ? 0.f : ex2_ftz(v[j] - mj[e]);
          if (j & 1) pk[j >> 1] = F16 ? pack_f16x2(r[j - 1], r[j]) : pack_bf16x2(r[j - 1], r[j]);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; u++)
        *reinterpret_cast<uint4*>(pbuf + sw128((uint32_t)m, (uint32_t)(hh * 64 + u * 16))) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sm.p_ready);
      l_part += lane_columns<false>(r, lane);         // beside the product, not before it
    }

    // ---------------- output
    if (c_lo < c_hi) {
      for (int t = 0; t < 4; t++) ok = ka_wait(&sm.pv_done[t], ph ^ 1u, sm, p.hdr, 47) && ok;
      tc::fence_after_sync();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    sm.red[warp][lane] = l_part;
    named_sync(2 + hh, 128);
    const float l = sm.red[4 * hh][lane] + sm.red[4 * hh + 1][lane] + sm.red[4 * hh + 2][lane] + sm.red[4 * hh + 3][lane];
    if (!SPLIT) {
      if (p.lse && q4 == 0)
        p.lse[bq * H + 32 * hh + lane] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * KA_LN2;
      const float inv = l == 0.f ? 0.f : 1.0f / l;    // no visible key: zeros
      uint16_t* out = p.out + bq * H * D + (int64_t)(32 * hh) * D + m;
#pragma unroll 1
      for (int u = 0; u < 4; u++) {
        uint32_t o[32];
        if (c_lo < c_hi) tmem_ld32(tmem + lane_off + KA_O_COL + 64 * u + 32 * hh, o);
#pragma unroll
        for (int j = 0; j < 32; j++) {
          const float i = __shfl_sync(0xFFFFFFFFu, inv, j);
          const float x = c_lo < c_hi ? __uint_as_float(o[j]) * i : 0.f;
          out[j * D + 128 * u] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xFFFFu);
        }
      }
    } else {
      float* part = p.part + (int64_t)blockIdx.x * KA_PART_FLOATS;
      if (q4 == 0) {
        part[32 * hh + lane] = m_used;
        part[H + 32 * hh + lane] = l;
      }
      float* op = part + 2 * H + (int64_t)(32 * hh) * D + m;
      if (c_lo < c_hi) {
#pragma unroll 1
        for (int u = 0; u < 4; u++) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_off + KA_O_COL + 64 * u + 32 * hh, o);
#pragma unroll
          for (int j = 0; j < 32; j++) op[j * D + 128 * u] = __uint_as_float(o[j]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == KA_MMA_WARP) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, KA_TMEM_COLS);
  }
}

// One query's output from its CTAs' partial states: with m = max_s m_s and
// w_s = 2^(m_s - m), O = sum_s w_s O_s / sum_s w_s l_s.  One warp per (head,
// half of the dims); the weights of 32 states at a time lie in the lanes.
__global__ void __launch_bounds__(256) keys_combine_kernel(const float* __restrict__ part, int split,
                                                           uint16_t* __restrict__ out, float* __restrict__ lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t bq = blockIdx.x >> 4;
  const int h = (blockIdx.x & 15) * 4 + (threadIdx.x >> 6), d0 = ((threadIdx.x >> 5) & 1) * (D / 2) + 4 * lane;
  const float* pb = part + bq * split * KA_PART_FLOATS;
  float mx = -INFINITY;
  for (int s = lane; s < split; s += 32) mx = fmaxf(mx, pb[(int64_t)s * KA_PART_FLOATS + h]);
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
  float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float L = 0.f;
  for (int s0 = 0; s0 < split; s0 += 32) {
    float w = 0.f;
    if (s0 + lane < split) {
      const float* ps = pb + (int64_t)(s0 + lane) * KA_PART_FLOATS;
      const float l = ps[H + h];
      if (l != 0.f) {                                 // a state that saw a key
        w = exp2f(ps[h] - mx);
        L += w * l;
      }
    }
    const int n = min(32, split - s0);
#pragma unroll 4
    for (int i = 0; i < n; i++) {
      const float wi = __shfl_sync(0xFFFFFFFFu, w, i);
      const float* o = pb + (int64_t)(s0 + i) * KA_PART_FLOATS + 2 * H + h * D + d0;
      if (wi != 0.f) {                                // a state without keys holds no O
        const float4 x = *reinterpret_cast<const float4*>(o), y = *reinterpret_cast<const float4*>(o + 128);
        a[0] += wi * x.x;
        a[1] += wi * x.y;
        a[2] += wi * x.z;
        a[3] += wi * x.w;
        a[4] += wi * y.x;
        a[5] += wi * y.y;
        a[6] += wi * y.z;
        a[7] += wi * y.w;
      }
    }
  }
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, k);
  const float inv = L == 0.f ? 0.f : 1.0f / L;        // no visible key: zeros
  if (lse && (threadIdx.x & 63) == 0) lse[bq * H + h] = L == 0.f ? -INFINITY : (mx + log2f(L)) * KA_LN2;
  uint16_t* o = out + (bq * H + h) * D + d0;
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
  *reinterpret_cast<uint2*>(o + 128) = make_uint2(pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
}

// ------------------------------------------------------------------ host side
// CTAs per query: the number whose time, in chunks, is least.  A CTA costs its
// chunks and about KA_FIXED more (set-up, the first keys, the output), a split
// call KA_JOIN more; CTAs run one to an SM.  The GPU's 152 SMs are a constant
// here so that the workspace can be sized without a device.
constexpr int KA_SMS = 152;
constexpr int KA_FIXED = 3, KA_JOIN = 3;

int keys_split(int64_t BQ, int64_t chunks) {
  if (BQ <= 0 || BQ >= 4 * KA_SMS) return 1;
  int best = 1;
  int64_t best_cost = ceil_div(BQ, KA_SMS) * (KA_FIXED + chunks);
  for (int s = 2; s <= KA_SMS && s <= chunks; s++) {
    const int64_t cost = ceil_div(BQ * s, KA_SMS) * (KA_FIXED + ceil_div(chunks, s)) + KA_JOIN;
    if (cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

size_t keys_part_bytes(int64_t BQ, int64_t chunks) {
  const int s = keys_split(BQ, chunks);
  return s > 1 ? (size_t)(BQ * s) * KA_PART_FLOATS * sizeof(float) : 0;
}

template <bool F16>
static cudaError_t keys_launch(const KeysParams& p, int64_t BQ, const CUtensorMap& mq, const CUtensorMap& mr,
                               const CUtensorMap& ms, cudaStream_t stream) {
  static PerDeviceOnce attrs;
  cudaError_t e = attrs.ensure([](int) {
    cudaError_t r = cudaFuncSetAttribute(keys_attn_kernel<F16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, KA_SMEM);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(keys_attn_kernel<F16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, KA_SMEM);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(BQ * p.split));
  cfg.blockDim = dim3(KA_THREADS);
  cfg.dynamicSmemBytes = KA_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set-up overlaps the previous kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = p.split > 1 ? cudaLaunchKernelEx(&cfg, keys_attn_kernel<F16, true>, p, mq, mr, ms)
                  : cudaLaunchKernelEx(&cfg, keys_attn_kernel<F16, false>, p, mq, mr, ms);
  if (e != cudaSuccess || p.split == 1) return e;
  cudaLaunchConfig_t cc = {};
  cc.gridDim = dim3((unsigned)(BQ * 16));
  cc.blockDim = dim3(256);
  cc.stream = stream;
  cc.attrs = attr;
  cc.numAttrs = 1;
  return cudaLaunchKernelEx(&cc, keys_combine_kernel, (const float*)p.part, p.split, p.out, p.lse);
}

cudaError_t launch_keys_attention(KeysParams p, int B, int64_t chunks, void* part, cudaStream_t stream) {
  const int64_t BQ = (int64_t)B * p.Q;
  if (BQ == 0) return cudaSuccess;
  p.split = keys_split(BQ, chunks);
  p.part = reinterpret_cast<float*>(part);
  CUtensorMap mq, mr, ms;
  if (!encode_bf16_rows512(&mq, p.q, (uint64_t)BQ * H, H)) return cudaErrorInvalidValue;
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
  return p.main_kv ? keys_launch<true>(p, BQ, mq, mr, ms, stream) : keys_launch<false>(p, BQ, mq, mr, ms, stream);
}

}  // namespace csa2
