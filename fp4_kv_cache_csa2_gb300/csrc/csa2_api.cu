// C ABI of the CSA2 layer: argument checks, workspace carving and launches.
// The operations themselves are defined in include/csa2.h.
#include <cmath>
#include <cstring>
#include <thread>
#include <vector>

#include "common.cuh"
#include "host_once.cuh"
#include "params.cuh"

using namespace csa2;

namespace {

constexpr size_t HDR = CSA2_WS_HEADER_BYTES;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned8(const void* p) { return ((uintptr_t)p & 7u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// [a, a + an) and [b, b + bn) share a byte
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// what a call that reads no index key needs of a cache
csa2_status check_cache_entries(const csa2_cache* c) {
  if (!c || !c->main_kv || !c->n_entries) return CSA2_ERR_INVALID_ARG;
  if (c->cap < 0 || (c->cap % BLK) != 0) return CSA2_ERR_INVALID_ARG;
  if (c->m != 1 && c->m != 2) return CSA2_ERR_UNSUPPORTED;
  return aligned16(c->main_kv) ? CSA2_OK : CSA2_ERR_INVALID_ARG;
}

csa2_status check_cache(const csa2_cache* c) {
  if (!c || !c->idx_codes || !c->idx_scales) return CSA2_ERR_INVALID_ARG;
  const csa2_status st = check_cache_entries(c);
  if (st != CSA2_OK) return st;
  return aligned16(c->idx_codes) && aligned16(c->idx_scales) ? CSA2_OK : CSA2_ERR_INVALID_ARG;
}

csa2_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return CSA2_ERR_WORKSPACE;
  if (((uintptr_t)ws & 255u) != 0) return CSA2_ERR_INVALID_ARG;
  if (ws_bytes < need) return CSA2_ERR_WORKSPACE;
  return CSA2_OK;
}

csa2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

WsHeader* header(void* ws) { return reinterpret_cast<WsHeader*>(ws); }
unsigned char* scratch(void* ws) { return reinterpret_cast<unsigned char*>(ws) + HDR; }

size_t gkeys_bytes(int B, int Q, int64_t max_n) {
  return align256((size_t)B * Q * (size_t)ceil_div(max_n, BLK) * sizeof(uint32_t));
}

bool long_rows(int64_t max_n) { return max_n > ROW_SELECT_MIN_KEYS; }

// scratch of the Full selections: per-row histograms and lists for long rows,
// block-maximum keys otherwise
size_t select_scratch_bytes(int B, int Q, int64_t max_n, bool blocks) {
  if (long_rows(max_n)) return align256(row_select_bytes((int64_t)B * Q));
  return blocks ? gkeys_bytes(B, Q, max_n) : 0;
}

// B * Q queries per call at most: every grid stays a 1-D grid below 2^31 CTAs
constexpr int64_t MAX_QUERIES = (int64_t)1 << 26;

csa2_status check_q(int B, int Q) {
  if (B < 0 || Q < 0) return CSA2_ERR_INVALID_ARG;
  if ((int64_t)B * Q > MAX_QUERIES) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

// ---------------------------------------------------------------- the calls
csa2_status do_index_score(const csa2_cache* cache, const uint16_t* q_idx, const float* w_head,
                           const int64_t* q_pos, const int32_t* pool, int M, float* scores, int B, int Q,
                           int64_t max_n, WsHeader* hdr, cudaStream_t stream) {
  IsParams p{};
  p.idx_codes = cache->idx_codes;
  p.idx_scales = cache->idx_scales;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.m = cache->m;
  p.q_idx = q_idx;
  p.w_head = w_head;
  p.q_pos = q_pos;
  p.pool = pool;
  p.M = M;
  p.scores = scores;
  p.B = B;
  p.Q = Q;
  p.max_n = max_n;
  p.hdr = hdr;
  return from_cuda(launch_index_score(p, stream));
}

csa2_status do_attention(const csa2_cache* cache, const uint16_t* q, const int32_t* sel, int K,
                         const uint16_t* swa, const int64_t* swa_base, int S, const int64_t* q_pos, float scale,
                         uint16_t* out, int B, int Q, void* part_ws, WsHeader* hdr, cudaStream_t stream,
                         const uint8_t* packed_in = nullptr, uint8_t* packed_out = nullptr, bool swa_fp8 = false,
                         int split = 1) {
  AttnParams p{};
  p.main_kv = cache->main_kv;
  p.cap = cache->cap;
  p.q = q;
  p.sel = sel;
  p.K = K;
  p.swa = swa;
  p.swa_base = swa_base;
  p.S = S;
  p.swa_fp8 = swa_fp8 ? 1 : 0;
  p.q_pos = q_pos;
  p.scale = scale;
  p.out = out;
  p.Q = Q;
  p.hdr = hdr;
  p.packed_in = packed_in;
  p.packed_out = packed_out;
  p.split = split;
  return from_cuda(launch_attention(p, B, reinterpret_cast<float*>(part_ws), stream));
}

}  // namespace

extern "C" {

int csa2_layout_version(void) { return CSA2_LAYOUT_VERSION; }

const char* csa2_status_string(csa2_status s) {
  switch (s) {
    case CSA2_OK: return "CSA2_OK";
    case CSA2_ERR_INVALID_ARG: return "CSA2_ERR_INVALID_ARG";
    case CSA2_ERR_UNSUPPORTED: return "CSA2_ERR_UNSUPPORTED";
    case CSA2_ERR_WORKSPACE: return "CSA2_ERR_WORKSPACE";
    case CSA2_ERR_CUDA: return "CSA2_ERR_CUDA";
    case CSA2_ERR_TIMEOUT: return "CSA2_ERR_TIMEOUT";
    case CSA2_ERR_BOUNDS: return "CSA2_ERR_BOUNDS";
  }
  return "CSA2_ERR_UNKNOWN";
}

csa2_status csa2_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  csa2_status st = check_ws(ws, ws_bytes, HDR);
  if (st != CSA2_OK) return st;
  return from_cuda(cudaMemsetAsync(ws, 0, HDR, (cudaStream_t)stream));
}

csa2_status csa2_sync_status(void* ws, void* stream, int64_t* detail) {
  if (!ws) return CSA2_ERR_WORKSPACE;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return CSA2_ERR_CUDA;
  WsHeader h;
  if (cudaMemcpy(&h, ws, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess) return CSA2_ERR_CUDA;
  if (detail) *detail = (int64_t)h.detail;
  if (h.status != 0) {
    if (cudaMemset(ws, 0, HDR) != cudaSuccess) return CSA2_ERR_CUDA;
  }
  return (csa2_status)h.status;
}

csa2_status csa2_rope_table(float* cs, int64_t P, double theta) {
  if (!cs || P < 0) return CSA2_ERR_INVALID_ARG;
  double inv_freq[32];
  for (int i = 0; i < 32; i++) inv_freq[i] = std::pow(theta, -(double)(2 * i) / 64.0);
  unsigned nt = std::thread::hardware_concurrency();
  if (nt == 0) nt = 1;
  if (nt > 32) nt = 32;
  if (P < 65536) nt = 1;
  auto work = [&](int64_t p0, int64_t p1) {
    for (int64_t p = p0; p < p1; p++)
      for (int i = 0; i < 32; i++) {
        double ang = (double)p * inv_freq[i];
        cs[(p * 32 + i) * 2 + 0] = (float)std::cos(ang);
        cs[(p * 32 + i) * 2 + 1] = (float)std::sin(ang);
      }
  };
  std::vector<std::thread> th;
  int64_t per = (P + nt - 1) / nt;
  for (unsigned k = 0; k < nt; k++) {
    int64_t a = k * per, b = std::min<int64_t>(P, a + per);
    if (a >= b) break;
    th.emplace_back(work, a, b);
  }
  for (auto& x : th) x.join();
  return CSA2_OK;
}

csa2_status csa2_compress_quantize(const csa2_cache* cache, const uint16_t* x, int B, int T,
                                   const int64_t* entry_start, const float* w0, const float* w1,
                                   const float* rope_cs, int64_t rope_P, const uint16_t* w_idx, void* ws,
                                   size_t ws_bytes, void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if (B < 0 || T < 0 || rope_P < 0) return CSA2_ERR_INVALID_ARG;
  if (T % cache->m != 0) return CSA2_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return check_ws(ws, ws_bytes, HDR);
  if (!x || !entry_start || !rope_cs || !w_idx) return CSA2_ERR_INVALID_ARG;
  if (cache->m == 2 && (!w0 || !w1)) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(rope_cs) || !aligned16(w_idx)) return CSA2_ERR_INVALID_ARG;
  if (cache->m == 2 && (!aligned16(w0) || !aligned16(w1))) return CSA2_ERR_INVALID_ARG;
  st = check_ws(ws, ws_bytes, HDR);
  if (st != CSA2_OK) return st;
  CwParams p{};
  p.main_kv = cache->main_kv;
  p.idx_codes = cache->idx_codes;
  p.idx_scales = cache->idx_scales;
  p.cap = cache->cap;
  p.m = cache->m;
  p.x = x;
  p.B = B;
  p.T = T;
  p.entry_start = entry_start;
  p.w0 = w0;
  p.w1 = w1;
  p.rope_cs = rope_cs;
  p.rope_P = rope_P;
  p.w_idx = w_idx;
  p.hdr = header(ws);
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return CSA2_ERR_CUDA;
  return from_cuda(launch_cache_write(p, (cudaStream_t)stream, sms));
}

csa2_status csa2_index_score(const csa2_cache* cache, const uint16_t* q_idx, const float* w_head,
                             const int64_t* q_pos, const int32_t* pool_blocks, int M, float* scores, int B, int Q,
                             int64_t max_n, void* ws, size_t ws_bytes, void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if ((st = check_q(B, Q)) != CSA2_OK) return st;
  if (max_n < 0) return CSA2_ERR_INVALID_ARG;
  if (pool_blocks && (M < 1 || M > CSA2_MAX_M)) return CSA2_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, HDR)) != CSA2_OK) return st;
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!q_idx || !w_head || !q_pos || !scores) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(q_idx)) return CSA2_ERR_INVALID_ARG;
  return do_index_score(cache, q_idx, w_head, q_pos, pool_blocks, M, scores, B, Q, max_n, header(ws),
                        (cudaStream_t)stream);
}

size_t csa2_block_topk_workspace_size(int B, int Q, int64_t max_n) {
  if (B < 0 || Q < 0 || max_n < 0) return 0;
  return HDR + select_scratch_bytes(B, Q, max_n, true);
}

csa2_status csa2_block_topk(const csa2_cache* cache, const float* scores, const int64_t* q_pos, int B, int Q,
                            int64_t max_n, int M, int32_t* pool_blocks, void* ws, size_t ws_bytes, void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if ((st = check_q(B, Q)) != CSA2_OK) return st;
  if (max_n < 0) return CSA2_ERR_INVALID_ARG;
  if (M < 1 || M > CSA2_MAX_M) return CSA2_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, csa2_block_topk_workspace_size(B, Q, max_n))) != CSA2_OK) return st;
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!scores || !q_pos || !pool_blocks) return CSA2_ERR_INVALID_ARG;
  if (long_rows(max_n))
    return from_cuda(launch_row_select(scores, q_pos, cache->n_entries, cache->m, B, Q, max_n, 0, nullptr, M,
                                       pool_blocks, scratch(ws), (cudaStream_t)stream));
  return from_cuda(launch_block_topk(scores, q_pos, cache->n_entries, cache->m, B, Q, max_n, M, pool_blocks,
                                     reinterpret_cast<uint32_t*>(scratch(ws)), (cudaStream_t)stream));
}

size_t csa2_select_topk_workspace_size(int B, int Q, int64_t max_n) {
  if (B < 0 || Q < 0 || max_n < 0) return 0;
  return HDR + select_scratch_bytes(B, Q, max_n, false);
}

csa2_status csa2_select_topk(const csa2_cache* cache, const float* scores, const int64_t* q_pos,
                             const int32_t* pool_blocks, int M, int K, int32_t* sel, int B, int Q, int64_t max_n,
                             void* ws, size_t ws_bytes, void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if ((st = check_q(B, Q)) != CSA2_OK) return st;
  if (max_n < 0) return CSA2_ERR_INVALID_ARG;
  if (K < 1 || K > CSA2_MAX_K) return CSA2_ERR_UNSUPPORTED;
  if (pool_blocks && (M < 1 || M > CSA2_MAX_M)) return CSA2_ERR_UNSUPPORTED;
  const size_t need = pool_blocks ? HDR : csa2_select_topk_workspace_size(B, Q, max_n);
  if ((st = check_ws(ws, ws_bytes, need)) != CSA2_OK) return st;
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!scores || !q_pos || !sel) return CSA2_ERR_INVALID_ARG;
  if (!pool_blocks && long_rows(max_n))
    return from_cuda(launch_row_select(scores, q_pos, cache->n_entries, cache->m, B, Q, max_n, K, sel, 0, nullptr,
                                       scratch(ws), (cudaStream_t)stream));
  return from_cuda(launch_select_topk(scores, q_pos, cache->n_entries, cache->m, pool_blocks, M, K, sel, B, Q,
                                      max_n, (cudaStream_t)stream));
}

csa2_status csa2_swa_quantize_fp8(const uint16_t* x, int64_t n_rows, uint8_t* out, void* stream) {
  if (n_rows < 0) return CSA2_ERR_INVALID_ARG;
  if (n_rows == 0) return CSA2_OK;
  if (!x || !out || !aligned16(x) || !aligned16(out)) return CSA2_ERR_INVALID_ARG;
  return from_cuda(launch_swa_fp8(x, n_rows, out, (cudaStream_t)stream));
}

size_t csa2_attn_workspace_size(int B, int Q, int K) {
  if (B < 0 || Q < 0 || K < 0) return 0;
  return HDR + align256(attn_partials_bytes((int64_t)B * Q, K));
}

csa2_status csa2_sparse_swa_attn(const csa2_cache* cache, const uint16_t* q, const int32_t* sel, int K,
                                 const uint16_t* swa, const int64_t* swa_base_pos, int S, const int64_t* q_pos,
                                 float scale, uint16_t* out, int B, int Q, void* ws, size_t ws_bytes,
                                 void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if ((st = check_q(B, Q)) != CSA2_OK) return st;
  if (K < 0 || K > CSA2_MAX_K) return CSA2_ERR_UNSUPPORTED;
  if (S < 0 || !std::isfinite(scale)) return CSA2_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, csa2_attn_workspace_size(B, Q, K))) != CSA2_OK) return st;
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!q || (K > 0 && !sel) || !swa || !swa_base_pos || !q_pos || !out) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(swa) || !aligned16(out)) return CSA2_ERR_INVALID_ARG;
  return do_attention(cache, q, sel, K, swa, swa_base_pos, S, q_pos, scale, out, B, Q, scratch(ws), header(ws),
                      (cudaStream_t)stream);
}

csa2_status csa2_block_summary(const csa2_cache* cache, const int64_t* first_block, int64_t n_blocks, int B,
                               uint8_t* sum_codes, uint8_t* sum_scales, int64_t sum_cap, void* ws, size_t ws_bytes,
                               void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if (B < 0 || n_blocks < 0 || sum_cap < 0) return CSA2_ERR_INVALID_ARG;
  if ((sum_cap % BLK) != 0) return CSA2_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, HDR)) != CSA2_OK) return st;
  if (B == 0 || n_blocks == 0) return CSA2_OK;
  if (!first_block || !sum_codes || !sum_scales) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(sum_codes) || !aligned16(sum_scales)) return CSA2_ERR_INVALID_ARG;
  HsParams p{};
  p.idx_codes = cache->idx_codes;
  p.idx_scales = cache->idx_scales;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.first_block = first_block;
  p.B = B;
  p.n_blocks = n_blocks;
  p.sum_codes = sum_codes;
  p.sum_scales = sum_scales;
  p.sum_cap = sum_cap;
  p.hdr = header(ws);
  return from_cuda(launch_block_summary(p, (cudaStream_t)stream));
}

csa2_status csa2_qk_norm_rope(const csa2_qk_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return CSA2_ERR_INVALID_ARG;
  if (a->T < 0 || a->rope_P < 0 || a->n_rows < 0) return CSA2_ERR_INVALID_ARG;
  if (a->T > MAX_QUERIES || a->n_rows > ((int64_t)1 << 40)) return CSA2_ERR_UNSUPPORTED;
  if (!std::isfinite(a->eps) || a->eps < 0.f) return CSA2_ERR_INVALID_ARG;
  if (a->rows_fp8 != 0 && a->rows_fp8 != 1) return CSA2_ERR_INVALID_ARG;
  csa2_status st = check_ws(ws, ws_bytes, HDR);
  if (st != CSA2_OK) return st;
  if (a->T == 0 || (!a->q && !a->k)) return CSA2_OK;
  if (!a->pos || !aligned8(a->pos) || !a->rope_cs || !aligned16(a->rope_cs)) return CSA2_ERR_INVALID_ARG;
  const int64_t max_stride = (int64_t)1 << 32;
  int64_t q_bytes = 0, k_bytes = 0, out_bytes = 0, row_bytes = 0;
  if (a->q) {
    if (!a->q_out || !aligned16(a->q) || !aligned16(a->q_out)) return CSA2_ERR_INVALID_ARG;
    if (a->q_weight && !aligned16(a->q_weight)) return CSA2_ERR_INVALID_ARG;
    if (a->q_stride < H * D || a->q_stride > max_stride || a->q_stride % 8 != 0) return CSA2_ERR_INVALID_ARG;
    q_bytes = ((a->T - 1) * a->q_stride + H * D) * 2;
    out_bytes = a->T * H * D * 2;
  }
  if (a->k) {
    if (!a->rows || !aligned16(a->k) || !aligned16(a->rows)) return CSA2_ERR_INVALID_ARG;
    if (a->k_weight && !aligned16(a->k_weight)) return CSA2_ERR_INVALID_ARG;
    if (a->k_slot && !aligned8(a->k_slot)) return CSA2_ERR_INVALID_ARG;
    if (a->k_stride < D || a->k_stride > max_stride || a->k_stride % 8 != 0) return CSA2_ERR_INVALID_ARG;
    k_bytes = ((a->T - 1) * a->k_stride + D) * 2;
    row_bytes = a->n_rows * D * (a->rows_fp8 ? 1 : 2);
  }
  const bool in_place = a->q && a->q_out == a->q && a->q_stride == H * D;
  if (!in_place && overlap(a->q, q_bytes, a->q_out, out_bytes)) return CSA2_ERR_INVALID_ARG;
  if (overlap(a->k, k_bytes, a->rows, row_bytes) || overlap(a->k, k_bytes, a->q_out, out_bytes) ||
      overlap(a->q, q_bytes, a->rows, row_bytes) || overlap(a->q_out, out_bytes, a->rows, row_bytes))
    return CSA2_ERR_INVALID_ARG;
  const int64_t weight = D * 4, table = a->rope_P < ((int64_t)1 << 48) ? a->rope_P * D_ROPE * 4 : INT64_MAX / 2;
  const struct { const void* a; int64_t n; } in[] = {{a->pos, a->T * 8}, {a->rope_cs, table}, {ws, (int64_t)HDR},
      {a->q_weight, a->q && a->q_weight ? weight : 0}, {a->k_weight, a->k && a->k_weight ? weight : 0},
      {a->k_slot, a->k && a->k_slot ? a->T * 8 : 0}};
  for (const auto& x : in)
    if (overlap(x.a, x.n, a->q_out, out_bytes) || overlap(x.a, x.n, a->rows, row_bytes)) return CSA2_ERR_INVALID_ARG;
  QkParams p{};
  p.T = a->T;
  p.pos = a->pos;
  p.rope_cs = a->rope_cs;
  p.rope_P = a->rope_P;
  p.eps = a->eps;
  p.q = a->q;
  p.q_stride = a->q_stride;
  p.q_weight = a->q_weight;
  p.q_out = a->q_out;
  p.k = a->k;
  p.k_stride = a->k_stride;
  p.k_weight = a->k_weight;
  p.rows = static_cast<uint8_t*>(a->rows);
  p.n_rows = a->n_rows;
  p.k_slot = a->k_slot;
  p.rows_fp8 = a->rows_fp8;
  p.hdr = header(ws);
  return from_cuda(launch_qk_norm_rope(p, (cudaStream_t)stream));
}

// The attentions over every visible key: their queries, rows and outputs.
constexpr int64_t MAX_KEY_QUERIES = (int64_t)1 << 24;   // 64 rows each below 2^31 (tensor-map coordinates)

static csa2_status check_keys_call(const KeysParams& p, int B, int Q, size_t need, void* ws, size_t ws_bytes) {
  const bool rows = p.W > 0;                          // (an 8-bit cache may be attended without a window)
  if (B < 0 || Q < 0 || p.S < 0 || p.n_sink < 0 || p.W < (p.scales8 ? 0 : 1) || !std::isfinite(p.scale))
    return CSA2_ERR_INVALID_ARG;
  if (p.rows_fp8 != 0 && p.rows_fp8 != 1) return CSA2_ERR_INVALID_ARG;
  const int64_t BQ = (int64_t)B * Q, nr = B * p.S, nk = (int64_t)B * p.n_sink, lim = (int64_t)1 << 31;
  if (BQ > MAX_KEY_QUERIES || nr >= lim || nk >= lim) return CSA2_ERR_UNSUPPORTED;
  csa2_status st = check_ws(ws, ws_bytes, need);
  if (st != CSA2_OK || BQ == 0) return st;
  if (!p.q || !p.q_pos || (rows && !p.base_pos) || !p.out || (nr > 0 && !p.rows) || (nk > 0 && !p.sinks))
    return CSA2_ERR_INVALID_ARG;
  if (!aligned16(p.q) || !aligned16(p.rows) || !aligned16(p.sinks) || !aligned16(p.out) || !aligned8(p.q_pos) ||
      !aligned8(p.base_pos) || ((uintptr_t)p.lse & 3u) != 0)
    return CSA2_ERR_INVALID_ARG;
  const int64_t row = D * (p.rows_fp8 ? 1 : 2), out_n = BQ * H * D * 2, lse_n = p.lse ? BQ * H * 4 : 0;
  const struct { const void* a; int64_t n; } in[] = {{p.q, out_n}, {p.q_pos, BQ * 8}, {p.base_pos, rows ? (int64_t)B * 8 : 0},
      {p.rows, nr * row}, {p.sinks, nk * row}, {ws, (int64_t)need},
      {p.main_kv, p.main_kv ? B * p.cap * (p.scales8 ? D : MAIN_BYTES) : 0},
      {p.scales8, p.scales8 ? B * (p.cap / BLK) * 4 : 0}, {p.n_entries, p.n_entries ? (int64_t)B * 4 : 0}};
  for (const auto& x : in)
    if (overlap(x.a, x.n, p.out, out_n) || overlap(x.a, x.n, p.lse, lse_n)) return CSA2_ERR_INVALID_ARG;
  return overlap(p.out, out_n, p.lse, lse_n) ? CSA2_ERR_INVALID_ARG : CSA2_OK;
}

// runs of keys that a query of a window call / a dense call sees at most
static int64_t window_chunks(int64_t W, int64_t n_sink) { return ceil_div(W, KEYS_CHUNK) + ceil_div(n_sink, KEYS_CHUNK); }
static int64_t dense_chunks(int64_t max_n) {
  const int64_t most = INT32_MAX;                     // n_entries is 32 bits: no query sees more
  return WIN / KEYS_CHUNK + ceil_div(max_n < most ? max_n : most, KEYS_CHUNK);
}

size_t csa2_window_attn_workspace_size(int B, int Q, int W, int n_sink) {
  if (B < 0 || Q < 0 || W < 1 || n_sink < 0 || (int64_t)B * Q > MAX_KEY_QUERIES) return 0;
  return HDR + align256(keys_part_bytes((int64_t)B * Q, window_chunks(W, n_sink)));
}

csa2_status csa2_window_attn(const csa2_window_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (!a) return CSA2_ERR_INVALID_ARG;
  KeysParams p{};
  p.q = a->q;
  p.q_pos = a->q_pos;
  p.Q = a->Q;
  p.rows = static_cast<const uint8_t*>(a->rows);
  p.base_pos = a->swa_base_pos;
  p.S = a->S;
  p.sinks = static_cast<const uint8_t*>(a->sinks);
  p.n_sink = a->n_sink;
  p.rows_fp8 = a->rows_fp8;
  p.W = a->W;
  p.scale = a->scale;
  p.out = a->out;
  p.lse = a->lse;
  const csa2_status st = check_keys_call(p, a->B, a->Q, csa2_window_attn_workspace_size(a->B, a->Q, a->W, a->n_sink),
                                         ws, ws_bytes);
  if (st != CSA2_OK || a->B == 0 || a->Q == 0) return st;
  p.hdr = header(ws);
  return from_cuda(launch_keys_attention(p, a->B, window_chunks(a->W, a->n_sink), scratch(ws), (cudaStream_t)stream));
}

size_t csa2_dense_attn_workspace_size(int B, int Q, int64_t max_n) {
  if (B < 0 || Q < 0 || max_n < 0 || (int64_t)B * Q > MAX_KEY_QUERIES) return 0;
  return HDR + align256(keys_part_bytes((int64_t)B * Q, dense_chunks(max_n)));
}

csa2_status csa2_dense_attn(const csa2_cache* cache, const csa2_dense_args* a, void* ws, size_t ws_bytes,
                            void* stream) {
  csa2_status st = check_cache_entries(cache);
  if (st != CSA2_OK) return st;
  if (!a || a->max_n < 0 || ((uintptr_t)cache->n_entries & 3u) != 0) return CSA2_ERR_INVALID_ARG;
  KeysParams p{};
  p.q = a->q;
  p.q_pos = a->q_pos;
  p.Q = a->Q;
  p.rows = static_cast<const uint8_t*>(a->swa);
  p.base_pos = a->swa_base_pos;
  p.S = a->S;
  p.rows_fp8 = a->swa_fp8;
  p.W = WIN;
  p.main_kv = cache->main_kv;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.m = cache->m;
  p.scale = a->scale;
  p.out = a->out;
  p.lse = a->lse;
  st = check_keys_call(p, a->B, a->Q, csa2_dense_attn_workspace_size(a->B, a->Q, a->max_n), ws, ws_bytes);
  if (st != CSA2_OK || a->B == 0 || a->Q == 0) return st;
  p.hdr = header(ws);
  return from_cuda(launch_keys_attention(p, a->B, dense_chunks(a->max_n), scratch(ws), (cudaStream_t)stream));
}

// ---------------------------------------------------------------- the 8-bit cache
static csa2_status check_cache8(const csa2_cache8* c, int B) {
  if (!c || !c->codes || !c->scales || !c->n_entries || B < 0) return CSA2_ERR_INVALID_ARG;
  if (c->cap < 0 || c->cap % BLK != 0) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(c->codes) || !aligned4(c->scales) || !aligned4(c->n_entries)) return CSA2_ERR_INVALID_ARG;
  if (c->m != 1 && c->m != 2) return CSA2_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 31;
  return c->cap < lim && B * c->cap < lim ? CSA2_OK : CSA2_ERR_UNSUPPORTED;
}

csa2_status csa2_cache8_write(const csa2_cache8* cache, const csa2_cache8_write_args* a, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!a) return CSA2_ERR_INVALID_ARG;
  csa2_status st = check_cache8(cache, a->B);
  if (st != CSA2_OK) return st;
  if ((st = check_q(a->B, a->T)) != CSA2_OK) return st;
  if ((st = check_ws(ws, ws_bytes, HDR)) != CSA2_OK || a->B == 0 || a->T == 0) return st;
  if (!a->x || !aligned16(a->x) || !a->entry_start || !aligned8(a->entry_start) || !aligned4(a->n_new))
    return CSA2_ERR_INVALID_ARG;
  if (a->x_stride < D || a->x_stride > ((int64_t)1 << 32) || a->x_stride % 8 != 0) return CSA2_ERR_INVALID_ARG;
  const int64_t n = (int64_t)a->B * cache->cap, scale_n = n / BLK * 4;
  const struct { const void* a; int64_t n; } in[] = {
      {a->x, (((int64_t)a->B * a->T - 1) * a->x_stride + D) * 2}, {a->entry_start, (int64_t)a->B * 8},
      {a->n_new, a->n_new ? (int64_t)a->B * 4 : 0}, {cache->n_entries, (int64_t)a->B * 4}, {ws, (int64_t)HDR}};
  for (const auto& x : in)
    if (overlap(x.a, x.n, cache->codes, n * D) || overlap(x.a, x.n, cache->scales, scale_n)) return CSA2_ERR_INVALID_ARG;
  if (overlap(cache->codes, n * D, cache->scales, scale_n)) return CSA2_ERR_INVALID_ARG;
  C8WriteParams p{};
  p.codes = reinterpret_cast<uint8_t*>(cache->codes);
  p.scales = cache->scales;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.x = a->x;
  p.x_stride = a->x_stride;
  p.B = a->B;
  p.T = a->T;
  p.start = a->entry_start;
  p.n_new = a->n_new;
  p.hdr = header(ws);
  return from_cuda(launch_cache8_write(p, (cudaStream_t)stream));
}

static int64_t cache8_chunks(int64_t max_n, int W) {
  return dense_chunks(max_n) - WIN / KEYS_CHUNK + ceil_div(W, KEYS_CHUNK);
}

size_t csa2_cache8_attn_workspace_size(int B, int Q, int64_t max_n, int W) {
  if (B < 0 || Q < 0 || max_n < 0 || W < 0 || (int64_t)B * Q > MAX_KEY_QUERIES) return 0;
  return HDR + align256(cache8_part_bytes(B, Q, cache8_chunks(max_n, W)));
}

int csa2_test_cache8_attn_plan(int B, int Q, int64_t max_n, int W, int* split) {
  if (B < 0 || Q < 0 || max_n < 0 || W < 0 || (int64_t)B * Q > MAX_KEY_QUERIES || !split) return -1;
  const Cache8Plan plan = cache8_plan(B, Q, cache8_chunks(max_n, W));
  *split = plan.split;
  return plan.pairs ? 1 : 0;
}

csa2_status csa2_cache8_attn(const csa2_cache8* cache, const csa2_cache8_attn_args* a, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!a || a->max_n < 0 || a->W < 0) return CSA2_ERR_INVALID_ARG;
  csa2_status st = check_cache8(cache, a->B);
  if (st != CSA2_OK) return st;
  KeysParams p{};
  p.q = a->q;
  p.q_pos = a->q_pos;
  p.Q = a->Q;
  p.W = a->W;
  if (a->W > 0) {
    p.rows = static_cast<const uint8_t*>(a->swa);
    p.base_pos = a->swa_base_pos;
    p.S = a->S;
    p.rows_fp8 = a->swa_fp8;
  }
  p.main_kv = reinterpret_cast<const uint8_t*>(cache->codes);
  p.scales8 = cache->scales;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.m = cache->m;
  p.scale = a->scale;
  p.out = a->out;
  p.lse = a->lse;
  st = check_keys_call(p, a->B, a->Q, csa2_cache8_attn_workspace_size(a->B, a->Q, a->max_n, a->W), ws, ws_bytes);
  if (st != CSA2_OK || a->B == 0 || a->Q == 0) return st;
  p.hdr = header(ws);
  return from_cuda(launch_keys_attention(p, a->B, cache8_chunks(a->max_n, a->W), scratch(ws), (cudaStream_t)stream));
}

// ---------------------------------------------------------------- gathered weights
static int64_t weights_n(int64_t max_n) { return max_n < INT32_MAX ? max_n : INT32_MAX; }   // n_entries is 32 bits

size_t csa2_attn_weights_workspace_size(int B, int Q, int64_t max_n) {
  if (B < 0 || Q < 0 || max_n < 0 || (int64_t)B * Q > MAX_KEY_QUERIES) return 0;
  const int64_t n = weights_n(max_n);
  const AwPlan plan = attn_weights_plan(B, Q, n);
  return HDR + (plan.splits > 1 ? align256((size_t)plan.splits * B * attn_weights_pitch(n) * sizeof(float)) : 0);
}

// p: the cache's part, filled in; entry: bytes of one of its entries
static csa2_status do_attn_weights(AwParams p, int64_t entry, const csa2_weights_args* a, void* ws, size_t ws_bytes,
                                   void* stream) {
  if (a->Q < 0 || a->max_n < 0 || !std::isfinite(a->scale) || !std::isfinite(a->decay)) return CSA2_ERR_INVALID_ARG;
  const int64_t BQ = (int64_t)a->B * a->Q, out_n = a->B * p.cap * 4;
  if (BQ > MAX_KEY_QUERIES || a->B > MAX_KEY_QUERIES) return CSA2_ERR_UNSUPPORTED;
  const size_t need = csa2_attn_weights_workspace_size(a->B, a->Q, a->max_n);
  csa2_status st = check_ws(ws, ws_bytes, need);
  if (st != CSA2_OK || a->B == 0) return st;
  if (!a->weights || !aligned4(a->weights) || !aligned4(a->prev) || !aligned4(p.n_entries)) return CSA2_ERR_INVALID_ARG;
  if (BQ > 0 && (!a->q || !aligned16(a->q) || !a->q_pos || !aligned8(a->q_pos) || !a->lse || !aligned4(a->lse)))
    return CSA2_ERR_INVALID_ARG;
  const struct { const void* a; int64_t n; } in[] = {
      {a->q, BQ * H * D * 2}, {a->q_pos, BQ * 8}, {a->lse, BQ * H * 4}, {ws, (int64_t)need}, {p.kv, a->B * p.cap * entry},
      {p.scales8, p.scales8 ? a->B * (p.cap / BLK) * 4 : 0}, {p.n_entries, (int64_t)a->B * 4},
      {a->prev, a->prev && a->prev != a->weights ? out_n : 0}};
  for (const auto& x : in)
    if (overlap(x.a, x.n, a->weights, out_n)) return CSA2_ERR_INVALID_ARG;
  p.q = a->q;
  p.q_pos = a->q_pos;
  p.lse = a->lse;
  p.scale = a->scale;
  p.decay = a->decay;
  p.prev = a->prev;
  p.out = a->weights;
  p.B = a->B;
  p.Q = a->Q;
  p.max_n = weights_n(a->max_n);
  p.hdr = header(ws);
  p.part = reinterpret_cast<float*>(scratch(ws));
  return from_cuda(launch_attn_weights(p, (cudaStream_t)stream));
}

csa2_status csa2_attn_weights(const csa2_cache* cache, const csa2_weights_args* a, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!a || a->B < 0) return CSA2_ERR_INVALID_ARG;
  const csa2_status st = check_cache_entries(cache);
  if (st != CSA2_OK) return st;
  AwParams p{};
  p.kv = cache->main_kv;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.m = cache->m;
  return do_attn_weights(p, MAIN_BYTES, a, ws, ws_bytes, stream);
}

csa2_status csa2_cache8_attn_weights(const csa2_cache8* cache, const csa2_weights_args* a, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!a) return CSA2_ERR_INVALID_ARG;
  const csa2_status st = check_cache8(cache, a->B);
  if (st != CSA2_OK) return st;
  AwParams p{};
  p.kv = reinterpret_cast<const uint8_t*>(cache->codes);
  p.scales8 = cache->scales;
  p.cap = cache->cap;
  p.n_entries = cache->n_entries;
  p.m = cache->m;
  return do_attn_weights(p, D, a, ws, ws_bytes, stream);
}

// ---------------------------------------------------------------- eviction
size_t csa2_evict_workspace_size(int B, int64_t budget, int unit) {
  if (B < 0 || budget < 1 || budget > INT32_MAX || (unit != 1 && unit != 8) || budget % unit != 0) return 0;
  // the chunks of an 8-bit cache are the smaller ones
  const int64_t chunks = evict_chunks(unit == 8 ? 8 : 4, unit, budget / unit);
  return HDR + align256(sizeof(uint32_t)) + align256((size_t)B * 4) + align256((size_t)B * chunks * 4);
}

// p: the caches' part, filled in.  An array of either cache: its bytes for one entry times 8.
struct EvArray {
  const void* from;
  void* to;
  int64_t bytes8;
};

static csa2_status do_evict(EvParams p, const EvArray* arrays, int n_arrays, int bits, const csa2_evict_args* a, void* ws,
                            size_t ws_bytes, void* stream) {
  const int64_t unit = a->unit, lim = INT32_MAX;
  if (a->B < 0 || a->budget < 1 || a->budget % unit != 0 || a->n_first < 0 || a->n_recent < 0) return CSA2_ERR_INVALID_ARG;
  if (p.cap > lim || p.to_cap > lim || a->budget > lim) return CSA2_ERR_UNSUPPORTED;
  if (a->n_first > a->budget || a->n_recent > a->budget || a->budget > p.to_cap) return CSA2_ERR_INVALID_ARG;
  const int64_t first = ceil_div(a->n_first, unit), recent = ceil_div(a->n_recent, unit) + (unit > 1 ? 1 : 0);
  if (first + recent > a->budget / unit) return CSA2_ERR_INVALID_ARG;
  // a chunk of the moves is 40 entries or more: every grid stays below 2^31 CTAs
  if (a->B > (1 << 20) || a->B * (a->budget / 40 + p.to_cap / 8192 + 2) >= lim) return CSA2_ERR_UNSUPPORTED;
  const size_t need = csa2_evict_workspace_size(a->B, a->budget, a->unit);
  csa2_status st = check_ws(ws, ws_bytes, need);
  if (st != CSA2_OK || a->B == 0) return st;
  if (!a->weights || !aligned16(a->weights) || !aligned4(a->to_weights) || !a->kept || !aligned4(a->kept) || !a->n_out ||
      !aligned4(a->n_out) || !aligned4(p.n_entries))
    return CSA2_ERR_INVALID_ARG;
  // in place: every array the same
  int same = 0;
  for (int i = 0; i < n_arrays; i++) same += arrays[i].from == arrays[i].to;
  if (same != 0 && (same != n_arrays || p.cap != p.to_cap)) return CSA2_ERR_INVALID_ARG;
  p.in_place = same != 0;
  // what the call writes and what it reads; [from, from + n) are pairs that may be one
  struct Range { const void* a; int64_t n; } out[8], in[12];
  int n_out = 0, n_in = 0;
  for (int i = 0; i < n_arrays; i++) {
    out[n_out++] = {arrays[i].to, a->B * (p.to_cap / 8) * arrays[i].bytes8};
    if (!p.in_place) in[n_in++] = {arrays[i].from, a->B * (p.cap / 8) * arrays[i].bytes8};
  }
  if (a->to_weights) out[n_out++] = {a->to_weights, a->B * p.to_cap * 4};
  out[n_out++] = {a->kept, a->B * (a->budget / unit) * 4};
  out[n_out++] = {a->n_out, (int64_t)a->B * 4};
  if (!(p.in_place && a->to_weights == a->weights)) in[n_in++] = {a->weights, a->B * p.cap * 4};
  if (a->n_out != p.n_entries) in[n_in++] = {p.n_entries, (int64_t)a->B * 4};
  in[n_in++] = {ws, (int64_t)need};
  for (int i = 0; i < n_out; i++) {
    for (int k = 0; k < n_in; k++)
      if (overlap(out[i].a, out[i].n, in[k].a, in[k].n)) return CSA2_ERR_INVALID_ARG;
    for (int k = 0; k < i; k++)
      if (overlap(out[i].a, out[i].n, out[k].a, out[k].n)) return CSA2_ERR_INVALID_ARG;
  }
  p.B = a->B;
  p.units = a->budget / unit;
  p.first = first;
  p.recent = a->n_recent;
  p.weights = a->weights;
  p.to_weights = a->to_weights;
  p.kept = a->kept;
  p.n_out = a->n_out;
  p.hdr = header(ws);
  unsigned char* cur = scratch(ws);
  p.ticket = reinterpret_cast<uint32_t*>(cur);
  cur += align256(sizeof(uint32_t));
  p.n_new = reinterpret_cast<int32_t*>(cur);
  cur += align256((size_t)a->B * 4);
  p.flags = reinterpret_cast<int32_t*>(cur);
  return from_cuda(launch_evict(p, bits, a->unit, (cudaStream_t)stream));
}

csa2_status csa2_evict(const csa2_cache* cache, const csa2_cache* to, const csa2_evict_args* a, void* ws, size_t ws_bytes,
                       void* stream) {
  if (!a || (a->unit != 1 && a->unit != 8)) return CSA2_ERR_INVALID_ARG;
  if (!to) to = cache;
  csa2_status st = check_cache_entries(cache);
  if (st != CSA2_OK) return st;
  if (!to->main_kv || !aligned16(to->main_kv) || to->cap < 0 || to->cap % BLK != 0) return CSA2_ERR_INVALID_ARG;
  const bool index = cache->idx_codes && cache->idx_scales && to->idx_codes && to->idx_scales;
  if (index && (!aligned16(cache->idx_codes) || !aligned16(cache->idx_scales) || !aligned16(to->idx_codes) ||
                !aligned16(to->idx_scales)))
    return CSA2_ERR_INVALID_ARG;
  EvParams p{};
  p.rows = cache->main_kv;
  p.to_rows = to->main_kv;
  if (index) {
    p.idx_codes = cache->idx_codes;
    p.idx_scales = cache->idx_scales;
    p.to_idx_codes = to->idx_codes;
    p.to_idx_scales = to->idx_scales;
  }
  p.cap = cache->cap;
  p.to_cap = to->cap;
  p.n_entries = cache->n_entries;
  const EvArray arrays[] = {{p.rows, p.to_rows, 8 * MAIN_BYTES}, {p.idx_codes, p.to_idx_codes, 8 * IDX_CODE_BYTES},
                            {p.idx_scales, p.to_idx_scales, 8 * IDX_SCALE_BYTES}};
  return do_evict(p, arrays, index ? 3 : 1, 4, a, ws, ws_bytes, stream);
}

csa2_status csa2_cache8_evict(const csa2_cache8* cache, const csa2_cache8* to, const csa2_evict_args* a, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!a) return CSA2_ERR_INVALID_ARG;
  if (a->unit != 8) return a->unit == 1 ? CSA2_ERR_UNSUPPORTED : CSA2_ERR_INVALID_ARG;
  if (!to) to = cache;
  csa2_status st = check_cache8(cache, a->B);
  if (st != CSA2_OK) return st;
  if (!to->codes || !to->scales || !aligned16(to->codes) || !aligned4(to->scales) || to->cap < 0 || to->cap % BLK != 0)
    return CSA2_ERR_INVALID_ARG;
  EvParams p{};
  p.rows = reinterpret_cast<const uint8_t*>(cache->codes);
  p.scales = cache->scales;
  p.to_rows = reinterpret_cast<uint8_t*>(to->codes);
  p.to_scales = to->scales;
  p.cap = cache->cap;
  p.to_cap = to->cap;
  p.n_entries = cache->n_entries;
  const EvArray arrays[] = {{p.rows, p.to_rows, 8 * D}, {p.scales, p.to_scales, 4}};
  return do_evict(p, arrays, 2, 8, a, ws, ws_bytes, stream);
}

// HISA keeps up to 2048 of its summary rows: past 4096 blocks a row goes to
// the multi-CTA selection (a single CTA spends most of its time on the
// output once M is a large part of the row)
constexpr int64_t HISA_ROW_SELECT_MIN = 4096;
bool hisa_long_rows(int64_t nb) { return nb > HISA_ROW_SELECT_MIN; }

size_t csa2_hisa_blocks_workspace_size(int B, int Q, int64_t max_n) {
  if (B < 0 || Q < 0 || max_n < 0) return 0;
  const int64_t nb = ceil_div(max_n, BLK);
  return HDR + align256((size_t)B * Q * sizeof(int64_t)) + align256((size_t)B * sizeof(int32_t)) +
         align256((size_t)B * Q * nb * sizeof(float)) +
         (hisa_long_rows(nb) ? align256(row_select_bytes((int64_t)B * Q)) : 0);
}

csa2_status csa2_hisa_blocks(const csa2_cache* cache, const uint8_t* sum_codes, const uint8_t* sum_scales,
                             int64_t sum_cap, const uint16_t* q_idx, const float* w_head, const int64_t* q_pos,
                             int B, int Q, int64_t max_n, int M, int32_t* pool_blocks, void* ws, size_t ws_bytes,
                             void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if ((st = check_q(B, Q)) != CSA2_OK) return st;
  if (max_n < 0 || sum_cap < 0 || (sum_cap % BLK) != 0) return CSA2_ERR_INVALID_ARG;
  if (M < 1 || M > CSA2_MAX_M) return CSA2_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, csa2_hisa_blocks_workspace_size(B, Q, max_n))) != CSA2_OK) return st;
  if (B == 0 || Q == 0) return CSA2_OK;
  if (!sum_codes || !sum_scales || !q_idx || !w_head || !q_pos || !pool_blocks) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(sum_codes) || !aligned16(sum_scales) || !aligned16(q_idx)) return CSA2_ERR_INVALID_ARG;
  // rows past the summary store cannot be scored
  if (ceil_div(cache->cap, BLK) > sum_cap) return CSA2_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  WsHeader* hdr = header(ws);
  unsigned char* cur = scratch(ws);
  const int64_t nb = ceil_div(max_n, BLK);
  HvParams vp{};
  vp.q_pos = q_pos;
  vp.n_entries = cache->n_entries;
  vp.m = cache->m;
  vp.B = B;
  vp.Q = Q;
  vp.cap = cache->cap;
  vp.max_n = max_n;
  vp.view_pos = reinterpret_cast<int64_t*>(cur);
  cur += align256((size_t)B * Q * sizeof(int64_t));
  vp.view_n = reinterpret_cast<int32_t*>(cur);
  cur += align256((size_t)B * sizeof(int32_t));
  float* scores = reinterpret_cast<float*>(cur);
  cur += align256((size_t)B * Q * nb * sizeof(float));
  st = from_cuda(launch_hisa_view(vp, s));
  if (st != CSA2_OK) return st;
  // the summary store read as an m = 1 cache of ceil(n / 8) rows per sequence
  csa2_cache view{};
  view.main_kv = cache->main_kv;
  view.idx_codes = const_cast<uint8_t*>(sum_codes);
  view.idx_scales = const_cast<uint8_t*>(sum_scales);
  view.cap = sum_cap;
  view.n_entries = vp.view_n;
  view.m = 1;
  st = do_index_score(&view, q_idx, w_head, vp.view_pos, nullptr, M, scores, B, Q, nb, hdr, s);
  if (st != CSA2_OK) return st;
  if (hisa_long_rows(nb))
    return from_cuda(launch_row_select(scores, vp.view_pos, vp.view_n, 1, B, Q, nb, M, pool_blocks, 0, nullptr,
                                       cur, s));
  return from_cuda(launch_select_topk(scores, vp.view_pos, vp.view_n, 1, nullptr, M, M, pool_blocks, B, Q, nb, s));
}

size_t csa2_decode_workspace_size(csa2_mode mode, int B, int Q, int64_t max_n, int M, int K) {
  if (B < 0 || Q < 0 || max_n < 0 || M < 0 || K < 0) return 0;
  size_t need = HDR + align256(attn_partials_bytes((int64_t)B * Q, K));
  if (mode == CSA2_MODE_FULL) {
    need += align256((size_t)B * Q * max_n * sizeof(float)) + select_scratch_bytes(B, Q, max_n, true);
  } else if (mode == CSA2_MODE_REINDEX) {
    need += align256((size_t)B * Q * M * BLK * sizeof(float));
  }
  return need;
}

csa2_status csa2_decode(const csa2_cache* cache, const csa2_decode_args* a, void* ws, size_t ws_bytes,
                        void* stream) {
  csa2_status st = check_cache(cache);
  if (st != CSA2_OK) return st;
  if (!a) return CSA2_ERR_INVALID_ARG;
  if (a->mode != CSA2_MODE_FULL && a->mode != CSA2_MODE_REINDEX && a->mode != CSA2_MODE_REUSE)
    return CSA2_ERR_INVALID_ARG;
  if ((st = check_q(a->B, a->Q)) != CSA2_OK) return st;
  if (a->K < 1 || a->K > CSA2_MAX_K) return CSA2_ERR_UNSUPPORTED;
  if (a->mode != CSA2_MODE_REUSE && (a->M < 1 || a->M > CSA2_MAX_M)) return CSA2_ERR_UNSUPPORTED;
  if (a->S < 0 || a->max_n < 0 || !std::isfinite(a->scale)) return CSA2_ERR_INVALID_ARG;
  const size_t need = csa2_decode_workspace_size(a->mode, a->B, a->Q, a->max_n, a->M, a->K);
  if ((st = check_ws(ws, ws_bytes, need)) != CSA2_OK) return st;
  if (a->B == 0 || a->Q == 0) return CSA2_OK;
  if (!a->q_pos || !a->q || !a->swa || !a->swa_base_pos || !a->sel || !a->out) return CSA2_ERR_INVALID_ARG;
  if (a->mode != CSA2_MODE_REUSE && (!a->q_idx || !a->w_head || !a->pool_blocks)) return CSA2_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->swa) || !aligned16(a->out)) return CSA2_ERR_INVALID_ARG;
  if (a->mode != CSA2_MODE_REUSE && !aligned16(a->q_idx)) return CSA2_ERR_INVALID_ARG;
  if (a->packed_sel && !aligned16(a->packed_sel)) return CSA2_ERR_INVALID_ARG;
  if (a->swa_fp8 != 0 && a->swa_fp8 != 1) return CSA2_ERR_INVALID_ARG;
  if (a->attn_split < 0) return CSA2_ERR_INVALID_ARG;
  const int split = a->attn_split > 1 ? a->attn_split : 1;
  if (split > 1 && (int64_t)a->B * a->Q > attn_split_max_queries()) return CSA2_ERR_UNSUPPORTED;
  const uint8_t* packed_in = a->mode == CSA2_MODE_REUSE ? a->packed_sel : nullptr;
  uint8_t* packed_out = a->mode == CSA2_MODE_REUSE ? nullptr : a->packed_sel;

  cudaStream_t s = (cudaStream_t)stream;
  WsHeader* hdr = header(ws);
  unsigned char* cur = scratch(ws);
  void* part = cur;
  cur += align256(attn_partials_bytes((int64_t)a->B * a->Q, a->K));
  if (a->mode == CSA2_MODE_FULL) {
    float* scores = reinterpret_cast<float*>(cur);
    cur += align256((size_t)a->B * a->Q * a->max_n * sizeof(float));
    uint32_t* gkeys = reinterpret_cast<uint32_t*>(cur);
    st = do_index_score(cache, a->q_idx, a->w_head, a->q_pos, nullptr, a->M, scores, a->B, a->Q, a->max_n, hdr, s);
    if (st != CSA2_OK) return st;
    if (long_rows(a->max_n)) {
      st = from_cuda(launch_row_select(scores, a->q_pos, cache->n_entries, cache->m, a->B, a->Q, a->max_n, a->K,
                                       a->sel, a->M, a->pool_blocks, cur, s));
      if (st != CSA2_OK) return st;
      return do_attention(cache, a->q, a->sel, a->K, a->swa, a->swa_base_pos, a->S, a->q_pos, a->scale, a->out,
                          a->B, a->Q, part, hdr, s, packed_in, packed_out, a->swa_fp8 != 0, split);
    }
    st = from_cuda(launch_block_topk(scores, a->q_pos, cache->n_entries, cache->m, a->B, a->Q, a->max_n, a->M,
                                     a->pool_blocks, gkeys, s));
    if (st != CSA2_OK) return st;
    st = from_cuda(launch_select_topk(scores, a->q_pos, cache->n_entries, cache->m, nullptr, a->M, a->K, a->sel,
                                      a->B, a->Q, a->max_n, s));
    if (st != CSA2_OK) return st;
  } else if (a->mode == CSA2_MODE_REINDEX) {
    IsParams ip{};
    ip.idx_codes = cache->idx_codes;
    ip.idx_scales = cache->idx_scales;
    ip.cap = cache->cap;
    ip.n_entries = cache->n_entries;
    ip.m = cache->m;
    ip.q_idx = a->q_idx;
    ip.w_head = a->w_head;
    ip.q_pos = a->q_pos;
    ip.pool = a->pool_blocks;
    ip.M = a->M;
    ip.B = a->B;
    ip.Q = a->Q;
    ip.max_n = a->max_n;
    ip.sel = a->sel;
    ip.K = a->K;
    ip.hdr = hdr;
    ip.scores = reinterpret_cast<float*>(cur);                   // the pool slots' keys
    st = from_cuda(launch_reindex_select(ip, s));
    if (st != CSA2_OK) return st;
  }
  return do_attention(cache, a->q, a->sel, a->K, a->swa, a->swa_base_pos, a->S, a->q_pos, a->scale, a->out, a->B,
                      a->Q, part, hdr, s, packed_in, packed_out, a->swa_fp8 != 0, split);
}

}  // extern "C"
