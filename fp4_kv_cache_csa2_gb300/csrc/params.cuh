// Launch parameters and launcher declarations shared by the CSA2 translation units.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace csa2 {

struct CwParams {
  uint8_t* main_kv;
  uint8_t* idx_codes;
  uint8_t* idx_scales;
  int64_t cap;
  int m;
  const uint16_t* x;        // [B][T][512]
  int B, T;
  const int64_t* entry_start;
  const float* w0;
  const float* w1;
  const float* rope_cs;     // [P][32][2]
  int64_t rope_P;
  const uint16_t* w_idx;    // [128][512]
  WsHeader* hdr;
};

struct IsParams {
  const uint8_t* idx_codes;
  const uint8_t* idx_scales;
  int64_t cap;
  const int32_t* n_entries;
  int m;
  const uint16_t* q_idx;      // [B][Q][32][128]
  const float* w_head;        // [B][Q][32]
  const int64_t* q_pos;       // [B][Q]
  const int32_t* pool;        // [B][Q][M] or null
  int M;
  float* scores;              // [B][Q][max_n] or [B][Q][M*8]
  int B, Q;
  int64_t max_n;
  int64_t entries_per_cta;    // set by the launcher
  int64_t group0;             // first query group of this launch (index scan; set by the launcher)
  int32_t* sel;               // fused Reindex: [B][Q][K] output
  int K;
  WsHeader* hdr;
  int test_withhold;          // test hook: the producer waits on a barrier nobody arrives on (0 = off)
};

struct AttnParams {
  const uint8_t* main_kv;
  int64_t cap;
  const uint16_t* q;          // [BQ][64][512]
  const int32_t* sel;         // [BQ][K]
  int K;
  const uint16_t* swa;        // [B][S][512] bf16, or E4M3 bytes when swa_fp8
  const int64_t* swa_base;    // [B]
  int S;
  int swa_fp8;
  const int64_t* q_pos;       // [BQ]
  float scale;
  uint16_t* out;              // [BQ][64][512]
  int Q;
  const uint8_t* packed_in;   // [BQ][K][288] selected entries to read instead of gathering, or null
  uint8_t* packed_out;        // [BQ][K][288] where to write the gathered selected entries, or null
  int split;                  // CTAs per query (1: the whole query in one CTA)
  float* opart;               // split > 1: the partial states, [BQ * split][2 * 64 + 64 * 512]
  WsHeader* hdr;
};

struct HsParams {             // HISA block summaries
  const uint8_t* idx_codes;
  const uint8_t* idx_scales;
  int64_t cap;
  const int32_t* n_entries;
  const int64_t* first_block; // [B]
  int B;
  int64_t n_blocks;           // blocks per sequence from first_block
  uint8_t* sum_codes;         // [B][sum_cap][64]
  uint8_t* sum_scales;        // [B][sum_cap][4]
  int64_t sum_cap;
  WsHeader* hdr;
};

struct HvParams {             // HISA view of the summary store as an m = 1 cache
  const int64_t* q_pos;       // [B][Q]
  const int32_t* n_entries;   // [B]
  int m, B, Q;
  int64_t cap, max_n;
  int64_t* view_pos;          // [B][Q] out
  int32_t* view_n;            // [B] out
};

struct QkParams {             // norm and rotation of queries and window keys
  int64_t T;
  const int64_t* pos;         // [T], -1: padding
  const float* rope_cs;       // [rope_P][32][2]
  int64_t rope_P;
  float eps;
  const uint16_t* q;          // token t at t * q_stride: [64][512], or null
  int64_t q_stride;
  const float* q_weight;      // [512] or null
  uint16_t* q_out;            // [T][64][512]
  const uint16_t* k;          // token t at t * k_stride: [512], or null
  int64_t k_stride;
  const float* k_weight;      // [512] or null
  uint8_t* rows;              // [n_rows][512] bf16, or E4M3 bytes when rows_fp8
  int64_t n_rows;
  const int64_t* k_slot;      // [T] row of each token (-1: none), or null: row = token
  int rows_fp8;
  WsHeader* hdr;
};

struct KeysParams {           // attention over every visible key
  const uint16_t* q;          // [BQ][64][512] bf16
  const int64_t* q_pos;       // [BQ]
  int Q;
  const uint8_t* rows;        // [B][S][512] bf16, or E4M3 bytes when rows_fp8
  const int64_t* base_pos;    // [B] position of row 0
  int64_t S;
  const uint8_t* sinks;       // [B][n_sink][512] rows of positions 0 .. n_sink - 1, or null
  int n_sink;
  int rows_fp8;
  int64_t W;                  // window
  const uint8_t* main_kv;     // [B][cap][288], with scales8 [B][cap][512]; or null: no cache entries
  const float* scales8;       // 8-bit entries: [B][cap / 8]; null: 4-bit
  int64_t cap;
  const int32_t* n_entries;   // [B]
  int m;
  float scale;
  uint16_t* out;              // [BQ][64][512] bf16
  float* lse;                 // [BQ][64] or null
  int split;                  // CTAs per query (set by the launcher)
  float* part;                // split > 1: partial states
  WsHeader* hdr;
};

struct C8WriteParams {        // entries of the 8-bit cache
  uint8_t* codes;             // [B][cap][512]
  float* scales;              // [B][cap / 8]
  int64_t cap;
  const int32_t* n_entries;
  const uint16_t* x;          // token i of sequence b at (b * T + i) * x_stride
  int64_t x_stride;
  int B, T;
  const int64_t* start;       // [B]
  const int32_t* n_new;       // [B] or null
  WsHeader* hdr;
};

struct AwParams {             // attention weight that entries gather
  const uint8_t* kv;          // [B][cap][288], with scales8 [B][cap][512]
  const float* scales8;       // 8-bit entries: [B][cap / 8]; null: 4-bit
  int64_t cap;
  const int32_t* n_entries;   // [B]
  int m;
  const uint16_t* q;          // [BQ][64][512] bf16
  const int64_t* q_pos;       // [BQ]
  const float* lse;           // [BQ][64]
  float scale, decay;
  const float* prev;          // [B][cap] or null
  float* out;                 // [B][cap]
  int B, Q;
  int64_t max_n;
  float* part;                // splits > 1: [splits][B][pitch]
  int64_t pitch;              // set by the launcher, as the next two
  int runs, splits;
  WsHeader* hdr;
};

struct EvParams {             // eviction; `to_`: where entries go
  const uint8_t *rows, *idx_codes, *idx_scales;   // idx_*: null when not moved
  const float* scales;        // 8-bit entries
  uint8_t *to_rows, *to_idx_codes, *to_idx_scales;
  float* to_scales;
  int64_t cap, to_cap;
  const int32_t* n_entries;   // [B]
  int B;
  int64_t units;              // units that stay at most
  int64_t first;              // first units that stay
  int64_t recent;             // last entries that stay
  const float* weights;       // [B][cap]
  float* to_weights;          // [B][to_cap] or null
  int32_t* kept;              // [B][units]
  int32_t* n_out;             // [B]
  int in_place;
  uint32_t* ticket;           // scratch: the next chunk
  int32_t* n_new;             // scratch: [B] entries that stay
  int32_t* flags;             // scratch: [B][chunks] chunks that have been read
  int64_t chunks;             // set by the launcher
  WsHeader* hdr;
};

cudaError_t launch_cache_write(const CwParams& p, cudaStream_t stream, int num_sms);
cudaError_t launch_swa_fp8(const uint16_t* x, int64_t n_rows, uint8_t* out, cudaStream_t stream);
cudaError_t launch_index_score(IsParams p, cudaStream_t stream);
cudaError_t launch_reindex_select(IsParams p, cudaStream_t stream);
cudaError_t launch_block_topk(const float* scores, const int64_t* q_pos, const int32_t* n_entries, int m,
                              int B, int Q, int64_t max_n, int M, int32_t* pool_blocks, uint32_t* gkeys,
                              cudaStream_t stream);
cudaError_t launch_select_topk(const float* scores, const int64_t* q_pos, const int32_t* n_entries, int m,
                               const int32_t* pool, int M, int K, int32_t* sel, int B, int Q, int64_t max_n,
                               cudaStream_t stream);
// Full rows longer than ROW_SELECT_MIN_KEYS entries are selected by the
// multi-CTA histogram/filter path, with row_select_bytes(B*Q) of scratch.
constexpr int64_t ROW_SELECT_MIN_KEYS = 16384;
size_t row_select_bytes(int64_t BQ);
cudaError_t launch_row_select(const float* scores, const int64_t* q_pos, const int32_t* n_entries, int m, int B,
                              int Q, int64_t max_n, int K, int32_t* sel, int M, int32_t* pool, void* scratch,
                              cudaStream_t stream);
cudaError_t launch_attention(AttnParams p, int B, float* partials, cudaStream_t stream);
size_t attn_partials_bytes(int64_t BQ, int K);
int attn_split_max_queries();
cudaError_t launch_block_summary(const HsParams& p, cudaStream_t stream);
cudaError_t launch_hisa_view(const HvParams& p, cudaStream_t stream);
// `chunks`: runs of KEYS_CHUNK keys of the longest query (for the split over CTAs);
// `part`: keys_part_bytes(B * Q, chunks) of scratch
constexpr int KEYS_CHUNK = 64;
cudaError_t launch_keys_attention(KeysParams p, int B, int64_t chunks, void* part, cudaStream_t stream);
// The same for a call without cache entries whose windows are short enough (window_ring_fits):
// many queries in a row over a ring of rows in shared memory
cudaError_t launch_window_ring(const KeysParams& p, int B, cudaStream_t stream);
bool window_ring_fits(int64_t W, int n_sink);
size_t keys_part_bytes(int64_t BQ, int64_t chunks);
struct Cache8Plan { bool pairs; int split; };             // of a call with scales8
Cache8Plan cache8_plan(int B, int Q, int64_t chunks);
size_t cache8_part_bytes(int B, int Q, int64_t chunks);
// Several queries of an 8-bit cache (p.split and p.part set; the maps of q, the rows and the codes)
cudaError_t launch_pair_attention(const KeysParams& p, int B, const CUtensorMap& mr8, cudaStream_t stream);
struct AwPlan { int runs, splits; };    // of a sequence's tiles, of its queries
AwPlan attn_weights_plan(int B, int Q, int64_t max_n);
int64_t attn_weights_pitch(int64_t max_n);
cudaError_t launch_attn_weights(AwParams p, cudaStream_t stream);
int64_t evict_chunks(int bits, int unit, int64_t units);
cudaError_t launch_evict(EvParams p, int bits, int unit, cudaStream_t stream);
cudaError_t launch_cache8_write(const C8WriteParams& p, cudaStream_t stream);
cudaError_t launch_qk_norm_rope(const QkParams& p, cudaStream_t stream);

}  // namespace csa2
