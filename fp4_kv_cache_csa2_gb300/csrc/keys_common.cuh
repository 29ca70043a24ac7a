// What the attentions over every key share: the softmax's reference and the partial states.
#pragma once

#include "common.cuh"
#include "params.cuh"

namespace csa2 {

constexpr float KA_LOG2E = 1.4426950408889634f;
constexpr float KA_LN2 = 0.6931471805599453f;
// The reference of a head moves when a score (in powers of two) lies KA_TAU (bf16, where P has
// binary32's range) or KA_MOST (F16) above it.  F16: P of the largest score is 2^KA_TOP when the reference is set,
// and at most 2^KA_MOST, f16's range less a little, before it moves.  Weights down to 2^-22 of the largest
// keep f16's 11 bits, and what lies below loses 2^-33 of it at most: with a reference at the largest
// score itself one key 17.3 above 131,072 others alike lost all of their 0.4 %.  The room between
// the two (5.5 in logits) keeps rescalings rare: 2048 queries over 8192 entries took 1911 us, with
// 2^0 at the top 1910, with 2^10 1933, with 2^11 1971 (and 15 more each with the check of q's range).
constexpr float KA_TAU = 8.0f * KA_LOG2E;
constexpr float KA_TOP = 8.0f, KA_MOST = 15.9f;
// 8-bit entries: codes times a block's scale s.  The tensor cores see the codes; s enters the scores, and the
// weights that go to the second product are P s, so the reference follows the scores plus log2 s.  The
// sum of the softmax is of P without s, which is why s counts as KA_FLOOR8 at least there: P stays below
// 2^(KA_MOST + 60), its sum inside binary32.  (Up to s = 2^80 the largest P is 2^-72 or more, so that weights down to
// 2^-54 of it are in the sum.)
constexpr float KA_FLOOR8 = 0x1p-60f;
constexpr int KA_SMS = 152;                               // GB300; CTAs a query is divided over at most
constexpr int KA_PART_FLOATS = 2 * H + H * D;             // one partial state: references, sums, O [dims / 4][head][4]

// Joins the partial states of BQ queries (p.part, p.split > 1) into p.out and p.lse.
cudaError_t launch_keys_join(const KeysParams& p, int64_t BQ, cudaStream_t stream);

}  // namespace csa2
