// Rotating cache writes and latent attention: what their C ABI
// (pkv_latent_api.cu) hands to the kernel units.
#pragma once

#include "pkv_ops.h"

namespace pkv {

constexpr int kRopeDim = 64;  // rotated dims of a latent row and of its queries

// Rotation of a set of query heads: q [T, H, D] into q_out, `stride` elements
// from token to token and `head` from head to head.
struct RopeQuery {
    const void *q;
    void *out;
    int64_t stride, head, out_stride, out_head;
    int num_heads;           // 0: no queries
};

// What both cache writes share.
struct RopeTokens {
    const int32_t *positions;  // [T]
    const float *table;        // [max_positions, rot]: cosines, then sines
    const int64_t *slots;      // [T]
    int32_t *status;           // optional
    int num_tokens, rot, max_positions, num_blocks;
    int interleaved;           // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
    int in_dtype;
};

// K rotated and V as it is into their slots of caches [N, Hkv, D, 16].
struct RopeAppendParams {
    RopeTokens t;
    RopeQuery q;
    const void *k, *v;  // [T, Hkv, D]
    int64_t k_stride, v_stride;
    void *k_cache, *v_cache;
    int kv_dtype, num_kv_heads, head_dim;
    float k_scale, v_scale;
};

// Rows (latent | rotated key) of a cache [N, 16, R + 64].
struct LatentAppendParams {
    RopeTokens t;
    RopeQuery q;
    const void *latent, *k_rope;  // [T, R], [T, 64]
    int64_t latent_stride, k_rope_stride;
    void *cache;
    int cache_dtype, latent_dim;
};

// Latent attention, one query per sequence (absorbed form): over the rows
// [R + 64] of a paged cache [N, 16, R + 64], whose first R numbers are the values.
struct LatentDecodeParams {
    const void *q;       // [S, H, R + 64]
    const void *cache;
    const int32_t *block_tables;
    const int32_t *seq_lens;
    void *out;           // [S, H, R]
    int32_t *status;     // optional
    int num_seqs, num_heads, latent_dim, num_blocks, max_blocks, max_len;
    float score_scale;   // |scale| * log2(e), at least 2^-120
    int negate;          // scale < 0: the scores are negated
    int drop_first_copy; // test hook: never issue the first copy of CTA 0
    // The schedule (latent_plan).
    int tile_heads, head_tiles, teams;
    int whole;           // sequences are not cut
    float *part;         // [2 teams][head tiles][tile_heads][R] sums of weights times rows
    float2 *part_ml;     // [2 teams][head tiles][tile_heads] reference of the weights (log2), their sum
    int *pieces;         // [teams] sequence cut by a team's start (-1: none)
};

// Latent attention over whole prompts with keys and values expanded per head.
struct LatentPromptParams {
    const void *q;       // [T, H, Dn + 64]
    const void *k;       // [T, H, Dn]
    const void *k_rope;  // [T, 64]
    const void *v;       // [T, H, Dn]
    void *out;           // [T, H, Dn]
    int64_t q_stride, k_stride, k_head, k_rope_stride, v_stride, v_head;  // elements
    int nope;
    PromptParams items;  // sequences and heads, for the look-up of work items
    int drop_first_copy; // test hook: never issue the first copy of CTA 0
};

constexpr int kLatentSms = 152;    // SMs that a plan counts on
constexpr int kLatentTokens = 64;  // tokens of a tile: the decode's unit of work
constexpr int kLatentMaxSeqs = 1 << 20;  // every CTA reads all lengths once

// Heads of a tile, tiles per sequence and teams for a call: set in p.  Returns
// the bytes of workspace, 0 for sizes without a plan.
size_t latent_plan(LatentDecodeParams &p, int dtype);
size_t latent_part_rows(const LatentDecodeParams &p);  // of partial sums in the workspace

pkv_status launch_latent_decode_simt(const LatentDecodeParams &p, cudaStream_t stream);
pkv_status launch_latent_decode_tc(const LatentDecodeParams &p, cudaStream_t stream);
pkv_status launch_latent_merge(const LatentDecodeParams &p, int dtype, cudaStream_t stream);
pkv_status launch_latent_prompt_simt(const LatentPromptParams &p, cudaStream_t stream);
pkv_status launch_latent_prompt_tc(const LatentPromptParams &p, cudaStream_t stream);
pkv_status launch_rope_append(const RopeAppendParams &p, cudaStream_t stream);
pkv_status launch_latent_append(const LatentAppendParams &p, cudaStream_t stream);

}  // namespace pkv
