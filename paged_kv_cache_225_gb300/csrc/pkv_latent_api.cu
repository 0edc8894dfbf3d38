// C ABI of the rotating cache writes and of the latent attention (declared in
// include/pkv.h): argument validation and dispatch.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "pkv_latent.h"

using namespace pkv;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_float(pkv_dtype t) { return t == PKV_F32 || t == PKV_BF16; }

// A distance in elements of `dtype`: at least `least`, a multiple of 16 bytes, below 2^36.
bool stride_ok(int64_t stride, int64_t least, pkv_dtype dtype)
{
    return stride >= least && stride % (dtype == PKV_F32 ? 4 : 8) == 0 && stride < (int64_t{1} << 36);
}

// Whether `count` runs of `dim` numbers, `step` apart (positive), fit in `room`; their
// extent may pass 64 bits.
bool fits(int count, int64_t step, int dim, int64_t room)
{
    return room >= dim && (count <= 1 || step <= (room - dim) / (count - 1));
}

// Heads of `dim` numbers, token by token or head by head, that do not overlap.
bool heads_apart(int num_tokens, int num_heads, int64_t stride, int64_t head, int dim)
{
    return fits(num_heads, head, dim, stride) || fits(num_tokens, stride, dim, head);
}

// Queries turned in place lie where they are read: other strides would write rows that
// another warp has yet to read.
bool in_place_ok(const RopeQuery &q, int num_tokens)
{
    return q.q != q.out || q.num_heads == 0 ||
           ((num_tokens <= 1 || q.stride == q.out_stride) && (q.num_heads <= 1 || q.head == q.out_head));
}

// The kernels work with a positive factor: the sign goes to the scores, and a zero
// becomes a factor too small to tell weights apart, which keeps masked scores (-inf)
// out all the same.
float score_factor(float scale)
{
    const float factor = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
    const float least = std::ldexp(1.0f, -120), most = std::ldexp(1.0f, 127);
    return factor < least ? least : factor > most ? most : factor;
}

// Arguments that both cache writes share.
pkv_status check_tokens(RopeTokens &t, pkv_dtype in_dtype, const int32_t *positions, const float *table, int rot_dim,
                        int max_positions, const int64_t *slots, int num_tokens, int block_size, int num_blocks,
                        int flags, int32_t *status)
{
    if (num_tokens < 0 || max_positions <= 0 || num_blocks <= 0 || (flags & ~PKV_FLAG_ROPE_INTERLEAVED) != 0)
        return PKV_ERR_INVALID_ARG;
    if (!is_float(in_dtype) || block_size != kBlockSize)
        return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return PKV_OK;
    if (!positions || !table || !slots)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(table, 16) || !aligned(slots, 8) || !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    t.positions = positions;
    t.table = table;
    t.slots = slots;
    t.status = status;
    t.num_tokens = num_tokens;
    t.rot = rot_dim;
    t.max_positions = max_positions;
    t.num_blocks = num_blocks;
    t.interleaved = (flags & PKV_FLAG_ROPE_INTERLEAVED) ? 1 : 0;
    t.in_dtype = in_dtype;
    return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_append(const void *q, const void *k, const void *v, pkv_dtype in_dtype, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int32_t *positions, const float *table,
                           int rot_dim, int max_positions, const int64_t *slot_mapping, int num_tokens,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                           void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache, pkv_dtype kv_dtype,
                           float k_scale, float v_scale, int flags, int32_t *status, void *stream)
{
    if (num_q_heads < 0 || num_kv_heads <= 0 || rot_dim <= 0 || rot_dim > head_dim)
        return PKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || rot_dim % 16 != 0)
        return PKV_ERR_UNSUPPORTED;
    if (!is_float(kv_dtype) && !is_scaled(kv_dtype))
        return PKV_ERR_UNSUPPORTED;
    if (is_scaled(kv_dtype) &&
        (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale == 0.f || v_scale == 0.f))
        return PKV_ERR_INVALID_ARG;
    RopeAppendParams p;
    std::memset(&p, 0, sizeof p);
    const pkv_status rc = check_tokens(p.t, in_dtype, positions, table, rot_dim, max_positions, slot_mapping,
                                       num_tokens, block_size, num_blocks, flags, status);
    if (rc != PKV_OK || num_tokens == 0)
        return rc;
    if (!k || !v || !k_cache || !v_cache || (num_q_heads > 0 && (!q || !q_out)))
        return PKV_ERR_INVALID_ARG;
    for (const void *a : {q, k, v, static_cast<const void *>(q_out), static_cast<const void *>(k_cache),
                          static_cast<const void *>(v_cache)})
        if (!aligned(a, 16))
            return PKV_ERR_INVALID_ARG;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    if (!stride_ok(k_stride, kv_row, in_dtype) || !stride_ok(v_stride, kv_row, in_dtype))
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!stride_ok(q_stride, q_row, in_dtype) || !stride_ok(q_out_stride, q_row, in_dtype)))
        return PKV_ERR_INVALID_ARG;
    p.q.q = q;
    p.q.out = q_out;
    p.q.stride = q_stride;
    p.q.out_stride = q_out_stride;
    p.q.head = p.q.out_head = head_dim;
    p.q.num_heads = num_q_heads;
    if (!in_place_ok(p.q, num_tokens))
        return PKV_ERR_INVALID_ARG;
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.kv_dtype = kv_dtype;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return launch_rope_append(p, static_cast<cudaStream_t>(stream));
}

pkv_status pkv_latent_append(const void *latent, const void *k_rope, pkv_dtype in_dtype, int64_t latent_stride,
                             int64_t k_rope_stride, const void *q_rope, int64_t q_stride, int64_t q_head_stride,
                             const int32_t *positions, const float *table, int max_positions,
                             const int64_t *slot_mapping, int num_tokens, int num_q_heads, int latent_dim,
                             int rope_dim, int block_size, int num_blocks, void *q_out, int64_t q_out_stride,
                             int64_t q_out_head_stride, void *cache, pkv_dtype cache_dtype, int flags,
                             int32_t *status, void *stream)
{
    if (num_q_heads < 0)
        return PKV_ERR_INVALID_ARG;
    if ((latent_dim != 256 && latent_dim != 512) || rope_dim != kRopeDim || !is_float(cache_dtype))
        return PKV_ERR_UNSUPPORTED;
    LatentAppendParams p;
    std::memset(&p, 0, sizeof p);
    const pkv_status rc = check_tokens(p.t, in_dtype, positions, table, rope_dim, max_positions, slot_mapping,
                                       num_tokens, block_size, num_blocks, flags, status);
    if (rc != PKV_OK || num_tokens == 0)
        return rc;
    if (!latent || !k_rope || !cache || (num_q_heads > 0 && (!q_rope || !q_out)))
        return PKV_ERR_INVALID_ARG;
    for (const void *a : {latent, k_rope, q_rope, static_cast<const void *>(q_out), static_cast<const void *>(cache)})
        if (!aligned(a, 16))
            return PKV_ERR_INVALID_ARG;
    if (!stride_ok(latent_stride, latent_dim, in_dtype) || !stride_ok(k_rope_stride, rope_dim, in_dtype))
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        for (const int64_t st : {q_stride, q_head_stride, q_out_stride, q_out_head_stride})
            if (!stride_ok(st, rope_dim, in_dtype))
                return PKV_ERR_INVALID_ARG;
        if (!heads_apart(num_tokens, num_q_heads, q_out_stride, q_out_head_stride, rope_dim))
            return PKV_ERR_INVALID_ARG;
    }
    p.q.q = q_rope;
    p.q.out = q_out;
    p.q.stride = q_stride;
    p.q.head = q_head_stride;
    p.q.out_stride = q_out_stride;
    p.q.out_head = q_out_head_stride;
    p.q.num_heads = num_q_heads;
    if (!in_place_ok(p.q, num_tokens))
        return PKV_ERR_INVALID_ARG;
    p.latent = latent;
    p.k_rope = k_rope;
    p.latent_stride = latent_stride;
    p.k_rope_stride = k_rope_stride;
    p.cache = cache;
    p.cache_dtype = cache_dtype;
    p.latent_dim = latent_dim;
    return launch_latent_append(p, static_cast<cudaStream_t>(stream));
}

// Sizes of a decode call; PKV_OK fills the plan in.
static pkv_status plan_decode(LatentDecodeParams &p, pkv_dtype dtype, int num_seqs, int num_q_heads, int latent_dim,
                              int rope_dim, int block_size, int max_seq_len, size_t *bytes)
{
    if (num_seqs < 0 || num_q_heads <= 0 || max_seq_len < 0)
        return PKV_ERR_INVALID_ARG;
    if (!is_float(dtype) || (latent_dim != 256 && latent_dim != 512) || rope_dim != kRopeDim ||
        block_size != kBlockSize || num_q_heads > 128 || num_seqs > kLatentMaxSeqs)
        return PKV_ERR_UNSUPPORTED;
    // Lengths are rounded up to whole pages and tiles in 32 bits, one clamped to the bound too.
    if (max_seq_len > INT_MAX - kLatentTokens)
        return PKV_ERR_UNSUPPORTED;
    // Tiles are counted in 32 bits, the ends of a team's range included.
    if (static_cast<int64_t>(num_seqs) * (max_seq_len / kLatentTokens + 1) >= INT64_C(1) << 30)
        return PKV_ERR_UNSUPPORTED;
    p.num_seqs = num_seqs;
    p.num_heads = num_q_heads;
    p.latent_dim = latent_dim;
    p.max_len = max_seq_len;
    *bytes = latent_plan(p, dtype);
    return PKV_OK;
}

size_t pkv_latent_attn_workspace_size(pkv_dtype dtype, int num_seqs, int num_q_heads, int latent_dim, int rope_dim,
                                      int block_size, int max_seq_len)
{
    LatentDecodeParams p;
    std::memset(&p, 0, sizeof p);
    size_t bytes = 0;
    return plan_decode(p, dtype, num_seqs, num_q_heads, latent_dim, rope_dim, block_size, max_seq_len, &bytes) ==
                   PKV_OK
               ? (bytes > 256 ? bytes : 256)
               : 0;
}

pkv_status pkv_latent_attn_decode(const void *q, const void *cache, pkv_dtype dtype, const int32_t *block_tables,
                                  const int32_t *seq_lens, int num_seqs, int num_q_heads, int latent_dim,
                                  int rope_dim, int block_size, int num_blocks, int max_blocks_per_seq,
                                  int max_seq_len, float scale, void *out, void *workspace, size_t workspace_bytes,
                                  int32_t *status, int flags, void *stream)
{
    LatentDecodeParams p;
    std::memset(&p, 0, sizeof p);
    size_t bytes = 0;
    const pkv_status rc = plan_decode(p, dtype, num_seqs, num_q_heads, latent_dim, rope_dim, block_size, max_seq_len,
                                      &bytes);
    if (rc != PKV_OK)
        return rc;
    if (num_blocks <= 0 || max_blocks_per_seq <= 0 ||
        max_seq_len > static_cast<int64_t>(max_blocks_per_seq) * block_size || !std::isfinite(scale) ||
        (flags & ~PKV_FLAG_TEST_DROP_FIRST_COPY) != 0 || (flags != 0 && dtype != PKV_BF16))
        return PKV_ERR_INVALID_ARG;
    if (num_blocks > 0x7fffffff / kBlockSize)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0)
        return PKV_OK;
    if (!q || !cache || !block_tables || !seq_lens || !out)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(out, 16) || !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < bytes)
        return PKV_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return PKV_ERR_INVALID_ARG;
    p.q = q;
    p.cache = cache;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.out = out;
    p.status = status;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.score_scale = score_factor(scale);
    p.negate = scale < 0.f ? 1 : 0;
    p.drop_first_copy = (flags & PKV_FLAG_TEST_DROP_FIRST_COPY) ? 1 : 0;
    const size_t rows = latent_part_rows(p);
    p.part = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.part + rows * latent_dim);
    p.pieces = reinterpret_cast<int *>(p.part_ml + rows);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const pkv_status done = dtype == PKV_F32 ? launch_latent_decode_simt(p, st) : launch_latent_decode_tc(p, st);
    return done != PKV_OK ? done : launch_latent_merge(p, dtype, st);
}

pkv_status pkv_latent_prompt_attn(const void *q, const void *k, const void *k_rope, const void *v, pkv_dtype dtype,
                                  int64_t q_stride, int64_t k_stride, int64_t k_head_stride, int64_t k_rope_stride,
                                  int64_t v_stride, int64_t v_head_stride, const int32_t *q_start, int num_seqs,
                                  int num_tokens, int num_heads, int nope_dim, int rope_dim, int max_q_len,
                                  float scale, void *out, int32_t *status, int flags, void *stream)
{
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || max_q_len < 0)
        return PKV_ERR_INVALID_ARG;
    if (!is_float(dtype) || (nope_dim != 64 && nope_dim != 128) || rope_dim != kRopeDim || num_heads > 65535 ||
        num_seqs > kPromptMaxSeqs)
        return PKV_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || (flags & ~PKV_FLAG_TEST_DROP_FIRST_COPY) != 0 || (flags != 0 && dtype != PKV_BF16))
        return PKV_ERR_INVALID_ARG;
    const bool no_rows = num_tokens == 0 || max_q_len == 0;
    if (no_rows && (num_seqs == 0 || !q_start || !status))
        return PKV_OK;
    LatentPromptParams p;
    std::memset(&p, 0, sizeof p);
    p.items.q_start = q_start;
    p.items.status = status;
    p.items.num_seqs = num_seqs;
    p.items.num_tokens = num_tokens;
    if (!aligned(q_start, 4) || !aligned(status, 4))
        return PKV_ERR_INVALID_ARG;
    // A call without rows computes nothing, but its ranges are looked at all the same.
    if (no_rows)
        return launch_prompt_ranges(p.items, static_cast<cudaStream_t>(stream));
    if (num_seqs == 0)
        return PKV_OK;
    if (!q || !k || !k_rope || !v || !q_start || !out)
        return PKV_ERR_INVALID_ARG;
    for (const void *a : {q, k, k_rope, v, static_cast<const void *>(out)})
        if (!aligned(a, 16))
            return PKV_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, static_cast<int64_t>(num_heads) * (nope_dim + rope_dim), dtype) ||
        !stride_ok(k_rope_stride, rope_dim, dtype))
        return PKV_ERR_INVALID_ARG;
    for (const int64_t st : {k_stride, k_head_stride, v_stride, v_head_stride})
        if (!stride_ok(st, nope_dim, dtype))
            return PKV_ERR_INVALID_ARG;
    p.q = q;
    p.k = k;
    p.k_rope = k_rope;
    p.v = v;
    p.out = out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.k_head = k_head_stride;
    p.k_rope_stride = k_rope_stride;
    p.v_stride = v_stride;
    p.v_head = v_head_stride;
    p.nope = nope_dim;
    p.items.num_kv_heads = p.items.num_q_heads = num_heads;
    p.items.group = 1;
    p.items.max_q_len = max_q_len < num_tokens ? max_q_len : num_tokens;
    p.items.score_scale = score_factor(scale);
    p.items.negate = scale < 0.f ? 1 : 0;
    p.drop_first_copy = (flags & PKV_FLAG_TEST_DROP_FIRST_COPY) ? 1 : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_F32 ? launch_latent_prompt_simt(p, st) : launch_latent_prompt_tc(p, st);
}

}  // extern "C"
