// C ABI of the whole-prompt attention and of the device block tables
// (declared in include/pkv.h): argument validation and dispatch.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "pkv_ops.h"

using namespace pkv;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes that the table calls share.
bool tables_sizes_ok(int num_seqs, int max_blocks_per_seq, int num_blocks)
{
    // A row's tokens stay below 2^30.
    return num_seqs >= 0 && num_blocks > 0 && max_blocks_per_seq > 0 &&
           max_blocks_per_seq <= (1 << 26) - 1;
}

}  // namespace

extern "C" {

pkv_status pkv_prompt_attn(const void *q, const void *k, const void *v, pkv_dtype dtype,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           const int32_t *q_start, int num_seqs, int num_tokens, int num_q_heads,
                           int num_kv_heads, int head_dim, int max_q_len, float scale, void *out,
                           pkv_dtype out_dtype, int32_t *status, int flags, void *stream)
{
    if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_q_len < 0 ||
        num_q_heads % num_kv_heads != 0)
        return PKV_ERR_INVALID_ARG;
    if ((dtype != PKV_F32 && dtype != PKV_BF16) || (out_dtype != PKV_F32 && out_dtype != PKV_BF16))
        return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128)
        return PKV_ERR_UNSUPPORTED;
    if (num_q_heads / num_kv_heads > 16 || num_seqs > kPromptMaxSeqs)
        return PKV_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || (flags & ~(PKV_FLAG_TEST_DROP_FIRST_COPY | PKV_FLAG_TEST_SLOW_GATE)) != 0 ||
        (flags != 0 && dtype != PKV_BF16))
        return PKV_ERR_INVALID_ARG;
    // A call without rows computes nothing, but its ranges are looked at all the same.
    const bool no_rows = num_tokens == 0 || max_q_len == 0;
    if (num_seqs == 0 || (no_rows && (!status || !q_start)))
        return PKV_OK;
    if (no_rows) {
        if (!aligned(q_start, 4) || !aligned(status, 4))
            return PKV_ERR_INVALID_ARG;
        PromptParams p;
        std::memset(&p, 0, sizeof p);
        p.q_start = q_start;
        p.status = status;
        p.num_seqs = num_seqs;
        p.num_tokens = num_tokens;
        return launch_prompt_ranges(p, static_cast<cudaStream_t>(stream));
    }
    if (!q || !k || !v || !q_start || !out)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(q_start, 4) || (status && !aligned(status, 4)))
        return PKV_ERR_INVALID_ARG;
    // Rows that do not overlap and start on 16-byte boundaries.
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
    const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    const int64_t unit = dtype == PKV_F32 ? 4 : 8;
    const int64_t limit = int64_t{1} << 36;  // elements: the byte stride stays below 2^40
    for (const int64_t st : {q_stride, k_stride, v_stride})
        if (st % unit != 0 || st >= limit)
            return PKV_ERR_INVALID_ARG;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
        return PKV_ERR_INVALID_ARG;
    PromptParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_start = q_start;
    p.out = out;
    p.status = status;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.dtype = dtype;
    p.out_dtype = out_dtype;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.group = num_q_heads / num_kv_heads;
    p.max_q_len = max_q_len < num_tokens ? max_q_len : num_tokens;
    // The kernels work with a positive factor: the sign is applied to Q (or the
    // score), and a zero becomes a factor too small to tell weights apart, which
    // keeps masked scores (-inf) out all the same.
    const float factor = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
    const float least = std::ldexp(1.0f, -120), most = std::ldexp(1.0f, 127);
    p.score_scale = factor < least ? least : factor > most ? most : factor;
    p.negate = scale < 0.f ? 1 : 0;
    p.drop_first_copy = (flags & PKV_FLAG_TEST_DROP_FIRST_COPY) ? 1 : 0;
    p.slow_gate = (flags & PKV_FLAG_TEST_SLOW_GATE) ? 1 : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? launch_prompt_tc(p, st) : launch_prompt_simt(p, st);
}

pkv_status pkv_tables_step(int32_t *seq_lens, int32_t *block_tables, int32_t *ref_counts,
                           int num_seqs, int max_blocks_per_seq, int block_size, int num_blocks,
                           const int32_t *drop_lens, const int32_t *new_lens, int32_t *q_start,
                           int64_t *slot_mapping, int max_tokens, int32_t *copy_pairs,
                           int32_t *status, void *stream)
{
    if (!tables_sizes_ok(num_seqs, max_blocks_per_seq, num_blocks) || max_tokens < 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != kBlockSize || num_seqs > kTablesMaxRows)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 && max_tokens == 0 && !q_start)
        return PKV_OK;
    if (!ref_counts || (num_seqs > 0 && (!seq_lens || !block_tables)))
        return PKV_ERR_INVALID_ARG;
    if (max_tokens > 0 && !slot_mapping)
        return PKV_ERR_INVALID_ARG;
    for (const void *a : {static_cast<const void *>(seq_lens), static_cast<const void *>(block_tables),
                          static_cast<const void *>(drop_lens), static_cast<const void *>(new_lens),
                          static_cast<const void *>(q_start), static_cast<const void *>(copy_pairs),
                          static_cast<const void *>(status)})
        if (!aligned(a, 4))
            return PKV_ERR_INVALID_ARG;
    if (!aligned(ref_counts, 16) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    TablesParams p;
    std::memset(&p, 0, sizeof p);
    p.drop_lens = num_seqs > 0 ? drop_lens : nullptr;
    p.new_lens = new_lens;
    p.seq_lens = seq_lens;
    p.block_tables = block_tables;
    p.ref_counts = ref_counts;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.max_tokens = max_tokens;
    p.q_start = q_start;
    p.slot_mapping = slot_mapping;
    p.wide_slots = aligned(slot_mapping, 16) ? 1 : 0;
    p.copy_pairs = copy_pairs;
    p.status = status;
    return launch_tables_step(p, static_cast<cudaStream_t>(stream));
}

pkv_status pkv_tables_fork(const int32_t *pairs, int num_pairs, int32_t *seq_lens,
                           int32_t *block_tables, int32_t *ref_counts, int num_seqs,
                           int max_blocks_per_seq, int block_size, int num_blocks,
                           int32_t *status, void *stream)
{
    if (!tables_sizes_ok(num_seqs, max_blocks_per_seq, num_blocks) || num_pairs < 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != kBlockSize)
        return PKV_ERR_UNSUPPORTED;
    if (num_pairs == 0)
        return PKV_OK;
    if (!pairs || !seq_lens || !block_tables || !ref_counts)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(pairs, 4) || !aligned(seq_lens, 4) || !aligned(block_tables, 4) ||
        !aligned(ref_counts, 4) || (status && !aligned(status, 4)))
        return PKV_ERR_INVALID_ARG;
    return launch_tables_fork(pairs, num_pairs, seq_lens, block_tables, ref_counts, num_seqs,
                              max_blocks_per_seq, num_blocks, status,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
