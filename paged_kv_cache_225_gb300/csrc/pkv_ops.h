// Whole-prompt attention and device block tables: what their C ABI
// (pkv_ops_api.cu) hands to the kernel units.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Causal attention over whole prompts.  Sequence s is rows q_start[s] ..
// q_start[s + 1] - 1 of q, k, v and out; row i attends rows 0 .. i of it.
struct PromptParams {
    const void *q;           // [T, Hq, D], rows q_stride elements apart
    const void *k;           // [T, Hkv, D]
    const void *v;
    const int32_t *q_start;  // [S + 1]
    void *out;               // [T, Hq, D]
    int32_t *status;         // optional
    int64_t q_stride, k_stride, v_stride;  // elements
    int dtype, out_dtype;
    int num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, group;
    int max_q_len;           // bound on a sequence's rows
    unsigned max_items;      // bound on the work items of a valid q_start (set at launch)
    float score_scale;       // |scale| * log2(e), at least 2^-120
    int negate;              // scale < 0: the kernels negate the scores
    int drop_first_copy;     // test hook: never issue the first copy of CTA 0
    int slow_gate;           // test hook: the warp that watches the loads looks 20 us late
};

// Every look-up of an item may walk all row starts once per cost class (2^20 of
// them, most empty: 10 ms a class, and a 32K prompt has some 20 classes), while
// the bf16 kernel's other roles wait for at most a second.
constexpr int kPromptMaxSeqs = 1 << 20;

// One scheduling step of a page pool kept in device memory.
struct TablesParams {
    const int32_t *drop_lens;  // [S] or null
    const int32_t *new_lens;   // [S] or null
    int32_t *seq_lens;         // [S]
    int32_t *block_tables;     // [S, max_blocks]
    int32_t *ref_counts;       // [num_blocks]
    int num_seqs, max_blocks, num_blocks, max_tokens;
    int32_t *q_start;          // [S + 1] or null
    int64_t *slot_mapping;     // [max_tokens]
    int wide_slots;            // slot_mapping is 16-byte aligned
    int32_t *copy_pairs;       // [S, 2] or null
    int32_t *status;           // optional
};
constexpr int kTablesMaxRows = 8192;  // rows whose prefix sums fit shared memory
constexpr int kTablesRowBytes = 16;   // shared memory per row

// Each launches on `stream` and returns a status, as the units of pkv_internal.h.
pkv_status launch_prompt_simt(const PromptParams &p, cudaStream_t stream);  // fp32
pkv_status launch_prompt_tc(const PromptParams &p, cudaStream_t stream);    // bf16
// Row ranges alone, for calls without a row to attend: invalid ones are reported.
pkv_status launch_prompt_ranges(const PromptParams &p, cudaStream_t stream);
pkv_status launch_tables_step(const TablesParams &p, cudaStream_t stream);
pkv_status launch_tables_fork(const int32_t *pairs, int num_pairs, int32_t *seq_lens,
                              int32_t *block_tables, int32_t *ref_counts, int num_seqs,
                              int max_blocks, int num_blocks, int32_t *status, cudaStream_t stream);

}  // namespace pkv
