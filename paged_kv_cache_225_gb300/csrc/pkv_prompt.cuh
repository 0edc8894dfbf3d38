// Work items of the whole-prompt attention, shared by its kernels.
//
// A row is one (token, grouped query head) pair of a KV head: G rows per
// token, tokens first, so that the rows of one tile read the same K and V.
// An item is a block of `tokens` consecutive tokens of one sequence for one KV
// head.  Item i of a sequence attends about (i + 1) * tokens keys, so items
// are numbered from the costliest down: all sequences' items of the largest
// index, then the next index, KV heads innermost.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

struct PromptItem {
    int s, hkv;  // sequence (-1: no such item), KV head
    int row0, n; // first row of the sequence in q / k / v, its length
    int index;   // item's index in its sequence
};

// Rows [start, end) of sequence s; empty and reported when q_start is not a
// valid range of at most max_q_len rows.
__device__ __forceinline__ int prompt_len(const PromptParams &p, int s, int &start, bool report)
{
    start = __ldg(p.q_start + s);
    const int end = __ldg(p.q_start + s + 1);
    const bool ok = start >= 0 && end >= start && end <= p.num_tokens && end - start <= p.max_q_len;
    if (!ok && report)
        set_status(p.status, PKV_ERR_OUT_OF_RANGE);
    return ok ? end - start : 0;
}

// Items there can be at most (host): every sequence's tokens / `tokens` and one
// more, or the longest's for each of them.
inline long prompt_max_items(const PromptParams &p, long tokens)
{
    const long per_seq = (static_cast<long>(p.max_q_len) + tokens - 1) / tokens;
    const long a = static_cast<long>(p.num_tokens) / tokens + p.num_seqs, b = per_seq * p.num_seqs;
    return (a < b ? a : b) * p.num_kv_heads;
}

// One warp looks items up by number.  With P_s items in sequence s, the items
// of index >= i number C(i) = sum_s max(0, P_s - i) per KV head, so item
// number u has the largest index i with C(i) > u / num_kv_heads: a binary search.
struct PromptScan {
    int top;  // items of the longest sequence

    __device__ __forceinline__ static int items_of(int n, int tokens) { return (n + tokens - 1) / tokens; }

    __device__ unsigned count(const PromptParams &p, int tokens, int index, int lane) const
    {
        unsigned c = 0;
        for (int s = lane; s < p.num_seqs; s += 32) {
            int start;
            c += max(items_of(prompt_len(p, s, start, false), tokens) - index, 0);
        }
        return __reduce_add_sync(kFullMask, c);
    }

    __device__ void init(const PromptParams &p, int tokens, int lane, bool report)
    {
        int t = 0;
        for (int s = lane; s < p.num_seqs; s += 32) {
            int start;
            t = max(t, items_of(prompt_len(p, s, start, report), tokens));
        }
        top = __reduce_max_sync(kFullMask, t);
    }

    // Item number u; s = -1 past the last one.
    __device__ PromptItem find(const PromptParams &p, int tokens, unsigned u, int lane) const
    {
        PromptItem it;
        it.s = -1;
        it.hkv = it.row0 = it.n = it.index = 0;
        const unsigned unit = u / p.num_kv_heads;
        int lo = -1, hi = top;       // C(lo) > unit or lo = -1; C(hi) <= unit
        unsigned above = 0;          // C(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const unsigned c = count(p, tokens, mid, lane);
            if (c > unit) {
                lo = mid;
            } else {
                hi = mid;
                above = c;
            }
        }
        if (lo < 0)
            return it;
        int r = static_cast<int>(unit - above);  // the r-th sequence with an item lo
        it.hkv = static_cast<int>(u - unit * p.num_kv_heads);
        it.index = lo;
        for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
            const int s = s0 + lane;
            int start = 0, n = 0;
            if (s < p.num_seqs)
                n = prompt_len(p, s, start, false);
            const unsigned m = __ballot_sync(kFullMask, items_of(n, tokens) > lo);
            const int c = __popc(m);
            if (r < c) {
                const int at = __fns(m, 0, r + 1);
                it.s = s0 + at;
                it.row0 = __shfl_sync(kFullMask, start, at);
                it.n = __shfl_sync(kFullMask, n, at);
                return it;
            }
            r -= c;
        }
        return it;
    }
};

}  // namespace pkv
