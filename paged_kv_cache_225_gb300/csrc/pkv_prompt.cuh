// Work items of the whole-prompt attention, shared by its kernels.
//
// A row is one (token, grouped query head) pair of a KV head: G rows per
// token, tokens first, so that the rows of one tile read the same K and V.
// An item is a block of `tokens` consecutive tokens of one sequence for one KV
// head.  Block i of a sequence attends about (i + 1) * tokens keys.  Items are
// numbered by falling cost: in classes of block indices [3/4 h, h), from the
// longest sequence's last block down, in a class sequence by sequence from the
// largest index to the smallest, KV heads innermost.  CTAs that take items
// from such a list in turn end within about one short item of each other
// (sixteen prompts of 512 to 4096 tokens on the tensor cores, same box: 575 us,
// sequence after sequence 646 us).
#pragma once

#include "pkv_common.cuh"
#include "pkv_ops.h"

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
// more, or the longest's for each of them.  Row starts that step back can
// make sequences that overlap, and any number of items: the look-up stops at
// this bound.
inline long prompt_max_items(const PromptParams &p, long tokens)
{
    const long per_seq = (static_cast<long>(p.max_q_len) + tokens - 1) / tokens;
    const long a = static_cast<long>(p.num_tokens) / tokens + p.num_seqs, b = per_seq * p.num_seqs;
    return (a < b ? a : b) * p.num_kv_heads;
}

// One warp looks items up by ascending number.  It stands at one class and 32
// sequences, a lane each, and moves on when their items are used up: a CTA's
// look-ups together read q_start once per class (about log_4/3 of the longest
// sequence's items).
struct PromptScan {
    int lo = 0, hi = 0;   // the class: block indices lo .. hi - 1
    int s0 = 0;           // first of the 32 sequences
    unsigned before = 0;  // items (per KV head) ahead of them
    unsigned here = 0;    // and theirs
    int start, n;         // this lane's sequence
    unsigned upto;        // items in the class of the lanes up to this one

    __device__ __forceinline__ void load(const PromptParams &p, int tokens, int lane)
    {
        const int s = s0 + lane;
        start = n = 0;
        if (s < p.num_seqs)
            n = prompt_len(p, s, start, false);
        upto = max(min((n + tokens - 1) / tokens, hi) - lo, 0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(kFullMask, upto, d);
            if (lane >= d)
                upto += y;
        }
        here = __shfl_sync(kFullMask, upto, 31);
    }

    // `report`: invalid ranges are recorded.
    __device__ __forceinline__ void init(const PromptParams &p, int tokens, int lane, bool report)
    {
        int top = 0;
        for (int s = lane; s < p.num_seqs; s += 32) {
            int at;
            top = max(top, (prompt_len(p, s, at, report) + tokens - 1) / tokens);
        }
        lo = __reduce_max_sync(kFullMask, top);
        s0 = p.num_seqs;  // past the sequences of an empty class
    }

    // Item number u (not below an earlier u); s = -1 past the last one.
    __device__ PromptItem find(const PromptParams &p, int tokens, unsigned u, int lane)
    {
        PromptItem it;
        it.s = -1;
        it.hkv = it.row0 = it.n = it.index = 0;
        if (u >= p.max_items)
            return it;
        const unsigned unit = u / p.num_kv_heads;
        while (unit >= before + here) {
            before += here;
            here = 0;
            s0 += 32;
            if (s0 >= p.num_seqs) {
                if (lo == 0)
                    return it;
                hi = lo;
                lo = min(hi - 1, hi * 3 / 4);
                s0 = 0;
            }
            load(p, tokens, lane);
        }
        const unsigned r = unit - before;
        const int at = __ffs(__ballot_sync(kFullMask, upto > r)) - 1;
        it.s = s0 + at;
        it.hkv = static_cast<int>(u - unit * p.num_kv_heads);
        it.row0 = __shfl_sync(kFullMask, start, at);
        it.n = __shfl_sync(kFullMask, n, at);
        // Its last item in the class comes last.
        it.index = lo + static_cast<int>(__shfl_sync(kFullMask, upto, at) - 1 - r);
        return it;
    }
};

}  // namespace pkv
