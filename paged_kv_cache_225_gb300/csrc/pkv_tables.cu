// Block tables, cache slots and page reference counts kept on the GPU.
//
// The same bookkeeping as the host block manager ("Inference optimization"
// lesson, section "PagedAttention": a page table per request, pages anywhere,
// shared pages stored once and copied when a request diverges; "Continuous
// Batching e PagedAttention no vLLM", section 3), on tensors that stay in
// device memory, so that a scheduling step needs no host round trip and can
// be part of a CUDA graph.
//
// With kept_s = L_s - min(drop_s, L_s), pages(x) = ceil(x / 16) and copy_s = 1
// for a row whose part-filled last page has other holders left (row order
// decides which of them is the last, who writes in place), row s takes
//   need_s = pages(kept_s + n_s) - pages(kept_s) + copy_s   (0 when n_s = 0)
// pages, and the r-th page taken in row order is the r-th lowest id whose
// count is zero.  Both orders are prefix sums: over the rows in shared memory,
// over the pool by counting zero counts per warp and ranking them by ballot.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// Inclusive prefix sum over the block; *total is the block's sum.  `part`
// holds kWarps entries and is free to be reused on return.
__device__ unsigned long long block_scan(unsigned long long x, unsigned long long *part,
                                         unsigned long long *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFullMask, x, d);
        if (lane >= d)
            x += y;
    }
    if (lane == 31)
        part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        unsigned long long p = part[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long y = __shfl_up_sync(kFullMask, p, d);
            if (lane >= d)
                p += y;
        }
        part[lane] = p;
    }
    __syncthreads();
    if (warp > 0)
        x += part[warp - 1];
    *total = part[kWarps - 1];
    __syncthreads();
    return x;
}

// First row whose inclusive end lies above i (ends is non-decreasing).
__device__ __forceinline__ int row_of(const int *ends, int n, int i)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Ids in [lo, lo + 32) whose count is zero, as a lane mask.
__device__ __forceinline__ unsigned zero_mask(const int32_t *ref, int lo, int hi, int lane)
{
    const int p = lo + lane;
    return __ballot_sync(kFullMask, p < hi && __ldcg(ref + p) == 0);
}

__global__ void __launch_bounds__(kThreads, 1) tables_step_kernel(const TablesParams p)
{
    extern __shared__ int rows_smem[];
    __shared__ unsigned long long s_part[kWarps];
    __shared__ int s_warp_base[kWarps + 1];
    __shared__ int s_bad;
    const int S = p.num_seqs;
    int *tok_end = rows_smem;                                        // tokens reserved, inclusive
    int *page_end = tok_end + S;                                     // pages taken, inclusive
    unsigned *kept2 = reinterpret_cast<unsigned *>(page_end + S);    // 2 * kept + copy
    int *shared_last = reinterpret_cast<int *>(kept2 + S);           // shared part-filled last page
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int max_len = p.max_blocks * kBlockSize;
    const size_t width = p.max_blocks;

    if (threadIdx.x == 0)
        s_bad = 0;

    // Drops, a warp per row.
    if (p.drop_lens) {
        for (int s = warp; s < S; s += kWarps) {
            const int L = p.seq_lens[s], d = __ldg(p.drop_lens + s);
            if (L < 0 || L > max_len || d < 0) {
                if (lane == 0)
                    set_status(p.status, PKV_ERR_OUT_OF_RANGE);
                continue;
            }
            int32_t *row = p.block_tables + s * width;
            for (int j = pages_of(L - min(d, L)) + lane; j < pages_of(L); j += 32) {
                const int32_t page = row[j];
                bool ok = page >= 0 && page < p.num_blocks;
                if (ok && atomicSub(p.ref_counts + page, 1) <= 0) {
                    atomicAdd(p.ref_counts + page, 1);  // nobody held it: put it back
                    ok = false;
                }
                if (!ok)
                    set_status(p.status, PKV_ERR_OUT_OF_RANGE);
                row[j] = -1;
            }
        }
    }
    __syncthreads();

    // Rows: what is kept, and which part-filled last pages are shared.
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int L = p.seq_lens[s], d = p.drop_lens ? __ldg(p.drop_lens + s) : 0;
        const int n = p.new_lens ? __ldg(p.new_lens + s) : 0;
        const bool len_ok = L >= 0 && L <= max_len;
        const int kept = len_ok ? L - (d > 0 ? min(d, L) : 0) : 0;
        bool bad = !len_ok || n < 0 || n > max_len - kept;
        int shared = -1;
        if (!bad && n > 0 && kept % kBlockSize != 0) {
            const int32_t page = p.block_tables[s * width + pages_of(kept) - 1];
            const int refs = page >= 0 && page < p.num_blocks ? __ldcg(p.ref_counts + page) : 0;
            bad = refs <= 0;
            if (refs > 1)
                shared = page;
        }
        kept2[s] = 2u * static_cast<unsigned>(kept);
        shared_last[s] = shared;
        if (bad)
            s_bad = 1;
    }
    __syncthreads();
    // A sharing row copies unless every other holder of the page is an
    // earlier row that has copied already.
    bool want_pair = false;
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int page = shared_last[s];
        if (page < 0)
            continue;
        const int others = __ldcg(p.ref_counts + page) - 1;
        int before = 0;
        for (int t = 0; t < s && before < others; ++t)
            before += shared_last[t] == page;
        if (before < others) {
            kept2[s] |= 1u;
            want_pair = true;
        }
    }
    if (want_pair && !p.copy_pairs)
        s_bad = 1;
    // Prefix sums of the tokens and pages, 1024 rows at a time.
    unsigned long long tokens = 0, pages = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        unsigned long long n = 0, need = 0;
        if (s < S) {
            const int kept = static_cast<int>(kept2[s] >> 1);
            const int nn = p.new_lens ? __ldg(p.new_lens + s) : 0;
            if (nn > 0 && nn <= max_len - kept) {
                n = nn;
                need = pages_of(kept + nn) - pages_of(kept) + (kept2[s] & 1u);
            }
        }
        unsigned long long sum;
        const unsigned long long te = tokens + block_scan(n, s_part, &sum);
        tokens += sum;
        const unsigned long long pe = pages + block_scan(need, s_part, &sum);
        pages += sum;
        if (s < S) {  // read only when both totals fit an int (checked below)
            tok_end[s] = static_cast<int>(te);
            page_end[s] = static_cast<int>(pe);
        }
    }

    // Zero counts per warp, each over a contiguous range of the pool.
    const int per_warp = (p.num_blocks / kWarps + 32) & ~31;
    const int lo = static_cast<int>(min(static_cast<long>(warp) * per_warp, static_cast<long>(p.num_blocks)));
    const int hi = static_cast<int>(min(static_cast<long>(lo) + per_warp, static_cast<long>(p.num_blocks)));
    int zeros = 0;
    for (int b = lo; b < hi; b += 32)
        zeros += __popc(zero_mask(p.ref_counts, b, hi, lane));
    if (lane == 0)
        s_warp_base[warp + 1] = zeros;
    __syncthreads();
    if (threadIdx.x == 0) {
        s_warp_base[0] = 0;
        for (int w = 0; w < kWarps; ++w)
            s_warp_base[w + 1] += s_warp_base[w];
    }
    __syncthreads();
    const bool enough = pages <= static_cast<unsigned long long>(s_warp_base[kWarps]);
    const bool bad = s_bad || tokens > static_cast<unsigned long long>(p.max_tokens);
    const bool ok = !bad && enough;
    if (!ok && threadIdx.x == 0)
        set_status(p.status, bad ? PKV_ERR_OUT_OF_RANGE : PKV_ERR_NO_BLOCKS);
    const int total = ok ? static_cast<int>(tokens) : 0;
    const int taken = ok ? static_cast<int>(pages) : 0;

    if (p.copy_pairs)
        for (int s = threadIdx.x; s < S; s += kThreads)
            if (!ok || !(kept2[s] & 1u))
                p.copy_pairs[2 * s] = p.copy_pairs[2 * s + 1] = -1;
    // Hand out the pages: the r-th zero count goes to the row that owns r.
    int rank = s_warp_base[warp];
    for (int b = lo; b < hi && rank < taken; b += 32) {
        const unsigned m = zero_mask(p.ref_counts, b, hi, lane);
        const int r = rank + __popc(m & ((1u << lane) - 1u));
        if ((m >> lane & 1u) && r < taken) {
            const int s = row_of(page_end, S, r);
            const int j = r - (s ? page_end[s - 1] : 0);
            const unsigned k2 = kept2[s];
            const int copy = k2 & 1u;
            int32_t *entry = p.block_tables + s * width + pages_of(static_cast<int>(k2 >> 1)) - copy + j;
            if (copy && j == 0) {
                const int32_t src = *entry;
                p.copy_pairs[2 * s] = src;
                p.copy_pairs[2 * s + 1] = b + lane;
                atomicSub(p.ref_counts + src, 1);  // at least one holder is left
            }
            *entry = b + lane;
            p.ref_counts[b + lane] = 1;
        }
        rank += __popc(m);
    }
    __syncthreads();

    // Slots of the reserved tokens (-1 past them), row starts, lengths.
    for (int i = threadIdx.x; i < p.max_tokens; i += kThreads) {
        int64_t slot = -1;
        if (i < total) {
            const int s = row_of(tok_end, S, i);
            const int pos = static_cast<int>(kept2[s] >> 1) + i - (s ? tok_end[s - 1] : 0);
            const int32_t page = __ldcg(p.block_tables + s * width + pos / kBlockSize);
            slot = static_cast<int64_t>(page) * kBlockSize + pos % kBlockSize;
        }
        p.slot_mapping[i] = slot;
    }
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int end = ok ? tok_end[s] : 0;
        const int n = ok ? end - (s ? tok_end[s - 1] : 0) : 0;
        if (p.q_start)
            p.q_start[s + 1] = end;
        const int L = p.seq_lens[s];
        if (L >= 0 && L <= max_len)
            p.seq_lens[s] = static_cast<int>(kept2[s] >> 1) + n;
    }
    if (p.q_start && threadIdx.x == 0)
        p.q_start[0] = 0;
}

// One CTA per (parent, child) pair.
constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads)
    tables_fork_kernel(const int32_t *pairs, int num_pairs, int32_t *seq_lens,
                       int32_t *block_tables, int32_t *ref_counts, int num_seqs, int max_blocks,
                       int num_blocks, int32_t *status)
{
    const int i = blockIdx.x;
    const int parent = __ldg(pairs + 2 * i), child = __ldg(pairs + 2 * i + 1);
    if (parent < 0 && child < 0)
        return;  // padding
    bool bad = parent < 0 || child < 0 || parent >= num_seqs || child >= num_seqs;
    // A child is nobody's parent in this call and listed once: its row is
    // written by this CTA alone, and the parent's row by none.
    for (int t = threadIdx.x; t < num_pairs; t += kForkThreads)
        bad = bad || __ldg(pairs + 2 * t) == child || (t < i && __ldg(pairs + 2 * t + 1) == child);
    bad = __syncthreads_or(bad);
    int L = 0;
    if (!bad) {
        L = __ldcg(seq_lens + parent);
        bad = L < 0 || L > max_blocks * kBlockSize || __ldcg(seq_lens + child) != 0;
    }
    __syncthreads();  // every thread has read the child's length
    if (bad) {
        if (threadIdx.x == 0)
            set_status(status, PKV_ERR_OUT_OF_RANGE);
        return;
    }
    const int32_t *src = block_tables + static_cast<size_t>(parent) * max_blocks;
    int32_t *dst = block_tables + static_cast<size_t>(child) * max_blocks;
    for (int j = threadIdx.x; j < pages_of(L); j += kForkThreads) {
        int32_t page = src[j];
        bool ok = page >= 0 && page < num_blocks;
        if (ok && atomicAdd(ref_counts + page, 1) <= 0) {
            atomicSub(ref_counts + page, 1);  // not a held page: nothing to share
            ok = false;
        }
        if (!ok) {
            set_status(status, PKV_ERR_OUT_OF_RANGE);
            page = -1;
        }
        dst[j] = page;
    }
    if (threadIdx.x == 0)
        seq_lens[child] = L;
}

}  // namespace

pkv_status launch_tables_step(const TablesParams &p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(tables_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kTablesMaxRows * kTablesRowBytes) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    tables_step_kernel<<<1, kThreads, static_cast<size_t>(p.num_seqs) * kTablesRowBytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status launch_tables_fork(const int32_t *pairs, int num_pairs, int32_t *seq_lens,
                              int32_t *block_tables, int32_t *ref_counts, int num_seqs,
                              int max_blocks, int num_blocks, int32_t *status, cudaStream_t stream)
{
    tables_fork_kernel<<<static_cast<unsigned>(num_pairs), kForkThreads, 0, stream>>>(
        pairs, num_pairs, seq_lens, block_tables, ref_counts, num_seqs, max_blocks, num_blocks,
        status);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
