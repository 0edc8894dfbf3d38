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
// CTAs of the cluster: the largest there is, which was never slower than fewer
// (us a step on 1 / 4 / 16: 128 rows of a 31K-page pool 17.2 / 11.9 / 10.7, 64
// prompts admitted 120.7 / 37.8 / 18.3, 512 rows of a 288K-page pool 154.9 /
// 53.1 / 22.1).
constexpr int kStepCtas = 16;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// Orders every CTA's accesses (shared and global) before the barrier with
// those after it.  A cluster of one needs only the block's barrier.
__device__ __forceinline__ void sync_all(int ctas)
{
    if (ctas == 1) {
        __syncthreads();
        return;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive prefix sums of a pair over the block; *ta, *tb are the block's
// sums.  `part` holds 2 * kWarps entries and is free to be reused on return.
__device__ void block_scan2(unsigned long long &a, unsigned long long &b, unsigned long long *part,
                            unsigned long long *ta, unsigned long long *tb)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFullMask, a, d);
        const unsigned long long z = __shfl_up_sync(kFullMask, b, d);
        if (lane >= d) {
            a += y;
            b += z;
        }
    }
    if (lane == 31) {
        part[warp] = a;
        part[kWarps + warp] = b;
    }
    __syncthreads();
    if (warp < 2) {
        unsigned long long p = part[kWarps * warp + lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long y = __shfl_up_sync(kFullMask, p, d);
            if (lane >= d)
                p += y;
        }
        part[kWarps * warp + lane] = p;
    }
    __syncthreads();
    if (warp > 0) {
        a += part[warp - 1];
        b += part[kWarps + warp - 1];
    }
    *ta = part[kWarps - 1];
    *tb = part[2 * kWarps - 1];
    __syncthreads();
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

// Which of the four counts from id on are zero (bits 0..3); ids from `end` on
// are not.  id is a multiple of 4 and the counts are 16-byte aligned.
__device__ __forceinline__ unsigned zeros4(const int32_t *ref, long id, long end)
{
    if (id + 4 <= end) {
        const int4 v = __ldcg(reinterpret_cast<const int4 *>(ref + id));
        return (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
    }
    unsigned m = 0;
    for (int c = 0; c < 4; ++c)
        m |= (id + c < end && __ldcg(ref + id + c) == 0 ? 1u : 0u) << c;
    return m;
}

constexpr int kStep = 4;  // loads of 128 counts a warp has in flight

// A cluster of CTAs runs the whole step: the pool's counts and the rows' pages
// and slots are spread over the cluster's warps, the (small) row sums are
// computed by every CTA for itself, and three cluster barriers separate drops,
// counting, handing out and writing slots.  All of it is a few dependent trips
// to L2: bound by latency, not by bytes.
__global__ void __launch_bounds__(kThreads, 1) tables_step_kernel(const TablesParams p, int ctas)
{
    extern __shared__ int rows_smem[];
    __shared__ unsigned long long s_part[2 * kWarps];
    __shared__ int s_warp_base[kWarps + 1];
    __shared__ int s_zeros[kStepCtas];  // zero counts of every CTA's part of the pool
    __shared__ int s_bad;
    const int S = p.num_seqs;
    int *tok_end = rows_smem;                                        // tokens reserved, inclusive
    int *page_end = tok_end + S;                                     // pages taken, inclusive
    unsigned *kept2 = reinterpret_cast<unsigned *>(page_end + S);    // 2 * kept + copy
    int *shared_last = reinterpret_cast<int *>(kept2 + S);           // shared part-filled last page
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = blockIdx.x;  // the grid is one cluster
    const int max_len = p.max_blocks * kBlockSize;
    const size_t width = p.max_blocks;

    if (threadIdx.x == 0)
        s_bad = 0;

    // Drops: as many warps per row as there are for all rows.
    if (p.drop_lens) {
        const int per_row = max(1, ctas * kWarps / S);
        const int gw = cta * kWarps + warp;
        const int sub = gw % per_row;
        for (int s = gw / per_row; s < S; s += ctas * kWarps / per_row) {
            if (gw / per_row >= ctas * kWarps / per_row)
                break;  // warps left over
            const int L = __ldcg(p.seq_lens + s), d = __ldg(p.drop_lens + s);
            if (L < 0 || L > max_len || d < 0) {
                if (lane == 0 && sub == 0)
                    set_status(p.status, PKV_ERR_OUT_OF_RANGE);
                continue;
            }
            int32_t *row = p.block_tables + s * width;
            const int last = pages_of(L);
            for (int j0 = pages_of(L - min(d, L)) + sub * 32 + lane; j0 < last;
                 j0 += kStep * 32 * per_row) {
                int32_t page[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int j = j0 + i * 32 * per_row;
                    page[i] = j < last ? __ldcg(row + j) : -1;
                }
                bool bad = false;
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int j = j0 + i * 32 * per_row;
                    if (j >= last)
                        continue;
                    row[j] = -1;
                    bool ok = page[i] >= 0 && page[i] < p.num_blocks;
                    if (ok && atomicSub(p.ref_counts + page[i], 1) <= 0) {
                        atomicAdd(p.ref_counts + page[i], 1);  // nobody held it: put it back
                        ok = false;
                    }
                    bad = bad || !ok;
                }
                if (bad)
                    set_status(p.status, PKV_ERR_OUT_OF_RANGE);
            }
        }
    }
    sync_all(ctas);  // also: every CTA runs, before its shared memory is written

    // Zero counts: the pool in ranges of `per_warp` ids, one per warp of the
    // cluster, in order.
    const long per_warp = (p.num_blocks / (ctas * kWarps) + 128) & ~127;
    const long lo = min(static_cast<long>(cta * kWarps + warp) * per_warp, static_cast<long>(p.num_blocks));
    const long hi = min(lo + per_warp, static_cast<long>(p.num_blocks));
    int zeros = 0;
    for (long b = lo; b < hi; b += 128 * kStep) {
        unsigned m[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            m[i] = zeros4(p.ref_counts, min(b + 128 * i + 4 * lane, hi), hi);
#pragma unroll
        for (int i = 0; i < kStep; ++i)
            zeros += __popc(m[i]);
    }
    zeros = __reduce_add_sync(kFullMask, zeros);
    if (lane == 0)
        s_warp_base[warp + 1] = zeros;

    // Rows: what is kept, and which part-filled last pages are shared.
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int L = __ldcg(p.seq_lens + s), d = p.drop_lens ? __ldg(p.drop_lens + s) : 0;
        const int n = p.new_lens ? __ldg(p.new_lens + s) : 0;
        const bool len_ok = L >= 0 && L <= max_len;
        const int kept = len_ok ? L - (d > 0 ? min(d, L) : 0) : 0;
        bool bad = !len_ok || n < 0 || n > max_len - kept;
        int shared = -1;
        if (!bad && n > 0 && kept % kBlockSize != 0) {
            const int32_t page = __ldcg(p.block_tables + s * width + pages_of(kept) - 1);
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
    if (threadIdx.x < 32) {  // this CTA's zero counts: per-warp bases, total to every CTA
        int z = s_warp_base[lane + 1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFullMask, z, d);
            if (lane >= d)
                z += y;
        }
        s_warp_base[lane + 1] = z;
        if (lane == 0)
            s_warp_base[0] = 0;
        const int all = __shfl_sync(kFullMask, z, 31);
        if (lane < ctas) {
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(remote)
                         : "r"(smem_u32(&s_zeros[cta])), "r"(lane));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(all) : "memory");
        }
    }
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
        unsigned long long sum_n, sum_need;
        block_scan2(n, need, s_part, &sum_n, &sum_need);
        if (s < S) {  // read only when both totals fit an int (checked below)
            tok_end[s] = static_cast<int>(tokens + n);
            page_end[s] = static_cast<int>(pages + need);
        }
        tokens += sum_n;
        pages += sum_need;
    }
    sync_all(ctas);

    int rank = s_warp_base[warp];
    int total_zeros = 0;
    for (int c = 0; c < ctas; ++c) {
        const int z = s_zeros[c];
        rank += c < cta ? z : 0;
        total_zeros += z;
    }
    const bool enough = pages <= static_cast<unsigned long long>(total_zeros);
    const bool bad = s_bad || tokens > static_cast<unsigned long long>(p.max_tokens);
    const bool ok = !bad && enough;
    if (!ok && cta == 0 && threadIdx.x == 0)
        set_status(p.status, bad ? PKV_ERR_OUT_OF_RANGE : PKV_ERR_NO_BLOCKS);
    const int total = ok ? static_cast<int>(tokens) : 0;
    const int taken = ok ? static_cast<int>(pages) : 0;

    const int thread = cta * kThreads + threadIdx.x, threads = ctas * kThreads;
    if (p.copy_pairs)
        for (int s = thread; s < S; s += threads)
            if (!ok || !(kept2[s] & 1u))
                p.copy_pairs[2 * s] = p.copy_pairs[2 * s + 1] = -1;
    // Hand out the pages: the r-th zero count goes to the row that owns r.
    for (long b = lo; b < hi && rank < taken; b += 128) {
        unsigned m = zeros4(p.ref_counts, min(b + 4 * lane, hi), hi);
        const int c = __popc(m);
        int upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFullMask, upto, d);
            if (lane >= d)
                upto += y;
        }
        for (int r = rank + upto - c; m && r < taken; ++r, m &= m - 1) {
            const int32_t page = static_cast<int32_t>(b) + 4 * lane + __ffs(m) - 1;
            const int s = row_of(page_end, S, r);
            const int j = r - (s ? page_end[s - 1] : 0);
            const unsigned k2 = kept2[s];
            const int copy = k2 & 1u;
            int32_t *entry = p.block_tables + s * width + pages_of(static_cast<int>(k2 >> 1)) - copy + j;
            if (copy && j == 0) {
                const int32_t src = __ldcg(entry);
                p.copy_pairs[2 * s] = src;
                p.copy_pairs[2 * s + 1] = page;
                atomicSub(p.ref_counts + src, 1);  // at least one holder is left
            }
            *entry = page;
            p.ref_counts[page] = 1;
        }
        rank += __shfl_sync(kFullMask, upto, 31);
    }
    sync_all(ctas);

    // Slots of the reserved tokens (-1 past them), row starts, lengths.
    for (int i = thread; i < p.max_tokens; i += threads) {
        int64_t slot = -1;
        if (i < total) {
            const int s = row_of(tok_end, S, i);
            const int pos = static_cast<int>(kept2[s] >> 1) + i - (s ? tok_end[s - 1] : 0);
            const int32_t page = __ldcg(p.block_tables + s * width + pos / kBlockSize);
            slot = static_cast<int64_t>(page) * kBlockSize + pos % kBlockSize;
        }
        p.slot_mapping[i] = slot;
    }
    for (int s = thread; s < S; s += threads) {
        const int end = ok ? tok_end[s] : 0;
        const int n = ok ? end - (s ? tok_end[s - 1] : 0) : 0;
        if (p.q_start)
            p.q_start[s + 1] = end;
        const int L = __ldcg(p.seq_lens + s);
        if (L >= 0 && L <= max_len)
            p.seq_lens[s] = static_cast<int>(kept2[s] >> 1) + n;
    }
    if (p.q_start && thread == 0)
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
        if (cudaFuncSetAttribute(tables_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kTablesMaxRows * kTablesRowBytes) != cudaSuccess ||
            cudaFuncSetAttribute(tables_step_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                 1) != cudaSuccess)
            return PKV_ERR_CUDA;
        return PKV_OK;
    });
    if (rc != PKV_OK)
        return rc;
    const int ctas = kStepCtas;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.num_seqs) * kTablesRowBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tables_step_kernel, p, ctas) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
