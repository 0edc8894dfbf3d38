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
#include "pkv_ops.h"

namespace pkv {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// CTAs of the cluster: the largest there is.  us a step on 2 / 4 / 8 / 16: 128
// rows of a 31K-page pool 13.3 / 11.0 / 10.9 / 11.2, 64 prompts admitted 46.5 /
// 28.1 / 18.8 / 14.7, 512 rows of a 288K-page pool 73.6 / 43.1 / 29.1 / 21.6.
constexpr int kStepCtas = 16;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// A cluster barrier in two halves: what a CTA did before the first (shared and
// global memory) is visible to every CTA after the second.  `.aligned`: a
// warp's lanes arrive together.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
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

// Lanes whose count is zero among the 32 from id on (ids from p.num_blocks on
// are not).  A count below zero, of a page dropped more often than held, is
// reported and becomes zero.
__device__ __forceinline__ unsigned zero_mask(const TablesParams &p, long id, int lane)
{
    const bool in = id + lane < p.num_blocks;
    const int refs = in ? __ldcg(p.ref_counts + id + lane) : 1;
    if (refs < 0) {
        p.ref_counts[id + lane] = 0;
        set_status(p.status, PKV_ERR_OUT_OF_RANGE);
    }
    return __ballot_sync(kFullMask, refs <= 0);
}

constexpr int kStep = 4;     // loads of table entries in flight
constexpr int kRounds = 8;   // turns that the warps take through the pool (a multiple of kStep)
constexpr unsigned kInvalid = ~0u;

// A cluster of CTAs runs the whole step: the pool's counts and the rows' pages
// and slots are spread over the cluster's warps, the (small) row sums are
// computed by every CTA for itself, and three cluster barriers separate drops,
// counting, handing out and writing slots.  All of it is a few dependent trips to L2, each of
// which the code starts as early as it can: bound by latency, not by bytes.
__global__ void __launch_bounds__(kThreads, 1) tables_step_kernel(const TablesParams p)
{
    extern __shared__ int rows_smem[];
    __shared__ unsigned long long s_part[2 * kWarps];
    __shared__ int s_warp_base[kRounds][kWarps];  // zero counts, then those of the warps before
    __shared__ int s_zeros[kRounds][kStepCtas];   // zero counts of every CTA
    __shared__ int s_bad;
    const int S = p.num_seqs;
    int *tok_end = rows_smem;     // tokens asked for; then reserved, inclusive sums
    int *page_end = tok_end + S;  // length before the step; then pages taken, inclusive sums
    // 2 * kept + copy, or kInvalid for a row of invalid length.
    unsigned *kept2 = reinterpret_cast<unsigned *>(page_end + S);
    // 2 * page + shared of the part-filled page that the row grows into, else kInvalid.
    unsigned *last2 = kept2 + S;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = blockIdx.x;  // the grid is one cluster
    const int gw = cta * kWarps + warp, warps = kStepCtas * kWarps;
    const int thread = cta * kThreads + threadIdx.x, threads = kStepCtas * kThreads;
    const int max_len = p.max_blocks * kBlockSize;
    const size_t width = p.max_blocks;

    if (!p.drop_lens)
        cluster_arrive();  // only says that this CTA runs
    if (threadIdx.x == 0)
        s_bad = 0;
    __syncthreads();

    // Rows: what is kept, and the part-filled last pages (which no drop touches).
    int32_t page0 = -1;  // that of row threadIdx.x, on its way during the drops
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int L = __ldcg(p.seq_lens + s), d = p.drop_lens ? __ldg(p.drop_lens + s) : 0;
        const int n = p.new_lens ? __ldg(p.new_lens + s) : 0;
        const bool len_ok = L >= 0 && L <= max_len;
        const int kept = len_ok ? L - (d > 0 ? min(d, L) : 0) : 0;
        if (!len_ok || n < 0 || n > max_len - kept)
            s_bad = 1;
        else if (n > 0 && kept % kBlockSize != 0) {
            const int32_t page = __ldcg(p.block_tables + s * width + pages_of(kept) - 1);
            if (s == threadIdx.x)
                page0 = page;
            else
                last2[s] = page >= 0 && page < p.num_blocks ? 2u * static_cast<unsigned>(page) : kInvalid;
        }
        if (p.drop_lens && (!len_ok || d < 0) && cta == 0)
            set_status(p.status, PKV_ERR_OUT_OF_RANGE);
        tok_end[s] = n;
        page_end[s] = L;
        kept2[s] = len_ok ? 2u * static_cast<unsigned>(kept) : kInvalid;
    }

    // Drops: as many warps per row as there are for all rows.
    if (p.drop_lens) {
        __syncthreads();
        const int per_row = max(1, warps / S);
        const int sub = gw % per_row;
        for (int s = gw / per_row; s < S && gw / per_row < warps / per_row; s += warps / per_row) {
            if (kept2[s] == kInvalid)
                continue;
            int32_t *row = p.block_tables + s * width;
            const int last = pages_of(page_end[s]);
            for (int j0 = pages_of(static_cast<int>(kept2[s] >> 1)) + sub * 32 + lane; j0 < last;
                 j0 += kStep * 32 * per_row) {
                int32_t page[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int j = j0 + i * 32 * per_row;
                    page[i] = j < last ? __ldcg(row + j) : -1;
                }
                // A page that nobody held falls below zero: the counting below
                // finds and mends it, so that nothing waits for a result here.
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int j = j0 + i * 32 * per_row;
                    if (j >= last)
                        continue;
                    row[j] = -1;
                    if (page[i] >= 0 && page[i] < p.num_blocks)
                        atomicSub(p.ref_counts + page[i], 1);
                    else
                        set_status(p.status, PKV_ERR_OUT_OF_RANGE);
                }
            }
        }
        cluster_arrive();
        cluster_wait();
    }

    // Zero counts.  The warps go through the pool in turns of `chunk` ids each,
    // so that the low ids, where the free pages are taken, are spread over all.
    const int chunk = static_cast<int>((p.num_blocks / (static_cast<long>(warps) * kRounds) + 32) & ~31L);
#pragma unroll 1
    for (int r0 = 0; r0 < kRounds; r0 += kStep) {
        int zeros[kStep] = {};
#pragma unroll 1
        for (int i = 0; i < chunk; i += 32)
#pragma unroll
            for (int x = 0; x < kStep; ++x)
                zeros[x] += __popc(zero_mask(p, (static_cast<long>(r0 + x) * warps + gw) * chunk + i, lane));
        if (lane == 0)
#pragma unroll
            for (int x = 0; x < kStep; ++x)
                s_warp_base[r0 + x][warp] = zeros[x];
    }
    // Counts of the rows' last pages, as the drops left them.
    for (int s = threadIdx.x; s < S; s += kThreads) {
        const int n = tok_end[s];
        const unsigned k2 = kept2[s];
        unsigned l2 = kInvalid;
        if (k2 != kInvalid && n > 0 && n <= max_len - static_cast<int>(k2 >> 1) && (k2 >> 1) % kBlockSize != 0) {
            if (s == threadIdx.x)
                l2 = page0 >= 0 && page0 < p.num_blocks ? 2u * static_cast<unsigned>(page0) : kInvalid;
            else
                l2 = last2[s];
            const int refs = l2 == kInvalid ? 0 : __ldcg(p.ref_counts + (l2 >> 1));
            if (refs <= 0)
                s_bad = 1;
            if (refs > 1)
                l2 |= 1u;
        }
        last2[s] = l2;
    }
    if (!p.drop_lens)
        cluster_wait();  // every CTA runs: their shared memory may be written
    __syncthreads();
    if (warp < kRounds) {  // a turn's zero counts: per-warp bases, this CTA's total to every CTA
        const int own = s_warp_base[warp][lane];
        int z = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFullMask, z, d);
            if (lane >= d)
                z += y;
        }
        s_warp_base[warp][lane] = z - own;
        const int all = __shfl_sync(kFullMask, z, 31);
        if (lane < kStepCtas) {
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(remote)
                         : "r"(smem_u32(&s_zeros[warp][cta])), "r"(lane));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(all) : "memory");
        }
    }
    // A sharing row copies unless every other holder of the page is an
    // earlier row that has copied already.  A warp per row.
    for (int s = warp; s < S; s += kWarps) {
        const unsigned l2 = last2[s];
        if (l2 == kInvalid || !(l2 & 1u))
            continue;
        const int others = __ldcg(p.ref_counts + (l2 >> 1)) - 1;
        int before = 0;
        for (int t = lane; t < s; t += 32)
            before += last2[t] == l2;
        before = __reduce_add_sync(kFullMask, before);
        if (before < others && lane == 0) {
            kept2[s] |= 1u;
            if (!p.copy_pairs)
                s_bad = 1;
        }
    }
    __syncthreads();
    // Prefix sums of the tokens and pages, 1024 rows at a time.
    unsigned long long tokens = 0, pages = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        unsigned long long n = 0, need = 0;
        if (s < S && kept2[s] != kInvalid) {
            const int kept = static_cast<int>(kept2[s] >> 1);
            const int nn = tok_end[s];
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
    cluster_arrive();
    cluster_wait();

    // Lane r: the zero counts ahead of this CTA's in turn r, and of the turn.
    int ahead = 0, total_zeros = 0;
    if (lane < kRounds)
        for (int c = 0; c < kStepCtas; ++c) {
            const int z = s_zeros[lane][c];
            ahead += c < cta ? z : 0;
            total_zeros += z;
        }
    {
        int upto = total_zeros;  // turns up to this lane's
#pragma unroll
        for (int d = 1; d < kRounds; d <<= 1) {
            const int y = __shfl_up_sync(kFullMask, upto, d);
            if (lane >= d)
                upto += y;
        }
        ahead += upto - total_zeros;
        total_zeros = __shfl_sync(kFullMask, upto, kRounds - 1);
    }
    const bool enough = pages <= static_cast<unsigned long long>(total_zeros);
    const bool bad = s_bad || tokens > static_cast<unsigned long long>(p.max_tokens);
    const bool ok = !bad && enough;
    if (!ok && thread == 0)
        set_status(p.status, bad ? PKV_ERR_OUT_OF_RANGE : PKV_ERR_NO_BLOCKS);
    const int total = ok ? static_cast<int>(tokens) : 0;
    const int taken = ok ? static_cast<int>(pages) : 0;

    // Hand out the pages: the r-th zero count goes to the row that owns r.
#pragma unroll 1
    for (int r = 0; r < kRounds; ++r) {
        const long b = (static_cast<long>(r) * warps + gw) * chunk;
        int rank = __shfl_sync(kFullMask, ahead, r) + s_warp_base[r][warp];
        if (b >= p.num_blocks || rank >= taken)
            break;
#pragma unroll 1
        for (int i = 0; i < chunk && rank < taken; i += 32) {
            const unsigned m = zero_mask(p, b + i, lane);
            const int at = rank + __popc(m & ((1u << lane) - 1u));
            rank += __popc(m);
            if (!(m >> lane & 1u) || at >= taken)
                continue;
            const int32_t page = static_cast<int32_t>(b + i + lane);
            const int s = row_of(page_end, S, at);
            const int j = at - (s ? page_end[s - 1] : 0);
            const unsigned k2 = kept2[s];
            const int copy = k2 & 1u;
            if (copy && j == 0) {
                const unsigned src = last2[s] >> 1;
                p.copy_pairs[2 * s] = static_cast<int32_t>(src);
                p.copy_pairs[2 * s + 1] = page;
                atomicSub(p.ref_counts + src, 1);  // at least one holder is left
            }
            p.block_tables[s * width + pages_of(static_cast<int>(k2 >> 1)) - copy + j] = page;
            p.ref_counts[page] = 1;
        }
    }
    cluster_arrive();
    for (int s = thread; s < S; s += threads) {
        const int end = ok ? tok_end[s] : 0;
        const int n = ok ? end - (s ? tok_end[s - 1] : 0) : 0;
        if (p.q_start)
            p.q_start[s + 1] = end;
        if (p.copy_pairs && (!ok || !(kept2[s] & 1u)))
            p.copy_pairs[2 * s] = p.copy_pairs[2 * s + 1] = -1;
        if (kept2[s] != kInvalid)
            p.seq_lens[s] = static_cast<int>(kept2[s] >> 1) + n;
    }
    if (p.q_start && thread == 0)
        p.q_start[0] = 0;
    cluster_wait();  // the tables are written

    // Slots of the reserved tokens, -1 past them: four tokens in a row per
    // thread, which mostly share their row and page.
    for (long i0 = 4L * thread; i0 < p.max_tokens; i0 += 4L * threads) {
        const int *last = tok_end + S;
        const int *e = i0 < total ? tok_end + row_of(tok_end, S, static_cast<int>(i0)) : last;
        int64_t slot[4];
        int at = -1;  // table entry in `page`
        int32_t page = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            slot[x] = -1;
            if (i0 + x >= total)
                continue;
            const int i = static_cast<int>(i0) + x;
            for (; *e <= i; ++e)
                at = -1;
            const int s = static_cast<int>(e - tok_end);
            const int pos = static_cast<int>(kept2[s] >> 1) + i - (s ? e[-1] : 0);
            if (at != pos / kBlockSize) {
                at = pos / kBlockSize;
                page = __ldcg(p.block_tables + s * width + at);
            }
            slot[x] = static_cast<int64_t>(page) * kBlockSize + pos % kBlockSize;
        }
        if (i0 + 4 <= p.max_tokens && p.wide_slots) {
            longlong2 *dst = reinterpret_cast<longlong2 *>(p.slot_mapping + i0);
            dst[0] = make_longlong2(slot[0], slot[1]);
            dst[1] = make_longlong2(slot[2], slot[3]);
        } else {
            for (int x = 0; x < 4; ++x)
                if (i0 + x < p.max_tokens)
                    p.slot_mapping[i0 + x] = slot[x];
        }
    }
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
    // No pair of the call drops a page or adds one that nobody holds: a count
    // read as positive stays so.
    const int pages = pages_of(L);
    for (int j0 = threadIdx.x; j0 < pages; j0 += kStep * kForkThreads) {
        int32_t page[kStep];
        int refs[kStep];
#pragma unroll
        for (int x = 0; x < kStep; ++x)
            page[x] = j0 + x * kForkThreads < pages ? __ldcg(src + j0 + x * kForkThreads) : -1;
#pragma unroll
        for (int x = 0; x < kStep; ++x)
            refs[x] = page[x] >= 0 && page[x] < num_blocks ? __ldcg(ref_counts + page[x]) : 0;
#pragma unroll
        for (int x = 0; x < kStep; ++x) {
            if (j0 + x * kForkThreads >= pages)
                continue;
            if (refs[x] > 0)
                atomicAdd(ref_counts + page[x], 1);
            else
                set_status(status, PKV_ERR_OUT_OF_RANGE);  // not a held page: nothing to share
            dst[j0 + x * kForkThreads] = refs[x] > 0 ? page[x] : -1;
        }
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
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kStepCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kStepCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.num_seqs) * kTablesRowBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tables_step_kernel, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
