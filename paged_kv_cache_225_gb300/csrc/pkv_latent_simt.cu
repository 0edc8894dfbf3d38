// Latent attention for one query per sequence on the CUDA cores (fp32), and the
// kernel that joins the partial sums of sequences that a range's end cut.
//
// Absorbed form: out[s, h] = sum_t softmax_t(scale q[s, h] . row_t) row_t[:R], the
// scaled_dot_product_attention of the "Inference optimization" lesson (Step 2) in
// which all heads share one row of R + 64 numbers per token, key and value at once.
//
// A CTA of 256 threads has 16 heads of a sequence and walks its pages: scores of
// 16 heads x 16 tokens (a warp: 4 heads, all tokens, half the dims; a lane 4 heads x
// 2 tokens on every fourth of those dims), one pass of the softmax with a thread
// per score, then R / 256 output dims of all heads per thread.  Shared-memory loads and
// the steps of a page bound it: 16 sequences of 4096 tokens, 32 heads, R = 512: 157 us (29
// TFLOP/s); 8 of up to 4096, 16 heads, R = 256: 24 us.  With the four lanes of a token next to each other
// (two rows to a load's phase, in the same banks) 213 and 29 us.
#include "pkv_latent.cuh"

namespace pkv {

namespace {

constexpr int kSimtThreads = 256;
constexpr int kSimtHeads = 16;

template <int R> struct LatentSimt {
    static constexpr int kRow = R + kRopeDim;
    static constexpr int kLd = kRow + 4;  // rows 4 banks apart
    static constexpr int kPages = R == 256 ? 4 : 2;  // in shared memory, two CTAs to an SM
    static constexpr int kSmem = (1 + kPages) * 16 * kLd * 4;
};

__device__ __forceinline__ float sum2(uint64_t v)
{
    const float2 r = unpair(v);
    return r.x + r.y;
}

// 16 rows of 16-byte pieces into shared memory; rows past `rows` are zero.
template <int R> __device__ __forceinline__ void load_rows(float *dst, const float *src, int rows)
{
    constexpr int kRow = LatentSimt<R>::kRow, kLd = LatentSimt<R>::kLd;
    for (int e = threadIdx.x; e < 16 * (kRow / 4); e += kSimtThreads) {
        const int r = e / (kRow / 4), d = 4 * (e % (kRow / 4));
        float *to = dst + r * kLd + d;
        if (r < rows)
            cp_async_16(to, src + r * kRow + d);
        else
            *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    cp_async_commit();
}

template <int R>
__global__ void __launch_bounds__(kSimtThreads, 2) latent_simt_kernel(const LatentDecodeParams p)
{
    constexpr int kRow = LatentSimt<R>::kRow, kLd = LatentSimt<R>::kLd, kDims = R / kSimtThreads;
    constexpr int kPages = LatentSimt<R>::kPages;
    extern __shared__ __align__(16) float smem_f[];
    float *sq = smem_f, *sk = sq + 16 * kLd;  // the queries, the pages
    __shared__ float s_half[2][16][17];       // scores of half the dims
    __shared__ __align__(16) float s_p[16][16], s_alpha[16];
    __shared__ float2 s_ml[16];
    __shared__ LatentPiece s_piece;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int team = blockIdx.x / p.head_tiles, h0 = blockIdx.x % p.head_tiles * kSimtHeads;
    const int heads = min(kSimtHeads, p.num_heads - h0);
    const float c = p.negate ? -p.score_scale : p.score_scale;

    // The kernel that joins cut sequences may be set up; it waits for this one's end.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    LatentWalk walk;
    if (warp == 0)
        walk.init(p, team, lane, blockIdx.x == 0);
    int cut = -1;
    for (;;) {
        if (warp == 0) {
            const LatentPiece next = walk.next(p);
            if (lane == 0)
                s_piece = next;
        }
        __syncthreads();
        const LatentPiece piece = s_piece;
        if (piece.s < 0)
            break;
        if (piece.first > 0)
            cut = piece.s;
        load_rows<R>(sq, static_cast<const float *>(p.q) + (static_cast<size_t>(piece.s) * p.num_heads + h0) * kRow,
                     heads);
        const int from = piece.first * (kLatentTokens / 16);  // pages
        const int to = min(piece.last * (kLatentTokens / 16), (piece.len + 15) / 16);
        const int32_t *table = p.block_tables + static_cast<size_t>(piece.s) * p.max_blocks;
        auto load_page = [&](int page) {
            const int block = __ldg(table + page);
            const bool ok = static_cast<unsigned>(block) < static_cast<unsigned>(p.num_blocks);
            if (!ok && threadIdx.x == 0)
                set_status(p.status, PKV_ERR_OUT_OF_RANGE);
            load_rows<R>(sk + page % kPages * 16 * kLd,
                         static_cast<const float *>(p.cache) + static_cast<size_t>(ok ? block : 0) * 16 * kRow,
                         ok ? min(16, piece.len - 16 * page) : 0);
        };
        uint64_t o[kDims == 2 ? 16 : 8];  // heads x dims, in pairs
#pragma unroll
        for (int i = 0; i < (kDims == 2 ? 16 : 8); ++i)
            o[i] = 0;
        float m = -INFINITY, l = 0.f;  // of head threadIdx.x / 16
        // Every page counts as a group of copies, also one that is not there.
#pragma unroll
        for (int i = 0; i < kPages - 1; ++i) {
            if (from + i < to)
                load_page(from + i);
            else
                cp_async_commit();
        }
        for (int page = from; page < to; ++page) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kPages - 2) : "memory");
            __syncthreads();
            if (page + kPages - 1 < to)
                load_page(page + kPages - 1);
            else
                cp_async_commit();
            const float *k = sk + page % kPages * 16 * kLd;
            {
                // Heads 4 (warp % 4) .., dims of half warp / 4, tokens lane % 8 and lane % 8 + 8:
                // the eight lanes of a load's phase lie in eight rows, 4 banks apart.
                const int half = warp >> 2, hq = 4 * (warp & 3);
                uint64_t acc[4][2] = {};
                const float *kq = sq + hq * kLd + half * (kRow / 2) + 4 * (lane >> 3);
                const float *kr = k + (lane & 7) * kLd + half * (kRow / 2) + 4 * (lane >> 3);
#pragma unroll 2
                for (int d = 0; d < kRow / 2; d += 16) {
                    ulonglong2 kf[2];
                    kf[0] = *reinterpret_cast<const ulonglong2 *>(kr + d);
                    kf[1] = *reinterpret_cast<const ulonglong2 *>(kr + 8 * kLd + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const ulonglong2 qf = *reinterpret_cast<const ulonglong2 *>(kq + i * kLd + d);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            fma2(acc[i][j], qf.x, kf[j].x);
                            fma2(acc[i][j], qf.y, kf[j].y);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = sum2(acc[i][j]);
                        x += __shfl_xor_sync(kFullMask, x, 8);
                        x += __shfl_xor_sync(kFullMask, x, 16);
                        if (lane < 8)
                            s_half[half][hq + i][lane + 8 * j] = x;
                    }
            }
            __syncthreads();
            {
                const int h = threadIdx.x >> 4, t = threadIdx.x & 15;
                const float x = 16 * page + t < piece.len ? (s_half[0][h][t] + s_half[1][h][t]) * c : -INFINITY;
                float mx = x;
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, w));
                const float m_new = fmaxf(m, mx);
                const float off = m_new == -INFINITY ? 0.f : m_new;  // nothing but -inf: weights 0
                const float alpha = exp2f(m - off), w = exp2f(x - off);
                m = m_new;
                l = l * alpha + w;
                s_p[t][h] = w;
                if (t == 0)
                    s_alpha[h] = alpha;
            }
            __syncthreads();
            // Output dims 2 threadIdx.x and the next, or dim threadIdx.x.
            if constexpr (kDims == 2) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = s_alpha[i];
                    mul2(o[i], pair(a, a));
                }
#pragma unroll 4
                for (int t = 0; t < 16; ++t) {
                    const uint64_t v = *reinterpret_cast<const uint64_t *>(k + t * kLd + 2 * threadIdx.x);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(&s_p[t][i]);
                        const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            fma2(o[i + e], pair(ww[e], ww[e]), v);
                    }
                }
            } else {
                // One dim: pairs of heads.
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mul2(o[i], *reinterpret_cast<const uint64_t *>(&s_alpha[2 * i]));
                }
#pragma unroll 4
                for (int t = 0; t < 16; ++t) {
                    const float x = k[t * kLd + threadIdx.x];
                    const uint64_t v = pair(x, x);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&s_p[t][2 * i]);
                        fma2(o[i], w.x, v);
                        fma2(o[i + 1], w.y, v);
                    }
                }
            }
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1)
            l += __shfl_xor_sync(kFullMask, l, w);
        if ((threadIdx.x & 15) == 0)
            s_ml[threadIdx.x >> 4] = make_float2(m, l);
        cp_async_wait_all();
        __syncthreads();
        const bool whole = piece.whole();
        const size_t slot = static_cast<size_t>(latent_slot(team, piece)) * p.head_tiles + blockIdx.x % p.head_tiles;
#pragma unroll
        for (int h = 0; h < 16; ++h) {
            if (h >= heads)
                break;
            float2 y;
            if constexpr (kDims == 2) {
                y = unpair(o[h]);
            } else {
                const float2 z = unpair(o[h / 2]);
                y.x = h & 1 ? z.y : z.x;
                y.y = 0.f;
            }
            const int d = kDims * threadIdx.x;
            if (!whole) {
                float *dst = p.part + (slot * kSimtHeads + h) * R + d;
                dst[0] = y.x;
                if constexpr (kDims == 2)
                    dst[1] = y.y;
                if (threadIdx.x == 0)
                    p.part_ml[slot * kSimtHeads + h] = s_ml[h];
                continue;
            }
            const float sum = s_ml[h].y;
            // An empty sequence's row is zero.
            y.x = piece.len > 0 ? y.x / sum : 0.f;
            y.y = piece.len > 0 ? y.y / sum : 0.f;
            float *dst = static_cast<float *>(p.out) + (static_cast<size_t>(piece.s) * p.num_heads + h0 + h) * R + d;
            dst[0] = y.x;
            if constexpr (kDims == 2)
                dst[1] = y.y;
        }
        __syncthreads();  // s_ml, the queries and the piece are read
    }
    if (threadIdx.x == 0 && blockIdx.x % p.head_tiles == 0)
        p.pieces[team] = cut;
}

// ------------------------------------------------------------------ joining

constexpr int kMergeWarps = 4;  // of a block in which each has a unit of its own

// Joins the pieces of cut sequences.  blockIdx.x is a sequence (fewer sequences than
// teams) or a team but the first, which stands for the sequence that its start cuts if
// that begins in the team before.  For one head and 128 of its dims
//   M = max_i m_i,  out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i
// over the pieces i, four at a time.  A warp has 256 dims of a head and all pieces, or,
// with many pieces to a sequence, kShare warps take them in turn for 128 dims and add up
// in order.  Either way the result does not depend on who wrote first.
//
// What bounds it: three dependent trips to L2 and the partial sums, which are there (64
// sequences of 64 heads, 28 MB: 8.5 us of 62; a warp to 128 dims 11.4, to 512 9).
template <typename T, int R, int kShare>
__global__ void __launch_bounds__(32 * (kShare > 1 ? kShare : kMergeWarps))
    latent_merge_kernel(const LatentDecodeParams p, int by_sequence)
{
    constexpr bool kShared = kShare > 1;
    constexpr int kVec = kShared ? 1 : 2;
    constexpr int kParts = R / 128 / kVec;
    __shared__ float4 s_sum[kShare][32];
    __shared__ float2 s_ml[kShare];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = kShared ? blockIdx.y : blockIdx.y * kMergeWarps + warp;
    const int h = unit / kParts, d = unit % kParts * (128 * kVec) + 4 * lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (h >= p.num_heads)
        return;
    // The sequence that each team's start cuts, lane by lane; at most 304 teams.
    constexpr int kMost = (2 * kLatentSms + 31) / 32;
    int cut[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i)
        cut[i] = 32 * i + lane < p.teams ? p.pieces[32 * i + lane] : -1;
    int s = blockIdx.x;
    if (!by_sequence) {
        const int team = blockIdx.x + 1;
        s = p.pieces[team];
        // The piece before starts the sequence if nothing before that one belongs to it.
        if (s < 0 || p.pieces[team - 1] == s)
            return;
    }
    int team = p.teams, count = 0;  // the first team that goes on with s, and how many do
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const unsigned same = __ballot_sync(kFullMask, cut[i] == s);
        if (same && count == 0)
            team = 32 * i + __ffs(same) - 1;
        count += __popc(same);  // its teams are neighbours
    }
    if (count == 0)
        return;
    const int last = team + count - 1;
    const int ht = h / p.tile_heads, hh = h % p.tile_heads;
    auto row = [&](int t) {  // t = team - 1: the piece the sequence starts with
        const size_t slot = t < team ? 2 * t + 1 : 2 * t;
        return (slot * p.head_tiles + ht) * p.tile_heads + hh;
    };
    // A few pieces at a time, their loads before anything that needs one.
    constexpr int kDeep = 4;
    float4 sums[kVec] = {};
    float top = -INFINITY, total = 0.f;
    for (int t0 = team - 1 + (kShared ? kDeep * warp : 0); t0 <= last; t0 += kDeep * kShare) {
        float4 x[kDeep][kVec];
        float2 ml[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int t = min(t0 + i, last);
            ml[i] = p.part_ml[row(t)];
#pragma unroll
            for (int v = 0; v < kVec; ++v)
                x[i][v] = *reinterpret_cast<const float4 *>(p.part + row(t) * R + d + 128 * v);
        }
        float up = top;
#pragma unroll
        for (int i = 0; i < kDeep; ++i)
            up = fmaxf(up, ml[i].x);
        const float old = top == -INFINITY ? 0.f : exp2f(top - up);
        top = up;
        total *= old;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            sums[v].x *= old;
            sums[v].y *= old;
            sums[v].z *= old;
            sums[v].w *= old;
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            if (t0 + i > last)
                break;
            const float w = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - up);
            total = fmaf(w, ml[i].y, total);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                sums[v].x = fmaf(w, x[i][v].x, sums[v].x);
                sums[v].y = fmaf(w, x[i][v].y, sums[v].y);
                sums[v].z = fmaf(w, x[i][v].z, sums[v].z);
                sums[v].w = fmaf(w, x[i][v].w, sums[v].w);
            }
        }
    }
    if constexpr (kShared) {
        s_sum[warp][lane] = sums[0];
        if (lane == 0)
            s_ml[warp] = make_float2(top, total);
        __syncthreads();
        if (warp > 0)
            return;
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kShare; ++i)
            top = fmaxf(top, s_ml[i].x);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        total = 0.f;
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const float4 x = s_sum[i][lane];
            const float w = s_ml[i].x == -INFINITY ? 0.f : exp2f(s_ml[i].x - top);
            total = fmaf(w, s_ml[i].y, total);
            sum.x = fmaf(w, x.x, sum.x);
            sum.y = fmaf(w, x.y, sum.y);
            sum.z = fmaf(w, x.z, sum.z);
            sum.w = fmaf(w, x.w, sum.w);
        }
        sums[0] = sum;
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
        const size_t at = (static_cast<size_t>(s) * p.num_heads + h) * R + d + 128 * v;
        const float4 y = make_float4(sums[v].x / total, sums[v].y / total, sums[v].z / total, sums[v].w / total);
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = y;
        else
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
}

template <int R> pkv_status launch_simt(const LatentDecodeParams &p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(latent_simt_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    LatentSimt<R>::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    latent_simt_kernel<R><<<p.teams * p.head_tiles, kSimtThreads, LatentSimt<R>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, int R, int kShare> pkv_status launch_merge(const LatentDecodeParams &p, cudaStream_t stream)
{
    const int by_sequence = p.num_seqs < p.teams;
    const int units = p.num_heads * (R / 128) / (kShare > 1 ? 1 : 2);
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(by_sequence ? p.num_seqs : p.teams - 1,
                          kShare > 1 ? units : (units + kMergeWarps - 1) / kMergeWarps);
    config.blockDim = dim3(32 * (kShare > 1 ? kShare : kMergeWarps));
    config.stream = stream;
    // Set up while the attention kernel runs.
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, latent_merge_kernel<T, R, kShare>, p, by_sequence) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}
template <typename T, int R> pkv_status launch_merge_by(const LatentDecodeParams &p, cudaStream_t stream)
{
    // Eight pieces to a sequence and more (4 x 32K tokens, 128 heads, 19 pieces: 57 us, alone
    // or with eight warps 59), and 32 and more (32K tokens, 32 heads, 152 pieces: 25 us, with
    // four warps 30, alone 60 with an earlier form).
    return p.teams >= 32 * p.num_seqs  ? launch_merge<T, R, 8>(p, stream)
           : p.teams >= 8 * p.num_seqs ? launch_merge<T, R, 4>(p, stream)
                                       : launch_merge<T, R, 1>(p, stream);
}

}  // namespace

// Cut / whole, us, when the rule was chosen: one sequence of 200 tokens, 32 heads 10.7 / 10.4, of 512 9.4 / 14.1; 128
// of 256 to 512 31 / 30, of 500 to 1000 37 / 46.
constexpr double kCut = 4, kCutAll = 1.5;

size_t latent_part_rows(const LatentDecodeParams &p)
{
    return p.whole ? 0 : 2 * static_cast<size_t>(p.teams) * p.head_tiles * p.tile_heads;
}

size_t latent_plan(LatentDecodeParams &p, int dtype)
{
    // fp32: two CTAs to an SM.  bf16: one, with the fewest head columns that hold the heads
    // (columns cost time, and the room they leave holds more tiles): 256 x 4096 tokens of 16
    // heads took 192 us with 16 columns, 194 with 32, 202 with 64 on one card; 128 of 500 to
    // 1000 tokens, 32 heads, 36.3 with 32 columns, 38.3 with 64.
    p.tile_heads = dtype == PKV_F32 || p.num_heads <= 16 ? 16 : p.num_heads <= 32 ? 32 : 64;
    p.head_tiles = (p.num_heads + p.tile_heads - 1) / p.tile_heads;
    const long ctas = dtype == PKV_F32 ? 2 * kLatentSms : kLatentSms;
    const long tiles = (static_cast<long>(p.max_len) + kLatentTokens - 1) / kLatentTokens;
    const long units = static_cast<long>(p.num_seqs) * (tiles > 1 ? tiles : 1);
    const long most = ctas / p.head_tiles;
    p.teams = static_cast<int>(units < most ? units : most);
    // Cutting evens the teams out and costs partial sums and the second kernel, in tiles
    // of a team about kCut and, by the share of the teams that cut, kCutAll more.  Without
    // it a team has whole sequences, of which the longest counts.  The lengths are not
    // known here: three quarters of the bound on average are supposed.  (Figures: bf16.)
    const double rounds = static_cast<double>((p.num_seqs + most - 1) / most) * tiles;
    const double even = 0.75 * p.num_seqs * tiles / most;
    p.whole = rounds <= even + kCut + kCutAll * p.teams / most;
    if (p.whole && p.num_seqs < p.teams)
        p.teams = p.num_seqs > 0 ? p.num_seqs : 1;
    const size_t rows = latent_part_rows(p);
    return (rows * (p.latent_dim * sizeof(float) + sizeof(float2)) + p.teams * sizeof(int) + 255) / 256 * 256;
}

pkv_status launch_latent_decode_simt(const LatentDecodeParams &p, cudaStream_t stream)
{
    return p.latent_dim == 512 ? launch_simt<512>(p, stream) : launch_simt<256>(p, stream);
}

pkv_status launch_latent_merge(const LatentDecodeParams &p, int dtype, cudaStream_t stream)
{
    if (p.teams <= 1 || p.whole)
        return PKV_OK;
    if (dtype == PKV_F32)
        return p.latent_dim == 512 ? launch_merge_by<float, 512>(p, stream) : launch_merge_by<float, 256>(p, stream);
    return p.latent_dim == 512 ? launch_merge_by<__nv_bfloat16, 512>(p, stream)
                               : launch_merge_by<__nv_bfloat16, 256>(p, stream);
}

}  // namespace pkv
