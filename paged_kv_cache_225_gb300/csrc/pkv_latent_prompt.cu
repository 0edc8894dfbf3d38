// Latent attention over whole prompts, keys and values expanded per head, on the
// CUDA cores (fp32).
//
// Expanded form: row i of a sequence and head h attends its rows j <= i with score
// scale (q[i, h, :Dn] . k[j, h] + q[i, h, Dn:] . k_rope[j]), the rotated key being
// shared by all heads, and values v[j, h] of Dn dims (causal
// scaled_dot_product_attention of the "Inference optimization" lesson, Step 2).
// One pass over the keys with the running maximum and sum of the softmax.
//
// A CTA of 256 threads holds 64 rows of a head and walks 32 keys at a time, all in
// shared memory, so that two CTAs fit an SM; a thread owns 4 rows x 2 keys of the
// scores and 4 rows x Dn / 16 columns of the output; products are packed two to an
// instruction.
//
// What bounds it (8 prompts of 256 to 1024 tokens, 32 heads of 128 + 64: 1.32 ms, 27
// TFLOP/s), by its code: a block's K and V are asked for when the last one is done, so only
// the other CTA of the SM covers their way, and sixteen packed multiply-adds of the scores
// take six shared-memory loads.
#include "pkv_latent.h"
#include "pkv_prompt.cuh"

namespace pkv {

namespace {

constexpr int kRows = 64;
constexpr int kKeys = 32;
constexpr int kRpt = 4;  // rows per thread
constexpr int kTy = kRows / kRpt;
constexpr int kSimtThreads = 16 * kTy;

template <int DN> struct LpGeom {
    static constexpr int kDk = DN + kRopeDim;
    static constexpr int kLd = kDk + 4;     // rows of Q and K: 4 banks apart
    static constexpr int kPLd = kKeys + 4;  // and of the weights
    // The weights take K's place once the scores are done.
    static constexpr int kKP = kKeys * kLd > kRows * kPLd ? kKeys * kLd : kRows * kPLd;
    static constexpr int kSmem = (kRows * kLd + kKP + kKeys * DN) * 4;
};

template <int DN>
__global__ void __launch_bounds__(kSimtThreads, 2) latent_prompt_simt_kernel(const LatentPromptParams p)
{
    using Geo = LpGeom<DN>;
    constexpr int kDk = Geo::kDk, kLd = Geo::kLd, kPLd = Geo::kPLd;
    constexpr int kCols = DN / 64;  // float4 columns of the output per thread
    extern __shared__ __align__(16) float smem_f[];
    float *sq = smem_f, *sk = sq + kRows * kLd, *sv = sk + Geo::kKP, *sp = sk;
    __shared__ PromptItem s_item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float *q = static_cast<const float *>(p.q), *k = static_cast<const float *>(p.k);
    const float *kr = static_cast<const float *>(p.k_rope), *v = static_cast<const float *>(p.v);
    const int H = p.items.num_kv_heads;
    const float c = p.items.negate ? -p.items.score_scale : p.items.score_scale;

    PromptScan scan;
    if (warp == 0)
        scan.init(p.items, kRows, lane, blockIdx.x == 0);
    for (unsigned u = blockIdx.x;; u += gridDim.x) {
        if (warp == 0) {
            const PromptItem found = scan.find(p.items, kRows, u, lane);
            if (lane == 0)
                s_item = found;
        }
        __syncthreads();
        const PromptItem it = s_item;
        if (it.s < 0)
            return;
        const int t0 = it.index * kRows;       // first token of the item
        const int nt = min(kRows, it.n - t0);  // its tokens
        const int end = t0 + nt;               // keys any of its rows sees

        for (int e = threadIdx.x; e < kRows * (kDk / 4); e += kSimtThreads) {
            const int r = e / (kDk / 4), d = 4 * (e % (kDk / 4));
            if (r < nt)
                cp_async_16(sq + r * kLd + d, q + (static_cast<int64_t>(it.row0) + t0 + r) * p.q_stride +
                                            static_cast<int64_t>(it.hkv) * kDk + d);
            else
                *reinterpret_cast<float4 *>(sq + r * kLd + d) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        cp_async_commit();

        uint64_t o[kRpt][2 * kCols];
        float m[kRpt], l[kRpt];
        int pos[kRpt];
#pragma unroll
        for (int i = 0; i < kRpt; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            pos[i] = t0 + min(ty + kTy * i, nt - 1);  // rows past the item repeat its last token
#pragma unroll
            for (int x = 0; x < 2 * kCols; ++x)
                o[i][x] = 0;
        }

        for (int k0 = 0; k0 < end; k0 += kKeys) {
            __syncthreads();  // the last block's reads are done
            for (int e = threadIdx.x; e < kKeys * (kDk / 4); e += kSimtThreads) {
                const int r = e / (kDk / 4), d = 4 * (e % (kDk / 4));
                float *dk = sk + r * kLd + d;
                const int64_t row = static_cast<int64_t>(it.row0) + k0 + r;
                if (k0 + r >= end)
                    *reinterpret_cast<float4 *>(dk) = make_float4(0.f, 0.f, 0.f, 0.f);
                else if (d < DN)
                    cp_async_16(dk, k + row * p.k_stride + it.hkv * p.k_head + d);
                else
                    cp_async_16(dk, kr + row * p.k_rope_stride + d - DN);
            }
            cp_async_commit();
            for (int e = threadIdx.x; e < kKeys * (DN / 4); e += kSimtThreads) {
                const int r = e / (DN / 4), d = 4 * (e % (DN / 4));
                float *dv = sv + r * DN + d;
                if (k0 + r < end)
                    cp_async_16(dv, v + (static_cast<int64_t>(it.row0) + k0 + r) * p.v_stride + it.hkv * p.v_head + d);
                else
                    *reinterpret_cast<float4 *>(dv) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            cp_async_commit();
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // Q and K; V may still be on its way
            __syncthreads();
            uint64_t acc[kRpt][2];
#pragma unroll
            for (int i = 0; i < kRpt; ++i)
                acc[i][0] = acc[i][1] = 0;
#pragma unroll 4
            for (int d = 0; d < kDk; d += 4) {
                ulonglong2 kf[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    kf[j] = *reinterpret_cast<const ulonglong2 *>(sk + (tx + 16 * j) * kLd + d);
#pragma unroll
                for (int i = 0; i < kRpt; ++i) {
                    const ulonglong2 qf = *reinterpret_cast<const ulonglong2 *>(sq + (ty + kTy * i) * kLd + d);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        fma2(acc[i][j], qf.x, kf[j].x);
                        fma2(acc[i][j], qf.y, kf[j].y);
                    }
                }
            }
            cp_async_wait_all();
            __syncthreads();  // K is read, V is there

            const bool masked = k0 + kKeys > t0 + 1;  // some row does not see some key
#pragma unroll
            for (int i = 0; i < kRpt; ++i) {
                float x[2];
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = unpair(acc[i][j]);
                    x[j] = k0 + tx + 16 * j <= pos[i] ? (s.x + s.y) * c : -INFINITY;
                    mx = fmaxf(mx, x[j]);
                }
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, w));
                const float m_new = fmaxf(m[i], mx);
                // Nothing but -inf so far: any finite offset gives weights 0.
                const float off = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[i] - off);
                m[i] = m_new;
                l[i] *= alpha;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float w = exp2f(x[j] - off);
                    l[i] += w;
                    sp[(ty + kTy * i) * kPLd + tx + 16 * j] = w;
                }
                const uint64_t a2 = pair(alpha, alpha);
#pragma unroll
                for (int x2 = 0; x2 < 2 * kCols; ++x2)
                    mul2(o[i][x2], a2);
            }
            // A key a row does not see adds nothing to it, not even 0 * inf:
            // with infinities or NaN among V, a masked block goes key by key.
            bool careful = false;
            if (masked) {
                for (int e = threadIdx.x; e < kKeys * (DN / 4); e += kSimtThreads) {
                    const float4 x = *reinterpret_cast<const float4 *>(sv + 4 * e);
                    careful = careful || !(x.x * 0.f == 0.f && x.y * 0.f == 0.f && x.z * 0.f == 0.f &&
                                           x.w * 0.f == 0.f);
                }
                careful = __syncthreads_or(careful);
            }
            __syncwarp();  // a row's weights are written and read by one half warp
            if (!careful) {
#pragma unroll 1
                for (int key = 0; key < kKeys; key += 4) {
                    ulonglong2 vf[4][kCols];
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int x = 0; x < kCols; ++x)
                            vf[kk][x] = *reinterpret_cast<const ulonglong2 *>(sv + (key + kk) * DN + 4 * tx + 64 * x);
#pragma unroll
                    for (int i = 0; i < kRpt; ++i) {
                        const float4 w = *reinterpret_cast<const float4 *>(sp + (ty + kTy * i) * kPLd + key);
                        const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t w2 = pair(ww[kk], ww[kk]);
#pragma unroll
                            for (int x = 0; x < kCols; ++x) {
                                fma2(o[i][2 * x], w2, vf[kk][x].x);
                                fma2(o[i][2 * x + 1], w2, vf[kk][x].y);
                            }
                        }
                    }
                }
            } else {
                const int keys = min(kKeys, end - k0);
#pragma unroll 1
                for (int key = 0; key < keys; ++key)
#pragma unroll
                    for (int i = 0; i < kRpt; ++i) {
                        if (k0 + key > pos[i])
                            continue;
                        const float w1 = sp[(ty + kTy * i) * kPLd + key];
                        const uint64_t w = pair(w1, w1);
#pragma unroll
                        for (int x = 0; x < kCols; ++x) {
                            const ulonglong2 vf =
                                *reinterpret_cast<const ulonglong2 *>(sv + key * DN + 4 * tx + 64 * x);
                            fma2(o[i][2 * x], w, vf.x);
                            fma2(o[i][2 * x + 1], w, vf.y);
                        }
                    }
            }
        }

#pragma unroll
        for (int i = 0; i < kRpt; ++i) {
            float sum = l[i];
#pragma unroll
            for (int w = 8; w >= 1; w >>= 1)
                sum += __shfl_xor_sync(kFullMask, sum, w);
            const int r = ty + kTy * i;
            if (r >= nt)
                continue;
            const size_t orow = ((static_cast<size_t>(it.row0) + t0 + r) * H + it.hkv) * DN;
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
                const size_t off = orow + 4 * tx + 64 * x;
                const float2 a = unpair(o[i][2 * x]), b = unpair(o[i][2 * x + 1]);
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off) =
                    make_float4(a.x / sum, a.y / sum, b.x / sum, b.y / sum);
            }
        }
        __syncthreads();  // the item and its rows are read before the next ones are written
    }
}

template <int DN> pkv_status launch_lp(LatentPromptParams p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(latent_prompt_simt_kernel<DN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    LpGeom<DN>::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    const long items = prompt_max_items(p.items, kRows);
    if (items <= 0)
        return PKV_OK;
    if (items > 0x40000000L)
        return PKV_ERR_UNSUPPORTED;
    p.items.max_items = static_cast<unsigned>(items);
    // Two CTAs to an SM; the costliest items go first, one at a time.
    const long slots = 2L * device_sm_count();
    latent_prompt_simt_kernel<DN><<<static_cast<unsigned>(items < slots ? items : slots), kSimtThreads,
                                       LpGeom<DN>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_latent_prompt_simt(const LatentPromptParams &p, cudaStream_t stream)
{
    return p.nope == 128 ? launch_lp<128>(p, stream) : launch_lp<64>(p, stream);
}

}  // namespace pkv
