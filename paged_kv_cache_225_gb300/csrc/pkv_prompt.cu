// Causal attention over whole fp32 prompts on the CUDA cores.
//
// softmax(scale * q K^T) V of the "Inference optimization" lesson (Step 2,
// scaled_dot_product_attention with its causal mask) for every sequence of a
// packed batch: row i of a sequence attends rows 0 .. i of the same sequence,
// query head h uses KV head h / G.
//
// One pass over the keys with the running maximum m and sum l of the softmax
// (scores in log2 units): for a block of keys with scores x,
//   m' = max(m, max x),  l' = l 2^(m - m') + sum 2^(x - m'),
//   o' = o 2^(m - m') + sum 2^(x - m') v,   out = o / l.
// A CTA holds 64 rows (token, grouped head) and walks 64 keys at a time, all
// operands in shared memory as f32; a thread owns 8 rows x 4 keys of the
// scores and 8 rows x D / 16 columns of the output.
#include "pkv_prompt.cuh"

namespace pkv {

namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kSimtThreads = 128;

template <int D> struct SimtGeom {
    static constexpr int kLd = D + 4;  // row stride of Q and K: rows 4 banks apart
    static constexpr int kPLd = kKeys + 4;
    static constexpr int kFloats = kRows * kLd + kKeys * kLd + kKeys * D + kRows * kPLd;
    static constexpr int kSmem = kFloats * 4;
};

__device__ __forceinline__ float4 load4(const void *base, size_t off)
{
    return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off));
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 2) prompt_simt_kernel(const PromptParams p)
{
    using Geo = SimtGeom<D>;
    constexpr int kLd = Geo::kLd, kPLd = Geo::kPLd;
    constexpr int kCols = D / 64;  // float4 columns of the output per thread
    extern __shared__ __align__(16) float smem_f[];
    float *sq = smem_f, *sk = sq + kRows * kLd, *sv = sk + kKeys * kLd, *sp = sv + kKeys * D;
    __shared__ PromptItem s_item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.group;
    const int tokens = kRows / G;  // tokens per item
    if (warp == 0) {
        PromptScan scan;
        scan.init(p, tokens, lane, blockIdx.x == 0);
        const PromptItem it = scan.find(p, tokens, blockIdx.x, lane);
        if (lane == 0)
            s_item = it;
    }
    __syncthreads();
    const PromptItem it = s_item;
    if (it.s < 0)
        return;
    const int t0 = it.index * tokens;               // first token of the item
    const int nt = min(tokens, it.n - t0);          // its tokens
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

    for (int e = threadIdx.x; e < kRows * (D / 4); e += kSimtThreads) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nt * G)
            v = load4(p.q,
                      (static_cast<size_t>(it.row0) + t0 + r / G) * p.q_stride +
                          static_cast<size_t>(it.hkv * G + r % G) * D + c);
        *reinterpret_cast<float4 *>(sq + r * kLd + c) = v;
    }

    float o[8][4 * kCols], m[8], l[8];
    int pos[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        pos[i] = t0 + min((ty + 8 * i) / G, nt - 1);  // rows past the item repeat its last token
#pragma unroll
        for (int c = 0; c < 4 * kCols; ++c)
            o[i][c] = 0.f;
    }

    const int end = t0 + nt;  // keys any row of the item sees
    for (int k0 = 0; k0 < end; k0 += kKeys) {
        __syncthreads();  // the last block's reads are done
        for (int e = threadIdx.x; e < kKeys * (D / 4); e += kSimtThreads) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4));
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (k0 + r < end) {
                const size_t tok = static_cast<size_t>(it.row0) + k0 + r;
                const size_t col = static_cast<size_t>(it.hkv) * D + c;
                kk = load4(p.k, tok * p.k_stride + col);
                vv = load4(p.v, tok * p.v_stride + col);
            }
            *reinterpret_cast<float4 *>(sk + r * kLd + c) = kk;
            *reinterpret_cast<float4 *>(sv + r * D + c) = vv;
        }
        __syncthreads();
        float x[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][j] = 0.f;
#pragma unroll 2
        for (int d = 0; d < D; d += 4) {
            float4 kf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kf[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * kLd + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 qf = *reinterpret_cast<const float4 *>(sq + (ty + 8 * i) * kLd + d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = fmaf(qf.x, kf[j].x, fmaf(qf.y, kf[j].y, fmaf(qf.z, kf[j].z, fmaf(qf.w, kf[j].w, x[i][j]))));
            }
        }
        const float c = p.negate ? -p.score_scale : p.score_scale;
        const bool masked = k0 + kKeys > t0 + 1;  // some row does not see some key
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool seen = k0 + tx + 16 * j <= pos[i];
                x[i][j] = seen ? x[i][j] * c : -INFINITY;
                mx = fmaxf(mx, x[i][j]);
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
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(x[i][j] - off);
                l[i] += w;
                sp[(ty + 8 * i) * kPLd + tx + 16 * j] = w;
            }
#pragma unroll
            for (int c = 0; c < 4 * kCols; ++c)
                o[i][c] *= alpha;
        }
        __syncwarp();  // a row's weights are written and read by one half warp
        const int keys = min(kKeys, end - k0);
        if (!masked) {
#pragma unroll 1
            for (int k = 0; k < kKeys; k += 4) {
                float4 vf[4][kCols];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        vf[kk][c] = *reinterpret_cast<const float4 *>(sv + (k + kk) * D + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 w = *reinterpret_cast<const float4 *>(sp + (ty + 8 * i) * kPLd + k);
                    const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int c = 0; c < kCols; ++c) {
                            o[i][4 * c] = fmaf(ww[kk], vf[kk][c].x, o[i][4 * c]);
                            o[i][4 * c + 1] = fmaf(ww[kk], vf[kk][c].y, o[i][4 * c + 1]);
                            o[i][4 * c + 2] = fmaf(ww[kk], vf[kk][c].z, o[i][4 * c + 2]);
                            o[i][4 * c + 3] = fmaf(ww[kk], vf[kk][c].w, o[i][4 * c + 3]);
                        }
                }
            }
        } else {
            // Masked block: a key a row does not see adds nothing to it, not
            // even 0 * inf.
#pragma unroll 1
            for (int k = 0; k < keys; ++k) {
                float4 vf[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    vf[c] = *reinterpret_cast<const float4 *>(sv + k * D + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (k0 + k > pos[i])
                        continue;
                    const float w = sp[(ty + 8 * i) * kPLd + k];
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        o[i][4 * c] = fmaf(w, vf[c].x, o[i][4 * c]);
                        o[i][4 * c + 1] = fmaf(w, vf[c].y, o[i][4 * c + 1]);
                        o[i][4 * c + 2] = fmaf(w, vf[c].z, o[i][4 * c + 2]);
                        o[i][4 * c + 3] = fmaf(w, vf[c].w, o[i][4 * c + 3]);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float sum = l[i];
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1)
            sum += __shfl_xor_sync(kFullMask, sum, w);
        const int r = ty + 8 * i;
        if (r >= nt * G)
            continue;
        const size_t orow = ((static_cast<size_t>(it.row0) + t0 + r / G) * p.num_q_heads +
                             it.hkv * G + r % G) * D;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const size_t off = orow + 4 * tx + 64 * c;
            const float4 v = make_float4(o[i][4 * c] / sum, o[i][4 * c + 1] / sum,
                                         o[i][4 * c + 2] / sum, o[i][4 * c + 3] / sum);
            if (p.out_dtype == PKV_F32) {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off) = v;
            } else {
                uint2 w;
                w.x = pack_bf16(v.x, v.y);
                w.y = pack_bf16(v.z, v.w);
                *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(p.out) + off) = w;
            }
        }
    }
}

template <int D> pkv_status launch_simt_d(const PromptParams &p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(prompt_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    SimtGeom<D>::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    const long items = prompt_max_items(p, kRows / p.group);
    if (items <= 0)
        return PKV_OK;
    if (items > 0x7fffffffL)
        return PKV_ERR_UNSUPPORTED;
    prompt_simt_kernel<D><<<static_cast<unsigned>(items), kSimtThreads, SimtGeom<D>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_prompt_simt(const PromptParams &p, cudaStream_t stream)
{
    return p.head_dim == 128 ? launch_simt_d<128>(p, stream) : launch_simt_d<64>(p, stream);
}

}  // namespace pkv
