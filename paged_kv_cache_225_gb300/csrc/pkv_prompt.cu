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
// Everything stays in f32: tensor-core products of split operands would lose
// the last bits in their accumulation.
//
// A CTA of 256 threads holds 64 rows (token, grouped head) and walks 64 keys at a
// time, all operands in shared memory; a thread owns 4 rows x 4 keys of the scores
// and 4 rows x D / 16 columns of the output.  Products are packed two to an
// instruction (fma.rn.f32x2): the scores sum even and odd dims in the halves, the
// output holds pairs of columns.  Shared-memory loads and their latency bound it.
// Rows per thread trade loads for warps that hide them: 8 rows (128 threads, 250
// registers) load least, but two CTAs are then 8 warps to an SM; 2 rows load twice
// as often as 4.  8 prompts of 256 to 1024 tokens, 32 heads of 128 over 8 KV
// heads: 919 us with 8 rows, 898 us (33 TFLOP/s) with 4, 1241 us with 2; four
// prompts of 1 to 64 tokens 11.8, 10.0 and 10.5 us.  Single multiply-adds with one
// shared load per operand pair took 1233 us.
#include "pkv_prompt.cuh"

namespace pkv {

namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kRpt = 4;  // rows per thread
constexpr int kTy = kRows / kRpt;
constexpr int kSimtThreads = 16 * kTy;

template <int D> struct SimtGeom {
    static constexpr int kLd = D + 4;          // row stride of Q and K: rows 4 banks apart
    static constexpr int kPLd = kKeys + 4;     // and of the weights
    // The weights take K's place once the scores are done.
    static constexpr int kKP = kKeys * kLd > kRows * kPLd ? kKeys * kLd : kRows * kPLd;
    static constexpr int kFloats = kRows * kLd + kKP + kKeys * D;
    static constexpr int kSmem = kFloats * 4;
};

__device__ __forceinline__ void fma2(uint64_t &c, uint64_t a, uint64_t b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ void mul2(uint64_t &c, uint64_t a)
{
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(c) : "l"(a));
}
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 2) prompt_simt_kernel(const PromptParams p)
{
    using Geo = SimtGeom<D>;
    constexpr int kLd = Geo::kLd, kPLd = Geo::kPLd;
    constexpr int kCols = D / 64;  // float4 columns of the output per thread
    extern __shared__ __align__(16) float smem_f[];
    float *sq = smem_f, *sk = sq + kRows * kLd, *sv = sk + Geo::kKP, *sp = sk;
    __shared__ PromptItem s_item;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.group;
    const int tokens = kRows / G;  // tokens per item
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float *q = static_cast<const float *>(p.q);
    const float *k = static_cast<const float *>(p.k), *v = static_cast<const float *>(p.v);
    const float c = p.negate ? -p.score_scale : p.score_scale;

    PromptScan scan;
    if (warp == 0)
        scan.init(p, tokens, lane, blockIdx.x == 0);
    for (unsigned u = blockIdx.x;; u += gridDim.x) {
        if (warp == 0) {
            const PromptItem found = scan.find(p, tokens, u, lane);
            if (lane == 0)
                s_item = found;
        }
        __syncthreads();
        const PromptItem it = s_item;
        if (it.s < 0)
            return;
        const int t0 = it.index * tokens;       // first token of the item
        const int nt = min(tokens, it.n - t0);  // its tokens
        const int end = t0 + nt;                // keys any of its rows sees

        for (int e = threadIdx.x; e < kRows * (D / 4); e += kSimtThreads) {
            const int r = e / (D / 4), d = 4 * (e % (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nt * G)
                x = __ldg(reinterpret_cast<const float4 *>(
                    q + (static_cast<size_t>(it.row0) + t0 + r / G) * p.q_stride +
                    static_cast<size_t>(it.hkv * G + r % G) * D + d));
            *reinterpret_cast<float4 *>(sq + r * kLd + d) = x;
        }

        uint64_t o[kRpt][2 * kCols];
        float m[kRpt], l[kRpt];
        int pos[kRpt];
#pragma unroll
        for (int i = 0; i < kRpt; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            pos[i] = t0 + min((ty + kTy * i) / G, nt - 1);  // rows past the item repeat its last token
#pragma unroll
            for (int x = 0; x < 2 * kCols; ++x)
                o[i][x] = 0;
        }

        for (int k0 = 0; k0 < end; k0 += kKeys) {
            __syncthreads();  // the last block's reads are done
            for (int e = threadIdx.x; e < kKeys * (D / 4); e += kSimtThreads) {
                const int r = e / (D / 4), d = 4 * (e % (D / 4));
                float *dk = sk + r * kLd + d;
                if (k0 + r < end)
                    cp_async_16(dk, k + (static_cast<size_t>(it.row0) + k0 + r) * p.k_stride +
                                        static_cast<size_t>(it.hkv) * D + d);
                else
                    *reinterpret_cast<float4 *>(dk) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            cp_async_commit();
            for (int e = threadIdx.x; e < kKeys * (D / 4); e += kSimtThreads) {
                const int r = e / (D / 4), d = 4 * (e % (D / 4));
                float *dv = sv + r * D + d;
                if (k0 + r < end)
                    cp_async_16(dv, v + (static_cast<size_t>(it.row0) + k0 + r) * p.v_stride +
                                        static_cast<size_t>(it.hkv) * D + d);
                else
                    *reinterpret_cast<float4 *>(dv) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            cp_async_commit();
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // K; V may still be on its way
            __syncthreads();
            uint64_t acc[kRpt][4];
#pragma unroll
            for (int i = 0; i < kRpt; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = 0;
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                ulonglong2 kf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    kf[j] = *reinterpret_cast<const ulonglong2 *>(sk + (tx + 16 * j) * kLd + d);
#pragma unroll
                for (int i = 0; i < kRpt; ++i) {
                    const ulonglong2 qf = *reinterpret_cast<const ulonglong2 *>(sq + (ty + kTy * i) * kLd + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
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
                float x[4];
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
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
                for (int j = 0; j < 4; ++j) {
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
                for (int e = threadIdx.x; e < kKeys * (D / 4); e += kSimtThreads) {
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
                            vf[kk][x] = *reinterpret_cast<const ulonglong2 *>(sv + (key + kk) * D + 4 * tx + 64 * x);
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
                                *reinterpret_cast<const ulonglong2 *>(sv + key * D + 4 * tx + 64 * x);
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
            if (r >= nt * G)
                continue;
            const size_t orow = ((static_cast<size_t>(it.row0) + t0 + r / G) * p.num_q_heads +
                                 it.hkv * G + r % G) * D;
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
                const size_t off = orow + 4 * tx + 64 * x;
                const float2 a = unpair(o[i][2 * x]), b = unpair(o[i][2 * x + 1]);
                const float4 y = make_float4(a.x / sum, a.y / sum, b.x / sum, b.y / sum);
                if (p.out_dtype == PKV_F32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off) = y;
                } else {
                    uint2 w;
                    w.x = pack_bf16(y.x, y.y);
                    w.y = pack_bf16(y.z, y.w);
                    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(p.out) + off) = w;
                }
            }
        }
        __syncthreads();  // the item is read before the next one is written
    }
}

__global__ void __launch_bounds__(kSimtThreads) prompt_ranges_kernel(const PromptParams p)
{
    int start;
    for (int s = threadIdx.x; s < p.num_seqs; s += kSimtThreads)
        prompt_len(p, s, start, true);
}

template <int D> pkv_status launch_simt_d(PromptParams p, cudaStream_t stream)
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
    if (items > 0x40000000L)
        return PKV_ERR_UNSUPPORTED;
    p.max_items = static_cast<unsigned>(items);
    // Two CTAs to an SM; the costliest items go first, one at a time.
    const long slots = 2L * device_sm_count();
    prompt_simt_kernel<D><<<static_cast<unsigned>(items < slots ? items : slots), kSimtThreads,
                            SimtGeom<D>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_prompt_ranges(const PromptParams &p, cudaStream_t stream)
{
    prompt_ranges_kernel<<<1, kSimtThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status launch_prompt_simt(const PromptParams &p, cudaStream_t stream)
{
    return p.head_dim == 128 ? launch_simt_d<128>(p, stream) : launch_simt_d<64>(p, stream);
}

}  // namespace pkv
