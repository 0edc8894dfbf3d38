// Helpers that the tensor-core kernels of whole prompts share: waits that sleep,
// tensor-memory loads, packed arithmetic, the weights of a row of scores.
#pragma once

#include "pkv_tc.cuh"

namespace pkv {

namespace {

// As tc_wait, but asleep until the phase ends: try_wait gives up soon by itself,
// and a thread that then reads the timer and the flag and looks again notices
// the end late and takes issue slots from the softmax warps.  The softmax warps' own
// waits are short and keep tc_wait.  Asleep none / the others / all: a chat batch
// (128 prompts of 256 to 512 tokens, 64 heads over 8) 516 / 498 / 498 us, a 32K prompt 5.59 / 5.50 / 5.75 ms.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)  // ns
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool sleep_wait(uint64_t *bar, uint32_t parity, const volatile int *abort)
{
    if (mbar_try_wait_long(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_long(bar, parity))
            return true;
        if (*abort)
            return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs)
            return false;
    }
}
__device__ __forceinline__ bool warp_sleep_wait(uint64_t *bar, uint32_t parity, const volatile int *abort)
{
    return __all_sync(kFullMask, sleep_wait(bar, parity, abort));
}

// 32 columns of the warp's 32 lanes.  Load and wait are one statement: between
// two, the compiler may copy registers that the load has yet to fill.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
          "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
          "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
          "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
          "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
// 64 columns.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&x)[32], float (&y)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,"
        "%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,"
        "%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
          "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]),
          "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]),
          "=f"(x[18]), "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]),
          "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]), "=f"(x[28]), "=f"(x[29]),
          "=f"(x[30]), "=f"(x[31]),
          "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]),
          "=f"(y[6]), "=f"(y[7]), "=f"(y[8]), "=f"(y[9]), "=f"(y[10]), "=f"(y[11]),
          "=f"(y[12]), "=f"(y[13]), "=f"(y[14]), "=f"(y[15]), "=f"(y[16]), "=f"(y[17]),
          "=f"(y[18]), "=f"(y[19]), "=f"(y[20]), "=f"(y[21]), "=f"(y[22]), "=f"(y[23]),
          "=f"(y[24]), "=f"(y[25]), "=f"(y[26]), "=f"(y[27]), "=f"(y[28]), "=f"(y[29]),
          "=f"(y[30]), "=f"(y[31])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}

// Two f32 fused multiply-adds / adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t x, y, z, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t x, y, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}

// Scores at and past `lim` become -inf.
__device__ __forceinline__ void mask32(float (&x)[32], int lim)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        x[e] = e < lim ? x[e] : -INFINITY;
}

__device__ __forceinline__ float max32(const float (&x)[32])
{
    float a[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
        a[f] = fmaxf(x[f], x[4 + f]);
#pragma unroll
    for (int e = 8; e < 32; e += 8)
#pragma unroll
        for (int f = 0; f < 4; ++f)
            a[f] = fmaxf(a[f], fmaxf(x[e + f], x[e + 4 + f]));
    return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

// Weights 2^(c x + off) of 32 scores: added to the sums l, stored as bf16 pairs
// at column `col` (and what the rounding leaves, 16 columns on).  Sixteen at
// a time, stage by stage, so that neighbouring instructions are independent.
template <bool kSplit>
__device__ __forceinline__ void weights32(const float (&x)[32], float c, float off, float2 (&l)[2], uint32_t col)
{
    const float2 c2 = make_float2(c, c), off2 = make_float2(off, off);
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float2 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = fma2(make_float2(x[16 * g + 2 * e], x[16 * g + 2 * e + 1]), c2, off2);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = make_float2(MmaSoftmax::ex2(w[e].x), MmaSoftmax::ex2(w[e].y));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            hi[8 * g + e] = pack_bf16(w[e].x, w[e].y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            l[e % 2] = add2(l[e % 2], w[e]);
        if constexpr (kSplit)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                lo[8 * g + e] = pack_bf16(w[e].x - bf16_lo(hi[8 * g + e]), w[e].y - bf16_hi(hi[8 * g + e]));
    }
    tmem_st16u(col, hi);
    if constexpr (kSplit)
        tmem_st16u(col + 16, lo);
}

}  // namespace

}  // namespace pkv
