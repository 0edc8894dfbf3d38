// Causal attention over whole prompts on the tcgen05 tensor cores (bf16).
//
// softmax(scale * q K^T) V of the "Inference optimization" lesson (Step 2,
// scaled_dot_product_attention with its causal mask), one pass over the keys
// with the running maximum and sum of the softmax.  A row is one (token,
// grouped query head) pair; the G heads of a group read the same K and V.
//
// Layout on the GPU:
//  * A tile is 128 rows: R = 128 / G consecutive tokens (rounded down) with
//    their G heads.  An item is two neighbouring tiles of one sequence and KV
//    head: every K and V block of 128 keys that reaches shared memory serves
//    256 rows (a tile alone would ask L2 for 64 bytes a cycle and SM).  One
//    persistent CTA per SM walks the items.
//  * Warps 0-3 own the rows of tile 0 (a thread per row, which is its TMEM
//    lane), 4-7 those of tile 1.  One thread of warp 8 issues the TMA loads, one
//    of warp 9 the MMAs; warp 10 looks the items up ahead of all of them, warp
//    11 watches the loads for the MMA thread, warps 12-15 write the outputs.
//  * TMEM: scores of both tiles (2 x 128 columns, P written back over them as
//    bf16) and both outputs (2 x head_dim columns).  Per block and tile:
//    S = Q K^T from shared memory; the rows' threads read S, apply the limit
//    and the softmax and write P; O += P V with P read from TMEM.  While one
//    tile's threads work, the tensor cores run the other tile's products; P is
//    handed over in two parts of 64 keys, so that P V starts before the last
//    weights are there.
//  * All shared-memory operands are in the 128-byte swizzle mode: [128 rows]
//    [64 elements] per half of head_dim, K-major for Q and K, MN-major for V.
//  * The last block of an item is cut to its keys in steps of 16 (N of S, K of
//    P V).
//  * The running maximum is raised only when a score exceeds it by 2^8; O is
//    then rescaled in TMEM by the rows' threads.
//  * P V multiplies a masked weight 0 with the V rows of later tokens in the
//    diagonal block, which may hold infinities or NaN.  Rows past the item's
//    keys are zeroed in shared memory; items with an output that is not finite
//    are looked at again by all warps after the CTA's last one (redo_items): in
//    between, the other roles would have to wait for it.
//  * Every wait is bounded; a timeout records PKV_ERR_TIMEOUT, stops every role,
//    lets copies and MMAs in flight finish and frees TMEM.
//
// What bounds it.  Long prompts: the tensor cores (a 32K prompt of 32 heads of
// 128 over 8 KV heads: 5.7 to 5.85 ms, 1.5 PFLOP/s, 90% of what a cuBLAS product
// sustains on the same part; a burst takes 5.5 ms).  A block takes them 2 x 1024 cycles; a tile's
// softmax of about 1200 cycles hides behind the other tile's products.  The
// queue of the tensor cores holds about three MMAs, so the issuing thread may
// spend only some 200 cycles between two groups: hence one barrier per group
// (the gate), one commit per step for the ring, and a loop of its own for
// whole blocks.  Short prompts (128 of 256 to 512 tokens, 64 heads: 500 us,
// 3.6 TB/s): the chain load - S - softmax - P V - store of items two blocks long,
// and the issuing thread's general steps.  With heads of 64 (37 prompts of up to
// 1000 tokens, 24/2 heads: 96 us): the same steps, some 4500 cycles each for 1000
// of products, and scores that wait for P V because P lies over them.
//
// Bits of P.  A bf16 output takes its weights rounded to bf16 (2^-8 of each at
// most), an f32 output in two bf16 parts (2^-16), which is twice the products of
// P V.  Against 64 bits the bf16 outputs are then 0.0017 to 0.0020 off (2-norm),
// of which 0.0014 to 0.0016 is the rounding of the output itself.  One part / two,
// us: chat batch 499 / 676, 16 prompts of 512 to 4096 tokens 530 / 739, 32K prompt
// 5713 / 7997, heads of 64 above 104 / 131.
//
// Measured and not taken (32K prompt / chat batch, 5.7 ms / 521 us then): an issuing thread
// per tile 8.1 ms / 501 us (both tiles' products run interleaved, then both
// softmaxes; taking turns costs more), scores kept in registers between the
// maximum and the weights 5.9 ms / 530 us (spills, and code that leaves the
// instruction caches), two threads per row 8.3 ms / 945 us, the outputs written by
// the softmax warps 5.8 ms / 525 us, Q prefetched into L2 5.7 ms / 558 us.
#include <climits>
#include <type_traits>

#include "pkv_prompt.cuh"
#include "pkv_tc.cuh"

namespace pkv {

namespace {

constexpr int kM = 128;     // rows of a tile
constexpr int kKeys = 128;  // keys of a block
constexpr int kThreads = 512;
constexpr int kTileWarps = 4;     // warps 0 .. 7: the rows of two tiles
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kItemWarp = 10;
constexpr int kGateWarp = 11;     // 12 .. 15: the outputs
constexpr int kSteps = 4;         // barriers of the MMA thread's steps
constexpr int kParts = 2;         // a block's P is handed to the MMAs in parts
constexpr int kPart = kKeys / kParts;
constexpr int kQueue = 4;         // items looked up ahead
constexpr int kHalf = 128 * 128;  // bytes of [128 rows][64 bf16]

template <int D> struct PtGeom {
    static constexpr int kTile = D / 64 * kHalf;
    static constexpr int NS = D == 128 ? 5 : 8;   // K / V tiles in the ring
    static constexpr int kSmem = (2 + NS) * kTile + 1024;
    static constexpr int kOCol = 2 * kKeys;       // outputs follow the scores
    static_assert(kOCol + 2 * D <= 512, "scores and outputs fill TMEM");
};

struct PromptMaps {
    CUtensorMap q, k, v;
};

// One queue entry: an item, or s < 0 for the end of the work.
struct PtItem {
    int s, hkv, row0, n, tok0;
    int nt[2];   // tokens of the two tiles
    int end[2];  // keys a tile sees
    int nb[2];   // its blocks
    int blocks;  // blocks loaded

    __device__ __forceinline__ void fill(const int *w, int R)
    {
        s = w[0];
        hkv = w[1];
        row0 = w[2];
        n = w[3];
        tok0 = w[4];
        nt[0] = min(R, n - tok0);
        nt[1] = max(0, min(R, n - tok0 - R));
        end[0] = tok0 + nt[0];
        end[1] = end[0] + nt[1];
        nb[0] = (end[0] + kKeys - 1) / kKeys;
        nb[1] = nt[1] > 0 ? (end[1] + kKeys - 1) / kKeys : 0;
        blocks = max(nb[0], nb[1]);
    }
};

// Keys of block j that a tile of nb blocks ending at key `end` multiplies, in
// steps of 16.
__device__ __forceinline__ int block_cols(int nb, int end, int j)
{
    return j + 1 < nb ? kKeys : (end - j * kKeys + 15) & ~15;
}

// As tc_wait, but asleep until the phase ends: try_wait gives up soon by itself,
// and a thread that then reads the timer and the flag and looks again notices
// the end late and takes issue slots from the softmax warps.  The softmax warps' own
// waits are short and keep tc_wait.  Asleep none / the others / all: chat batch
// (above) 516 / 498 / 498 us, a 32K prompt 5.59 / 5.50 / 5.75 ms.
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

// Shared-memory descriptor of a 128-byte-swizzled operand (atoms of 8 rows x
// 128 bytes).  Low word: address / 16, and from bit 16 the distance / 16 of
// atoms along the contiguous axis (MN-major only).  High word: the distance /
// 16 of 8-row groups, descriptor version 1 (bit 14), layout code 2 (bit 29).
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi)
{
    return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u));
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

// 32 consecutive columns of an output row, f32 or bf16.  With 32-byte stores a
// lane fills whole sectors (`wide`: the output is aligned for them).
template <bool kF32>
__device__ __forceinline__ void store_out32(const PromptParams &p, size_t off, const float *v, bool wide)
{
    unsigned char *dst = static_cast<unsigned char *>(p.out) + off * (kF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = kF32 ? __float_as_uint(v[8 * i + e]) : pack_bf16(v[16 * i + 2 * e], v[16 * i + 2 * e + 1]);
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 32 * i),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
                         "r"(w[7])
                         : "memory");
        } else {
            uint4 *d = reinterpret_cast<uint4 *>(dst + 32 * i);
            d[0] = make_uint4(w[0], w[1], w[2], w[3]);
            d[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// ------------------------------------------- rows with values not to be seen

// Where V is not finite, the products above may be wrong: a masked weight 0
// times an infinity or NaN of a later row is NaN, and with P in two parts so is
// an infinity that the row does see times a part that is zero or negative.  The
// output warps note the items with an output that is not finite; when the CTA's
// last item is done, all its warps go through them again.
//
// A dim of a row is told from the first NaN and infinities of either sign that
// V holds in it: those at or before the row decide the output (NaN; or the
// infinity, as the weight of a finite score is positive), those after it must
// not reach it.  Only where the row sees none and a later one spoilt the sum is
// the sum computed again, with V's NaN and infinities as zeros and the item's
// keys in steps of 64 through shared memory (mma.sync, a warp for 16 rows, P in
// two parts).  So a row costs at most one such pass, and nothing but the look at
// V where the NaN is its own.  An 8K prompt of 32/8 heads (371 us): V all NaN
// 1.1 ms, its last token NaN 1.3 ms, every 10^4-th value NaN 3.1 ms; a chat batch
// (500 us) at most 3.9 ms.
constexpr int kRedoKeys = 64;

template <int D> struct RedoSmem {
    static constexpr int kLd = D + 8;           // rows of Q and K: 4 banks apart
    static constexpr int kVLd = kRedoKeys + 8;  // and of V, which is transposed
    int nan_at[D], pinf_at[D], ninf_at[D];      // first row of V with one
    int last[2][D];                             // last one among a tile's products
    int first;                                  // first token with an output to look at
    int upto;                                   // last token to be computed again
    int key_bad;                                // first row of K that is not finite
    alignas(16) unsigned short q[2 * kM * kLd];
    alignas(16) unsigned short k[kRedoKeys * kLd];
    alignas(16) unsigned short v[D * kVLd];
};

// The e-th bf16 of two or four loaded as one word, as its bits.
__device__ __forceinline__ uint32_t bf16_bits(uint32_t x, int e) { return e ? x >> 16 : x & 0xffffu; }
__device__ __forceinline__ uint32_t bf16_bits(uint2 x, int e) { return bf16_bits(e & 2 ? x.y : x.x, e & 1); }
__device__ __forceinline__ bool bf16_bad(uint32_t bits) { return (bits & 0x7fffu) >= 0x7f80u; }
template <typename Dims, int kPer> __device__ __forceinline__ bool any_bad(Dims x)
{
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        bad = bad || bf16_bad(bf16_bits(x, e));
    return bad;
}

template <bool kF32> __device__ __forceinline__ float load_out(const PromptParams &p, size_t at)
{
    if constexpr (kF32)
        return static_cast<const float *>(p.out)[at];
    else
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.out)[at]);
}
template <bool kF32> __device__ __forceinline__ void store_out(const PromptParams &p, size_t at, float y)
{
    if constexpr (kF32)
        static_cast<float *>(p.out)[at] = y;
    else
        static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16(y);
}

// Rows [from, to) of the item's V (and K): first and last bad ones per dim.  A
// lane has D / 32 dims, a warp eight rows at a time so that their loads overlap.
template <int D>
__device__ __noinline__ void redo_look(const PromptParams &p, RedoSmem<D> &sm, const PtItem &it, int from, int to,
                                       int end0, int end1)
{
    constexpr int kPer = D / 32;
    using Dims = std::conditional_t<kPer == 4, uint2, uint32_t>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned short *kb = static_cast<const unsigned short *>(p.k) +
                               static_cast<size_t>(it.row0) * p.k_stride + it.hkv * D + lane * kPer;
    const unsigned short *vb = static_cast<const unsigned short *>(p.v) +
                               static_cast<size_t>(it.row0) * p.v_stride + it.hkv * D + lane * kPer;
    int first_nan[kPer], first_p[kPer], first_n[kPer], last0[kPer], last1[kPer], key_bad = INT_MAX;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        first_nan[e] = first_p[e] = first_n[e] = INT_MAX;
        last0[e] = last1[e] = -1;
    }
    for (int j0 = from + 8 * warp; j0 < to; j0 += 8 * (kThreads / 32)) {
        Dims kw[8], vw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t j = min(j0 + i, to - 1);
            kw[i] = *reinterpret_cast<const Dims *>(kb + j * p.k_stride);
            vw[i] = *reinterpret_cast<const Dims *>(vb + j * p.v_stride);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = min(j0 + i, to - 1);
            // A score that is not finite gives an infinite V row no positive weight.
            const bool kbad = __any_sync(kFullMask, any_bad<Dims, kPer>(kw[i]));
            if (kbad)
                key_bad = min(key_bad, j);
            if (!any_bad<Dims, kPer>(vw[i]))
                continue;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t x = bf16_bits(vw[i], e);
                if (!bf16_bad(x))
                    continue;
                if ((x & 0x7fffu) != 0x7f80u || kbad)
                    first_nan[e] = min(first_nan[e], j);
                else if (x & 0x8000u)
                    first_n[e] = min(first_n[e], j);
                else
                    first_p[e] = min(first_p[e], j);
                if (j < end0)
                    last0[e] = max(last0[e], j);
                if (j < end1)
                    last1[e] = max(last1[e], j);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int d = lane * kPer + e;
        atomicMin(&sm.nan_at[d], first_nan[e]);
        atomicMin(&sm.pinf_at[d], first_p[e]);
        atomicMin(&sm.ninf_at[d], first_n[e]);
        atomicMax(&sm.last[0][d], last0[e]);
        atomicMax(&sm.last[1][d], last1[e]);
    }
    if (lane == 0)
        atomicMin(&sm.key_bad, key_bad);
}

// Dim d of a row at token `pos`: NaN or an infinity when the row sees one, else 0.
template <int D> __device__ __forceinline__ float seen_value(const RedoSmem<D> &sm, int d, int pos)
{
    const bool up = sm.pinf_at[d] <= pos, down = sm.ninf_at[d] <= pos;
    if (sm.nan_at[d] <= pos || (up && down))
        return __int_as_float(0x7fffffff);
    return up ? INFINITY : down ? -INFINITY : 0.f;
}

// The sums of the rows `rows` of this warp's 16 once more, and their outputs where they
// were not finite.  All warps of the CTA call it.
template <int D, bool kF32>
__device__ __noinline__ void redo_rows(const PromptParams &p, RedoSmem<D> &sm, const PtItem &it, unsigned rows)
{
    using Sm = RedoSmem<D>;
    constexpr int kLd = Sm::kLd, kVLd = Sm::kVLd;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, tq = lane & 3;  // fragment row, and pair of columns
    const int G = p.group, R = kM / G;
    const unsigned short *qb = static_cast<const unsigned short *>(p.q) + static_cast<size_t>(it.hkv) * G * D;
    const unsigned short *kb = static_cast<const unsigned short *>(p.k) + it.hkv * D;
    const unsigned short *vb = static_cast<const unsigned short *>(p.v) + it.hkv * D;
    const int keys = min(sm.upto + 1, it.n);

    for (int e = threadIdx.x; e < 2 * kM * (D / 8); e += kThreads) {
        const int r = e / (D / 8), c = e % (D / 8), t = r / kM, rr = r % kM;
        const int nt = t ? it.nt[1] : it.nt[0];
        uint4 x = make_uint4(0, 0, 0, 0);
        if (rr < nt * G)
            x = *reinterpret_cast<const uint4 *>(
                qb + (static_cast<size_t>(it.row0) + it.tok0 + t * R + rr / G) * p.q_stride + (rr % G) * D + 8 * c);
        *reinterpret_cast<uint4 *>(sm.q + r * kLd + 8 * c) = x;
    }

    int pos[2];        // tokens of fragment rows g and g + 8, or -1
    size_t orow[2];    // and their outputs
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int rr = 16 * (warp & 7) + g + 8 * i, t = warp >> 3;
        const int tok = it.tok0 + t * R + rr / G;
        pos[i] = rows >> (g + 8 * i) & 1u ? tok : -1;
        orow[i] = (static_cast<size_t>(it.row0 + tok) * p.num_q_heads + it.hkv * G + rr % G) * D;
    }
    const int my_keys = rows ? __reduce_max_sync(kFullMask, max(pos[0], pos[1])) + 1 : 0;
    const float c = p.negate ? -p.score_scale : p.score_scale;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[n][e] = 0.f;

    for (int k0 = 0; k0 < keys; k0 += kRedoKeys) {
        __syncthreads();  // the keys before these are used
        for (int e = threadIdx.x; e < kRedoKeys * (D / 8); e += kThreads) {
            const int r = e / (D / 8), d = 8 * (e % (D / 8));
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (k0 + r < keys) {
                const int64_t row = static_cast<int64_t>(it.row0) + k0 + r;
                x = *reinterpret_cast<const uint4 *>(kb + row * p.k_stride + d);
                y = *reinterpret_cast<const uint4 *>(vb + row * p.v_stride + d);
            }
            *reinterpret_cast<uint4 *>(sm.k + r * kLd + d) = x;
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = bf16_bits(w[i / 2], i & 1);
                sm.v[(d + i) * kVLd + r] = static_cast<unsigned short>(bf16_bad(b) ? 0u : b);
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int h = k0; h < min(k0 + kRedoKeys, my_keys); h += 32) {
            const int at = h - k0;
            float s[4][4] = {};
#pragma unroll 2
            for (int ks = 0; ks < D / 16; ++ks) {
                const unsigned short *qr = sm.q + (16 * warp + g) * kLd + 16 * ks + 2 * tq;
                const uint32_t a[4] = {*reinterpret_cast<const uint32_t *>(qr),
                                       *reinterpret_cast<const uint32_t *>(qr + 8 * kLd),
                                       *reinterpret_cast<const uint32_t *>(qr + 8),
                                       *reinterpret_cast<const uint32_t *>(qr + 8 * kLd + 8)};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const unsigned short *kr = sm.k + (at + 8 * n + g) * kLd + 16 * ks + 2 * tq;
                    mma_bf16(s[n], a, *reinterpret_cast<const uint32_t *>(kr),
                             *reinterpret_cast<const uint32_t *>(kr + 8));
                }
            }
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[n][2 * i + e];
                        x = h + 8 * n + 2 * tq + e <= pos[i] ? x * c : -INFINITY;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
                mx = fmaxf(mx, m[i]);
                // Nothing but -inf so far: any finite offset gives weights 0.
                const float off = mx == -INFINITY ? 0.f : mx;
                alpha[i] = MmaSoftmax::ex2(m[i] - off);
                m[i] = mx;
                l[i] *= alpha[i];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[n][2 * i + e];
                        x = MmaSoftmax::ex2(x - off);
                        l[i] += x;
                    }
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[n][e] *= alpha[e / 2];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // rows g, g + 8 of the chunk's keys, then of its last eight
                    const float x = s[2 * kc + i / 2][2 * (i & 1)], y = s[2 * kc + i / 2][2 * (i & 1) + 1];
                    hi[i] = pack_bf16(x, y);
                    lo[i] = pack_bf16(x - bf16_lo(hi[i]), y - bf16_hi(hi[i]));
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    const unsigned short *vr = sm.v + (8 * n + g) * kVLd + at + 16 * kc + 2 * tq;
                    const uint32_t b0 = *reinterpret_cast<const uint32_t *>(vr),
                                   b1 = *reinterpret_cast<const uint32_t *>(vr + 8);
                    mma_bf16(o[n], hi, b0, b1);
                    mma_bf16(o[n], lo, b0, b1);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float sum = l[i];
        sum += __shfl_xor_sync(kFullMask, sum, 1);
        sum += __shfl_xor_sync(kFullMask, sum, 2);
        if (pos[i] < 0)
            continue;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = 8 * n + 2 * tq + e;
                const float y = load_out<kF32>(p, orow[i] + d);
                if (!(y * 0.f == 0.f))  // the others stand
                    store_out<kF32>(p, orow[i] + d, seen_value(sm, d, pos[i]) + o[n][2 * i + e] / sum);
            }
    }
}

// The k-th item of this CTA.  Alternating direction: a CTA late in one row of
// items is early in the next, so that the CTAs' totals stay even.
__device__ __forceinline__ unsigned item_number(unsigned k)
{
    return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// The items first .. last of this CTA once more, by all its warps: warp w has rows
// 16 w .. 16 w + 15 of an item's 256.
template <int D, bool kSplit>
__device__ __noinline__ void redo_items(const PromptParams &p, unsigned char *smem, unsigned first, unsigned last)
{
    constexpr int kPer = D / 32;
    using Dims = std::conditional_t<kPer == 4, uint2, uint32_t>;
    RedoSmem<D> &sm = *reinterpret_cast<RedoSmem<D> *>(smem);
    static_assert(sizeof(RedoSmem<D>) <= PtGeom<D>::kSmem - 1024, "fits where the ring was");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.group, R = kM / G;
    const int t = warp >> 3;
    PromptScan scan;
    scan.init(p, 2 * R, lane, false);
    for (unsigned k = first; k <= last; ++k) {
        const PromptItem found = scan.find(p, 2 * R, item_number(k), lane);
        const int w[5] = {found.s, found.hkv, found.row0, found.n, found.index * 2 * R};
        PtItem it;
        it.fill(w, R);
        // Keys that the products of the tiles have gone through.
        const int item_end = max(it.end[0], it.end[1]);
        int key_end[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            key_end[x] = it.nb[x] == 0 ? 0
                                       : min((it.nb[x] - 1) * kKeys + block_cols(it.nb[x], it.end[x], it.nb[x] - 1),
                                             item_end);
        const int tok = it.tok0 + t * R, nt = t ? it.nt[1] : it.nt[0];
        __syncthreads();  // the item before has left shared memory
        if (threadIdx.x < D) {
            sm.nan_at[threadIdx.x] = sm.pinf_at[threadIdx.x] = sm.ninf_at[threadIdx.x] = INT_MAX;
            sm.last[0][threadIdx.x] = sm.last[1][threadIdx.x] = -1;
        }
        if (threadIdx.x == 0) {
            sm.first = sm.key_bad = INT_MAX;
            sm.upto = -1;
        }
        __syncthreads();
        // Outputs of this lane's dims that are not finite, kPer bits a row.
        uint64_t bad = 0;
        unsigned rows = 0;
        for (int i = 0; i < 16; ++i) {
            const int r = 16 * (warp & 7) + i;
            if (r >= nt * G)
                break;
            const size_t at = (static_cast<size_t>(it.row0 + tok + r / G) * p.num_q_heads + it.hkv * G + r % G) * D;
            uint64_t b = 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float y = load_out<kSplit>(p, at + lane * kPer + e);
                b |= static_cast<uint64_t>(!(y * 0.f == 0.f)) << e;
            }
            bad |= b << (kPer * i);
            rows |= __any_sync(kFullMask, b != 0) ? 1u << i : 0u;
        }
        if (rows && lane == 0)
            atomicMin(&sm.first, tok + (16 * (warp & 7) + __ffs(rows) - 1) / G);
        if (!__syncthreads_or(rows != 0))
            continue;
        // What they must not see first: mostly nothing, and the outputs stand.
        const int from = kSplit ? 0 : sm.first + 1;
        redo_look<D>(p, sm, it, from, max(key_end[0], key_end[1]), key_end[0], key_end[1]);
        __syncthreads();
        if (!kSplit) {
            bool hidden = false;
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    hidden = hidden || ((bad >> (kPer * i + e) & 1) &&
                                        sm.last[t][lane * kPer + e] > tok + (16 * (warp & 7) + i) / G);
            if (!__syncthreads_or(hidden))
                continue;
            redo_look<D>(p, sm, it, 0, from, key_end[0], key_end[1]);
            __syncthreads();
        }
        unsigned again = 0;  // rows whose sums are computed again
        for (unsigned left = rows; left; left &= left - 1) {
            const int i = __ffs(left) - 1, r = 16 * (warp & 7) + i, pos = tok + r / G;
            const size_t head = it.hkv * G + r % G, row = it.row0 + pos;
            float y[kPer];
            int write = 0;  // dims of this lane to be written
            bool sum = false;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int d = lane * kPer + e;
                const bool here = bad >> (kPer * i + e) & 1, hidden = sm.last[t][d] > pos;
                y[e] = seen_value(sm, d, pos);
                sum = sum || (here && hidden && y[e] == 0.f);
                if (here && (kSplit || hidden) && fabsf(y[e]) == INFINITY)
                    write |= 1 << e;
            }
            sum = __any_sync(kFullMask, sum);
            if (!sum && !__any_sync(kFullMask, write != 0))
                continue;
            if (!sum) {
                // An infinity has a positive weight if the scores are finite: else look.
                const Dims qw = *reinterpret_cast<const Dims *>(static_cast<const unsigned short *>(p.q) +
                                                                row * p.q_stride + head * D + lane * kPer);
                sum = sm.key_bad <= pos || __any_sync(kFullMask, any_bad<Dims, kPer>(qw));
            }
            if (sum) {
                again |= 1u << i;
                continue;
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (write >> e & 1)
                    store_out<kSplit>(p, (row * p.num_q_heads + head) * D + lane * kPer + e, y[e]);
        }
        if (again && lane == 0)
            atomicMax(&sm.upto, tok + (16 * (warp & 7) + 31 - __clz(again)) / G);
        if (__syncthreads_or(again != 0))
            redo_rows<D, kSplit>(p, sm, it, again);
    }
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ PromptMaps maps)
{
    using Geo = PtGeom<D>;
    constexpr int NS = Geo::NS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], step_done[kSteps];
    __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][kParts], o_full[2],
        o_free[2], l_full[2];
    __shared__ __align__(8) uint64_t item_full[kQueue], item_empty[kQueue], drain;
    __shared__ int s_item[kQueue][5];
    __shared__ float s_sum[2][kM];  // the rows' sums of weights, for the output warps
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ unsigned s_redo[2];  // first and last item with an output that is not finite
    volatile int *abort = &s_abort;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t smem0 = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (smem0 - raw);
    const int G = p.group;
    const int R = kM / G;  // tokens of a tile

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
        }
        for (int i = 0; i < kSteps; ++i)
            mbar_init(&step_done[i], 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_empty[t], 1);
            mbar_init(&s_full[t], 1);
            for (int i = 0; i < kParts; ++i)
                mbar_init(&p_full[t][i], kTileWarps + (t == 0 && i == 0));  // and the gate
            mbar_init(&o_full[t], 1);
            mbar_init(&l_full[t], kTileWarps);
            mbar_init(&o_free[t], kTileWarps);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 3 * kTileWarps + 3);
        }
        mbar_init(&drain, 1);
        s_abort = 0;
        s_redo[0] = ~0u;
        s_redo[1] = 0;
        fence_mbar_init();
    }
    if (warp == kProducerWarp && lane < 3) {
        const CUtensorMap *map = lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Q rows past G * R are never loaded: zero.
    for (int e = threadIdx.x; e < 2 * (D / 64) * (kM - G * R) * 8; e += kThreads) {
        const int per = (kM - G * R) * 8;  // 16-byte pieces of one half
        *reinterpret_cast<uint4 *>(smem + (e / per) * kHalf + (G * R * 8 + e % per) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const uint32_t ring0 = smem0 + 2 * Geo::kTile;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------- copies
        if (lane == 0) {
            uint32_t kv = 0;          // tiles issued
            uint32_t steps = 0;       // steps of the MMA thread seen done
            uint32_t qn[2] = {0, 0};  // Q tiles issued
            bool ok = true;
            auto load = [&](const CUtensorMap *map, const PtItem &it, int j) {
                const uint32_t st = kv % NS;
                // Step i (from 0) gives back tiles 2 i - 1 and 2 i of the ring's
                // sequence K, V, K, V, ...: V of a block and the next K.
                for (; kv >= NS && 2 * steps < kv - NS + 2; ++steps)
                    if (!sleep_wait(&step_done[steps % kSteps], (steps / kSteps) & 1, abort))
                        return false;
                mbar_arrive_expect_tx(&full[st], Geo::kTile);
                for (int h = 0; h < D / 64; ++h) {
                    if (p.drop_first_copy && blockIdx.x == 0 && kv == 0 && h == 0)
                        continue;
                    tma_load_3d(smem + (2 + st) * Geo::kTile + h * kHalf, map, 64 * h, it.hkv,
                                it.row0 + j * kKeys, &full[st]);
                }
                ++kv;
                return true;
            };
            for (unsigned k = 0; ok; ++k) {
                const int slot = k % kQueue;
                ok = sleep_wait(&item_full[slot], (k / kQueue) & 1, abort);
                if (!ok)
                    break;
                PtItem it;
                it.fill(s_item[slot], R);
                mbar_arrive(&item_empty[slot]);
                if (it.s < 0)
                    break;
                for (int j = 0; j < it.blocks && ok; ++j) {
                    ok = load(&maps.k, it, j);
                    for (int t = 0; t < 2 && j == 0 && ok; ++t) {
                        if (it.nt[t] == 0)
                            continue;
                        if (qn[t] > 0)
                            ok = sleep_wait(&q_empty[t], (qn[t] - 1) & 1, abort);
                        if (!ok)
                            break;
                        mbar_arrive_expect_tx(&q_full[t], (D / 64) * G * R * 128);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(smem + t * Geo::kTile + h * kHalf, &maps.q, 64 * h,
                                        it.hkv * G, it.row0 + it.tok0 + t * R, &q_full[t]);
                        ++qn[t];
                    }
                    ok = ok && load(&maps.v, it, j);
                }
            }
            if (!ok) {
                set_status(p.status, PKV_ERR_TIMEOUT);
                *abort = 1;
            }
            // Every copy still in flight lands before the CTA exits, also when
            // another role gives up after the last one was issued.
            for (uint32_t c = kv > NS ? kv - NS : 0; c < kv; ++c)
                mbar_wait_bounded(&full[c % NS], (c / NS) & 1, kWaitLimitNs);
            for (int t = 0; t < 2; ++t)
                if (qn[t] > 0)
                    mbar_wait_bounded(&q_full[t], (qn[t] - 1) & 1, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == kGateWarp) {
        // ------------------------------------------------------- K / V gate
        // Waits for V of block j and K of the next one and counts as the fifth
        // arrival on tile 0's first part of P, so that the MMA thread has one
        // barrier to look at where it would have three.  It looks at no other
        // load: the ring gives a slot back when the MMA thread has used it, and
        // only the arrival that follows holds the MMA thread back until the
        // gate has seen the slot full.  A wait for K of an item's first block,
        // or for V that only tile 1 sees, could come a whole turn of the ring
        // late and never end.
        if (lane == 0) {
            uint32_t st = 0, par = 0;
            uint32_t blocks = 0;  // of tile 0
            bool ok = true;
            auto pass = [&](bool look) {  // one tile of the ring
                if (look && p.slow_gate)
                    for (int i = 0; i < 20; ++i)
                        __nanosleep(1000);
                ok = ok && (!look || sleep_wait(&full[st], par, abort));
                if (++st == NS) {
                    st = 0;
                    par ^= 1;
                }
            };
            for (unsigned k = 0; ok; ++k) {
                const int slot = k % kQueue;
                ok = sleep_wait(&item_full[slot], (k / kQueue) & 1, abort);
                if (!ok)
                    break;
                PtItem it;
                it.fill(s_item[slot], R);
                mbar_arrive(&item_empty[slot]);
                if (it.s < 0)
                    break;
                // K of block 0, which the MMA thread waits for itself, is tile 0.
                for (int i = 0, tiles = 2 * it.blocks; i < tiles && ok; ++i) {
                    const int j = (i - 1) >> 1;  // the block whose step uses it
                    const bool gated = i > 0 && j < it.nb[0];
                    pass(gated);
                    // After K of the next block, or the last V.
                    if (!gated || ((i & 1) && i + 1 < tiles))
                        continue;
                    // Not before the block before has all its arrivals.
                    if (blocks > 0)
                        ok = ok && sleep_wait(&p_full[0][0], (blocks - 1) & 1, abort);
                    ++blocks;
                    if (ok)
                        mbar_arrive(&p_full[0][0]);
                }
            }
            if (!ok) {
                set_status(p.status, PKV_ERR_TIMEOUT);
                *abort = 1;
            }
        }
        __syncwarp();
    } else if (warp == kItemWarp) {
        // -------------------------------------------------- item look-up
        PromptScan scan;
        scan.init(p, 2 * R, lane, blockIdx.x == 0);
        bool ok = true;
        for (unsigned k = 0; ok; ++k) {
            const PromptItem found = scan.find(p, 2 * R, item_number(k), lane);
            if (lane == 0) {
                const int slot = k % kQueue;
                if (k >= kQueue)
                    ok = sleep_wait(&item_empty[slot], ((k / kQueue) - 1) & 1, abort);
                if (ok) {
                    int *w = s_item[slot];
                    w[0] = found.s;
                    w[1] = found.hkv;
                    w[2] = found.row0;
                    w[3] = found.n;
                    w[4] = found.index * 2 * R;
                    mbar_arrive(&item_full[slot]);
                } else {
                    set_status(p.status, PKV_ERR_TIMEOUT);
                    *abort = 1;
                }
            }
            ok = __shfl_sync(kFullMask, ok ? 1 : 0, 0) != 0 && found.s >= 0;
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------- MMA issue
        // One thread for both tiles, which keeps them out of phase: while one
        // tile's rows are in the softmax the other's products run.  A step is,
        // tile after tile, P V of block j and the scores of the next block;
        // after an item's last block these are the next item's first scores,
        // which its threads find when their output is written.  The tensor
        // cores queue about three MMAs (200 cycles), so little may stand
        // between one group of eight and the next: the steps in which every
        // block is whole have a loop of their own.
        if (lane == 0) {
            // A negative scale negates Q (instruction descriptor bit 13).
            const uint32_t id_s0 = tc_idesc(kM, 0, false) | (p.negate ? 1u << 13 : 0u);
            constexpr uint32_t kIdPV = tc_idesc(kM, D, true);
            constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
            constexpr uint32_t kTileLo = Geo::kTile >> 4;
            const uint32_t qlo = (smem0 >> 4) | 1u << 16;
            const uint32_t klo0 = (ring0 >> 4) | 1u << 16, vlo0 = (ring0 >> 4) | (kHalf >> 4) << 16;
            uint32_t vst = NS - 1, vpar = 1, kst = 0, kpar = 0;  // ring positions of V (j) and K (next)
            uint32_t q_par = 0, o_par = 3, p_par = 0;            // bit t
            uint32_t step = 0;
            unsigned k = 0;
            bool ok = true;
            // Eight MMAs of S (head_dim 128) for tile t, and of P V per part.
            auto mma_s = [&](uint32_t t, uint32_t id) {
                const uint32_t klo = klo0 + kst * kTileLo, q = qlo + t * kTileLo;
                const uint32_t d = tmem + t * kKeys;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * kHalf + (ks % 4) * 32) >> 4;
                    tc_mma_ss(d, desc64(q + o, kDescHi), desc64(klo + o, kDescHi), id, ks > 0);
                }
            };
            auto mma_pv = [&](uint32_t t, int part, int steps, bool first) {
                const uint32_t vlo = vlo0 + vst * kTileLo + part * (kPart / 16) * (2048 >> 4);
                const uint32_t a = tmem + t * kKeys + part * kPart, d = tmem + Geo::kOCol + t * D;
#pragma unroll
                for (int ks = 0; ks < kPart / 16; ++ks) {
                    if (ks >= steps)
                        break;
                    const uint64_t vd = desc64(vlo + ks * (2048 >> 4), kDescHi);
                    tc_mma_ta(d, a + 32 * (ks / 2) + 8 * (ks % 2), vd, kIdPV, !(first && ks == 0));
                    if constexpr (kSplit)
                        tc_mma_ta(d, a + 32 * (ks / 2) + 16 + 8 * (ks % 2), vd, kIdPV, true);
                }
            };
            auto next_kv = [&] {  // V of the block just scored follows its K, then the next K
                vst = kst + 1 == NS ? 0 : kst + 1;
                vpar = kst + 1 == NS ? kpar ^ 1 : kpar;
                kst = vst + 1 == NS ? 0 : vst + 1;
                kpar = vst + 1 == NS ? vpar ^ 1 : vpar;
            };
            int nb0 = 0, nb1 = 0, end0 = 0, end1 = 0, blocks = 0;        // the item; 0 blocks: none
            int nnb0 = 0, nnb1 = 0, nend0 = 0, nend1 = 0, nblocks = 0;   // the next one
            auto next_item = [&] {
                const int slot = k % kQueue;
                ok = ok && sleep_wait(&item_full[slot], (k / kQueue) & 1, abort);
                nblocks = 0;
                if (!ok)
                    return;
                PtItem it;
                it.fill(s_item[slot], R);
                mbar_arrive(&item_empty[slot]);
                ++k;
                if (it.s < 0)
                    return;
                nnb0 = it.nb[0];
                nnb1 = it.nb[1];
                nend0 = it.end[0];
                nend1 = it.end[1];
                nblocks = it.blocks;
            };
            int j = -1;
            next_item();
            blocks = nblocks;
            nb0 = nnb0;
            nb1 = nnb1;
            end0 = nend0;
            end1 = nend1;
            while (ok && blocks > 0) {
                // Steps whose blocks, and the ones scored in them, are whole
                // for both tiles.
                const uint32_t id_whole = id_s0 | (kKeys >> 3) << 17;
                const int whole = min(nb0, nb1) - 2;
                for (; j >= 0 && j < whole && ok; ++j) {
                    if (j == 0) {
                        ok = sleep_wait(&o_free[0], o_par & 1, abort) && sleep_wait(&o_free[1], o_par >> 1, abort);
                        o_par ^= 3;
                    }
#pragma unroll
                    for (uint32_t t = 0; t < 2; ++t) {
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            ok = ok && sleep_wait(&p_full[t][part], p_par >> t & 1, abort);
                            tc_fence_after();
                            if (ok)
                                mma_pv(t, part, kPart / 16, j == 0 && part == 0);
                        }
                        if (!ok)
                            break;
                        mma_s(t, id_whole);
                        tc_commit(&s_full[t]);
                    }
                    p_par ^= 3;
                    tc_commit(&step_done[step++ % kSteps]);
                    next_kv();
                }
                if (!ok)
                    break;
                // The other steps.
                const bool last = j + 1 == blocks;
                const int nj = last ? 0 : j + 1;
                bool more = !last;
#pragma unroll 1
                for (uint32_t t = 0; t < 2; ++t) {
                    const int nb = t ? nb1 : nb0, end = t ? end1 : end0;
                    if (j >= 0 && j < nb) {
                        if (j == 0) {  // the output of the tile's item before this one is read
                            ok = ok && sleep_wait(&o_free[t], o_par >> t & 1, abort);
                            o_par ^= 1u << t;
                        }
                        // V is there: the gate's arrival stands for it, and tile
                        // 0 comes first in the step.
                        if (j >= nb0)
                            ok = ok && sleep_wait(&full[vst], vpar, abort);
                        const int steps = block_cols(nb, end, j) / 16;
                        for (int part = 0; part < kParts && kPart / 16 * part < steps; ++part) {
                            ok = ok && sleep_wait(&p_full[t][part], p_par >> t & 1, abort);
                            tc_fence_after();
                            if (ok)
                                mma_pv(t, part, steps - kPart / 16 * part, j == 0 && part == 0);
                        }
                        p_par ^= 1u << t;
                        if (j + 1 == nb)
                            tc_commit(&o_full[t]);
                    }
                    if (last && t == 0) {
                        next_item();
                        more = nblocks > 0;
                    }
                    const int qnb = last ? (t ? nnb1 : nnb0) : nb, qend = last ? (t ? nend1 : nend0) : end;
                    if (ok && more && nj < qnb) {
                        if (nj == 0) {
                            ok = sleep_wait(&q_full[t], q_par >> t & 1, abort);
                            q_par ^= 1u << t;
                        }
                        // So is K, but for an item's first block and those that
                        // tile 0 does not see.
                        if (t == 0 ? nj == 0 : nj >= (last ? nnb0 : nb0))
                            ok = ok && sleep_wait(&full[kst], kpar, abort);
                        tc_fence_after();
                        if (ok)
                            mma_s(t, id_s0 | (static_cast<uint32_t>(block_cols(qnb, qend, nj)) >> 3) << 17);
                        tc_commit(&s_full[t]);
                        if (nj + 1 == qnb)
                            tc_commit(&q_empty[t]);
                    }
                }
                if (!ok || !more)
                    break;
                tc_commit(&step_done[step++ % kSteps]);
                next_kv();
                if (last) {
                    blocks = nblocks;
                    nb0 = nnb0;
                    nb1 = nnb1;
                    end0 = nend0;
                    end1 = nend1;
                }
                j = nj;
            }
            if (!ok) {
                set_status(p.status, PKV_ERR_TIMEOUT);
                *abort = 1;
            }
            // Every MMA issued has completed before TMEM is freed.
            tc_commit(&drain);
            mbar_wait_bounded(&drain, 0, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp < 2 * kTileWarps) {
        // ------------------------------------------------------- softmax
        const int t = warp >> 2;                // tile
        const int r = threadIdx.x & (kM - 1);   // row of the tile = TMEM lane
        const int r_tok = r / G;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t scol = tmem + lanes + t * kKeys;
        const uint32_t ocol = tmem + lanes + Geo::kOCol + t * D;
        const float c = p.score_scale;  // positive
        constexpr float kLazy = MmaSoftmax::kLazy;
        uint32_t cnt = 0;   // blocks of this tile
        uint32_t items = 0; // its items
        uint32_t base = 0;  // ring index of the item's first K tile
        bool failed = false;
        for (unsigned k = 0; !failed; ++k) {
            const int slot = k % kQueue;
            if (!warp_wait(&item_full[slot], (k / kQueue) & 1, abort)) {
                failed = true;
                break;
            }
            PtItem it;
            it.fill(s_item[slot], R);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_empty[slot]);
            if (it.s < 0)
                break;
            // Selected, not indexed: the item stays in registers.
            const int nt = t ? it.nt[1] : it.nt[0], nb = t ? it.nb[1] : it.nb[0];
            const int end = t ? it.end[1] : it.end[0], item_end = max(it.end[0], it.end[1]);
            const int first = it.tok0 + t * R;  // token of row 0
            const int pos = first + min(r_tok, nt - 1);
            float m = -INFINITY;                // running maximum, log2 units
            float2 l2[2] = {};                  // its sum, in four parts
            const int whole = (first + 1) / kKeys;  // leading blocks that every row sees whole
            for (int j = 0; j < nb; ++j, ++cnt) {
                if (!warp_wait(&s_full[t], cnt & 1, abort)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const bool tail = j >= whole;
                const int cols = tail ? block_cols(nb, end, j) : kKeys;
                const bool second = cols > kPart;  // the block has keys in its second part
                // Twice through the scores, for the maximum and for the weights:
                // keeping them would not fit the registers without spilling,
                // and loops this short stay in the instruction caches.
                const int lim = pos - j * kKeys + 1;  // keys this row sees
                float mx = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < (second ? kKeys : kPart); c0 += 64) {
                    float x[32], y[32];
                    tmem_ld64(scol + c0, x, y);
                    if (tail) {
                        mask32(x, lim - c0);
                        mask32(y, lim - c0 - 32);
                    }
                    mx = fmaxf(mx, fmaxf(max32(x), max32(y)));
                }
                mx *= c;
                const bool need = mx > m + kLazy;  // false when nothing is visible
                if (__any_sync(kFullMask, need)) {
                    float alpha = 1.f;
                    if (need) {
                        alpha = m == -INFINITY ? 0.f : MmaSoftmax::ex2(m - mx);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            l2[i].x *= alpha;
                            l2[i].y *= alpha;
                        }
                        m = mx;
                    }
                    if (j > 0) {
                        // O holds earlier blocks, whose P V is done: these
                        // scores were issued, and so completed, after it.
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            float ov[16];
                            tmem_ld16(ocol + c0, ov);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                ov[e] *= alpha;
                            tmem_st16(ocol + c0, ov);
                        }
                        tmem_wait_st();
                    }
                }
                // V rows past the item's keys may hold anything.
                const int zero0 = item_end - j * kKeys;
                if (tail && zero0 < cols) {
                    const uint32_t vc = base + 2 * j + 1;
                    if (!warp_wait(&full[vc % NS], (vc / NS) & 1, abort)) {
                        failed = true;
                        break;
                    }
                    unsigned char *vt = smem + (2 + vc % NS) * Geo::kTile;
                    for (int e = r; e < (cols - zero0) * (D / 8); e += kM) {
                        const int row = zero0 + e / (D / 8), piece = e % (D / 8);
                        *reinterpret_cast<uint4 *>(vt + (piece >> 3) * kHalf + row * 128 +
                                                   (piece & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                // Weights 2^(c x - m), in bf16 pairs over the consumed scores; a
                // row of nothing but -inf so far has weights 0.
                const float off = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
                for (int part = 0; part < kParts; ++part) {
                    if (kPart * part < cols) {
                        const uint32_t pc = scol + kPart * part;
                        float x[32], y[32];
                        tmem_ld64(pc, x, y);
                        if (tail) {
                            mask32(x, lim - kPart * part);
                            mask32(y, lim - kPart * part - 32);
                        }
                        weights32<kSplit>(x, c, off, l2, pc);
                        weights32<kSplit>(y, c, off, l2, pc + 32);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                    }
                    if (lane == 0)  // both parts' barriers count every block
                        mbar_arrive(&p_full[t][part]);
                }
            }
            base += 2 * it.blocks;
            if (failed)
                break;
            if (nb == 0)
                continue;

            // The sums go to the output warps, once they have read the last ones.
            if (items > 0 && !warp_wait(&o_free[t], (items - 1) & 1, abort)) {
                failed = true;
                break;
            }
            ++items;
            const float2 lsum = add2(l2[0], l2[1]);
            s_sum[t][r] = lsum.x + lsum.y;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&l_full[t]);
        }
        if (failed && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    } else {
        // --------------------------------------------------- output rows
        // Four warps of their own, for both tiles in turn: the rows' threads go
        // on with the next item while its predecessor's output is read, scaled
        // and stored.
        const int r = 32 * (warp & 3) + lane;
        const int r_tok = r / G, r_head = r % G;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t par = 0;  // bit t: parity of the tile's barriers
        unsigned redo0 = ~0u, redo1 = 0;  // first and last item with a row that is not finite
        bool failed = false;
        for (unsigned k = 0; !failed; ++k) {
            const int slot = k % kQueue;
            if (!warp_sleep_wait(&item_full[slot], (k / kQueue) & 1, abort)) {
                failed = true;
                break;
            }
            PtItem it;
            it.fill(s_item[slot], R);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_empty[slot]);
            if (it.s < 0)
                break;
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? it.nt[1] : it.nt[0], nb = t ? it.nb[1] : it.nb[0];
                if (nb == 0)
                    continue;
                const int first = it.tok0 + t * R;
                const uint32_t ocol = tmem + lanes + Geo::kOCol + t * D;
                if (!warp_sleep_wait(&l_full[t], par >> t & 1, abort) ||
                    !warp_sleep_wait(&o_full[t], par >> t & 1, abort)) {
                    failed = true;
                    break;
                }
                par ^= 1u << t;
                tc_fence_after();
                const float inv = 1.f / s_sum[t][r];
                const bool live = r < nt * G;
                const size_t orow = (static_cast<size_t>(it.row0 + first + min(r_tok, nt - 1)) * p.num_q_heads +
                                     it.hkv * G + r_head) * D;
                float bad = 0.f;  // NaN once an output is not finite
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float ov[32];
                    tmem_ld32(ocol + c0, ov);
                    if (c0 + 32 == D) {  // read whole: the next item's P V may start
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&o_free[t]);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        ov[e] *= inv;
                        bad = fmaf(ov[e], 0.f, bad);
                    }
                    if (live)
                        store_out32<kSplit>(p, orow + c0, ov, wide);
                }
                if (__any_sync(kFullMask, live && bad != 0.f)) {
                    redo0 = min(redo0, k);
                    redo1 = k;
                }
            }
        }
        if (lane == 0 && redo0 <= redo1) {
            atomicMin(&s_redo[0], redo0);
            atomicMax(&s_redo[1], redo1);
        }
        if (failed && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
    // Every copy has landed and every MMA is done: shared memory is free.
    if (s_redo[0] <= s_redo[1] && !s_abort)
        redo_items<D, kSplit>(p, smem, s_redo[0], s_redo[1]);
}

// ------------------------------------------------------------------ host

// Rows of [num_tokens][heads][D] bf16, `stride` elements apart: boxes of 64
// elements x `box_heads` heads x `box_tokens` tokens in the 128-byte swizzle mode.
bool encode_rows(EncodeTiledFn enc, CUtensorMap *map, const void *base, int D, int heads, int64_t tokens,
                 int64_t stride, int box_heads, int box_tokens)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads),
                               static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kSplit> pkv_status launch_ptc(PromptParams p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(prompt_tc_kernel<D, kSplit>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    PtGeom<D>::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    EncodeTiledFn enc = encoder();
    if (!enc)
        return PKV_ERR_CUDA;
    const int R = kM / p.group;
    PromptMaps maps;
    if (!encode_rows(enc, &maps.q, p.q, D, p.num_q_heads, p.num_tokens, p.q_stride, p.group, R) ||
        !encode_rows(enc, &maps.k, p.k, D, p.num_kv_heads, p.num_tokens, p.k_stride, 1, kKeys) ||
        !encode_rows(enc, &maps.v, p.v, D, p.num_kv_heads, p.num_tokens, p.v_stride, 1, kKeys))
        return PKV_ERR_CUDA;
    const long items = prompt_max_items(p, 2 * R);
    if (items <= 0)
        return PKV_OK;
    if (items > 0x40000000L)
        return PKV_ERR_UNSUPPORTED;
    p.max_items = static_cast<unsigned>(items);
    const long sms = device_sm_count();
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    prompt_tc_kernel<D, kSplit><<<grid, kThreads, PtGeom<D>::kSmem, stream>>>(p, maps);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_prompt_tc(const PromptParams &p, cudaStream_t stream)
{
    const bool split = p.out_dtype == PKV_F32;
    if (p.head_dim == 128)
        return split ? launch_ptc<128, true>(p, stream) : launch_ptc<128, false>(p, stream);
    return split ? launch_ptc<64, true>(p, stream) : launch_ptc<64, false>(p, stream);
}

}  // namespace pkv
