// Cache writes that rotate on the way: new tokens' queries and keys are turned
// by their positions and the keys and values go to their slots.
//
// The "Inference optimization" lesson (section "Caches de KV") appends only the
// new token's K and V; a model with rotary positions turns each pair (a, b) of a
// query's and a key's dims by the angle of the token's position first:
//   (a, b) -> (a cos - b sin, b cos + a sin).
// Both products and their sum are rounded (no fused multiply-add): the result
// does not depend on the order in which a compiler would fuse them, and an
// 8-bit code is the one that element-wise f32 arithmetic gives.
//
// A unit is 16 dims of a head whose pairs lie among them: dims 8u .. 8u + 7 and
// rot / 2 + 8u .. (halves), or 16u .. 16u + 15 (neighbours); both take cosines and
// sines 8u .. 8u + 7.  Dims past `rot` are copied.
//
// Queries: a warp has one token; its lanes hold the units of 32 / (D / 16) heads
// at a time and keep their cosines and sines over all of the warp's heads, which
// would otherwise be read again for every head (twice the bytes of the rows).
//
// Keys and values: the caches hold the 16 tokens of a page side by side for each
// (head, dim).  A CTA takes one KV head of some tokens through shared memory (as
// codes of the cache's type) and writes every page that 16 consecutive tokens
// fill as a whole, 64 bytes a thread; tokens of part-filled pages are written
// element by element.  A page belongs to the CTA that has its first token, which
// loads up to 15 tokens past its own.
//
// What bounds it: bytes in flight.  A row's numbers are kept as loaded until they are
// used; with the registers that saves four CTAs fit an SM and a warp has two sets of
// heads on their way.  A chat batch (128 prompts of 256 to 512 tokens, 64/8 heads, bf16):
// 366 us, 5.4 TB/s (80% of a plain copy); as f32 numbers and three CTAs 417 us; one set 381,
// four (which spill) 416 us.  With an fp8 cache of heads of 64 (37 prompts of up to 1000
// tokens, 24/2 heads) 41 us, 4.0 TB/s: 24 heads are three sets of eight, so that a warp's
// second turn of two sets is half empty.  The latent rows of 16 prompts of 512 to 4096 tokens
// with 32 query heads: 97 us, 4.5 TB/s (their 128-byte pieces lie 384 and 1152 bytes apart);
// two sets or four CTAs were no faster.  The same rows in f32: 201 us, 4.3 TB/s.  There the
// bound of five CTAs, chosen on bf16 (12 bytes spilled), spills 100 bytes.
#include "pkv_convert.cuh"
#include "pkv_latent.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;                // tokens of a CTA at most
constexpr int kHalo = kBlockSize - 1;    // tokens past them that fill its last page

struct Vec8 {
    float x[8];
};

// 8 numbers as they lie in memory: rows are read once and kept so until they are used,
// in half the registers for bf16.
template <typename In> struct Raw8 {
    uint4 w[sizeof(In) / 2];
};
__device__ __forceinline__ uint4 load_once(const void *p)
{
    uint4 v;
    // Not volatile: what is stored where it was read (queries in place) depends on it.
    asm("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <typename In> __device__ __forceinline__ Raw8<In> load_raw(const In *p)
{
    Raw8<In> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(In)) / 2; ++i)
        r.w[i] = load_once(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
__device__ __forceinline__ Vec8 widen(const Raw8<float> &r)
{
    const uint4 a = r.w[0], b = r.w[1];
    return {{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
             __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)}};
}
__device__ __forceinline__ Vec8 widen(const Raw8<__nv_bfloat16> &r)
{
    const uint4 a = r.w[0];
    return {{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(a.z), bf16_hi(a.z), bf16_lo(a.w),
             bf16_hi(a.w)}};
}
// 8 of the table's numbers, which neighbouring warps read too.
__device__ __forceinline__ Vec8 load8(const float *p)
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(float *p, const Vec8 &v)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Vec8 &v)
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v.x[0], v.x[1]), pack_bf16(v.x[2], v.x[3]),
                                               pack_bf16(v.x[4], v.x[5]), pack_bf16(v.x[6], v.x[7]));
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}

// One unit's place in a head and its angles.
struct Unit {
    int lo, hi;    // first dims of its two runs of 8
    bool turned;
    Vec8 c, s;

    __device__ __forceinline__ void init(const RopeTokens &t, int u, int pos)
    {
        place(t, u);
        angles(t, u, pos);
    }
    __device__ __forceinline__ void place(const RopeTokens &t, int u)
    {
        turned = 16 * u < t.rot;
        const bool halves = turned && !t.interleaved;
        lo = halves ? 8 * u : 16 * u;
        hi = halves ? t.rot / 2 + 8 * u : 16 * u + 8;
    }
    __device__ __forceinline__ void angles(const RopeTokens &t, int u, int pos)
    {
        if (turned) {
            const float *row = t.table + static_cast<size_t>(pos) * t.rot + 8 * u;
            c = load8(row);
            s = load8(row + t.rot / 2);
        }
    }
    __device__ __forceinline__ void apply(Vec8 &a, Vec8 &b, int interleaved) const
    {
        if (!turned)
            return;
        if (interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                turn(a.x[2 * e], a.x[2 * e + 1], c.x[e], s.x[e]);
                turn(b.x[2 * e], b.x[2 * e + 1], c.x[4 + e], s.x[4 + e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                turn(a.x[e], b.x[e], c.x[e], s.x[e]);
        }
    }
};

// Slot and position of token i; false for padding and, reported when `report`
// is set, for a slot or position outside its range.
__device__ __forceinline__ bool token_ok(const RopeTokens &t, int i, int64_t &slot, int &pos, bool report)
{
    slot = __ldg(t.slots + i);
    pos = __ldg(t.positions + i);
    if (slot < 0)
        return false;
    const bool ok = slot < static_cast<int64_t>(t.num_blocks) * kBlockSize &&
                    static_cast<unsigned>(pos) < static_cast<unsigned>(t.max_positions);
    if (!ok && report)
        set_status(t.status, PKV_ERR_OUT_OF_RANGE);
    return ok;
}

// Warp `w` of the queries' warps: token w / groups, every groups-th set of heads.
// kDeep: sets of heads whose loads are on their way together.
template <typename In, int kDim, int kDeep>
__device__ __forceinline__ void rotate_queries(const RopeTokens &t, const RopeQuery &q, int64_t w, int groups)
{
    constexpr int kUnits = kDim / 16, kAtOnce = 32 / kUnits;  // heads in a warp
    const int lane = threadIdx.x & 31;
    const int i = static_cast<int>(w / groups), group = static_cast<int>(w % groups);
    if (i >= t.num_tokens)
        return;
    int64_t slot;
    int pos;
    if (!token_ok(t, i, slot, pos, false))
        return;
    Unit unit;
    unit.init(t, lane % kUnits, pos);
    const In *src = static_cast<const In *>(q.q) + i * q.stride;
    In *dst = static_cast<In *>(q.out) + i * q.out_stride;
    for (int h0 = group * kAtOnce + lane / kUnits; h0 < q.num_heads; h0 += kDeep * groups * kAtOnce) {
        Raw8<In> ra[kDeep], rb[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int h = h0 + j * groups * kAtOnce;
            if (h < q.num_heads) {
                ra[j] = load_raw(src + h * q.head + unit.lo);
                rb[j] = load_raw(src + h * q.head + unit.hi);
            }
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int h = h0 + j * groups * kAtOnce;
            if (h < q.num_heads) {
                Vec8 a = widen(ra[j]), b = widen(rb[j]);
                unit.apply(a, b, t.interleaved);
                store8(dst + h * q.out_head + unit.lo, a);
                store8(dst + h * q.out_head + unit.hi, b);
            }
        }
    }
}

// The code of x in a cache of `dtype` (INT4: its low nibble).
template <typename Code> __device__ __forceinline__ Code code_of(float x, int dtype, float scale)
{
    if constexpr (sizeof(Code) == 4) {
        return __float_as_uint(x);
    } else if constexpr (sizeof(Code) == 2) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    } else {
        if (dtype == PKV_INT4) {
            const float r = rintf(x / scale);
            return static_cast<Code>(static_cast<int>(r != r ? 0.f : fminf(fmaxf(r, -8.f), 7.f)) & 0xf);
        }
        return static_cast<Code>(
            __nv_cvt_float_to_fp8(x / scale, __NV_SATFINITE, dtype == PKV_FP8_E4M3 ? __NV_E4M3 : __NV_E5M2));
    }
}

template <typename Code>
__device__ __forceinline__ void put_codes(Code *dst, const Vec8 &v, int dtype, float scale)
{
    constexpr int kPer = 4 / sizeof(Code);
    uint32_t w[8 / kPer];
#pragma unroll
    for (int e = 0; e < 8 / kPer; ++e) {
        w[e] = 0;
#pragma unroll
        for (int f = 0; f < kPer; ++f)
            w[e] |= static_cast<uint32_t>(code_of<Code>(v.x[kPer * e + f], dtype, scale)) << (8 * sizeof(Code) * f);
    }
    if constexpr (sizeof(Code) == 1) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int e = 0; e < 8 / kPer / 4; ++e)
            reinterpret_cast<uint4 *>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    }
}

// Row stride of the shared-memory tile: 4 banks past a multiple of 32, so that
// rows of 16-byte pieces and columns both spread.
template <typename Code, int D> struct TileGeom {
    static constexpr int kRow = D * static_cast<int>(sizeof(Code)) + 16;
};

// A whole page of one (KV head): the words of a tile column, 16 tokens of one
// word each (1, 2 or 4 dims), become 64 bytes of the page's rows (INT4: 32).
template <typename Code>
__device__ __forceinline__ void put_page(unsigned char *page, int word, const uint32_t (&w)[16], int dtype)
{
    uint32_t o[16];
    if constexpr (sizeof(Code) == 4) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = w[e];
    } else if constexpr (sizeof(Code) == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o[e] = prmt(w[2 * e], w[2 * e + 1], 0x5410);
            o[8 + e] = prmt(w[2 * e], w[2 * e + 1], 0x7632);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 4 tokens x 4 dims
            const uint32_t a = prmt(w[4 * e], w[4 * e + 1], 0x5140), b = prmt(w[4 * e], w[4 * e + 1], 0x7362);
            const uint32_t c = prmt(w[4 * e + 2], w[4 * e + 3], 0x5140),
                           d = prmt(w[4 * e + 2], w[4 * e + 3], 0x7362);
            o[e] = prmt(a, c, 0x5410);
            o[4 + e] = prmt(a, c, 0x7632);
            o[8 + e] = prmt(b, d, 0x5410);
            o[12 + e] = prmt(b, d, 0x7632);
        }
        if (dtype == PKV_INT4) {
            // Token 2j in the low nibble of byte j of its dim's 8 bytes.
            uint32_t n[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = o[2 * e] | o[2 * e] >> 4, y = o[2 * e + 1] | o[2 * e + 1] >> 4;
                n[e] = prmt(x, y, 0x6420);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(page + word * 32);
            dst[0] = make_uint4(n[0], n[1], n[2], n[3]);
            dst[1] = make_uint4(n[4], n[5], n[6], n[7]);
            return;
        }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(page + word * 64);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
}

__device__ __forceinline__ void put_nibble(unsigned char *cache, size_t i, uint32_t code)
{
    const size_t byte = i >> 1;
    unsigned int *word = reinterpret_cast<unsigned int *>(cache + (byte & ~static_cast<size_t>(3)));
    const int shift = static_cast<int>((byte & 3) * 8 + (i & 1) * 4);
    atomicAnd(word, ~(0xfu << shift));
    atomicOr(word, code << shift);
}

// Tokens [t0, t0 + tile) of KV head h.
template <typename In, typename Code, int D>
__device__ __forceinline__ void write_tile(const RopeAppendParams &p, unsigned char *smem, int t0, int tile, int h)
{
    constexpr int kRow = TileGeom<Code, D>::kRow;
    constexpr int kUnits = D / 16, kAtOnce = 32 / kUnits;  // tokens in a warp's load
    constexpr int kWords = D * static_cast<int>(sizeof(Code)) / 4;
    __shared__ int64_t s_slot[kHalo + kTile + kHalo];  // of tokens t0 - 15 ..; -1: not written
    __shared__ int s_pos[kHalo + kTile + kHalo];
    __shared__ int s_page[kHalo + kTile];              // token 0 of a whole page: its block, else -1
    __shared__ unsigned char s_part[kTile];            // 1: a token of a part-filled page
    __shared__ int s_end;                              // tokens to load
    const RopeTokens &t = p.t;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = min(tile, t.num_tokens - t0);
    for (int e = threadIdx.x; e < kHalo + n + kHalo; e += kThreads) {
        const int i = t0 - kHalo + e;
        int64_t slot = -1;
        int pos = 0;
        if (i >= 0 && i < t.num_tokens && !token_ok(t, i, slot, pos, h == 0 && e >= kHalo && e < kHalo + n))
            slot = -1;
        s_slot[e] = slot;
        s_pos[e] = pos;
    }
    if (threadIdx.x == 0)
        s_end = n;
    __syncthreads();
    // Whole pages whose first token is among t0 - 15 .. t0 + n - 1.
    for (int e = threadIdx.x; e < kHalo + n; e += kThreads) {
        const int64_t slot = s_slot[e];
        bool whole = slot >= 0 && slot % kBlockSize == 0;
        for (int j = 1; whole && j < kBlockSize; ++j)
            whole = s_slot[e + j] == slot + j;
        s_page[e] = whole ? static_cast<int>(slot / kBlockSize) : -1;
        if (whole && e >= kHalo)
            atomicMax(&s_end, e - kHalo + kBlockSize);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += kThreads) {
        const int64_t slot = s_slot[kHalo + e];
        const int first = kHalo + e - static_cast<int>(slot & (kBlockSize - 1));
        s_part[e] = slot >= 0 && s_page[first] < 0;
    }
    const int end = s_end;
    unsigned char *sk = smem, *sv = smem + (tile + kHalo) * kRow;
    const In *k = static_cast<const In *>(p.k) + static_cast<size_t>(h) * D;
    const In *v = static_cast<const In *>(p.v) + static_cast<size_t>(h) * D;
    for (int e = warp * kAtOnce + lane / kUnits; e < end; e += kWarps * kAtOnce) {
        if (s_slot[kHalo + e] < 0)
            continue;
        const int64_t i = t0 + e;
        Unit unit;
        unit.place(t, lane % kUnits);
        const Raw8<In> ka = load_raw(k + i * p.k_stride + unit.lo), kb = load_raw(k + i * p.k_stride + unit.hi);
        const Raw8<In> va = load_raw(v + i * p.v_stride + unit.lo), vb = load_raw(v + i * p.v_stride + unit.hi);
        unit.angles(t, lane % kUnits, s_pos[kHalo + e]);
        Vec8 a = widen(ka), b = widen(kb);
        unit.apply(a, b, t.interleaved);
        Code *dk = reinterpret_cast<Code *>(sk + e * kRow), *dv = reinterpret_cast<Code *>(sv + e * kRow);
        put_codes(dk + unit.lo, a, p.kv_dtype, p.k_scale);
        put_codes(dk + unit.hi, b, p.kv_dtype, p.k_scale);
        put_codes(dv + unit.lo, widen(va), p.kv_dtype, p.v_scale);
        put_codes(dv + unit.hi, widen(vb), p.kv_dtype, p.v_scale);
    }
    __syncthreads();

    // Whole pages, a warp each.
    const size_t page_bytes = p.kv_dtype == PKV_INT4 ? D * kBlockSize / 2 : D * kBlockSize * sizeof(Code);
    unsigned char *caches[2] = {static_cast<unsigned char *>(p.k_cache), static_cast<unsigned char *>(p.v_cache)};
    for (int e = warp; e < n; e += kWarps) {
        const int block = s_page[kHalo + e];
        if (block < 0)
            continue;
        for (int x = lane; x < 2 * kWords; x += 32) {
            const int which = x >= kWords, word = which ? x - kWords : x;
            const unsigned char *src = (which ? sv : sk) + e * kRow + 4 * word;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[j] = *reinterpret_cast<const uint32_t *>(src + j * kRow);
            put_page<Code>(caches[which] + (static_cast<size_t>(block) * p.num_kv_heads + h) * page_bytes, word, w,
                           p.kv_dtype);
        }
    }
    // The other tokens, neighbouring tokens on neighbouring lanes.
    constexpr int kDims = 4 / static_cast<int>(sizeof(Code));
    for (int x = threadIdx.x; x < 2 * kWords * n; x += kThreads) {
        const int e = x % n, at = x / n;
        if (!s_part[e])
            continue;
        const int which = at >= kWords, word = which ? at - kWords : at;
        const uint32_t w = *reinterpret_cast<const uint32_t *>((which ? sv : sk) + e * kRow + 4 * word);
        const int64_t slot = s_slot[kHalo + e];
        const size_t cell = ((static_cast<size_t>(slot / kBlockSize) * p.num_kv_heads + h) * D + kDims * word) *
                                kBlockSize + static_cast<size_t>(slot % kBlockSize);
#pragma unroll
        for (int f = 0; f < kDims; ++f) {
            const Code code = static_cast<Code>(w >> (8 * sizeof(Code) % 32 * f));
            if (sizeof(Code) == 1 && p.kv_dtype == PKV_INT4)
                put_nibble(caches[which], cell + f * kBlockSize, code);
            else
                reinterpret_cast<Code *>(caches[which])[cell + f * kBlockSize] = code;
        }
    }
}

// CTAs [0, kv_ctas) write the caches, the others turn the queries.
// The CTAs of an SM (four, with f32 three) are as many as the registers allow with next to
// nothing spilled.
template <typename In, typename Code, int D>
__global__ void __launch_bounds__(kThreads, sizeof(In) == 2 ? 4 : 3)
    rope_append_kernel(const RopeAppendParams p, int tile, int kv_ctas, int groups)
{
    extern __shared__ __align__(16) unsigned char smem_rope[];
    const int b = static_cast<int>(blockIdx.x);
    if (b < kv_ctas) {
        write_tile<In, Code, D>(p, smem_rope, b / p.num_kv_heads * tile, tile, b % p.num_kv_heads);
        return;
    }
    rotate_queries<In, D, sizeof(In) == 2 ? 2 : 1>(p.t, p.q, static_cast<int64_t>(b - kv_ctas) * kWarps + (threadIdx.x >> 5), groups);
}

// Sets of heads that a token's queries are shared between: one, unless there
// are too few tokens to fill the GPU.
int query_groups(int tokens, int heads, int at_once)
{
    const int most = (heads + at_once - 1) / at_once;
    const long want = (static_cast<long>(device_sm_count()) * 2 * kWarps + tokens - 1) / tokens;
    return static_cast<int>(want < most ? want : most);
}

template <typename In, typename Code, int D>
pkv_status launch_append(const RopeAppendParams &p, cudaStream_t stream)
{
    // Tokens of a CTA: as many as leave two CTAs to an SM, at most 64, or 32 for f32
    // caches, whose tiles of 64 (83 KB) leave room for two CTAs only (64 prompts of 256 to 512
    // tokens, 32/8 heads, f32: 284 us against 256).
    constexpr int kMost = sizeof(Code) == 4 ? kTile / 2 : kTile;
    const long want = static_cast<long>(p.t.num_tokens) * p.num_kv_heads / (2L * device_sm_count());
    const int tile = want >= kMost ? kMost : want < 1 ? 1 : static_cast<int>(want);
    const long kv = (static_cast<long>(p.t.num_tokens) + tile - 1) / tile * p.num_kv_heads;
    int groups = 1;
    long warps = 0;
    if (p.q.num_heads > 0) {
        groups = query_groups(p.t.num_tokens, p.q.num_heads, 32 / (D / 16));
        warps = static_cast<long>(p.t.num_tokens) * groups;
    }
    const long grid = kv + (warps + kWarps - 1) / kWarps;
    if (grid > 0x7fffffffL)
        return PKV_ERR_UNSUPPORTED;
    const int smem = 2 * (tile + kHalo) * TileGeom<Code, D>::kRow;
    constexpr int most = 2 * (kMost + kHalo) * TileGeom<Code, D>::kRow;
    if (most > 48 * 1024) {
        static ContextCache cache;
        int set = 0;
        const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
            *out = 1;
            return cudaFuncSetAttribute(rope_append_kernel<In, Code, D>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess
                       ? PKV_OK
                       : PKV_ERR_CUDA;
        });
        if (rc != PKV_OK)
            return rc;
    }
    rope_append_kernel<In, Code, D><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(
        p, tile, static_cast<int>(kv), groups);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename In, typename Code> pkv_status launch_append_d(const RopeAppendParams &p, cudaStream_t stream)
{
    return p.head_dim == 64 ? launch_append<In, Code, 64>(p, stream) : launch_append<In, Code, 128>(p, stream);
}
template <typename In> pkv_status launch_append_in(const RopeAppendParams &p, cudaStream_t stream)
{
    if (p.kv_dtype == PKV_F32)
        return launch_append_d<In, uint32_t>(p, stream);
    if (p.kv_dtype == PKV_BF16)
        return launch_append_d<In, unsigned short>(p, stream);
    return launch_append_d<In, unsigned char>(p, stream);
}

// ------------------------------------------------------------ latent rows

// CTAs [0, row_ctas): a warp per token copies its latent vector and turns its
// key; the others turn the queries.
template <typename In, typename Out>
__global__ void __launch_bounds__(kThreads, 5)
    latent_append_kernel(const LatentAppendParams p, int row_ctas, int groups)
{
    const int b = static_cast<int>(blockIdx.x), lane = threadIdx.x & 31;
    if (b >= row_ctas) {
        rotate_queries<In, kRopeDim, 1>(p.t, p.q, static_cast<int64_t>(b - row_ctas) * kWarps + (threadIdx.x >> 5),
                                     groups);
        return;
    }
    const int64_t i = static_cast<int64_t>(b) * kWarps + (threadIdx.x >> 5);
    if (i >= p.t.num_tokens)
        return;
    int64_t slot;
    int pos;
    if (!token_ok(p.t, static_cast<int>(i), slot, pos, lane == 0))
        return;
    Out *dst = static_cast<Out *>(p.cache) + static_cast<size_t>(slot) * (p.latent_dim + kRopeDim);
    const In *src = static_cast<const In *>(p.latent) + i * p.latent_stride;
    for (int d = 8 * lane; d < p.latent_dim; d += 256) {
        if constexpr (sizeof(In) == 2 && sizeof(Out) == 2)  // the bits
            *reinterpret_cast<uint4 *>(dst + d) = load_once(src + d);
        else
            store8(dst + d, widen(load_raw(src + d)));
    }
    if (lane < kRopeDim / 16) {
        Unit unit;
        unit.init(p.t, lane, pos);
        const In *key = static_cast<const In *>(p.k_rope) + i * p.k_rope_stride;
        Vec8 a = widen(load_raw(key + unit.lo)), c = widen(load_raw(key + unit.hi));
        unit.apply(a, c, p.t.interleaved);
        store8(dst + p.latent_dim + unit.lo, a);
        store8(dst + p.latent_dim + unit.hi, c);
    }
}

template <typename In, typename Out> pkv_status launch_rows(const LatentAppendParams &p, cudaStream_t stream)
{
    const long rows = (static_cast<long>(p.t.num_tokens) + kWarps - 1) / kWarps;
    int groups = 1;
    long warps = 0;
    if (p.q.num_heads > 0) {
        groups = query_groups(p.t.num_tokens, p.q.num_heads, 32 / (kRopeDim / 16));
        warps = static_cast<long>(p.t.num_tokens) * groups;
    }
    const long grid = rows + (warps + kWarps - 1) / kWarps;
    if (grid > 0x7fffffffL)
        return PKV_ERR_UNSUPPORTED;
    latent_append_kernel<In, Out><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(
        p, static_cast<int>(rows), groups);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_rope_append(const RopeAppendParams &p, cudaStream_t stream)
{
    return p.t.in_dtype == PKV_F32 ? launch_append_in<float>(p, stream)
                                   : launch_append_in<__nv_bfloat16>(p, stream);
}

pkv_status launch_latent_append(const LatentAppendParams &p, cudaStream_t stream)
{
    if (p.t.in_dtype == PKV_F32)
        return p.cache_dtype == PKV_F32 ? launch_rows<float, float>(p, stream)
                                        : launch_rows<float, __nv_bfloat16>(p, stream);
    return p.cache_dtype == PKV_F32 ? launch_rows<__nv_bfloat16, float>(p, stream)
                                    : launch_rows<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace pkv
