// Latent attention for one query per sequence on the tcgen05 tensor cores (bf16).
//
// Absorbed form: out[s, h] = sum_t softmax_t(scale q[s, h] . row_t) row_t[:R] (the
// scaled_dot_product_attention of the "Inference optimization" lesson, Step 2, with
// one row of R + 64 numbers per token, key and value at once).  One pass over the
// rows with the running maximum and sum of the softmax.
//
// Layout on the GPU:
//  * Tokens lie on the rows of the products and heads on their columns: S^T = rows
//    Q^T (M = 64 tokens, N = heads) and O^T = rows^T P^T (M = 128 dims at a time).
//    So a call pays for the heads it has, in steps of 16, 32 and 64, and the same
//    shared-memory copy of a row (64 tokens x 64 dims, 128-byte swizzle) is the
//    K-major operand of the one and the M-major operand of the other.
//  * A CTA (one per SM) has up to 64 heads and walks a range of tiles of 64 tokens
//    (pkv_latent.cuh).  Warps 0-7 compute the softmax, four for each half of the heads;
//    warps 8 to 15 issue the TMA loads, one for each 8 tokens of a tile.
//  * TMEM: two buffers of S^T, and O^T.  P^T goes through shared memory.
//  * A tile comes in two parts, each with a ring of its own: the scores start with the
//    first that lands, and a part's slot is filled again when its half of O^T is done.
//    A box is 8 tokens of one page x half the dims: groups of 8 tokens then lie a fixed
//    distance apart, whatever the pages, which is all that the operands ask for.
//  * A warp issues the scores' MMAs, another those of P V, which free the ring.
//  * The reference of a head's weights is raised only when a score exceeds it by 2^8;
//    O^T is then rescaled in TMEM.  All weights of a head and tile share it, so the
//    four warps of a half agree through a barrier.
//  * Weights are rounded to bf16 (off by 2^-8 at most), their sum is that of the f32 ones.
//    A second part of each, for 16 bits, would double the products of P V and needs 8 KB
//    more with 64 heads, where two tiles leave 1 KB.
//  * Rows past the sequence's end are zeroed in shared memory before P V, which
//    multiplies them with 0: they may hold anything.
//  * Every wait is bounded; a timeout records PKV_ERR_TIMEOUT, stops every role, lets
//    copies and MMAs in flight finish and frees TMEM.  The warps of a half leave
//    together: none waits at a barrier for one that has gone.
//
// What the layout costs the tensor cores (counted alone, cycles per MMA of 16 dims or
// tokens): the scores 32, 24 and 23 for 64, 32 and 16 heads (M = 64), P V 48, 40 and 39
// (M = 128): the larger of half or full rate and of the operands' shared-memory bytes at
// 128 a cycle.  A tile of 64 tokens takes 1940 cycles with 64 heads, HBM 3170 to bring it.
// Heads on the rows would take 2176 with 64 heads and as much with 16.
//
// What bounds it.  Few heads: HBM (256 x 4096 tokens, 16 heads: 196 us, 6.2 TB/s, 91% of a
// plain copy).  64 heads (64 x 8192 tokens: 118 us, 5.2 TB/s): queries and weights leave
// room for two tiles, and a tile's slot is taken for some 3300 cycles between its landing
// and the end of P V (scores 900, softmax 1000, P V 700, hand-overs) and 2300 more until
// the next one has landed; that alone would leave 6.0 TB/s (16 heads in 64 columns), the
// rest are the partial sums of cut sequences, 128 KB each.  128 heads are two CTAs that read the same rows
// (128 x 4096 tokens: 170 us, 860 TFLOP/s): the same chain, with 1940 cycles of products in
// 2800.  Short calls: about 6000 cycles until the first tile lands (the lengths and the
// table are two dependent trips to memory) and the joining kernel (64 sequences of a
// mean of 2900 tokens, 64 heads: 53 + 8.5 us).  Many sequences: every CTA reads all lengths,
// a run of neighbours to a lane (2^17 empty ones 0.8 ms, of 16 tokens and one head 2.3 ms:
// the rest is a chain for each).
//
// Measured and not kept: one warp for all MMAs that takes what is ready (64 x 64 heads
// 76 us against 66 then: it looks as long as it issues); one copying warp, two, four (73,
// 66, 63; eight 62.5 with the later steps); 16-token boxes of 64 dims instead of 8-token
// boxes of half the row (66 against 63); two tiles of 32 heads instead of one of 64 (64 x
// 8192 tokens 130 against 118); partial sums with the heads next to each other (32 bytes to
// a lane: 78 against 65); the barrier of the softmax warps also telling failures apart
// without a second look (the same).
#include "pkv_latent.cuh"
#include "pkv_tc.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 608;
constexpr int kSoftWarps = 8;
constexpr int kProducerWarp = 8;  // one for each group of 8 tokens
constexpr int kGroups = kLatentTokens / 8;
constexpr int kTok = kLatentTokens;
constexpr int kPages = kTok / kBlockSize;
constexpr int kScoreWarp = kProducerWarp + kGroups;
constexpr int kValueWarp = kScoreWarp + 1;
constexpr int kAheadWarp = kValueWarp + 1;
constexpr int kAhead = 2;  // tiles asked of HBM ahead of the rings
constexpr int kAtom = 1024;  // bytes of 8 tokens x 64 dims

// A tile lies in shared memory in two parts, chunks (of 64 dims) 0 .. CA - 1 and the rest
// with the rotated chunk: [8 groups of 8 tokens][chunks][8 tokens][64 dims].
template <int R, int NH> struct LtGeom {
    static constexpr int CA = R / 128, CB = R / 128 + 1;
    static constexpr int kTilesA = CA / 2, kTilesB = CA - kTilesA;  // 128-dim tiles of O^T in each part
    static constexpr int kA = 8 * CA * kAtom, kB = 8 * CB * kAtom;
    static constexpr int kQ = (R / 64 + 1) * NH * 128;  // bytes of the queries
    static constexpr int kP = NH * 128;
    // Slots of each part: as many as fit.
    static constexpr int kRoom = 229 * 1024 - 4096 - kQ - kP;
    static constexpr int kBoth = kRoom / (kA + kB);
    static constexpr int NA = kBoth;
    static constexpr int NB = kBoth + (kRoom - kBoth * (kA + kB) >= kB ? 1 : 0);
    static constexpr int kSmem = 1024 + kQ + kP + NA * kA + NB * kB;
    static constexpr int kOCol = 2 * NH;
    static constexpr int kCols = kOCol + CA * NH;  // TMEM columns
    static constexpr int kAlloc = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kBoth >= 2 && kCols <= 512, "two tiles fit");
};

struct LatentMaps {
    CUtensorMap q, a, b;
};

// One box of 64 numbers x rows x chunks.
__device__ __forceinline__ void load_elected(uint32_t dst, const CUtensorMap *map, int row, int chunk, int outer, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(outer), "r"(smem_u32(bar))
        : "memory");
}

// 16 lanes x 8 J columns of f32 as fragments: registers 4j, 4j + 1 of a thread are row
// lane / 4, columns 8j + 2 (lane % 4) and the next; 4j + 2, 4j + 3 the same of row + 8.
// Load and wait are one statement: between two, the compiler may copy registers that
// the load has yet to fill.
template <int J> __device__ __forceinline__ void tmem_ld_rows(uint32_t addr, float (&x)[4 * J])
{
    if constexpr (J == 1) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
            : "r"(addr)
            : "memory");
    } else if constexpr (J == 2) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
            : "r"(addr)
            : "memory");
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
              "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
            : "r"(addr)
            : "memory");
    }
}

// 8 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float (&v)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// 8 x 8 matrices of 16-bit fragments, transposed: lane l gives the address of row
// l % 8 of matrix l / 8.
__device__ __forceinline__ void stsm_t4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void stsm_t2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b)
                 : "memory");
}

// Hands the warp's part of O^T, `mine` columns of each of kTiles tiles NH columns apart,
// to put(tile, column, value of this lane's dim).
template <int kTiles, int NH, int kCols, typename Put>
__device__ __forceinline__ void store_heads(uint32_t col, int mine, Put put)
{
#pragma unroll 1
    for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 8) {
            if (c0 >= mine)
                break;
            float o[8];
            tmem_ld8(col + t * NH + c0, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e < mine)
                    put(t, c0 + e, o[e]);
        }
    }
}

// Barrier of the four softmax warps of half g; the second form also ORs a predicate.
__device__ __forceinline__ void half_sync(int g)
{
    asm volatile("barrier.sync %0, 128;" ::"r"(g + 1) : "memory");
}
__device__ __forceinline__ bool half_any(int g, bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\t"
        "barrier.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(g + 1), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}

// A ring's position: slot and parity of its phase.
template <int N> struct Ring {
    uint32_t at = 0, par = 0;
    __device__ __forceinline__ void step()
    {
        if (++at == N) {
            at = 0;
            par ^= 1;
        }
    }
};

template <int R, int NH>
__global__ void __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const __grid_constant__ LatentDecodeParams p, const __grid_constant__ LatentMaps maps)
{
    using Geo = LtGeom<R, NH>;
    constexpr int NA = Geo::NA, NB = Geo::NB, CA = Geo::CA, CB = Geo::CB;
    constexpr int kTiles = CA;          // 128-dim tiles of O^T
    constexpr int J = NH / 16;          // octets of columns per half
    constexpr int kHalfCols = NH / 2;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t a_full[NA], a_empty[NA], b_full[NB], b_empty[NB];
    __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], s_free[2], p_full, pv_done, o_free,
        drain[2];
    __shared__ __align__(16) float s_red[2][4][32];  // per half and warp: maxima or sums of its heads
    __shared__ __align__(16) float s_col[NH];        // per head: a factor of its column of O^T
    __shared__ LatentWalk s_walk;
    __shared__ uint32_t s_tmem, s_issued;  // tiles whose copies have been issued
    __shared__ int s_abort, s_never, s_failed[2][2];
    volatile int *abort = &s_abort;
    const volatile int &no_abort = s_never;  // for what has to end before the CTA may

    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t smem0 = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (smem0 - raw);
    constexpr int kPOff = Geo::kQ, kAOff = kPOff + Geo::kP, kBOff = kAOff + NA * Geo::kA;
    const int team = blockIdx.x / p.head_tiles, ht = blockIdx.x % p.head_tiles;
    const int h0 = ht * NH;

    if (warp == 0) {
        // A lane for each barrier.
        if (lane < NA) {
            mbar_init(&a_full[lane], kGroups);
            mbar_init(&a_empty[lane], 1);
        }
        if (lane < NB) {
            mbar_init(&b_full[lane], kGroups);
            mbar_init(&b_empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&s_full[lane], 1);
            mbar_init(&s_free[lane], kSoftWarps);
            mbar_init(&drain[lane], 1);
            s_failed[lane][0] = s_failed[lane][1] = 0;
        }
        if (lane == 2) {
            mbar_init(&q_full, 1);
            mbar_init(&q_empty, 1);
            mbar_init(&p_full, kSoftWarps);
        }
        if (lane == 3) {
            mbar_init(&pv_done, 1);
            mbar_init(&o_free, kSoftWarps);
            s_abort = s_never = 0;
            s_issued = 0;
        }
        fence_mbar_init();
    }
    if (warp == kScoreWarp && lane < 3) {
        const CUtensorMap *map = lane == 0 ? &maps.q : lane == 1 ? &maps.a : &maps.b;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == kProducerWarp) {
        LatentWalk walk;
        walk.init(p, team, lane, blockIdx.x == 0);
        if (lane == 0)
            s_walk = walk;
    }
    if (warp == kValueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(Geo::kAlloc)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The kernel that joins cut sequences may be set up; it waits for this one's end.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = s_tmem;
    LatentWalk walk = s_walk;

    if (warp >= kProducerWarp && warp < kProducerWarp + kGroups) {
        // ------------------------------------------------------- copies
        // A warp for each group of 8 tokens: a warp issues a box only every 150 to 400
        // cycles, by its size (one warp 22 bytes a cycle, four 80).
        const int mine = warp - kProducerWarp;
        Ring<NA> a;
        Ring<NB> b;
        uint32_t tiles = 0, b_tiles = 0, pieces = 0;
        bool ok = true;
        for (;;) {
            const LatentPiece piece = walk.next(p);
            if (piece.s < 0 || !ok)
                break;
            if (piece.len == 0)
                continue;
            if (mine == 0) {
                if (pieces > 0)
                    ok = warp_wait(&q_empty, (pieces - 1) & 1, abort);
                if (!ok)
                    break;
                expect_elected(&q_full, Geo::kQ);
                load_elected(smem0, &maps.q, h0, 0, piece.s, &q_full);
            }
            ++pieces;
            const int32_t *table = p.block_tables + static_cast<size_t>(piece.s) * p.max_blocks;
            const int pages = (piece.len + kBlockSize - 1) / kBlockSize;
            // This warp's block ids of 32 tiles, a lane each, the next 32 on their way.
            auto ids_at = [&](int j) {
                const int page = (j + lane) * kPages + mine / 2;
                return page < pages ? __ldg(table + page) : 0;
            };
            int ids = 0, next_ids = ids_at(piece.first);
            for (int j = piece.first; j < piece.last; ++j) {
                const int at = (j - piece.first) & 31;
                if (at == 0) {
                    ids = next_ids;
                    if (static_cast<unsigned>(ids) >= static_cast<unsigned>(p.num_blocks)) {
                        set_status(p.status, PKV_ERR_OUT_OF_RANGE);
                        ids = p.num_blocks;  // past the map: zeros
                    }
                    next_ids = j + 32 < piece.last ? ids_at(j + 32) : 0;
                }
                const bool there = j * kTok + 8 * mine < piece.len;
                const int id = __shfl_sync(kFullMask, ids, at);
                ok = warp_wait(&a_empty[a.at], a.par ^ 1, abort);
                if (!ok)
                    break;
                {
                    uint64_t *bar = &a_full[a.at];
                    expect_elected(bar, there ? Geo::kA / kGroups : 0);
                    if (there && !(p.drop_first_copy && blockIdx.x == 0 && tiles == 0 && mine == 0))
                        load_elected(smem0 + kAOff + a.at * Geo::kA + mine * (Geo::kA / kGroups), &maps.a,
                                     8 * (mine & 1), 0, id, bar);
                }
                a.step();
                ++tiles;
                if (mine == 0 && lane == 0)
                    *static_cast<volatile uint32_t *>(&s_issued) = tiles;
                ok = warp_wait(&b_empty[b.at], b.par ^ 1, abort);
                if (!ok)
                    break;
                {
                    uint64_t *bar = &b_full[b.at];
                    expect_elected(bar, there ? Geo::kB / kGroups : 0);
                    if (there)
                        load_elected(smem0 + kBOff + b.at * Geo::kB + mine * (Geo::kB / kGroups), &maps.b,
                                     8 * (mine & 1), CA, id, bar);
                }
                b.step();
                ++b_tiles;
            }
        }
        if (!ok && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        // Every copy still in flight lands before the CTA exits.
        if (lane == 0) {
            for (uint32_t c = tiles > NA ? tiles - NA : 0; c < tiles; ++c)
                tc_wait(&a_full[c % NA], (c / NA) & 1, &no_abort);
            for (uint32_t c = b_tiles > NB ? b_tiles - NB : 0; c < b_tiles; ++c)
                tc_wait(&b_full[c % NB], (c / NB) & 1, &no_abort);
            if (pieces > 0 && mine == 0)
                tc_wait(&q_full, (pieces - 1) & 1, &no_abort);
        }
        __syncwarp();
    } else if (warp == kAheadWarp && p.head_tiles > 1) {
        // --------------------------------------------- HBM, ahead of the rings
        // With two head tiles, each row is read by two CTAs, and the rings hold half as many
        // bytes of HBM: pages are fetched into L2 while the rings are still full.  Two tiles
        // at a time, a lane for each page; the head tiles share the pages out.  128 x 4096
        // tokens, 128 heads, when it was added: 174 us, without 198; four tiles ahead 182.
        // With one head tile the rings are enough, and it costs (256 x 4096, 16 heads, then:
        // 194 us without, 207 two ahead, 275 four: more than L2 keeps).  The wait below ends
        // with the copying warp, which issues every tile or gives up at its limit and says so.
        const volatile uint32_t *issued = &s_issued;
        uint32_t tiles = 0;
        for (bool on = true; on;) {
            const LatentPiece piece = walk.next(p);
            if (piece.s < 0)
                break;
            const int32_t *table = p.block_tables + static_cast<size_t>(piece.s) * p.max_blocks;
            const int pages = min((piece.len + kBlockSize - 1) / kBlockSize, piece.last * kPages);
            const int tile_count = piece.len > 0 ? piece.last - piece.first : 0;
            for (int j = 0; j < tile_count; j += 2, tiles += 2) {
                const int page = (piece.first + j) * kPages + lane;
                const int id = lane < 2 * kPages && page < pages && page % p.head_tiles == ht ? __ldg(table + page) : -1;
                while (on && static_cast<int>(tiles - *issued) > kAhead) {
                    on = !*abort;
                    __nanosleep(100);
                }
                on = __all_sync(kFullMask, on);
                if (!on)
                    break;
                constexpr int kLines = kBlockSize * (R + kRopeDim) * 2 / 128;
#pragma unroll 1
                for (int i = 0; i < 2 * kPages; ++i) {
                    const int one = __shfl_sync(kFullMask, id, i);
                    if (static_cast<unsigned>(one) >= static_cast<unsigned>(p.num_blocks))
                        continue;
                    const char *at = static_cast<const char *>(p.cache) + static_cast<size_t>(one) * (kLines * 128);
                    for (int x = lane; x < kLines; x += 32)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + x * 128));
                }
            }
            tiles -= tile_count & 1;
        }
    } else if (warp == kScoreWarp) {
        // ------------------------------------------------- MMA issue: scores
        // A warp for the scores and one for P V, each with its own waits: one warp that
        // took whichever was ready spent as long on looking as on issuing.
        const uint32_t id_s = tc_idesc(kTok, NH, false) | (p.negate ? 1u << 13 : 0u);
        const uint64_t qd = operand(smem0, kAtom);
        const uint64_t ad = operand(smem0 + kAOff, CA * kAtom), bd = operand(smem0 + kBOff, CB * kAtom);
        Ring<NA> a;
        Ring<NB> b;
        uint32_t tiles = 0, pieces = 0;
        bool ok = true;
        for (;;) {
            const LatentPiece piece = walk.next(p);
            if (piece.s < 0 || !ok)
                break;
            if (piece.len == 0)
                continue;
            ok = warp_wait(&q_full, pieces & 1, abort);
            for (int j = piece.first; j < piece.last && ok; ++j) {
                const uint32_t d = tmem + (tiles & 1) * NH;
                // The softmax has read the buffer's last scores.
                if (tiles > 1)
                    ok = warp_wait(&s_free[tiles & 1], ((tiles >> 1) - 1) & 1, abort);
                ok = ok && warp_wait(&a_full[a.at], a.par, abort);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t x = ad + a.at * (Geo::kA >> 4), y = bd + b.at * (Geo::kB >> 4);
#pragma unroll
                for (int c = 0; c < CA; ++c)
                    mma4<2, 2>(d, x + c * (kAtom >> 4), qd + c * (NH * 128 >> 4), id_s, c > 0);
                a.step();
                ok = warp_wait(&b_full[b.at], b.par, abort);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    mma4<2, 2>(d, y + c * (kAtom >> 4), qd + (CA + c) * (NH * 128 >> 4), id_s, true);
                b.step();
                commit_elected(&s_full[tiles & 1]);
                ++tiles;
            }
            if (ok)
                commit_elected(&q_empty);
            ++pieces;
        }
        if (!ok && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        // Every MMA issued has completed before TMEM is freed.
        commit_elected(&drain[0]);
        warp_wait(&drain[0], 0, &no_abort);
    } else if (warp == kValueWarp) {
        // ------------------------------------------------- MMA issue: P V
        constexpr uint32_t kIdPV = tc_idesc(128, NH, false) | 1u << 15;  // A is M-major
        const uint64_t pd = operand(smem0 + kPOff, kAtom);
        const uint64_t ad = operand(smem0 + kAOff, CA * kAtom, kAtom), bd = operand(smem0 + kBOff, CB * kAtom, kAtom);
        Ring<NA> a;
        Ring<NB> b;
        uint32_t tiles = 0, pieces = 0;
        bool ok = true;
        for (;;) {
            const LatentPiece piece = walk.next(p);
            if (piece.s < 0 || !ok)
                break;
            if (piece.len == 0)
                continue;
            for (int j = piece.first; j < piece.last; ++j) {
                ok = warp_wait(&p_full, tiles & 1, abort);
                // The last piece's sums have been read.
                if (j == piece.first && pieces > 0)
                    ok = ok && warp_wait(&o_free, (pieces - 1) & 1, abort);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t x = ad + a.at * (Geo::kA >> 4), y = bd + b.at * (Geo::kB >> 4);
                // 16 tokens to a step: two groups.
#pragma unroll
                for (int m = 0; m < Geo::kTilesA; ++m)
                    mma4<(2 * CA * kAtom >> 4), 2>(tmem + Geo::kOCol + m * NH, x + 2 * m * (kAtom >> 4), pd, kIdPV,
                                                   j > piece.first);
                commit_elected(&a_empty[a.at]);
                a.step();
#pragma unroll
                for (int m = 0; m < Geo::kTilesB; ++m)
                    mma4<(2 * CB * kAtom >> 4), 2>(tmem + Geo::kOCol + (Geo::kTilesA + m) * NH,
                                                   y + 2 * m * (kAtom >> 4), pd, kIdPV, j > piece.first);
                commit_elected(&b_empty[b.at]);
                b.step();
                commit_elected(&pv_done);
                ++tiles;
            }
            ++pieces;
        }
        if (!ok && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        commit_elected(&drain[1]);
        warp_wait(&drain[1], 0, &no_abort);
    } else if (warp < kSoftWarps) {
        // ------------------------------------------------------- softmax
        const int g = warp >> 2, quad = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t ocol = tmem + lanes + Geo::kOCol + g * kHalfCols;
        const float c = p.score_scale;  // positive
        constexpr float kLazy = MmaSoftmax::kLazy;
        const int tok0 = 16 * quad + (lane >> 2);  // this thread's tokens: tok0 and tok0 + 8
        // Where this lane's row of a weights matrix goes: head, then 8 tokens.
        const int m_head = g * kHalfCols + 8 * (lane >> 4) + (lane & 7), m_piece = 2 * quad + ((lane >> 3) & 1);
        const uint32_t p_addr = smem0 + kPOff + m_head * 128 + ((m_piece ^ (m_head & 7)) << 4);
        uint32_t cnt = 0;  // tiles
        int cut = -1;
        bool failed = false, gone = false;
        for (;;) {
            const LatentPiece piece = walk.next(p);
            if (piece.s < 0)
                break;
            if (piece.first > 0)
                cut = piece.s;
            const int heads = min(NH, p.num_heads - h0);
            if (piece.len == 0) {
                const size_t at = (static_cast<size_t>(piece.s) * p.num_heads + h0) * R;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at);
                for (int e = threadIdx.x; e < heads * R / 8; e += 32 * kSoftWarps)
                    dst[e] = make_uint4(0, 0, 0, 0);
                continue;
            }
            float m[2 * J], l[2 * J];  // reference and partial sum of columns 8j + 2 (lane % 4) + e
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            for (int j = piece.first; j < piece.last; ++j, ++cnt) {
                failed = !warp_wait(&s_full[cnt & 1], (cnt >> 1) & 1, abort) || failed;
                tc_fence_after();
                float x[4 * J];
                tmem_ld_rows<J>(tmem + lanes + (cnt & 1) * NH + g * kHalfCols, x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s_free[cnt & 1]);
                const int valid = piece.len - j * kTok;  // tokens of the tile
                const bool tail = valid < kTok;
                if (tail) {
#pragma unroll
                    for (int i = 0; i < 4 * J; ++i)
                        if (tok0 + (i & 2 ? 8 : 0) >= valid)
                            x[i] = -INFINITY;
                }
                bool need = false;
                float mx[2 * J];
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    const int r = 4 * (i >> 1) + (i & 1);
                    mx[i] = fmaxf(x[r], x[r + 2]) * c;
                    need = need || mx[i] > m[i] + kLazy;
                }
                if (failed && lane == 0)
                    s_failed[g][cnt & 1] = 1;
                need = half_any(g, need);
                gone = *reinterpret_cast<volatile int *>(&s_failed[g][cnt & 1]) != 0;
                if (gone)
                    break;
                if (need) {
                    // Maxima over the tile's tokens, of every head of this half.
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
#pragma unroll
                        for (int w = 4; w <= 16; w <<= 1)
                            mx[i] = fmaxf(mx[i], __shfl_xor_sync(kFullMask, mx[i], w));
                        if (lane < 4)
                            s_red[g][quad][8 * (i >> 1) + 2 * lane + (i & 1)] = mx[i];
                    }
                    half_sync(g);
                    float alpha[2 * J];
#pragma unroll
                    for (int i = 0; i < 2 * J; ++i) {
                        const int col = 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                        const float top = fmaxf(fmaxf(s_red[g][0][col], s_red[g][1][col]),
                                                fmaxf(s_red[g][2][col], s_red[g][3][col]));
                        const float up = fmaxf(m[i], top);
                        alpha[i] = up == m[i] ? 1.f : MmaSoftmax::ex2(m[i] - up);
                        m[i] = up;
                        l[i] *= alpha[i];
                        if (quad == 0 && lane < 4)
                            s_col[g * kHalfCols + col] = alpha[i];
                    }
                    half_sync(g);
                    if (j > piece.first) {
                        // O^T holds earlier tiles: all their products are done.
                        failed = !warp_wait(&pv_done, (cnt - 1) & 1, abort) || failed;
                        tc_fence_after();
#pragma unroll 1
                        for (int t = 0; t < kTiles; ++t)
#pragma unroll
                            for (int c0 = 0; c0 < kHalfCols; c0 += 8) {
                                float o[8];
                                tmem_ld8(ocol + t * NH + c0, o);
                                const float4 a = *reinterpret_cast<const float4 *>(&s_col[g * kHalfCols + c0]);
                                const float4 b = *reinterpret_cast<const float4 *>(&s_col[g * kHalfCols + c0 + 4]);
                                o[0] *= a.x;
                                o[1] *= a.y;
                                o[2] *= a.z;
                                o[3] *= a.w;
                                o[4] *= b.x;
                                o[5] *= b.y;
                                o[6] *= b.z;
                                o[7] *= b.w;
                                tmem_st8(ocol + t * NH + c0, o);
                            }
                        tmem_wait_st();
                    }
                }
                // Weights 2^(c x - m); a head of nothing but -inf so far has weights 0.
                uint32_t w[2 * J];
#pragma unroll
                for (int i = 0; i < 2 * J; i += 2) {
                    const float o0 = m[i] == -INFINITY ? 0.f : -m[i], o1 = m[i + 1] == -INFINITY ? 0.f : -m[i + 1];
                    const float a0 = MmaSoftmax::ex2(fmaf(x[2 * i], c, o0));
                    const float a1 = MmaSoftmax::ex2(fmaf(x[2 * i + 1], c, o1));
                    const float b0 = MmaSoftmax::ex2(fmaf(x[2 * i + 2], c, o0));
                    const float b1 = MmaSoftmax::ex2(fmaf(x[2 * i + 3], c, o1));
                    l[i] += a0 + b0;
                    l[i + 1] += a1 + b1;
                    w[i] = pack_bf16(a0, a1);
                    w[i + 1] = pack_bf16(b0, b1);
                }
                // The last tile's products with P are done: P may be written.
                if (cnt > 0)
                    failed = !warp_wait(&pv_done, (cnt - 1) & 1, abort) || failed;
                if constexpr (J == 1) {
                    stsm_t2(p_addr, w[0], w[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * J; i += 4)
                        stsm_t4(p_addr + 8 * (i / 2) * 128, w[i], w[i + 1], w[i + 2], w[i + 3]);
                }
                if (tail) {
                    // Rows past the end may hold anything.
                    const int rows = kTok - valid;
                    unsigned char *pa = smem + kAOff + cnt % NA * Geo::kA, *pb = smem + kBOff + cnt % NB * Geo::kB;
                    for (int e = threadIdx.x; e < rows * (CA + CB) * 8; e += 32 * kSoftWarps) {
                        const int row = valid + e / (8 * (CA + CB)), x = e % (8 * (CA + CB));  // 16-byte pieces
                        unsigned char *at = x < 8 * CA ? pa + (row >> 3) * (CA * kAtom) + (x >> 3) * kAtom
                                                       : pb + (row >> 3) * (CB * kAtom) + ((x >> 3) - CA) * kAtom;
                        *reinterpret_cast<uint4 *>(at + (row & 7) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full);
            }
            if (gone)
                break;
            // Sums of the heads' weights.
#pragma unroll
            for (int i = 0; i < 2 * J; ++i) {
#pragma unroll
                for (int w = 4; w <= 16; w <<= 1)
                    l[i] += __shfl_xor_sync(kFullMask, l[i], w);
                if (lane < 4)
                    s_red[g][quad][8 * (i >> 1) + 2 * lane + (i & 1)] = l[i];
            }
            half_sync(g);
            const bool whole = piece.whole();
            const size_t slot = (static_cast<size_t>(latent_slot(team, piece)) * p.head_tiles + ht) * NH;
            if (quad == 0 && lane < 4) {
#pragma unroll
                for (int i = 0; i < 2 * J; ++i) {
                    const int col = 8 * (i >> 1) + 2 * lane + (i & 1), h = g * kHalfCols + col;
                    const float sum = s_red[g][0][col] + s_red[g][1][col] + s_red[g][2][col] + s_red[g][3][col];
                    s_col[h] = whole ? 1.f / sum : 1.f;
                    if (!whole && h < heads)
                        p.part_ml[slot + h] = make_float2(m[i], sum);
                }
            }
            half_sync(g);
            failed = !warp_wait(&pv_done, (cnt - 1) & 1, abort) || failed;
            tc_fence_after();
            {
                const int d = 32 * quad + lane, h = g * kHalfCols;
                const int mine = min(kHalfCols, heads - h);
                const float *f = s_col + h;
                if (whole)
                    store_heads<kTiles, NH, kHalfCols>(ocol, mine, [&](int t, int e, float x) {
                        static_cast<__nv_bfloat16 *>(p.out)[(static_cast<size_t>(piece.s) * p.num_heads + h0 + h + e) * R +
                                                            128 * t + d] = __float2bfloat16(x * f[e]);
                    });
                else
                    store_heads<kTiles, NH, kHalfCols>(ocol, mine, [&](int t, int e, float x) {
                        p.part[(slot + h + e) * R + 128 * t + d] = x;
                    });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&o_free);
        }
        if ((failed || gone) && lane == 0) {
            set_status(p.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        if (threadIdx.x == 0 && ht == 0)
            p.pieces[team] = cut;
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kValueWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Geo::kAlloc)
                     : "memory");
    }
}

// ------------------------------------------------------------------ host

// [outer][rows][numbers] bf16, dense, as [outer][chunks][rows][64]: boxes of `box_rows` rows
// x `box_chunks` chunks in the 128-byte swizzle mode; zeros past the edges.
bool encode_chunks(EncodeTiledFn enc, CUtensorMap *map, const void *base, int numbers, int rows, int64_t outer,
                   int box_rows, int box_chunks)
{
    const cuuint64_t row = static_cast<cuuint64_t>(numbers) * 2;
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(numbers / 64),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[3] = {row, 128, row * rows};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_chunks), 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, int NH> pkv_status launch_tc(const LatentDecodeParams &p, cudaStream_t stream)
{
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(latent_tc_kernel<R, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    LtGeom<R, NH>::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    EncodeTiledFn enc = encoder();
    if (!enc)
        return PKV_ERR_UNSUPPORTED;
    LatentMaps maps;
    using Geo = LtGeom<R, NH>;
    constexpr int kRow = R + kRopeDim;
    if (!encode_chunks(enc, &maps.q, p.q, kRow, p.num_heads, p.num_seqs, NH, kRow / 64) ||
        !encode_chunks(enc, &maps.a, p.cache, kRow, kBlockSize, p.num_blocks, 8, Geo::CA) ||
        !encode_chunks(enc, &maps.b, p.cache, kRow, kBlockSize, p.num_blocks, 8, Geo::CB))
        return PKV_ERR_INVALID_ARG;
    latent_tc_kernel<R, NH><<<p.teams * p.head_tiles, kThreads, LtGeom<R, NH>::kSmem, stream>>>(p, maps);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int R> pkv_status launch_tc_r(const LatentDecodeParams &p, cudaStream_t stream)
{
    return p.tile_heads == 16 ? launch_tc<R, 16>(p, stream)
                              : p.tile_heads == 32 ? launch_tc<R, 32>(p, stream) : launch_tc<R, 64>(p, stream);
}

}  // namespace

pkv_status launch_latent_decode_tc(const LatentDecodeParams &p, cudaStream_t stream)
{
    return p.latent_dim == 512 ? launch_tc_r<512>(p, stream) : launch_tc_r<256>(p, stream);
}

}  // namespace pkv
