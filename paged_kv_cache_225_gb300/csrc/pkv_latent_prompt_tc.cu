// Latent attention over whole prompts, keys and values expanded per head, on the
// tcgen05 tensor cores (bf16).
//
// Expanded form: row i of a sequence and head h attends its rows j <= i with score
// scale (q[i, h, :Dn] . k[j, h] + q[i, h, Dn:] . k_rope[j]), the rotated key being
// shared by all heads, and values v[j, h] of Dn dims (causal
// scaled_dot_product_attention of the "Inference optimization" lesson, Step 2).
// One pass over the keys with the running maximum and sum of the softmax.
//
// Layout on the GPU:
//  * A tile is 128 tokens of one head.  An item is two neighbouring tiles: every block
//    of 128 keys that reaches shared memory serves both.  One persistent CTA per SM
//    walks the items (pkv_prompt.cuh).
//  * Warps 0-3 own the rows of tile 0 (a thread per row, which is its TMEM lane), 4-7
//    those of tile 1.  Warps 8 and 9 issue the TMA loads, warp 10 the MMAs, warp 11
//    looks the items up, warps 12-15 write the outputs.
//  * TMEM: scores of both tiles (2 x 128 columns, P written back over them as bf16) and
//    both outputs.  Per block and tile: S = Q K^T from shared memory, the softmax, O +=
//    P V with P read from TMEM, in two parts of 64 keys.  While one tile's threads work,
//    the tensor cores run the other tile's products.
//  * Q of both tiles takes 96 KB (Dn = 128), a block's K and V 80: what is left for them
//    holds one block and a half.  So the ring's slots are single chunks of [128 keys]
//    [64 dims], in the order of their use: K, V, the next K.  The two
//    halves of V may lie at either end of the ring: their distance goes into the operand,
//    and the half with the lower dims into the lower slot.
//  * Tiles begin at multiples of 128 tokens, so a tile sees its last block by a triangle
//    and all others whole.  P V multiplies a masked weight 0 with V rows of later tokens
//    in that block: NaN and infinities there are replaced by zeros in shared memory before
//    the product, their first rows noted per dim, and added to the outputs of the rows
//    that see them (s_seen).  Rows past the sequence are zeroed.
//  * Weights are rounded to bf16 (off by 2^-8 at most), their sum is that of the f32 ones:
//    two parts of each would double the products of P V, on the unit that bounds this.
//  * Every wait is bounded; a timeout records PKV_ERR_TIMEOUT, stops every role, lets
//    copies and MMAs in flight finish and frees TMEM.
//
// What bounds it.  Long prompts: the tensor cores and their power (one of 16K tokens, 32
// heads: 1.63 to 1.77 ms by the card, 1550 to 1690 TFLOP/s, 83 to 90% of a cuBLAS burst, 91 to 99% of what
// cuBLAS sustains): a block takes them 2560 cycles for both tiles, a step 3600, of which the
// issuing warp waits 570 for the softmax and 320 for K and V.  16 prompts of 512 to 4096
// tokens: 855 us, 1160 TFLOP/s: steps of 4150 cycles, 1160 of them waiting for the softmax
// (an item is 10 blocks, and its ends do not overlap as well).  128 prompts of 256 to 512
// tokens: 441 us, 60% of HBM's bytes; heads of 64 + 64 (37 prompts of up to 1000 tokens,
// 32 heads): 181 us; both are chains of load, scores, softmax, P V and store of items two
// or three blocks long.
//
// V with values that are not finite, one prompt of 8192 tokens, 32 heads: 438 us without,
// all NaN 626, the last token 440, every 10^4-th value 457.
//
// Measured and not kept: a barrier for each chunk instead of one for a block's K and one
// for its V (888 us against 842 on the 16 prompts, 1863 against 1717 on the long one);
// some of the exponentials by polynomial on the multiply-add units (852 us without, 885 to
// 965 with one to four in eight: issue slots, not the special function units, are short);
// the maximum with three operands to an instruction (the same).

#include "pkv_latent.h"
#include "pkv_prompt.cuh"
#include "pkv_prompt_tc.cuh"

namespace pkv {

namespace {

constexpr int kM = 128;     // rows of a tile, keys of a block
constexpr int kThreads = 512;
constexpr int kTileWarps = 4;  // warps 0 .. 7: the rows of two tiles
constexpr int kProducerWarp = 8;
constexpr int kProducers = 2;
constexpr int kMmaWarp = 10;
constexpr int kItemWarp = 11;
constexpr int kParts = 2;  // a block's P is handed to the MMAs in parts
constexpr int kPart = kM / kParts;
constexpr int kQueue = 4;  // items looked up ahead
constexpr int kChunk = kM * 128;  // bytes of [128 rows][64 bf16]
constexpr int kTurns = 4;  // barriers of the blocks in turn: more than any role is ahead of another
constexpr unsigned kNone = 0xffffu;

template <int DN> struct LpGeom {
    static constexpr int CK = DN / 64 + 1, CV = DN / 64;  // chunks of K and V of a block
    static constexpr int NS = DN == 128 ? 8 : 10;         // slots of the ring
    static constexpr int kRing = 2 * CK * kChunk;
    static constexpr int kOCol = 2 * kM;
    static_assert(kOCol + 2 * DN <= 512 && NS >= CK + CV && NS % kProducers == 0, "TMEM and the ring");
    struct Small {
        uint64_t k_full[kTurns], v_full[kTurns], k_done[kTurns], v_done[kTurns];  // block by block
        uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][kParts], o_full[2], o_free[2], l_full[2];
        uint64_t item_full[kQueue], item_empty[kQueue], drain;
        uint64_t done[2], out_sync;  // an item's outputs are written; the output warps meet
        float sum[2][kM];  // the rows' sums of weights, for the output warps
        // Per dim the first row of the item's last blocks with a NaN, +inf, -inf in V, from
        // the item's first token; two items' worth.
        unsigned short seen[2][3][DN];
        int any[2];        // an entry of seen is set
        int item[kQueue][5];
        uint32_t tmem;
        int abort, never;
    };
    static constexpr int kSmem = kRing + NS * kChunk + static_cast<int>(sizeof(Small));
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

struct LpMaps {
    CUtensorMap q, k, kr, v;
};

// One queue entry: an item, or s < 0 for the end of the work.
struct LpItem {
    int s, head, row0, n, tok0;
    int nt[2];  // tokens of the two tiles
    int nb[2];  // blocks a tile sees
    int blocks;

    __device__ __forceinline__ void fill(const int *w)
    {
        s = w[0];
        head = w[1];
        row0 = w[2];
        n = w[3];
        tok0 = w[4];
        nt[0] = min(kM, n - tok0);
        nt[1] = max(0, min(kM, n - tok0 - kM));
        nb[0] = tok0 / kM + 1;
        nb[1] = nt[1] > 0 ? nb[0] + 1 : 0;
        blocks = max(nb[0], nb[1]);
    }
};

// One box [128 rows][64 dims] of a head.
__device__ __forceinline__ void load_elected(uint32_t dst, const CUtensorMap *map, int dim, int head, int row,
                                             uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(dim), "r"(head), "r"(row), "r"(smem_u32(bar))
        : "memory");
}

// D (+)= P V over 16 keys, P from TMEM.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t}" ::"r"(d),
        "r"(p), "l"(v), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void note_first(unsigned short *at, unsigned short row)
{
    unsigned short old = *at;
    while (row < old) {
        const unsigned short was = atomicCAS(at, old, row);
        if (was == old)
            break;
        old = was;
    }
}

// What dim d of V adds to a row that sees rows up to `upto`: NaN, an infinity, or 0.
template <int DN> __device__ __forceinline__ float seen_value(const unsigned short (&seen)[3][DN], int d, int upto)
{
    const bool up = seen[1][d] <= upto, down = seen[2][d] <= upto;
    if (seen[0][d] <= upto || (up && down))
        return __int_as_float(0x7fffffff);
    return up ? INFINITY : down ? -INFINITY : 0.f;
}

template <int DN>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prompt_tc_kernel(const __grid_constant__ LatentPromptParams p, const __grid_constant__ LpMaps maps)
{
    using Geo = LpGeom<DN>;
    constexpr int NS = Geo::NS, CK = Geo::CK, CV = Geo::CV, CB = CK + CV;
    // No static shared memory: the operands begin on a 1 KB boundary.
    extern __shared__ __align__(1024) unsigned char smem[];
    typename Geo::Small &sm = *reinterpret_cast<typename Geo::Small *>(smem + Geo::kRing + NS * kChunk);
    volatile int *abort = &sm.abort;
    const volatile int *no_abort = &sm.never;  // for what has to end before the CTA may

    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t smem0 = smem_u32(smem);
    const PromptParams &pi = p.items;
    if (smem0 & 1023) {  // the operands' swizzle counts on it
        set_status(pi.status, PKV_ERR_CUDA);
        return;
    }

    if (warp == 0) {
        if (lane < kTurns) {
            mbar_init(&sm.k_full[lane], 1);
            mbar_init(&sm.v_full[lane], 1);
            mbar_init(&sm.k_done[lane], 1);
            mbar_init(&sm.v_done[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&sm.q_full[lane], 1);
            mbar_init(&sm.q_empty[lane], 1);
            mbar_init(&sm.s_full[lane], 1);
            for (int i = 0; i < kParts; ++i)
                mbar_init(&sm.p_full[lane][i], kTileWarps);
            mbar_init(&sm.o_full[lane], 1);
            mbar_init(&sm.l_full[lane], kTileWarps);
            mbar_init(&sm.o_free[lane], kTileWarps);
            mbar_init(&sm.done[lane], kTileWarps);
            sm.any[lane] = 0;
        }
        if (lane < kQueue) {
            mbar_init(&sm.item_full[lane], 1);
            mbar_init(&sm.item_empty[lane], 3 * kTileWarps + kProducers + 1);
        }
        if (lane == 0) {
            mbar_init(&sm.drain, 1);
            mbar_init(&sm.out_sync, kTileWarps);
            sm.abort = sm.never = 0;
        }
        fence_mbar_init();
    }
    for (int e = threadIdx.x; e < 2 * 3 * DN; e += kThreads)
        (&sm.seen[0][0][0])[e] = kNone;
    if (warp == kProducerWarp && lane < 4) {
        const CUtensorMap *map = lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.kr : &maps.v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    // Lane 0 of a warp gives an item's slot back.
    auto next_item = [&](unsigned k, LpItem &it) {
        const int slot = k % kQueue;
        if (!warp_sleep_wait(&sm.item_full[slot], (k / kQueue) & 1, abort))
            return false;
        it.fill(sm.item[slot]);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.item_empty[slot]);
        return true;
    };
    // Slot of chunk c, counted over all blocks.
    auto slot_of = [](uint32_t c) { return c % NS; };

    if (warp == kProducerWarp || warp == kProducerWarp + 1) {
        // ------------------------------------------------------- copies
        // One warp loads K (its own dims, then the rotated ones) and Q of tile 0, the other V
        // and Q of tile 1.  A chunk's slot is free when the block that had it NS chunks ago
        // has been used.
        const uint32_t mine = warp - kProducerWarp;
        uint32_t b = 0;   // blocks
        uint32_t qn = 0;  // Q tiles of this warp
        uint64_t *const filled = mine ? sm.v_full : sm.k_full;
        bool ok = true;
        for (unsigned k = 0; ok; ++k) {
            LpItem it;
            ok = next_item(k, it);
            if (!ok || it.s < 0)
                break;
            const int nt = mine ? it.nt[1] : it.nt[0];
            if (nt > 0) {
                if (qn > 0)
                    ok = warp_sleep_wait(&sm.q_empty[mine], (qn - 1) & 1, abort);
                if (!ok)
                    break;
                expect_elected(&sm.q_full[mine], CK * kChunk);
#pragma unroll 1
                for (int i = 0; i < CK; ++i)
                    load_elected(smem0 + (mine * CK + i) * kChunk, &maps.q, 64 * i, it.head,
                                 it.row0 + it.tok0 + static_cast<int>(mine) * kM, &sm.q_full[mine]);
                ++qn;
            }
            for (int j = 0; j < it.blocks && ok; ++j) {
                const int row = it.row0 + j * kM;
                uint64_t *bar = &filled[b % kTurns];
                const uint32_t v_slot = slot_of(b * CB + CK);
                bool asked = false;
#pragma unroll
                for (int i = 0; i < CB; ++i) {
                    if ((i >= CK) != (mine == 1))
                        continue;
                    const uint32_t c = b * CB + i, slot = slot_of(c);
                    if (c >= NS && ok) {
                        const uint32_t was = c - NS, block = was / CB;
                        uint64_t *done = was % CB < CK ? sm.k_done : sm.v_done;
                        ok = warp_sleep_wait(&done[block % kTurns], (block / kTurns) & 1, abort);
                    }
                    if (!ok)
                        break;
                    if (!asked)
                        expect_elected(bar, (mine ? CV : CK) * kChunk);
                    asked = true;
                    const uint32_t dst = smem0 + Geo::kRing + slot * kChunk;
                    if (p.drop_first_copy && blockIdx.x == 0 && c == 0)
                        continue;
                    if (i < CK - 1) {
                        load_elected(dst, &maps.k, 64 * i, it.head, row, bar);
                    } else if (i == CK - 1) {
                        load_elected(dst, &maps.kr, 0, 0, row, bar);
                    } else {
                        // V's halves at the ends of the ring trade places.
                        const int half = CV == 2 && v_slot == NS - 1 ? 1 - (i - CK) : i - CK;
                        load_elected(dst, &maps.v, 64 * half, it.head, row, bar);
                    }
                }
                // Copies of it are under way: all or, where a wait gave up, the first.
                b += asked ? 1 : 0;
            }
        }
        if (!ok && lane == 0) {
            set_status(pi.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        // Every copy still in flight lands before the CTA exits.  (One whose block was not
        // asked for whole is waited for until the limit.)
        if (lane == 0) {
            for (uint32_t x = b > kTurns ? b - kTurns : 0; x < b; ++x)
                sleep_wait(&filled[x % kTurns], (x / kTurns) & 1, no_abort);
            if (qn > 0)
                sleep_wait(&sm.q_full[mine], (qn - 1) & 1, no_abort);
        }
        __syncwarp();
    } else if (warp == kItemWarp) {
        // -------------------------------------------------- item look-up
        PromptScan scan;
        scan.init(pi, 2 * kM, lane, blockIdx.x == 0);
        bool ok = true;
        for (unsigned k = 0; ok; ++k) {
            // In alternating direction over the CTAs: a round's costliest item goes to the
            // CTA that had the cheapest of the round before.
            const unsigned at = k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
            const PromptItem found = scan.find(pi, 2 * kM, k * gridDim.x + at, lane);
            if (lane == 0) {
                const int slot = k % kQueue;
                if (k >= kQueue)
                    ok = sleep_wait(&sm.item_empty[slot], ((k / kQueue) - 1) & 1, abort);
                if (ok) {
                    int *w = sm.item[slot];
                    w[0] = found.s;
                    w[1] = found.hkv;
                    w[2] = found.row0;
                    w[3] = found.n;
                    w[4] = found.index * 2 * kM;
                    mbar_arrive(&sm.item_full[slot]);
                } else {
                    set_status(pi.status, PKV_ERR_TIMEOUT);
                    *abort = 1;
                }
            }
            ok = __shfl_sync(kFullMask, ok ? 1 : 0, 0) != 0 && found.s >= 0;
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------- MMA issue
        // A step is, tile after tile, P V of block j and the scores of block j + 1; in an
        // item's last step the scores are the next item's first ones.
        const uint32_t id_s0 = tc_idesc(kM, 0, false) | (pi.negate ? 1u << 13 : 0u);
        constexpr uint32_t kIdPV = tc_idesc(kM, DN, true);
        const uint64_t qd = operand(smem0, 1024), kd = operand(smem0 + Geo::kRing, 1024);
        uint32_t b = 0;                            // the block whose scores come next
        uint32_t q_par = 0, o_par = 3, p_par = 0;  // bit t
        unsigned k = 0;
        bool ok = true;
        LpItem it, next;
        // Scores of tile t with block b: `first` of its users waits for it,
        // `last` gives it back; the tile's `final` one gives Q back.
        auto scores = [&](int t, int cols, bool first, bool last, bool fresh, bool final) {
            if (fresh) {
                ok = ok && warp_sleep_wait(&sm.q_full[t], q_par >> t & 1, abort);
                q_par ^= 1u << t;
            }
            const uint32_t id = id_s0 | static_cast<uint32_t>(cols >> 3) << 17;
            if (first)
                ok = ok && warp_sleep_wait(&sm.k_full[b % kTurns], (b / kTurns) & 1, abort);
            if (!ok)
                return;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < CK; ++i)
                mma4<2, 2>(tmem + t * kM, qd + (t * CK + i) * (kChunk >> 4),
                           kd + slot_of(b * CB + i) * (kChunk >> 4), id, i > 0);
            commit_elected(&sm.s_full[t]);
            if (last)
                commit_elected(&sm.k_done[b % kTurns]);
            if (final)
                commit_elected(&sm.q_empty[t]);
        };
        auto cols_of = [&](const LpItem &x, int t, int j) {
            return j + 1 < x.nb[t] ? kM : (x.nt[t] + 15) & ~15;
        };
        ok = next_item(k++, it);
        bool more = ok && it.s >= 0;
        if (more) {
            scores(0, cols_of(it, 0, 0), true, it.nb[1] == 0, true, it.nb[0] == 1);
            if (ok && it.nb[1] > 0)
                scores(1, cols_of(it, 1, 0), false, true, true, it.nb[1] == 1);
        }
        while (more && ok) {
            for (int j = 0; j < it.blocks && ok; ++j) {
                const uint32_t vb = b++;  // V of this block, K of the next
                const bool end = j + 1 == it.blocks;
                if (end) {
                    ok = next_item(k++, next);
                    more = ok && next.s >= 0;
                    if (!ok)
                        break;
                }
                const uint32_t vs = slot_of(vb * CB + CK);
                const bool split = CV == 2 && vs == NS - 1;
                const uint64_t vd = operand(smem0 + Geo::kRing + (split ? 0 : vs) * kChunk, 1024,
                                            split ? (NS - 1) * kChunk : kChunk);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < it.nb[t]) {
                        if (j == 0) {  // the output of the tile's item before this one is read
                            ok = ok && warp_sleep_wait(&sm.o_free[t], o_par >> t & 1, abort);
                            o_par ^= 1u << t;
                        }
                        if (t == 0 || j >= it.nb[0])
                            ok = ok && warp_sleep_wait(&sm.v_full[vb % kTurns], (vb / kTurns) & 1, abort);
                        const int steps = cols_of(it, t, j) / 16;
                        const uint32_t d = tmem + Geo::kOCol + t * DN;
#pragma unroll
                        for (int part = 0; part < kParts; ++part) {
                            if (part * (kPart / 16) >= steps)
                                break;
                            ok = ok && warp_sleep_wait(&sm.p_full[t][part], p_par >> t & 1, abort);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint32_t a = tmem + t * kM + part * kPart;
#pragma unroll
                            for (int ks = 0; ks < kPart / 16; ++ks) {
                                if (part * (kPart / 16) + ks >= steps)
                                    break;
                                mma_pv(d, a + 32 * (ks / 2) + 8 * (ks % 2),
                                       vd + (part * (kPart / 16) + ks) * (2048 >> 4), kIdPV, j > 0 || part + ks > 0);
                            }
                        }
                        p_par ^= 1u << t;
                        if (!ok)
                            break;
                        if (t == 1 || j >= it.nb[1])
                            commit_elected(&sm.v_done[vb % kTurns]);
                        if (j + 1 == it.nb[t])
                            commit_elected(&sm.o_full[t]);
                    }
                    if (!end) {
                        const int n = j + 1;
                        if (n < it.nb[t])
                            scores(t, cols_of(it, t, n), t == 0 || n >= it.nb[0], t == 1 || n >= it.nb[1], false,
                                   n + 1 == it.nb[t]);
                    } else if (more && next.nt[t] > 0) {
                        scores(t, cols_of(next, t, 0), t == 0, t == 1 || next.nb[1] == 0, true, next.nb[t] == 1);
                    }
                    if (!ok)
                        break;
                }
            }
            it = next;
        }
        if (!ok && lane == 0) {
            set_status(pi.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        // Every MMA issued has completed before TMEM is freed.
        commit_elected(&sm.drain);
        warp_sleep_wait(&sm.drain, 0, no_abort);
    } else if (warp < 2 * kTileWarps) {
        // ------------------------------------------------------- softmax
        const int t = warp >> 2;               // tile
        const int r = threadIdx.x & (kM - 1);  // row of the tile = TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t scol = tmem + lanes + t * kM;
        const uint32_t ocol = tmem + lanes + Geo::kOCol + t * DN;
        const float c = pi.score_scale;  // positive
        constexpr float kLazy = MmaSoftmax::kLazy;
        uint32_t cnt = 0;    // blocks of this tile
        uint32_t items = 0;  // its items
        uint32_t base = 0;   // the item's first block
        bool failed = false;
        for (unsigned k = 0; !failed; ++k) {
            LpItem it;
            if (!next_item(k, it)) {
                failed = true;
                break;
            }
            if (it.s < 0)
                break;
            // Selected, not indexed: the item stays in registers.
            const int nt = t ? it.nt[1] : it.nt[0], nb = t ? it.nb[1] : it.nb[0];
            float m = -INFINITY;  // running maximum, log2 units
            float2 l2[2] = {};    // its sum, in four parts
            for (int j = 0; j < nb; ++j, ++cnt) {
                if (!warp_wait(&sm.s_full[t], cnt & 1, abort)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const bool tail = j + 1 == nb;
                const int cols = tail ? (nt + 15) & ~15 : kM;
                const bool second = cols > kPart;   // the block has keys in its second part
                const int lim = min(r, nt - 1) + 1; // keys this row sees of its last block
                // Twice through the scores, for the maximum and for the weights.
                float mx = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < (second ? kM : kPart); c0 += 64) {
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
                        // O holds earlier blocks, whose P V is done: these scores were
                        // issued, and so completed, after it.
#pragma unroll 1
                        for (int c0 = 0; c0 < DN; c0 += 16) {
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
                if (tail) {
                    // V of the last block: rows past the sequence become zero, and so do
                    // values that are not finite, which are noted.
                    const uint32_t vb = base + j, vs = slot_of(vb * CB + CK);
                    if (!warp_wait(&sm.v_full[vb % kTurns], (vb / kTurns) & 1, abort)) {
                        failed = true;
                        break;
                    }
                    const bool split = CV == 2 && vs == NS - 1;
                    const int first = j * kM - it.tok0, past = it.n - j * kM;
                    unsigned short(&seen)[3][DN] = sm.seen[k & 1];
                    for (int e = r; e < cols * (DN / 8); e += kM) {
                        const int row = e / (DN / 8), piece = e % (DN / 8), half = piece >> 3;
                        const uint32_t slot = split ? (half ? NS - 1 : 0) : vs + half;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + Geo::kRing + slot * kChunk + row * 128 +
                                                              (((piece & 7) ^ (row & 7)) << 4));
                        if (row >= past) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 v4 = *at;
                        uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
                        bool bad = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad = bad || (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
                        if (!bad)
                            continue;
                        // The outputs of the item that noted here before are written.
                        if (k >= 2 && !tc_wait(&sm.done[k & 1], ((k >> 1) - 1) & 1, abort))
                            continue;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t x = w[i >> 1] >> (16 * (i & 1)) & 0xffffu;
                            if ((x & 0x7f80u) != 0x7f80u)
                                continue;
                            const int kind = (x & 0x7fu) ? 0 : (x & 0x8000u) ? 2 : 1;
                            note_first(&seen[kind][8 * piece + i], static_cast<unsigned short>(first + row));
                            w[i >> 1] &= i & 1 ? 0xffffu : 0xffff0000u;
                        }
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                        sm.any[k & 1] = 1;
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
                // Weights 2^(c x - m), in bf16 pairs over the consumed scores; a row of
                // nothing but -inf so far has weights 0.
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
                        weights32<false>(x, c, off, l2, pc);
                        weights32<false>(y, c, off, l2, pc + 32);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                    }
                    if (lane == 0)  // both parts' barriers count every block
                        mbar_arrive(&sm.p_full[t][part]);
                }
            }
            base += it.blocks;
            if (failed)
                break;
            if (nb == 0)
                continue;
            // The sums go to the output warps, once they have read the last ones.
            if (items > 0 && !warp_wait(&sm.o_free[t], (items - 1) & 1, abort)) {
                failed = true;
                break;
            }
            ++items;
            const float2 lsum = add2(l2[0], l2[1]);
            sm.sum[t][r] = lsum.x + lsum.y;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.l_full[t]);
        }
        if (failed && lane == 0) {
            set_status(pi.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    } else {
        // --------------------------------------------------- output rows
        const int r = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t par = 0;  // bit t: parity of the tile's barriers
        uint32_t meets = 0;
        bool failed = false;
        for (unsigned k = 0; !failed; ++k) {
            LpItem it;
            if (!next_item(k, it)) {
                failed = true;
                break;
            }
            if (it.s < 0)
                break;
            bool bad = false;
            unsigned short(&seen)[3][DN] = sm.seen[k & 1];
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? it.nt[1] : it.nt[0];
                if (nt == 0)
                    continue;
                if (!warp_sleep_wait(&sm.l_full[t], par >> t & 1, abort) ||
                    !warp_sleep_wait(&sm.o_full[t], par >> t & 1, abort)) {
                    failed = true;
                    break;
                }
                par ^= 1u << t;
                tc_fence_after();
                const uint32_t ocol = tmem + lanes + Geo::kOCol + t * DN;
                const float inv = 1.f / sm.sum[t][r];
                bad = *reinterpret_cast<volatile int *>(&sm.any[k & 1]) != 0;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                     (static_cast<size_t>(it.row0 + it.tok0 + t * kM + min(r, nt - 1)) *
                                          pi.num_kv_heads + it.head) * DN;
#pragma unroll 1
                for (int c0 = 0; c0 < DN; c0 += 32) {
                    float ov[32];
                    tmem_ld32(ocol + c0, ov);
                    if (c0 + 32 == DN) {  // read whole: the next item's P V may start
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&sm.o_free[t]);
                    }
                    if (bad) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] = ov[e] * inv + seen_value<DN>(seen, c0 + e, t * kM + r);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] *= inv;
                    }
                    const bool live = r < nt;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16(ov[16 * i + 2 * e], ov[16 * i + 2 * e + 1]);
                        __nv_bfloat16 *at = dst + c0 + 16 * i;
                        if (live && wide) {  // whole sectors
                            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(w[0]),
                                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                         : "memory");
                        } else if (live) {
                            reinterpret_cast<uint4 *>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4 *>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (failed)
                break;
            if (bad) {  // the same for all four warps: the item's last tile has been handed over
                // What was noted goes once all of them have read it.
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.out_sync);
                if (!warp_sleep_wait(&sm.out_sync, meets++ & 1, abort)) {
                    failed = true;
                    break;
                }
                for (int e = r; e < 3 * DN; e += 32 * kTileWarps)
                    (&seen[0][0])[e] = kNone;
                if (r == 0)
                    sm.any[k & 1] = 0;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.done[k & 1]);
        }
        if (failed && lane == 0) {
            set_status(pi.status, PKV_ERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------------ host

// Rows of [tokens][heads][D] bf16, token and head strides in elements: boxes of 64
// elements x one head x 128 tokens in the 128-byte swizzle mode.
bool encode_rows(EncodeTiledFn enc, CUtensorMap *map, const void *base, int D, int heads, int64_t tokens,
                 int64_t stride, int64_t head)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, kM};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DN> pkv_status launch_lp_tc(LatentPromptParams p, cudaStream_t stream)
{
    using Geo = LpGeom<DN>;
    static ContextCache cache;
    int set = 0;
    const pkv_status rc = cache.get(&set, [](int *out) -> pkv_status {
        *out = 1;
        return cudaFuncSetAttribute(latent_prompt_tc_kernel<DN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Geo::kSmem) == cudaSuccess
                   ? PKV_OK
                   : PKV_ERR_CUDA;
    });
    if (rc != PKV_OK)
        return rc;
    EncodeTiledFn enc = encoder();
    if (!enc)
        return PKV_ERR_UNSUPPORTED;
    const int H = p.items.num_kv_heads;
    const int64_t T = p.items.num_tokens;
    LpMaps maps;
    if (!encode_rows(enc, &maps.q, p.q, DN + kRopeDim, H, T, p.q_stride, DN + kRopeDim) ||
        !encode_rows(enc, &maps.k, p.k, DN, H, T, p.k_stride, p.k_head) ||
        !encode_rows(enc, &maps.kr, p.k_rope, kRopeDim, 1, T, p.k_rope_stride, kRopeDim) ||
        !encode_rows(enc, &maps.v, p.v, DN, H, T, p.v_stride, p.v_head))
        return PKV_ERR_INVALID_ARG;
    const long items = prompt_max_items(p.items, 2 * kM);
    if (items <= 0)
        return PKV_OK;
    if (items > 0x40000000L)
        return PKV_ERR_UNSUPPORTED;
    p.items.max_items = static_cast<unsigned>(items);
    const long sms = device_sm_count();
    latent_prompt_tc_kernel<DN><<<static_cast<unsigned>(items < sms ? items : sms), kThreads, Geo::kSmem, stream>>>(
        p, maps);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_latent_prompt_tc(const LatentPromptParams &p, cudaStream_t stream)
{
    return p.nope == 128 ? launch_lp_tc<128>(p, stream) : launch_lp_tc<64>(p, stream);
}

}  // namespace pkv
