// Work of the latent decode, shared by its kernels.
//
// A tile is 64 tokens of one sequence.  The tiles of all sequences, one after
// another, are cut into one contiguous range per team (a team: the CTAs of a
// sequence's head tiles), as equal as whole tiles allow, whatever the lengths.
// A sequence cut by a range's end leaves partial sums, which a second kernel
// joins; the others are written at once.  Short sequences are not cut: a range then
// has the sequences that begin in it.
#pragma once

#include "pkv_common.cuh"
#include "pkv_latent.h"

namespace pkv {

// Length of sequence s; one outside [0, max_len] is clamped and reported.
__device__ __forceinline__ int latent_len(const LatentDecodeParams &p, int s, bool report)
{
    int L = __ldg(p.seq_lens + s);
    if (L < 0 || L > p.max_len) {
        if (report)
            set_status(p.status, PKV_ERR_OUT_OF_RANGE);
        L = L < 0 ? 0 : p.max_len;
    }
    return L;
}
// Its tiles; an empty sequence has one, whose output is zero.
__device__ __forceinline__ int latent_tiles(int len)
{
    return len > kLatentTokens ? (len + kLatentTokens - 1) / kLatentTokens : 1;
}

// Tiles [first, last) of sequence s, which has `tiles` and `len` tokens.
struct LatentPiece {
    int s, first, last, tiles, len;
    __device__ __forceinline__ bool whole() const { return first == 0 && last == tiles; }
};

// A team's walk over its range, by one warp.
struct LatentWalk {
    int left;  // tiles still to hand out
    int s, j;  // where they begin

    __device__ __forceinline__ void init(const LatentDecodeParams &p, int team, int lane, bool report)
    {
        // A lane has a run of neighbouring sequences.  The call has less than 2^31 tiles.
        const int per = (p.num_seqs + 31) >> 5;
        const int lo = min(per * lane, p.num_seqs), hi = min(lo + per, p.num_seqs);
        unsigned mine = 0;
        for (int i = lo; i < hi; ++i)
            mine += latent_tiles(latent_len(p, i, report));
        unsigned upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned y = __shfl_up_sync(kFullMask, upto, d);
            if (lane >= d)
                upto += y;
        }
        const unsigned total = __shfl_sync(kFullMask, upto, 31);
        // Every team that works has a tile at least.
        const unsigned teams = min(total, static_cast<unsigned>(p.teams));
        left = 0;
        s = j = 0;
        if (team >= static_cast<int>(teams))
            return;
        // The first total % teams teams have a tile more.
        const unsigned each = total / teams, extra = total - each * teams;
        const unsigned begin = each * team + min(static_cast<unsigned>(team), extra);
        left = each + (team < static_cast<int>(extra) ? 1 : 0);
        const unsigned past = __ballot_sync(kFullMask, upto > begin);
        const int at = __ffs(past) - 1;
        if (lane == at) {
            int b = begin - (upto - mine);
            for (s = lo; per > 1; ++s) {
                const int n = latent_tiles(latent_len(p, s, false));
                if (b < n)
                    break;
                b -= n;
            }
            j = b;
        }
        s = __shfl_sync(kFullMask, s, at);
        j = __shfl_sync(kFullMask, j, at);
        if (p.whole && j > 0) {
            // Sequences are not cut: they belong to the team whose range they begin in.
            left -= latent_tiles(latent_len(p, s, false)) - j;
            ++s;
            j = 0;
        }
    }

    // The next piece; s = -1 when the range is used up.
    __device__ __forceinline__ LatentPiece next(const LatentDecodeParams &p)
    {
        LatentPiece r;
        r.s = -1;
        r.first = r.last = r.tiles = r.len = 0;
        if (left <= 0)
            return r;
        r.s = s;
        r.len = latent_len(p, s, false);
        r.tiles = latent_tiles(r.len);
        r.first = j;
        r.last = p.whole ? r.tiles : min(r.tiles, j + left);
        left -= r.last - r.first;
        ++s;
        j = 0;
        return r;
    }
};

// Where a cut piece of a team leaves its sums: the piece that a sequence starts
// with in the odd slot, the others in the even one.
__device__ __forceinline__ int latent_slot(int team, const LatentPiece &piece)
{
    return 2 * team + (piece.first == 0 ? 1 : 0);
}

}  // namespace pkv
