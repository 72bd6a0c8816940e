// moe_ffn.h -- the order of a feed-forward launch's work: tiles in bands, and
// what each pair of blocks does (shared with the test of all plans).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kBand = 8;  // row tiles of a band of tiles

// i / d and the rest, 0 <= i, by d's reciprocal: the quotient is below 2^22, so a float is off by one at most.
static __host__ __device__ __forceinline__ int divide(int i, int d, float inverse, int &rest)
{
    int n = static_cast<int>(static_cast<float>(i) * inverse);
    rest = i - n * d;
    if (rest < 0) {
        --n;
        rest += d;
    } else if (rest >= d) {
        ++n;
        rest -= d;
    }
    return n;
}

// Tiles in bands of kBand row tiles, feature tiles one after the other within a band: tiles that run at a time share
// operands in L2. (Each role goes through this for each tile; divisions took 0.4 us of it.)
static __host__ __device__ __forceinline__ void tile_of(const FfnArgs &a, int i, int &m, int &n)
{
    int in, column;
    const int first = divide(i, kBand * a.m_tiles, a.band_inverse, in) * kBand, left = a.n_tiles - first;
    m = left >= kBand ? in / kBand : divide(in, left, a.rest_inverse, column);
    n = first + in - m * (left >= kBand ? kBand : left);
}

// A pair's work: a tile of product g over chunks [c0, c1) of K.
enum ItemKind { kWhole = 0, kPart, kLast };  // a part's sums go to memory; the last part of a tile adds the others'
struct Item {
    int g, tile, c0, c1, kind;
};

// In the order in which all roles go through it: the first part of a tile that later pairs end (whose reader then finds it:
// after the whole tiles the gradients of 700 rows, 1024 x 9000, take 102 us, 91 so); whole tiles, every pairs-th; tiles cut
// out of the last rounds in full; the last part of a tile that earlier pairs began.
struct Items {
    const FfnGroup &q;
    const int pair;
    int gb, tb, cb, ge, te, ce;  // the share of the cut rounds: from chunk cb of tile tb of product gb to ge, te, ce
    bool any;
    int phase, g, t;

    __host__ __device__ __forceinline__ Items(const FfnGroup &q_, int pair_) : q(q_), pair(pair_), phase(0)
    {
        any = q.begin[pair] < q.begin[pair + 1];
        locate(q.begin[pair], gb, tb, cb);
        locate(q.begin[pair + 1], ge, te, ce);
        g = 0;
        t = pair;
    }
    __host__ __device__ __forceinline__ void locate(int u, int &at_g, int &at_t, int &at_c) const
    {
        for (at_g = 0; at_g < q.count - 1; ++at_g) {
            const FfnArgs &a = q.p[at_g];
            const int units = (a.m_tiles * a.n_tiles - a.whole) * a.chunks;
            if (u < units)
                break;
            u -= units;
        }
        at_t = q.p[at_g].whole + u / q.p[at_g].chunks;
        at_c = u % q.p[at_g].chunks;
    }
    __host__ __device__ __forceinline__ bool part(Item &it) const
    {
        if (!any || ce == 0)
            return false;
        it = {ge, te, gb == ge && tb == te ? cb : 0, ce, kPart};
        return true;
    }
    __host__ __device__ __forceinline__ bool last(Item &it) const
    {
        if (!any || cb == 0 || (gb == ge && tb == te))  // all of the share is in one tile
            return false;
        it = {gb, tb, cb, q.p[gb].chunks, kLast};
        return true;
    }
    __host__ __device__ __forceinline__ bool next(Item &it)
    {
        if (phase == 0) {
            phase = 1;
            if (part(it))
                return true;
        }
        if (phase == 1) {
            if (t < q.whole) {
                int i = t;
                for (g = 0; g < q.count - 1 && i >= q.p[g].whole; ++g)
                    i -= q.p[g].whole;
                t += q.pairs;
                it = {g, i, 0, q.p[g].chunks, kWhole};
                return true;
            }
            phase = 2;
            g = gb;
            t = tb + (cb > 0);
        }
        if (phase == 2) {
            while (any && g < ge && t >= q.p[g].m_tiles * q.p[g].n_tiles)
                t = q.p[++g].whole;
            if (any && (g < ge || t < te)) {
                it = {g, t++, 0, q.p[g].chunks, kWhole};
                return true;
            }
            phase = 3;
            return last(it);
        }
        return false;
    }
    // The first of the pairs that have parts of the tile that this one ends.
    __host__ __device__ __forceinline__ int first_of_last() const
    {
        const int start = q.begin[pair] - cb;
        int p = pair - 1;
        while (p > 0 && q.begin[p] > start)
            --p;
        return p;
    }
};

}  // namespace moe
