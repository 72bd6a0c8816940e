// ffn_plan.cpp -- the plans of the feed-forward block's launches and the order of
// their work, on the CPU: linked with the library's objects and the stand-in runtime.
#include <vector>

#include "moe_ffn.h"

namespace {

using namespace moe;

struct Product {
    int M, N, K, a_mn, b_mn;
};

// Of one chunk of a pair's tile: its MMAs, or the copies.
int cycles(int n) { return 2 * n > 256 + n ? 2 * n : 256 + n; }

// 0, or what is wrong with the plan of one launch.
int look(int epilogue, const Product *products, int count, int sms, long long *most)
{
    FfnLaunch l = {};
    l.epilogue = epilogue;
    l.q.count = count;
    for (int g = 0; g < count; ++g) {
        FfnArgs &a = l.q.p[g];
        a.M = products[g].M;
        a.N = products[g].N;
        a.K = products[g].K;
        a.a_mn = products[g].a_mn;
        a.b_mn = products[g].b_mn;
    }
    ffn_plan(&l, sms);
    const FfnGroup &q = l.q;
    const int features = (epilogue == kFfnJoin ? 64 : 128) * (l.split ? 1 : 2);
    if (q.stages < 2 || q.bytes < 16384 || q.bytes % 1024)
        return 1;
    for (int g = 0; g < count; ++g) {
        const FfnArgs &a = q.p[g];
        const int rows = l.split ? a.tile_n : a.tile_n / 2;
        if (a.tile_n < 16 || a.tile_n > 256 || a.tile_n % 16 || rows % 8)
            return 2;
        if (static_cast<long long>(a.m_tiles) * features < a.M || static_cast<long long>(a.n_tiles) * a.tile_n < a.N)
            return 3;
        if (a.chunks * 64LL < a.K || (!a.b_mn && a.box_b != rows))
            return 4;
        if (16384 + (a.b_mn ? (rows + 63) / 64 * 8192 : rows * 128) > q.bytes)
            return 5;
    }
    most[4] = 0;
    for (int g = 0; g < count; ++g)
        most[4] += static_cast<long long>(q.p[g].m_tiles) * q.p[g].n_tiles * q.p[g].chunks * cycles(q.p[g].tile_n);
    if (l.split) {
        if (count != 1 || l.split > 8 || l.split > q.p[0].chunks || q.p[0].b_mn)
            return 6;
        if (static_cast<long long>(q.p[0].m_tiles) * q.p[0].n_tiles * l.split > 0x7FFFFFFF)
            return 7;
        return 0;
    }
    // every chunk of every tile once, in the shares of its tile's pairs; each part is awaited by the pair that ends the tile
    std::vector<std::vector<std::vector<int>>> done(count);
    for (int g = 0; g < count; ++g)
        done[g].assign(q.p[g].m_tiles * q.p[g].n_tiles, {});
    std::vector<int> written(q.pairs, 0), awaited(q.pairs, 0);
    const int busy = q.cut ? q.pairs : q.whole < q.pairs ? q.whole : q.pairs;
    for (int p = 0; p < busy; ++p) {
        Items w(q, p);
        Item it;
        bool last = false;
        long long units = 0;
        while (w.next(it)) {
            const FfnArgs &a = q.p[it.g];
            int m, n;
            if (it.g < 0 || it.g >= count || it.tile < 0 || it.tile >= a.m_tiles * a.n_tiles || it.c0 < 0 ||
                it.c0 >= it.c1 || it.c1 > a.chunks)
                return 8;
            tile_of(a, it.tile, m, n);
            if (m < 0 || m >= a.m_tiles || n < 0 || n >= a.n_tiles)
                return 9;
            Item end;
            if (last)
                return 10;  // what waits for others comes last
            if (w.last(end) != (it.kind == kLast) && it.kind == kLast)
                return 17;
            if (it.kind == kWhole && (it.c0 != 0 || it.c1 != a.chunks))
                return 11;
            if (it.kind == kPart && written[p]++)
                return 12;  // one part to a pair
            if (it.kind == kLast) {
                last = true;
                if (it.c1 != a.chunks || it.c0 == 0 || w.first_of_last() < 0 || w.first_of_last() >= p)
                    return 13;
                for (int o = w.first_of_last(); o < p; ++o)
                    if (q.begin[o] < q.begin[o + 1])
                        ++awaited[o];
            }
            units += static_cast<long long>(it.c1 - it.c0) * cycles(a.tile_n);
            auto &list = done[it.g][it.tile];
            for (int c = it.c0; c < it.c1; ++c)
                list.push_back(c);
        }
        *most = units > *most ? units : *most;
    }
    for (int g = 0; g < count; ++g)
        for (auto &list : done[g]) {
            if (static_cast<int>(list.size()) != q.p[g].chunks)
                return 14;
            std::vector<char> have(list.size(), 0);
            for (const int c : list)
                if (have[c]++)
                    return 15;
        }
    for (int p = 0; p < q.pairs; ++p)
        if (written[p] != awaited[p])
            return 16;
    return 0;
}

}  // namespace

extern "C" {

// The launches of every call of a block: 0, or 100 * the launch + what is wrong. v: the busiest pair's
// cycles of each, and all cycles of each.
int ffn_look(int T, int H, int I, int sms, int wanted, long long *v)
{
    const Product join = {I, T, H, 0, 0}, down = {H, T, I, 0, 0}, split = {I, T, H, 1, 0};
    const Product dx = {H, T, 2 * I, 1, 0}, up = {H, 2 * I, T, 1, 1}, low = {I, H, T, 1, 1};
    const Product all[3] = {2 * I > 16 * T ? up : dx, 2 * I > 16 * T ? low : up, 2 * I > 16 * T ? dx : low};  // as the calls order them
    for (int i = 0; i < 8; ++i)
        v[i] = 0;
    if (const int bad = look(moe::kFfnJoin, &join, 1, sms, v))
        return 100 + bad;
    if (const int bad = look(moe::kFfnStore, &down, 1, sms, v + 1))
        return 200 + bad;
    if (const int bad = look(moe::kFfnSplit, &split, 1, sms, v + 2))
        return 300 + bad;
    Product some[3];
    int n = 0;
    for (int g = 0; g < 3; ++g)
        if (wanted >> g & 1)
            some[n++] = all[g];
    if (n)
        if (const int bad = look(moe::kFfnStore, some, n, sms, v + 3))
            return 400 + bad;
    return 0;
}

}  // extern "C"
