// int4_rings.cpp -- prints, once each, the stage counts of the 4-bit kernel's
// rings (weights, tokens of the first product, of the second) that an accepted call can have.
#include <cstdio>
#include <set>
#include <tuple>

#include "moe_internal.h"

int main()
{
    std::set<std::tuple<int, int, int>> seen;
    for (const bool linear : {false, true})
        for (int tile = 8192 + 256; tile <= 8192 + 4 * 256 + 4 * 128; tile += 128)  // groups of 128 to 32, zero points
            for (int T = 1; T <= EP_MOE_MAX_TOKENS; ++T)
                for (int P = linear ? 0 : T; P <= (linear ? 0 : T * EP_MAX_TOP_K); P += T)
                    for (int E = 1; E <= (linear ? 1 : EP_MOE_MAX_EXPERTS); ++E)
                        for (int nmax = 8; nmax <= 32 && nmax <= ((T + 7) & ~7); nmax += 8) {
                            // the lists' bytes as the kernel counts them; any shared memory that it may have besides its rings
                            const int fixed = (linear ? 0 : T * moe::kTileRows * 4) + E * 22 + P * 5 + 4;
                            for (int own = 1024; own <= 2816; own += 256) {
                                const moe::Int4Layout l = moe::int4_layout(linear, moe::kSmemMax - own, fixed, 2 * tile, nmax);
                                seen.insert(std::make_tuple(l.stages, l.stages_b[0], l.stages_b[1]));
                            }
                        }
    for (const auto &s : seen)
        printf("%d %d %d\n", std::get<0>(s), std::get<1>(s), std::get<2>(s));
}
