// moe_sched.h -- what the two experts kernels share: the lists of chosen
// experts, the split of the work over the blocks, rings, and h.
#pragma once

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

static __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Position in a ring of n stages and the parity of its current round.
struct Cursor {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++s == n) {
            s = 0;
            parity ^= 1;
        }
    }
    // k <= n
    __device__ __forceinline__ void advance(int k, int n)
    {
        const int to = s + k;
        parity ^= to >= n ? 1 : 0;
        s = to >= n ? to - n : to;
    }
};

// Walks a block's share [begin, end) of one product's units (chunks of
// inputs), one run of chunks of one (expert i, row tile m) after the other.
// The first product goes expert by expert, the second row tile by row tile.
// Only the start costs divisions.
struct Walk {
    int i, m, k, len, left;
    const int chunks, inner;
    const bool second;

    __device__ __forceinline__ Walk(int begin, int end, int chunks_, int inner_, bool second_)
        : left(end - begin), chunks(chunks_), inner(inner_), second(second_)
    {
        const int tile = begin / chunks, outer = tile / inner, in = tile - outer * inner;
        k = begin - tile * chunks;
        i = second ? in : outer;
        m = second ? outer : in;
        len = min(chunks - k, left);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next()
    {
        left -= len;
        k = 0;
        len = min(chunks, left);
        int &in = second ? i : m;
        if (++in == inner) {
            in = 0;
            ++(second ? m : i);
        }
    }
};

// `total` units cut into contiguous shares, one per block, that differ by one
// at most; blocks beyond `total` have none, so every block of a run of blocks
// has a part in a tile they share.
struct Shares {
    int each, more;  // units of a share; the first `more` blocks have one more

    __device__ __forceinline__ Shares(int total, int G) : Shares(total / G, total, G) {}
    __device__ __forceinline__ Shares(int each_, int total, int G) : each(each_), more(total - each_ * G) {}
    __device__ __forceinline__ int begin(int b) const { return b * each + min(b, more); }
    __device__ __forceinline__ int owner(int u) const
    {
        const int edge = more * (each + 1);
        return u < edge ? u / (each + 1) : more + (u - edge) / each;
    }
};

// The same for units of different costs: block b has the units whose place, the
// cost of all before them, is in [b, b + 1) times total / blocks. No share is
// empty if that is at least the largest cost of a unit. Places fit 32 bits:
// weights that a GPU's memory holds are far fewer units.
struct CostShares {
    uint32_t total, each, more;
    int blocks;

    // blocks: as many as have a share, G at most
    __device__ __forceinline__ CostShares(uint32_t total_, uint32_t largest, int G)
        : total(total_), blocks(static_cast<int>(min(static_cast<uint32_t>(G), total_ / largest)))
    {
        each = total / blocks;
        more = total - each * blocks;
    }
    __device__ __forceinline__ uint32_t begin(int b) const
    {
        return b >= blocks ? total : each * b + (more * b + blocks - 1) / blocks;
    }
    __device__ __forceinline__ int owner(uint32_t place) const
    {
        int b = min(static_cast<int>(place / each), blocks - 1);  // or one of the few before it
        while (begin(b) > place)
            --b;
        return b;
    }
};

// A tile that blocks b0..b1 share: each keeps its part in one of two slots,
// the second if the tile begins after the block's share does.
struct Split {
    int b0, b1, slot0;

    Split() = default;
    __device__ __forceinline__ Split(const Shares &s, int first_unit, int units)
        : b0(s.owner(first_unit)), b1(s.owner(first_unit + units - 1)),
          slot0(2 * b0 + (first_unit > s.begin(b0) ? 1 : 0))
    {
    }
    __device__ __forceinline__ bool shared() const { return b0 != b1; }
    __device__ __forceinline__ int parts() const { return b1 - b0 + 1; }
    __device__ __forceinline__ int slot(int b) const { return b == b0 ? slot0 : 2 * b; }
    // As above where units' costs differ: the costs before the tile's first and last unit and before the unit that
    // precedes it.
    __device__ __forceinline__ Split(const CostShares &s, uint32_t first, uint32_t last, uint32_t before)
        : b0(s.owner(first)), b1(s.owner(last)), slot0(2 * b0 + (first > 0 && before >= s.begin(b0) ? 1 : 0))
    {
    }
    // Of n columns, the first that block b adds up (b == b1 + 1: n).
    __device__ __forceinline__ int column(int n, int b) const { return n * (b - b0) / parts(); }
};

// A run of chunks whose tile other blocks share is left as a part and settled
// after the product's last run, when the others are about to be done too:
// each of them then adds up the parts of some columns. A block has at most
// two such runs, the first and the last.
struct Rest {
    int i, m;
};
struct Rests {
    int n;
    Rest of[2];
};

// Sums v[c] of N values of a shared tile over the parts, in the order of the
// inputs: four columns, of which the first `cols` are there (the rest are 0),
// or twice four, `second` values apart. `base` is the first value in slot 0. Four parts'
// loads are in flight, or two.
template <int N>
static __device__ __forceinline__ void sum_parts(const float *base, int part_floats, const Split &sp, int cols, float *v,
                                                 int second = 0)
{
    static_assert(N == 4 || N == 8, "");
    constexpr int kFlight = N > 4 ? 2 : 4;
#pragma unroll
    for (int c = 0; c < N; ++c)
        v[c] = (c & 3) < cols ? __ldcg(base + static_cast<size_t>(sp.slot0) * part_floats + (c & 3) * kTileRows + (c >> 2) * second) : 0.0f;
    for (int b = sp.b0 + 1; b <= sp.b1; b += kFlight) {
        float x[kFlight][N];
#pragma unroll
        for (int q = 0; q < kFlight; ++q)
#pragma unroll
            for (int c = 0; c < N; ++c)
                x[q][c] = b + q <= sp.b1 && (c & 3) < cols
                              ? __ldcg(base + static_cast<size_t>(2 * (b + q)) * part_floats + (c & 3) * kTileRows + (c >> 2) * second)
                              : 0.0f;
#pragma unroll
        for (int q = 0; q < kFlight; ++q)
#pragma unroll
            for (int c = 0; c < N; ++c)
                v[c] += x[q][c];
    }
}

// Two bf16 values whose sum carries 16 bits of v's mantissa (v itself where it is not finite).
static __device__ __forceinline__ void split(float v, __nv_bfloat16 &hi, __nv_bfloat16 &lo)
{
    hi = __float2bfloat16_rn(v);
    const float r = v - __bfloat162float(hi);
    lo = __float2bfloat16_rn(isfinite(r) ? r : 0.0f);
}

static __device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// Lists of the chosen experts, in dynamic shared memory. An entry is an expert
// with up to `cap` of its tokens; an expert with more has two entries. What
// only building them needs lies in `scratch`, 6 P bytes: the kernels give the
// sums of y, which come into use long after (up to 12 KB less for the rings).
struct Lists {
    unsigned long long *mask;  // [E] tokens of each expert
    float *weight;             // [P] routing weight of each (entry, token) pair
    float *given;              // [P] the call's weights; scratch
    unsigned short *expert;    // [2 E] of each entry, ascending
    unsigned short *offset;    // [2 E + 1] the entry's first pair
    unsigned short *blocks;    // [2 E + 1] column blocks of 8 tokens before the entry
    unsigned short *start;     // [E] each active expert's first pair
    short *id;                 // [P] the call's ids, local; scratch
    unsigned char *token;      // [P] tokens, ascending per expert

    __device__ __forceinline__ Lists(void *at, void *scratch, int E, int P)
    {
        mask = static_cast<unsigned long long *>(at);
        weight = reinterpret_cast<float *>(mask + E);
        given = static_cast<float *>(scratch);
        expert = reinterpret_cast<unsigned short *>(weight + P);
        offset = expert + 2 * E;
        blocks = offset + 2 * E + 1;
        start = blocks + 2 * E + 1;
        id = reinterpret_cast<short *>(given + P);
        token = reinterpret_cast<unsigned char *>(start + E);
    }
    __device__ __forceinline__ int count(int i) const { return offset[i + 1] - offset[i]; }
};

static inline size_t lists_bytes(int E, int P) { return size_t(E) * 22 + size_t(P) * 5 + 4; }
static_assert(6 * EP_MAX_TOP_K <= 4 * kTileRows, "the scratch fits a token's row of the sums of y");

// Builds the lists; every block does, from the ids themselves, with one trip
// to memory and four barriers. A token's bit in its expert's mask makes the
// order of the threads irrelevant. All threads of the block call it; the
// caller synchronises before it reads them. sh.active: entries, sh.nmax: the
// most tokens of one, sh.totals: scratch.
template <class Args, class Shared>
static __device__ __forceinline__ void build_lists(const Args &a, const Lists &li, Shared &sh, int tid, int threads,
                                                   int cap)
{
    const int warp = tid >> 5, lane = tid & 31, batches = (a.E + 31) / 32;
    for (int i = tid; i < a.P; i += threads) {
        unsigned int e = ~0u;  // the local id; foreign ones, negative ones too, come out as a.E or more
        float w = 0.0f;
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + i, 4, a.ids, 4LL * a.P))
            e = static_cast<unsigned int>(a.ids[i]) - static_cast<unsigned int>(a.first);
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + i, 4, a.weights, 4LL * a.P))
            w = a.weights[i];
        li.id[i] = static_cast<short>(e < static_cast<unsigned int>(a.E) ? e : -1);
        li.given[i] = w;
    }
    for (int e = tid; e < a.E; e += threads)
        li.mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.P; i += threads)
        if (li.id[i] >= 0)
            atomicOr(&li.mask[li.id[i]], 1ULL << (i / a.K));
    __syncthreads();
    // 32 experts to a warp: entries, pairs and column blocks before each expert, first within the 32. Pairs are in the
    // low and blocks in the high half of a word.
    const auto counts = [&](int n) {
        const int n1 = n > cap ? (n + 1) / 2 : n;
        return n | ((n1 + 7) / 8 + (n - n1 + 7) / 8) << 16;
    };
    for (int b = warp; b < batches; b += threads / 32) {
        const int e = b * 32 + lane, n = e < a.E ? __popcll(li.mask[e]) : 0;
        const unsigned live = __ballot_sync(~0u, n > 0), two = __ballot_sync(~0u, n > cap);
        const int sum = __reduce_add_sync(~0u, counts(n)), most = __reduce_max_sync(~0u, n > cap ? (n + 1) / 2 : n);
        if (lane == 0)
            sh.totals[b] = make_int3(__popc(live) + __popc(two), sum, most);
    }
    __syncthreads();
    for (int b = warp; b < batches; b += threads / 32) {
        int entries = 0, sums = 0, most = 0;
        for (int c = 0; c < b; ++c) {
            entries += sh.totals[c].x;
            sums += sh.totals[c].y;
            most = max(most, sh.totals[c].z);
        }
        const int e = b * 32 + lane, n = e < a.E ? __popcll(li.mask[e]) : 0;
        const unsigned live = __ballot_sync(~0u, n > 0), two = __ballot_sync(~0u, n > cap), before = (1u << lane) - 1;
        if (live) {
            int sum = counts(n);  // inclusive prefix sum over the lanes
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, d);
                if (lane >= d)
                    sum += v;
            }
            if (n > 0) {
                const int at = entries + __popc(live & before) + __popc(two & before), to = sums + sum - counts(n);
                const int off = to & 0xFFFF, blk = to >> 16;
                li.expert[at] = static_cast<unsigned short>(e);
                li.offset[at] = li.start[e] = static_cast<unsigned short>(off);
                li.blocks[at] = static_cast<unsigned short>(blk);
                if (n > cap) {
                    li.expert[at + 1] = static_cast<unsigned short>(e);
                    li.offset[at + 1] = static_cast<unsigned short>(off + (n + 1) / 2);
                    li.blocks[at + 1] = static_cast<unsigned short>(blk + ((n + 1) / 2 + 7) / 8);
                }
            }
        }
        if (b == batches - 1 && lane == 0) {
            entries += sh.totals[b].x;
            sums += sh.totals[b].y;
            li.offset[entries] = static_cast<unsigned short>(sums & 0xFFFF);
            li.blocks[entries] = static_cast<unsigned short>(sums >> 16);
            sh.active = entries;
            sh.nmax = max(most, sh.totals[b].z);
        }
    }
    __syncthreads();
    for (int i = tid; i < a.P; i += threads) {
        const int e = li.id[i];
        if (e < 0)
            continue;
        const int t = i / a.K, first = t * a.K;
        float w = 0.0f;  // an expert named twice by a token counts twice, at its first place
        bool earlier = false;
        for (int k = first; k < first + a.K; ++k)
            if (li.id[k] == e) {
                earlier = earlier || k < i;
                w += li.given[k];
            }
        if (!earlier) {
            const int at = li.start[e] + __popcll(li.mask[e] & ((1ULL << t) - 1));
            li.token[at] = static_cast<unsigned char>(t);
            li.weight[at] = w;
        }
    }
}

// y = 0 where no token chose an expert of this handle.
template <class Args>
static __device__ __forceinline__ void clear_out(const Args &a, int blk, int G, int tid, int threads)
{
    for (long long i = static_cast<long long>(blk) * threads + tid; i < static_cast<long long>(a.T) * a.H;
         i += static_cast<long long>(G) * threads) {
        const long long t = i / a.H;
        uint16_t *const p = reinterpret_cast<uint16_t *>(a.out) + t * a.out_stride + (i - t * a.H);
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
            *p = 0;
    }
}

}  // namespace moe
