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

// Slot (first or last share) in which block b keeps its part of the tile that begins at unit `begin`.
static __device__ __forceinline__ int part_slot(int total, int b, int G, int begin)
{
    return 2 * b + (begin <= share_begin(total, b, G) ? 0 : 1);
}

// Two bf16 values whose sum carries 16 bits of v's mantissa (v itself where it is not finite).
static __device__ __forceinline__ void split(float v, __nv_bfloat16 &hi, __nv_bfloat16 &lo)
{
    hi = __float2bfloat16_rn(v);
    const float r = v - __bfloat162float(hi);
    lo = __float2bfloat16_rn(isfinite(r) ? r : 0.0f);
}

static __device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// Lists of the chosen experts, in dynamic shared memory.
struct Lists {
    unsigned long long *mask;  // [E] tokens of each expert
    float *weight;             // [P] routing weight of each (expert, token) pair
    unsigned short *expert;    // [E] active experts, ascending
    unsigned short *offset;    // [E + 1] their first pair
    unsigned char *token;      // [P] tokens, ascending per expert

    __device__ __forceinline__ Lists(void *at, int E, int P)
    {
        mask = static_cast<unsigned long long *>(at);
        weight = reinterpret_cast<float *>(mask + E);
        expert = reinterpret_cast<unsigned short *>(weight + P);
        offset = expert + E;
        token = reinterpret_cast<unsigned char *>(offset + E + 1);
    }
    __device__ __forceinline__ int count(int i) const { return offset[i + 1] - offset[i]; }
};

static inline size_t lists_bytes(int E, int P) { return size_t(E) * 12 + size_t(P) * 5 + 2; }

// Builds the lists; every block does, from the ids themselves. A token's bit
// in its expert's mask makes the order of the threads irrelevant. All
// threads of the block call it; the caller synchronises before the lists are
// read (active and nmax, the most tokens of one expert, before that too).
template <class Args, class Shared>
static __device__ __forceinline__ void build_lists(const Args &a, const Lists &li, Shared &sh, int tid, int threads)
{
    for (int e = tid; e < a.E; e += threads)
        li.mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.P; i += threads) {
        if (!EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + i, 4, a.ids, 4LL * a.P))
            continue;
        const int e = a.ids[i] - a.first;
        if (e >= 0 && e < a.E)
            atomicOr(&li.mask[e], 1ULL << (i / a.K));
    }
    __syncthreads();
    if (tid < 32) {
        const int lane = tid;
        int n_active = 0, n_pairs = 0, nmax = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < a.E ? __popcll(li.mask[e]) : 0;
            const unsigned live = __ballot_sync(~0u, n > 0);
            if (live == 0)
                continue;
            int sum = n;  // inclusive prefix sum over the lanes
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, d);
                if (lane >= d)
                    sum += v;
            }
            if (n > 0) {
                const int at = n_active + __popc(live & ((1u << lane) - 1));
                li.expert[at] = static_cast<unsigned short>(e);
                li.offset[at] = static_cast<unsigned short>(n_pairs + sum - n);
            }
            n_active += __popc(live);
            n_pairs += __shfl_sync(~0u, sum, 31);
            nmax = max(nmax, __reduce_max_sync(~0u, n));
        }
        if (lane == 0) {
            li.offset[n_active] = static_cast<unsigned short>(n_pairs);
            sh.active = n_active;
            sh.nmax = nmax;
        }
    }
    __syncthreads();
    for (int i = tid; i < sh.active; i += threads) {
        const int e = li.expert[i];
        int at = li.offset[i];
        for (unsigned long long m = li.mask[e]; m; m &= m - 1, ++at) {
            const int t = __ffsll(static_cast<long long>(m)) - 1;
            float w = 0.0f;  // an expert named twice by a token counts twice
            for (int k = 0; k < a.K; ++k)
                if (a.ids[t * a.K + k] - a.first == e &&
                    EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + t * a.K + k, 4, a.weights, 4LL * a.P))
                    w += a.weights[t * a.K + k];
            li.token[at] = static_cast<unsigned char>(t);
            li.weight[at] = w;
        }
    }
}

// Waits until every tile of the first product is announced; then orders TMA
// reads of h after that.
template <class Args>
static __device__ __forceinline__ bool wait_products(const Args &a, int tiles, volatile int *abort)
{
    const unsigned long long t0 = now_ns();
    while (ld_acquire(a.done) < tiles) {
        if (*abort)
            return false;
        if (now_ns() - t0 > kWaitNs) {
            *abort = kWaitDone;
            return false;
        }
    }
    fence_async_proxy();
    return true;
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
