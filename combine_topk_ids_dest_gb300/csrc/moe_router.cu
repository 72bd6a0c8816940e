// moe_router.cu -- a token's top-k experts and weights from its hidden row.
//
//   l = x Wg^T (fp32);  s = sigmoid(l) or softmax(l);  choose by s (+ bias)
//
// Two kernels, both from hidden rows to ids and weights:
//
//  - few tokens (up to kFewTokens): latency counts, the router's weight is
//    spread over the SMs. A block takes 16 experts, a slice of the inputs and
//    up to 16 tokens; its warps load MMA fragments straight from global
//    memory (any 16 inputs may be a k-step, so a lane's share of a 32-input
//    step is 16 contiguous bytes). Slices are written as fp32 parts and the
//    block that arrives last for its tokens adds them up, one warp a token.
//  - many tokens: a GEMM of [tokens x hidden] with the whole expert axis as
//    the accumulator's columns, D[128 tokens, E] in tensor memory, so each
//    thread finds all of a token's logits in its lane and no logit is written
//    out. Tiles are as high as one wave of blocks needs, up to 128 tokens.
//    With too few tiles for the SMs the inputs are split over blocks as well;
//    parts go through memory and each block of a tile chooses for its share
//    of the tokens. Otherwise two blocks multiply together, which halves the
//    weight's traffic into and out of shared memory (one block for itself,
//    with the weight multicast, left the MMAs waiting: 60 us for the products
//    below, now 38).
//
// What bounds them: latency for few tokens (one token, 128 experts x 4096: 5.6
// us in a graph, 10 with the host's launch; 128 tokens, 256 experts x 7168,
// inputs split over 16 blocks: 16 us). 16001 tokens x 7168 to 256 experts take
// 56 us, 4.2 TB/s: the products 38, at 35 us for their bytes and 31 for the
// MMAs, then scores 5, buckets 2.5 and eight picks 8, latency and issue of
// dependent comparisons, while no tile is left to multiply meanwhile. The
// tensor pipe is active 52 % of the time, DRAM 50 %.
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kFewTokens = kMaxTokens;
constexpr int kSlice = 256;         // tokens of one launch of the kernel for few
// A tile's scores of up to so many experts fit shared memory. Above, the kernel for few tokens takes slices of 256, one
// after the other: 65 tokens x 7168 to 512 experts 35 us, 256 tokens 88 us, 16001 tokens 5.8 ms, where 384 experts,
// in one launch, take 75 us.
constexpr int kManyExperts = 384;

// Order-preserving image of a float in the unsigned integers; NaN and -infinity give 0 (never chosen).
static __device__ __forceinline__ uint32_t ordered(float v)
{
    if (!(v > -INFINITY))
        return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

static __device__ __forceinline__ float unordered(uint32_t v)
{
    return v == 0 ? -INFINITY : __uint_as_float((v & 0x80000000u) ? (v & 0x7FFFFFFFu) : ~v);
}

static __device__ __forceinline__ bool ranks_by_logit(const RouterArgs &a)
{
    return a.scoring == EP_SCORE_SOFTMAX && a.bias == nullptr && a.groups == 1;
}

// From exp(-|l|), so that the divisor lies in [1, 2] and small scores keep their value down to the subnormal ones
// (1 / (1 + exp(-l)) is 0 from l = -88 on). The quotient is within 2 units of the last place; the correctly rounded
// one has a branch for each score.
static __device__ __forceinline__ float sigmoid(float l)
{
    const float x = expf(-fabsf(l));
    return __fdividef(l < 0.0f ? x : 1.0f, 1.0f + x);
}

static __device__ __forceinline__ void store_choice(const RouterArgs &a, int t, int k, int id, float w)
{
    const size_t at = static_cast<size_t>(t) * a.K + k;
    if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + at, 4, a.ids, 4LL * a.T * a.K))
        a.ids[at] = id;
    if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + at, 4, a.weights, 4LL * a.T * a.K))
        a.weights[at] = w * a.scale;
}

// One warp: the choice of one token from its logits; s[i] of lane l is expert l + 32 i.
template <int N> static __device__ void choose_warp(const RouterArgs &a, int t, float (&s)[N], int lane)
{
    uint32_t c[N];
    const bool by_logit = ranks_by_logit(a);
    if (a.scoring == EP_SCORE_SOFTMAX) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = fmaxf(top, s[i]);
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i < a.E) {
                c[i] = ordered(s[i]);
                s[i] = expf(s[i] - top);
                sum += s[i];
            }
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(~0u, sum, d);
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] = s[i] / sum;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] = sigmoid(s[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E)
            c[i] = 0;
        else if (!by_logit)
            c[i] = ordered(a.bias ? s[i] + a.bias[e] : s[i]);
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        uint32_t value = 0;  // of group `lane`
        if (per == 32) {  // group g is c[g] of the lanes
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t m1 = __reduce_max_sync(~0u, c[i]);
                const int owner = __ffs(__ballot_sync(~0u, c[i] == m1)) - 1;
                const uint32_t m2 = __reduce_max_sync(~0u, lane == owner ? 0 : c[i]);
                if (lane == i)
                    value = ordered(unordered(m1) + unordered(m2));
            }
        }
        for (int g = 0; per != 32 && g < a.groups; ++g) {
            uint32_t b1 = 0, b2 = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = lane + 32 * i;
                if (e >= g * per && e < (g + 1) * per) {
                    b2 = max(b2, min(b1, c[i]));
                    b1 = max(b1, c[i]);
                }
            }
            const uint32_t m1 = __reduce_max_sync(~0u, b1);
            const int owner = __ffs(__ballot_sync(~0u, b1 == m1)) - 1;
            const uint32_t m2 = __reduce_max_sync(~0u, lane == owner ? b2 : b1);
            if (lane == g)
                value = ordered(per == 1 ? unordered(m1) : unordered(m1) + unordered(m2));
        }
        unsigned keep = 0;
        bool open = lane < a.groups;
        for (int k = 0; k < a.top_groups; ++k) {
            const uint32_t m = __reduce_max_sync(~0u, open ? value : 0);
            const int g = __ffs(__ballot_sync(~0u, open && value == m)) - 1;
            keep |= 1u << g;
            if (lane == g)
                open = false;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!((keep >> min((lane + 32 * i) / per, 31)) & 1))
                c[i] = 0;
    }
    int id = EP_INVALID_EXPERT_ID;  // of choice `lane`
    float w = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            best = max(best, c[i]);
        const uint32_t m = __reduce_max_sync(~0u, best);
        if (m == 0)
            break;  // nothing left to choose
        int at = 0x7FFFFFFF;
        float v = 0.0f;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (c[i] == m) {
                at = lane + 32 * i;
                v = s[i];
            }
        const int e = __reduce_min_sync(~0u, at);
        v = __shfl_sync(~0u, v, e & 31);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane + 32 * i == e)
                c[i] = 0;
        if (lane == k) {
            id = e;
            w = v;
        }
    }
    if (a.renormalize) {
        float sum = w;  // lanes without a choice have 0
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(~0u, sum, d);
        w = id >= 0 && sum != 0.0f ? w / sum : w;
    }
    if (lane < a.K)
        store_choice(a, t, lane, id, w);
}

// The same, the logits being sums of `parts` rows of E, `next` apart.
template <int N>
static __device__ void choose_from_parts(const RouterArgs &a, int t, const float *p, size_t next, int parts, int lane)
{
    float l[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        l[i] = lane + 32 * i < a.E ? 0.0f : -INFINITY;
    for (int s = 0; s < parts; s += 4) {
        float v[4][N];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[q][i] = s + q < parts && lane + 32 * i < a.E ? __ldcg(p + (s + q) * next + lane + 32 * i) : 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i)
                l[i] += v[q][i];
    }
    choose_warp<N>(a, t, l, lane);
}

// ---- few tokens --------------------------------------------------------------------

// Sixteen bytes of a row, zeros past its end.
static __device__ __forceinline__ uint4 load_row(const uint16_t *row, int k, int H, bool valid)
{
    return valid && k < H ? __ldg(reinterpret_cast<const uint4 *>(row + k)) : make_uint4(0, 0, 0, 0);
}

// grid (16-expert blocks, input slices, token blocks of 8 NT); 8 NT warps that share the slice's 32-input steps,
// so that the last block has a warp for each token.
template <int NT, int N, bool BF16>
__global__ void __launch_bounds__(NT * 256) few_kernel(const __grid_constant__ RouterArgs a)
{
    constexpr int kWarps = NT * 8;
    __shared__ float red[kWarps][16][NT * 8 + 1];
    __shared__ int last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.z * NT * 8, splits = gridDim.y;
    const int steps = (a.H + 31) / 32, share = splits * kWarps, mine = blockIdx.y * kWarps + warp;
    const int s0 = steps * mine / share, s1 = steps * (mine + 1) / share;
    const uint16_t *const W = static_cast<const uint16_t *>(a.weight), *const X = static_cast<const uint16_t *>(a.x);
    const bool ok0 = e0 + g < a.E, ok1 = e0 + g + 8 < a.E;
    const uint16_t *const w0 = W + static_cast<size_t>(ok0 ? e0 + g : 0) * a.H;
    const uint16_t *const w1 = W + static_cast<size_t>(ok1 ? e0 + g + 8 : 0) * a.H;
    float c[NT][4] = {};
    for (int s = s0; s < s1; s += 4) {
        uint4 p[4], q[4], x[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = (s + i) * 32 + t4 * 8;
            const bool in = s + i < s1;
            p[i] = load_row(w0, k, a.H, in && ok0);
            q[i] = load_row(w1, k, a.H, in && ok1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int t = t0 + nt * 8 + g;
                x[i][nt] = load_row(X + (t < a.T ? t : 0) * a.x_stride, k, a.H, in && t < a.T);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t f0[4] = {p[i].x, q[i].x, p[i].y, q[i].y}, f1[4] = {p[i].z, q[i].z, p[i].w, q[i].w};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816<BF16, true>(c[nt], f0, x[i][nt].x, x[i][nt].y);
                mma_16816<BF16, true>(c[nt], f1, x[i][nt].z, x[i][nt].w);
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[warp][g + (i >> 1) * 8][nt * 8 + t4 * 2 + (i & 1)] = c[nt][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * 16; i += kWarps * 32) {
        const int t = i >> 4, e = i & 15;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += red[w][e][t];
        if (t0 + t < a.T && e0 + e < a.E)
            a.parts[(static_cast<size_t>(blockIdx.y) * a.T + t0 + t) * a.E + e0 + e] = v;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const int blocks = gridDim.x * splits;
        last = add_acq_rel(a.counters + blockIdx.z, 1) == blocks - 1;
        if (last)
            a.counters[blockIdx.z] = 0;  // for the next launch
    }
    __syncthreads();
    if (!last)
        return;
    const int t = t0 + warp;
    if (t < a.T)
        choose_from_parts<N>(a, t, a.parts + static_cast<size_t>(t) * a.E, static_cast<size_t>(a.T) * a.E, splits, lane);
}

// ---- many tokens -------------------------------------------------------------------

constexpr int kScorers = 512;  // threads that score and choose, four to a token
constexpr int kThreads = 128 + kScorers;  // warps: copies, MMA, -, -, then those
constexpr int kMaxStages = 8;
constexpr int kBuckets = 16;
// Scores lie [expert][token], 136 to a row: the choice's lanes, eight tokens times four experts in a row, then read 32
// banks, and the biases of the same place in several buckets of 32 lie in different ones.
constexpr int kScoreStride = 136;
static __host__ __device__ __forceinline__ int bias_at(int e) { return e + (e >> 5); }

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], done, drain;
    uint32_t tmem;
    int abort, issued;
};

// How a tile's experts are bucketed: a pick then looks through one bucket
// only. Groups are the buckets where there are 2 to 16 of them.
struct Buckets {
    int n, size;
    bool groups;
};

static __device__ __forceinline__ Buckets buckets_of(const RouterArgs &a)
{
    const bool groups = a.groups > 1 && a.groups <= kBuckets;
    return {groups ? a.groups : kBuckets, groups ? a.E / a.groups : (a.E + kBuckets - 1) / kBuckets, groups};
}

// The two largest choice values of experts [e0, e1) of a token (score[e * kScoreStride]).
static __device__ __forceinline__ void two_largest(const float *score, const float *bias, int e0, int e1, float &b1, float &b2)
{
    b1 = b2 = -INFINITY;
#pragma unroll 4
    for (int e = e0; e < e1; ++e) {
        const float c = score[e * kScoreStride] + bias[bias_at(e)];
        const float v = c > -INFINITY ? c : -INFINITY;  // NaN is never chosen
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
    }
}

// The groups that take part, as a bit set, from their values[g * kScoreStride].
static __device__ unsigned best_groups(const RouterArgs &a, const float *values)
{
    unsigned keep = 0;
    for (int k = 0; k < a.top_groups; ++k) {
        int best = -1;
        float most = 0.0f;
        for (int g = 0; g < a.groups; ++g) {
            const float v = values[g * kScoreStride];
            if (!((keep >> g) & 1) && (best < 0 || v > most)) {
                best = g;
                most = v;
            }
        }
        keep |= 1u << best;
    }
    return keep;
}

static __device__ __forceinline__ float group_value(float b1, float b2, int per)
{
    const float v = per == 1 ? b1 : b1 + b2;
    return v > -INFINITY ? v : -INFINITY;  // infinities of both signs
}

// Four neighbouring lanes, q = 0 to 3: the choice of one token; the warp is
// converged. score[e * kScoreStride] is expert e's score (its logit where the rank goes
// by logits), most_of[b * kScoreStride] bucket b's largest value and values[b * kScoreStride] a
// group's. A pick takes the bucket with the largest value and looks through it
// for the expert, whose score then becomes NaN, and for the next largest. With
// one thread a token the tile of 128 took longer although it had four warps
// only: 61 against 58 us for the call of 16001. live: the token exists, its
// results are written.
static __device__ void choose_quad(const RouterArgs &a, int t, bool live, float *score, const float *most_of,
                                   const float *values, const float *bias, float top, float sum, int q)
{
    constexpr int kMine = kBuckets / 4, kNone = 0x7FFFFFFF;
    const bool by_logit = ranks_by_logit(a);
    const Buckets bk = buckets_of(a);
    float most[kMine];  // of buckets 4 q .. 4 q + 3
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int b = q * kMine + i;
        most[i] = b < bk.n ? most_of[b * kScoreStride] : -INFINITY;
    }
    if (bk.groups) {  // a group takes part if fewer than top_groups come before it
        float v[kBuckets];
#pragma unroll
        for (int g = 0; g < kBuckets; ++g)
            v[g] = g < bk.n ? values[g * kScoreStride] : -INFINITY;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int b = q * kMine + i;
            const float own = b < bk.n ? values[b * kScoreStride] : -INFINITY;
            int before = 0;
#pragma unroll
            for (int g = 0; g < kBuckets; ++g)
                before += g < bk.n && (v[g] > own || (v[g] == own && g < b)) ? 1 : 0;
            most[i] = before < a.top_groups ? most[i] : -INFINITY;
        }
    }
    const size_t at = static_cast<size_t>(t) * a.K;
    float w[EP_MAX_TOP_K / 4], total = 0.0f;  // of choices q, q + 4, ...
    int count = 0;
    for (int n = 0; n < a.K; ++n) {
        float best = -INFINITY;
        int b = kNone;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (most[i] > best) {
                best = most[i];
                b = q * kMine + i;
            }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            const float v = __shfl_xor_sync(~0u, best, d);
            const int o = __shfl_xor_sync(~0u, b, d);
            const bool take = v > best || (v == best && o < b);
            best = take ? v : best;
            b = take ? o : b;
        }
        const bool any = b != kNone;  // something is left to choose
        float rest = -INFINITY;
        int id = kNone;
        const int end = any ? min((b + 1) * bk.size, a.E) : 0;
        for (int e0 = any ? b * bk.size + q : 0; e0 < end; e0 += 32) {
            float c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c[i] = e0 + 4 * i < end ? score[(e0 + 4 * i) * kScoreStride] + bias[bias_at(e0 + 4 * i)] : -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool hit = id == kNone && c[i] == best;
                id = hit ? e0 + 4 * i : id;
                rest = !hit && c[i] > rest ? c[i] : rest;
            }
        }
        __syncwarp();
        int first = id;
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
            first = min(first, __shfl_xor_sync(~0u, first, d));
        if (id != kNone && id != first)  // as large, but not the lowest index
            rest = best;
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
            rest = fmaxf(rest, __shfl_xor_sync(~0u, rest, d));
        const float x = any ? score[first * kScoreStride] : 0.0f, weight = by_logit && any ? expf(x - top) / sum : x;
        __syncwarp();
        if (any && q == 0)
            score[first * kScoreStride] = __uint_as_float(0x7FC00000u);  // NaN is never chosen
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            most[i] = q * kMine + i == b ? rest : most[i];
        total += weight;
        count += any ? 1 : 0;
        if ((n & 3) == q) {
#pragma unroll
            for (int i = 0; i < EP_MAX_TOP_K / 4; ++i)
                w[i] = i == n >> 2 ? weight : w[i];
            if (live && EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + at + n, 4, a.ids, 4LL * a.T * a.K))
                a.ids[at + n] = any ? first : EP_INVALID_EXPERT_ID;
        }
    }
    if (!a.renormalize || total == 0.0f)  // scores that are all 0 stay so
        total = 1.0f;
#pragma unroll
    for (int i = 0; i < EP_MAX_TOP_K / 4; ++i) {
        const int n = 4 * i + q;
        if (live && n < a.K && EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + at + n, 4, a.weights, 4LL * a.T * a.K))
            a.weights[at + n] = n < count ? w[i] / total * a.scale : 0.0f;
    }
}

// grid (token tiles, input splits). Without splits (PAIR) two blocks make a
// cluster and multiply together: each has its tokens and half of the weight's
// rows of a chunk in shared memory, so the weight is read once for 256 tokens.
// The first block issues, and both blocks' copies report to its barriers. Dynamic shared
// memory: the ring, used again for scores [E][136], 32 rows of bucket and group
// values, and the bias.
template <int N, bool BF16, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) many_kernel(const __grid_constant__ RouterArgs a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const uint32_t dyn0 = smem_u32(dyn), ring = (dyn0 + 1023u) & ~1023u;
    float *const scores = reinterpret_cast<float *>(dyn + (ring - dyn0));
    float *const bias = scores + (a.E + 32) * kScoreStride;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int tile = blockIdx.x, split = blockIdx.y, splits = gridDim.y;
    const int t0 = tile * a.rows, rows = min(a.rows, a.T - t0);
    const int half = router_columns(a.E), E16 = router_all_columns(a.E);  // columns of one MMA, of all
    const int bytes_x = a.rows * 128, bytes_w = E16 * (PAIR ? 64 : 128), stage = 16384 + bytes_w;
    const int chunks = (a.H + kChunk - 1) / kChunk;
    const int c0 = static_cast<int>(static_cast<long long>(chunks) * split / splits);
    const int c1 = static_cast<int>(static_cast<long long>(chunks) * (split + 1) / splits);
    volatile int *const abort = &sh.abort;

    const int rank = PAIR ? tile & 1 : 0;

    if (tid == 0) {
        sh.abort = sh.issued = 0;
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        mbar_init(smem_u32(&sh.done), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        mbar_init_fence();
        tma_prefetch_map(&a.mx);
        tma_prefetch_map(&a.mw);
    }
    if (warp == 1)
        tmem_alloc<PAIR>(smem_u32(&sh.tmem), a.tmem_cols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no copy reaches a block before its barriers are set
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Up to four accumulators along the inputs, added up in fp32: long sums in one lose twice the last bits.
    const int spans = min(4, a.tmem_cols / E16);

    if (warp == 0 && elect_one()) {
        int s = 0, it = 0;
        uint32_t parity = 0;
        for (int c = c0; c < c1; ++c, ++it) {
            if (!mbar_wait(smem_u32(&sh.empty[s]), parity ^ 1, abort, kWaitEmptyA))
                break;
            const uint32_t at = ring + s * stage;
            const int part = E16 / 2;  // the map's box: half of the experts
            if (PAIR) {
                const uint32_t bar = in_first_block(smem_u32(&sh.full[s]));
                if (rank == 0)
                    mbar_expect(smem_u32(&sh.full[s]), 2 * (bytes_x + bytes_w));
                tma_load_2d_pair(at, &a.mx, bar, c * kChunk, t0);
                tma_load_2d_pair(at + 16384, &a.mw, bar, c * kChunk, rank * part);
            } else {
                const uint32_t bar = smem_u32(&sh.full[s]);
                mbar_expect(bar, bytes_x + bytes_w);
                tma_load_2d(at, &a.mx, bar, c * kChunk, t0);
                tma_load_2d(at + 16384, &a.mw, bar, c * kChunk, 0);
                tma_load_2d(at + 16384 + part * 128, &a.mw, bar, c * kChunk, part);
            }
            if (++s == a.stages) {
                s = 0;
                parity ^= 1;
            }
        }
        sh.issued = it;
    } else if (warp == 1) {
        int s = 0;
        uint32_t parity = 0;
        const uint32_t idesc = idesc_f16(PAIR ? 256 : 128, half, BF16);
        int span = 0, next = c0;  // the accumulator in use, and the chunk from which it is another
        uint32_t d = tmem;
        for (int c = c0; c < c1 && rank == 0; ++c) {
            const bool first = c == next;
            if (first) {
                d = tmem + span * E16;
                next = c0 + (c1 - c0) * ++span / spans;
                next = next > c ? next : c + 1;
            }
            if (!mbar_wait_warp(smem_u32(&sh.full[s]), parity, abort, kWaitFullA))
                break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t at = ring + s * stage;
                const uint64_t da = desc_sw128(at), db = desc_sw128(at + 16384);
                for (int e = 0; e < E16; e += half)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (PAIR)
                            mma_ss_pair(d + e, da + 2 * q, db + e * 4 + 2 * q, idesc, !first || q > 0);
                        else
                            mma_ss(d + e, da + 2 * q, db + e * 8 + 2 * q, idesc, !first || q > 0);
                    }
                if (PAIR)
                    tc_commit_pair(smem_u32(&sh.empty[s]));
                else
                    tc_commit(smem_u32(&sh.empty[s]));
            }
            if (++s == a.stages) {
                s = 0;
                parity ^= 1;
            }
        }
        if (rank == 0 && elect_one()) {
            if (PAIR) {
                tc_commit_pair(smem_u32(&sh.done));
                tc_commit_pair(smem_u32(&sh.drain));
            } else {
                tc_commit(smem_u32(&sh.done));
                tc_commit(smem_u32(&sh.drain));
            }
        }
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= 4) {
        // four threads to a token, each with a quarter of the experts' scores
        constexpr int kParts = kScorers / 128;
        const int row = tid & 127, part = (warp - 4) >> 2, wtid = tid - 128;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const int mine8 = (a.E + 8 * kParts - 1) / (8 * kParts) * 8, b0 = min(part * mine8, a.E), b1 = min(b0 + mine8, a.E);
        bool run = mbar_wait_warp(smem_u32(&sh.done), 0, abort, kWaitFullD);
        run = named_all(2, kScorers, run);
        tc_fence_after();
        const int used = min(spans, c1 - c0);
        // A pair's second instruction (more than 256 experts) takes the second half of each block's experts.
        auto logits = [&](int e, float (&v)[8]) {
            float x[8];
            const int all = E16 / 2, in = e % all, col = !PAIR || half == E16 ? e : (2 * in >= half ? half / 2 : 0) + in + (e >= all ? half / 2 : 0);
            tmem_ld8(lanes + col, v);
            for (int i = 1; i < used; ++i) {
                tmem_ld8(lanes + i * E16 + col, x);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += x[j];
            }
            tmem_wait_ld();
        };
        float top = -INFINITY, sum = 0.0f;
        if (run && PAIR) {
            for (int e = b0; e < b1; e += 8) {
                float v[8];
                logits(e, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i < b1) {
                        top = fmaxf(top, v[i]);
                        scores[(e + i) * kScoreStride + row] = a.scoring == EP_SCORE_SIGMOID ? sigmoid(v[i]) : v[i];
                    }
            }
        } else if (run) {  // parts: [tile][split][token][E]
            float *const p = a.parts + ((static_cast<size_t>(tile) * splits + split) * 128 + row) * a.E;
            for (int e = b0; e < b1; e += 8) {
                float v[8];
                logits(e, v);
                if (row >= rows)
                    continue;
                if (a.E % 4 == 0 && e + 8 <= b1) {  // a sector for each thread
                    *reinterpret_cast<float4 *>(p + e) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(p + e + 4) = make_float4(v[4], v[5], v[6], v[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (e + i < b1)
                            p[e + i] = v[i];
                }
            }
            named_sync(1, kScorers);
            if (wtid == 0) {
                add_acq_rel(a.counters + tile, 1);
                run = wait_count(a.counters + tile, splits, abort, kWaitOther);
            }
            run = named_all(2, kScorers, run);
            // this block's tokens of the tile, a warp each
            const int r0 = rows * split / splits, r1 = rows * (split + 1) / splits;
            const float *const from = a.parts + static_cast<size_t>(tile) * splits * 128 * a.E;
            for (int r = r0 + warp - 4; run && r < r1; r += kScorers / 32)
                choose_from_parts<N>(a, t0 + r, from + static_cast<size_t>(r) * a.E, static_cast<size_t>(128) * a.E, splits,
                                     lane);
        }
        if (run && PAIR) {
            for (int e = wtid; e < a.E; e += kScorers)
                bias[bias_at(e)] = a.bias ? a.bias[e] : 0.0f;
            float *const mine = scores + row, *const most = mine + a.E * kScoreStride, *const values = most + kBuckets * kScoreStride;
            float *const xch = bias + bias_at(a.E);  // [parts][128]
            if (a.scoring == EP_SCORE_SOFTMAX) {  // the threads of a token exchange the largest logit and the sum
                xch[part * 128 + row] = top;
                named_sync(1, kScorers);
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    top = fmaxf(top, xch[i * 128 + row]);
                named_sync(1, kScorers);
                const bool keep = ranks_by_logit(a);
#pragma unroll 4
                for (int e = b0; e < b1; ++e) {
                    const float x = expf(mine[e * kScoreStride] - top);
                    sum += x;
                    if (!keep)
                        mine[e * kScoreStride] = x;
                }
                xch[part * 128 + row] = sum;
                named_sync(1, kScorers);
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    sum += xch[i * 128 + row];
                if (!keep) {
#pragma unroll 4
                    for (int e = b0; e < b1; ++e)
                        mine[e * kScoreStride] = mine[e * kScoreStride] / sum;
                }
                named_sync(1, kScorers);
                if (part == 0) {
                    xch[row] = top;
                    xch[128 + row] = sum;
                }
            }
            named_sync(1, kScorers);
            const Buckets bk = buckets_of(a);
            if (a.groups > kBuckets) {  // many small groups: NaN for the experts of those that do not take part
                const int per = a.E / a.groups;
                float b1v, b2v;
                for (int g = part; g < a.groups; g += kParts) {
                    two_largest(mine, bias, g * per, (g + 1) * per, b1v, b2v);
                    most[g * kScoreStride] = group_value(b1v, b2v, per);
                }
                named_sync(1, kScorers);
                const unsigned kept = best_groups(a, most);
                named_sync(1, kScorers);
                for (int g = part; g < a.groups; g += kParts)
                    if (!((kept >> g) & 1))
                        for (int e = g * per; e < (g + 1) * per; ++e)
                            mine[e * kScoreStride] = __uint_as_float(0x7FC00000u);
                named_sync(1, kScorers);
            }
            for (int b = part; b < bk.n; b += kParts) {
                float b1v, b2v;
                two_largest(mine, bias, b * bk.size, min((b + 1) * bk.size, a.E), b1v, b2v);
                most[b * kScoreStride] = b1v;
                if (bk.groups)
                    values[b * kScoreStride] = group_value(b1v, b2v, bk.size);
            }
            named_sync(1, kScorers);
            const int token = wtid >> 2;
            float *const its = scores + token;
            const bool softmax = a.scoring == EP_SCORE_SOFTMAX;
            choose_quad(a, t0 + token, token < rows, its, its + a.E * kScoreStride, its + (a.E + kBuckets) * kScoreStride, bias,
                        softmax ? xch[token] : 0.0f, softmax ? xch[128 + token] : 0.0f, wtid & 3);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort) {
        if (tid == 0) {
            bool landed = true;
            for (int i = max(0, sh.issued - a.stages); rank == 0 && landed && i < sh.issued; ++i)
                landed = mbar_wait(smem_u32(&sh.full[i % a.stages]), (i / a.stages) & 1, nullptr, kWaitOther);
            if (PAIR)  // copies that the first block no longer counts land meanwhile
                for (const long long from = clock64(); clock64() - from < 1000000;) {
                }
            atomicAdd_system(a.err + sh.abort, 1u);
            __threadfence_system();
            atomicAdd_system(a.err, 1u);
        }
        __syncthreads();
    }
    if (warp == 1)
        tmem_free<PAIR>(tmem, a.tmem_cols);
    cluster_sync();  // the other block's copies and arrivals have come
    if (splits > 1 && tid == 0 && add_acq_rel(a.counters + gridDim.x + tile, 1) == splits - 1)
        a.counters[tile] = a.counters[gridDim.x + tile] = 0;  // for the next launch
}

int few_splits(const RouterArgs &a) { return (((a.H + 31) / 32) + 31) / 32; }  // four steps a warp, two of 16 warps

struct ManyPlan {
    int rows, tiles, splits;
};

// Up to 16 splits of the inputs, as far as they leave one wave of blocks with
// tiles of at most 128 tokens (a block then chooses for a few tokens, a warp
// each), and tiles as high as that many blocks need. Tiles come first: 1300
// tokens are 11 of them, 13 splits of which fit 152 SMs; 14, which the SMs
// would hold by the number of tokens, leave blocks for 10.
ManyPlan plan_many(const RouterArgs &a)
{
    ManyPlan p;
    const int chunks = (a.H + kChunk - 1) / kChunk;
    const int full = static_cast<int>((a.T + 127LL) / 128);  // tiles of 128
    p.splits = a.sms / full;
    p.splits = p.splits > 16 ? 16 : p.splits;
    p.splits = p.splits > chunks ? chunks : p.splits;
    if (p.splits <= 1) {
        const long long wave = (full + a.sms - 1) / a.sms * static_cast<long long>(a.sms);
        p.splits = 1;
        p.rows = static_cast<int>((a.T + wave - 1) / wave);
    } else {
        const int tiles = a.sms / p.splits;  // full or more
        p.rows = (a.T + tiles - 1) / tiles;
    }
    p.tiles = static_cast<int>((a.T + p.rows - 1LL) / p.rows);
    return p;
}

}  // namespace

bool router_many(const RouterArgs &a) { return a.T > kFewTokens && a.E <= kManyExperts; }

size_t router_workspace(const RouterArgs &a)
{
    if (a.T <= kFewTokens)
        return 0;
    if (!router_many(a))
        return static_cast<size_t>(few_splits(a)) * (a.T < kSlice ? a.T : kSlice) * a.E * sizeof(float);
    const ManyPlan p = plan_many(a);
    return p.splits == 1 ? 0 : static_cast<size_t>(p.tiles) * p.splits * a.E * 128 * sizeof(float);
}

int router_counters(int sms) { return (2 * sms + kSlice + 63) & ~63; }

size_t router_few_parts(const RouterArgs &a) { return static_cast<size_t>(few_splits(a)) * kFewTokens * a.E * sizeof(float); }


int router_rows(const RouterArgs &a) { return plan_many(a).rows; }

namespace {

using Kernel = void (*)(RouterArgs);

template <int NT> Kernel few_of(const RouterArgs &a)
{
    if (a.E <= 128)
        return a.bf16 ? few_kernel<NT, 4, true> : few_kernel<NT, 4, false>;
    if (a.E <= 256)
        return a.bf16 ? few_kernel<NT, 8, true> : few_kernel<NT, 8, false>;
    return a.bf16 ? few_kernel<NT, 16, true> : few_kernel<NT, 16, false>;
}

template <bool PAIR> Kernel many_of(const RouterArgs &a)
{
    if (a.E <= 128)
        return a.bf16 ? many_kernel<4, true, PAIR> : many_kernel<4, false, PAIR>;
    if (a.E <= 256)
        return a.bf16 ? many_kernel<8, true, PAIR> : many_kernel<8, false, PAIR>;
    return a.bf16 ? many_kernel<12, true, PAIR> : many_kernel<12, false, PAIR>;
}

template <int NT> cudaError_t launch_few(const RouterArgs &a, cudaStream_t stream)
{
    const dim3 grid((a.E + 15) / 16, few_splits(a), (a.T + NT * 8 - 1) / (NT * 8));
    few_of<NT>(a)<<<grid, NT * 256, 0, stream>>>(a);
    return cudaGetLastError();
}

template <bool PAIR> cudaError_t launch_many(RouterArgs a, const ManyPlan &p, cudaStream_t stream)
{
    const int E16 = router_all_columns(a.E), stage = 16384 + E16 * (PAIR ? 64 : 128);
    a.rows = p.rows;
    a.tmem_cols = 512;
    a.stages = (kSmemMax - 2048 - static_cast<int>(sizeof(Shared))) / stage;
    if (a.stages > kMaxStages)
        a.stages = kMaxStages;
    const size_t choice = (static_cast<size_t>(a.E + 32) * kScoreStride + bias_at(a.E) + kScorers) * 4;
    size_t smem = static_cast<size_t>(a.stages) * stage;
    smem = 1024 + (smem > choice ? smem : choice);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(PAIR ? (p.tiles + 1) & ~1 : p.tiles, p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    if (!PAIR) {  // the blocks of a tile wait for one another's parts
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
    } else {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, many_of<PAIR>(a), a);
}

}  // namespace

cudaError_t router_setup(const RouterArgs &a)
{
    cudaError_t ce = cudaSuccess;
    // the experts kernel that usually follows needs all of the SM's memory as shared memory: no change of the split
    for (const Kernel k : {few_of<1>(a), few_of<2>(a)})
        if (ce == cudaSuccess)
            ce = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    for (const Kernel k : {many_of<true>(a), many_of<false>(a)})
        if (ce == cudaSuccess && a.E <= kManyExperts)
            ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSmemMax - 64 - static_cast<int>(sizeof(Shared)));
    return ce;
}

cudaError_t launch_router(const RouterArgs &all, cudaStream_t stream)
{
    if (router_many(all)) {
        const ManyPlan p = plan_many(all);
        return p.splits == 1 ? launch_many<true>(all, p, stream) : launch_many<false>(all, p, stream);
    }
    RouterArgs a = all;
    for (int t = 0; t < all.T; t += kSlice) {
        a.T = all.T - t < kSlice ? all.T - t : kSlice;
        a.x = static_cast<const uint16_t *>(all.x) + t * all.x_stride;
        a.ids = all.ids + static_cast<size_t>(t) * a.K;
        a.weights = all.weights + static_cast<size_t>(t) * a.K;
        const cudaError_t ce = a.T <= 8 ? launch_few<1>(a, stream) : launch_few<2>(a, stream);
        if (ce != cudaSuccess)
            return ce;
    }
    return cudaSuccess;
}

std::vector<const void *> router_kernels()
{
#define FEW(NT, BF16)                                                                                   \
    reinterpret_cast<const void *>(few_kernel<NT, 4, BF16>), reinterpret_cast<const void *>(few_kernel<NT, 8, BF16>), \
        reinterpret_cast<const void *>(few_kernel<NT, 16, BF16>)
#define MANY(BF16, PAIR)                                                                                \
    reinterpret_cast<const void *>(many_kernel<4, BF16, PAIR>), reinterpret_cast<const void *>(many_kernel<8, BF16, PAIR>), \
        reinterpret_cast<const void *>(many_kernel<12, BF16, PAIR>)
    return {FEW(1, true), FEW(1, false), FEW(2, true), FEW(2, false), MANY(true, false), MANY(false, false), MANY(true, true), MANY(false, true)};
#undef FEW
#undef MANY
}

}  // namespace moe
