// moe_router.cu -- a token's top-k experts and weights from its hidden row.
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kPerLane = kMaxLocal / 32;

template <typename T> static __device__ __forceinline__ float2 unpack(uint32_t v);
template <> __device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t v)
{
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}
template <> __device__ __forceinline__ float2 unpack<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
}

// One warp per (token, expert).
template <typename T>
__global__ void __launch_bounds__(256) logits_kernel(const __grid_constant__ RouterArgs a)
{
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= a.E)
        return;
    for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
        const uint4 *const x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + t * a.x_stride);
        const uint4 *const w = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.weight) +
                                                              static_cast<size_t>(e) * a.H);
        float s = 0.0f;
        for (int i = lane; i < a.H / 8; i += 32) {
            const uint4 p = x[i], q = w[i];
            const uint32_t pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 f = unpack<T>(pv[c]), g = unpack<T>(qv[c]);
                s = fmaf(f.x, g.x, s);
                s = fmaf(f.y, g.y, s);
            }
        }
        for (int d = 16; d; d >>= 1)
            s += __shfl_xor_sync(~0u, s, d);
        if (lane == 0)
            a.logits[static_cast<size_t>(t) * a.E + e] = s;
    }
}

// Order-preserving image of a float in the unsigned integers; NaN and -infinity give 0 (never chosen).
static __device__ __forceinline__ uint32_t ordered(float v)
{
    if (!(v > -INFINITY))
        return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp: the choice of one token from its logits. Lane l holds experts l, l + 32, ...
static __device__ void choose(const RouterArgs &a, int t, const float *logits, int lane)
{
    float s[kPerLane];
    uint32_t c[kPerLane];
    const int n = (a.E + 31) / 32;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int e = lane + 32 * i;
        s[i] = (i < n && e < a.E) ? logits[e] : -INFINITY;
        top = fmaxf(top, s[i]);
    }
    float inv = 1.0f;
    const bool by_logit = a.scoring == EP_SCORE_SOFTMAX && a.bias == nullptr && a.groups == 1;
    if (a.scoring == EP_SCORE_SOFTMAX) {
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = lane + 32 * i;
            if (i < n && e < a.E) {
                if (by_logit)
                    c[i] = ordered(s[i]);
                s[i] = expf(s[i] - top);
                sum += s[i];
            }
        }
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(~0u, sum, d);
        inv = sum;
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int e = lane + 32 * i;
        if (i < n && e < a.E) {
            s[i] = a.scoring == EP_SCORE_SOFTMAX ? s[i] / inv : 1.0f / (1.0f + expf(-s[i]));
            if (!by_logit)
                c[i] = ordered(a.bias ? s[i] + a.bias[e] : s[i]);
        } else {
            c[i] = 0;
        }
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        uint32_t value = 0;  // of group `lane`
        for (int g = 0; g < a.groups; ++g) {
            uint32_t b1 = 0, b2 = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if (i < n && (lane + 32 * i) / per == g) {
                    b2 = max(b2, min(b1, c[i]));
                    b1 = max(b1, c[i]);
                }
            const uint32_t m1 = __reduce_max_sync(~0u, b1);
            const int owner = __ffs(__ballot_sync(~0u, b1 == m1)) - 1;
            const uint32_t m2 = __reduce_max_sync(~0u, lane == owner ? b2 : b1);
            auto back = [](uint32_t v) {
                return v == 0 ? -INFINITY : __uint_as_float((v & 0x80000000u) ? (v & 0x7FFFFFFFu) : ~v);
            };
            const float sum = per == 1 ? back(m1) : back(m1) + back(m2);
            if (lane == g)
                value = ordered(sum);
        }
        unsigned keep = 0;
        bool open = lane < a.groups;
        for (int k = 0; k < a.top_groups; ++k) {
            const uint32_t m = __reduce_max_sync(~0u, open ? value : 0);
            const unsigned eq = __ballot_sync(~0u, open && value == m);
            const int g = __ffs(eq) - 1;
            keep |= 1u << g;
            if (lane == g)
                open = false;
        }
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i < n && !((keep >> min((lane + 32 * i) / per, 31)) & 1))
                c[i] = 0;
    }
    int id = EP_INVALID_EXPERT_ID;  // of choice `lane`
    float w = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i < n)
                best = max(best, c[i]);
        const uint32_t m = __reduce_max_sync(~0u, best);
        if (m == 0)
            break;  // nothing left to choose
        int at = 0x7FFFFFFF;
        float v = 0.0f;
#pragma unroll
        for (int i = kPerLane - 1; i >= 0; --i)
            if (i < n && c[i] == m) {
                at = lane + 32 * i;
                v = s[i];
            }
        const int e = __reduce_min_sync(~0u, at);
        v = __shfl_sync(~0u, v, e & 31);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (lane + 32 * i == e)
                c[i] = 0;
        if (lane == k) {
            id = e;
            w = v;
        }
    }
    if (a.renormalize) {
        float sum = lane < a.K ? w : 0.0f;
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(~0u, sum, d);
        w = id >= 0 ? w / sum : 0.0f;
    }
    if (lane < a.K) {
        const size_t at = static_cast<size_t>(t) * a.K + lane;
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + at, 4, a.ids, 4LL * a.T * a.K))
            a.ids[at] = id;
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + at, 4, a.weights, 4LL * a.T * a.K))
            a.weights[at] = w * a.scale;
    }
}

__global__ void __launch_bounds__(256) choose_kernel(const __grid_constant__ RouterArgs a)
{
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t < a.T)
        choose(a, t, a.logits + static_cast<size_t>(t) * a.E, threadIdx.x & 31);
}

}  // namespace

size_t router_workspace(const RouterArgs &a) { return static_cast<size_t>(a.T) * a.E * sizeof(float); }

cudaError_t launch_router(const RouterArgs &a, cudaStream_t stream)
{
    const dim3 grid((a.E + 7) / 8, a.T < 65535 ? a.T : 65535);
    if (a.bf16)
        logits_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    else
        logits_kernel<__half><<<grid, 256, 0, stream>>>(a);
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess)
        return ce;
    choose_kernel<<<(a.T + 7) / 8, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t router_binary_version(int *v)
{
    cudaFuncAttributes fa;
    cudaError_t ce = cudaFuncGetAttributes(&fa, choose_kernel);
    if (ce == cudaSuccess)
        *v = fa.binaryVersion;
    return ce;
}

}  // namespace moe
