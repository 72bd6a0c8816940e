// moe_norm.cu -- the residual's addition, the root-mean-square norm of each
// row, rows in 8 bits with a scale per 128 columns, and the backward pass.
//
//   s = x + residual;  r = 1 / sqrt(mean(s^2) + eps);  y = s r w
//   backward:  n = h r;  g = dy w;  dx = r (g - n mean(g n)) + dh;  dw = sum_t dy n
//
// A row is read once and stays in registers, 8 columns to a unit; a block has
// one row, or several short ones.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kUnit = 8;             // columns that a thread takes at a time
constexpr float kScaled = 0x1p-80f;  // squares of rows whose sum exceeds fp32 are taken of s * this

struct Raw16 {
    uint4 v;
};
struct Raw32 {
    uint4 v[2];
};

// Eight columns as they lie in memory.
template <class T> struct UnitOf {
    using type = Raw16;
};
template <> struct UnitOf<float> {
    using type = Raw32;
};
template <class T> using Unit = typename UnitOf<T>::type;

static __device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

static __device__ __forceinline__ Raw16 load(const Raw16 *p) { return {load16(&p->v)}; }
static __device__ __forceinline__ Raw32 load(const Raw32 *p) { return {{load16(&p->v[0]), load16(&p->v[1])}}; }

template <class T> static __device__ __forceinline__ float2 widen(uint32_t v);
template <> __device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 widen<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

template <class T> static __device__ __forceinline__ uint32_t narrow(float a, float b);
template <> __device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t narrow<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <class T> static __device__ __forceinline__ void widen_unit(const Raw16 &u, float (&f)[kUnit])
{
    const uint32_t w[4] = {u.v.x, u.v.y, u.v.z, u.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = widen<T>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
template <class T> static __device__ __forceinline__ void widen_unit(const Raw32 &u, float (&f)[kUnit])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(u.v[i].x);
        f[4 * i + 1] = __uint_as_float(u.v[i].y);
        f[4 * i + 2] = __uint_as_float(u.v[i].z);
        f[4 * i + 3] = __uint_as_float(u.v[i].w);
    }
}

template <class T> static __device__ __forceinline__ void store_unit(Raw16 *p, const float (&f)[kUnit])
{
    p->v = make_uint4(narrow<T>(f[0], f[1]), narrow<T>(f[2], f[3]), narrow<T>(f[4], f[5]), narrow<T>(f[6], f[7]));
}
template <class T> static __device__ __forceinline__ void store_unit(Raw32 *p, const float (&f)[kUnit])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Unit u of row t, of type T.
template <class T> static __device__ __forceinline__ Unit<T> *unit_at(void *p, long long stride, long long t, int u)
{
    return reinterpret_cast<Unit<T> *>(static_cast<T *>(p) + t * stride) + u;
}
template <class T>
static __device__ __forceinline__ const Unit<T> *unit_at(const void *p, long long stride, long long t, int u)
{
    return reinterpret_cast<const Unit<T> *>(static_cast<const T *>(p) + t * stride) + u;
}

// The norm's weight of unit u: of type T, or fp32. It is read by every row: from L1 where it can be.
template <class T> static __device__ __forceinline__ void load_weight(const void *w, bool fp32, int u, float (&f)[kUnit])
{
    if (sizeof(T) == 4 || fp32) {
        const float4 *const p = static_cast<const float4 *>(w) + 2 * u;
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else if constexpr (sizeof(T) == 2) {
        widen_unit<T>(Raw16{__ldg(static_cast<const uint4 *>(w) + u)}, f);
    }
}

// Sums of N values over the `warps` warps of a row, in the same order in every thread. slots: [N][32] of this row. All
// threads of the block call it.
template <int N> static __device__ __forceinline__ void row_sums(float (&v)[N], float (*slots)[32], int warps, int warp, int lane)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = 16; d; d >>= 1)
            v[i] += __shfl_xor_sync(~0u, v[i], d);
    if (warps == 1)
        return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            slots[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = lane < warps ? slots[i][lane] : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1)
            v[i] += __shfl_xor_sync(~0u, v[i], d);
    }
}

// 1 / sqrt(sum / H + eps); for a sum of squares of finite values that exceeds fp32, from the sum of (s kScaled)^2,
// next to which eps is nothing.
static __device__ __forceinline__ float rstd_of(float sum, int H, float eps)
{
    return 1.0f / sqrtf(sum / static_cast<float>(H) + eps);
}
static __device__ __forceinline__ float rstd_scaled(float sum, int H)
{
    return kScaled / sqrtf(sum / static_cast<float>(H));
}

// blockDim (threads of a row, rows of a block); thread i of a row has its units i, i + blockDim.x, ...: U of them.
template <class T, int U> __global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float slots[kNormRows][2][1][32];
    const int units = a.H / kUnit, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = t < a.T;
    float s[U][kUnit];
    float sum[1] = {0.0f};
    {
        Unit<T> x[U], r[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (live && u < units) {
                x[i] = load(unit_at<T>(a.x, a.x_stride, t, u));
                if (a.residual)
                    r[i] = load(unit_at<T>(a.residual, a.residual_stride, t, u));
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (live && u < units) {
                widen_unit<T>(x[i], s[i]);
                if (a.residual) {
                    float f[kUnit];
                    widen_unit<T>(r[i], f);
#pragma unroll
                    for (int j = 0; j < kUnit; ++j)
                        s[i][j] += f[j];
                }
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    sum[0] = fmaf(s[i][j], s[i][j], sum[0]);
            } else {
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    s[i][j] = 0.0f;
            }
        }
    }
    row_sums<1>(sum, slots[threadIdx.y][0], warps, warp, lane);
    float rstd = rstd_of(sum[0], a.H, a.eps);
    // rare: squares that exceed fp32 (all rows of the block take part, for the barrier)
    if (__syncthreads_or(isinf(sum[0]))) {
        float again[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                again[0] = fmaf(s[i][j] * kScaled, s[i][j] * kScaled, again[0]);
        row_sums<1>(again, slots[threadIdx.y][1], warps, warp, lane);
        if (isinf(sum[0]))
            rstd = rstd_scaled(again[0], a.H);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        const bool mine = live && u < units;
        float y[kUnit];
        uint32_t most = 0;  // of |y|, as bits: NaN is largest
        if (mine) {
            if (a.residual_out && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, unit_at<T>(a.residual_out, a.residual_out_stride, t, u), sizeof(Unit<T>), a.residual_out, sizeof(T) * ((a.T - 1LL) * a.residual_out_stride + a.H)))
                store_unit<T>(unit_at<T>(a.residual_out, a.residual_out_stride, t, u), s[i]);
            float w[kUnit];
            load_weight<T>(a.weight, a.weight_fp32, u, w);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                y[j] = s[i][j] * rstd * w[j];
                most = max(most, __float_as_uint(fabsf(y[j])));
            }
            if (a.out && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, unit_at<T>(a.out, a.out_stride, t, u), sizeof(Unit<T>), a.out, sizeof(T) * ((a.T - 1LL) * a.out_stride + a.H)))
                store_unit<T>(unit_at<T>(a.out, a.out_stride, t, u), y);
        }
        if (a.q) {  // a group is 16 threads' units
#pragma unroll
            for (int d = 8; d; d >>= 1)
                most = max(most, __shfl_xor_sync(~0u, most, d));
            const float scale = most >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                                    : fmaxf(__uint_as_float(most) / 448.0f, 0x1p-126f);
            const float inverse = 1.0f / scale;
            if (mine) {
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(y[4 * j] * inverse, y[4 * j + 1] * inverse), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(y[4 * j + 2] * inverse, y[4 * j + 3] * inverse), __NV_SATFINITE, __NV_E4M3);
                    w[j] = lo | (hi << 16);
                }
                uint2 *const q = reinterpret_cast<uint2 *>(a.q + t * a.H) + u;
                if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, q, 8, a.q, a.T * static_cast<long long>(a.H)))
                    *q = make_uint2(w[0], w[1]);
                float *const to = a.scales + t * a.groups + u / 16;
                if ((u & 15) == 0 &&
                    EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, to, 4, a.scales, 4LL * a.T * a.groups))
                    *to = scale;
            }
        }
    }
}

// One block has rows blockIdx.x + i gridDim.x, and the sums of its rows' parts of dw, per column in one thread.
template <class T, int U> __global__ void __launch_bounds__(1024) back_kernel(const __grid_constant__ NormBackArgs a)
{
    __shared__ float slots[2][2][32];
    __shared__ float slots_again[2][2][32];
    const int units = a.H / kUnit, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    float acc[U][kUnit];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
            acc[i][j] = 0.0f;
    int turn = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        Unit<T> rh[U], rdy[U], rdh[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) {
                rh[i] = load(unit_at<T>(a.h, a.h_stride, t, u));
                rdy[i] = load(unit_at<T>(a.dy, a.dy_stride, t, u));
                if (a.dx && a.dh)
                    rdh[i] = load(unit_at<T>(a.dh, a.dh_stride, t, u));
            }
        }
        float sums[2] = {0.0f, 0.0f};  // of h^2 and of dy w h
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) {
                float h[kUnit], dy[kUnit], w[kUnit];
                widen_unit<T>(rh[i], h);
                widen_unit<T>(rdy[i], dy);
                load_weight<T>(a.weight, a.weight_fp32, u, w);
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    sums[0] = fmaf(h[j], h[j], sums[0]);
                    sums[1] = fmaf(dy[j] * w[j], h[j], sums[1]);
                }
            }
        }
        row_sums<2>(sums, slots[turn], warps, warp, lane);
        float rstd = rstd_of(sums[0], a.H, a.eps), mean = rstd * sums[1] / static_cast<float>(a.H);  // of g n
        if (!isfinite(sums[0]) || !isfinite(sums[1])) {  // squares that exceed fp32; the same in all threads
            float again[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = threadIdx.x + i * blockDim.x;
                if (u < units) {
                    float h[kUnit], dy[kUnit], w[kUnit];
                    widen_unit<T>(rh[i], h);
                    widen_unit<T>(rdy[i], dy);
                    load_weight<T>(a.weight, a.weight_fp32, u, w);
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) {
                        again[0] = fmaf(h[j] * kScaled, h[j] * kScaled, again[0]);
                        again[1] = fmaf(dy[j] * w[j], h[j] * kScaled, again[1]);
                    }
                }
            }
            __syncthreads();
            row_sums<2>(again, slots_again[turn], warps, warp, lane);
            if (isinf(sums[0]))
                rstd = rstd_scaled(again[0], a.H);
            mean = rstd / kScaled * again[1] / static_cast<float>(a.H);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) {
                float h[kUnit], dy[kUnit], w[kUnit], dx[kUnit];
                widen_unit<T>(rh[i], h);
                widen_unit<T>(rdy[i], dy);
                load_weight<T>(a.weight, a.weight_fp32, u, w);
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const float n = h[j] * rstd;
                    acc[i][j] = fmaf(dy[j], n, acc[i][j]);
                    dx[j] = rstd * fmaf(-n, mean, dy[j] * w[j]);
                }
                if (a.dx) {
                    if (a.dh) {
                        float dh[kUnit];
                        widen_unit<T>(rdh[i], dh);
#pragma unroll
                        for (int j = 0; j < kUnit; ++j)
                            dx[j] += dh[j];
                    }
                    if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, unit_at<T>(a.dx, a.dx_stride, t, u), sizeof(Unit<T>), a.dx, sizeof(T) * ((a.T - 1LL) * a.dx_stride + a.H)))
                        store_unit<T>(unit_at<T>(a.dx, a.dx_stride, t, u), dx);
                }
            }
        }
    }
    if (!a.parts)
        return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (u < units)
            store_unit<float>(reinterpret_cast<Raw32 *>(a.parts + static_cast<size_t>(blockIdx.x) * a.H) + u, acc[i]);
    }
}

// dw from the blocks' parts [blocks, H]: 32 columns a block, a warp adds every 32nd block's part, then the warps' sums in turn.
__global__ void __launch_bounds__(1024) parts_kernel(const __grid_constant__ NormBackArgs a, int blocks)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < a.H)
        for (int b = warp; b < blocks; b += 32)
            s += a.parts[static_cast<size_t>(b) * a.H + col];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < a.H) {
        float total = sums[0][lane];
        for (int i = 1; i < 32; ++i)
            total += sums[i][lane];
        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, a.dweight + col, 4, a.dweight, 4LL * a.H))
            a.dweight[col] = total;
    }
}

struct Shape {
    int units, threads, rows;  // units of a thread, threads of a row, rows of a block
};

// Threads of a row: `u` units each, in whole warps. Short rows share a block.
Shape shape_of(int H, int u, bool one_row)
{
    const int units = H / kUnit;
    Shape s;
    s.units = u;
    s.threads = ((units + u - 1) / u + 31) / 32 * 32;
    s.rows = one_row || s.threads >= 128 ? 1 : 128 / s.threads;
    return s;
}

template <class T> cudaError_t launch(const NormArgs &a, const Shape &s, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.T + static_cast<long long>(s.rows) - 1) / s.rows)), block(s.threads, s.rows);
    if (s.units == 1)
        norm_kernel<T, 1><<<grid, block, 0, stream>>>(a);
    else if (s.units == 2)
        norm_kernel<T, 2><<<grid, block, 0, stream>>>(a);
    else
        norm_kernel<T, 4><<<grid, block, 0, stream>>>(a);
    return cudaGetLastError();
}

template <class T> cudaError_t launch_back(const NormBackArgs &a, const Shape &s, int blocks, cudaStream_t stream)
{
    if (s.units == 1)
        back_kernel<T, 1><<<blocks, s.threads, 0, stream>>>(a);
    else
        back_kernel<T, 2><<<blocks, s.threads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    // Few rows: as many threads as there are units, for the shortest way through a row; many: 4 units a thread
    const int least = (a.H / kUnit + 1023) / 1024, u = a.T <= 2 * a.sms ? (least > 1 ? 2 : 1) : 4;
    const Shape s = shape_of(a.H, u, false);
    switch (a.dtype) {
    case EP_DTYPE_BF16: return launch<__nv_bfloat16>(a, s, stream);
    case EP_DTYPE_FP16: return launch<__half>(a, s, stream);
    default: return launch<float>(a, s, stream);
    }
}

int norm_back_blocks(int T, int sms) { return T < 2 * sms ? T : 2 * sms; }

cudaError_t launch_norm_back(const NormBackArgs &a, cudaStream_t stream)
{
    const int blocks = norm_back_blocks(a.T, a.sms);
    cudaError_t ce = cudaSuccess;
    if (blocks > 0) {
        const Shape s = shape_of(a.H, a.H / kUnit > 512 ? 2 : 1, true);
        ce = a.dtype == EP_DTYPE_BF16   ? launch_back<__nv_bfloat16>(a, s, blocks, stream)
             : a.dtype == EP_DTYPE_FP16 ? launch_back<__half>(a, s, blocks, stream)
                                        : launch_back<float>(a, s, blocks, stream);
    }
    if (ce == cudaSuccess && a.dweight) {
        parts_kernel<<<(a.H + 31) / 32, 1024, 0, stream>>>(a, blocks);
        ce = cudaGetLastError();
    }
    return ce;
}

std::vector<const void *> norm_kernels()
{
#define NORM(T)                                                                                             \
    reinterpret_cast<const void *>(norm_kernel<T, 1>), reinterpret_cast<const void *>(norm_kernel<T, 2>),   \
        reinterpret_cast<const void *>(norm_kernel<T, 4>), reinterpret_cast<const void *>(back_kernel<T, 1>), \
        reinterpret_cast<const void *>(back_kernel<T, 2>)
    return {NORM(__nv_bfloat16), NORM(__half), NORM(float), reinterpret_cast<const void *>(parts_kernel)};
#undef NORM
}

}  // namespace moe
