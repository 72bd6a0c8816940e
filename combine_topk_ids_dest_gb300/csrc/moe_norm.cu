// moe_norm.cu -- the residual's addition, the root-mean-square norm of each
// row, rows in 8 bits with a scale per 128 columns, and the backward pass.
//
//   s = x + residual;  r = 1 / sqrt(mean(s^2) + eps);  y = s r w
//   backward:  n = h r;  g = dy w;  dx = r (g - n mean(g n)) + dh;  dw = sum_t dy n
//
// Both read each row once. Forward, a row stays in registers, 8 columns to a
// unit; a block has one row, or several of one warp. Backward, one persistent
// block an SM takes rows from a ring of shared memory that bulk copies fill:
// with the loads in registers too few were on their way, and the sums of dw need
// the registers (8192 x 4096 60 us, now 47). Its arithmetic is two numbers an
// instruction: near the rate of instructions otherwise (69 us).
//
// What bounds them: DRAM. bf16 rows with residual and 8-bit rows, 16001 x 7168
// (1.04 GB) 153 us, 6.8 TB/s, the rate of a copy (fp32 316, 6.2 TB/s); backward with dh, 8192 x 4096
// (268 MB) 46 to 48 us, 5.7 TB/s, 3 of them the sum of the blocks' parts of dw. Narrow
// rows reach 5.3 to 6 TB/s (16000 x 256 7.0 us). A few rows are launch and one
// trip to memory: one row of 4096 2.0 us, 128 of 7168 3.4 us in a graph. Rows of
// more than 8192 columns spill registers backward (4000 x 16384 142 us, 3.7 TB/s).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kUnit = 8;             // columns that a thread takes at a time
constexpr int kBackThreads = 17 * 32;  // of the backward pass: 16 warps that compute, one that copies
constexpr int kFewUnits = 2, kMostUnits = 4;  // units of a lane: the more up to 16384 columns in 16 warps
constexpr int kBackStages = 32, kBackRing = 200 * 1024;
constexpr float kScaled = 0x1p-80f;  // squares of rows whose sum exceeds fp32 are taken of s * this, of small rows of s / this
constexpr float kLeastMean = 0x1p-80f;  // of squares, with eps: what is below fp32's 2^-149 is nothing next to it

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

// Sums of N values over the `warps` warps of a row, in the same order in every thread. slots: [N][32] of this row.
// Rows of several warps have a block for themselves (barriers by a register's number would cost a block all 16).
template <int N>
static __device__ __forceinline__ void row_sums(float (&v)[N], float (*slots)[32], int warps, int warp, int lane)
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

// Two sums over a team's warps, in the same order in all its threads.
static __device__ __forceinline__ void team_sums(float (&v)[2], float (*slots)[16], int warps, int place, int team, int lane)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        v[0] += __shfl_xor_sync(~0u, v[0], d);
        v[1] += __shfl_xor_sync(~0u, v[1], d);
    }
    if (warps == 1)
        return;
    if (lane < 2)
        slots[lane][place] = lane ? v[1] : v[0];
    named_sync(1 + team, warps * 32);
    // lanes 0 to 15 have the first sum's parts, 16 to 31 the second's
    float x = (lane & 15) < warps ? slots[lane >> 4][lane & 15] : 0.0f;
#pragma unroll
    for (int d = 8; d; d >>= 1)
        x += __shfl_xor_sync(~0u, x, d);
    v[0] = __shfl_sync(~0u, x, 0);
    v[1] = __shfl_sync(~0u, x, 16);
}

// r = 1 / sqrt(sum / H + eps) of a sum of squares. Where that leaves fp32 (an infinite sum of finite values, or so little
// that squares may have vanished), the sum is taken again of (s f)^2, f a power of two: r = f / sqrt(sum / H + eps f^2).
struct Root {
    float mean, rstd;
    __device__ __forceinline__ Root(float sum, int H, float eps) : mean(sum / static_cast<float>(H) + eps), rstd(1.0f / sqrtf(mean)) {}
    // with eps above the one no square counts that vanished; NaN stays NaN
    __device__ __forceinline__ bool left() const { return mean < kLeastMean || isinf(mean); }
    __device__ __forceinline__ float factor() const { return mean < kLeastMean ? 1.0f / kScaled : kScaled; }
    __device__ __forceinline__ void again(float sum, int H, float eps)
    {
        const float f = factor();
        rstd = f / sqrtf(sum / static_cast<float>(H) + eps * f * f);
    }
};

// Two fp32 numbers at a time (one instruction each; both kernels would be near the rate of instructions otherwise).
static __device__ __forceinline__ uint64_t as64(float2 v) { return *reinterpret_cast<uint64_t *>(&v); }
static __device__ __forceinline__ float2 as2(uint64_t v) { return *reinterpret_cast<float2 *>(&v); }
static __device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as64(a)), "l"(as64(b)));
    return as2(d);
}
static __device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as64(a)), "l"(as64(b)), "l"(as64(c)));
    return as2(d);
}
constexpr int kPairs = kUnit / 2;

// Four values in e4m3.
static __device__ __forceinline__ uint32_t codes(float2 a, float2 b)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// blockDim (threads of a row, rows of a block); thread i of a row has its units i, i + blockDim.x, ...: U of them.
template <class T, int U> __global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float slots[kNormRows][2][1][32];
    const int units = a.H / kUnit, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = t < a.T;
    pdl_wait();
    pdl_launch_next();
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
    Root root(sum[0], a.H, a.eps);
    if (root.left()) {  // rare; the same in all threads of the row
        const float f = root.factor();
        float again[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                again[0] = fmaf(s[i][j] * f, s[i][j] * f, again[0]);
        row_sums<1>(again, slots[threadIdx.y][1], warps, warp, lane);
        root.again(again[0], a.H, a.eps);
    }
    const float rstd = root.rstd;
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
            for (int j = 0; j < kUnit; j += 2) {
                const float2 v = mul2(mul2(make_float2(s[i][j], s[i][j + 1]), make_float2(rstd, rstd)), make_float2(w[j], w[j + 1]));
                y[j] = v.x;
                y[j + 1] = v.y;
                most = max(most, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))));
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
            if (mine) {
                // Codes of y / scale. A division for each y takes 16001 x 7168 from 153 to some 165 us: where the products with a
                // little less and a little more than 1 / scale have the same code, so has the quotient. (1 / scale, what is
                // more or less, the product and the quotient itself are each off by 2^-24 at most, together 2^-22.)
                const float inverse = 1.0f / scale, l = inverse * (1.0f - 0x1p-21f), m = inverse * (1.0f + 0x1p-21f);
                const float2 less = make_float2(l, l), more = make_float2(m, m);
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 a2 = make_float2(y[4 * j], y[4 * j + 1]), b2 = make_float2(y[4 * j + 2], y[4 * j + 3]);
                    w[j] = codes(mul2(a2, less), mul2(b2, less));
                    if (w[j] != codes(mul2(a2, more), mul2(b2, more)))
                        w[j] = codes(make_float2(a2.x / scale, a2.y / scale), make_float2(b2.x / scale, b2.y / scale));
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

template <class T> static __device__ __forceinline__ void widen_pairs(const Raw16 &u, float2 (&f)[kPairs])
{
    f[0] = widen<T>(u.v.x), f[1] = widen<T>(u.v.y), f[2] = widen<T>(u.v.z), f[3] = widen<T>(u.v.w);
}
template <class T> static __device__ __forceinline__ void widen_pairs(const Raw32 &u, float2 (&f)[kPairs])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(u.v[i].x), __uint_as_float(u.v[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(u.v[i].z), __uint_as_float(u.v[i].w));
    }
}

// The backward pass: one block an SM. Rows of h, dy and dh are copied into a ring of shared memory, as many as it holds
// on their way at a time, and taken in turn by teams of warps (a.team warps; a lane has up to U units of a row).
// A stage of the ring has a.rows rows that follow one another, block b's are b, b + gridDim.x, ...; team r takes the
// stage's rows r, r + a.teams, ... Where rows are contiguous in memory a stage is one copy per operand. A lane keeps the sum of its columns' parts of
// dw; at the end the teams' sums are added in their order.
//   p = dy h;  dw += p r;  dx = dy w r - h (r^2 mean(g n)) + dh,  mean(g n) = r sum(p w) / H
template <class T, int U> __global__ void __launch_bounds__(kBackThreads, 1) back_kernel(const __grid_constant__ NormBackArgs a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t full[kBackStages], empty[kBackStages];
    __shared__ float slots[16][2][2][16];  // [team][turn][sum][warp]
    __shared__ int abort_, issued_, stopped[16];  // stopped: the stage from which on a team gave up
    uint8_t *const ring = dyn + (128 - (smem_u32(dyn) & 127)) % 128;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int team = warp / a.team, place = warp - team * a.team, units = a.H / kUnit;
    const int groups = (a.T - 1) / a.rows + 1, mine = (groups - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;
    const uint32_t row_bytes = a.H * sizeof(T);
    const bool has_dh = a.dx && a.dh;
    volatile int *const abort = &abort_;

    if (tid == 0) {
        abort_ = issued_ = 0;
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), a.team * a.teams);
        }
        mbar_init_fence();
    } else if (tid >= 32 && tid < 48) {
        stopped[tid - 32] = mine;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_next();

    if (warp == kBackThreads / 32 - 1) {
        // ---- copies ----
        fence_async_proxy();  // what the kernel before stored from registers is read by copies
        int s = 0, i = 0;
        uint32_t parity = 0;
        for (; i < mine; ++i) {
            if (!mbar_wait_warp(smem_u32(&empty[s]), parity ^ 1, abort, kWaitEmptyB))
                break;
            const long long t = (blockIdx.x + static_cast<long long>(i) * gridDim.x) * a.rows;
            const int rows = static_cast<int>(a.T - t < a.rows ? a.T - t : a.rows);
            const uint32_t bar = smem_u32(&full[s]);
            if (lane == 0)
                mbar_expect(bar, row_bytes * rows * (has_dh ? 3 : 2));
            __syncwarp();
            for (int o = 0; o < (has_dh ? 3 : 2); ++o) {
                const T *const from = static_cast<const T *>(o == 0 ? a.h : o == 1 ? a.dy : a.dh);
                const long long stride = o == 0 ? a.h_stride : o == 1 ? a.dy_stride : a.dh_stride;
                const uint32_t to = smem_u32(ring) + s * a.stage + o * a.rows * row_bytes;
                // Of the checked build: rows outside are not copied, and the wait for them runs out.
                const auto there = [&](const T *p, int n) {
                    return EP_IN_BOUNDS(a.chk, epk::kSiteMoeRows, p, row_bytes * n, from, sizeof(T) * ((a.T - 1LL) * stride + a.H));
                };
                if (stride == a.H) {
                    if (lane == o && there(from + t * stride, rows))
                        bulk_load_plain(to, from + t * stride, row_bytes * rows, bar);
                } else {
                    for (int r = lane; r < rows; r += 32)
                        if (there(from + (t + r) * stride, 1))
                            bulk_load_plain(to + r * row_bytes, from + (t + r) * stride, row_bytes, bar);
                }
            }
            if (++s == a.stages) {
                s = 0;
                parity ^= 1;
            }
        }
        if (lane == 0)
            issued_ = i;
    } else if (team < a.teams) {
        // ---- a team's rows ----
        float2 acc[U][kPairs], w[U][kPairs];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int u = (k * a.team + place) * 32 + lane;
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                acc[k][j] = w[k][j] = make_float2(0.0f, 0.0f);
            if (u < units) {
                float f[kUnit];
                load_weight<T>(a.weight, a.weight_fp32, u, f);
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    w[k][j] = make_float2(f[2 * j], f[2 * j + 1]);
            }
        }
        int turn = 0, s = 0;
        uint32_t parity = 0;
        for (int i = 0; i < mine; ++i) {
            bool run = mbar_wait(smem_u32(&full[s]), parity, abort, kWaitFullB);
            run = a.team > 1 ? named_all(1 + team, a.team * 32, run) : __all_sync(~0u, run);
            if (!run) {
                stopped[team] = i;
                break;
            }
            const long long t0 = (blockIdx.x + static_cast<long long>(i) * gridDim.x) * a.rows;
            const int rows = static_cast<int>(a.T - t0 < a.rows ? a.T - t0 : a.rows);
            for (int row = team; row < rows; row += a.teams, turn ^= 1) {
                const uint8_t *const at = ring + s * a.stage + row * row_bytes;
                const uint32_t next = a.rows * row_bytes;  // operand
                const Unit<T> *const h_at = reinterpret_cast<const Unit<T> *>(at) + place * 32 + lane;
                const Unit<T> *const dy_at = reinterpret_cast<const Unit<T> *>(at + next) + place * 32 + lane;
                const Unit<T> *const dh_at = reinterpret_cast<const Unit<T> *>(at + 2 * next) + place * 32 + lane;
                Unit<T> rh[U], rdy[U];
                float2 sums[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};  // of h^2 and of dy w h
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if ((k * a.team + place) * 32 + lane < units) {
                        rh[k] = h_at[k * a.team * 32];
                        rdy[k] = dy_at[k * a.team * 32];
                        float2 h[kPairs], dy[kPairs];
                        widen_pairs<T>(rh[k], h);
                        widen_pairs<T>(rdy[k], dy);
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            sums[0] = fma2(h[j], h[j], sums[0]);
                            sums[1] = fma2(mul2(dy[j], h[j]), w[k][j], sums[1]);
                        }
                    }
                float sum[2] = {sums[0].x + sums[0].y, sums[1].x + sums[1].y};
                team_sums(sum, slots[team][turn], a.team, place, team, lane);
                Root root(sum[0], a.H, a.eps);
                float mean = root.rstd * sum[1] / static_cast<float>(a.H);  // of g n
                if (root.left() || !isfinite(sum[1])) {  // rare; the same in all threads of the team
                    const float f = root.factor();
                    float again[2] = {0.0f, 0.0f};
                    for (int u = place * 32 + lane; u < units; u += a.team * 32) {
                        float h[kUnit], dy[kUnit], wu[kUnit];
                        widen_unit<T>(h_at[u - place * 32 - lane], h);
                        widen_unit<T>(dy_at[u - place * 32 - lane], dy);
                        load_weight<T>(a.weight, a.weight_fp32, u, wu);
#pragma unroll
                        for (int j = 0; j < kUnit; ++j) {
                            again[0] = fmaf(h[j] * f, h[j] * f, again[0]);
                            again[1] = fmaf(dy[j] * wu[j], h[j] * f, again[1]);
                        }
                    }
                    if (a.team > 1)
                        named_sync(1 + team, a.team * 32);  // the slots are read
                    team_sums(again, slots[team][turn], a.team, place, team, lane);
                    if (root.left())
                        root.again(again[0], a.H, a.eps);
                    mean = root.rstd / f * again[1] / static_cast<float>(a.H);
                }
                const float2 r2 = make_float2(root.rstd, root.rstd);
                // h r is n, which may be large where r^2 alone is too small for fp32
                const float2 m2 = make_float2(-mean, -mean);
                const long long t = t0 + row;
                Unit<T> *const to = a.dx ? unit_at<T>(a.dx, a.dx_stride, t, place * 32 + lane) : nullptr;
#pragma unroll
                for (int k = 0; k < U; ++k)
                    if ((k * a.team + place) * 32 + lane < units) {
                        float2 h[kPairs], dy[kPairs], dx[kPairs];
                        widen_pairs<T>(rh[k], h);
                        widen_pairs<T>(rdy[k], dy);
                        if (has_dh) {
                            widen_pairs<T>(dh_at[k * a.team * 32], dx);
                        } else {
#pragma unroll
                            for (int j = 0; j < kPairs; ++j)
                                dx[j] = make_float2(0.0f, 0.0f);
                        }
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            const float2 n = mul2(h[j], r2);
                            acc[k][j] = fma2(dy[j], n, acc[k][j]);
                            dx[j] = fma2(fma2(n, m2, mul2(dy[j], w[k][j])), r2, dx[j]);
                        }
                        if (to && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, to + k * a.team * 32, sizeof(Unit<T>), a.dx, sizeof(T) * ((a.T - 1LL) * a.dx_stride + a.H))) {
                            const float f[kUnit] = {dx[0].x, dx[0].y, dx[1].x, dx[1].y, dx[2].x, dx[2].y, dx[3].x, dx[3].y};
                            store_unit<T>(to + k * a.team * 32, f);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&empty[s]));
            if (++s == a.stages) {
                s = 0;
                parity ^= 1;
            }
        }
        if (a.parts) {  // the teams' sums, one after the other, where the ring was
            float *const sums = reinterpret_cast<float *>(ring) + static_cast<size_t>(team) * a.H;
            named_sync(15, a.teams * a.team * 32);  // all rows are read (or given up)
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int u = (k * a.team + place) * 32 + lane;
                if (u < units) {
                    const float f[kUnit] = {acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y,
                                            acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y};
                    store_unit<float>(reinterpret_cast<Raw32 *>(sums) + u, f);
                }
            }
            named_sync(15, a.teams * a.team * 32);
            for (int c = tid; c < a.H; c += a.teams * a.team * 32) {
                float total = *abort ? __uint_as_float(0x7FC00000u) : 0.0f;
                for (int r = 0; r < a.teams; ++r)
                    total += reinterpret_cast<float *>(ring)[static_cast<size_t>(r) * a.H + c];
                a.parts[static_cast<size_t>(blockIdx.x) * a.H + c] = total;
            }
        }
    }
    __syncthreads();
    if (abort_) {
        // rows of dx that were given up are NaN: there is no handle that could report it
        for (int r = 0; a.dx && r < a.teams; ++r)
            for (int i = stopped[r]; i < mine; ++i) {
                const long long t0 = (blockIdx.x + static_cast<long long>(i) * gridDim.x) * a.rows;
                for (long long t = t0 + r; t < t0 + a.rows && t < a.T; t += a.teams)
                    for (int u = tid; u < units; u += kBackThreads) {
                        const float f[kUnit] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
                        Unit<T> *const to = unit_at<T>(a.dx, a.dx_stride, t, u);
                        if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, to, sizeof(Unit<T>), a.dx, sizeof(T) * ((a.T - 1LL) * a.dx_stride + a.H)))
                            store_unit<T>(to, f);
                    }
            }
        if (tid == 0)  // copies in flight land before the block's memory is given back
            for (int i = max(0, issued_ - a.stages); i < issued_; ++i)
                mbar_wait(smem_u32(&full[i % a.stages]), (i / a.stages) & 1, nullptr, kWaitOther);
    }
}

// dw from the blocks' parts [blocks, H]: 32 columns a block, a warp adds every 32nd block's part, then the warps' sums in turn.
__global__ void __launch_bounds__(1024) parts_kernel(const __grid_constant__ NormBackArgs a, int blocks)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    pdl_wait();
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

// Threads of a row: `u` units each, in whole warps. Rows of one warp share a block.
Shape shape_of(int H, int u)
{
    const int units = H / kUnit;
    Shape s;
    s.units = u;
    s.threads = ((units + u - 1) / u + 31) / 32 * 32;
    s.rows = s.threads == 32 ? kNormRows : 1;
    return s;
}

// A launch whose blocks may start while the kernel before it ends; they wait for its end before they read anything.
template <class... Args, class... Given>
cudaError_t launch_early(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const Given &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T> cudaError_t launch(const NormArgs &a, const Shape &s, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.T + static_cast<long long>(s.rows) - 1) / s.rows)), block(s.threads, s.rows);
    if constexpr (sizeof(T) == 2)
        if (s.units == 4)
            return launch_early(norm_kernel<T, 4>, grid, block, 0, stream, a);
    return launch_early(s.units == 1 ? norm_kernel<T, 1> : norm_kernel<T, 2>, grid, block, 0, stream, a);
}

template <class T> cudaError_t launch_back(NormBackArgs a, int *blocks, cudaStream_t stream)
{
    const int row = a.H * static_cast<int>(sizeof(T)), copies = a.dx && a.dh ? 3 : 2;
    const int lane_units = a.H > kFewUnits * 16 * 32 * kUnit ? kMostUnits : kFewUnits;
    a.team = (a.H / kUnit + 32 * lane_units - 1) / (32 * lane_units);
    a.teams = (kBackThreads / 32 - 1) / a.team;
    // as many rows to a stage as there are teams, unless that leaves blocks without any
    a.rows = (a.T - 1) / a.sms + 1 < a.teams ? (a.T - 1) / a.sms + 1 : a.teams;
    a.stage = (copies * row * a.rows + 127) & ~127;
    a.stages = kBackRing / a.stage < kBackStages ? kBackRing / a.stage : kBackStages;
    const int groups = (a.T - 1) / a.rows + 1;
    *blocks = groups < a.sms ? groups : a.sms;
    const int ring = a.stages * a.stage, sums = a.teams * a.H * 4;  // sums: 64 KB at most
    return launch_early(lane_units == kFewUnits ? back_kernel<T, kFewUnits> : back_kernel<T, kMostUnits>, dim3(*blocks), dim3(kBackThreads), 128 + (ring > sums ? ring : sums), stream, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    // Few rows: as many threads as there are units, for the shortest way through a row. Many: units of a thread that
    // keep a row's loads on their way at once and its warps few (bf16, 8-bit rows too: 16000 x 256 6.9, 8.3, 12.1 us
    // with 1, 2, 4; 8000 x 2048 27.4, 24.6, 25.5; 16001 x 7168 290, 182, 153; fp32 with 4 does not fit the registers)
    const int units = a.H / kUnit;
    const int u = a.T <= 2 * a.sms ? (units > 1024 ? 2 : 1) : units <= 32 ? 1 : units <= 256 || a.dtype == EP_DTYPE_FP32 ? 2 : 4;
    const Shape s = shape_of(a.H, u);
    switch (a.dtype) {
    case EP_DTYPE_BF16: return launch<__nv_bfloat16>(a, s, stream);
    case EP_DTYPE_FP16: return launch<__half>(a, s, stream);
    default: return launch<float>(a, s, stream);
    }
}

int norm_back_blocks(int T, int sms) { return T < sms ? T : sms; }  // at most

cudaError_t launch_norm_back(const NormBackArgs &a, cudaStream_t stream)
{
    int blocks = norm_back_blocks(a.T, a.sms);
    cudaError_t ce = cudaSuccess;
    if (blocks > 0) {
        ce = a.dtype == EP_DTYPE_BF16   ? launch_back<__nv_bfloat16>(a, &blocks, stream)
             : a.dtype == EP_DTYPE_FP16 ? launch_back<__half>(a, &blocks, stream)
                                        : launch_back<float>(a, &blocks, stream);
    }
    if (ce == cudaSuccess && a.dweight) {
        ce = launch_early(parts_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, stream, a, blocks);
    }
    return ce;
}

// On the current device: every kernel is loaded (the first call may be captured), the backward ones get their shared memory.
cudaError_t norm_setup()
{
    cudaError_t ce = cudaSuccess;
    cudaFuncAttributes attr;
    for (const void *k : norm_kernels())
        if (ce == cudaSuccess)
            ce = cudaFuncGetAttributes(&attr, k);
    for (const auto k : {back_kernel<__nv_bfloat16, kFewUnits>, back_kernel<__half, kFewUnits>, back_kernel<float, kFewUnits>,
                         back_kernel<__nv_bfloat16, kMostUnits>, back_kernel<__half, kMostUnits>, back_kernel<float, kMostUnits>})
        if (ce == cudaSuccess)
            ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBackRing + 128);
    return ce;
}

std::vector<const void *> norm_kernels()
{
#define NORM(T)                                                                                           \
    reinterpret_cast<const void *>(norm_kernel<T, 1>), reinterpret_cast<const void *>(norm_kernel<T, 2>), \
        reinterpret_cast<const void *>(back_kernel<T, kFewUnits>), reinterpret_cast<const void *>(back_kernel<T, kMostUnits>)
    return {NORM(__nv_bfloat16), NORM(__half), NORM(float), reinterpret_cast<const void *>(norm_kernel<__nv_bfloat16, 4>),
            reinterpret_cast<const void *>(norm_kernel<__half, 4>), reinterpret_cast<const void *>(parts_kernel)};
#undef NORM
}

}  // namespace moe
