// moe_ffn.cu -- the products of a gated feed-forward block for many rows, and
// of its gradients.
//
//   h = silu(x W1^T) (x W3^T);  y = h W2^T
//   dh = dy W2;  dg = dh u silu'(g);  du = dh silu(g)
//   dx = dg W1 + du W3;  dW1 = dg^T x;  dW3 = du^T x;  dW2 = dy^T h
//
// Every one is D[features, rows] = A B^T with the features (the columns of the
// result in memory) along the MMA's M and the rows of x along its N, which may
// be any multiple of 16: a ragged number of rows wastes little, and a warp's 32
// lanes store 32 neighbouring columns of a row straight from registers. For the
// weights' gradients the "rows" are the weight's. Operands whose k are not
// contiguous in memory (W2 and W1 | W3 for dh and dx, everything for the
// weights' gradients) are read as MN-major tiles, so nothing is transposed.
//
// What follows a product is in its epilogue, in fp32 from tensor memory: gate
// and up joined (a block's 128 MMA rows are 64 of gate and the same 64 of up),
// or the gradient of h split into those of gate and up.
//
// Two shapes of one kernel:
//  - pairs: two neighbouring blocks multiply together (cta_group::2), 256
//    features x up to 256 rows a tile, persistent, accumulators in two halves of
//    tensor memory, so that one tile's epilogue runs under the next one's MMAs;
//  - splits: for few tiles. A block has 128 features, a cluster of 1 to 8 blocks
//    shares a tile's K. Their sums meet in distributed shared memory, added in
//    the order of K, a share of the rows in each block.
#include <cmath>

#include <cuda_bf16.h>

#include "moe_sched.h"

namespace moe {

namespace {

// Threads that store results: of a pair's block 16 warps, which have the next tile's MMAs to hide under; of a split's 8.
static __host__ __device__ constexpr int storers(bool pair) { return pair ? 512 : 256; }
// Warp 0 copies, warp 1 multiplies, warps from the fourth on store.
static __host__ __device__ constexpr int threads(bool pair) { return 128 + storers(pair); }
constexpr int kMaxStages = 12;
constexpr int kBlockA = 16384;      // 128 features x 64 k
constexpr int kHalfTmem = 256;      // columns of one accumulator
// Shared memory through which a pair's results leave: of four warps, two boxes of 16 rows, one of fp32 or of three results;
// joined, also the halves of gate and up that 8 pairs of warps exchange.
static __host__ __device__ constexpr int box_bytes(int epi) { return epi == kFfnStore ? 8192 : epi == kFfnJoin ? 4096 : 12288; }
static __host__ __device__ constexpr int out_bytes(int epi) { return 4 * box_bytes(epi) + (epi == kFfnJoin ? 8 * 2048 : 0); }
constexpr int kBand = 8;            // row tiles of a band of tiles

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t full_d[2], empty_d[2];
    uint64_t drain;
    uint32_t tmem;
    int abort, issued;
};

// Tensor memory is given out in powers of two from 32 columns on.
static __host__ __device__ __forceinline__ uint32_t tmem_columns(int n)
{
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
}

// silu of g and its derivative, to some 5e-6 of their values (the fast exponential and division; the results are rounded
// to 2^-8). e = exp(-g), bounded for the derivative: sigma is then 1e-35 where it would be less.
static __device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

struct Gate {
    float silu, slope;
    __device__ __forceinline__ explicit Gate(float g)
    {
        const float e = __expf(fminf(-g, 80.0f)), s = __fdividef(1.0f, 1.0f + e);
        silu = g * s;
        slope = s * fmaf(g, e * s, 1.0f);
    }
};

static __device__ __forceinline__ void add4(float4 &a, const float4 &b)
{
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

static __device__ __forceinline__ uint2 pack4(float a, float b, float c, float d)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// Whether a store is inside a call's result (of the checked build; h, saved and dgu are workspace).
template <int EPI> static __device__ __forceinline__ bool inside(const FfnArgs &a, const void *p, int bytes, int size)
{
    return EPI != kFfnStore ||
           EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, bytes, a.out, size * ((a.N - 1LL) * a.out_stride + a.M));
}

// Of a split: what one thread does with the results of four features (col ..) of a row. Feature counts are multiples of 8: all four
// are there, or none.
// WEIGHT: of a weight's gradient, which may be fp32 and is aligned.
template <int EPI, bool WEIGHT> struct Sink {
    const FfnArgs &a;
    const int col;

    struct Kept {
        float4 g, u;
    };

    __device__ __forceinline__ Sink(const FfnArgs &a_, int col_) : a(a_), col(col_) {}

    __device__ __forceinline__ bool live(int t) const { return col < a.M && t < a.N; }

    // split: the kept g and u of row t, ahead of their use
    __device__ __forceinline__ void fetch(int t, Kept &k) const
    {
        if (EPI == kFfnSplit && live(t)) {
            const float *const s = a.saved + 2LL * t * a.M + col;
            k.g = *reinterpret_cast<const float4 *>(s);
            k.u = *reinterpret_cast<const float4 *>(s + a.M);
        }
    }

    // v: the results; joined: of gate, those of up are in k.u
    __device__ __forceinline__ void put(int t, const float4 &v, const Kept &k) const
    {
        if (!live(t))
            return;
        const long long at = t * a.out_stride + col;
        if (WEIGHT && a.fp32) {
            float4 *const p = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
            if (inside<EPI>(a, p, 16, 4)) {
                const float4 o = a.accumulate ? *p : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                *p = a.accumulate ? make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w) : v;
            }
            return;
        }
        uint2 r;
        if (EPI == kFfnStore) {
            r = pack4(v.x, v.y, v.z, v.w);
        } else if (EPI == kFfnJoin) {
            r = pack4(silu(v.x) * k.u.x, silu(v.y) * k.u.y, silu(v.z) * k.u.z, silu(v.w) * k.u.w);
            if (a.saved) {
                float *const s = a.saved + 2LL * t * a.M + col;
                *reinterpret_cast<float4 *>(s) = v;
                *reinterpret_cast<float4 *>(s + a.M) = k.u;
            }
        } else {
            const Gate x(k.g.x), y(k.g.y), z(k.g.z), w(k.g.w);
            __nv_bfloat16 *const d = a.dgu + 2LL * t * a.M + col;
            *reinterpret_cast<uint2 *>(d) = pack4(v.x * k.u.x * x.slope, v.y * k.u.y * y.slope, v.z * k.u.z * z.slope,
                                                  v.w * k.u.w * w.slope);
            *reinterpret_cast<uint2 *>(d + a.M) = pack4(v.x * x.silu, v.y * y.silu, v.z * z.silu, v.w * w.silu);
            r = pack4(x.silu * k.u.x, y.silu * k.u.y, z.silu * k.u.z, w.silu * k.u.w);
        }
        __nv_bfloat16 *const p = static_cast<__nv_bfloat16 *>(a.out) + at;
        if (!inside<EPI>(a, p, 8, 2))
            return;
        if (EPI != kFfnStore || WEIGHT || a.aligned) {
            *reinterpret_cast<uint2 *>(p) = r;
        } else {
            uint16_t *const e = reinterpret_cast<uint16_t *>(p);
            e[0] = r.x & 0xFFFF, e[1] = r.x >> 16, e[2] = r.y & 0xFFFF, e[3] = r.y >> 16;
        }
    }

};

// Tiles in bands of kBand row tiles, feature tiles one after the other within a band: tiles that run at a time share
// operands in L2.
static __device__ __forceinline__ void tile_of(const FfnArgs &a, int i, int &m, int &n)
{
    const int band = i / (kBand * a.m_tiles), first = band * kBand, wide = min(kBand, a.n_tiles - first);
    const int in = i - first * a.m_tiles;
    m = in / wide;
    n = first + in - m * wide;
}

template <int EPI, bool A_MN, bool B_MN, bool PAIR>
__global__ void __launch_bounds__(threads(PAIR), PAIR ? 1 : 2) ffn_kernel(const __grid_constant__ FfnArgs a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const uint32_t dyn0 = smem_u32(dyn), ring = (dyn0 + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int group = PAIR ? 2 : a.split;  // blocks of a cluster
    const int rank = blockIdx.x % group, first = blockIdx.x / group, next = gridDim.x / group;
    const int tiles = a.m_tiles * a.n_tiles, chunks = (a.K + kChunk - 1) / kChunk;
    const int c0 = PAIR ? 0 : static_cast<int>(static_cast<long long>(chunks) * rank / a.split);
    const int c1 = PAIR ? chunks : static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / a.split);
    const int rows_b = PAIR ? a.tile_n / 2 : a.tile_n, blocks_b = (rows_b + 63) / 64;
    const int bytes = kBlockA + (B_MN ? blocks_b * 8192 : rows_b * 128);
    constexpr int kFeatures = EPI == kFfnJoin ? 64 : 128;  // of a block
    constexpr int kEpilogue = storers(PAIR);
    using To = Sink<EPI, A_MN && B_MN>;
    volatile int *const abort = &sh.abort;

    if (tid == 0) {
        sh.abort = sh.issued = 0;
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.full_d[i]), 1);
            mbar_init(smem_u32(&sh.empty_d[i]), (PAIR ? 2 : 1) * kEpilogue / 32);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        mbar_init_fence();
        tma_prefetch_map(&a.ma);
        tma_prefetch_map(&a.mb);
    }
    const uint32_t columns = PAIR ? 2 * kHalfTmem : tmem_columns(a.tile_n);
    if (warp == 1)
        tmem_alloc<PAIR>(smem_u32(&sh.tmem), columns);
    tc_fence_before();
    __syncthreads();
    if (PAIR)
        cluster_sync();  // no copy or arrival reaches a block before its barriers are set
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0 && elect_one()) {
        // ---- copies ----
        auto load = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int x, int y) {
            if (PAIR)
                tma_load_2d_pair(dst, map, in_first_block(full), x, y);
            else
                tma_load_2d(dst, map, full, x, y);
        };
        auto expect = [&](uint32_t full) {
            if (!PAIR || rank == 0)
                mbar_expect(full, PAIR ? 2 * bytes : bytes);
        };
        auto load_a = [&](uint32_t dst, uint32_t full, int m, int k) {
            const int m0 = (PAIR ? 2 * m + rank : m) * kFeatures;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int f = EPI == kFfnJoin ? m0 + j * a.M : m0 + j * 64;
                load(dst + j * 8192, &a.ma, full, A_MN ? f : k, A_MN ? k : f);
            }
        };
        auto load_b = [&](uint32_t dst, uint32_t full, int n, int k) {
            const int n0 = n * a.tile_n + (PAIR ? rank * rows_b : 0);
            if (B_MN) {
                for (int j = 0; j < blocks_b; ++j)
                    load(dst + kBlockA + j * 8192, &a.mb, full, n0 + j * 64, k);
            } else {
                load(dst + kBlockA, &a.mb, full, k, n0);
            }
        };
        int m, n, ahead = 0;  // the ring's first round: weights that are copied before the rows are there
        if (a.early == kFfnWeights && first < tiles) {
            tile_of(a, first, m, n);
            for (; ahead < a.stages && c0 + ahead < c1; ++ahead) {
                expect(smem_u32(&sh.full[ahead]));
                load_a(ring + ahead * bytes, smem_u32(&sh.full[ahead]), m, (c0 + ahead) * kChunk);
            }
        }
        if (a.early != kFfnAll) {
            pdl_wait();
            fence_async_proxy();  // what the kernel before stored from registers is read by copies
        }
        pdl_launch_next();
        Cursor at;
        int issued = 0;
        bool run = true;
        for (int i = first; run && i < tiles; i += next) {
            tile_of(a, i, m, n);
            for (int c = c0; c < c1; ++c) {
                const uint32_t to = ring + at.s * bytes, full = smem_u32(&sh.full[at.s]);
                if (issued >= ahead) {
                    run = mbar_wait(smem_u32(&sh.empty[at.s]), at.parity ^ 1, abort, kWaitEmptyA);
                    if (!run)
                        break;
                    expect(full);
                    load_a(to, full, m, c * kChunk);
                }
                load_b(to, full, n, c * kChunk);
                at.next(a.stages);
                ++issued;
            }
        }
        sh.issued = issued;
    } else if (warp == 1) {
        // ---- matrix instructions, of a pair in its first block ----
        Cursor at, at_d;
        bool run = true;
        const uint32_t idesc =
            idesc_f16(PAIR ? 256 : 128, a.tile_n, 1) | (A_MN ? kIdescAmn : 0u) | (B_MN ? kIdescBmn : 0u);
        for (int i = first; run && i < tiles && (!PAIR || rank == 0); i += next) {
            run = mbar_wait_warp(smem_u32(&sh.empty_d[at_d.s]), at_d.parity ^ 1, abort, kWaitEmptyD);
            const uint32_t d = tmem + at_d.s * kHalfTmem;
            for (int c = c0; run && c < c1; ++c) {
                run = mbar_wait_warp(smem_u32(&sh.full[at.s]), at.parity, abort, kWaitFullA);
                if (!run)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t from = ring + at.s * bytes;
                    const uint64_t da = A_MN ? desc_mn(from) : desc_sw128(from);
                    const uint64_t db = B_MN ? desc_mn(from + kBlockA) : desc_sw128(from + kBlockA);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // 16 k each: 32 bytes of a row, or 16 rows of 128, in 16-byte units
                        const uint64_t qa = da + q * (A_MN ? 128 : 2), qb = db + q * (B_MN ? 128 : 2);
                        if (PAIR)
                            mma_ss_pair(d, qa, qb, idesc, c > c0 || q > 0);
                        else
                            mma_ss(d, qa, qb, idesc, c > c0 || q > 0);
                    }
                    if (PAIR)
                        tc_commit_pair(smem_u32(&sh.empty[at.s]));
                    else
                        tc_commit(smem_u32(&sh.empty[at.s]));
                }
                at.next(a.stages);
            }
            if (elect_one()) {
                if (PAIR)
                    tc_commit_pair(smem_u32(&sh.full_d[at_d.s]));
                else
                    tc_commit(smem_u32(&sh.full_d[at_d.s]));
            }
            at_d.next(2);
        }
        if ((!PAIR || rank == 0) && elect_one()) {
            if (PAIR)
                tc_commit_pair(smem_u32(&sh.drain));
            else
                tc_commit(smem_u32(&sh.drain));
        }
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= 4 && PAIR) {
        // ---- results, under the next tile's products ----
        // A step is 16 rows. Four warps with the four quarters of the features take every fourth step, give each row's
        // features their place in shared memory, and one of them sends it off as a box (out of bounds is cut off by the
        // map). Joined: a warp of quarters 0 and 1 has gate, the one two quarters on up of the same 32 features; they
        // exchange halves, and each joins 8 of the 16 rows.
        Cursor at_d;
        const int quarter = warp & 3, turn = (warp - 4) >> 2, steps = a.tile_n / 16;
        const bool second = EPI == kFfnJoin && quarter >= 2, sender = quarter == 0 && elect_one();
        const int f = (EPI == kFfnJoin ? quarter & 1 : quarter) * 32 + lane;  // of the block's features
        constexpr int kRows = EPI == kFfnJoin ? 8 : 16;                       // of a warp
        const int row0 = second ? 8 : 0;
        uint8_t *const stage = dyn + (ring - dyn0) + a.stages * bytes + turn * box_bytes(EPI);
        float *const exchange = reinterpret_cast<float *>(dyn + (ring - dyn0) + a.stages * bytes + 4 * box_bytes(EPI)) +
                                (turn * 2 + (quarter & 1)) * 512 + lane;  // [gate, up][8][32]
        constexpr bool kWeight = A_MN && B_MN;
        const bool boxes = a.boxes != 0;
        int sent = 0;
        for (int i = first; i < tiles; i += next) {
            int m, n;
            tile_of(a, i, m, n);
            const int m0 = (2 * m + rank) * kFeatures, col = m0 + f, t0 = n * a.tile_n;
            float g[16], u[16];
            auto fetch = [&](int step) {  // the kept g and u, ahead of their use
                if (EPI == kFfnSplit && step < steps) {
                    const float *s = a.saved + 2LL * (t0 + step * 16) * a.M + col;
#pragma unroll
                    for (int r = 0; r < 16; ++r, s += 2LL * a.M)
                        if (col < a.M && t0 + step * 16 + r < a.N) {
                            g[r] = s[0];
                            u[r] = s[a.M];
                        } else {
                            g[r] = u[r] = 0.0f;
                        }
                }
            };
            fetch(turn);
            const bool run = mbar_wait(smem_u32(&sh.full_d[at_d.s]), at_d.parity, abort, kWaitFullD);
            if (!named_all(1, kEpilogue, run))
                break;
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21) + at_d.s * kHalfTmem;
            for (int step = turn; step < steps; step += 4) {
                const int t = t0 + step * 16;
                float v[16];
                tmem_ld16(d + step * 16, v);
                tmem_wait_ld();
                if (EPI == kFfnJoin) {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        exchange[(second ? 256 : 0) + r * 32] = v[second ? r : r + 8];
                    named_sync(6 + turn * 2 + (quarter & 1), 64);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float other = exchange[(second ? 0 : 256) + r * 32];
                        g[r] = second ? other : v[r];
                        u[r] = second ? v[r + 8] : other;
                    }
                    if (a.saved && col < a.M) {
                        float *s = a.saved + 2LL * (t + row0) * a.M + col;
#pragma unroll
                        for (int r = 0; r < 8; ++r, s += 2LL * a.M)
                            if (t + row0 + r < a.N) {
                                s[0] = g[r];
                                s[a.M] = u[r];
                            }
                    }
                }
                if (boxes) {
                    // two boxes of bf16 in turn, of fp32 or of three results one
                    const bool one = EPI == kFfnSplit || (kWeight && a.fp32);
                    uint8_t *const box = stage + (one || (sent & 1) == 0 ? 0 : kFeatures * 32);
                    ++sent;
                    if (sender) {
                        if (one)
                            bulk_wait_read<0>();
                        else
                            bulk_wait_read<1>();
                    }
                    named_sync(2 + turn, 128);
                    if (kWeight && a.fp32) {
                        float *const to = reinterpret_cast<float *>(box) + f;
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            to[r * 128] = v[r];
                    } else {
                        __nv_bfloat16 *const to = reinterpret_cast<__nv_bfloat16 *>(box) + row0 * kFeatures + f;
#pragma unroll
                        for (int r = 0; r < kRows; ++r) {
                            if (EPI == kFfnStore) {
                                to[r * 128] = __float2bfloat16_rn(v[r]);
                            } else if (EPI == kFfnJoin) {
                                to[r * 64] = __float2bfloat16_rn(silu(g[r]) * u[r]);
                            } else {
                                const Gate gate(g[r]);
                                to[r * 128] = __float2bfloat16_rn(gate.silu * u[r]);
                                to[r * 128 + 2048] = __float2bfloat16_rn(v[r] * u[r] * gate.slope);
                                to[r * 128 + 4096] = __float2bfloat16_rn(v[r] * gate.silu);
                            }
                        }
                    }
                    fence_async_shared();
                    named_sync(2 + turn, 128);
                    if (sender && m0 < a.M && t < a.N) {
                        const uint32_t from = smem_u32(box);
                        if (kWeight && a.accumulate)
                            tma_add_2d(&a.mo, from, m0, t);
                        else
                            tma_store_2d(&a.mo, from, m0, t);
                        if (EPI == kFfnSplit) {
                            tma_store_3d(&a.md, from + 4096, m0, t, 0);
                            tma_store_3d(&a.md, from + 8192, m0, t, 1);
                        }
                    }
                    if (sender)
                        bulk_commit();
                } else {  // y or dx with rows that a map does not take (or checked): one by one
                    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + (t + row0) * a.out_stride + col;
#pragma unroll
                    for (int r = 0; r < kRows; ++r, p += a.out_stride)
                        if (col < a.M && t + row0 + r < a.N && inside<EPI>(a, p, 2, 2))
                            *p = __float2bfloat16_rn(v[r]);
                }
                fetch(step + 4);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(in_first_block(smem_u32(&sh.empty_d[at_d.s])));
            at_d.next(2);
        }
        if (sender)
            bulk_wait<0>();
    }
    if (!PAIR) {
        // ---- a split's sums into this block's memory, then a share of the rows from all of the cluster's ----
        float *const sums = reinterpret_cast<float *>(dyn + (ring - dyn0));  // [rows][128 features]
        int m, n;
        tile_of(a, first, m, n);
        if (warp >= 4) {
            const bool run = mbar_wait(smem_u32(&sh.full_d[0]), 0, abort, kWaitFullD);
            if (named_all(1, kEpilogue, run)) {
                tc_fence_after();
                const int quarter = warp & 3;
                const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21);
                float *const to = sums + quarter * 32 + lane;
                for (int j = (warp - 4) / 4 * 16; j < a.tile_n; j += 32) {
                    float v[16];
                    tmem_ld16(d + j, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        to[(j + r) * 128] = v[r];
                }
                tc_fence_before();
            }
        }
        __syncwarp();
        if (a.split > 1)
            cluster_sync();
        else
            __syncthreads();
        if (warp >= 4 && !sh.abort) {
            constexpr int kLanes = kFeatures / 4, kStep = kEpilogue / kLanes, R = EPI == kFfnStore ? 2 : 1;  // lanes of a row, rows at a time
            const int f = lane % kLanes * 4;
            const int lo = a.tile_n * rank / a.split, hi = a.tile_n * (rank + 1) / a.split;
            const uint32_t at = smem_u32(sums) + f * 4;
            const To sink(a, m * kFeatures + f);
            for (int j = lo + (tid - 128) / kLanes; j < hi; j += kStep * R) {
                float4 v[R];
                typename To::Kept k[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (EPI == kFfnJoin)
                        k[r].u = v[r];
                    if (j + r * kStep < hi)
                        sink.fetch(n * a.tile_n + j + r * kStep, k[r]);
                }
                for (int s0 = 0; s0 < a.split; s0 += 4) {
                    float4 x[4][R], y[4][R];
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (s0 + s < a.split) {
                            const uint32_t from = in_block(at, s0 + s);
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                if (j + r * kStep < hi) {
                                    x[s][r] = ld_cluster4(from + (j + r * kStep) * 512);
                                    if (EPI == kFfnJoin)
                                        y[s][r] = ld_cluster4(from + (j + r * kStep) * 512 + 256);
                                }
                        }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (s0 + s < a.split)
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                add4(v[r], x[s][r]);
                                if (EPI == kFfnJoin)
                                    add4(k[r].u, y[s][r]);
                            }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (j + r * kStep < hi)  // the others are another block's
                        sink.put(n * a.tile_n + j + r * kStep, v[r], k[r]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort) {  // copies in flight land before the block's memory is given back
        if (tid == 0) {
            bool landed = true;
            for (int i = max(0, sh.issued - a.stages); (!PAIR || rank == 0) && landed && i < sh.issued; ++i)
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
        tmem_free<PAIR>(tmem, columns);
    if (PAIR || a.split > 1)
        cluster_sync();  // the other blocks' copies, arrivals and reads have come
    if (a.early == kFfnAll && tid == 0)
        pdl_wait();  // what follows this kernel follows the one before it too
}

// Gradients of no rows.
__global__ void __launch_bounds__(256) zero_kernel(uint32_t *p, size_t words)
{
    for (size_t i = blockIdx.x * size_t(256) + threadIdx.x; i < words; i += size_t(gridDim.x) * 256)
        p[i] = 0;
}

using Kernel = void (*)(FfnArgs);

template <bool PAIR> Kernel kernel_of(const FfnProduct &p)
{
    if (p.epilogue == kFfnJoin)
        return ffn_kernel<kFfnJoin, false, false, PAIR>;
    if (p.epilogue == kFfnSplit)
        return ffn_kernel<kFfnSplit, true, false, PAIR>;
    if (!p.a_mn)
        return ffn_kernel<kFfnStore, false, false, PAIR>;
    return p.b_mn ? ffn_kernel<kFfnStore, true, true, PAIR> : ffn_kernel<kFfnStore, true, false, PAIR>;
}

int div_up(int a, int b) { return (a + b - 1) / b; }

int stage_bytes(const FfnProduct &p)
{
    const int rows = p.pair ? p.a.tile_n / 2 : p.a.tile_n;
    return kBlockA + (p.b_mn ? div_up(rows, 64) * 8192 : rows * 128);
}

// Dynamic shared memory of a block that has an SM for itself, and of one that shares it with another.
constexpr int kRoom = kSmemMax - 64 - static_cast<int>(sizeof(Shared));
constexpr int kHalfRoom = (228 * 1024) / 2 - 1024 - 64 - static_cast<int>(sizeof(Shared));
constexpr int kShareRows = 128;  // up to so many rows a tile, a split's blocks can share an SM

}  // namespace

// The plan of least cost, in cycles. A tile's 64 k take 2 cycles a row in the MMAs or 64 bytes a cycle of the copies
// of a block's operands, whichever is more; the weights, or all operands, have to come from DRAM once.
void ffn_plan(FfnProduct *p, int sms)
{
    FfnArgs &a = p->a;
    const int chunks = div_up(a.K, kChunk), features = p->epilogue == kFfnJoin ? 64 : 128;
    const double dram = 2.0 * a.K * (static_cast<double>(a.M) * (p->epilogue == kFfnJoin ? 2 : 1) + a.N) / 3500.0;
    double best = 0.0;
    bool any = false;
    int best_n = 16, best_split = 1;
    bool best_pair = false;
    for (int pair = 0; pair < 2; ++pair)
        for (int n = 16; n <= 256; n += 16) {
            const int n_tiles = div_up(a.N, n);
            if (n > 16 && div_up(a.N, n - 16) == n_tiles)
                continue;  // the same tiles with more waste
            const double tiles = static_cast<double>(n_tiles) * div_up(a.M, features * (pair ? 2 : 1));
            const double mma = 2.0 * n, copy = (kBlockA + 128.0 * (pair ? n / 2 : n)) / 64.0;
            const double chunk = mma > copy ? mma : copy;
            for (int split = 1; split <= (pair ? 1 : 8) && split <= chunks; split *= 2) {
                double cost;
                if (pair) {
                    const double waves = std::ceil(tiles / (sms / 2));
                    cost = waves * (chunks * chunk + 400.0);
                    cost = (cost > dram ? cost : dram) + 3000.0 + 10.0 * n;
                } else {
                    const int resident = n <= kShareRows ? 2 : 1;  // they share the SM's MMAs and copies
                    const double blocks = tiles * split, mine = std::ceil(blocks / sms);
                    cost = mine * div_up(chunks, split) * chunk;
                    cost = (cost > dram ? cost : dram) + std::ceil(blocks / (resident * sms)) * (3000.0 + 16.0 * n);
                }
                if (!any || cost < best) {
                    any = true;
                    best = cost;
                    best_n = n;
                    best_split = split;
                    best_pair = pair != 0;
                }
            }
        }
    a.tile_n = best_n;
    a.split = best_split;
    p->pair = best_pair;
    a.m_tiles = div_up(a.M, features * (best_pair ? 2 : 1));
    a.n_tiles = div_up(a.N, best_n);
    p->box_b = best_pair ? best_n / 2 : best_n;
    // Two blocks of a split on an SM where there are more blocks than SMs
    const bool share = !best_pair && best_n <= kShareRows && static_cast<long long>(a.m_tiles) * a.n_tiles * best_split > sms;
    const int room = share ? kHalfRoom : kRoom - (best_pair ? out_bytes(p->epilogue) : 0), stage = stage_bytes(*p);
    a.stages = (room - 1024) / stage < kMaxStages ? (room - 1024) / stage : kMaxStages;
}

cudaError_t ffn_setup()
{
    cudaError_t ce = cudaSuccess;
    for (const void *f : ffn_kernels())
        if (ce == cudaSuccess && f != reinterpret_cast<const void *>(zero_kernel))
            ce = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    return ce;
}

cudaError_t launch_ffn(const FfnProduct &p, int sms, cudaStream_t stream)
{
    const FfnArgs &a = p.a;
    const int tiles = a.m_tiles * a.n_tiles;
    size_t ring = static_cast<size_t>(a.stages) * stage_bytes(p);
    const size_t sums = static_cast<size_t>(a.tile_n) * 512;  // no more than a stage or two
    if (!p.pair && ring < sums)
        ring = sums;
    cudaLaunchConfig_t cfg = {};
    const int pairs = sms / 2;
    cfg.gridDim = dim3(p.pair ? 2 * (tiles < pairs ? tiles : pairs) : tiles * a.split);
    cfg.blockDim = dim3(threads(p.pair));
    cfg.dynamicSmemBytes = 1024 + ring + (p.pair ? out_bytes(p.epilogue) : 0);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.pair ? 2 : a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, p.pair ? kernel_of<true>(p) : kernel_of<false>(p), a);
}

cudaError_t launch_ffn_zero(void *p, size_t bytes, cudaStream_t stream)
{
    zero_kernel<<<1024, 256, 0, stream>>>(static_cast<uint32_t *>(p), bytes / 4);
    return cudaGetLastError();
}

std::vector<const void *> ffn_kernels()
{
#define FFN(PAIR)                                                                           \
    reinterpret_cast<const void *>(ffn_kernel<kFfnJoin, false, false, PAIR>),               \
        reinterpret_cast<const void *>(ffn_kernel<kFfnSplit, true, false, PAIR>),           \
        reinterpret_cast<const void *>(ffn_kernel<kFfnStore, false, false, PAIR>),          \
        reinterpret_cast<const void *>(ffn_kernel<kFfnStore, true, false, PAIR>),           \
        reinterpret_cast<const void *>(ffn_kernel<kFfnStore, true, true, PAIR>)
    return {FFN(true), FFN(false), reinterpret_cast<const void *>(zero_kernel)};
#undef FFN
}

}  // namespace moe
