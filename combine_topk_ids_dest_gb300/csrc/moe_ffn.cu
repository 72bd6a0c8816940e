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
#include <cuda_bf16.h>

#include "moe_sched.h"

namespace moe {

namespace {

constexpr int kThreads = 384;       // warp 0 copies, warp 1 multiplies, warps 4 to 11 store
constexpr int kEpilogue = 256;
constexpr int kMaxStages = 12;
constexpr int kBlockA = 16384;      // 128 features x 64 k
constexpr int kHalfTmem = 256;      // columns of one accumulator
constexpr int kExchange = 4 * 2 * 2 * 1024;  // gate and up: [pair of warps][turn][which][8 rows][32 lanes] floats
constexpr int kBand = 8;            // row tiles of a band of tiles

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t full_d[2], empty_d[2];
    uint64_t drain;
    uint32_t tmem;
    int abort, issued;
};

static __device__ __forceinline__ void tmem_ld8_wait(uint32_t addr, float (&v)[8])
{
    tmem_ld8(addr, v);
    tmem_wait_ld();
}

// silu and its derivative times what reaches them. e = exp(-g), bounded: sigma is then 1e-35 where it would be less.
struct Gate {
    float silu, slope;
    __device__ __forceinline__ explicit Gate(float g)
    {
        const float e = expf(fminf(-g, 80.0f)), s = 1.0f / (1.0f + e);
        silu = g * s;
        slope = s * fmaf(g, e * s, 1.0f);
    }
};

// What one thread does with the results of one feature for successive rows.
template <int EPI> struct Sink {
    const FfnArgs &a;
    const int col;
    __device__ __forceinline__ Sink(const FfnArgs &a_, int col_) : a(a_), col(col_) {}

    // n results v[0..n) (joined: of gate, with those of up in w) for rows t, t + step, ...
    template <int R> __device__ __forceinline__ void put(int t, int step, const float (&v)[R], const float (&w)[R])
    {
        if (col >= a.M)
            return;
        if (EPI == kFfnStore) {
            if (a.fp32) {
                float *p = static_cast<float *>(a.out) + static_cast<long long>(t) * a.out_stride + col;
#pragma unroll
                for (int i = 0; i < R; ++i, p += step * a.out_stride)
                    if (t + i * step < a.N && inside(p, 4))
                        *p = a.accumulate ? *p + v[i] : v[i];
            } else {
                __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + static_cast<long long>(t) * a.out_stride + col;
#pragma unroll
                for (int i = 0; i < R; ++i, p += step * a.out_stride)
                    if (t + i * step < a.N && inside(p, 2))
                        *p = __float2bfloat16_rn(v[i]);
            }
        } else if (EPI == kFfnJoin) {
            __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + static_cast<long long>(t) * a.out_stride + col;
            float *s = a.saved + 2LL * t * a.M + col;
#pragma unroll
            for (int i = 0; i < R; ++i, p += step * a.out_stride, s += 2LL * step * a.M)
                if (t + i * step < a.N) {
                    *p = __float2bfloat16_rn(swiglu(v[i], w[i]));
                    if (a.saved) {
                        s[0] = v[i];
                        s[a.M] = w[i];
                    }
                }
        } else {
            __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + static_cast<long long>(t) * a.out_stride + col;
            __nv_bfloat16 *d = a.dgu + 2LL * t * a.M + col;
            const float *s = a.saved + 2LL * t * a.M + col;
            float g[R], u[R];
#pragma unroll
            for (int i = 0; i < R; ++i, s += 2LL * step * a.M) {
                const bool live = t + i * step < a.N;
                g[i] = live ? s[0] : 0.0f;
                u[i] = live ? s[a.M] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < R; ++i, p += step * a.out_stride, d += 2LL * step * a.M)
                if (t + i * step < a.N) {
                    const Gate gate(g[i]);
                    d[0] = __float2bfloat16_rn(v[i] * u[i] * gate.slope);
                    d[a.M] = __float2bfloat16_rn(v[i] * gate.silu);
                    *p = __float2bfloat16_rn(swiglu(g[i], u[i]));
                }
        }
    }
    __device__ __forceinline__ bool inside(const void *p, int bytes) const
    {
        return EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, bytes, a.out, bytes * ((a.N - 1LL) * a.out_stride + a.M));
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
__global__ void __launch_bounds__(kThreads, 1) ffn_kernel(const __grid_constant__ FfnArgs a)
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
    if (warp == 1)
        tmem_alloc<PAIR>(smem_u32(&sh.tmem), 2 * kHalfTmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no copy or arrival reaches a block before its barriers are set
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0 && elect_one()) {
        // ---- copies ----
        Cursor at;
        int issued = 0;
        bool run = true;
        for (int i = first; run && i < tiles; i += next) {
            int m, n;
            tile_of(a, i, m, n);
            const int m0 = (PAIR ? 2 * m + rank : m) * kFeatures, n0 = n * a.tile_n + (PAIR ? rank * rows_b : 0);
            for (int c = c0; c < c1; ++c) {
                run = mbar_wait(smem_u32(&sh.empty[at.s]), at.parity ^ 1, abort, kWaitEmptyA);
                if (!run)
                    break;
                const uint32_t to = ring + at.s * bytes, mine = smem_u32(&sh.full[at.s]);
                const uint32_t bar = PAIR ? in_first_block(mine) : mine;
                if (!PAIR || rank == 0)
                    mbar_expect(mine, PAIR ? 2 * bytes : bytes);
                auto load = [&](uint32_t dst, const CUtensorMap *map, int x, int y) {
                    if (PAIR)
                        tma_load_2d_pair(dst, map, bar, x, y);
                    else
                        tma_load_2d(dst, map, bar, x, y);
                };
                const int k = c * kChunk;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int f = EPI == kFfnJoin ? m0 + j * a.M : m0 + j * 64;
                    load(to + j * 8192, &a.ma, A_MN ? f : k, A_MN ? k : f);
                }
                if (B_MN) {
                    for (int j = 0; j < blocks_b; ++j)
                        load(to + kBlockA + j * 8192, &a.mb, n0 + j * 64, k);
                } else {
                    load(to + kBlockA, &a.mb, k, n0);
                }
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
        Cursor at_d;
        const int quarter = warp & 3, half = (warp - 4) >> 2, span = a.tile_n / 2;  // two warps share the lanes' rows
        float *const exchange = reinterpret_cast<float *>(dyn + (ring - dyn0) + a.stages * bytes);
        for (int i = first; i < tiles; i += next) {
            const bool run = mbar_wait(smem_u32(&sh.full_d[at_d.s]), at_d.parity, abort, kWaitFullD);
            if (!named_all(1, kEpilogue, run))
                break;
            tc_fence_after();
            int m, n;
            tile_of(a, i, m, n);
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21) + at_d.s * kHalfTmem + half * span;
            const int t0 = n * a.tile_n + half * span, m0 = (2 * m + rank) * kFeatures;
            if (EPI == kFfnJoin) {
                // A warp has gate (quarters 0, 1) or up (2, 3) of 32 features for the same rows as another has the
                // other: the first joins them for the even steps of 8 rows, the second for the odd ones.
                const bool up = quarter >= 2;
                const int pair = half * 2 + (quarter & 1);
                Sink<EPI> sink(a, m0 + (quarter & 1) * 32 + lane);
                for (int j = 0, turn = 0; j < span; j += 16, turn ^= 1) {
                    float even[8], odd[8], got[8];
                    tmem_ld8(d + j, even);
                    if (j + 8 < span)
                        tmem_ld8(d + j + 8, odd);
                    tmem_wait_ld();
                    float *const slot = exchange + ((pair * 2 + turn) * 2) * 256 + lane;
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        slot[(up ? 256 : 0) + r * 32] = up ? even[r] : odd[r];
                    named_sync(2 + pair, 64);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        got[r] = slot[(up ? 0 : 256) + r * 32];
                    if (!up)
                        sink.put(t0 + j, 1, even, got);
                    else if (j + 8 < span)
                        sink.put(t0 + j + 8, 1, got, odd);
                }
            } else {
                Sink<EPI> sink(a, m0 + quarter * 32 + lane);
                for (int j = 0; j < span; j += 8) {
                    float v[8];
                    tmem_ld8_wait(d + j, v);
                    sink.put(t0 + j, 1, v, v);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(in_first_block(smem_u32(&sh.empty_d[at_d.s])));
            at_d.next(2);
        }
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
                const int quarter = warp & 3, half = (warp - 4) >> 2, span = a.tile_n / 2;
                const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21) + half * span;
                float *const to = sums + half * span * 128 + quarter * 32 + lane;
                for (int j = 0; j < span; j += 8) {
                    float v[8];
                    tmem_ld8_wait(d + j, v);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        to[(j + r) * 128] = v[r];
                }
                tc_fence_before();
            }
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && !sh.abort) {
            constexpr int kWarps = kFeatures / 32, kStep = kEpilogue / 32 / kWarps;  // warps side by side; rows at a time
            const int f = (warp - 4) % kWarps * 32 + lane;
            const int lo = a.tile_n * rank / a.split, hi = a.tile_n * (rank + 1) / a.split;
            const uint32_t at = smem_u32(sums) + f * 4;
            Sink<EPI> sink(a, m * kFeatures + f);
            constexpr int R = 4;
            for (int j = lo + (warp - 4) / kWarps; j < hi; j += kStep * R) {
                float v[R], w[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    v[r] = w[r] = 0.0f;
                for (int s = 0; s < a.split; ++s) {
                    const uint32_t from = in_block(at, s);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int row = j + r * kStep;
                        if (row < hi) {
                            v[r] += ld_cluster(from + row * 512);
                            if (EPI == kFfnJoin)
                                w[r] += ld_cluster(from + row * 512 + 256);
                        }
                    }
                }
                // rows of another block's share are not this one's to store
                if (j + (R - 1) * kStep < hi) {
                    sink.put(n * a.tile_n + j, kStep, v, w);
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (j + r * kStep < hi) {
                            const float v1[1] = {v[r]}, w1[1] = {w[r]};
                            sink.put(n * a.tile_n + j + r * kStep, kStep, v1, w1);
                        }
                }
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
        tmem_free<PAIR>(tmem, 2 * kHalfTmem);
    cluster_sync();  // the other blocks' copies, arrivals and reads have come
}

// Gradients of no rows; the routing weights of a block that is one expert.
__global__ void __launch_bounds__(256) fill_kernel(uint32_t *p, size_t words, uint32_t value)
{
    for (size_t i = blockIdx.x * size_t(256) + threadIdx.x; i < words; i += size_t(gridDim.x) * 256)
        p[i] = value;
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

constexpr int kRoom = kSmemMax - 1024 - 64 - static_cast<int>(sizeof(Shared));

}  // namespace

// Cycles of a tile's 64 k, as measured: the MMAs need 2 a row, the copies of a block's operands 64 bytes a cycle.
// The plan with the smallest product of waves of blocks and cycles of a block.
void ffn_plan(FfnProduct *p, int sms)
{
    FfnArgs &a = p->a;
    const int chunks = div_up(a.K, kChunk), features = p->epilogue == kFfnJoin ? 64 : 128;
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
            for (int split = 1; split <= (pair ? 1 : 8) && split <= chunks; split *= 2) {
                const double mma = 2.0 * n, copy = (kBlockA + 128.0 * (pair ? n / 2 : n)) / 64.0;
                const double chunk = mma > copy ? mma : copy;
                const double slots = pair ? sms / 2 : sms;
                const double waves = static_cast<double>(static_cast<long long>((tiles * split + slots - 1) / slots));
                const double block = div_up(chunks, split) * chunk;
                const double cost = pair ? 3000 + waves * (block + 400) + 10 * n : waves * (3000 + block + 16 * n);
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
    const int room = kRoom - (best_pair ? kExchange : 0), stage = stage_bytes(*p);
    a.stages = room / stage < kMaxStages ? room / stage : kMaxStages;
}

cudaError_t ffn_setup()
{
    cudaError_t ce = cudaSuccess;
    for (const void *f : ffn_kernels())
        if (ce == cudaSuccess && f != reinterpret_cast<const void *>(fill_kernel))
            ce = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom + 1024);
    return ce;
}

cudaError_t launch_ffn(const FfnProduct &p, int sms, cudaStream_t stream)
{
    const FfnArgs &a = p.a;
    const int tiles = a.m_tiles * a.n_tiles;
    size_t ring = static_cast<size_t>(a.stages) * stage_bytes(p);
    const size_t sums = static_cast<size_t>(a.tile_n) * 512;
    if (!p.pair && ring < sums)
        ring = sums;
    cudaLaunchConfig_t cfg = {};
    const int pairs = sms / 2;
    cfg.gridDim = dim3(p.pair ? 2 * (tiles < pairs ? tiles : pairs) : tiles * a.split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + ring + (p.pair ? kExchange : 0);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.pair ? 2 : a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.pair ? kernel_of<true>(p) : kernel_of<false>(p), a);
}

cudaError_t launch_ffn_zero(void *p, size_t bytes, cudaStream_t stream)
{
    fill_kernel<<<1024, 256, 0, stream>>>(static_cast<uint32_t *>(p), bytes / 4, 0u);
    return cudaGetLastError();
}

cudaError_t launch_ffn_ones(float *p, int n, cudaStream_t stream)
{
    fill_kernel<<<1, 256, 0, stream>>>(reinterpret_cast<uint32_t *>(p), n, 0x3F800000u);
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
    return {FFN(true), FFN(false), reinterpret_cast<const void *>(fill_kernel)};
#undef FFN
}

}  // namespace moe
