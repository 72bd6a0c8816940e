// moe_ffn.cu -- the products of a gated feed-forward block for many rows, and
// of its gradients.
//
//   h = silu(x W1^T) (x W3^T);  y = h W2^T
//   dh = dy W2;  dg = dh u silu'(g);  du = dh silu(g)
//   dx = dg W1 + du W3;  dW1 = dg^T x;  dW3 = du^T x;  dW2 = dy^T h
//
// Every one is D[features, rows] = A B^T with the features (the columns of the
// result in memory) along the MMA's M and the rows of x along its N, which may
// be any multiple of 16: a ragged number of rows wastes little. For the weights'
// gradients the "rows" are the weight's. Operands whose k are not
// contiguous in memory (W2 and W1 | W3 for dh and dx, everything for the
// weights' gradients) are read as MN-major tiles, so nothing is transposed.
//
// What follows a product is in its epilogue, in fp32 from tensor memory: gate
// and up joined (a block's 128 MMA rows are 64 of gate and the same 64 of up),
// or the gradient of h split into those of gate and up.
//
// Roundings: sums, g and u are fp32, y and the gradients are rounded once. h, and
// the gradients of g and u, are rounded to bf16 before the product that takes
// them: a result's error is then 1.41 times its own rounding's. In two bf16 parts,
// as the experts' kernels keep h for a few rows, that product would take twice the
// MMAs, which bound it for many rows.
//
// Two kernels:
//  - pairs: two neighbouring blocks multiply together (cta_group::2), 256
//    features x up to 256 rows a tile, persistent, accumulators in two halves of
//    tensor memory, so that one tile's epilogue runs under the next one's MMAs.
//    The three products that follow the split are one launch: whole tiles go
//    round the pairs, the last one or two rounds are cut along K where that evens the
//    pairs out. A tile that pairs share: all but the last one's sums go through memory;
//    the last pair, which ends with it, puts them into tensor memory and adds its
//    own there, in the order of K. Waits go to lower pairs only;
//  - splits: for few tiles. A block has 128 features, a cluster of 1 to 8 blocks
//    shares a tile's K. Their sums meet in distributed shared memory, added in
//    the order of K, a share of the rows in each block.
// No sum depends on timing. Kernels of a call overlap (programmatic launches):
// the next one is set up, and has its first weights on their way, while this one
// ends.
//
// What bounds them: for many rows the MMAs, then the power limit (a step of
// 4096 rows, 4096 x 14336, 4.3 TFLOP: 2.54 to 2.7 ms in captured calls, 1.6 to
// 1.7 PFLOP/s where cuBLAS sustains 1.72 and reaches 1.89 for a moment; 8191 rows,
// 7168 x 2048, forward 408 to 425 us, 1.7 PFLOP/s; tensor pipe active 86 % in the three
// gradients of 2048 x 4096 x 4096). Below 256 rows a tile the copies: 57 bytes a
// cycle come into an SM, a chunk of 64 k takes 0.23 us with 176 rows, 0.31 with
// 256 (515 rows, 4096 x 14336: 121 to 142 us as the clock is, floor 96). For few
// rows DRAM and a fixed part of some 4 us a kernel, of which the wait for the kernel
// before, the first copy and the results are one each: one row, 7168 x 2048, 19.4
// us, 14 of them at 6.6 TB/s; 128 rows 24.7. Rows whose length is no multiple of 128
// bytes cost up to a quarter more (2056 x 1400 against 2048 x 1408: 110 and 88 us):
// each of a tile's rows lies in two lines.
#include <cmath>

#include <cuda_bf16.h>

#include "moe_ffn.h"
#include "moe_sched.h"

namespace moe {

namespace {

constexpr int kMaxStages = 12;
constexpr int kBlockA = 16384;      // 128 features x 64 k
constexpr int kHalfTmem = 256;      // columns of one accumulator
constexpr int kPairStore = 512;     // threads that store a pair's results: 16 warps, under the next tile's MMAs
constexpr int kSplitStore = 256;
constexpr int kFirstStore = 4;      // warp 0 copies, warp 1 multiplies, warps from this one on store

// Shared memory through which a pair's results leave: of four warps, two boxes of 16 rows, one of fp32 or of three results;
// joined, also the halves of gate and up that 8 pairs of warps exchange.
static __host__ __device__ constexpr int box_bytes(int epi) { return epi == kFfnStore ? 8192 : epi == kFfnJoin ? 4096 : 12288; }
static __host__ __device__ constexpr int out_bytes(int epi) { return 4 * box_bytes(epi) + (epi == kFfnJoin ? 8 * 2048 : 0); }
static __host__ __device__ constexpr int features_of(int epi) { return epi == kFfnJoin ? 64 : 128; }  // of a block

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t full_d[2], empty_d[2];
    uint64_t drain, loaded;
    uint32_t tmem;
    int abort, issued, reset;
};

// Tensor memory is given out in powers of two from 32 columns on.
static __host__ __device__ __forceinline__ uint32_t tmem_columns(int n)
{
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
}

// silu of g and its derivative, to some 1e-5 of their values (the fast exponential and division; the results are rounded
// to 2^-8). From exp(-|g|), so that the divisor lies in [1, 2] and sigma and 1 - sigma keep their value down to fp32's
// smallest numbers (1 / (1 + exp(-g)) is 0 from g = -87.4 on).
struct Sigma {
    float s, rest;  // sigma and 1 - sigma
    __device__ __forceinline__ explicit Sigma(float g)
    {
        const float x = __expf(-fabsf(g)), large = __fdividef(1.0f, 1.0f + x), small = x * large;
        s = g < 0.0f ? small : large;
        rest = g < 0.0f ? large : small;
    }
};
static __device__ __forceinline__ float silu(float g) { return g * Sigma(g).s; }

struct Gate {
    float silu, slope;
    __device__ __forceinline__ explicit Gate(float g)
    {
        const Sigma sigma(g);
        silu = g * sigma.s;
        slope = sigma.s * fmaf(g, sigma.rest, 1.0f);
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
template <int EPI> struct Sink {
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
        if (EPI != kFfnStore || a.aligned) {
            *reinterpret_cast<uint2 *>(p) = r;
        } else {
            uint16_t *const e = reinterpret_cast<uint16_t *>(p);
            e[0] = r.x & 0xFFFF, e[1] = r.x >> 16, e[2] = r.y & 0xFFFF, e[3] = r.y >> 16;
        }
    }
};

// What both kernels do before their work, and after it.
static __device__ __forceinline__ void set_barriers(Shared &sh, int storers)
{
    sh.abort = sh.issued = sh.reset = 0;
    for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(smem_u32(&sh.full[i]), 1);
        mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sh.full_d[i]), 1);
        mbar_init(smem_u32(&sh.empty_d[i]), storers);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    mbar_init(smem_u32(&sh.loaded), storers);
    mbar_init_fence();
}

static __device__ __forceinline__ void report(const Shared &sh, unsigned int *err)
{
    atomicAdd_system(err + sh.abort, 1u);
    __threadfence_system();
    atomicAdd_system(err, 1u);
}

// Bytes of B in a stage: rows (k contiguous), or blocks of 64 rows.
static __host__ __device__ __forceinline__ int bytes_b(int rows, bool mn) { return mn ? (rows + 63) / 64 * 8192 : rows * 128; }

// The kernels' operands: A is MN-major in what follows the forward pass (GRAD), B in the weights' gradients only.
template <int EPI, bool GRAD> constexpr bool kAmn = EPI == kFfnSplit || GRAD;

// One chunk of 64 k: four instructions of 16, which are 32 bytes of a row apart, or 16 rows of 128 bytes.
template <bool A_MN, bool B_MN, bool PAIR>
static __device__ __forceinline__ void multiply(uint32_t d, uint32_t from, int tile_n, bool add)
{
    const uint32_t idesc =
        idesc_f16(PAIR ? 256 : 128, tile_n, 1) | (A_MN ? kIdescAmn : 0u) | (B_MN ? kIdescBmn : 0u);
    const uint64_t da = A_MN ? desc_mn(from) : desc_sw128(from);
    const uint64_t db = B_MN ? desc_mn(from + kBlockA) : desc_sw128(from + kBlockA);
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // in 16-byte units
        const uint64_t qa = da + q * (A_MN ? 128 : 2), qb = db + q * (B_MN ? 128 : 2);
        if (PAIR)
            mma_ss_pair(d, qa, qb, idesc, add || q > 0);
        else
            mma_ss(d, qa, qb, idesc, add || q > 0);
    }
}

template <bool PAIR>
static __device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t full, int x, int y)
{
    if (PAIR)
        tma_load_2d_pair(dst, map, in_first_block(full), x, y);
    else
        tma_load_2d(dst, map, full, x, y);
}

// 128 features from m0 on (joined: 64 of gate, and of up), and `rows` rows from n0 on, of 64 k.
template <int EPI, bool A_MN, bool PAIR>
static __device__ __forceinline__ void load_a(const FfnArgs &a, uint32_t dst, uint32_t full, int m0, int k)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int f = EPI == kFfnJoin ? m0 + j * a.M : m0 + j * 64;
        load_box<PAIR>(dst + j * 8192, &a.ma, full, A_MN ? f : k, A_MN ? k : f);
    }
}
template <bool PAIR>
static __device__ __forceinline__ void load_b(const FfnArgs &a, bool mn, uint32_t dst, uint32_t full, int n0, int rows, int k)
{
    if (mn) {
        for (int j = 0; j < rows; j += 64)
            load_box<PAIR>(dst + kBlockA + j * 128, &a.mb, full, n0 + j, k);
    } else {
        load_box<PAIR>(dst + kBlockA, &a.mb, full, k, n0);
    }
}

// ---- pairs -------------------------------------------------------------------------------

// GRAD: dx and the weights' gradients, up to three products; else one product.
template <int EPI, bool GRAD> __global__ void __launch_bounds__(128 + kPairStore, 1) pair_kernel(const __grid_constant__ FfnGroup q)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const uint32_t dyn0 = smem_u32(dyn), ring = (dyn0 + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
    constexpr int kFeatures = features_of(EPI);
    constexpr bool A_MN = kAmn<EPI, GRAD>;
    volatile int *const abort = &sh.abort;

    if (tid == 0)
        set_barriers(sh, 2 * kPairStore / 32);
    else if (tid >= 64 && tid < 64 + q.count) {
        tma_prefetch_map(&q.p[tid - 64].ma);
        tma_prefetch_map(&q.p[tid - 64].mb);
    }
    if (warp == 1)
        tmem_alloc<true>(smem_u32(&sh.tmem), 2 * kHalfTmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no copy or arrival reaches a block before its barriers are set
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0 && elect_one()) {
        // ---- copies ----
        auto expect = [&](uint32_t full, int bytes) {
            if (rank == 0)
                mbar_expect(full, 2 * bytes);
        };
        Item it;
        int ahead = 0;  // the ring's first round: weights that are copied before the rows are there
        {
            Items first(q, pair);
            if (first.next(it) && q.p[GRAD ? it.g : 0].early) {
                const FfnArgs &a = q.p[GRAD ? it.g : 0];
                int m, n;
                tile_of(a, it.tile, m, n);
                for (; ahead < q.stages && it.c0 + ahead < it.c1; ++ahead) {
                    expect(smem_u32(&sh.full[ahead]), kBlockA + bytes_b(a.tile_n / 2, GRAD && a.b_mn));
                    load_a<EPI, A_MN, true>(a, ring + ahead * q.bytes, smem_u32(&sh.full[ahead]), (2 * m + rank) * kFeatures,
                                      (it.c0 + ahead) * kChunk);
                }
            }
        }
        pdl_wait();
        fence_async_proxy();  // what the kernel before stored from registers is read by copies
        pdl_launch_next();
        Cursor at;
        int issued = 0;
        bool run = true;
        for (Items w(q, pair); run && w.next(it);) {
            const FfnArgs &a = q.p[GRAD ? it.g : 0];
            int m, n;
            tile_of(a, it.tile, m, n);
            const int m0 = (2 * m + rank) * kFeatures, rows = a.tile_n / 2, n0 = n * a.tile_n + rank * rows;
            const int bytes = kBlockA + bytes_b(rows, GRAD && a.b_mn);
            for (int c = it.c0; c < it.c1; ++c) {
                const uint32_t to = ring + at.s * q.bytes, full = smem_u32(&sh.full[at.s]);
                if (issued >= ahead) {
                    run = mbar_wait(smem_u32(&sh.empty[at.s]), at.parity ^ 1, abort, kWaitEmptyA);
                    if (!run)
                        break;
                    expect(full, bytes);
                    load_a<EPI, A_MN, true>(a, to, full, m0, c * kChunk);
                }
                load_b<true>(a, GRAD && a.b_mn, to, full, n0, rows, c * kChunk);
                at.next(q.stages);
                ++issued;
            }
        }
        sh.issued = issued;
    } else if (warp == 1) {
        // ---- matrix instructions, in the first block ----
        pdl_wait();  // waits are for this kernel's copies: the kernel before may take longer than their limit
        Cursor at, at_d;
        bool run = rank == 0;
        Item it;
        for (Items w(q, pair); run && w.next(it);) {
            const FfnArgs &a = q.p[GRAD ? it.g : 0];
            // one value for all lanes, which the compiler then keeps in uniform registers
            const int tile_n = __shfl_sync(~0u, a.tile_n, 0), b_mn = GRAD ? __shfl_sync(~0u, a.b_mn, 0) : 0;
            run = mbar_wait_warp(smem_u32(&sh.empty_d[at_d.s]), at_d.parity ^ 1, abort, kWaitEmptyD);
            const uint32_t d = tmem + at_d.s * kHalfTmem;
            const bool add = GRAD && it.kind == kLast;  // to the sums of the tile's other parts
            if (run && add)
                run = mbar_wait_warp(smem_u32(&sh.loaded), 0, abort, kWaitDone);
            for (int c = it.c0; run && c < it.c1; ++c) {
                run = mbar_wait_warp(smem_u32(&sh.full[at.s]), at.parity, abort, kWaitFullA);
                if (!run)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    if (GRAD && b_mn)
                        multiply<A_MN, true, true>(d, ring + at.s * q.bytes, tile_n, add || c > it.c0);
                    else
                        multiply<A_MN, false, true>(d, ring + at.s * q.bytes, tile_n, add || c > it.c0);
                    tc_commit_pair(smem_u32(&sh.empty[at.s]));
                }
                at.next(q.stages);
            }
            if (elect_one())
                tc_commit_pair(smem_u32(&sh.full_d[at_d.s]));
            at_d.next(2);
        }
        if (rank == 0 && elect_one())
            tc_commit_pair(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= kFirstStore) {
        // ---- results, under the next tile's products ----
        // A step is 16 rows. Four warps with the four quarters of the features take every fourth step, give each row's
        // features their place in shared memory, and one of them sends it off as a box (out of bounds is cut off by the
        // map). Joined: a warp of quarters 0 and 1 has gate, the one two quarters on up of the same 32 features; they
        // exchange halves, and each joins 8 of the 16 rows.
        Cursor at_d;
        const int quarter = warp & 3, turn = (warp - kFirstStore) >> 2;
        const bool second = EPI == kFfnJoin && quarter >= 2, sender = quarter == 0 && elect_one();
        const int f = (EPI == kFfnJoin ? quarter & 1 : quarter) * 32 + lane;  // of the block's features
        constexpr int kRows = EPI == kFfnJoin ? 8 : 16;                       // of a warp
        const int row0 = second ? 8 : 0;
        uint8_t *const stage = dyn + (ring - dyn0) + q.stages * q.bytes + turn * box_bytes(EPI);
        float *const exchange = reinterpret_cast<float *>(dyn + (ring - dyn0) + q.stages * q.bytes + 4 * box_bytes(EPI)) +
                                (turn * 2 + (quarter & 1)) * 512 + lane;  // [gate, up][8][32]
        // a block's part of a tile: [row][128 MMA rows]
        const auto part_of = [&](int p) { return q.parts + (static_cast<size_t>(2 * p + rank) * 256) * 128 + quarter * 32 + lane; };
        // The sums of the other parts of the tile that this pair ends go into tensor memory, where its own are added:
        // under the item before, unless that is this pair's part, for which others may be waiting.
        Item it, last;
        int left = -1;  // items before they are loaded
        if (Items w(q, pair); GRAD && w.last(last)) {
            int before = kPart, at = 0;
            while (w.next(it) && it.kind != kLast) {
                before = it.kind;
                ++at;
            }
            left = before == kPart ? at : at - 1;
        }
        auto load_parts = [&](uint32_t d) {
            Items w(q, pair);
            bool run = true;
            if (tid == kFirstStore * 32)
                for (int p = w.first_of_last(); run && p < pair; ++p)
                    if (q.begin[p] < q.begin[p + 1])
                        run = wait_count(q.flags + 2 * p + rank, 1, abort, kWaitDone);
            if (!named_all(1, kPairStore, run))
                return false;
            for (int step = turn; step < q.p[GRAD ? last.g : 0].tile_n / 16; step += 4) {
                float v[16];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    v[r] = 0.0f;
                for (int p = w.first_of_last(); p < pair; p += 2) {  // two parts' loads in flight
                    float x[16], y[16];
                    const bool has_x = q.begin[p] < q.begin[p + 1], has_y = p + 1 < pair && q.begin[p + 1] < q.begin[p + 2];
                    const float *const at_x = part_of(p) + step * 16 * 128, *const at_y = part_of(p + 1) + step * 16 * 128;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        x[r] = has_x ? __ldcg(at_x + r * 128) : 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        y[r] = has_y ? __ldcg(at_y + r * 128) : 0.0f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        v[r] = v[r] + x[r] + y[r];
                }
                tmem_st16(d + step * 16, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(in_first_block(smem_u32(&sh.loaded)));
            return true;
        };
        bool one = EPI == kFfnSplit;
        for (int i = 0; GRAD && i < q.count; ++i)
            one = one || q.p[i].fp32;
        int sent = 0, items = 0;
        pdl_wait();  // flags, and what is fetched ahead of the sums, are the kernel's before until then
        for (Items w(q, pair); w.next(it);) {
            const FfnArgs &a = q.p[GRAD ? it.g : 0];
            const int steps = a.tile_n / 16;
            const bool weight = GRAD && a.fp32, boxes = EPI != kFfnStore || a.boxes;
            int m, n;
            tile_of(a, it.tile, m, n);
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
            bool run = true;
            if (GRAD && items++ == left) {  // the last item's half of tensor memory is this one's, or the other
                const int half = at_d.s ^ (it.kind == kLast ? 0 : 1);
                run = load_parts(tmem + (static_cast<uint32_t>(quarter) << 21) + half * kHalfTmem);
                if (!run)
                    break;
            }
            fetch(turn);
            run = mbar_wait(smem_u32(&sh.full_d[at_d.s]), at_d.parity, abort, kWaitFullD);
            if (!named_all(1, kPairStore, run))
                break;
            tc_fence_after();
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21) + at_d.s * kHalfTmem;
            if (GRAD && it.kind == kPart) {
                float *const part = part_of(pair);
                for (int step = turn; step < steps; step += 4) {
                    float v[16];
                    tmem_ld16(d + step * 16, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        part[(step * 16 + r) * 128] = v[r];
                }
                named_sync(1, kPairStore);
                if (tid == kFirstStore * 32)
                    add_acq_rel(q.flags + 2 * pair + rank, 1);
            } else {
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
                        // two boxes of bf16 in turn; one of fp32 (in the whole launch then) or of three results
                        uint8_t *const box = stage + (one || (sent & 1) == 0 ? 0 : kFeatures * 32);
                        ++sent;
                        if (sender) {
                            if (one)
                                bulk_wait_read<0>();
                            else
                                bulk_wait_read<1>();
                        }
                        named_sync(2 + turn, 128);
                        if (weight) {
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
                            if (weight && a.accumulate)
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
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort) {  // copies in flight land before the block's memory is given back
        if (tid == 0) {
            bool landed = true;
            for (int i = max(0, sh.issued - q.stages); rank == 0 && landed && i < sh.issued; ++i)
                landed = mbar_wait(smem_u32(&sh.full[i % q.stages]), (i / q.stages) & 1, nullptr, kWaitOther);
            // copies that the first block no longer counts land meanwhile
            for (const long long from = clock64(); clock64() - from < 1000000;) {
            }
            report(sh, q.err);
        }
        __syncthreads();
    }
    if (warp == 1)
        tmem_free<true>(tmem, 2 * kHalfTmem);
    cluster_sync();  // the other block's copies and arrivals have come
    if (GRAD && q.cut) {  // the last block to leave clears the flags for the next launch
        if (tid == 0)
            sh.reset = add_acq_rel(q.flags + 2 * kFfnMaxPairs, 1) == static_cast<int>(gridDim.x) - 1;
        __syncthreads();
        if (sh.reset) {
            if (tid < 2 * kFfnMaxPairs)
                q.flags[tid] = 0;
            if (tid == 0)
                q.flags[2 * kFfnMaxPairs] = 0;
        }
    }
}

// ---- splits --------------------------------------------------------------------------------

template <int EPI> __global__ void __launch_bounds__(128 + kSplitStore, 2) split_kernel(const __grid_constant__ FfnSplit q)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const FfnArgs &a = q.a;
    const uint32_t dyn0 = smem_u32(dyn), ring = (dyn0 + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int rank = blockIdx.x % q.split;
    const int c0 = a.chunks * rank / q.split, c1 = a.chunks * (rank + 1) / q.split;
    const int bytes = kBlockA + bytes_b(a.tile_n, false);
    constexpr int kFeatures = features_of(EPI);
    constexpr bool A_MN = kAmn<EPI, false>;
    volatile int *const abort = &sh.abort;
    int m, n;
    tile_of(a, blockIdx.x / q.split, m, n);

    if (tid == 0) {
        set_barriers(sh, 1);
    } else if (tid == 64) {
        tma_prefetch_map(&a.ma);
        tma_prefetch_map(&a.mb);
    }
    const uint32_t columns = tmem_columns(a.tile_n);
    if (warp == 1)
        tmem_alloc(smem_u32(&sh.tmem), columns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 0 && elect_one()) {
        // ---- copies ----
        auto a_of = [&](int s, int c) {
            mbar_expect(smem_u32(&sh.full[s]), bytes);
            load_a<EPI, A_MN, false>(a, ring + s * bytes, smem_u32(&sh.full[s]), m * kFeatures, c * kChunk);
        };
        int ahead = 0;  // the ring's first round: weights that are copied before the rows are there
        if (a.early)
            for (; ahead < q.stages && c0 + ahead < c1; ++ahead)
                a_of(ahead, c0 + ahead);
        pdl_wait();
        fence_async_proxy();  // what the kernel before stored from registers is read by copies
        pdl_launch_next();
        Cursor at;
        int issued = 0;
        for (int c = c0; c < c1; ++c) {
            if (issued >= ahead) {
                if (!mbar_wait(smem_u32(&sh.empty[at.s]), at.parity ^ 1, abort, kWaitEmptyA))
                    break;
                a_of(at.s, c);
            }
            load_b<false>(a, false, ring + at.s * bytes, smem_u32(&sh.full[at.s]), n * a.tile_n, a.tile_n, c * kChunk);
            at.next(q.stages);
            ++issued;
        }
        sh.issued = issued;
    } else if (warp == 1) {
        // ---- matrix instructions ----
        pdl_wait();  // waits are for this kernel's copies: the kernel before may take longer than their limit
        Cursor at;
        for (int c = c0; c < c1; ++c) {
            if (!mbar_wait_warp(smem_u32(&sh.full[at.s]), at.parity, abort, kWaitFullA))
                break;
            tc_fence_after();
            if (elect_one()) {
                multiply<A_MN, false, false>(tmem, ring + at.s * bytes, a.tile_n, c > c0);
                tc_commit(smem_u32(&sh.empty[at.s]));
            }
            at.next(q.stages);
        }
        if (elect_one()) {
            tc_commit(smem_u32(&sh.full_d[0]));
            tc_commit(smem_u32(&sh.drain));
        }
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    }
    // ---- this block's sums into its memory, then a share of the rows from all of the cluster's ----
    float *const sums = reinterpret_cast<float *>(dyn + (ring - dyn0));  // [rows][128 features]
    if (warp >= kFirstStore) {
        pdl_wait();
        const bool run = mbar_wait(smem_u32(&sh.full_d[0]), 0, abort, kWaitFullD);
        if (named_all(1, kSplitStore, run)) {
            tc_fence_after();
            const int quarter = warp & 3;
            const uint32_t d = tmem + (static_cast<uint32_t>(quarter) << 21);
            float *const to = sums + quarter * 32 + lane;
            for (int j = (warp - kFirstStore) / 4 * 16; j < a.tile_n; j += 32) {
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
    if (q.split > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp >= kFirstStore && !sh.abort) {
        constexpr int kLanes = kFeatures / 4, kStep = kSplitStore / kLanes;  // lanes of a row, rows at a time
        constexpr int R = EPI == kFfnStore ? 2 : 1;
        const int f = lane % kLanes * 4;
        const int lo = a.tile_n * rank / q.split, hi = a.tile_n * (rank + 1) / q.split;
        const uint32_t at = smem_u32(sums) + f * 4;
        const Sink<EPI> sink(a, m * kFeatures + f);
        for (int j = lo + (tid - kFirstStore * 32) / kLanes; j < hi; j += kStep * R) {
            float4 v[R];
            typename Sink<EPI>::Kept k[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (EPI == kFfnJoin)
                    k[r].u = v[r];
                if (j + r * kStep < hi)
                    sink.fetch(n * a.tile_n + j + r * kStep, k[r]);
            }
            for (int s0 = 0; s0 < q.split; s0 += 4) {
                float4 x[4][R], y[4][R];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (s0 + s < q.split) {
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
                    if (s0 + s < q.split)
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
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort) {  // copies in flight land before the block's memory is given back
        if (tid == 0) {
            bool landed = true;
            for (int i = max(0, sh.issued - q.stages); landed && i < sh.issued; ++i)
                landed = mbar_wait(smem_u32(&sh.full[i % q.stages]), (i / q.stages) & 1, nullptr, kWaitOther);
            report(sh, q.err);
        }
        __syncthreads();
    }
    if (warp == 1)
        tmem_free(tmem, columns);
    if (q.split > 1)
        cluster_sync();  // the other blocks have read this one's sums
}

// Gradients of no rows.
__global__ void __launch_bounds__(256) zero_kernel(uint32_t *p, size_t words)
{
    for (size_t i = blockIdx.x * size_t(256) + threadIdx.x; i < words; i += size_t(gridDim.x) * 256)
        p[i] = 0;
}

// ---- plans ---------------------------------------------------------------------------------

// Dynamic shared memory of a block that has an SM for itself, and of one that shares it with another.
constexpr int kRoom = kSmemMax - 64 - static_cast<int>(sizeof(Shared));
constexpr int kHalfRoom = (228 * 1024) / 2 - 1024 - 64 - static_cast<int>(sizeof(Shared));
constexpr int kShareRows = 128;  // up to so many rows a tile, a split's blocks can share an SM

int div_up(int a, int b) { return (a + b - 1) / b; }

// Cycles of a tile's 64 k: 2 a row in the MMAs, or 64 bytes a cycle of the copies of a block's operands.
double chunk_cycles(int n, bool pair)
{
    const double mma = 2.0 * n, copy = (kBlockA + 128.0 * (pair ? n / 2 : n)) / 64.0;
    return mma > copy ? mma : copy;
}

// Of a pair's tile of n rows: its products, under which its epilogue is hidden, or that.
double tile_cycles(const FfnArgs &a, int n)
{
    const double products = a.chunks * chunk_cycles(n, true) + 200, store = 1500 + 18.0 * n;
    return products > store ? products : store;
}

struct Choice {
    double cost;
    int n, split;  // split 0: pairs
    bool cut;
};

// All operands come from DRAM once, whoever asks for them.
double dram_cycles(const FfnArgs &a, int epilogue)
{
    return 2.0 * a.K * (static_cast<double>(a.M) * (epilogue == kFfnJoin ? 2 : 1) + a.N) / 3500.0;
}

// A part costs a trip of its sums through memory, on both sides. So rounds whose whole tiles leave little to gain are not
// cut, and pairs that have nearly their share in whole tiles get no more (gradients of 700 rows, 2048 x 768: 22 us, with
// cuts wherever they even the pairs out 37; 1500 rows, 4096 x 1536: 80 and 85; others within 1 %).
constexpr double kCutGain = 8000, kLeastShare = 4000;  // cycles

// Cycles of a product's pairs with tiles of n rows: rounds of whole tiles, or an even share of them, cut. Gradients of
// different K in one launch are balanced by cutting. One product is not, unless its tiles are few: pairs that go through K
// out of step read the weights once for each tile of rows (y of 515 rows, 4096 x 14336: 50 us over all pairs, 45 over 64 of
// 76 in step), and a pair with nothing but a tile's last part waits for the others' before it begins. (dx and what it needs,
// 64 rows, 4096 x 4096: 33 us cut, 43 whole; 512 rows: 68 and 55.)
Choice pair_choice(const FfnArgs &a, int epilogue, int n, int count, bool grad, int sms)
{
    const double tiles = static_cast<double>(div_up(a.N, n)) * div_up(a.M, 2 * features_of(epilogue));
    const double rounds = tiles / (sms / 2), tile = tile_cycles(a, n), dram = dram_cycles(a, epilogue);
    const double whole = std::ceil(rounds) * tile;
    const double even = count > 1 ? rounds * tile : 2.0 * rounds * tile + 10.0 * n / rounds + kCutGain;
    const bool cut = grad && (count > 1 || (rounds < 0.5 && even < whole));
    return {std::fmax(cut ? even : whole, dram) + 7000 + 10.0 * n, n, 0, cut};
}

// Whether a split's blocks take half of an SM's memory: where there are more blocks than SMs, or half holds all that a block
// copies. The next kernel's blocks then start beside them (1 row, 1024 x 1024: 7.9 us, alone on the SMs 11.5; 128 rows,
// 7168 x 2048, whose copies need the room: 24.7, alone 22.0).
bool shares_sm(const FfnArgs &a, double blocks, int n, int split, int sms)
{
    return n <= kShareRows && (blocks > sms || div_up(a.chunks, split) <= (kHalfRoom - 1024) / (kBlockA + 128 * n));
}

// A cluster's sums meet at a cost that grows with its blocks. A block alone on its SM leaves no room for the next kernel's
// first copies.
Choice split_choice(const FfnArgs &a, int epilogue, int n, int split, int sms)
{
    const double tiles = static_cast<double>(div_up(a.N, n)) * div_up(a.M, features_of(epilogue)), blocks = tiles * split;
    const bool share = shares_sm(a, blocks, n, split, sms);
    const double copy = (kBlockA + 128.0 * n) / 45.0, chunk = copy > 2.0 * n ? copy : 2.0 * n;  // mostly from DRAM
    const double cost = std::ceil(blocks / sms) * div_up(a.chunks, split) * chunk;
    const double after = std::ceil(blocks / (share ? 2 * sms : sms)) * (3000.0 + n * (8.0 + 4.0 * split));
    const double dram = dram_cycles(a, epilogue);
    return {(cost > dram ? cost : dram) + after + (share ? 0.0 : 800.0), n, split, false};
}

template <class F> Choice least(const FfnArgs &a, F &&cost)
{
    // Of rows that lie along memory a pair's halves are whole lines: 128 rows or 256. Other heights read up to twice as
    // much (the gradients of 1999 rows, 2056 x 1400: 51 us instead of 33).
    const int step = a.b_mn ? 128 : 16;
    Choice best = {-1.0, step, 0, false};
    for (int n = step; n <= 256; n += step) {
        if (n > step && div_up(a.N, n - step) == div_up(a.N, n))
            continue;  // the same tiles with more waste
        const Choice c = cost(n);
        if (best.cost < 0.0 || c.cost < best.cost)
            best = c;
    }
    return best;
}

// Cycles of a pair's whole tiles: every pairs-th of those of all products.
double whole_cycles(const FfnGroup &q, int pair)
{
    double sum = 0.0;
    int first = 0;  // the pair that has the product's first one
    for (int g = 0; g < q.count; ++g) {
        const FfnArgs &a = q.p[g];
        const int skip = ((pair - first) % q.pairs + q.pairs) % q.pairs;
        const int n = a.whole > skip ? (a.whole - skip + q.pairs - 1) / q.pairs : 0;
        sum += n * tile_cycles(a, a.tile_n);
        first = (first + a.whole) % q.pairs;
    }
    return sum;
}

// Which tiles are whole and which are cut. Tiles of a product whose shares end within a few chunks of a tile's edge are
// not cut there.
void cut_rounds(FfnGroup *q, bool cut)
{
    const int pairs = q->pairs;
    int tiles = 0;
    double all = 0.0, most = 0.0;
    for (int g = 0; g < q->count; ++g) {
        FfnArgs &a = q->p[g];
        a.whole = a.m_tiles * a.n_tiles;
        tiles += a.whole;
        all += a.whole * tile_cycles(a, a.tile_n);
    }
    for (int p = 0; p < pairs; ++p)
        most = std::fmax(most, whole_cycles(*q, p));
    cut = cut && most > all / pairs + kCutGain;
    // a last round of few tiles is cut together with the one before: a tile has few parts
    const int rounds = tiles / pairs, rest_tiles = tiles % pairs;
    q->whole = !cut ? tiles : (rest_tiles * 3 >= pairs || rounds == 0 ? rounds : rounds - 1) * pairs;
    for (int g = 0, left = q->whole; g < q->count; ++g) {
        FfnArgs &a = q->p[g];
        a.whole = a.whole < left ? a.whole : left;
        left -= a.whole;
    }
    // shares of the cut rounds: what a pair's whole tiles leave of its part of everything
    double want[kFfnMaxPairs], sum = 0.0, rest = all, largest = 0.0;
    for (int p = 0; p < pairs; ++p) {
        const double whole = whole_cycles(*q, p);
        rest -= whole;
        want[p] = std::fmax(all / pairs - whole, 0.0);
        largest = std::fmax(largest, want[p]);
    }
    const int apart = largest > 0.0 && largest < kLeastShare ? static_cast<int>(std::ceil(kLeastShare / largest)) : 1;
    for (int p = 0; p < pairs; ++p) {  // shares that would be too small go to the others
        want[p] = apart > 1 ? (p % apart == 0 ? largest : 0.0) : want[p] < kLeastShare ? 0.0 : want[p];
        sum += want[p];
    }
    double to = 0.0;
    for (int p = 0; p <= kFfnMaxPairs; ++p)
        q->begin[p] = 0;
    int unit = 0;
    for (int p = 0; p < pairs; ++p) {
        q->begin[p] = unit;
        to += sum > 0.0 ? want[p] * rest / sum : 0.0;
        // the unit at `to` cycles
        double at = 0.0;
        unit = 0;
        for (int g = 0; g < q->count; ++g) {
            const FfnArgs &a = q->p[g];
            const double one = tile_cycles(a, a.tile_n) / a.chunks;
            const int have = (a.m_tiles * a.n_tiles - a.whole) * a.chunks;
            if (p == pairs - 1 || at + have * one <= to) {
                at += have * one;
                unit += have;
                continue;
            }
            int here = static_cast<int>((to - at) / one + 0.5);
            const int edge = a.chunks / 32 > 2 ? a.chunks / 32 : 2, in = here % a.chunks;
            if (in <= edge)
                here -= in;
            else if (a.chunks - in <= edge)
                here += a.chunks - in;
            unit += here;
            break;
        }
        if (unit < q->begin[p])
            unit = q->begin[p];
    }
    for (int p = pairs; p <= kFfnMaxPairs; ++p)
        q->begin[p] = unit;
}

}  // namespace

void ffn_plan(FfnLaunch *l, int sms)
{
    FfnGroup &q = l->q;
    q.pairs = sms / 2 < kFfnMaxPairs ? sms / 2 : kFfnMaxPairs;
    const bool grad = q.p[0].a_mn && l->epilogue == kFfnStore;  // dx, or the weights' gradients: pairs
    l->split = 0;
    bool cut = false;
    for (int g = 0; g < q.count; ++g) {
        FfnArgs &a = q.p[g];
        a.chunks = div_up(a.K, kChunk);
        Choice c = least(a, [&](int n) { return pair_choice(a, l->epilogue, n, q.count, grad, 2 * q.pairs); });
        if (q.count == 1) {
            for (int split = 1; !grad && split <= 8 && split <= a.chunks; split *= 2) {
                const Choice s = least(a, [&](int n) { return split_choice(a, l->epilogue, n, split, sms); });
                if (s.cost < c.cost)
                    c = s;
            }
            l->split = c.split;
        }
        a.tile_n = c.n;
        cut = c.cut;
        a.m_tiles = div_up(a.M, features_of(l->epilogue) * (c.split ? 1 : 2));
        a.n_tiles = div_up(a.N, c.n);
        a.box_b = c.split ? c.n : c.n / 2;
        a.band_inverse = 1.0f / static_cast<float>(kBand * a.m_tiles);
        a.rest_inverse = 1.0f / static_cast<float>(a.n_tiles % kBand ? a.n_tiles % kBand : kBand);
    }
    if (l->split) {
        const FfnArgs &a = q.p[0];
        const bool share = shares_sm(a, static_cast<double>(a.m_tiles) * a.n_tiles * l->split, a.tile_n, l->split, sms);
        q.bytes = kBlockA + bytes_b(a.tile_n, a.b_mn);
        q.stages = ((share ? kHalfRoom : kRoom) - 1024) / q.bytes;
    } else {
        q.bytes = 0;
        for (int g = 0; g < q.count; ++g) {
            const int bytes = kBlockA + bytes_b(q.p[g].tile_n / 2, q.p[g].b_mn);
            q.bytes = bytes > q.bytes ? bytes : q.bytes;
        }
        q.stages = (kRoom - 1024 - out_bytes(l->epilogue)) / q.bytes;
        cut_rounds(&q, cut);
        q.cut = q.begin[q.pairs] > 0;
    }
    q.stages = q.stages < kMaxStages ? q.stages : kMaxStages;
    l->parts = !l->split && q.cut ? static_cast<size_t>(2 * q.pairs) * 256 * 128 * sizeof(float) : 0;
}

namespace {

using PairKernel = void (*)(FfnGroup);
using SplitKernel = void (*)(FfnSplit);

PairKernel pair_of(int epilogue, bool grad)
{
    return epilogue == kFfnJoin    ? pair_kernel<kFfnJoin, false>
           : epilogue == kFfnSplit ? pair_kernel<kFfnSplit, false>
           : grad                  ? pair_kernel<kFfnStore, true>
                                   : pair_kernel<kFfnStore, false>;
}
SplitKernel split_of(int epilogue)
{
    return epilogue == kFfnJoin ? split_kernel<kFfnJoin> : epilogue == kFfnSplit ? split_kernel<kFfnSplit> : split_kernel<kFfnStore>;
}

}  // namespace

cudaError_t ffn_setup()
{
    cudaError_t ce = cudaSuccess;
    for (const void *f : ffn_kernels())
        if (ce == cudaSuccess && f != reinterpret_cast<const void *>(zero_kernel))
            ce = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    return ce;
}

cudaError_t launch_ffn(const FfnLaunch &l, cudaStream_t stream)
{
    const FfnGroup &q = l.q;
    const FfnArgs &a = q.p[0];
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = l.split ? l.split : 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    size_t ring = static_cast<size_t>(q.stages) * q.bytes;
    if (l.split) {
        const size_t sums = static_cast<size_t>(a.tile_n) * 512;  // no more than a few stages
        FfnSplit s;
        s.a = a;
        s.stages = q.stages;
        s.split = l.split;
        s.err = q.err;
        cfg.gridDim = dim3(a.m_tiles * a.n_tiles * l.split);
        cfg.blockDim = dim3(128 + kSplitStore);
        cfg.dynamicSmemBytes = 1024 + (ring > sums ? ring : sums);
        return cudaLaunchKernelEx(&cfg, split_of(l.epilogue), s);
    }
    int busy = q.cut ? q.pairs : q.whole < q.pairs ? q.whole : q.pairs;
    cfg.gridDim = dim3(2 * busy);
    cfg.blockDim = dim3(128 + kPairStore);
    cfg.dynamicSmemBytes = 1024 + ring + out_bytes(l.epilogue);
    return cudaLaunchKernelEx(&cfg, pair_of(l.epilogue, a.a_mn != 0), q);
}

cudaError_t launch_ffn_zero(void *p, size_t bytes, cudaStream_t stream)
{
    zero_kernel<<<1024, 256, 0, stream>>>(static_cast<uint32_t *>(p), bytes / 4);
    return cudaGetLastError();
}

std::vector<const void *> ffn_kernels()
{
    std::vector<const void *> all = {reinterpret_cast<const void *>(zero_kernel)};
    all.push_back(reinterpret_cast<const void *>(pair_of(kFfnStore, true)));
    for (const int e : {kFfnStore, kFfnJoin, kFfnSplit}) {
        all.push_back(reinterpret_cast<const void *>(pair_of(e, false)));
        all.push_back(reinterpret_cast<const void *>(split_of(e)));
    }
    return all;
}

}  // namespace moe
