// moe_int4.cu -- products of a few tokens with 4-bit weights and group scales:
// a linear layer, and the experts of an MoE layer.
//
//   w = s (q - z):  q 0..15, one scale s and zero point z (8 without) per `group` inputs
//   linear:   y = x W^T
//   experts:  as in moe_experts.cu
//
// Work is cut and shared tiles are settled as in moe_experts.cu. A weight is
// repacked once, when it is taken, to tiles of 128 rows x 128 inputs: 8 KB of
// codes, their scales and zero points. A unit of work, and a stage of the
// weights' ring, is two tiles that lie side by side: the gate and the up tile
// of a chunk of inputs, or two chunks of the other products; one copy of 17
// KB each, since a copy's issue costs the producer more than its bytes. Four
// groups of four warps take the tiles in turn (the first tile of a unit falls
// to groups 0 and 2, the second to 1 and 3); a tile of experts with many
// tokens costs more, so their shares are cut by cost. The linear layer, which
// needs no list and no share of another's work, starts its copies before the
// kernel before it is done; the last of the blocks that share a tile adds its
// parts up. A warp has 32 rows of its tile:
//
//  - codes are packed in the order of the MMA's A fragment, so a 16-byte
//    load is four fragments; two or three instructions turn a pair of codes
//    into 16-bit whole numbers q - z, which bf16 and fp16 hold exactly;
//  - mma.sync adds a group's products in fp32, and s times that sum goes to
//    the row's fp32 accumulators: no weight is rounded, and a scale costs
//    one instruction per four sums instead of one per pair of weights;
//  - the second product's token tile has the high and the low part of h, in
//    columns side by side for up to four tokens, else in two tiles that are
//    added to the same sums.
//
// Why warp-level MMA here: at 4 bits a weight the SM has 366 cycles for a
// tile. Decoding takes 224 of them on the integer pipe whatever follows;
// mma.sync takes 131 per 8 tokens from registers the decode has just
// written. The same tile through tensor memory (16-bit weights stored as
// tcgen05's A operand, 128 x 16 x 16 MMAs) was built first and took about
// 1000: each tile passed through four hand-overs between warps.
//
// What bounds it: instructions. A tile of up to 8 tokens costs a scheduler some
// 345 of them (220 decode, multiply and scale; the rest walks the rings) and
// about 450 cycles, 4.9 TB/s of packed weights, 57 % of the DRAM's cycles over
// a whole call; from 17 tokens on the MMAs count. Measured (GB300): experts of
// one token, 8 of 256 of 7168 x 2048, 49 us in the kernel, 62 with the router;
// 41 tokens, 8 of 128 experts of 4096 x 1408, 253 us, 4.4 TB/s; linear
// 28672 x 4096, one row, 18.9 us, 3.3 TB/s; 7168 x 18432, 47 rows, 58 us.
#include <type_traits>

#include "moe_sched.h"

namespace moe {

namespace {

constexpr int kGroups = kInt4Groups;
constexpr int kWorkers = kGroups * 128;
// then a warpgroup for results, a warp that brings weights and two that bring tokens
constexpr int kResults = 128;
constexpr int kThreads = kWorkers + kResults + 96;
constexpr int kCopyWarp = (kWorkers + kResults) / 32;  // brings weights; the next ones tokens
constexpr int kMaxStagesA = kInt4StagesA, kMaxStagesB = kInt4StagesB;
constexpr int kCap = 32;                   // tokens of an entry: 4 column blocks of 8
constexpr int kSideBySide = 4;             // up to so many tokens have both parts of h in one column block

struct Shared {
    uint64_t full_a[kMaxStagesA], empty_a[kMaxStagesA];
    uint64_t full_b[2][kMaxStagesB], empty_b[2][kMaxStagesB];  // a ring for each product
    uint64_t full_s, empty_s;  // the groups' sums of a run
    int abort;
    int active, nmax;
    int issued_a, issued_b[2][2];  // of each product by each warp
    int reset, last;
    int3 totals[kMaxLocal / 32];
    Rests rests[2];
    int cut[4];  // this block's shares: where the first and the second product's begin and end
    // what run_tiles needs; offsets are from the dynamic shared memory's start
    uint32_t ring_a, ring_b, sums;
    int stages, stage_a, stages_b[2], stage_b[2], tile[2], zeros[2], cols, scale_fp16;
};

__shared__ Shared sh;
extern __shared__ uint8_t dyn[];

// Cost of a unit of an entry with this many column blocks. Measured for one to
// four of them 16, 21, 32 and 40 (0.47 to 1.18 us) in the first product, which
// these fit, and 18, 29, 45 and 62 in the second, where they are up to a third
// too low for large entries.
constexpr int kUnitCost = 9, kBlockCost = 8;

// Eight codes to the four registers of an A fragment: pair p has its codes at
// bits 4p and 4p + 16, so a shift and a mask leave a pair; or-ing the exponent
// of 128 (bf16; 1024 in fp16) makes them 128 + q (published for fp16 by Kim et
// al., arXiv 2211.10017). za and zb hold 128 + z twice, for the fragment's rows
// r and r + 8.
template <bool BF16> static __device__ __forceinline__ void decode(uint32_t w, uint32_t za, uint32_t zb, uint32_t *out)
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t v;  // (w >> 4p & mask) | exponent: one instruction after the shift, which two constants in C are not
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(BF16 ? 0x43004300u : 0x64006400u));
        if (BF16)
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[p]) : "r"(v), "r"(p & 1 ? zb : za));
        else
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[p]) : "r"(v), "r"(p & 1 ? zb : za));
    }
}

// Adds one weight tile times NT * 8 tokens (in PLANES parts) to the sums of
// this warp's 32 rows: acc[column block][16-row half][fragment]. SHIFT:
// log2(group / 32). tile: the tile in shared memory; tokens: [PLANES][4][NT * 8][32] 16-bit. meanwhile() is
// called where its loads' latency is hidden.
template <int NT, int SHIFT, int PLANES, bool BF16, class Meanwhile>
static __device__ __forceinline__ void add_tile(float (&acc)[NT][2][4], const uint8_t *tile, int rows32, int lane,
                                                const uint8_t *tokens, bool with_zeros, bool scale_fp16,
                                                Meanwhile meanwhile)
{
    constexpr int kQ = 1 << SHIFT;  // 32-input steps of a group
    // From three column blocks on, a group's sum is scaled in steps of 32 inputs: it then needs registers for one
    // block at a time, and the MMAs take longer than the scaling.
    constexpr bool kSteps = NT >= 3 || kQ == 1;
    const uint4 *const codes = reinterpret_cast<const uint4 *>(tile + rows32 * 2048) + lane;
    const int row = rows32 * 32 + (lane >> 2);
    const uint16_t *const scales = reinterpret_cast<const uint16_t *>(tile + 8192) + row;
    const uint8_t *const zeros = tile + 8192 + (1024 >> SHIFT) + row;
    const uint4 *const tok = reinterpret_cast<const uint4 *>(tokens) + lane;
    constexpr uint32_t one = BF16 ? 0x43004300u : 0x64006400u;
    uint32_t z[4] = {one + 0x00080008u, one + 0x00080008u, one + 0x00080008u, one + 0x00080008u};
    float s[4], c[kSteps ? 1 : NT][2][4];
    uint4 w = codes[0];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (q % kQ == 0 && with_zeros) {
#pragma unroll
            for (int h = 0; h < 4; ++h)  // rows r, r + 8, r + 16, r + 24
                z[h] = one + zeros[(q >> SHIFT) * 128 + h * 8] * 0x00010001u;
        }
        if (kSteps ? q % kQ == 0 : q % kQ == kQ - 1) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t raw = scales[(q >> SHIFT) * 128 + h * 8];
                s[h] = scale_fp16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(raw)))
                                  : __uint_as_float(raw << 16);
            }
        }
        uint32_t f[4][4];  // [2 * sixteen inputs + 16-row half]
        decode<BF16>(w.x, z[0], z[1], f[0]);
        decode<BF16>(w.y, z[2], z[3], f[1]);
        decode<BF16>(w.z, z[0], z[1], f[2]);
        decode<BF16>(w.w, z[2], z[3], f[3]);
        if (q < 3)
            w = codes[(q + 1) * 32];
        else
            meanwhile();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float(&d)[2][4] = c[kSteps ? 0 : nt];
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                const uint4 b = tok[((p * 4 + q) * NT + nt) * 32];
                if (p == 0 && (kSteps || q % kQ == 0)) {
                    mma_16816<BF16, false>(d[0], f[0], b.x, b.y);
                    mma_16816<BF16, false>(d[1], f[1], b.x, b.y);
                } else {
                    mma_16816<BF16, true>(d[0], f[0], b.x, b.y);
                    mma_16816<BF16, true>(d[1], f[1], b.x, b.y);
                }
                mma_16816<BF16, true>(d[0], f[2], b.z, b.w);
                mma_16816<BF16, true>(d[1], f[3], b.z, b.w);
            }
            if (kSteps || q % kQ == kQ - 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float &y = acc[nt][i >> 2][i & 3];
                    y = fmaf(s[(i >> 2) * 2 + ((i >> 1) & 1)], d[i >> 2][i & 3], y);
                }
            }
        }
    }
}

// Where a worker warp is in the rings, in one word.
struct Place {
    Cursor a, b;          // its group's next unit
    int turn;             // units until then
    uint32_t ready;       // whether that unit has landed
    uint32_t run_parity;  // of empty_s
    bool run;

    __device__ __forceinline__ explicit Place(uint32_t w)
        : turn(w >> 12 & 1), ready(w >> 13 & 1), run_parity(w >> 14 & 1), run(w >> 15)
    {
        a.s = w & 31;
        a.parity = w >> 5 & 1;
        b.s = w >> 6 & 31;
        b.parity = w >> 11 & 1;
    }
    __device__ __forceinline__ uint32_t word() const
    {
        return a.s | a.parity << 5 | b.s << 6 | b.parity << 11 | turn << 12 | ready << 13 | run_parity << 14 |
               uint32_t(run) << 15;
    }
    // Before the first unit of a product: group pairs take the units in turn. The weights' ring goes on.
    static __device__ __forceinline__ uint32_t first(int turn) { return turn | turn << 6 | turn << 12 | 1 << 14 | 1 << 15; }
    static __device__ __forceinline__ uint32_t second(uint32_t w)
    {
        return (w & ~(63u << 6) & ~(1u << 13)) | (w >> 12 & 1) << 6;
    }
};

// A worker warp's tiles of a run of `units`, of which its group has one in the
// first `valid`; its sums go to shared memory. PLANES: 0 for the first product
// (PAIR: the unit is a gate and an up tile with one token tile), else the parts
// of h in a token tile of the second. Not inlined: among thirty of them and the
// rest of the kernel the compiler kept some fifteen of the loop's values in
// memory, each time round.
template <int NT, int SHIFT, int PLANES, bool PAIR, bool BF16>
static __device__ __noinline__ uint32_t run_tiles(uint32_t word, int units, int valid)
{
    constexpr bool SECOND = PLANES != 0;
    constexpr uint32_t empty_a = offsetof(Shared, empty_a) - offsetof(Shared, full_a);
    constexpr uint32_t empty_b = offsetof(Shared, empty_b) - offsetof(Shared, full_b);
    Place at(word);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = warp >> 2, rows32 = warp & 3, tile = grp & 1;
    const int stages = sh.stages, stages_b = sh.stages_b[SECOND], stage_a = sh.stage_a, stage_b = sh.stage_b[SECOND];
    const uint8_t *const ring_a = dyn + sh.ring_a + tile * sh.tile[SECOND];
    // rows of 32 inputs and one token are 64 bytes: the second chunk's token tile
    const uint8_t *const ring_b = dyn + sh.ring_b + (PAIR ? 0 : tile * NT * 8 * 256 * (SECOND ? PLANES : 1));
    const bool with_zeros = sh.zeros[SECOND], scale_fp16 = sh.scale_fp16;
    volatile int *const abort = &sh.abort;
    float acc[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[nt][i >> 2][i & 3] = 0.0f;
    int turn = at.turn;
    for (; turn < units; turn += 2) {
        const uint32_t fa = smem_u32(&sh.full_a[at.a.s]), fb = smem_u32(&sh.full_b[SECOND][at.b.s]);
        if (!mbar_wait2_warp(at.ready, fa, at.a.parity, fb, at.b.parity, abort, kWaitFullA, kWaitFullB)) {
            at.run = false;
            return at.word();
        }
        const uint8_t *const weights = ring_a + at.a.s * stage_a, *const tokens = ring_b + at.b.s * stage_b;
        at.a.advance(2, stages);  // the group's next unit
        at.b.advance(2, stages_b);
        auto peek = [&] {
            at.ready = mbar_peek2(smem_u32(&sh.full_a[at.a.s]), at.a.parity, smem_u32(&sh.full_b[SECOND][at.b.s]),
                                  at.b.parity);
        };
        if (PAIR || turn < valid)
            add_tile<NT, SHIFT, SECOND ? PLANES : 1, BF16>(acc, weights, rows32, lane, tokens, with_zeros, scale_fp16, peek);
        else
            peek();
        __syncwarp();
        mbar_arrive2_if(lane == 0, fa + empty_a, fb + empty_b);
    }
    at.turn = turn - units;
    // the sums of the run before have been read
    at.run = mbar_wait_warp(smem_u32(&sh.empty_s), at.run_parity, abort, kWaitEmptyD);
    at.run_parity ^= 1;
    if (at.run) {
        float *const mine = reinterpret_cast<float *>(dyn + sh.sums) + (grp * sh.cols + (lane & 3) * 2) * kInt4SumStride +
                            rows32 * 32 + (lane >> 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mine[(nt * 8 + (i & 1)) * kInt4SumStride + (i >> 1) * 8] = acc[nt][i >> 2][i & 3];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sh.full_s));
    }
    return at.word();
}

template <bool LINEAR, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) int4_kernel(const __grid_constant__ Int4Args a)
{
    const uint32_t dyn0 = smem_u32(dyn), base = (dyn0 + 127u) & ~127u;
    // dynamic shared memory: y's accumulators, lists, the groups' sums, the rings
    float *const acc_y = reinterpret_cast<float *>(dyn + (base - dyn0));  // [T][128], of the second product
    const Lists li(acc_y + (LINEAR ? 0 : a.T * kTileRows), acc_y, a.E, a.P);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int G = gridDim.x, blk = blockIdx.x;
    volatile int *const abort = &sh.abort;

    // With up to 8 tokens every expert's token tile is all of x: a sum's column is the token. Else the tokens are
    // gathered, half the inputs by each of two warps: a gather of four rows of 64 bytes costs its thread 85 cycles,
    // and a unit of an expert with five tokens would take 10 % longer.
    const bool whole = LINEAR || a.T <= 8;

    // The weights' warp sets up its own barriers: in the linear layer, whose weights and share need no list and no
    // earlier kernel, it starts before the block has met.
    if (warp == kCopyWarp && lane < kMaxStagesA) {
        mbar_init(smem_u32(&sh.full_a[lane]), 1);
        mbar_init(smem_u32(&sh.empty_a[lane]), 8);
    } else if (tid >= 32 && tid < 32 + 2 * kMaxStagesB) {
        mbar_init(smem_u32(&sh.full_b[0][tid - 32]), !whole && tid < 32 + kMaxStagesB ? 2 : 1);
        mbar_init(smem_u32(&sh.empty_b[0][tid - 32]), 8);
    } else if (tid == 64) {
        mbar_init(smem_u32(&sh.full_s), kWorkers / 32);
        mbar_init(smem_u32(&sh.empty_s), kResults / 32);
        sh.abort = sh.reset = sh.rests[0].n = sh.rests[1].n = sh.issued_a = 0;
        for (int i = 0; i < 4; ++i)
            sh.issued_b[i >> 1][i & 1] = 0;
        tma_prefetch_map(&a.mx);
    }
    mbar_init_fence();
    if (!LINEAR) {
        build_lists(a, li, sh, tid, kThreads, kCap);
        __syncthreads();
    }
    // the linear layer: one "expert" whose tokens are the rows of x, or two with half of them each
    const int rows = a.box_bytes / 512;  // int4_linear_rows
    const int A = LINEAR ? (a.T > rows ? 2 : 1) : sh.active, nmax = LINEAR ? rows : sh.nmax;

    if (A == 0) {
        clear_out(a, blk, G, tid, kThreads);
        return;
    }

    // units along the inputs; the last one of an odd number of chunks is half empty
    const int ku1 = LINEAR ? (a.kc1 + 1) / 2 : a.kc1, ku2 = (a.kc2 + 1) / 2;
    const int total1 = A * a.mt1 * ku1;
    // Costs: of a unit of entry i, of a unit of every entry before it
    const auto cost = [&](int i) { return kUnitCost + kBlockCost * (li.blocks[i + 1] - li.blocks[i]); };
    const auto costs = [&](int i) { return static_cast<uint32_t>(kUnitCost * i + kBlockCost * li.blocks[i]); };
    const Shares shares(total1, G);  // of the linear layer, whose units are alike
    const uint32_t units1 = a.mt1 * ku1, units2 = ku2;  // of an entry, or of one in a row tile
    const auto cost_shares = [&](bool second) {
        return CostShares(costs(A) * (second ? a.mt2 * units2 : units1), kUnitCost + kBlockCost * ((nmax + 7) / 8), G);
    };
    if (!LINEAR && warp < 4) {  // a warp finds one end of a share
        const bool second = warp & 2;
        const int b = blk + (warp & 1);
        const uint32_t units = second ? units2 : units1;
        if (nmax <= 8) {  // all units cost the same
            sh.cut[warp] = CostShares(A * units * (second ? a.mt2 : 1), 1, G).begin(b);
        } else {
            const uint32_t all = units * costs(A), place = cost_shares(second).begin(b), outer = place / all;
            const uint32_t rest = place - outer * all;
            int i = 0;  // entries that begin there or before
#pragma unroll 1
            for (int k = lane; k < A; k += 32)
                i += rest >= units * costs(k) ? 1 : 0;
            i = __reduce_add_sync(~0u, i) - 1;
            sh.cut[warp] = (outer * A + i) * units + (rest - units * costs(i) + cost(i) - 1) / cost(i);
        }
    }
    const int pairs = LINEAR ? a.T : li.offset[A];
    const Int4Layout lay = int4_layout(LINEAR, a.smem - static_cast<int>(base - dyn0), a.fixed_bytes, a.stage_a, nmax);
    const int cols = lay.cols, stages = lay.stages, stage_b1 = lay.stage_b[0], stage_b2 = lay.stage_b[1];
    const int stages_b1 = lay.stages_b[0], stages_b2 = lay.stages_b[1];
    float *const sums = reinterpret_cast<float *>(dyn + (base - dyn0) + lay.sums);  // [group][column][kInt4SumStride]
    const uint32_t ring_a = base + lay.ring_a, ring_b = base + lay.ring_b;
    if (tid == kThreads - 1) {
        sh.ring_a = ring_a - dyn0;
        sh.ring_b = ring_b - dyn0;
        sh.sums = base + lay.sums - dyn0;
        sh.stages = stages;
        sh.stage_a = a.stage_a;
        sh.stages_b[0] = stages_b1;
        sh.stages_b[1] = stages_b2;
        sh.stage_b[0] = stage_b1;
        sh.stage_b[1] = stage_b2;
        sh.tile[0] = a.tile1;
        sh.tile[1] = a.tile2;
        sh.zeros[0] = a.zeros1;
        sh.zeros[1] = a.zeros2;
        sh.cols = cols;
        sh.scale_fp16 = a.scale_fp16;
    }
    if (!LINEAR)
        __syncthreads();
    const int begin1 = LINEAR ? shares.begin(blk) : sh.cut[0], end1 = LINEAR ? shares.begin(blk + 1) : sh.cut[1];
    const int begin2 = LINEAR ? 0 : sh.cut[2], end2 = LINEAR ? 0 : sh.cut[3];
    // h: per entry and chunk a tile [2 parts][4][tokens][32], tokens a multiple of 8; or, for up to kSideBySide
    // tokens, [4][8][32] with the low parts in rows 4 to 7
    const auto h_entry = [&](int i) { return a.h + static_cast<size_t>(li.blocks[i] * 8) * a.h_stride; };

    // tiles of w1: [matrix][row tile][chunk]; gate and up tiles side by side
    const int tiles1 = LINEAR ? a.kc1 : 2 * a.kc1;
    const auto w1_tiles = [&](int expert, int m, int k) {
        return a.w1 + ((static_cast<size_t>(expert) * a.mt1 + m) * tiles1 + 2 * k) * a.tile1;
    };
    int ahead = 0;  // weight tiles of the linear layer on their way before the block has met
    if (LINEAR) {
        pdl_launch_next();
        if (warp == kCopyWarp) {
            __syncwarp();
            if (elect_one()) {
                const uint64_t policy = policy_evict_first();
                for (Walk w(begin1, end1, ku1, a.mt1, false); ahead < stages && w.more(); w.next()) {
                    const uint8_t *src = w1_tiles(0, w.m, w.k);
                    for (int k = w.k; ahead < stages && k < w.k + w.len; ++k, ++ahead, src += 2 * a.tile1) {
                        const uint32_t bar = smem_u32(&sh.full_a[ahead]), bytes = 2 * k + 1 < tiles1 ? 2 * a.tile1 : a.tile1;
                        mbar_expect(bar, bytes);
                        bulk_load(ring_a + ahead * a.stage_a, src, bytes, bar, policy);
                    }
                }
            }
        } else {
            if (tid == 96) {
                li.expert[0] = li.expert[1] = 0;
                li.offset[0] = 0;
                li.offset[1] = static_cast<unsigned short>(min(a.T, rows));
                li.offset[A] = static_cast<unsigned short>(a.T);
            }
            pdl_wait();  // x, y, the parts and the counters are the earlier kernel's until it is done
        }
        __syncthreads();
    }

    if (warp == kCopyWarp && elect_one()) {
        // ---- weight tiles ----
        const uint64_t policy = policy_evict_first();
        Cursor at;
        int issued = 0;
        bool run = true;
        auto load = [&](const uint8_t *src, uint32_t bytes) {
            if (issued >= ahead) {
                if (!mbar_wait(smem_u32(&sh.empty_a[at.s]), at.parity ^ 1, abort, kWaitEmptyA))
                    return false;
                const uint32_t bar = smem_u32(&sh.full_a[at.s]);
                mbar_expect(bar, bytes);
                bulk_load(ring_a + at.s * a.stage_a, src, bytes, bar, policy);
            }
            at.next(stages);
            ++issued;
            return true;
        };
        for (Walk w(begin1, end1, ku1, a.mt1, false); run && w.more(); w.next()) {
            const uint8_t *src = w1_tiles(li.expert[w.i], w.m, w.k);
            for (int k = w.k; run && k < w.k + w.len; ++k, src += 2 * a.tile1)
                run = load(src, 2 * k + 1 < tiles1 ? 2 * a.tile1 : a.tile1);
        }
        for (Walk w(begin2, end2, ku2, A, true); run && w.more(); w.next()) {
            const uint8_t *src = a.w2 + ((static_cast<size_t>(li.expert[w.i]) * a.mt2 + w.m) * a.kc2 + 2 * w.k) * a.tile2;
            for (int k = w.k; run && k < w.k + w.len; ++k, src += 2 * a.tile2)
                run = load(src, 2 * k + 1 < a.kc2 ? 2 * a.tile2 : a.tile2);
        }
        sh.issued_a = issued;
    } else if (warp > kCopyWarp && elect_one()) {
        // ---- token tiles ----
        const int half = warp - kCopyWarp - 1;
        if (LINEAR)
            fence_async_global();  // what the kernel before stored from registers is read by copies
        Cursor at;
        int issued = 0;
        bool run = true;
        uint32_t dst = 0, bar = 0;
        auto acquire = [&](int product, uint32_t bytes) {
            if (!mbar_wait(smem_u32(&sh.empty_b[product][at.s]), at.parity ^ 1, abort, kWaitEmptyB))
                return false;
            bar = smem_u32(&sh.full_b[product][at.s]);
            dst = ring_b + at.s * (product ? stage_b2 : stage_b1);
            mbar_expect(bar, bytes);
            at.next(product ? stages_b2 : stages_b1);
            ++issued;
            return true;
        };
        for (Walk w(begin1, end1, ku1, a.mt1, false); (half == 0 || !whole) && run && w.more(); w.next()) {
            const int n = li.count(w.i), n8 = (n + 7) & ~7, off = li.offset[w.i];
            const unsigned char *const tok = li.token + off;
            const uint32_t bytes = whole ? a.box_bytes : ((n + 3) & ~3) * 128;
            for (int k = w.k; k < w.k + w.len && (run = acquire(0, bytes)); ++k) {
                if (whole) {  // [inputs / 32][tokens][32]
                    tma_load_box(dst, &a.mx, bar, 0, LINEAR ? off : 0, LINEAR ? 8 * k : 4 * k);
                } else {
                    for (int j = 0; j < n; j += 4) {  // short of a fourth row: the last one again
                        const int r0 = tok[j], r1 = tok[min(j + 1, n - 1)], r2 = tok[min(j + 2, n - 1)],
                                  r3 = tok[min(j + 3, n - 1)];
                        for (int q = 2 * half; q < 2 * half + 2; ++q)
                            tma_gather4(dst + (q * n8 + j) * 64, &a.mx, bar, k * 128 + q * 32, r0, r1, r2, r3);
                    }
                }
            }
        }
        sh.issued_b[0][half] = issued;
        if (run && half == 0 && begin2 < end2) {  // h is complete
            run = wait_count(a.done, a.mt1 * pairs, abort, kWaitDone);
            fence_async_proxy();
        }
        issued = 0;
        at = Cursor();
        const uint64_t policy = policy_evict_first();
        for (Walk w(begin2, end2, ku2, A, true); half == 0 && run && w.more(); w.next()) {
            const int n = li.count(w.i);
            const uint32_t chunk = n <= kSideBySide ? 2048 : ceil_div(n, 8) * 4096;
            const uint8_t *src = reinterpret_cast<const uint8_t *>(h_entry(w.i)) + static_cast<size_t>(2 * w.k) * chunk;
            for (int k = w.k; run && k < w.k + w.len; ++k, src += 2 * chunk) {
                const uint32_t bytes = 2 * k + 1 < a.kc2 ? 2 * chunk : chunk;
                run = acquire(1, bytes);
                if (run)
                    bulk_load(dst, src, bytes, bar, policy);
            }
        }
        sh.issued_b[1][half] = issued;
    } else if (warp < kWorkers / 32) {
        // ---- products ----
        const int tile = warp >> 2 & 1;  // of a unit
        uint32_t at = Place::first(warp >> 3);
        // A run of `units` from unit k on, kc chunks along the inputs.
        auto by_group = [&](auto blocks, auto planes, int units, int k, int kc) {
            constexpr int NT = decltype(blocks)::value, PLANES = decltype(planes)::value;
            constexpr bool PAIR = !LINEAR && PLANES == 0;
            const int shift = PLANES ? a.shift2 : a.shift1, valid = (kc - tile + 1) / 2 - k;
            if (shift == 0)
                at = run_tiles<NT, 0, PLANES, PAIR, BF16>(at, units, valid);
            else if (shift == 1)
                at = run_tiles<NT, 1, PLANES, PAIR, BF16>(at, units, valid);
            else
                at = run_tiles<NT, 2, PLANES, PAIR, BF16>(at, units, valid);
        };
        auto run_products = [&](auto planes, int n, int units, int k, int kc) {
            if (n <= 8)
                by_group(std::integral_constant<int, 1>{}, planes, units, k, kc);
            else if (n <= 16)
                by_group(std::integral_constant<int, 2>{}, planes, units, k, kc);
            else if (n <= 24)
                by_group(std::integral_constant<int, 3>{}, planes, units, k, kc);
            else
                by_group(std::integral_constant<int, 4>{}, planes, units, k, kc);
        };
        for (Walk w(begin1, end1, ku1, a.mt1, false); Place(at).run && w.more(); w.next())
            run_products(std::integral_constant<int, 0>{}, LINEAR ? nmax : li.count(w.i), w.len, w.k, a.kc1);
        if constexpr (!LINEAR) {
            at = Place::second(at);
            for (Walk w(begin2, end2, ku2, A, true); Place(at).run && w.more(); w.next())
                if (li.count(w.i) <= kSideBySide)
                    by_group(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{}, w.len, w.k, a.kc2);
                else
                    run_products(std::integral_constant<int, 2>{}, li.count(w.i), w.len, w.k, a.kc2);
        }
    } else if (warp < (kWorkers + kResults) / 32) {
        // ---- results: a thread is a row of a tile ----
        const int row = tid - kWorkers;
        uint32_t parity = 0;  // of full_s
        bool run = true;
        // Waits for a run's sums. The four warps leave together, or not at all.
        auto sums_ready = [&] {
            const bool ok = named_all(2, kResults, mbar_wait(smem_u32(&sh.full_s), parity, abort, kWaitFullD));
            parity ^= 1;
            return ok;
        };
        auto sums_read = [&] {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sh.empty_s));
        };
        // Four columns of the sums from column c[0] .. c[3] on, this thread's row: of the even (0) or odd (1)
        // groups, or all. The loads of all four are in flight at once.
        auto sum_half = [&](const int (&c)[4], int odd, float (&v)[4]) {
            const float *const s = sums + odd * cols * kInt4SumStride + row;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = s[c[i] * kInt4SumStride] + s[(2 * cols + c[i]) * kInt4SumStride];
        };
        auto sum_all = [&](const int (&c)[4], float (&v)[4]) {
            float x[4];
            sum_half(c, 0, v);
            sum_half(c, 1, x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] += x[i];
        };

        // As in moe_experts.cu: tiles shared with other blocks are settled after a product's last run.
        auto arrive = [&](const Rests &rests, int *counters, bool second) {
            named_sync(1, kResults);
            if (row < rests.n)
                add_acq_rel(counters + (second ? rests.of[row].m : rests.of[row].i * a.mt1 + rests.of[row].m), 1);
        };
        auto parts_written = [&](int *counter, const Split &sp) {
            return named_all(2, kResults, row != 0 || wait_count(counter, sp.parts(), abort, kWaitOther));
        };
        // h of these columns of a tile goes out to the copies of every block.
        auto announce = [&](int columns) {
            fence_async_proxy();
            named_sync(1, kResults);
            if (row == 0)
                add_acq_rel(a.done, columns);
        };
        // column j of row tile m: h, or y of the linear layer
        auto result = [&](int i, int m, int j, float gate, float up) {
            const int col = m * kTileRows + row;
            if (LINEAR) {
                uint16_t *const p = static_cast<uint16_t *>(a.out) + (li.offset[i] + j) * a.out_stride + col;
                if (col < a.I &&
                    EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.I)))
                    *p = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(gate))
                              : __half_as_ushort(__float2half_rn(gate));
            } else {  // rows past the intermediate size have scales of 0: their h is 0, as the token tiles need
                const int n = li.count(i), n8 = (n + 7) & ~7;
                const bool side = n <= kSideBySide;
                __nv_bfloat16 *const p = h_entry(i) + static_cast<size_t>(m) * n8 * (side ? 128 : 256) +
                                         ((row >> 5) * n8 + j) * 32 + (row & 31);
                split(swiglu(gate, up), p[0], p[side ? kSideBySide * 32 : n8 * 128]);
            }
        };
        // A run's part: the block's second slot unless it is the first run of its share.
        auto part_of = [&](bool first) {
            return a.part + static_cast<size_t>(2 * blk + (first ? 0 : 1)) * a.part_floats + row;
        };

        int announced = 0;  // columns of h that are written and not yet announced
        for (Walk w(begin1, end1, ku1, a.mt1, false); w.more(); w.next()) {
            const int n = li.count(w.i);
            const unsigned char *const tok = li.token + li.offset[w.i];
            const bool shared = w.k != 0 || w.len != ku1, first = w.left == end1 - begin1;
            run = sums_ready();
            if (!run)
                break;
            float *const part = part_of(first);
            for (int j = 0; j < n; j += 4) {
                int c[4];  // the sums' columns
                float g[4], u[4] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = min(j + i, n - 1);
                    c[i] = !LINEAR && whole ? tok[k] : k;
                }
                if (LINEAR) {
                    sum_all(c, g);
                } else {
                    sum_half(c, 0, g);
                    sum_half(c, 1, u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (j + i >= n)
                        break;
                    if (shared) {
                        part[(j + i) * kTileRows] = g[i];
                        if (!LINEAR)
                            part[(n + j + i) * kTileRows] = u[i];
                    } else {
                        result(w.i, w.m, j + i, g[i], u[i]);
                    }
                }
            }
            sums_read();
            if (!shared)
                announced += n;
            else if (row == 0)
                sh.rests[0].of[sh.rests[0].n++] = Rest{w.i, w.m};
        }
        if (LINEAR && run) {  // the block whose part of a tile is the last adds them up: no block waits for another
            named_sync(1, kResults);
            for (int r = 0; r < sh.rests[0].n; ++r) {
                const int i = sh.rests[0].of[r].i, m = sh.rests[0].of[r].m, n = li.count(i), tile = i * a.mt1 + m;
                const Split sp(shares, tile * ku1, ku1);
                if (row == 0)
                    sh.last = add_acq_rel(a.tiles + tile, 1) == sp.parts() - 1;
                named_sync(1, kResults);
                for (int j = 0; sh.last && j < n; j += 4) {
                    float y[4];
                    sum_parts<4>(a.part + j * kTileRows + row, a.part_floats, sp, n - j, y);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (j + c < n)
                            result(i, m, j + c, y[c], 0.0f);
                }
                named_sync(1, kResults);
            }
        }
        if (!LINEAR && run) {
            arrive(sh.rests[0], a.tiles, false);
            for (int r = 0; run && r < sh.rests[0].n; ++r) {
                const int i = sh.rests[0].of[r].i, m = sh.rests[0].of[r].m, n = li.count(i);
                const uint32_t first = costs(i) * units1 + m * ku1 * cost(i);
                const Split sp(cost_shares(false), first, first + (ku1 - 1) * cost(i), first - cost(m > 0 || i == 0 ? i : i - 1));
                const int lo = sp.column(n, blk), hi = sp.column(n, blk + 1);
                if (lo == hi)
                    continue;
                run = parts_written(a.tiles + i * a.mt1 + m, sp);
                for (int j = lo; run && j < hi; j += 4) {
                    float v[8];  // gate, up
                    sum_parts<8>(a.part + j * kTileRows + row, a.part_floats, sp, hi - j, v, n * kTileRows);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (j + c < hi)
                            result(i, m, j + c, v[c], v[4 + c]);
                }
                announced += hi - lo;
            }
            if (run && announced > 0)
                announce(announced);
        }

        const int group = LINEAR ? 1 : A * ku2;
        auto store_y = [&](int m, int t, float r) {
            const int col = m * kTileRows + row;
            __nv_bfloat16 *const p = static_cast<__nv_bfloat16 *>(a.out) + t * a.out_stride + col;
            if (col < a.H && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
                *p = __float2bfloat16_rn(r);
        };
        for (Walk w(begin2, end2, ku2, A, true); !LINEAR && run && w.more();) {
            const int m = w.m, i0 = w.i;
            const bool first = w.left == end2 - begin2;
            bool shared = w.i != 0 || w.k != 0;  // an earlier block began this row tile
            for (int t = 0; t < a.T; ++t)  // a thread's own row: no barrier
                acc_y[t * kTileRows + row] = 0.0f;
            for (; w.more() && w.m == m; w.next()) {
                const int off = li.offset[w.i], n = li.count(w.i);
                run = sums_ready();
                if (!run)
                    break;
                for (int j = 0; j < n; j += 4) {
                    int c[4];
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = min(j + i, n - 1);
                    sum_all(c, v);
                    if (n <= kSideBySide) {  // the low parts' columns
                        float x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            c[i] += kSideBySide;
                        sum_all(c, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] += x[i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j + i < n) {  // a token is in one column of an entry
                            float *const y = acc_y + li.token[off + j + i] * kTileRows + row;
                            *y = fmaf(li.weight[off + j + i], v[i], *y);
                        }
                }
                sums_read();
            }
            if (!run)
                break;
            shared = shared || (!w.more() && end2 != (m + 1) * group);  // a later block ends it
            if (shared) {
                float *const part = part_of(first);
                for (int t = 0; t < a.T; ++t)
                    part[t * kTileRows] = acc_y[t * kTileRows + row];
                if (row == 0)
                    sh.rests[1].of[sh.rests[1].n++] = Rest{i0, m};
            } else {
                for (int t = 0; t < a.T; ++t)
                    store_y(m, t, acc_y[t * kTileRows + row]);
            }
        }
        if (!LINEAR && run) {
            int *const counters = a.tiles + 2 * a.E * a.mt1;
            arrive(sh.rests[1], counters, true);
            for (int r = 0; run && r < sh.rests[1].n; ++r) {
                const int m = sh.rests[1].of[r].m;
                const uint32_t one = costs(A) * units2, first = one * m;
                const Split sp(cost_shares(true), first, first + one - cost(A - 1), first - cost(A - 1));
                const int lo = sp.column(a.T, blk), hi = sp.column(a.T, blk + 1);
                if (lo == hi)
                    continue;
                run = parts_written(counters + m, sp);
                for (int t = lo; run && t < hi; t += 4) {
                    float y[4];
                    sum_parts<4>(a.part + t * kTileRows + row, a.part_floats, sp, hi - t, y);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (t + c < hi)
                            store_y(m, t + c, y[c]);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();

    if (sh.abort) {  // copies in flight land before the block's memory is given back
        if (tid == 0) {
            for (int i = max(0, sh.issued_a - stages); i < sh.issued_a; ++i)
                mbar_wait(smem_u32(&sh.full_a[i % stages]), (i / stages) & 1, nullptr, kWaitOther);
            for (int product = 0; product < 2; ++product) {
                const int n = product ? stages_b2 : stages_b1, i0 = sh.issued_b[product][0], i1 = sh.issued_b[product][1];
                const int both = product || whole ? max(i0, i1) : min(i0, i1);
                for (int i = max(0, max(i0, i1) - n); i < max(i0, i1); ++i) {
                    const uint32_t bar = smem_u32(&sh.full_b[product][i % n]);
                    if (i >= both)  // for the warp that gave up before
                        mbar_arrive(bar);
                    mbar_wait(bar, (i / n) & 1, nullptr, kWaitOther);
                }
            }
            atomicAdd_system(a.err + sh.abort, 1u);
            __threadfence_system();
            atomicAdd_system(a.err, 1u);
        }
        __syncthreads();
    }

    if (tid == 0)
        sh.reset = add_acq_rel(a.leaving, 1) == G - 1;
    __syncthreads();
    if (sh.reset) {
        for (int i = tid; i < A * a.mt1; i += kThreads)
            a.tiles[i] = 0;
        for (int i = tid; !LINEAR && i < a.mt2; i += kThreads)
            a.tiles[2 * a.E * a.mt1 + i] = 0;
        if (tid == 0)
            *a.done = *a.leaving = 0;
    }
}

// One thread per 32 codes of a tile. Codes: [4 x 32 rows][4 x 32 inputs][lane][4 words];
// word 2 s + f of lane 4 g + t is the A fragment of rows 16 f + g and + 8, inputs 8 t + 4 s
// .. + 3 (the MMA's sixteen inputs are any sixteen, the token tiles are read in the same
// order). Then scales and zero points [groups][128 rows]. Rows and inputs outside the
// matrix become codes of 0 with a scale of 0.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int lane = static_cast<int>(id & 31), q = static_cast<int>((id >> 5) & 3), rb = static_cast<int>((id >> 7) & 3);
    const long long tile = id >> 9;
    if (tile >= a.mats * a.mt * a.kc)
        return;
    const long long mat = tile / (static_cast<long long>(a.mt) * a.kc);
    const int m = static_cast<int>(tile / a.kc - mat * a.mt), kc = static_cast<int>(tile % a.kc);
    const int k = kc * 128 + q * 32 + (lane & 3) * 8;  // cols is a multiple of 32
    uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
    for (int half = 0; half < 4; ++half) {  // rows g, g + 8 of fragment 0, then of fragment 1
        const int r = m * 128 + rb * 32 + half * 8 + (lane >> 2);
        uint32_t in = 0;  // the row's 8 codes from k on
        if (r < a.rows && k < a.cols) {
            const uint8_t *const p = a.codes + (mat * a.rows + r) * (a.cols / 2) + k / 2;
            in = p[0] | p[1] << 8 | p[2] << 16 | static_cast<uint32_t>(p[3]) << 24;
        }
        const int f = half >> 1, low = half & 1;  // fragment; its row r (0) or r + 8 (1)
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // input 4 s + 2 v + e: word 2 s + f, pair 2 v + low, element e
            const int s = c >> 2, v = (c >> 1) & 1, e = c & 1;
            word[2 * s + f] |= ((in >> (4 * c)) & 15u) << ((2 * v + low) * 4 + e * 16);
        }
    }
    const long long to = a.pairs ? ((mat / 2 * a.mt + m) * a.kc + kc) * 2 + mat % 2 : tile;
    uint8_t *const dst = a.dst + to * a.tile_bytes;
    *reinterpret_cast<uint4 *>(dst + ((rb * 4 + q) * 32 + lane) * 16) = make_uint4(word[0], word[1], word[2], word[3]);
    const int groups = 128 / a.group, row = rb * 32 + lane, r = m * 128 + row;
    if (q < groups) {
        const int kg = kc * 128 + q * a.group;
        const bool in = r < a.rows && kg < a.cols;
        const long long at = (mat * a.rows + r) * (a.cols / a.group) + kg / a.group;
        reinterpret_cast<uint16_t *>(dst + 8192)[q * 128 + row] = in ? a.scales[at] : 0;
        if (a.zeros)
            (dst + 8192 + groups * 256)[q * 128 + row] = in ? (a.zeros[at] & 15) : 0;
    }
}

}  // namespace

int int4_tile_bytes(int group, bool zeros)
{
    return 8192 + 128 / group * 256 + (zeros ? 128 / group * 128 : 0);
}

size_t int4_part_floats(int T, bool linear)
{
    const int n = T < kCap ? T : kCap;  // columns of an entry, gate and up, or tokens of a row tile of y
    const int cols = linear ? n : (2 * n > T ? 2 * n : T);
    return static_cast<size_t>(cols) * kTileRows;
}

size_t int4_h_rows(int T, int K, int E)
{
    // an entry's rows are rounded up to a multiple of 8: 7 more for each of up to two entries per expert
    const int pairs = T * K, entries = pairs < 2 * E ? pairs : 2 * E;
    return static_cast<size_t>(pairs) + 7 * static_cast<size_t>(entries) + 8;
}

int int4_linear_rows(int T)
{
    const int n = T > kCap ? (T + 1) / 2 : T;
    return (n + 7) & ~7;
}

size_t int4_smem(Int4Args *a, bool linear)
{
    a->fixed_bytes = (linear ? 0 : a->T * kTileRows * 4) + static_cast<int>(lists_bytes(a->E, a->P));
    a->shift1 = a->group1 == 32 ? 0 : a->group1 == 64 ? 1 : 2;
    a->shift2 = a->group2 == 32 ? 0 : a->group2 == 64 ? 1 : 2;
    a->stage_a = 2 * (a->tile1 > a->tile2 ? a->tile1 : a->tile2);
    a->part_floats = static_cast<int>(int4_part_floats(a->T, linear));
    a->smem = (kSmemMax - static_cast<int>(sizeof(Shared)) - 64) & ~127;  // all of it: the rings take the rest
    return a->smem;
}

namespace {

using Kernel = void (*)(Int4Args);

Kernel kernel_of(bool linear, bool bf16)
{
    return !linear ? int4_kernel<false, true> : bf16 ? int4_kernel<true, true> : int4_kernel<true, false>;
}

}  // namespace

cudaError_t int4_setup(bool linear)
{
    cudaError_t ce = cudaSuccess;
    for (const bool bf16 : {true, false})
        if (ce == cudaSuccess && (linear || bf16))
            ce = cudaFuncSetAttribute(kernel_of(linear, bf16), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSmemMax - 64 - static_cast<int>(sizeof(Shared)));
    return ce;
}

cudaError_t launch_int4(const Int4Args &a, bool linear, bool bf16, int grid, size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    if (linear) {  // weights are fetched while the kernel before is finishing
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
    } else {  // the blocks wait for one another's h
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel_of(linear, bf16), a);
}

cudaError_t launch_pack(const PackArgs &a, cudaStream_t stream)
{
    const long long threads = a.mats * a.mt * a.kc * 512;
    pack_kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

std::vector<const void *> int4_kernels()
{
    return {reinterpret_cast<const void *>(int4_kernel<false, true>), reinterpret_cast<const void *>(int4_kernel<true, true>),
            reinterpret_cast<const void *>(int4_kernel<true, false>), reinterpret_cast<const void *>(pack_kernel)};
}

}  // namespace moe
