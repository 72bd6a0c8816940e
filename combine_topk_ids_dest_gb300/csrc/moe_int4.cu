// moe_int4.cu -- products of a few tokens with 4-bit weights and group scales:
// a linear layer, and the experts of an MoE layer.
//
//   w = s (q - z):  q 0..15, one scale s and zero point z (8 without) per `group` inputs
//   linear:   y = x W^T
//   experts:  as in moe_experts.cu
//
// The kernel is that of moe_experts.cu, with the weights' way to the MMA
// lengthened by one step. A stage of the ring is a tile of 128 rows x 128
// inputs, repacked once when the weight was taken: 8 KB of codes, its scales
// and zero points. Two warpgroups (a thread is a weight row) turn codes into
// q - z, whole numbers that 16 bits hold exactly, and store them to tensor
// memory as the MMA's A operand: shared memory could not carry the 16-bit
// tile's write and read at this rate. Scales are applied to sums, not to
// weights: each group's sum is an accumulator of its own, and two more
// warpgroups add s times it to fp32 registers. So no weight is rounded.
#include "moe_sched.h"

namespace moe {

namespace {

constexpr int kThreads = 640;      // warps: weights, MMA, tokens, -, 8 x codes, 8 x results
constexpr int kMaxStagesA = 24;
constexpr int kMaxStagesB = 16;
constexpr int kTmemA = 4;          // 16-bit weight tiles in tensor memory, 64 columns each
constexpr int kMaxSums = 16;       // accumulators in tensor memory, in the other 256 columns
constexpr int kResults = 256;      // threads of the result warps

struct Shared {
    uint64_t full_a[kMaxStagesA], empty_a[kMaxStagesA];
    uint64_t full_b[kMaxStagesB], empty_b[kMaxStagesB];
    uint64_t full_t[kTmemA], empty_t[kTmemA];
    uint64_t full_d[kMaxSums], empty_d[kMaxSums];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int active, nmax;
    int issued_a, issued_b;
    int reset;
    Rests rests[2];  // of the two products
};

// Eight codes to four pairs q - z. Code 2p is at bits 4p, code 2p + 1 at bits
// 4p + 16, so a shift and a mask leave a pair; or-ing the exponent of 128
// (bf16; 1024 in fp16) makes them 128 + q, and `zz` holds 128 + z twice.
template <bool BF16> static __device__ __forceinline__ void decode(uint32_t w, uint32_t zz, uint32_t *out)
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t v = ((w >> (4 * p)) & 0x000F000Fu) | (BF16 ? 0x43004300u : 0x64006400u);
        if (BF16)
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[p]) : "r"(v), "r"(zz));
        else
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(out[p]) : "r"(v), "r"(zz));
    }
}

static __device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

template <bool LINEAR, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) int4_kernel(const __grid_constant__ Int4Args a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const uint32_t dyn0 = smem_u32(dyn);
    const uint32_t ring_b = (dyn0 + 1023u) & ~1023u;
    const uint32_t ring_a = ring_b + a.bytes_b;
    uint8_t *const ring_a_p = dyn + (ring_a - dyn0);
    const int T8 = (a.T + 7) & ~7;
    float *const acc = reinterpret_cast<float *>(ring_a_p + a.stages * a.stage_a);
    const Lists li(acc + (LINEAR ? 0 : T8 * kTileRows), a.E, a.P);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
    const int G = gridDim.x, blk = blockIdx.x;
    volatile int *const abort = &sh.abort;

    if (tid == 0) {
        sh.abort = sh.reset = sh.rests[0].n = sh.rests[1].n = sh.issued_a = sh.issued_b = 0;
        for (int i = 0; i < kMaxStagesA; ++i) {
            mbar_init(smem_u32(&sh.full_a[i]), 1);
            mbar_init(smem_u32(&sh.empty_a[i]), 4 + 8);  // the warps that read codes, then scales
        }
        for (int i = 0; i < kMaxStagesB; ++i) {
            mbar_init(smem_u32(&sh.full_b[i]), 1);
            mbar_init(smem_u32(&sh.empty_b[i]), 1);
        }
        for (int i = 0; i < kTmemA; ++i) {
            mbar_init(smem_u32(&sh.full_t[i]), 4);
            mbar_init(smem_u32(&sh.empty_t[i]), 1);
        }
        for (int i = 0; i < kMaxSums; ++i) {
            mbar_init(smem_u32(&sh.full_d[i]), 1);
            mbar_init(smem_u32(&sh.empty_d[i]), 8);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        mbar_init_fence();
        tma_prefetch_map(&a.mx);
        if (!LINEAR)
            tma_prefetch_map(&a.mh);
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&sh.tmem), 512);

    if (LINEAR) {  // one "expert" whose tokens are the rows of x
        if (tid == 0) {
            li.expert[0] = 0;
            li.offset[0] = 0;
            li.offset[1] = static_cast<unsigned short>(a.T);
            sh.active = 1;
            sh.nmax = a.T;
        }
    } else {
        build_lists(a, li, sh, tid, kThreads);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int A = sh.active;

    if (A == 0) {
        clear_out(a, blk, G, tid, kThreads);
        __syncthreads();
        if (warp == 1)
            tmem_free(tmem, 512);
        return;
    }

    // gate and up (or one) tiles of the first product; the second product of the experts
    constexpr int kParts = LINEAR ? 1 : 2;
    const int total1 = A * a.mt1 * a.kc1, total2 = LINEAR ? 0 : A * a.mt2 * a.kc2;
    const Shares shares1(total1, G), shares2(total2, G);
    const int begin1 = shares1.begin(blk), end1 = shares1.begin(blk + 1);
    const int begin2 = LINEAR ? 0 : shares2.begin(blk), end2 = LINEAR ? 0 : shares2.begin(blk + 1);
    const int pairs = li.offset[A];
    const int width = LINEAR ? ceil_div(sh.nmax, 16) * 16 : ceil_div(sh.nmax, 8) * 16;  // rows of a token tile, columns of a sum
    const int stage_b = width * 256;  // two 64-input halves
    const int stages_b = min(kMaxStagesB, a.bytes_b / stage_b);
    const int sums = min(kMaxSums, 256 / width);
    const int groups1 = 4 >> a.shift1, groups2 = 4 >> a.shift2;

    if (warp == 0 && elect_one()) {
        // ---- weight tiles ----
        const uint64_t policy = policy_evict_first();
        Cursor at;
        int issued = 0;
        bool run = true;
        auto load = [&](const uint8_t *src, uint32_t bytes) {
            if (!mbar_wait(smem_u32(&sh.empty_a[at.s]), at.parity ^ 1, abort, kWaitEmptyA))
                return false;
            const uint32_t bar = smem_u32(&sh.full_a[at.s]);
            mbar_expect(bar, bytes);
            bulk_load(ring_a + at.s * a.stage_a, src, bytes, bar, policy);
            at.next(a.stages);
            ++issued;
            return true;
        };
        const size_t up = static_cast<size_t>(a.mt1) * a.kc1 * a.tile1;  // from a gate tile to its up tile
        for (Walk w(begin1, end1, a.kc1, a.mt1, false); run && w.more(); w.next()) {
            const uint8_t *src =
                a.w1 + ((static_cast<size_t>(li.expert[w.i]) * kParts * a.mt1 + w.m) * a.kc1 + w.k) * a.tile1;
            for (int k = 0; run && k < w.len; ++k, src += a.tile1)
                run = load(src, a.tile1) && (LINEAR || load(src + up, a.tile1));
        }
        for (Walk w(begin2, end2, a.kc2, A, true); run && w.more(); w.next()) {
            const uint8_t *src = a.w2 + ((static_cast<size_t>(li.expert[w.i]) * a.mt2 + w.m) * a.kc2 + w.k) * a.tile2;
            for (int k = 0; run && k < w.len; ++k, src += a.tile2)
                run = load(src, a.tile2);
        }
        sh.issued_a = issued;
    } else if (warp == 2 && elect_one()) {
        // ---- token tiles ----
        Cursor at;
        int issued = 0;
        bool run = true;
        uint32_t dst = 0, bar = 0;
        const uint32_t half = width * 128;  // from the tile's first 64 inputs to the others
        auto acquire = [&](uint32_t bytes) {
            if (!mbar_wait(smem_u32(&sh.empty_b[at.s]), at.parity ^ 1, abort, kWaitEmptyB))
                return false;
            bar = smem_u32(&sh.full_b[at.s]);
            dst = ring_b + at.s * stage_b;
            mbar_expect(bar, bytes);
            at.next(stages_b);
            ++issued;
            return true;
        };
        for (Walk w(begin1, end1, a.kc1, a.mt1, false); run && w.more(); w.next()) {
            const int n = li.count(w.i);
            const unsigned char *const tok = li.token + li.offset[w.i];
            const uint32_t bytes = LINEAR ? ceil_div(n, 8) * 2048 : ceil_div(n, 4) * 1024;
            for (int k = w.k; k < w.k + w.len && (run = acquire(bytes)); ++k) {
                if (LINEAR)
                    for (int j = 0; j < n; j += 8) {
                        tma_load_2d(dst + j * 128, &a.mx, bar, k * 128, j);
                        tma_load_2d(dst + half + j * 128, &a.mx, bar, k * 128 + 64, j);
                    }
                else
                    for (int j = 0; j < n; j += 4) {  // short of a fourth row: the last one again
                        const int r0 = tok[j], r1 = tok[min(j + 1, n - 1)], r2 = tok[min(j + 2, n - 1)],
                                  r3 = tok[min(j + 3, n - 1)];
                        tma_gather4(dst + j * 128, &a.mx, bar, k * 128, r0, r1, r2, r3);
                        tma_gather4(dst + half + j * 128, &a.mx, bar, k * 128 + 64, r0, r1, r2, r3);
                    }
            }
        }
        if (run && begin2 < end2) {
            run = wait_count(a.done, a.mt1 * pairs, abort, kWaitDone);
            fence_async_proxy();
        }
        for (Walk w(begin2, end2, a.kc2, A, true); run && w.more(); w.next()) {
            const int off = li.offset[w.i], n8 = ceil_div(li.count(w.i), 8);
            for (int k = w.k; k < w.k + w.len && (run = acquire(n8 * 4096)); ++k)
                for (int b = 0; b < n8; ++b) {
                    const int x = k * 128, r = off + b * 8;
                    tma_load_2d(dst + b * 1024, &a.mh, bar, x, r);
                    tma_load_2d(dst + (n8 + b) * 1024, &a.mh, bar, x, a.P + r);
                    tma_load_2d(dst + half + b * 1024, &a.mh, bar, x + 64, r);
                    tma_load_2d(dst + half + (n8 + b) * 1024, &a.mh, bar, x + 64, a.P + r);
                }
        }
        sh.issued_b = issued;
    } else if (warp == 1 && elect_one()) {
        // ---- matrix instructions ----
        Cursor at_t, at_b, at_d;
        bool run = true;
        for (int product = 0; run && product < 2; ++product) {
            const int parts = product ? 1 : kParts, groups = product ? groups2 : groups1, steps = 8 / groups;
            for (Walk w(product ? begin2 : begin1, product ? end2 : end1, product ? a.kc2 : a.kc1,
                        product ? A : a.mt1, product != 0);
                 run && w.more(); w.next()) {
                const int n = li.count(w.i);
                const int N = product ? ceil_div(n, 8) * 16 : ceil_div(n, 16) * 16;
                const uint32_t idesc = idesc_f16(kTileRows, N, BF16);
                for (int k = 0; run && k < w.len; ++k) {
                    run = mbar_wait(smem_u32(&sh.full_b[at_b.s]), at_b.parity, abort, kWaitFullB);
                    const uint64_t db = desc_sw128(ring_b + at_b.s * stage_b);
                    for (int g = 0; run && g < parts; ++g) {
                        run = mbar_wait(smem_u32(&sh.full_t[at_t.s]), at_t.parity, abort, kWaitFullA);
                        int k16 = 0;  // sixteenths of inputs within the tile
                        for (int q = 0; run && q < groups; ++q) {
                            run = mbar_wait(smem_u32(&sh.empty_d[at_d.s]), at_d.parity ^ 1, abort, kWaitEmptyD);
                            if (!run)
                                break;
                            tc_fence_after();
                            for (int c = 0; c < steps; ++c, ++k16)
                                mma_ts(tmem + 256 + at_d.s * width, tmem + at_t.s * 64 + k16 * 8,
                                       db + (k16 >> 2) * (width * 8) + 2 * (k16 & 3), idesc, c > 0);
                            tc_commit(smem_u32(&sh.full_d[at_d.s]));
                            at_d.next(sums);
                        }
                        tc_commit(smem_u32(&sh.empty_t[at_t.s]));
                        at_t.next(kTmemA);
                    }
                    tc_commit(smem_u32(&sh.empty_b[at_b.s]));
                    at_b.next(stages_b);
                }
            }
        }
        tc_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= 4 && warp < 12) {
        // ---- codes to 16-bit weights in tensor memory; the two warpgroups take tiles in turn ----
        const int wg = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const int tiles1 = (end1 - begin1) * kParts, tiles = tiles1 + (end2 - begin2);
        Cursor at_a, at_t;
        bool run = true;
        if (wg) {
            at_a.next(a.stages);
            at_t.next(kTmemA);
        }
        for (int it = wg; run && it < tiles; it += 2) {
            const bool second = it >= tiles1;
            const int shift = second ? a.shift2 : a.shift1;  // log2 of the group in 32 inputs
            const bool zeros = second ? a.zeros2 : a.zeros1;
            const int s = at_a.s, t = at_t.s;
            run = mbar_wait(smem_u32(&sh.full_a[s]), at_a.parity, abort, kWaitFullA) &&
                  mbar_wait(smem_u32(&sh.empty_t[t]), at_t.parity ^ 1, abort, kWaitEmptyA);
            at_a.next(a.stages);
            at_a.next(a.stages);
            at_t.next(kTmemA);
            at_t.next(kTmemA);
            run = __all_sync(~0u, run);
            if (!run)
                break;
            tc_fence_after();
            const uint8_t *const tile = ring_a_p + s * a.stage_a;
            const uint8_t *const zp = tile + 8192 + (1024 >> shift) + row;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(tile + q * 2048 + row * 16);
                const uint32_t z = zeros ? zp[(q >> shift) * 128] : 8;
                const uint32_t zz = (BF16 ? 0x43004300u : 0x64006400u) + z * 0x10001u;
                uint32_t r[16];
                decode<BF16>(w.x, zz, r);
                decode<BF16>(w.y, zz, r + 4);
                decode<BF16>(w.z, zz, r + 8);
                decode<BF16>(w.w, zz, r + 12);
                tmem_st16(lanes + t * 64 + q * 16, r);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sh.empty_a[s]));
                mbar_arrive(smem_u32(&sh.full_t[t]));
            }
        }
    } else if (warp >= 12) {
        // ---- scales and results; the two warpgroups share the columns ----
        const int wg = (warp - 12) >> 2, row = tid & 127, rtid = tid - 384;
        const uint32_t lanes = tmem + 256 + (static_cast<uint32_t>(warp & 3) << 21);
        Cursor at_a, at_d;
        bool run = true;
        float v[2][32];  // sums of this thread's row: gate and up (or the one product), up to 32 columns

        auto leave = [&](Rests &rests, int i, int m, const Split &sp, int *counter) {
            if (rtid == 0)
                rests.of[rests.n++] = Rest{i, m, sp};
            named_sync(1, kResults);
            if (rtid == 0)
                add_acq_rel(counter, 1);
        };
        auto parts_written = [&](int *counter, const Split &sp) {
            return named_all(2, kResults, rtid != 0 || wait_count(counter, sp.parts(), abort, kWaitOther));
        };
        auto announce = [&](int columns) {
            fence_async_proxy();
            named_sync(1, kResults);
            if (rtid == 0)
                add_acq_rel(a.done, columns);
        };
        // Adds s times the sum of each group of one weight tile to v[p], columns [c0, c0 + 8 nb) of the sum and,
        // where lo > 0, those `lo` further.
        auto add_tile = [&](float *p, int groups, int c0, int nb, int lo) {
            run = run && mbar_wait(smem_u32(&sh.full_a[at_a.s]), at_a.parity, abort, kWaitFullA);
            const uint8_t *const sc = ring_a_p + at_a.s * a.stage_a + 8192;
            for (int q = 0; q < groups; ++q) {
                const int d = at_d.s;
                run = run && mbar_wait(smem_u32(&sh.full_d[d]), at_d.parity, abort, kWaitFullD);
                run = __all_sync(~0u, run);
                if (!run)
                    return;
                tc_fence_after();
                const uint16_t raw = *reinterpret_cast<const uint16_t *>(sc + q * 256 + row * 2);
                const float s = a.scale_fp16 ? __half2float(__ushort_as_half(raw))
                                             : __uint_as_float(static_cast<uint32_t>(raw) << 16);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (b < nb) {
                        float x[8], y[8];
                        tmem_ld8(lanes + d * width + c0 + b * 8, x);
                        if (lo > 0)
                            tmem_ld8(lanes + d * width + lo + c0 + b * 8, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            p[b * 8 + c] = fmaf(s, lo > 0 ? x[c] + y[c] : x[c], p[b * 8 + c]);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sh.empty_d[d]));
                at_d.next(sums);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sh.empty_a[at_a.s]));
            at_a.next(a.stages);
        };

        // column j of row tile m: h, or y of the linear layer
        auto result = [&](int off, int m, int j, float gate, float up) {
            const int col = m * kTileRows + row;
            if (col >= a.I)
                return;
            if (LINEAR) {
                uint16_t *const p = static_cast<uint16_t *>(a.out) + j * a.out_stride + col;
                if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.I)))
                    *p = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(gate))
                              : __half_as_ushort(__float2half_rn(gate));
            } else {
                __nv_bfloat16 hi, lo;
                split(swiglu(gate, up), hi, lo);
                a.h[static_cast<size_t>(off + j) * a.h_stride + col] = hi;
                a.h[static_cast<size_t>(a.P + off + j) * a.h_stride + col] = lo;
            }
        };

        for (Walk w(begin1, end1, a.kc1, a.mt1, false); run && w.more(); w.next()) {
            const int off = li.offset[w.i], n = li.count(w.i), tile = w.i * a.mt1 + w.m;
            const int blocks = ceil_div(n, 8), half = ceil_div(blocks, 2);  // columns by eights: this warpgroup's
            const int c0 = wg ? half * 8 : 0, nb = wg ? blocks - half : half;
            const Split sp(shares1, tile * a.kc1, a.kc1);
#pragma unroll
            for (int c = 0; c < 32; ++c)
                v[0][c] = v[1][c] = 0.0f;
            for (int k = 0; run && k < w.len; ++k) {
                add_tile(v[0], groups1, c0, nb, 0);
                if (!LINEAR)
                    add_tile(v[1], groups1, c0, nb, 0);
            }
            run = named_all(2, kResults, run);
            if (!run)
                break;
            float *const part = a.part + static_cast<size_t>(sp.slot(blk)) * a.part_floats + row;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const int j = c0 + c;
                if (c < nb * 8 && j < n) {
                    if (sp.shared()) {
                        part[j * kTileRows] = v[0][c];
                        if (!LINEAR)
                            part[(n + j) * kTileRows] = v[1][c];
                    } else {
                        result(off, w.m, j, v[0][c], v[1][c]);
                    }
                }
            }
            if (sp.shared())
                leave(sh.rests[0], w.i, w.m, sp, a.tiles + tile);
            else if (!LINEAR)
                announce(n);
        }
        for (int r = 0; run && r < sh.rests[0].n; ++r) {
            const Rest &rest = sh.rests[0].of[r];
            const int i = rest.i, m = rest.m, off = li.offset[i], n = li.count(i);
            const Split sp = rest.sp;
            const int lo = sp.column(n, blk), hi = sp.column(n, blk + 1);
            if (lo == hi)
                continue;
            run = parts_written(a.tiles + i * a.mt1 + m, sp);
            if (!run)
                break;
            for (int j = lo + 2 * wg; j < hi; j += 4) {
                float g[2], u[2] = {};
                sum_parts<2>(a.part + j * kTileRows + row, a.part_floats, sp, hi - j, g);
                if (!LINEAR)
                    sum_parts<2>(a.part + (n + j) * kTileRows + row, a.part_floats, sp, hi - j, u);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (j + c < hi)
                        result(off, m, j + c, g[c], u[c]);
            }
            if (!LINEAR)
                announce(hi - lo);
        }

        const int group = LINEAR ? 1 : A * a.kc2;
        auto store_y = [&](int m, int t, float r) {
            const int col = m * kTileRows + row;
            __nv_bfloat16 *const p = static_cast<__nv_bfloat16 *>(a.out) + t * a.out_stride + col;
            if (col < a.H && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
                *p = __float2bfloat16_rn(r);
        };
        for (Walk w(begin2, end2, a.kc2, A, true); !LINEAR && run && w.more();) {
            const int m = w.m, i0 = w.i;
            const Split sp(shares2, m * group, group);
            for (int t = wg; t < a.T; t += 2)
                acc[t * kTileRows + row] = 0.0f;
            for (; run && w.more() && w.m == m; w.next()) {
                const int off = li.offset[w.i], n = li.count(w.i);
                const int blocks = ceil_div(n, 8), half = ceil_div(blocks, 2);
                const int c0 = wg ? half * 8 : 0, nb = wg ? blocks - half : half;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    v[0][c] = 0.0f;
                for (int k = 0; run && k < w.len; ++k)
                    add_tile(v[0], groups2, c0, nb, blocks * 8);
                // also: the other warpgroup's rows of acc for the experts before are written
                run = named_all(2, kResults, run);
                if (!run)
                    break;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < nb * 8 && c0 + c < n) {
                        float *const s = acc + li.token[off + c0 + c] * kTileRows + row;
                        *s = fmaf(li.weight[off + c0 + c], v[0][c], *s);
                    }
            }
            run = named_all(2, kResults, run);
            if (!run)
                break;
            if (sp.shared()) {
                float *const part = a.part + static_cast<size_t>(sp.slot(blk)) * a.part_floats + row;
                for (int t = wg; t < a.T; t += 2)
                    part[t * kTileRows] = acc[t * kTileRows + row];
                leave(sh.rests[1], i0, m, sp, a.tiles + a.E * a.mt1 + m);
            } else {
                for (int t = wg; t < a.T; t += 2)
                    store_y(m, t, acc[t * kTileRows + row]);
                named_sync(1, kResults);  // acc is read before the next row tile clears it
            }
        }
        for (int r = 0; !LINEAR && run && r < sh.rests[1].n; ++r) {
            const Rest &rest = sh.rests[1].of[r];
            const Split sp = rest.sp;
            const int m = rest.m, lo = sp.column(a.T, blk), hi = sp.column(a.T, blk + 1);
            if (lo == hi)
                continue;
            run = parts_written(a.tiles + a.E * a.mt1 + m, sp);
            if (!run)
                break;
            for (int t = lo + 2 * wg; t < hi; t += 4) {
                float x[2];
                sum_parts<2>(a.part + t * kTileRows + row, a.part_floats, sp, hi - t, x);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (t + c < hi)
                        store_y(m, t + c, x[c]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (sh.abort) {
        if (tid == 0) {
            for (int i = max(0, sh.issued_a - a.stages); i < sh.issued_a; ++i)
                mbar_wait(smem_u32(&sh.full_a[i % a.stages]), (i / a.stages) & 1, nullptr, kWaitOther);
            for (int i = max(0, sh.issued_b - stages_b); i < sh.issued_b; ++i)
                mbar_wait(smem_u32(&sh.full_b[i % stages_b]), (i / stages_b) & 1, nullptr, kWaitOther);
            atomicAdd_system(a.err + sh.abort, 1u);
            __threadfence_system();
            atomicAdd_system(a.err, 1u);
        }
        __syncthreads();
    }
    if (warp == 1)
        tmem_free(tmem, 512);

    if (tid == 0)
        sh.reset = add_acq_rel(a.leaving, 1) == G - 1;
    __syncthreads();
    if (sh.reset) {
        for (int i = tid; i < A * a.mt1; i += kThreads)
            a.tiles[i] = 0;
        for (int i = tid; !LINEAR && i < a.mt2; i += kThreads)
            a.tiles[a.E * a.mt1 + i] = 0;
        if (tid == 0)
            *a.done = *a.leaving = 0;
    }
}

// One thread per 32 codes of a tile: [4][128 rows][16 bytes], then scales and
// zero points [groups][128 rows]. Rows and inputs outside the matrix become
// codes of 0 with a scale of 0.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int row = static_cast<int>(id & 127), q = static_cast<int>((id >> 7) & 3);
    const long long tile = id >> 9;
    if (tile >= a.mats * a.mt * a.kc)
        return;
    const long long mat = tile / (static_cast<long long>(a.mt) * a.kc);
    const int m = static_cast<int>(tile / a.kc - mat * a.mt), kc = static_cast<int>(tile % a.kc);
    const int r = m * 128 + row, k = kc * 128 + q * 32;
    const bool inside = r < a.rows && k < a.cols;  // cols is a multiple of 32
    const long long src_row = mat * a.rows + r;
    uint32_t in[4] = {0, 0, 0, 0}, out[4];
    if (inside) {
        const uint8_t *const p = a.codes + src_row * (a.cols / 2) + k / 2;
        for (int i = 0; i < 16; ++i)
            in[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // codes 0..7 in order -> even ones in the low half, odd ones in the high half
        uint32_t o = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            o |= ((in[w] >> (4 * c)) & 15u) << ((c >> 1) * 4 + (c & 1) * 16);
        out[w] = o;
    }
    uint8_t *const dst = a.dst + tile * a.tile_bytes;
    *reinterpret_cast<uint4 *>(dst + q * 2048 + row * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    const int groups = 128 / a.group;
    for (int g = q; g < groups; g += 4) {
        const int kg = kc * 128 + g * a.group;
        const bool in_g = r < a.rows && kg < a.cols;
        const long long at = src_row * (a.cols / a.group) + kg / a.group;
        reinterpret_cast<uint16_t *>(dst + 8192)[g * 128 + row] = in_g ? a.scales[at] : 0;
        if (a.zeros)
            (dst + 8192 + groups * 256)[g * 128 + row] = in_g ? (a.zeros[at] & 15) : 0;
    }
}

}  // namespace

int int4_tile_bytes(int group, bool zeros)
{
    return 8192 + 128 / group * 256 + (zeros ? 128 / group * 128 : 0);
}

size_t int4_part_floats(int T, bool linear)
{
    const int T8 = (T + 7) & ~7;
    return static_cast<size_t>(linear ? 1 : 2) * T8 * kTileRows;
}

size_t int4_smem(Int4Args *a, bool linear)
{
    const int T8 = (a->T + 7) & ~7;
    const size_t lists = (linear ? 0 : static_cast<size_t>(T8) * kTileRows * 4) + lists_bytes(a->E, a->P);
    a->bytes_b = T8 <= 8 ? 32 * 1024 : 64 * 1024;  // at least 2 stages of the largest token tile
    a->shift1 = a->group1 == 32 ? 0 : a->group1 == 64 ? 1 : 2;
    a->shift2 = a->group2 == 32 ? 0 : a->group2 == 64 ? 1 : 2;
    a->stage_a = a->tile1 > a->tile2 ? a->tile1 : a->tile2;
    a->part_floats = static_cast<int>(int4_part_floats(a->T, linear));
    const size_t room = kSmemMax - sizeof(Shared) - 1024 - lists - a->bytes_b - 64;
    a->stages = static_cast<int>(room / a->stage_a);
    if (a->stages > kMaxStagesA)
        a->stages = kMaxStagesA;
    return 1024 + static_cast<size_t>(a->stages) * a->stage_a + a->bytes_b + lists;
}

cudaError_t launch_int4(const Int4Args &a, bool linear, bool bf16, int grid, size_t smem, cudaStream_t stream)
{
    using Kernel = void (*)(Int4Args);
    static const Kernel kernels[3] = {int4_kernel<false, true>, int4_kernel<true, true>, int4_kernel<true, false>};
    static const cudaError_t attr = [] {
        cudaError_t ce = cudaSuccess;
        for (Kernel k : kernels)
            if (ce == cudaSuccess)
                ce = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          kSmemMax - 64 - static_cast<int>(sizeof(Shared)));
        return ce;
    }();
    if (attr != cudaSuccess)
        return attr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernels[linear ? (bf16 ? 1 : 2) : 0], a);
}

cudaError_t launch_pack(const PackArgs &a, cudaStream_t stream)
{
    const long long threads = a.mats * a.mt * a.kc * 512;
    pack_kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t int4_binary_version(int *v)
{
    cudaFuncAttributes fa;
    const cudaError_t ce = cudaFuncGetAttributes(&fa, int4_kernel<false, true>);
    if (ce == cudaSuccess)
        *v = fa.binaryVersion;
    return ce;
}

}  // namespace moe
