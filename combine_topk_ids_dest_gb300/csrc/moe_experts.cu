// moe_experts.cu -- the experts of an MoE layer for a few tokens, bf16 weights.
//
//   y_t = sum_k w_tk * W2_e ( silu(W1_e x_t) * (W3_e x_t) ),   e = ids[t, k]
//
// One persistent kernel, one block per SM, streams the weights of the chosen
// experts once: 3 H I weights each, the only traffic that counts for 1..64
// tokens. Both products are skinny, D[128 weight rows, N token columns], so
// the weights are the MMA's A operand (M = 128) and the tokens its N:
//
//  - warp 0 streams weight tiles (128 rows x 64 inputs, 16 KB) through a ring
//    of shared memory with TMA; warp 2 brings the matching token tiles (rows
//    of x picked by index for the first product, rows of h for the second);
//    warp 1 issues the tcgen05 MMAs; warps 4-7 read the accumulators from
//    tensor memory.
//  - The work is cut evenly over the blocks in chunks of 64 inputs, wherever
//    row tiles begin and end: 8 experts' tiles divide 152 SMs badly, their
//    chunks do not. A tile that several blocks share is written as fp32
//    parts; after their last chunk each of them adds up the parts of some of
//    its columns, in the order of the inputs: results do not depend on timing.
//  - The second product's weights do not depend on the first's result, so the
//    ring runs on into them: while h is finished and its last tile announced,
//    the ring (up to 208 KB per SM) already fills with W2.
//  - h is kept as the sum of two bf16 values, 16 bits of mantissa: the second
//    product treats them as two columns, which costs nothing while the
//    weights are the bottleneck. x and the weights are used as they are, all
//    sums are fp32, y is rounded once. Against the 64-bit result that leaves
//    5 to 9 of 1000 values of y at the other bf16 neighbour (4-bit experts,
//    whose sums are shorter, 3; all 32-bit 0.4), and the norm of the error
//    at 1.00008 of what the rounding of y alone gives, or less.
//  - For each row tile of y a block adds its experts' contributions, times
//    the routing weight, in fp32 in ascending expert order.
//
// What bounds it: DRAM. 64 tokens, 8 of 128 experts of 4096 x 2048 (6.3 GB)
// take 922 to 949 us, 6.7 to 6.9 TB/s, the rate of a copy; 5 tokens, 2 of 8
// experts of 4096 x 14336, 313 us, 6.9 TB/s. One token's 8 of 256 experts of
// 7168 x 2048 (708 MB) take 127 us with the router: the first product streams
// at 6.7 TB/s, but the SMs' shares of the bandwidth differ by 10 % and all wait
// for the last before the second (ring full, some 8 us), and lists, settling
// and the launch take 10 more. With 2048 x 768 that fixed part is most of the
// 34 us.
#include "moe_sched.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxStagesA = 13;
constexpr int kMaxStagesB = 16;
constexpr int kTmemCols = 256;

struct Shared {
    uint64_t full_a[kMaxStagesA], empty_a[kMaxStagesA];
    uint64_t full_b[kMaxStagesB], empty_b[kMaxStagesB];
    uint64_t full_d[2], empty_d[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int active, nmax;   // experts that any token chose; the most tokens of one
    int issued_a, issued_b;
    int reset;
    int3 totals[kMaxLocal / 32];
    Rests rests[2];  // of the two products
};

__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ ExpertsArgs a)
{
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const uint32_t dyn0 = smem_u32(dyn);
    const uint32_t ring_a = (dyn0 + 1023u) & ~1023u;
    const uint32_t ring_b = ring_a + a.stages * kStageA;
    uint8_t *const after = dyn + (ring_b - dyn0) + a.bytes_b;
    const int T8 = (a.T + 7) & ~7;
    float *const acc = reinterpret_cast<float *>(after);
    const Lists li(acc + T8 * kTileRows, acc, a.E, a.P);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
    const int G = gridDim.x, blk = blockIdx.x;
    volatile int *const abort = &sh.abort;

    if (tid < kMaxStagesA) {
        mbar_init(smem_u32(&sh.full_a[tid]), 1);
        mbar_init(smem_u32(&sh.empty_a[tid]), 1);
    } else if (tid >= 64 && tid < 64 + kMaxStagesB) {
        mbar_init(smem_u32(&sh.full_b[tid - 64]), 1);
        mbar_init(smem_u32(&sh.empty_b[tid - 64]), 1);
    } else if (tid >= 96 && tid < 98) {
        mbar_init(smem_u32(&sh.full_d[tid - 96]), 1);
        mbar_init(smem_u32(&sh.empty_d[tid - 96]), 128);
    } else if (tid == 128) {
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort = sh.reset = sh.rests[0].n = sh.rests[1].n = sh.issued_a = sh.issued_b = 0;
    } else if (tid == 160) {
        tma_prefetch_map(&a.mx);
        tma_prefetch_map(&a.mw1);
        tma_prefetch_map(&a.mw2);
        tma_prefetch_map(&a.mh);
    }
    mbar_init_fence();
    if (warp == 1)
        tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
    build_lists(a, li, sh, tid, kThreads, kMaxTokens);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int A = sh.active;

    if (A == 0) {  // no token chose an expert of this handle
        clear_out(a, blk, G, tid, kThreads);
        __syncthreads();
        if (warp == 1)
            tmem_free(tmem, kTmemCols);
        return;
    }

    const int total1 = A * a.mt1 * a.kc1, total2 = A * a.mt2 * a.kc2;
    const Shares shares1(total1, G), shares2(total2, G);
    const int begin1 = shares1.begin(blk), end1 = shares1.begin(blk + 1);
    const int begin2 = shares2.begin(blk), end2 = shares2.begin(blk + 1);
    const int pairs = li.offset[A];
    const int stage_b = ceil_div(sh.nmax, 8) * 16 * 128;  // 8 tokens: up to 16 rows of 128 bytes
    const int stages_b = min(kMaxStagesB, a.bytes_b / stage_b);

    if (warp == 0 && elect_one()) {
        // ---- weight tiles ----
        const uint64_t policy = policy_evict_first();
        Cursor at;
        int issued = 0;
        bool run = true;
        auto load = [&](const CUtensorMap *map, int x, int y, int z) {
            if (!mbar_wait(smem_u32(&sh.empty_a[at.s]), at.parity ^ 1, abort, kWaitEmptyA))
                return false;
            const uint32_t bar = smem_u32(&sh.full_a[at.s]);
            mbar_expect(bar, kStageA);
            tma_load_3d(ring_a + at.s * kStageA, map, bar, x, y, z, policy);
            at.next(a.stages);
            ++issued;
            return true;
        };
        for (Walk w(begin1, end1, a.kc1, a.mt1, false); run && w.more(); w.next()) {
            const int e = li.expert[w.i];
            for (int k = w.k; run && k < w.k + w.len; ++k)
                run = load(&a.mw1, k * kChunk, w.m * kTileRows, 2 * e) &&
                      load(&a.mw1, k * kChunk, w.m * kTileRows, 2 * e + 1);
        }
        for (Walk w(begin2, end2, a.kc2, A, true); run && w.more(); w.next()) {
            const int e = li.expert[w.i];
            for (int k = w.k; run && k < w.k + w.len; ++k)
                run = load(&a.mw2, k * kChunk, w.m * kTileRows, e);
        }
        sh.issued_a = issued;
    } else if (warp == 2 && elect_one()) {
        // ---- token tiles ----
        Cursor at;
        int issued = 0;
        bool run = true;
        uint32_t dst = 0, bar = 0;
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
            const int n = li.count(w.i), quads = ceil_div(n, 4);
            const unsigned char *const tok = li.token + li.offset[w.i];
            for (int k = w.k; k < w.k + w.len && (run = acquire(quads * 512)); ++k)
                for (int j = 0; j < n; j += 4)  // short of a fourth row: the last one again
                    tma_gather4(dst + j * 128, &a.mx, bar, k * kChunk, tok[j], tok[min(j + 1, n - 1)],
                                tok[min(j + 2, n - 1)], tok[min(j + 3, n - 1)]);
        }
        if (run && begin2 < end2) {  // h is complete
            run = wait_count(a.done, a.mt1 * pairs, abort, kWaitDone);
            fence_async_proxy();
        }
        for (Walk w(begin2, end2, a.kc2, A, true); run && w.more(); w.next()) {
            const int off = li.offset[w.i], n8 = ceil_div(li.count(w.i), 8);
            for (int k = w.k; k < w.k + w.len && (run = acquire(n8 * 2048)); ++k)
                for (int b = 0; b < n8; ++b) {
                    tma_load_2d(dst + b * 1024, &a.mh, bar, k * kChunk, off + b * 8);
                    tma_load_2d(dst + (n8 + b) * 1024, &a.mh, bar, k * kChunk, a.P + off + b * 8);
                }
        }
        sh.issued_b = issued;
    } else if (warp == 1) {
        // ---- matrix instructions: the warp waits, one lane issues ----
        Cursor at_a, at_b, at_d;
        bool run = true;
        for (int product = 0; run && product < 2; ++product) {
            const int parts = product ? 1 : 2;  // gate and up share the token tile
            for (Walk w(product ? begin2 : begin1, product ? end2 : end1, product ? a.kc2 : a.kc1,
                        product ? A : a.mt1, product != 0);
                 run && w.more(); w.next()) {
                const int n = li.count(w.i);
                const int N = product ? ceil_div(n, 8) * 16 : ceil_div(n, 16) * 16;
                const uint32_t idesc = idesc_f16(kTileRows, N, 1);
                const uint32_t d = tmem + at_d.s * 128;
                run = mbar_wait_warp(smem_u32(&sh.empty_d[at_d.s]), at_d.parity ^ 1, abort, kWaitEmptyD);
                for (int k = 0; run && k < w.len; ++k) {
                    run = mbar_wait_warp(smem_u32(&sh.full_b[at_b.s]), at_b.parity, abort, kWaitFullB);
                    const uint64_t db = desc_sw128(ring_b + at_b.s * stage_b);
                    for (int g = 0; run && g < parts; ++g) {
                        run = mbar_wait_warp(smem_u32(&sh.full_a[at_a.s]), at_a.parity, abort, kWaitFullA);
                        if (!run)
                            break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t da = desc_sw128(ring_a + at_a.s * kStageA);
#pragma unroll
                            for (int q = 0; q < 4; ++q)  // 16 inputs each: 32 bytes further, in 16-byte units
                                mma_ss(d + g * N, da + 2 * q, db + 2 * q, idesc, k > 0 || q > 0);
                            tc_commit(smem_u32(&sh.empty_a[at_a.s]));
                            if (g == parts - 1)
                                tc_commit(smem_u32(&sh.empty_b[at_b.s]));
                        }
                        at_a.next(a.stages);
                    }
                    at_b.next(stages_b);
                }
                if (elect_one())
                    tc_commit(smem_u32(&sh.full_d[at_d.s]));
                at_d.next(2);
            }
        }
        if (elect_one())
            tc_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= 4) {
        // ---- results ----
        const int row = tid - 128;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp - 4) << 21);
        Cursor at_d;
        bool run = true;

        // Rests: counted once the product's last run is written.
        auto arrive = [&](const Rests &rests, int *counters, bool second) {
            named_sync(1, 128);
            if (row < rests.n)
                add_acq_rel(counters + (second ? rests.of[row].m : rests.of[row].i * a.mt1 + rests.of[row].m), 1);
        };
        auto parts_written = [&](int *counter, const Split &sp) {
            return named_all(2, 128, row != 0 || wait_count(counter, sp.parts(), abort, kWaitOther));
        };
        // h of these columns of a tile goes out to the TMA reads of every block.
        auto announce = [&](int columns) {
            fence_async_proxy();
            named_sync(1, 128);
            if (row == 0)
                add_acq_rel(a.done, columns);
        };
        // A run's part: the block's second slot unless it is the first run of its share.
        auto part_of = [&](bool first) {
            return a.part + static_cast<size_t>(2 * blk + (first ? 0 : 1)) * a.part_floats + row;
        };
        auto store_h = [&](int off, int j, int col, float gate, float up) {
            __nv_bfloat16 hi, lo;
            split(swiglu(gate, up), hi, lo);
            a.h[static_cast<size_t>(off + j) * a.h_stride + col] = hi;
            a.h[static_cast<size_t>(a.P + off + j) * a.h_stride + col] = lo;
        };

        int announced = 0;  // columns of h that are written and not yet announced
        for (Walk w(begin1, end1, a.kc1, a.mt1, false); run && w.more(); w.next()) {
            const int off = li.offset[w.i], n = li.count(w.i), N = ceil_div(n, 16) * 16, n8 = (n + 7) & ~7;
            const int col = w.m * kTileRows + row;  // of h
            const bool shared = w.k != 0 || w.len != a.kc1;
            float *const part = part_of(w.left == end1 - begin1);
            run = mbar_wait(smem_u32(&sh.full_d[at_d.s]), at_d.parity, abort, kWaitFullD);
            run = named_all(2, 128, run);  // the four warps leave together, or not at all
            if (!run)
                break;
            tc_fence_after();
            const uint32_t d = lanes + at_d.s * 128;
            for (int j = 0; j < n8; j += 8) {
                float g[8], v[8];
                tmem_ld8(d + j, g);
                tmem_ld8(d + N + j, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (j + c >= n)
                        break;
                    if (shared) {
                        part[(j + c) * kTileRows] = g[c];
                        part[(n + j + c) * kTileRows] = v[c];
                    } else if (col < a.I) {
                        store_h(off, j + c, col, g[c], v[c]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.empty_d[at_d.s]));
            at_d.next(2);
            if (!shared)
                announced += n;
            else if (row == 0)
                sh.rests[0].of[sh.rests[0].n++] = Rest{w.i, w.m};
        }
        if (run)
            arrive(sh.rests[0], a.tiles, false);
        for (int r = 0; run && r < sh.rests[0].n; ++r) {
            const int i = sh.rests[0].of[r].i, m = sh.rests[0].of[r].m, off = li.offset[i], n = li.count(i);
            const Split sp(shares1, (i * a.mt1 + m) * a.kc1, a.kc1);
            const int lo = sp.column(n, blk), hi = sp.column(n, blk + 1), col = m * kTileRows + row;
            if (lo == hi)
                continue;
            run = parts_written(a.tiles + i * a.mt1 + m, sp);
            if (!run)
                break;
            for (int j = lo; j < hi; j += 4) {
                float g[4], v[4];
                sum_parts<4>(a.part + j * kTileRows + row, a.part_floats, sp, hi - j, g);
                sum_parts<4>(a.part + (n + j) * kTileRows + row, a.part_floats, sp, hi - j, v);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (j + c < hi && col < a.I)
                        store_h(off, j + c, col, g[c], v[c]);
            }
            announced += hi - lo;
        }
        if (run && announced > 0)
            announce(announced);

        const int group = A * a.kc2;  // units of one row tile of y, over all experts
        auto store_y = [&](int m, int t, float v) {
            const int col = m * kTileRows + row;
            __nv_bfloat16 *const p = a.out + t * a.out_stride + col;
            if (col < a.H && EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
                *p = __float2bfloat16_rn(v);
        };
        for (Walk w(begin2, end2, a.kc2, A, true); run && w.more();) {
            const Walk first = w;
            for (int t = 0; t < a.T; ++t)
                acc[t * kTileRows + row] = 0.0f;
            for (; run && w.more() && w.m == first.m; w.next()) {
                const int off = li.offset[w.i], n = li.count(w.i), n8 = (n + 7) & ~7;
                run = mbar_wait(smem_u32(&sh.full_d[at_d.s]), at_d.parity, abort, kWaitFullD);
                run = named_all(2, 128, run);
                if (!run)
                    break;
                tc_fence_after();
                const uint32_t d = lanes + at_d.s * 128;
                for (int j = 0; j < n8; j += 8) {
                    float hi[8], lo[8];
                    tmem_ld8(d + j, hi);
                    tmem_ld8(d + n8 + j, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (j + c < n) {
                            float *const s = acc + li.token[off + j + c] * kTileRows + row;
                            *s = fmaf(li.weight[off + j + c], hi[c] + lo[c], *s);
                        }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(&sh.empty_d[at_d.s]));
                at_d.next(2);
            }
            if (!run)
                break;
            // an earlier block began this row tile, or a later one ends it
            if (first.i != 0 || first.k != 0 || (!w.more() && end2 != (first.m + 1) * group)) {
                float *const part = part_of(first.left == end2 - begin2);
                for (int t = 0; t < a.T; ++t)
                    part[t * kTileRows] = acc[t * kTileRows + row];
                if (row == 0)
                    sh.rests[1].of[sh.rests[1].n++] = Rest{first.i, first.m};
            } else {
                for (int t = 0; t < a.T; ++t)
                    store_y(first.m, t, acc[t * kTileRows + row]);
            }
        }
        if (run)
            arrive(sh.rests[1], a.tiles + a.E * a.mt1, true);
        for (int r = 0; run && r < sh.rests[1].n; ++r) {
            const int m = sh.rests[1].of[r].m;
            const Split sp(shares2, m * group, group);
            const int lo = sp.column(a.T, blk), hi = sp.column(a.T, blk + 1);
            if (lo == hi)
                continue;
            run = parts_written(a.tiles + a.E * a.mt1 + m, sp);
            if (!run)
                break;
            for (int t = lo; t < hi; t += 4) {
                float v[4];
                sum_parts<4>(a.part + t * kTileRows + row, a.part_floats, sp, hi - t, v);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (t + c < hi)
                        store_y(m, t + c, v[c]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (sh.abort) {  // copies in flight land before the block's memory is given back
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
        tmem_free(tmem, kTmemCols);

    // the last block to leave clears the counters for the next launch
    if (tid == 0)
        sh.reset = add_acq_rel(a.leaving, 1) == G - 1;
    __syncthreads();
    if (sh.reset) {
        for (int i = tid; i < A * a.mt1; i += kThreads)
            a.tiles[i] = 0;
        for (int i = tid; i < a.mt2; i += kThreads)
            a.tiles[a.E * a.mt1 + i] = 0;
        if (tid == 0)
            *a.done = *a.leaving = 0;
    }
}

}  // namespace

size_t experts_part_floats(int T)
{
    const int T8 = (T + 7) & ~7;
    return static_cast<size_t>(2) * T8 * kTileRows;
}

size_t experts_smem(ExpertsArgs *a)
{
    const int T8 = (a->T + 7) & ~7;
    const size_t lists = static_cast<size_t>(T8) * kTileRows * 4 + lists_bytes(a->E, a->P);
    a->bytes_b = T8 <= 8 ? 24 * 1024 : 48 * 1024;  // at least 12 and 3 stages of the largest token tile
    a->part_floats = static_cast<int>(experts_part_floats(a->T));
    const size_t room = kSmemMax - sizeof(Shared) - 1024 - lists - a->bytes_b - 64;
    a->stages = static_cast<int>(room / kStageA);
    if (a->stages > kMaxStagesA)
        a->stages = kMaxStagesA;
    return 1024 + static_cast<size_t>(a->stages) * kStageA + a->bytes_b + lists;
}

cudaError_t experts_setup()
{
    return cudaFuncSetAttribute(experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemMax - 64 - static_cast<int>(sizeof(Shared)));
}

cudaError_t launch_experts(const ExpertsArgs &a, int grid, size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;  // the blocks wait for one another's h
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, experts_kernel, a);
}

std::vector<const void *> experts_kernels() { return {reinterpret_cast<const void *>(experts_kernel)}; }

}  // namespace moe
