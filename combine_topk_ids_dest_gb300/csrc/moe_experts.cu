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
//    chunks do not. A tile that is shared by several blocks is written as
//    fp32 parts; the block whose part arrives last adds them up in order of
//    the inputs, so results do not depend on who is last.
//  - The second product's weights do not depend on the first's result, so the
//    ring runs on into them: while h is finished and its last tile announced,
//    the ring (up to 192 KB per SM) already fills with W2.
//  - h is kept as the sum of two bf16 values, 16 bits of mantissa: the second
//    product treats them as two columns, which costs nothing while the
//    weights are the bottleneck. x and the weights are used as they are, all
//    sums are fp32, y is rounded once.
//  - For each row tile of y a block adds its experts' contributions, times
//    the routing weight, in fp32 in ascending expert order.
#include "moe_device.h"
#include "moe_internal.h"

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
    int last, reset;
};

// Lists of the chosen experts, in dynamic shared memory.
struct Lists {
    unsigned long long *mask;  // [E] tokens of each expert
    float *weight;             // [P] routing weight of each (expert, token) pair
    unsigned short *expert;    // [E] active experts, ascending
    unsigned short *offset;    // [E + 1] their first pair
    unsigned char *token;      // [P] tokens, ascending per expert
};

static __device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Two bf16 values whose sum carries 16 bits of v's mantissa (v itself where it is not finite).
static __device__ __forceinline__ void split(float v, __nv_bfloat16 &hi, __nv_bfloat16 &lo)
{
    hi = __float2bfloat16_rn(v);
    const float r = v - __bfloat162float(hi);
    lo = __float2bfloat16_rn(isfinite(r) ? r : 0.0f);
}

static __device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.0f + expf(-gate)) * up; }

// Slot (first or last share) in which block b keeps its part of the tile that begins at unit `begin`.
static __device__ __forceinline__ int part_slot(int total, int b, int G, int begin)
{
    return 2 * b + (begin <= share_begin(total, b, G) ? 0 : 1);
}

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
    Lists li;
    li.mask = reinterpret_cast<unsigned long long *>(acc + T8 * kTileRows);
    li.weight = reinterpret_cast<float *>(li.mask + a.E);
    li.expert = reinterpret_cast<unsigned short *>(li.weight + a.P);
    li.offset = li.expert + a.E;
    li.token = reinterpret_cast<unsigned char *>(li.offset + a.E + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = gridDim.x, blk = blockIdx.x;
    volatile int *const abort = &sh.abort;

    if (tid == 0) {
        sh.abort = sh.reset = sh.issued_a = sh.issued_b = 0;
        for (int i = 0; i < kMaxStagesA; ++i) {
            mbar_init(smem_u32(&sh.full_a[i]), 1);
            mbar_init(smem_u32(&sh.empty_a[i]), 1);
        }
        for (int i = 0; i < kMaxStagesB; ++i) {
            mbar_init(smem_u32(&sh.full_b[i]), 1);
            mbar_init(smem_u32(&sh.empty_b[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.full_d[i]), 1);
            mbar_init(smem_u32(&sh.empty_d[i]), 128);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        mbar_init_fence();
        tma_prefetch_map(&a.mx);
        tma_prefetch_map(&a.mw1);
        tma_prefetch_map(&a.mw2);
        tma_prefetch_map(&a.mh);
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
    for (int e = tid; e < a.E; e += kThreads)
        li.mask[e] = 0;
    __syncthreads();

    // tokens of each expert (a bit set, so the order of the threads does not matter)
    for (int i = tid; i < a.P; i += kThreads) {
        if (!EP_IN_BOUNDS(a.chk, epk::kSiteMoeIds, a.ids + i, 4, a.ids, 4LL * a.P))
            continue;
        const int e = a.ids[i] - a.first;
        if (e >= 0 && e < a.E)
            atomicOr(&li.mask[e], 1ULL << (i / a.K));
    }
    __syncthreads();
    if (warp == 0) {
        int n_active = 0, n_pairs = 0, nmax = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < a.E ? __popcll(li.mask[e]) : 0;
            const unsigned live = __ballot_sync(~0u, n > 0);
            int sum = n;  // inclusive prefix sum over the lanes
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, d);
                if (lane >= d)
                    sum += v;
            }
            if (n > 0) {
                const int at = n_active + __popc(live & ((1u << lane) - 1));
                li.expert[at] = static_cast<unsigned short>(e);
                li.offset[at] = static_cast<unsigned short>(n_pairs + sum - n);
            }
            n_active += __popc(live);
            n_pairs += __shfl_sync(~0u, sum, 31);
            nmax = max(nmax, __reduce_max_sync(~0u, n));
        }
        if (lane == 0) {
            li.offset[n_active] = static_cast<unsigned short>(n_pairs);
            sh.active = n_active;
            sh.nmax = nmax;
        }
    }
    __syncthreads();
    const int A = sh.active;
    for (int i = tid; i < A; i += kThreads) {
        const int e = li.expert[i];
        int at = li.offset[i];
        for (unsigned long long m = li.mask[e]; m; m &= m - 1, ++at) {
            const int t = __ffsll(static_cast<long long>(m)) - 1;
            float w = 0.0f;  // an expert named twice by a token counts twice
            for (int k = 0; k < a.K; ++k)
                if (a.ids[t * a.K + k] - a.first == e &&
                    EP_IN_BOUNDS(a.chk, epk::kSiteMoeWeights, a.weights + t * a.K + k, 4, a.weights, 4LL * a.P))
                    w += a.weights[t * a.K + k];
            li.token[at] = static_cast<unsigned char>(t);
            li.weight[at] = w;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (A == 0) {  // no token chose an expert of this handle
        for (long long i = static_cast<long long>(blk) * kThreads + tid; i < static_cast<long long>(a.T) * a.H;
             i += static_cast<long long>(G) * kThreads) {
            const long long t = i / a.H;
            __nv_bfloat16 *const p = a.out + t * a.out_stride + (i - t * a.H);
            if (EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
                *p = __float2bfloat16_rn(0.0f);
        }
        __syncthreads();
        if (warp == 1)
            tmem_free(tmem, kTmemCols);
        return;
    }

    const int total1 = A * a.mt1 * a.kc1, total2 = A * a.mt2 * a.kc2;
    // no more shares than units: then every block of a run of blocks has a part in the tile they share
    const int G1 = min(G, total1), G2 = min(G, total2);
    const int begin1 = share_begin(total1, min(blk, G1), G1), end1 = share_begin(total1, min(blk + 1, G1), G1);
    const int begin2 = share_begin(total2, min(blk, G2), G2), end2 = share_begin(total2, min(blk + 1, G2), G2);
    const int stage_b = div_up(sh.nmax, 8) * 16 * 128;  // 8 tokens: up to 16 rows of 128 bytes
    const int stages_b = min(kMaxStagesB, a.bytes_b / stage_b);

    if (warp == 0 && lane == 0) {
        // ---- weight tiles ----
        const uint64_t policy = policy_evict_first();
        int it = 0;
        bool run = true;
        auto load = [&](const CUtensorMap *map, int x, int y, int z) {
            const int s = it % a.stages;
            if (!mbar_wait(smem_u32(&sh.empty_a[s]), ((it / a.stages) & 1) ^ 1, abort, kWaitEmptyA))
                return false;
            const uint32_t bar = smem_u32(&sh.full_a[s]);
            mbar_expect(bar, kStageA);
            tma_load_3d(ring_a + s * kStageA, map, bar, x, y, z, policy);
            ++it;
            return true;
        };
        for (int u = begin1; run && u < end1; ++u) {
            const int tile = u / a.kc1, kc = u - tile * a.kc1;
            const int i = tile / a.mt1, m = tile - i * a.mt1, e = li.expert[i];
            run = load(&a.mw1, kc * kChunk, m * kTileRows, 2 * e) &&
                  load(&a.mw1, kc * kChunk, m * kTileRows, 2 * e + 1);
        }
        for (int u = begin2; run && u < end2; ++u) {
            const int tile = u / a.kc2, kc = u - tile * a.kc2;
            const int m = tile / A, e = li.expert[tile - m * A];
            run = load(&a.mw2, kc * kChunk, m * kTileRows, e);
        }
        sh.issued_a = it;
    } else if (warp == 2 && lane == 0) {
        // ---- token tiles ----
        int it = 0;
        bool run = true;
        auto acquire = [&](uint32_t bytes, uint32_t &dst, uint32_t &bar) {
            const int s = it % stages_b;
            if (!mbar_wait(smem_u32(&sh.empty_b[s]), ((it / stages_b) & 1) ^ 1, abort, kWaitEmptyB))
                return false;
            bar = smem_u32(&sh.full_b[s]);
            dst = ring_b + s * stage_b;
            mbar_expect(bar, bytes);
            ++it;
            return true;
        };
        for (int u = begin1; run && u < end1; ++u) {
            const int tile = u / a.kc1, kc = u - tile * a.kc1, i = tile / a.mt1;
            const int off = li.offset[i], n = li.offset[i + 1] - off, quads = div_up(n, 4);
            uint32_t dst, bar;
            run = acquire(quads * 512, dst, bar);
            for (int q = 0; run && q < quads; ++q) {  // short of a fourth row: the last one again
                const int j = 4 * q, l = n - 1;
                tma_gather4(dst + q * 512, &a.mx, bar, kc * kChunk, li.token[off + j], li.token[off + min(j + 1, l)],
                            li.token[off + min(j + 2, l)], li.token[off + min(j + 3, l)]);
            }
        }
        if (run && begin2 < end2) {  // h is complete when every tile of the first product is
            const unsigned long long t0 = now_ns();
            while (ld_acquire(a.done) < A * a.mt1) {
                if (*abort || now_ns() - t0 > kWaitNs) {
                    *abort = *abort ? *abort : kWaitDone;
                    run = false;
                    break;
                }
            }
            fence_async_proxy();
        }
        for (int u = begin2; run && u < end2; ++u) {
            const int tile = u / a.kc2, kc = u - tile * a.kc2, i = tile % A;
            const int off = li.offset[i], n8 = div_up(li.offset[i + 1] - off, 8);
            uint32_t dst, bar;
            run = acquire(n8 * 2048, dst, bar);
            for (int b = 0; run && b < n8; ++b) {
                tma_load_2d(dst + b * 1024, &a.mh, bar, kc * kChunk, off + b * 8);
                tma_load_2d(dst + (n8 + b) * 1024, &a.mh, bar, kc * kChunk, a.P + off + b * 8);
            }
        }
        sh.issued_b = it;
    } else if (warp == 1 && lane == 0) {
        // ---- matrix instructions ----
        int it_a = 0, it_b = 0, seg = 0;
        bool run = true;
        for (int product = 0; run && product < 2; ++product) {
            const int kc_n = product ? a.kc2 : a.kc1, end = product ? end2 : end1;
            const int parts = product ? 1 : 2;  // gate and up share the token tile
            for (int u = product ? begin2 : begin1; run && u < end;) {
                const int tile = u / kc_n, k0 = u - tile * kc_n, k1 = min(kc_n, k0 + end - u);
                const int i = product ? tile % A : tile / a.mt1;
                const int n = li.offset[i + 1] - li.offset[i];
                const int N = product ? div_up(n, 8) * 16 : div_up(n, 16) * 16;
                const uint32_t idesc = idesc_f16(kTileRows, N, 1);
                const uint32_t d = tmem + (seg & 1) * 128;
                run = mbar_wait(smem_u32(&sh.empty_d[seg & 1]), ((seg >> 1) & 1) ^ 1, abort, kWaitEmptyD);
                tc_fence_after();
                for (int k = k0; run && k < k1; ++k) {
                    const int sb = it_b % stages_b;
                    run = mbar_wait(smem_u32(&sh.full_b[sb]), (it_b / stages_b) & 1, abort, kWaitFullB);
                    for (int g = 0; run && g < parts; ++g) {
                        const int sa = it_a % a.stages;
                        run = mbar_wait(smem_u32(&sh.full_a[sa]), (it_a / a.stages) & 1, abort, kWaitFullA);
                        if (!run)
                            break;
                        tc_fence_after();
                        const uint64_t da = desc_sw128(ring_a + sa * kStageA);
                        const uint64_t db = desc_sw128(ring_b + sb * stage_b);
#pragma unroll
                        for (int q = 0; q < 4; ++q)  // 16 inputs each: 32 bytes further, in 16-byte units
                            mma_ss(d + g * N, da + 2 * q, db + 2 * q, idesc, k > k0 || q > 0);
                        tc_commit(smem_u32(&sh.empty_a[sa]));
                        ++it_a;
                    }
                    tc_commit(smem_u32(&sh.empty_b[sb]));
                    ++it_b;
                }
                tc_commit(smem_u32(&sh.full_d[seg & 1]));
                ++seg;
                u += k1 - k0;
            }
        }
        tc_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0, nullptr, kWaitOther);
    } else if (warp >= 4) {
        // ---- results ----
        const int row = tid - 128;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp - 4) << 21);
        int seg = 0;
        bool run = true;

        // Counts this block's part of a tile; true in the block whose part was the last.
        auto arrive_last = [&](int *counter, int parts) {
            __threadfence();
            named_sync(1, 128);
            if (row == 0)
                sh.last = add_acq_rel(counter) == parts - 1;
            named_sync(1, 128);
            const bool last = sh.last != 0;
            if (last)
                __threadfence();
            return last;
        };

        for (int u = begin1; run && u < end1; ++seg) {
            const int tile = u / a.kc1, k0 = u - tile * a.kc1, k1 = min(a.kc1, k0 + end1 - u);
            const int i = tile / a.mt1, m = tile - i * a.mt1;
            const int off = li.offset[i], n = li.offset[i + 1] - off, N = div_up(n, 16) * 16, n8 = (n + 7) & ~7;
            const int first_unit = tile * a.kc1;
            const int b0 = share_owner(total1, first_unit, G1), b1 = share_owner(total1, first_unit + a.kc1 - 1, G1);
            const int col = m * kTileRows + row;  // of h
            run = mbar_wait(smem_u32(&sh.full_d[seg & 1]), (seg >> 1) & 1, abort, kWaitFullD);
            run = named_all(2, 128, run);  // the four warps leave together, or not at all
            if (!run)
                break;
            tc_fence_after();
            const uint32_t d = lanes + (seg & 1) * 128;
            float *const part = a.part + static_cast<size_t>(part_slot(total1, blk, G1, first_unit)) * a.part_floats;
            auto finish = [&](int j, float gate, float up) {
                if (j < n && col < a.I) {
                    __nv_bfloat16 hi, lo;
                    split(swiglu(gate, up), hi, lo);
                    a.h[static_cast<size_t>(off + j) * a.h_stride + col] = hi;
                    a.h[static_cast<size_t>(a.P + off + j) * a.h_stride + col] = lo;
                }
            };
            for (int j = 0; j < n8; j += 8) {
                float g[8], v[8];
                tmem_ld8(d + j, g);
                tmem_ld8(d + N + j, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (b0 == b1) {
                        finish(j + c, g[c], v[c]);
                    } else {
                        part[(j + c) * kTileRows + row] = g[c];
                        part[(n8 + j + c) * kTileRows + row] = v[c];
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&sh.empty_d[seg & 1]));
            bool mine = b0 == b1;
            if (!mine && arrive_last(a.tiles + tile, b1 - b0 + 1)) {
                mine = true;
                for (int j = 0; j < n8; j += 8) {
                    float g[8] = {}, v[8] = {};
                    for (int b = b0; b <= b1; ++b) {
                        const float *const p =
                            a.part + static_cast<size_t>(part_slot(total1, b, G1, first_unit)) * a.part_floats;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            g[c] += __ldcg(p + (j + c) * kTileRows + row);
                            v[c] += __ldcg(p + (n8 + j + c) * kTileRows + row);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        finish(j + c, g[c], v[c]);
                }
            }
            if (mine) {  // h of this tile goes out to the TMA reads of every block
                fence_async_proxy();
                __threadfence();
                named_sync(1, 128);
                if (row == 0)
                    add_acq_rel(a.done);
            }
            u += k1 - k0;
        }

        const int group = A * a.kc2;  // units of one row tile of y, over all experts
        for (int u = begin2; run && u < end2;) {
            const int m = u / group, stop = min(end2, (m + 1) * group), first_unit = m * group;
            const int b0 = share_owner(total2, first_unit, G2), b1 = share_owner(total2, first_unit + group - 1, G2);
            for (int t = 0; t < T8; ++t)
                acc[t * kTileRows + row] = 0.0f;
            for (; run && u < stop; ++seg) {
                const int tile = u / a.kc2, k0 = u - tile * a.kc2, k1 = min(a.kc2, k0 + stop - u);
                const int i = tile - m * A, off = li.offset[i], n = li.offset[i + 1] - off, n8 = (n + 7) & ~7;
                run = mbar_wait(smem_u32(&sh.full_d[seg & 1]), (seg >> 1) & 1, abort, kWaitFullD);
                run = named_all(2, 128, run);  // the four warps leave together, or not at all
                if (!run)
                    break;
                tc_fence_after();
                const uint32_t d = lanes + (seg & 1) * 128;
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
                mbar_arrive(smem_u32(&sh.empty_d[seg & 1]));
                u += k1 - k0;
            }
            if (!run)
                break;
            const int col = m * kTileRows + row;
            auto store = [&](int t, float v) {
                __nv_bfloat16 *const p = a.out + t * a.out_stride + col;
                if (t < a.T && col < a.H &&
                    EP_IN_BOUNDS(a.chk, epk::kSiteMoeOut, p, 2, a.out, 2 * ((a.T - 1) * a.out_stride + a.H)))
                    *p = __float2bfloat16_rn(v);
            };
            if (b0 == b1) {
                for (int t = 0; t < a.T; ++t)
                    store(t, acc[t * kTileRows + row]);
            } else {
                float *const part = a.part + static_cast<size_t>(part_slot(total2, blk, G2, first_unit)) * a.part_floats;
                for (int t = 0; t < a.T; ++t)
                    part[t * kTileRows + row] = acc[t * kTileRows + row];
                if (arrive_last(a.tiles + a.E * a.mt1 + m, b1 - b0 + 1)) {
                    for (int t = 0; t < a.T; t += 8) {
                        float v[8] = {};
                        for (int b = b0; b <= b1; ++b) {
                            const float *const p =
                                a.part + static_cast<size_t>(part_slot(total2, b, G2, first_unit)) * a.part_floats;
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (t + c < a.T)
                                    v[c] += __ldcg(p + (t + c) * kTileRows + row);
                        }
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            store(t + c, v[c]);
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
        sh.reset = add_acq_rel(a.leaving) == G - 1;
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
    size_t lists = static_cast<size_t>(T8) * kTileRows * 4 + static_cast<size_t>(a->E) * 8 + static_cast<size_t>(a->P) * 4 +
                   static_cast<size_t>(a->E) * 2 + static_cast<size_t>(a->E + 1) * 2 + static_cast<size_t>(a->P);
    a->bytes_b = T8 <= 8 ? 24 * 1024 : 48 * 1024;  // at least 12 and 3 stages of the largest token tile
    a->part_floats = static_cast<int>(experts_part_floats(a->T));
    const size_t room = kSmemMax - sizeof(Shared) - 1024 - lists - a->bytes_b - 64;
    a->stages = static_cast<int>(room / kStageA);
    if (a->stages > kMaxStagesA)
        a->stages = kMaxStagesA;
    return 1024 + static_cast<size_t>(a->stages) * kStageA + a->bytes_b + lists;
}

cudaError_t launch_experts(const ExpertsArgs &a, int grid, size_t smem, cudaStream_t stream)
{
    static const cudaError_t attr =
        cudaFuncSetAttribute(experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax - 64 - static_cast<int>(sizeof(Shared)));
    if (attr != cudaSuccess)
        return attr;
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

cudaError_t experts_binary_version(int *v)
{
    cudaFuncAttributes fa;
    const cudaError_t ce = cudaFuncGetAttributes(&fa, experts_kernel);
    if (ce == cudaSuccess)
        *v = fa.binaryVersion;
    return ce;
}

}  // namespace moe
