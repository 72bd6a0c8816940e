// moe_internal.h -- argument blocks and launchers shared by the C ABI of the
// MoE operators (moe_host.cu) and their kernels. Not installed.
#pragma once

#include <cstddef>
#include <cstdint>
#include <vector>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ep_internal.h"
#include "ep_moe.h"

namespace moe {

constexpr int kMaxTokens = EP_MOE_MAX_TOKENS;    // rows of one experts or linear call
constexpr int kMaxLocal = EP_MOE_MAX_EXPERTS;    // experts of one handle

constexpr int kTileRows = 128;              // weight rows of a tile: the MMA's M
constexpr int kSmemMax = 227 * 1024;        // shared memory of a block, static and dynamic
constexpr int kChunk = 64;                  // inputs of a 16-bit chunk: one 128-byte swizzled row

// ---- router (moe_router.cu) -------------------------------------------------------

// Experts of one MMA of the router: all, or half of them where there are more
// than 256, rounded up to a multiple of 32.
static __host__ __device__ inline int router_columns(int E)
{
    const int one = (E + 31) & ~31;
    return one <= 256 ? one : ((E + 1) / 2 + 31) & ~31;
}

// Columns of the router's accumulator.
static __host__ __device__ inline int router_all_columns(int E)
{
    const int one = router_columns(E);
    return E > one ? 2 * one : one;
}

struct RouterArgs {
    CUtensorMap mx;  // x [T, H], boxes 64 x rows (many tokens)
    CUtensorMap mw;  // weight [E, H], boxes 64 x half of the accumulator's columns
    const void *x, *weight;
    const float *bias;
    long long x_stride;
    int32_t *ids;
    float *weights;
    float *parts;   // workspace
    int *counters;  // zero between launches
    unsigned int *err;
    int T, H, E, K, bf16, scoring, groups, top_groups, renormalize, sms;
    int rows, stages, tmem_cols;
    float scale;
    epk::CheckCtx chk;
};

size_t router_workspace(const RouterArgs &a);
int router_counters(int sms);  // words, a multiple of 64
size_t router_few_parts(const RouterArgs &a);  // bytes of parts for up to kMaxTokens rows
bool router_many(const RouterArgs &a);  // whether the launch uses mx and mw
int router_rows(const RouterArgs &a);   // box rows of mx
// A kernel's attributes belong to one device's copy of it: the setups set, on the current device, those that the
// launches of a handle with these arguments need. Called whenever a handle is made.
cudaError_t router_setup(const RouterArgs &a);
cudaError_t launch_router(const RouterArgs &a, cudaStream_t stream);
std::vector<const void *> router_kernels();  // every kernel of the file

// ---- experts with dense bf16 weights (moe_experts.cu) ---------------------------

constexpr int kStageA = kTileRows * kChunk * 2;

struct ExpertsArgs {
    CUtensorMap mx;   // x [T, H], one-row boxes of 64 columns
    CUtensorMap mw1;  // w_gate_up [2 E, I, H], boxes 64 x 128
    CUtensorMap mw2;  // w_down [E, H, I], boxes 64 x 128
    CUtensorMap mh;   // h [2 P, I] (high parts, then low parts), boxes 64 x 8
    const int32_t *ids;
    const float *weights;
    __nv_bfloat16 *out;
    long long out_stride;
    __nv_bfloat16 *h;
    float *part;
    int *done;     // finished (row tile, token) pairs of the first product
    int *leaving;  // blocks that are done with the counters
    int *tiles;    // per tile: parts that have been written
    unsigned int *err;  // host memory: set when a wait ran out
    int T, K, P, H, I, E, first;
    int mt1, kc1, mt2, kc2;  // row tiles and chunks of the two products
    int h_stride;
    int stages, bytes_b, part_floats;
    epk::CheckCtx chk;
};

cudaError_t experts_setup();
cudaError_t launch_experts(const ExpertsArgs &a, int grid, size_t smem, cudaStream_t stream);
std::vector<const void *> experts_kernels();  // every kernel of the file
// Dynamic shared memory of a launch for T tokens; sets stages, bytes_b and part_floats.
size_t experts_smem(ExpertsArgs *a);
// Floats of one block's part (two per block) for up to T tokens.
size_t experts_part_floats(int T);

// ---- products with 4-bit weights (moe_int4.cu) -------------------------------------

struct Int4Args {
    CUtensorMap mx;  // x: boxes 32 x 1 of [T, H], or boxes 32 x tokens x 4 (linear: 8) of [H / 32, T, 32]
    const uint8_t *w1, *w2;  // packed tiles [matrix][row tile][chunk]
    const int32_t *ids;
    const float *weights;
    void *out;
    long long out_stride;
    __nv_bfloat16 *h;
    float *part;
    int *done, *leaving, *tiles;
    unsigned int *err;
    int T, K, P, E, first;
    int H, I;  // linear: inputs, outputs
    int mt1, kc1, mt2, kc2;
    int group1, group2, shift1, shift2;  // shift: log2(group / 32)
    int zeros1, zeros2, tile1, tile2, scale_fp16;
    int h_stride;
    int smem, fixed_bytes, stage_a, part_floats, box_bytes;
    epk::CheckCtx chk;
};

constexpr int kInt4StagesA = 12, kInt4StagesB = 16;  // most stages of the rings of weights and tokens
constexpr int kInt4SumStride = kTileRows + 4;        // column stride of the groups' sums: fragments' stores hit all banks
constexpr int kInt4Groups = 4;                       // groups of four warps that multiply

// Dynamic shared memory of the 4-bit kernel, in bytes from its first 128-byte
// boundary on: what does not depend on the ids (fixed_bytes), the groups' sums
// of this launch's largest entry, the rings. Two pairs of groups take the units
// in turn, each from its own stage on, so a ring has two stages at least: every
// handle that can be made has room for them (the CPU tests try all).
struct Int4Layout {
    int cols;                  // columns of a sum
    int stage_b[2], stages_b[2];  // token rings of the two products: bytes of a stage, stages
    int stages;                // of the weights' ring
    int sums, ring_b, ring_a;  // where they begin
};

// smem: bytes there are. A unit's token tile, in 8-token steps of 2 KB a chunk: two chunks, or one (and in the second
// product two chunks in two parts). The second product's ring begins where the first's did, which is empty by then: h
// is complete when every block is through with the first. The rings share the room so that about as many token tiles
// as weight tiles are on their way.
static __host__ __device__ __forceinline__ Int4Layout int4_layout(bool linear, int smem, int fixed_bytes, int stage_a,
                                                                  int nmax)
{
    const auto least = [](int x, int y) { return x < y ? x : y; };
    Int4Layout l;
    l.cols = (nmax + 7) & ~7;
    l.stage_b[0] = l.cols * (linear ? 512 : 256);
    l.stage_b[1] = l.cols * (linear ? 512 : 1024);
    l.sums = (fixed_bytes + 127) & ~127;
    l.ring_b = l.sums + kInt4Groups * l.cols * kInt4SumStride * 4;
    const int room = smem - l.ring_b, both = least(kInt4StagesB, room / (stage_a + l.stage_b[1]));
    l.stages_b[1] = both < 2 ? 2 : both;
    l.stages_b[0] = least(kInt4StagesB, l.stages_b[1] * l.stage_b[1] / l.stage_b[0]);
    l.ring_a = l.ring_b + l.stages_b[1] * l.stage_b[1];
    l.stages = least(kInt4StagesA, (smem - l.ring_a) / stage_a);
    return l;
}

struct PackArgs {
    const uint8_t *codes;    // [mats, rows, cols / 2]
    const uint16_t *scales;  // [mats, rows, cols / group]
    const uint8_t *zeros;    // likewise, or NULL
    uint8_t *dst;
    long long mats;
    int rows, cols, group, mt, kc, tile_bytes;
    int pairs;  // tiles of matrices 2 i and 2 i + 1 side by side
};

int int4_tile_bytes(int group, bool zeros);  // of one tile of 128 rows x 128 inputs
size_t int4_part_floats(int T, bool linear);
size_t int4_h_rows(int T, int K, int E);
int int4_linear_rows(int T);  // rows of x one run over the weight takes: T in one or two runs, a multiple of 8
size_t int4_smem(Int4Args *a, bool linear);
cudaError_t int4_setup(bool linear);
cudaError_t launch_int4(const Int4Args &a, bool linear, bool bf16, int grid, size_t smem, cudaStream_t stream);
cudaError_t launch_pack(const PackArgs &a, cudaStream_t stream);
std::vector<const void *> int4_kernels();  // every kernel of the file

// Binary versions of this library's MoE kernels, as epk::kernel_binary_versions.
cudaError_t kernel_binary_versions(int *out, int max, int *n);

}  // namespace moe
