// fake_runtime.cpp -- a stand-in for the CUDA runtime, on the CPU: the
// library's own objects are linked with it, so that what their host code asks
// of the runtime can be seen without a GPU. "Device memory" is host memory,
// nothing runs, every launch is recorded and refused where a device would
// refuse it: dynamic shared memory above 48 KB needs the kernel's attribute,
// which belongs to the device that was current when it was set.
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <utility>
#include <vector>

#include "moe_internal.h"

namespace {

struct Launch {
    std::string name;  // mangled
    int device;
    dim3 grid, block;
    size_t smem;
    std::vector<unsigned char> args;  // the argument block of kernels that have one of moe_internal.h's
};

struct State {
    int device = 0, sms = 152;
    std::map<const void *, std::string> names;
    std::map<std::pair<int, const void *>, int> smem;  // (device, kernel): largest dynamic shared memory
    std::vector<Launch> launches;
    std::vector<std::string> calls;  // that wait for a device or free memory, in order
    std::vector<unsigned int *> pinned;
    int box[3] = {0, 0, 0};  // of the last tensor map
    dim3 grid, block;        // of a launch that is being made
    size_t dyn = 0;
    cudaError_t last = cudaSuccess;
};

State &state()
{
    static State s;
    return s;
}

cudaError_t result(cudaError_t e)
{
    if (e != cudaSuccess)
        state().last = e;
    return e;
}

cudaError_t record(const void *func, dim3 grid, dim3 block, size_t smem, void **args)
{
    State &s = state();
    const auto name = s.names.find(func);
    if (name == s.names.end())
        return result(cudaErrorInvalidDeviceFunction);
    const auto at = s.smem.find({s.device, func});
    if (smem > static_cast<size_t>(at == s.smem.end() ? 48 * 1024 : at->second))
        return result(cudaErrorInvalidValue);
    Launch l{name->second, s.device, grid, block, smem, {}};
    const size_t bytes = l.name.find("many_kernel") != std::string::npos   ? sizeof(moe::RouterArgs)
                         : l.name.find("int4_kernel") != std::string::npos ? sizeof(moe::Int4Args)
                         : l.name.find("experts_kernel") != std::string::npos ? sizeof(moe::ExpertsArgs)
                                                                           : 0;
    if (bytes)
        l.args.assign(static_cast<unsigned char *>(args[0]), static_cast<unsigned char *>(args[0]) + bytes);
    s.launches.push_back(l);
    return cudaSuccess;
}

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t rank, void *, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *box, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    for (int i = 0; i < 3; ++i)
        state().box[i] = i < static_cast<int>(rank) ? static_cast<int>(box[i]) : 1;
    return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// ---- what compiled code registers and how it launches --------------------------

void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *,
                            int *)
{
    state().names[host] = name;
}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t *kernel, const void *func)
{
    *kernel = reinterpret_cast<cudaKernel_t>(const_cast<void *>(func));
    return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t)
{
    state().grid = grid;
    state().block = block;
    state().dyn = smem;
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream)
{
    *grid = state().grid;
    *block = state().block;
    *smem = state().dyn;
    *static_cast<cudaStream_t *>(stream) = nullptr;
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t kernel, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t)
{
    return record(kernel, grid, block, smem, args);
}

// ---- the runtime's functions that the library calls --------------------------------

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *func, void **args)
{
    return record(func, c->gridDim, c->blockDim, c->dynamicSmemBytes, args);
}
cudaError_t cudaFuncSetAttribute(const void *func, cudaFuncAttribute attr, int value)
{
    if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize)
        state().smem[{state().device, func}] = value;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *)
{
    memset(a, 0, sizeof(*a));
    a->binaryVersion = 103;
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int *d)
{
    *d = state().device;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int d)
{
    state().device = d;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr attr, int)
{
    *v = attr == cudaDevAttrComputeCapabilityMajor   ? 10
         : attr == cudaDevAttrComputeCapabilityMinor ? 3
         : attr == cudaDevAttrMultiProcessorCount    ? state().sms
                                                     : 0;
    return cudaSuccess;
}
cudaError_t cudaGetLastError()
{
    const cudaError_t e = state().last;
    state().last = cudaSuccess;
    return e;
}
const char *cudaGetErrorString(cudaError_t e) { return e == cudaSuccess ? "no error" : "refused by the stand-in runtime"; }
cudaError_t cudaMalloc(void **p, size_t n) { return (*p = aligned_alloc(256, (n + 255) & ~size_t(255))) ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaMemset(void *p, int v, size_t n)
{
    memset(p, v, n);
    return cudaSuccess;
}
cudaError_t cudaFree(void *p)
{
    state().calls.push_back("cudaFree");
    free(p);
    return cudaSuccess;
}
cudaError_t cudaHostAlloc(void **p, size_t n, unsigned)
{
    *p = calloc(1, n);
    state().pinned.push_back(static_cast<unsigned int *>(*p));
    return cudaSuccess;
}
cudaError_t cudaFreeHost(void *p)
{
    state().calls.push_back("cudaFreeHost");
    free(p);
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize()
{
    state().calls.push_back("cudaDeviceSynchronize " + std::to_string(state().device));
    return cudaSuccess;
}
cudaError_t cudaLaunchHostFunc(cudaStream_t, cudaHostFn_t, void *) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *)
{
    *p = nullptr;
    return cudaErrorInvalidSymbol;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *found)
{
    *fn = reinterpret_cast<void *>(&encode);
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

// ---- what the tests ask ---------------------------------------------------------------

void fake_device(int d) { state().device = d; }
void fake_sms(int n) { state().sms = n; }
int fake_launches() { return static_cast<int>(state().launches.size()); }
void fake_clear()
{
    state().launches.clear();
    state().calls.clear();
}
// Launch i: device, grid, block, dynamic shared memory.
const char *fake_launch(int i, long long *v)
{
    const Launch &l = state().launches[i];
    const long long all[8] = {l.device,  l.grid.x,  l.grid.y,  l.grid.z,
                              l.block.x, l.block.y, l.block.z, static_cast<long long>(l.smem)};
    memcpy(v, all, sizeof(all));
    return l.name.c_str();
}
int fake_calls() { return static_cast<int>(state().calls.size()); }
const char *fake_call(int i) { return state().calls[i].c_str(); }
void fake_box(int *box) { memcpy(box, state().box, sizeof(state().box)); }
// The error words of the handle that was made last.
unsigned int *fake_error_words() { return state().pinned.back(); }
// Launch i, of the router for many tokens: rows of a tile, ring stages.
void fake_router_args(int i, int *v)
{
    const moe::RouterArgs &a = *reinterpret_cast<const moe::RouterArgs *>(state().launches[i].args.data());
    v[0] = a.rows;
    v[1] = a.stages;
}
// Every accepted call of 4-bit experts: up to `tokens` tokens, `top_k` choices, `experts` experts, weight tiles of
// groups of 32 to 128 with and without zero points, entries of 8 to 32 tokens; and every linear call. v: the fewest stages
// of the three rings, and the configuration (T, K, E, group, zeros, nmax) where the weights' ring has fewest; the
// largest number of bytes by which a launch's memory ends after what it has.
void fake_int4_walk(int tokens, int top_k, int experts, int *v)
{
    v[0] = v[1] = v[2] = 1 << 30;
    v[9] = -(1 << 30);
    const auto look = [&](bool linear, int T, int K, int E, int group, int zeros) {
        moe::Int4Args a = {};
        a.T = T;
        a.E = E;
        a.P = linear ? 0 : T * K;
        a.group1 = a.group2 = group;
        a.tile1 = moe::int4_tile_bytes(group, zeros != 0);
        a.tile2 = moe::int4_tile_bytes(128, false);  // the largest tile sets the stage
        const int have = static_cast<int>(moe::int4_smem(&a, linear)) - 127;  // the worst alignment of its start
        for (int nmax = 8; nmax <= 32 && nmax <= ((T + 7) & ~7); nmax += 8) {
            const moe::Int4Layout l = moe::int4_layout(linear, have, a.fixed_bytes, a.stage_a, nmax);
            v[1] = l.stages_b[0] < v[1] ? l.stages_b[0] : v[1];
            v[2] = l.stages_b[1] < v[2] ? l.stages_b[1] : v[2];
            const int end = l.ring_a + l.stages * a.stage_a - have;
            v[9] = end > v[9] ? end : v[9];
            if (l.stages < v[0]) {
                const int at[7] = {l.stages, T, K, E, group, zeros, nmax};
                v[0] = at[0];
                memcpy(v + 3, at + 1, 6 * sizeof(int));
            }
        }
    };
    for (int group = 32; group <= 128; group *= 2)
        for (int zeros = 0; zeros < 2; ++zeros)
            for (int T = 1; T <= tokens; ++T) {
                look(true, T, 1, 1, group, zeros);
                for (int K = 1; K <= top_k; ++K)
                    for (int E = 1; E <= experts; ++E)
                        look(false, T, K, E, group, zeros);
            }
}
// Launch i, of the 4-bit kernel: what its layout follows from.
void fake_int4_args(int i, int *v)
{
    const moe::Int4Args &a = *reinterpret_cast<const moe::Int4Args *>(state().launches[i].args.data());
    v[0] = a.smem;
    v[1] = a.fixed_bytes;
    v[2] = a.stage_a;
}
// Launch i, of the bf16 experts: stages of the weights' ring, and of the tokens' for an entry of all tokens.
void fake_experts_args(int i, int *v)
{
    const moe::ExpertsArgs &a = *reinterpret_cast<const moe::ExpertsArgs *>(state().launches[i].args.data());
    v[0] = a.stages;
    v[1] = a.bytes_b / ((a.T + 7) / 8 * 16 * 128);
}

}  // extern "C"
