// moe_host.cu -- the C ABI of include/ep_moe.h: handles, argument checks,
// tensor maps and launches of the MoE operators.
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "moe_internal.h"

namespace {

using epk::set_error;

#define MOE_FAIL(...) return set_error(EP_ERR_INVALID_ARG, __VA_ARGS__)

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

ep_status cuda_error(cudaError_t ce, const char *what)
{
    cudaGetLastError();
    return set_error(ce == cudaErrorMemoryAllocation ? EP_ERR_OOM : EP_ERR_CUDA, "%s: %s", what,
                     cudaGetErrorString(ce));
}

// The current device, which must be able to run the library.
ep_status current_device(int *dev, int *sms)
{
    cudaError_t ce = cudaGetDevice(dev);
    if (ce != cudaSuccess)
        return cuda_error(ce, "cudaGetDevice");
    if (!ep_is_supported())
        return set_error(EP_ERR_UNSUPPORTED, "device %d is not compute capability 10.3 (sm_103)", *dev);
    if (sms) {
        ce = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
        if (ce != cudaSuccess)
            return cuda_error(ce, "cudaDeviceGetAttribute");
    }
#if EP_CHECKED
    if (!epk::check_record())
        return EP_ERR_CUDA;
#endif
    return EP_OK;
}

ep_status same_device(int want)
{
    int dev = -1;
    const cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess)
        return cuda_error(ce, "cudaGetDevice");
    if (dev != want)
        MOE_FAIL("handle lives on device %d but device %d is current", want, dev);
    return EP_OK;
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not link libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A 16-bit tensor [.., rows, cols]: row stride and matrix stride in elements,
// box_cols x box_rows boxes in 128-byte swizzled rows, zeros outside.
ep_status encode_map(CUtensorMap *m, const char *what, int fp16, const void *base, long long cols, long long rows,
                     long long mats, long long row_stride, long long mat_stride, int box_cols, int box_rows)
{
    EncodeTiled fn = encode_tiled();
    if (!fn)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint32_t rank = mats > 0 ? 3 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(mats > 0 ? mats : 1)};
    const cuuint64_t strides[2] = {cuuint64_t(row_stride) * 2, cuuint64_t(mat_stride) * 2};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1}, step[3] = {1, 1, 1};
    const CUresult r = fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                          const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled of %s: error %d", what, static_cast<int>(r));
    return EP_OK;
}

// Device words and the host flag of a handle whose blocks wait for one another.
struct Flags {
    unsigned int *err = nullptr;  // pinned host memory the kernels can write

    ep_status make()
    {
        const cudaError_t ce = cudaHostAlloc(reinterpret_cast<void **>(&err), 64, cudaHostAllocPortable);
        if (ce != cudaSuccess)
            return cuda_error(ce, "cudaHostAlloc");
        for (int i = 0; i < 16; ++i)
            err[i] = 0;
        return EP_OK;
    }
    void free()
    {
        if (err)
            cudaFreeHost(err);
        err = nullptr;
    }
    // EP_ERR_CUDA, once, after a call whose wait ran out.
    ep_status take() const
    {
        volatile unsigned int *v = err;  // [0] blocks that gave up, [site] those whose first wait to run out was there
        if (v[0] == 0)
            return EP_OK;
        unsigned int n[16];
        for (int i = 0; i < 16; ++i) {
            n[i] = v[i];
            v[i] = 0;
        }
        return set_error(EP_ERR_CUDA,
                         "waits inside an earlier call on this handle ran out in %u blocks, its output is undefined "
                         "(weights free %u, tokens free %u, sums free %u, weights %u, tokens %u, sums %u, products %u, "
                         "other %u)",
                         n[0], n[1], n[2], n[3], n[4], n[5], n[6], n[7], n[8]);
    }
};

ep_status finish(cudaError_t ce, const char *what, unsigned long long *rec, cudaStream_t stream)
{
    if (ce != cudaSuccess)
        return cuda_error(ce, what);
    const ep_status st = epk::check_after(rec, stream, what);
    return st == EP_OK ? set_error(EP_OK, "") : st;
}

}  // namespace

// ---- router ---------------------------------------------------------------------------

struct ep_router {
    ep_router_config cfg;
    int device;
};

namespace {

ep_status check_router(const ep_router_config *c)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (c->num_experts < 1 || c->num_experts > EP_MOE_MAX_EXPERTS)
        MOE_FAIL("num_experts=%d outside [1, %d]", c->num_experts, EP_MOE_MAX_EXPERTS);
    if (c->hidden < 8 || c->hidden > EP_MOE_MAX_DIM || c->hidden % 8)
        MOE_FAIL("hidden=%d must be a multiple of 8 in [8, %d]", c->hidden, EP_MOE_MAX_DIM);
    if (c->dtype != EP_DTYPE_BF16 && c->dtype != EP_DTYPE_FP16)
        MOE_FAIL("dtype %d: use bf16 or fp16", static_cast<int>(c->dtype));
    if (c->scoring != EP_SCORE_SOFTMAX && c->scoring != EP_SCORE_SIGMOID)
        MOE_FAIL("unknown scoring %d", static_cast<int>(c->scoring));
    if (c->num_groups < 1 || c->num_groups > 32 || c->num_experts % c->num_groups)
        MOE_FAIL("num_groups=%d must divide num_experts=%d and be at most 32", c->num_groups, c->num_experts);
    if (c->top_groups < 1 || c->top_groups > c->num_groups)
        MOE_FAIL("top_groups=%d outside [1, num_groups=%d]", c->top_groups, c->num_groups);
    const int open = c->num_experts / c->num_groups * c->top_groups;
    if (c->top_k < 1 || c->top_k > EP_MAX_TOP_K || c->top_k > open)
        MOE_FAIL("top_k=%d outside [1, %d] or above the %d experts that can be chosen", c->top_k, EP_MAX_TOP_K, open);
    if (!std::isfinite(c->scale))
        MOE_FAIL("scale is not finite");
    if (!c->weight || !aligned(c->weight, 16))
        MOE_FAIL("weight is NULL or not 16-byte aligned");
    if (!aligned(c->bias, 4))
        MOE_FAIL("bias is not 4-byte aligned");
    return EP_OK;
}

moe::RouterArgs router_args(const ep_router_config &c, int num_tokens)
{
    moe::RouterArgs a = {};
    a.weight = c.weight;
    a.bias = c.bias;
    a.T = num_tokens;
    a.H = c.hidden;
    a.E = c.num_experts;
    a.K = c.top_k;
    a.bf16 = c.dtype == EP_DTYPE_BF16;
    a.scoring = c.scoring;
    a.groups = c.num_groups;
    a.top_groups = c.top_groups;
    a.renormalize = c.renormalize != 0;
    a.scale = c.scale;
    return a;
}

}  // namespace

extern "C" {

ep_status ep_router_create(const ep_router_config *cfg, ep_router **out)
{
    if (!out)
        MOE_FAIL("out is NULL");
    *out = nullptr;
    ep_status st = check_router(cfg);
    if (st != EP_OK)
        return st;
    int dev = 0;
    st = current_device(&dev, nullptr);
    if (st != EP_OK)
        return st;
    ep_router *r = new (std::nothrow) ep_router();
    if (!r)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    r->cfg = *cfg;
    r->device = dev;
    *out = r;
    return set_error(EP_OK, "");
}

ep_status ep_router_workspace_size(const ep_router *r, int num_tokens, size_t *bytes)
{
    if (!r || !bytes)
        MOE_FAIL("handle or bytes is NULL");
    if (num_tokens < 0)
        MOE_FAIL("num_tokens=%d < 0", num_tokens);
    *bytes = moe::router_workspace(router_args(r->cfg, num_tokens));
    return set_error(EP_OK, "");
}

ep_status ep_router_run(ep_router *r, const void *x, long long x_stride, int num_tokens, int32_t *ids,
                        float *weights, void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("ep_router_run");
    if (!r)
        MOE_FAIL("handle is NULL");
    if (num_tokens < 0)
        MOE_FAIL("num_tokens=%d < 0", num_tokens);
    ep_status st = same_device(r->device);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    if (!x || !aligned(x, 16))
        MOE_FAIL("x is NULL or not 16-byte aligned");
    if (x_stride < r->cfg.hidden || x_stride % 8)
        MOE_FAIL("x_stride=%lld must be a multiple of 8 and at least hidden=%d", x_stride, r->cfg.hidden);
    if (!ids || !weights || !aligned(ids, 4) || !aligned(weights, 4))
        MOE_FAIL("ids or weights is NULL or not 4-byte aligned");
    moe::RouterArgs a = router_args(r->cfg, num_tokens);
    const size_t need = moe::router_workspace(a);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
        MOE_FAIL("workspace has %zu bytes, needs %zu, 256-byte aligned", workspace ? workspace_bytes : size_t(0), need);
    a.x = x;
    a.x_stride = x_stride;
    a.ids = ids;
    a.weights = weights;
    a.logits = static_cast<float *>(workspace);
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_router(a, s), "ep_router_run", rec, s);
}

ep_status ep_router_destroy(ep_router *r)
{
    delete r;
    return set_error(EP_OK, "");
}

}  // extern "C"

// ---- experts ----------------------------------------------------------------------------

struct ep_experts {
    ep_experts_config cfg;
    int device, sms;
    uint8_t *ws;
    bool owns_ws;
    Flags flags;
    CUtensorMap mw1, mw2;
};

namespace {

struct ExpertsLayout {
    size_t off_h, off_part, off_words, words, total;
    int h_stride, pairs;
};

// Workspace for the largest call: h [2][pairs][intermediate] bf16, two fp32
// parts per block, the counters.
ep_status plan_experts(const ep_experts_config *c, ExpertsLayout *l)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (c->num_experts < 1 || c->num_experts > EP_MOE_MAX_EXPERTS)
        MOE_FAIL("num_experts=%d outside [1, %d]", c->num_experts, EP_MOE_MAX_EXPERTS);
    if (c->first_expert < 0)
        MOE_FAIL("first_expert=%d < 0", c->first_expert);
    if (c->top_k < 1 || c->top_k > EP_MAX_TOP_K)
        MOE_FAIL("top_k=%d outside [1, %d]", c->top_k, EP_MAX_TOP_K);
    const int hi[2] = {c->hidden, c->intermediate};
    const char *const names[2] = {"hidden", "intermediate"};
    for (int i = 0; i < 2; ++i)
        if (hi[i] < 8 || hi[i] > EP_MOE_MAX_DIM || hi[i] % 8)
            MOE_FAIL("%s=%d must be a multiple of 8 in [8, %d]", names[i], hi[i], EP_MOE_MAX_DIM);
    if (c->max_tokens < 1 || c->max_tokens > EP_MOE_MAX_TOKENS)
        MOE_FAIL("max_tokens=%d outside [1, %d]", c->max_tokens, EP_MOE_MAX_TOKENS);
    const ep_weight *const w[2] = {&c->gate_up, &c->down};
    for (int i = 0; i < 2; ++i) {
        if (!w[i]->data || !aligned(w[i]->data, 16))
            MOE_FAIL("%s: data is NULL or not 16-byte aligned", i ? "down" : "gate_up");
        if (w[i]->group != 0)
            MOE_FAIL("%s: unknown group %d", i ? "down" : "gate_up", w[i]->group);
    }
    l->pairs = c->max_tokens * c->top_k;
    l->h_stride = (c->intermediate + 63) / 64 * 64;
    size_t off = 0;
    l->off_h = off;
    off += align256(size_t(2) * l->pairs * l->h_stride * 2);
    l->off_part = off;
    off += align256(moe::experts_part_floats(c->max_tokens) * 4 * 2 * 256);  // up to 256 blocks
    l->off_words = off;
    const size_t mt1 = (c->intermediate + moe::kTileRows - 1) / moe::kTileRows;
    const size_t mt2 = (c->hidden + moe::kTileRows - 1) / moe::kTileRows;
    l->words = 64 + c->num_experts * mt1 + mt2;
    off += align256(l->words * 4);
    l->total = off;
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_experts_workspace_size(const ep_experts_config *cfg, size_t *bytes)
{
    if (!bytes)
        MOE_FAIL("bytes is NULL");
    ExpertsLayout l{};
    const ep_status st = plan_experts(cfg, &l);
    if (st != EP_OK)
        return st;
    *bytes = l.total;
    return set_error(EP_OK, "");
}

ep_status ep_experts_create(const ep_experts_config *cfg, void *workspace, size_t bytes, ep_experts **out)
{
    if (!out)
        MOE_FAIL("out is NULL");
    *out = nullptr;
    ExpertsLayout l{};
    ep_status st = plan_experts(cfg, &l);
    if (st != EP_OK)
        return st;
    if (workspace && (!aligned(workspace, 256) || bytes < l.total))
        MOE_FAIL("workspace has %zu bytes, needs %zu, 256-byte aligned", bytes, l.total);
    int dev = 0, sms = 0;
    st = current_device(&dev, &sms);
    if (st != EP_OK)
        return st;
    ep_experts *h = new (std::nothrow) ep_experts();
    if (!h)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    h->cfg = *cfg;
    h->device = dev;
    h->sms = sms < 256 ? sms : 256;
    h->ws = static_cast<uint8_t *>(workspace);
    h->owns_ws = workspace == nullptr;
    const long long E = cfg->num_experts, H = cfg->hidden, I = cfg->intermediate;
    st = encode_map(&h->mw1, "gate_up", 0, cfg->gate_up.data, H, I, 2 * E, H, I * H, moe::kChunk, moe::kTileRows);
    if (st == EP_OK)
        st = encode_map(&h->mw2, "down", 0, cfg->down.data, I, H, E, I, H * I, moe::kChunk, moe::kTileRows);
    if (st == EP_OK)
        st = h->flags.make();
    if (st == EP_OK && h->owns_ws) {
        const cudaError_t ce = cudaMalloc(reinterpret_cast<void **>(&h->ws), l.total);
        if (ce != cudaSuccess) {
            h->ws = nullptr;
            st = cuda_error(ce, "cudaMalloc");
        }
    }
    if (st == EP_OK) {
        cudaError_t ce = cudaMemset(h->ws + l.off_words, 0, l.words * 4);
        if (ce == cudaSuccess)
            ce = cudaStreamSynchronize(nullptr);
        if (ce != cudaSuccess)
            st = cuda_error(ce, "clearing the counters");
    }
    if (st != EP_OK) {
        h->flags.free();
        if (h->owns_ws && h->ws)
            cudaFree(h->ws);
        delete h;
        return st;
    }
    *out = h;
    return set_error(EP_OK, "");
}

ep_status ep_experts_run(ep_experts *h, const void *x, long long x_stride, const int32_t *ids,
                         const float *weights, int num_tokens, void *out, long long out_stride, void *stream)
{
    Range range("ep_experts_run");
    if (!h)
        MOE_FAIL("handle is NULL");
    const ep_experts_config &c = h->cfg;
    if (num_tokens < 0 || num_tokens > c.max_tokens)
        MOE_FAIL("num_tokens=%d outside [0, max_tokens=%d]", num_tokens, c.max_tokens);
    ep_status st = same_device(h->device);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    if (!x || !aligned(x, 16))
        MOE_FAIL("x is NULL or not 16-byte aligned");
    if (x_stride < c.hidden || x_stride % 8)
        MOE_FAIL("x_stride=%lld must be a multiple of 8 and at least hidden=%d", x_stride, c.hidden);
    if (!ids || !weights || !aligned(ids, 4) || !aligned(weights, 4))
        MOE_FAIL("ids or weights is NULL or not 4-byte aligned");
    if (!out || !aligned(out, 2) || out_stride < c.hidden)
        MOE_FAIL("out is NULL, not 2-byte aligned, or out_stride=%lld < hidden=%d", out_stride, c.hidden);
    st = h->flags.take();
    if (st != EP_OK)
        return st;
    ExpertsLayout l{};
    st = plan_experts(&c, &l);
    if (st != EP_OK)
        return st;
    moe::ExpertsArgs a = {};
    a.mw1 = h->mw1;
    a.mw2 = h->mw2;
    a.T = num_tokens;
    a.K = c.top_k;
    a.P = num_tokens * c.top_k;
    a.H = c.hidden;
    a.I = c.intermediate;
    a.E = c.num_experts;
    a.first = c.first_expert;
    a.h = reinterpret_cast<__nv_bfloat16 *>(h->ws + l.off_h);
    a.h_stride = l.h_stride;
    st = encode_map(&a.mx, "x", 0, x, a.H, a.T, 0, x_stride, 0, moe::kChunk, 1);
    if (st == EP_OK)
        st = encode_map(&a.mh, "h", 0, a.h, a.I, 2LL * a.P, 0, a.h_stride, 0, moe::kChunk, 8);
    if (st != EP_OK)
        return st;
    a.ids = ids;
    a.weights = weights;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.out_stride = out_stride;
    a.part = reinterpret_cast<float *>(h->ws + l.off_part);
    int *const words = reinterpret_cast<int *>(h->ws + l.off_words);
    a.done = words;
    a.leaving = words + 32;
    a.tiles = words + 64;
    a.err = h->flags.err;
    a.mt1 = (a.I + moe::kTileRows - 1) / moe::kTileRows;
    a.kc1 = (a.H + moe::kChunk - 1) / moe::kChunk;
    a.mt2 = (a.H + moe::kTileRows - 1) / moe::kTileRows;
    a.kc2 = (a.I + moe::kChunk - 1) / moe::kChunk;
    const size_t smem = moe::experts_smem(&a);
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_experts(a, h->sms, smem, s), "ep_experts_run", rec, s);
}

ep_status ep_experts_destroy(ep_experts *h)
{
    if (h) {
        if (h->owns_ws && h->ws)
            cudaFree(h->ws);  // waits for work that uses it
        h->flags.free();
        delete h;
    }
    return set_error(EP_OK, "");
}

}  // extern "C"

cudaError_t moe::kernel_binary_versions(int *out, int max, int *n)
{
    cudaError_t (*const fns[])(int *) = {moe::router_binary_version, moe::experts_binary_version};
    *n = 0;
    for (auto *f : fns) {
        int v = 0;
        const cudaError_t ce = f(&v);
        if (ce != cudaSuccess)
            return ce;
        if (*n < max)
            out[(*n)++] = v;
    }
    return cudaSuccess;
}
