// moe_host.cu -- the C ABI of include/ep_moe.h: handles, argument checks,
// tensor maps and launches of the router, the experts and the 4-bit linear layer.
#include <climits>
#include <cmath>
#include <cstring>

#include "moe_host.h"

using namespace moe_host;

// ---- router ---------------------------------------------------------------------------

struct ep_router {
    ep_router_config cfg;
    int device, sms;
    int *counters;
    Flags flags;
    CUtensorMap mw;
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

moe::RouterArgs router_args(const ep_router_config &c, int sms, int num_tokens)
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
    a.sms = sms;
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
    int dev = 0, sms = 0;
    st = current_device(&dev, &sms);
    if (st != EP_OK)
        return st;
    ep_router *r = new (std::nothrow) ep_router();
    if (!r)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    r->cfg = *cfg;
    r->device = dev;
    r->sms = sms;
    st = encode_map(&r->mw, "weight", cfg->dtype == EP_DTYPE_FP16, cfg->weight, cfg->hidden, cfg->num_experts, 0,
                    cfg->hidden, 0, moe::kChunk, moe::router_all_columns(cfg->num_experts) / 2);
    if (st == EP_OK) {
        const cudaError_t ce = moe::router_setup(router_args(*cfg, sms, 1));
        if (ce != cudaSuccess)
            st = cuda_error(ce, "the router's kernels");
    }
    if (st == EP_OK)
        st = r->flags.make();
    if (st == EP_OK) {
        const size_t bytes = moe::router_counters(sms) * sizeof(int) + moe::router_few_parts(router_args(*cfg, sms, 1));
        cudaError_t ce = cudaMalloc(reinterpret_cast<void **>(&r->counters), bytes);
        if (ce == cudaSuccess)
            ce = cudaMemset(r->counters, 0, bytes);
        if (ce == cudaSuccess)
            ce = cudaStreamSynchronize(nullptr);
        if (ce != cudaSuccess)
            st = cuda_error(ce, "the router's counters");
    }
    if (st != EP_OK) {
        if (r->counters)
            cudaFree(r->counters);
        r->flags.free();
        delete r;
        return st;
    }
    *out = r;
    return set_error(EP_OK, "");
}

ep_status ep_router_workspace_size(const ep_router *r, int num_tokens, size_t *bytes)
{
    if (!r || !bytes)
        MOE_FAIL("handle or bytes is NULL");
    if (num_tokens < 0 || num_tokens > EP_ROUTER_MAX_TOKENS)
        MOE_FAIL("num_tokens=%d outside [0, %d]", num_tokens, EP_ROUTER_MAX_TOKENS);
    *bytes = moe::router_workspace(router_args(r->cfg, r->sms, num_tokens));
    return set_error(EP_OK, "");
}

ep_status ep_router_run(ep_router *r, const void *x, long long x_stride, int num_tokens, int32_t *ids,
                        float *weights, void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("ep_router_run");
    if (!r)
        MOE_FAIL("handle is NULL");
    if (num_tokens < 0 || num_tokens > EP_ROUTER_MAX_TOKENS)
        MOE_FAIL("num_tokens=%d outside [0, %d]", num_tokens, EP_ROUTER_MAX_TOKENS);
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
    moe::RouterArgs a = router_args(r->cfg, r->sms, num_tokens);
    const size_t need = moe::router_workspace(a);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
        MOE_FAIL("workspace has %zu bytes, needs %zu, 256-byte aligned", workspace ? workspace_bytes : size_t(0), need);
    a.x = x;
    a.x_stride = x_stride;
    a.ids = ids;
    a.weights = weights;
    st = r->flags.take();
    if (st == EP_OK && moe::router_many(a))
        st = encode_map(&a.mx, "x", r->cfg.dtype == EP_DTYPE_FP16, x, a.H, a.T, 0, x_stride, 0, moe::kChunk,
                        moe::router_rows(a));
    if (st != EP_OK)
        return st;
    a.mw = r->mw;
    a.counters = r->counters;
    // a few tokens' parts are the handle's own, behind the counters
    a.parts = need ? static_cast<float *>(workspace)
                   : reinterpret_cast<float *>(r->counters + moe::router_counters(r->sms));
    a.err = r->flags.err;
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_router(a, s), "ep_router_run", rec, s);
}

ep_status ep_router_destroy(ep_router *r)
{
    if (r) {
        wait_for_device(r->device);
        cudaFree(r->counters);
        r->flags.free();
        delete r;
    }
    return set_error(EP_OK, "");
}

}  // extern "C"

// ---- 4-bit weights ------------------------------------------------------------------------

namespace {

bool is_group(int g) { return g == 32 || g == 64 || g == 128; }

ep_status check_int_weight(const ep_int_weight *w)
{
    if (!w)
        MOE_FAIL("weight is NULL");
    if (!is_group(w->group))
        MOE_FAIL("group=%d: use 32, 64 or 128", w->group);
    if (w->mats < 1 || w->rows < 1 || w->cols < 1 || w->cols % w->group)
        MOE_FAIL("mats=%d, rows=%d, cols=%d: positive, cols a multiple of group=%d", w->mats, w->rows, w->cols, w->group);
    if (w->gate_up && w->mats % 2)
        MOE_FAIL("gate_up: mats=%d is odd", w->mats);
    if (w->cols > EP_MOE_MAX_DIM || w->rows > 16 * EP_MOE_MAX_DIM || w->mats > 2 * EP_MOE_MAX_EXPERTS)
        MOE_FAIL("mats=%d, rows=%d, cols=%d are limited to %d, %d, %d", w->mats, w->rows, w->cols,
                 2 * EP_MOE_MAX_EXPERTS, 16 * EP_MOE_MAX_DIM, EP_MOE_MAX_DIM);
    if (w->scale_dtype != EP_DTYPE_BF16 && w->scale_dtype != EP_DTYPE_FP16)
        MOE_FAIL("scale_dtype %d: use bf16 or fp16", static_cast<int>(w->scale_dtype));
    return EP_OK;
}

size_t packed_size(const ep_int_weight &w)
{
    return size_t(w.mats) * div_up(w.rows, 128) * div_up(w.cols, 128) *
           moe::int4_tile_bytes(w.group, w.zeros != nullptr);
}

// The parts that experts and linear handles share: the device, the workspace and the host flag.
struct Base {
    int device = 0, sms = 0;
    uint8_t *ws = nullptr;
    bool owns_ws = false;
    Flags flags;

    // setup: sets the attributes of the handle's kernels on the current device.
    template <class Setup>
    ep_status open(void *workspace, size_t bytes, size_t need, size_t off_words, size_t words, Setup setup)
    {
        if (workspace && (!aligned(workspace, 256) || bytes < need))
            MOE_FAIL("workspace has %zu bytes, needs %zu, 256-byte aligned", bytes, need);
        ep_status st = current_device(&device, &sms);
        if (st != EP_OK)
            return st;
        sms = sms < kMaxBlocks ? sms : kMaxBlocks;
        cudaError_t ce = setup();
        if (ce != cudaSuccess)
            return cuda_error(ce, "the handle's kernels");
        st = flags.make();
        if (st != EP_OK)
            return st;
        ws = static_cast<uint8_t *>(workspace);
        if (!ws) {
            ce = cudaMalloc(reinterpret_cast<void **>(&ws), need);
            if (ce != cudaSuccess) {
                ws = nullptr;
                return cuda_error(ce, "cudaMalloc");
            }
            owns_ws = true;
        }
        ce = cudaMemset(ws + off_words, 0, words * 4);
        if (ce == cudaSuccess)
            ce = cudaStreamSynchronize(nullptr);
        return ce == cudaSuccess ? EP_OK : cuda_error(ce, "clearing the counters");
    }
    void close()
    {
        if (ws)  // the handle was made: work that uses it may be queued
            wait_for_device(device);
        if (owns_ws && ws)
            cudaFree(ws);
        ws = nullptr;
        flags.free();
    }
    static constexpr int kMaxBlocks = 256;
};

constexpr size_t kWords = 64;  // done at 0, leaving at 32, then the tiles' counters

template <class Args> void set_words(Args &a, uint8_t *words)
{
    int *const w = reinterpret_cast<int *>(words);
    a.done = w;
    a.leaving = w + 32;
    a.tiles = w + kWords;
}

}  // namespace

extern "C" {

ep_status ep_weight_packed_size(const ep_int_weight *w, size_t *bytes)
{
    if (!bytes)
        MOE_FAIL("bytes is NULL");
    const ep_status st = check_int_weight(w);
    if (st != EP_OK)
        return st;
    *bytes = packed_size(*w);
    return set_error(EP_OK, "");
}

ep_status ep_weight_pack(const ep_int_weight *w, void *packed, size_t bytes, void *stream)
{
    Range range("ep_weight_pack");
    ep_status st = check_int_weight(w);
    if (st != EP_OK)
        return st;
    if (!w->codes || !w->scales || !aligned(w->scales, 2))
        MOE_FAIL("codes or scales is NULL or scales is not 2-byte aligned");
    if (!packed || !aligned(packed, 128) || bytes < packed_size(*w))
        MOE_FAIL("packed has %zu bytes, needs %zu, 128-byte aligned", bytes, packed_size(*w));
    int dev = 0;
    st = current_device(&dev, nullptr);
    if (st != EP_OK)
        return st;
    moe::PackArgs a = {};
    a.codes = w->codes;
    a.scales = static_cast<const uint16_t *>(w->scales);
    a.zeros = w->zeros;
    a.dst = static_cast<uint8_t *>(packed);
    a.mats = w->mats;
    a.rows = w->rows;
    a.cols = w->cols;
    a.group = w->group;
    a.mt = div_up(w->rows, 128);
    a.kc = div_up(w->cols, 128);
    a.tile_bytes = moe::int4_tile_bytes(w->group, w->zeros != nullptr);
    a.pairs = w->gate_up != 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t ce = moe::launch_pack(a, s);
    // A linear layer reads its weights while the kernel before it is finishing; what it waits for in full is
    // anything but a kernel.
    if (ce == cudaSuccess)
        ce = cudaLaunchHostFunc(s, [](void *) {}, nullptr);
    return ce == cudaSuccess ? set_error(EP_OK, "") : cuda_error(ce, "ep_weight_pack");
}

}  // extern "C"

// ---- linear -------------------------------------------------------------------------------

struct ep_linear {
    ep_linear_config cfg;
    Base base;
};

namespace {

struct LinearLayout {
    size_t off_words, words, total;
};

ep_status plan_linear(const ep_linear_config *c, LinearLayout *l)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (!is_group(c->weight.group))
        MOE_FAIL("weight: group=%d: use 32, 64 or 128", c->weight.group);
    if (c->inputs < 1 || c->inputs > EP_MOE_MAX_DIM || c->inputs % c->weight.group)
        MOE_FAIL("inputs=%d must be a multiple of group=%d in [1, %d]", c->inputs, c->weight.group, EP_MOE_MAX_DIM);
    if (c->outputs < 1 || c->outputs > 16 * EP_MOE_MAX_DIM)
        MOE_FAIL("outputs=%d outside [1, %d]", c->outputs, 16 * EP_MOE_MAX_DIM);
    if (c->max_tokens < 1 || c->max_tokens > EP_MOE_MAX_TOKENS)
        MOE_FAIL("max_tokens=%d outside [1, %d]", c->max_tokens, EP_MOE_MAX_TOKENS);
    if (c->weight.scale_dtype != EP_DTYPE_BF16 && c->weight.scale_dtype != EP_DTYPE_FP16)
        MOE_FAIL("weight: scale_dtype %d: use bf16 or fp16", static_cast<int>(c->weight.scale_dtype));
    if (!c->weight.data || !aligned(c->weight.data, 128))
        MOE_FAIL("weight: data is NULL or not 128-byte aligned");
    size_t off = align256(moe::int4_part_floats(c->max_tokens, true) * 4 * 2 * Base::kMaxBlocks);
    l->off_words = off;
    l->words = kWords + 2 * size_t(div_up(c->outputs, 128));  // up to two runs over the weight
    l->total = off + align256(l->words * 4);
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_linear_workspace_size(const ep_linear_config *cfg, size_t *bytes)
{
    if (!bytes)
        MOE_FAIL("bytes is NULL");
    LinearLayout l{};
    const ep_status st = plan_linear(cfg, &l);
    if (st != EP_OK)
        return st;
    *bytes = l.total;
    return set_error(EP_OK, "");
}

ep_status ep_linear_create(const ep_linear_config *cfg, void *workspace, size_t bytes, ep_linear **out)
{
    if (!out)
        MOE_FAIL("out is NULL");
    *out = nullptr;
    LinearLayout l{};
    ep_status st = plan_linear(cfg, &l);
    if (st != EP_OK)
        return st;
    ep_linear *h = new (std::nothrow) ep_linear();
    if (!h)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    h->cfg = *cfg;
    st = h->base.open(workspace, bytes, l.total, l.off_words, l.words, [] { return moe::int4_setup(true); });
    if (st != EP_OK) {
        h->base.close();
        delete h;
        return st;
    }
    *out = h;
    return set_error(EP_OK, "");
}

ep_status ep_linear_run(ep_linear *h, ep_dtype dtype, const void *x, long long x_stride, int num_tokens, void *y,
                        long long y_stride, void *stream)
{
    Range range("ep_linear_run");
    if (!h)
        MOE_FAIL("handle is NULL");
    const ep_linear_config &c = h->cfg;
    if (num_tokens < 0 || num_tokens > c.max_tokens)
        MOE_FAIL("num_tokens=%d outside [0, max_tokens=%d]", num_tokens, c.max_tokens);
    ep_status st = same_device(h->base.device);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    if (dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_FP16)
        MOE_FAIL("dtype %d: use bf16 or fp16", static_cast<int>(dtype));
    st = check_rows("x", x, x_stride, c.inputs, 16, 8);
    if (st == EP_OK)
        st = check_rows("y", y, y_stride, c.outputs, 2, 1);
    if (st == EP_OK)
        st = h->base.flags.take();
    if (st != EP_OK)
        return st;
    LinearLayout l{};
    plan_linear(&c, &l);
    moe::Int4Args a = {};
    a.T = num_tokens;
    a.E = 1;
    a.H = c.inputs;
    a.I = c.outputs;
    const int rows = moe::int4_linear_rows(a.T);
    a.box_bytes = rows * 512;
    st = encode_steps(&a.mx, "x", dtype == EP_DTYPE_FP16, x, a.H / 32, a.T, x_stride, rows, 8);
    if (st != EP_OK)
        return st;
    a.w1 = static_cast<const uint8_t *>(c.weight.data);
    a.out = y;
    a.out_stride = y_stride;
    a.part = reinterpret_cast<float *>(h->base.ws);
    set_words(a, h->base.ws + l.off_words);
    a.err = h->base.flags.err;
    a.mt1 = div_up(c.outputs, 128);
    a.kc1 = div_up(c.inputs, 128);
    a.mt2 = a.kc2 = 1;  // there is no second product
    a.group1 = a.group2 = c.weight.group;
    a.zeros1 = a.zeros2 = c.weight.has_zeros != 0;
    a.tile1 = a.tile2 = moe::int4_tile_bytes(c.weight.group, a.zeros1);
    a.scale_fp16 = c.weight.scale_dtype == EP_DTYPE_FP16;
    const size_t smem = moe::int4_smem(&a, true);
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_int4(a, true, dtype == EP_DTYPE_BF16, h->base.sms, smem, s), "ep_linear_run", rec, s);
}

ep_status ep_linear_destroy(ep_linear *h)
{
    if (h) {
        h->base.close();
        delete h;
    }
    return set_error(EP_OK, "");
}

}  // extern "C"

// ---- experts ----------------------------------------------------------------------------

struct ep_experts {
    ep_experts_config cfg;
    Base base;
    CUtensorMap mw1, mw2;  // of bf16 weights
};

namespace {

struct ExpertsLayout {
    size_t off_h, off_part, off_words, words, total;
    int h_stride;
};

// Workspace for the largest call: h [2][pairs][intermediate] bf16, two fp32
// parts per block, the counters.
ep_status plan_experts(const ep_experts_config *c, ExpertsLayout *l)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (c->num_experts < 1 || c->num_experts > EP_MOE_MAX_EXPERTS)
        MOE_FAIL("num_experts=%d outside [1, %d]", c->num_experts, EP_MOE_MAX_EXPERTS);
    if (c->first_expert < 0 || c->first_expert > INT_MAX - (c->num_experts - 1))
        MOE_FAIL("first_expert=%d: ids of %d experts must fit [0, 2^31)", c->first_expert, c->num_experts);
    if (c->top_k < 1 || c->top_k > EP_MAX_TOP_K)
        MOE_FAIL("top_k=%d outside [1, %d]", c->top_k, EP_MAX_TOP_K);
    if (c->max_tokens < 1 || c->max_tokens > EP_MOE_MAX_TOKENS)
        MOE_FAIL("max_tokens=%d outside [1, %d]", c->max_tokens, EP_MOE_MAX_TOKENS);
    const ep_weight *const w[2] = {&c->gate_up, &c->down};
    const char *const names[2] = {"gate_up", "down"};
    const int inputs[2] = {c->hidden, c->intermediate};
    const char *const of[2] = {"hidden", "intermediate"};
    if ((w[0]->group == 0) != (w[1]->group == 0))
        MOE_FAIL("gate_up and down must both be bf16 or both packed");
    for (int i = 0; i < 2; ++i) {
        if (w[i]->group != 0 && !is_group(w[i]->group))
            MOE_FAIL("%s: group=%d: use 0 (bf16), 32, 64 or 128", names[i], w[i]->group);
        const int step = w[i]->group ? w[i]->group : 8;
        if (inputs[i] < step || inputs[i] > EP_MOE_MAX_DIM || inputs[i] % step)
            MOE_FAIL("%s=%d must be a multiple of %d in [%d, %d]", of[i], inputs[i], step, step, EP_MOE_MAX_DIM);
        if (!w[i]->data || !aligned(w[i]->data, w[i]->group ? 128 : 16))
            MOE_FAIL("%s: data is NULL or not %d-byte aligned", names[i], w[i]->group ? 128 : 16);
        if (w[i]->group && (w[i]->scale_dtype != EP_DTYPE_BF16 && w[i]->scale_dtype != EP_DTYPE_FP16))
            MOE_FAIL("%s: scale_dtype %d: use bf16 or fp16", names[i], static_cast<int>(w[i]->scale_dtype));
    }
    if (w[0]->group && w[0]->scale_dtype != w[1]->scale_dtype)
        MOE_FAIL("gate_up and down must have the same scale_dtype");
    const int pairs = c->max_tokens * c->top_k;
    const size_t part = w[0]->group ? moe::int4_part_floats(c->max_tokens, false) : moe::experts_part_floats(c->max_tokens);
    size_t off = 0;
    l->off_h = off;
    if (w[0]->group) {  // a row of h in two parts, in chunks of 128 inputs
        l->h_stride = div_up(c->intermediate, 128) * 256;
        off += align256(moe::int4_h_rows(c->max_tokens, c->top_k, c->num_experts) * l->h_stride * 2);
    } else {
        l->h_stride = div_up(c->intermediate, 64) * 64;
        off += align256(size_t(2) * pairs * l->h_stride * 2);
    }
    l->off_part = off;
    off += align256(part * 4 * 2 * Base::kMaxBlocks);
    l->off_words = off;
    l->words = kWords + size_t(w[0]->group ? 2 : 1) * c->num_experts * div_up(c->intermediate, 128) +
               div_up(c->hidden, 128);
    off += align256(l->words * 4);
    l->total = off;
    return EP_OK;
}

// What both kernels' argument blocks have in common.
template <class Args>
ep_status experts_args(const ep_experts *h, Args &a, const ExpertsLayout &l, const void *x, long long x_stride,
                       int num_tokens, const int32_t *ids, const float *weights, long long out_stride, int chunk,
                       int box_cols)
{
    const ep_experts_config &c = h->cfg;
    a.T = num_tokens;
    a.K = c.top_k;
    a.P = num_tokens * c.top_k;
    a.H = c.hidden;
    a.I = c.intermediate;
    a.E = c.num_experts;
    a.first = c.first_expert;
    a.h = reinterpret_cast<__nv_bfloat16 *>(h->base.ws + l.off_h);
    a.h_stride = l.h_stride;
    a.ids = ids;
    a.weights = weights;
    a.out_stride = out_stride;
    a.part = reinterpret_cast<float *>(h->base.ws + l.off_part);
    set_words(a, h->base.ws + l.off_words);
    a.err = h->base.flags.err;
    a.mt1 = div_up(a.I, moe::kTileRows);
    a.kc1 = div_up(a.H, chunk);
    a.mt2 = div_up(a.H, moe::kTileRows);
    a.kc2 = div_up(a.I, chunk);
    if (box_cols == 32 && a.T <= 8)
        return encode_steps(&a.mx, "x", 0, x, a.H / 32, a.T, x_stride, 8, 4);
    return encode_map(&a.mx, "x", 0, x, a.H, a.T, 0, x_stride, 0, box_cols, 1);
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
    ep_experts *h = new (std::nothrow) ep_experts();
    if (!h)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    h->cfg = *cfg;
    const long long E = cfg->num_experts, H = cfg->hidden, I = cfg->intermediate;
    st = h->base.open(workspace, bytes, l.total, l.off_words, l.words,
                      [&] { return cfg->gate_up.group ? moe::int4_setup(false) : moe::experts_setup(); });
    if (st == EP_OK && cfg->gate_up.group == 0)
        st = encode_map(&h->mw1, "gate_up", 0, cfg->gate_up.data, H, I, 2 * E, H, I * H, moe::kChunk, moe::kTileRows);
    if (st == EP_OK && cfg->gate_up.group == 0)
        st = encode_map(&h->mw2, "down", 0, cfg->down.data, I, H, E, I, H * I, moe::kChunk, moe::kTileRows);
    if (st != EP_OK) {
        h->base.close();
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
    ep_status st = same_device(h->base.device);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    st = check_rows("x", x, x_stride, c.hidden, 16, 8);
    if (st == EP_OK)
        st = check_rows("out", out, out_stride, c.hidden, 2, 1);
    if (st != EP_OK)
        return st;
    if (!ids || !weights || !aligned(ids, 4) || !aligned(weights, 4))
        MOE_FAIL("ids or weights is NULL or not 4-byte aligned");
    st = h->base.flags.take();
    if (st != EP_OK)
        return st;
    ExpertsLayout l{};
    plan_experts(&c, &l);
    unsigned long long *rec = epk::check_record();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t ce;
    if (c.gate_up.group == 0) {
        moe::ExpertsArgs a = {};
        st = experts_args(h, a, l, x, x_stride, num_tokens, ids, weights, out_stride, moe::kChunk, moe::kChunk);
        if (st == EP_OK)
            st = encode_map(&a.mh, "h", 0, a.h, a.I, 2LL * a.P, 0, a.h_stride, 0, moe::kChunk, 8);
        if (st != EP_OK)
            return st;
        a.mw1 = h->mw1;
        a.mw2 = h->mw2;
        a.out = static_cast<__nv_bfloat16 *>(out);
        a.chk = epk::check_ctx(rec);
        const size_t smem = moe::experts_smem(&a);
        ce = moe::launch_experts(a, h->base.sms, smem, s);
    } else {
        moe::Int4Args a = {};
        st = experts_args(h, a, l, x, x_stride, num_tokens, ids, weights, out_stride, 128, 32);
        if (st != EP_OK)
            return st;
        a.w1 = static_cast<const uint8_t *>(c.gate_up.data);
        a.w2 = static_cast<const uint8_t *>(c.down.data);
        a.group1 = c.gate_up.group;
        a.group2 = c.down.group;
        a.zeros1 = c.gate_up.has_zeros != 0;
        a.zeros2 = c.down.has_zeros != 0;
        a.tile1 = moe::int4_tile_bytes(a.group1, a.zeros1);
        a.tile2 = moe::int4_tile_bytes(a.group2, a.zeros2);
        a.scale_fp16 = c.gate_up.scale_dtype == EP_DTYPE_FP16;
        a.out = out;
        a.box_bytes = 2048;
        a.chk = epk::check_ctx(rec);
        const size_t smem = moe::int4_smem(&a, false);
        ce = moe::launch_int4(a, false, true, h->base.sms, smem, s);
    }
    return finish(ce, "ep_experts_run", rec, s);
}

ep_status ep_layer_run(ep_router *r, ep_experts *h, const void *x, long long x_stride, int num_tokens,
                       int32_t *ids, float *weights, void *out, long long out_stride, void *stream)
{
    if (!r || !h)
        MOE_FAIL("a handle is NULL");
    if (r->cfg.hidden != h->cfg.hidden || r->cfg.top_k != h->cfg.top_k || r->cfg.dtype != EP_DTYPE_BF16)
        MOE_FAIL("router (hidden %d, top_k %d, dtype %d) and experts (hidden %d, top_k %d, bf16) differ", r->cfg.hidden,
                 r->cfg.top_k, static_cast<int>(r->cfg.dtype), h->cfg.hidden, h->cfg.top_k);
    if (num_tokens < 0 || num_tokens > h->cfg.max_tokens)
        MOE_FAIL("num_tokens=%d outside [0, max_tokens=%d]", num_tokens, h->cfg.max_tokens);
    // nothing is queued unless both calls will be: what only the second checks comes first
    ep_status st = same_device(h->base.device);
    if (st == EP_OK && num_tokens > 0)
        st = check_rows("out", out, out_stride, h->cfg.hidden, 2, 1);
    if (st == EP_OK && num_tokens > 0)
        st = h->base.flags.take();
    if (st != EP_OK)
        return st;
    st = ep_router_run(r, x, x_stride, num_tokens, ids, weights, nullptr, 0, stream);
    if (st != EP_OK)
        return st;
    return ep_experts_run(h, x, x_stride, ids, weights, num_tokens, out, out_stride, stream);
}

ep_status ep_experts_destroy(ep_experts *h)
{
    if (h) {
        h->base.close();
        delete h;
    }
    return set_error(EP_OK, "");
}

}  // extern "C"

cudaError_t moe::kernel_binary_versions(int *out, int max, int *n)
{
    *n = 0;
    for (const auto &list : {moe::router_kernels(), moe::experts_kernels(), moe::int4_kernels(), moe::norm_kernels(), moe::ffn_kernels()})
        for (const void *f : list) {
            cudaFuncAttributes attr;
            const cudaError_t ce = cudaFuncGetAttributes(&attr, f);
            if (ce != cudaSuccess)
                return ce;
            if (*n < max)
                out[(*n)++] = attr.binaryVersion;
        }
    return cudaSuccess;
}
