// moe_block_host.cu -- the C ABI of include/ep_moe.h, second part: the norm and
// the feed-forward block, their argument checks, tensor maps and launches.
#include <atomic>
#include <cmath>
#include <cstring>

#include "moe_host.h"

using namespace moe_host;

namespace {

int size_of(ep_dtype t) { return t == EP_DTYPE_FP32 ? 4 : 2; }

// An operand's memory: `rows` rows of `row` bytes, `pitch` bytes apart; p NULL: not there, nor without rows.
struct Span {
    const char *name;
    const void *p;
    long long rows;
    size_t row, pitch;
};

// Rows of `cols` elements of `size` bytes, `stride` elements apart.
Span rows_of(const char *name, const void *p, long long rows, long long cols, long long stride, int size)
{
    return {name, rows > 0 ? p : nullptr, rows, static_cast<size_t>(cols) * size, static_cast<size_t>(stride) * size};
}
Span whole(const char *name, const void *p, size_t bytes) { return {name, p, 1, bytes, bytes}; }

bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + (b.rows - 1) * b.pitch + b.row || y >= x + (a.rows - 1) * a.pitch + a.row)
        return false;
    if (a.pitch != b.pitch)
        return true;
    // columns of the same rows: b's begin where a's have ended, and end before a's begin again
    const size_t d = (y >= x ? y - x : a.pitch - (x - y) % a.pitch) % a.pitch;
    return d < a.row || d + b.row > a.pitch;
}

// An output that overlaps an input; in_place: other than as the very same rows.
ep_status check_overlap(const Span &out, const Span &in, bool in_place)
{
    if (overlap(out, in) && !(in_place && out.p == in.p && out.pitch == in.pitch))
        MOE_FAIL("%s overlaps %s", out.name, in.name);
    return EP_OK;
}

ep_status check_workspace(const void *workspace, size_t have, size_t need)
{
    if (need && (!workspace || !aligned(workspace, 256) || have < need))
        MOE_FAIL("workspace has %zu bytes, needs %zu, 256-byte aligned", workspace ? have : size_t(0), need);
    return EP_OK;
}

ep_status check_norm(const ep_norm_config *c, int num_tokens)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (c->hidden < 8 || c->hidden > EP_NORM_MAX_HIDDEN || c->hidden % 8)
        MOE_FAIL("hidden=%d must be a multiple of 8 in [8, %d]", c->hidden, EP_NORM_MAX_HIDDEN);
    if (c->dtype != EP_DTYPE_BF16 && c->dtype != EP_DTYPE_FP16 && c->dtype != EP_DTYPE_FP32)
        MOE_FAIL("dtype %d: use bf16, fp16 or fp32", static_cast<int>(c->dtype));
    if (c->weight_dtype != c->dtype && c->weight_dtype != EP_DTYPE_FP32)
        MOE_FAIL("weight_dtype %d: use dtype or fp32", static_cast<int>(c->weight_dtype));
    if (!std::isfinite(c->eps) || !(c->eps > 0.0f))
        MOE_FAIL("eps must be finite and above 0");
    if (!c->weight || !aligned(c->weight, 16))
        MOE_FAIL("weight is NULL or not 16-byte aligned");
    if (num_tokens < 0)
        MOE_FAIL("num_tokens=%d is negative", num_tokens);
    return EP_OK;
}

Span weight_span(const ep_norm_config &c) { return whole("weight", c.weight, size_t(c.hidden) * size_of(c.weight_dtype)); }

// The current device for the norm's calls, whose kernels have no handle: set up when a device is first seen.
ep_status norm_device(int *sms)
{
    static std::atomic<unsigned long long> seen{0};
    int dev = 0;
    ep_status st = current_device(&dev, sms);
    const unsigned long long bit = 1ULL << (dev & 63);
    if (st != EP_OK || (dev < 64 && (seen.load(std::memory_order_acquire) & bit)))
        return st;
    const cudaError_t ce = moe::norm_setup();
    if (ce != cudaSuccess)
        return cuda_error(ce, "the norm's kernels");
    seen.fetch_or(bit, std::memory_order_release);
    return EP_OK;
}

}  // namespace

extern "C" {

// ---- norm -----------------------------------------------------------------------------

ep_status ep_norm_run(const ep_norm_config *cfg, const ep_norm_rows *rows, int num_tokens, void *stream)
{
    Range range("ep_norm_run");
    ep_status st = check_norm(cfg, num_tokens);
    if (st != EP_OK)
        return st;
    if (!rows)
        MOE_FAIL("rows is NULL");
    moe::NormArgs a = {};
    st = norm_device(&a.sms);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    const ep_norm_rows &r = *rows;
    const int H = cfg->hidden, size = size_of(cfg->dtype), groups = div_up(H, EP_SCALE_GROUP);
    if (r.residual_out && !r.residual)
        MOE_FAIL("residual_out without residual");
    if ((r.q == nullptr) != (r.scales == nullptr))
        MOE_FAIL("q and scales must be given together");
    const long long strides[4] = {r.x_stride, r.residual_stride, r.residual_out_stride, r.out_stride};
    const Span all[4] = {rows_of("x", r.x, num_tokens, H, r.x_stride, size),
                         rows_of("residual", r.residual, num_tokens, H, r.residual_stride, size),
                         rows_of("residual_out", r.residual_out, num_tokens, H, r.residual_out_stride, size),
                         rows_of("out", r.out, num_tokens, H, r.out_stride, size)};
    for (int i = 0; i < 4; ++i)
        if (all[i].p || i == 0)
            if ((st = check_rows(all[i].name, all[i].p, strides[i], H, 16, 8)) != EP_OK)
                return st;
    if (!aligned(r.q, 8) || !aligned(r.scales, 4))
        MOE_FAIL("q is not 8-byte or scales not 4-byte aligned");
    const Span w = weight_span(*cfg);
    const Span eight[2] = {whole("q", r.q, size_t(num_tokens) * H), whole("scales", r.scales, size_t(num_tokens) * groups * 4)};
    for (int o = 2; o < 4 && st == EP_OK; ++o)
        for (int i = 0; i < o && st == EP_OK; ++i)
            st = check_overlap(all[o], all[i], i < 2);
    for (int o = 0; o < 4 && st == EP_OK; ++o)
        st = check_overlap(o < 2 ? all[2 + o] : eight[o - 2], w, false);
    for (int o = 0; o < 2 && st == EP_OK; ++o) {
        for (int i = 0; i < 4 && st == EP_OK; ++i)
            st = check_overlap(eight[o], all[i], false);
        for (int i = 0; i < o && st == EP_OK; ++i)
            st = check_overlap(eight[o], eight[i], false);
    }
    if (st != EP_OK)
        return st;
    a.x = r.x;
    a.residual = r.residual;
    a.weight = cfg->weight;
    a.x_stride = r.x_stride;
    a.residual_stride = r.residual_stride;
    a.residual_out_stride = r.residual_out_stride;
    a.out_stride = r.out_stride;
    a.residual_out = r.residual_out;
    a.out = r.out;
    a.q = static_cast<uint8_t *>(r.q);
    a.scales = r.scales;
    a.T = num_tokens;
    a.H = H;
    a.groups = groups;
    a.dtype = cfg->dtype;
    a.weight_fp32 = cfg->weight_dtype == EP_DTYPE_FP32;
    a.eps = cfg->eps;
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_norm(a, s), "ep_norm_run", rec, s);
}

ep_status ep_norm_backward_workspace_size(const ep_norm_config *cfg, int num_tokens, size_t *bytes)
{
    if (!bytes)
        MOE_FAIL("bytes is NULL");
    ep_status st = check_norm(cfg, num_tokens);
    if (st != EP_OK)
        return st;
    int sms = 0;
    st = norm_device(&sms);
    if (st != EP_OK)
        return st;
    *bytes = align256(size_t(moe::norm_back_blocks(num_tokens, sms)) * cfg->hidden * 4);
    return set_error(EP_OK, "");
}

ep_status ep_norm_backward(const ep_norm_config *cfg, const void *dy, long long dy_stride, const void *h,
                           long long h_stride, const void *dh, long long dh_stride, int num_tokens, void *dx,
                           long long dx_stride, float *dweight, void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("ep_norm_backward");
    ep_status st = check_norm(cfg, num_tokens);
    if (st != EP_OK)
        return st;
    moe::NormBackArgs a = {};
    st = norm_device(&a.sms);
    if (st != EP_OK)
        return st;
    const int H = cfg->hidden, size = size_of(cfg->dtype);
    if (!aligned(dweight, 4))
        MOE_FAIL("dweight is not 4-byte aligned");
    if ((!dx && !dweight) || (num_tokens == 0 && !dweight))
        return set_error(EP_OK, "");
    const bool any = num_tokens > 0;  // dweight is written without rows too
    const long long strides[3] = {dy_stride, h_stride, dh_stride};
    const Span in[4] = {rows_of("dy", dy, num_tokens, H, dy_stride, size), rows_of("h", h, num_tokens, H, h_stride, size),
                        rows_of("dh", dh, num_tokens, H, dh_stride, size), weight_span(*cfg)};
    const Span out[2] = {rows_of("dx", dx, num_tokens, H, dx_stride, size), whole("dweight", dweight, size_t(H) * 4)};
    for (int i = 0; i < 3 && st == EP_OK && any; ++i)
        if (i < 2 || dh)
            st = check_rows(in[i].name, in[i].p, strides[i], H, 16, 8);
    if (st == EP_OK && dx && any)
        st = check_rows("dx", dx, dx_stride, H, 16, 8);
    for (int o = 0; o < 2 && st == EP_OK; ++o)
        for (int i = 0; i < 4 && st == EP_OK; ++i)
            st = check_overlap(out[o], in[i], o == 0 && i < 3);
    if (st == EP_OK)
        st = check_overlap(out[0], out[1], false);
    const size_t need = dweight ? align256(size_t(moe::norm_back_blocks(num_tokens, a.sms)) * H * 4) : 0;
    if (st == EP_OK)
        st = check_workspace(workspace, workspace_bytes, need);
    if (st != EP_OK)
        return st;
    a.dy = dy;
    a.h = h;
    a.dh = dh;
    a.weight = cfg->weight;
    a.dy_stride = dy_stride;
    a.h_stride = h_stride;
    a.dh_stride = dh_stride;
    a.dx_stride = dx_stride;
    a.dx = dx;
    a.dweight = dweight;
    a.parts = dweight ? static_cast<float *>(workspace) : nullptr;
    a.T = num_tokens;
    a.H = H;
    a.dtype = cfg->dtype;
    a.weight_fp32 = cfg->weight_dtype == EP_DTYPE_FP32;
    a.eps = cfg->eps;
    unsigned long long *rec = epk::check_record();
    a.chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return finish(moe::launch_norm_back(a, s), "ep_norm_backward", rec, s);
}

}  // extern "C"

// ---- feed-forward ------------------------------------------------------------------------

enum Kind { kJoin = 0, kDown, kSplit, kGradients, kPlans = kGradients + 8 };  // kGradients + which are asked for

struct ep_ffn {
    ep_ffn_config cfg;
    int device, sms;
    Flags flags;
    int *parts;  // device: which parts of shared tiles are written, 0 between launches
    struct {
        int T;
        moe::FfnLaunch l;
    } plan[kPlans];  // of the last call of each kind
};

namespace {

ep_status check_ffn(const ep_ffn_config *c)
{
    if (!c)
        MOE_FAIL("config is NULL");
    if (c->hidden < 8 || c->hidden > EP_MOE_MAX_DIM || c->hidden % 8)
        MOE_FAIL("hidden=%d must be a multiple of 8 in [8, %d]", c->hidden, EP_MOE_MAX_DIM);
    if (c->intermediate < 8 || c->intermediate > EP_MOE_MAX_DIM || c->intermediate % 8)
        MOE_FAIL("intermediate=%d must be a multiple of 8 in [8, %d]", c->intermediate, EP_MOE_MAX_DIM);
    if (!c->gate_up || !aligned(c->gate_up, 16))
        MOE_FAIL("gate_up is NULL or not 16-byte aligned");
    if (!c->down || !aligned(c->down, 16))
        MOE_FAIL("down is NULL or not 16-byte aligned");
    return EP_OK;
}

ep_status check_ffn_tokens(const ep_ffn *h, int num_tokens)
{
    if (!h)
        MOE_FAIL("handle is NULL");
    if (num_tokens < 0 || num_tokens > EP_FFN_MAX_TOKENS)
        MOE_FAIL("num_tokens=%d outside [0, %d]", num_tokens, EP_FFN_MAX_TOKENS);
    return EP_OK;
}

// A matrix operand as it lies in memory: `rows` rows of `cols` bf16, `stride` apart.
struct Matrix {
    const char *name;
    const void *p;
    long long rows, cols, stride;
};

// One launch: up to three products D[M, N] = A B^T, each operand either [M or N, K], or [K, M or N] (mn).
struct Launch {
    moe::FfnLaunch l = {};
    int kind;
    Matrix a[3], b[3];

    Launch(int epilogue, int kind_) : kind(kind_) { l.epilogue = epilogue; }
    moe::FfnArgs &add(int M, int N, int K, bool a_mn, bool b_mn, const Matrix &ma, const Matrix &mb)
    {
        const int g = l.q.count++;
        a[g] = ma;
        b[g] = mb;
        moe::FfnArgs &p = l.q.p[g];
        p.M = M;
        p.N = N;
        p.K = K;
        p.a_mn = a_mn;
        p.b_mn = b_mn;
        return p;
    }
};

// The products of a call; pointers that a plan does not need may be missing.
Launch join_of(const ep_ffn_config &c, int T, const void *x, long long x_stride, void *h, float *saved)
{
    const int H = c.hidden, I = c.intermediate;
    Launch l(moe::kFfnJoin, kJoin);
    moe::FfnArgs &p = l.add(I, T, H, false, false, {"gate_up", c.gate_up, 2 * I, H, H}, {"x", x, T, H, x_stride});
    p.out = h;
    p.out_stride = I;
    p.saved = saved;
    return l;
}

Launch down_of(const ep_ffn_config &c, int T, const void *h, void *out, long long out_stride)
{
    const int H = c.hidden, I = c.intermediate;
    Launch l(moe::kFfnStore, kDown);
    moe::FfnArgs &p = l.add(H, T, I, false, false, {"down", c.down, H, I, I}, {"h", h, T, I, I});
    p.early = 1;
    p.out = out;
    p.out_stride = out_stride;
    return l;
}

Launch split_of(const ep_ffn_config &c, int T, const ep_ffn_grads &g, void *h, __nv_bfloat16 *dgu)
{
    const int H = c.hidden, I = c.intermediate;
    Launch l(moe::kFfnSplit, kSplit);
    moe::FfnArgs &p = l.add(I, T, H, true, false, {"down", c.down, H, I, I}, {"dy", g.dy, T, H, g.dy_stride});
    p.out = h;
    p.out_stride = I;
    p.saved = const_cast<float *>(g.saved);
    p.dgu = dgu;
    return l;
}

// dx and the weights' gradients, as far as they are asked for.
Launch gradients_of(const ep_ffn_config &c, int T, const ep_ffn_grads &g, const void *h, const __nv_bfloat16 *dgu)
{
    const int H = c.hidden, I = c.intermediate;
    const Matrix rows = {"gradients of gate and up", dgu, T, 2 * I, 2 * I}, x = {"x", g.x, T, H, g.x_stride};
    Launch l(moe::kFfnStore, kGradients + (g.dx ? 1 : 0) + (g.dgate_up ? 2 : 0) + (g.ddown ? 4 : 0));
    // Only the last rounds are cut over all pairs. A tile of dx goes through 2 I, one of the weights' gradients through T: where
    // that is so much more that few tiles of dx would fill a pair's share, dx comes last (all gradients of 700 rows, 1024 x
    // 9000: 90 us, first 120; 8192 rows, 2048 x 1000: 150, first 141).
    const bool dx_last = 2 * I > 16 * T;
    for (int turn = 0; turn < 2; ++turn) {
        if (g.dx && turn == dx_last) {
            moe::FfnArgs &p = l.add(H, T, 2 * I, true, false, {"gate_up", c.gate_up, 2 * I, H, H}, rows);
            p.early = 1;
            p.out = g.dx;
            p.out_stride = g.dx_stride;
        }
        if (g.dgate_up && turn != dx_last) {
            moe::FfnArgs &p = l.add(H, 2 * I, T, true, true, x, rows);
            p.early = 1;
            p.out = g.dgate_up;
            p.out_stride = H;
        }
        if (g.ddown && turn != dx_last) {
            moe::FfnArgs &p = l.add(I, H, T, true, true, {"h", h, T, I, I}, {"dy", g.dy, T, H, g.dy_stride});
            p.out = g.ddown;
            p.out_stride = I;
        }
    }
    for (int i = 0; i < l.l.q.count; ++i)
        if (l.l.q.p[i].b_mn) {
            l.l.q.p[i].fp32 = g.grad_dtype == EP_DTYPE_FP32;
            l.l.q.p[i].accumulate = g.accumulate != 0;
        }
    return l;
}

// The plan follows from the sizes alone: the last one of each kind is kept.
void plan(ep_ffn *h, int num_tokens, Launch &w)
{
    auto &kept = h->plan[w.kind];
    if (kept.T != num_tokens) {
        moe::ffn_plan(&w.l, h->sms);
        kept.l = w.l;
        kept.T = num_tokens;
        return;
    }
    moe::FfnGroup &q = w.l.q;
    const moe::FfnGroup &k = kept.l.q;
    for (int g = 0; g < q.count; ++g) {
        moe::FfnArgs &a = q.p[g];
        const moe::FfnArgs &b = k.p[g];
        a.tile_n = b.tile_n;
        a.m_tiles = b.m_tiles;
        a.n_tiles = b.n_tiles;
        a.chunks = b.chunks;
        a.box_b = b.box_b;
        a.whole = b.whole;
        a.band_inverse = b.band_inverse;
        a.rest_inverse = b.rest_inverse;
    }
    q.pairs = k.pairs;
    q.stages = k.stages;
    q.bytes = k.bytes;
    q.whole = k.whole;
    q.cut = k.cut;
    memcpy(q.begin, k.begin, sizeof(q.begin));
    w.l.split = kept.l.split;
    w.l.parts = kept.l.parts;
}

// An output that overlaps the weights.
ep_status check_weights(const Span &out, const ep_ffn_config &c)
{
    const size_t bytes = size_t(c.hidden) * c.intermediate * 2;
    const ep_status st = check_overlap(out, whole("gate_up", c.gate_up, 2 * bytes), false);
    return st == EP_OK ? check_overlap(out, whole("down", c.down, bytes), false) : st;
}

// The intermediate rows, for the backward pass the gradients of gate and up too, then the parts of shared tiles.
struct FfnLayout {
    size_t off_dgu, off_parts;
    FfnLayout(const ep_ffn_config &c, bool backward, int num_tokens)
    {
        const size_t row = size_t(c.intermediate) * 2;
        off_dgu = align256(num_tokens * row);
        off_parts = off_dgu + (backward ? align256(num_tokens * 2 * row) : 0);
    }
};

// Bytes of shared tiles' parts: only products that make gradients have such tiles, and only where their plan cuts rounds.
size_t parts_of(ep_ffn *h, int num_tokens, const ep_ffn_grads &g)
{
    Launch w = gradients_of(h->cfg, num_tokens, g, nullptr, nullptr);
    if (num_tokens == 0 || w.l.q.count == 0)
        return 0;
    plan(h, num_tokens, w);
    return align256(w.l.parts);
}

ep_status launch(ep_ffn *h, int num_tokens, Launch &w, void *parts, epk::CheckCtx chk, cudaStream_t s)
{
    moe::FfnGroup &q = w.l.q;
    plan(h, num_tokens, w);
    q.parts = static_cast<float *>(parts);
    q.flags = h->parts;
    q.err = h->flags.err;
    const int features = w.l.epilogue == moe::kFfnJoin ? 64 : 128;
    for (int g = 0; g < q.count; ++g) {
        moe::FfnArgs &a = q.p[g];
        const Matrix &ma = w.a[g], &mb = w.b[g];
        ep_status st = encode_map(&a.ma, ma.name, 0, ma.p, ma.cols, ma.rows, 0, ma.stride, 0, moe::kChunk, 64);
        if (st == EP_OK)
            st = encode_map(&a.mb, mb.name, 0, mb.p, mb.cols, mb.rows, 0, mb.stride, 0, moe::kChunk, a.b_mn ? 64 : a.box_b);
        const int size = a.fp32 ? 4 : 2;
        a.aligned = aligned(a.out, 8) && a.out_stride % 4 == 0;
        // The checked build tests the stores of y and dx one by one; all others are bounded by their maps.
        a.boxes = aligned(a.out, 16) && a.out_stride * size % 16 == 0 && !(EP_CHECKED && w.l.epilogue == moe::kFfnStore && !a.b_mn);
        if (st == EP_OK && !w.l.split && a.boxes)
            st = encode_result(&a.mo, "result", a.fp32 != 0, a.out, a.M, a.N, 0, a.out_stride, 0, features, 16);
        if (st == EP_OK && !w.l.split && a.dgu)
            st = encode_result(&a.md, "gradients of gate and up", false, a.dgu, a.M, a.N, 2, 2LL * a.M, a.M, features, 16);
        if (st != EP_OK)
            return st;
        a.chk = chk;
    }
    const cudaError_t ce = moe::launch_ffn(w.l, s);
    return ce == cudaSuccess ? EP_OK : cuda_error(ce, "launch");
}

}  // namespace

extern "C" {

ep_status ep_ffn_create(const ep_ffn_config *cfg, ep_ffn **out)
{
    if (!out)
        MOE_FAIL("out is NULL");
    *out = nullptr;
    ep_status st = check_ffn(cfg);
    if (st != EP_OK)
        return st;
    int dev = 0, sms = 0;
    st = current_device(&dev, &sms);
    if (st != EP_OK)
        return st;
    ep_ffn *h = new (std::nothrow) ep_ffn();
    if (!h)
        return set_error(EP_ERR_OOM, "host allocation of the handle failed");
    h->cfg = *cfg;
    h->device = dev;
    h->sms = sms;
    st = h->flags.make();
    if (st == EP_OK) {
        const size_t bytes = (2 * moe::kFfnMaxPairs + 1) * sizeof(int);
        cudaError_t ce = moe::ffn_setup();
        if (ce == cudaSuccess)
            ce = cudaMalloc(reinterpret_cast<void **>(&h->parts), bytes);
        if (ce == cudaSuccess)
            ce = cudaMemset(h->parts, 0, bytes);
        if (ce == cudaSuccess)
            ce = cudaStreamSynchronize(nullptr);
        if (ce != cudaSuccess)
            st = cuda_error(ce, "the handle's kernels and flags");
    }
    if (st != EP_OK) {
        if (h->parts)
            cudaFree(h->parts);
        h->flags.free();
        delete h;
        return st;
    }
    *out = h;
    return set_error(EP_OK, "");
}

ep_status ep_ffn_workspace_size(ep_ffn *h, ep_ffn_call call, int num_tokens, size_t *bytes)
{
    const ep_status st = check_ffn_tokens(h, num_tokens);
    if (st != EP_OK)
        return st;
    if (!bytes)
        MOE_FAIL("bytes is NULL");
    if (call != EP_FFN_RUN && call != EP_FFN_FORWARD && call != EP_FFN_BACKWARD)
        MOE_FAIL("unknown call %d", static_cast<int>(call));
    *bytes = FfnLayout(h->cfg, call == EP_FFN_BACKWARD, num_tokens).off_parts;
    size_t parts = 0;
    for (int asked = 1; asked < 8 && call == EP_FFN_BACKWARD; ++asked) {  // whichever gradients a call wants
        ep_ffn_grads g = {};
        g.dx = asked & 1 ? h : nullptr;
        g.dgate_up = asked & 2 ? h : nullptr;
        g.ddown = asked & 4 ? h : nullptr;
        const size_t here = parts_of(h, num_tokens, g);
        parts = here > parts ? here : parts;
    }
    *bytes += parts;
    return set_error(EP_OK, "");
}

ep_status ep_ffn_run(ep_ffn *h, const void *x, long long x_stride, int num_tokens, float *saved, void *out,
                     long long out_stride, void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("ep_ffn_run");
    ep_status st = check_ffn_tokens(h, num_tokens);
    if (st == EP_OK)
        st = same_device(h->device);
    if (st != EP_OK)
        return st;
    if (num_tokens == 0)
        return set_error(EP_OK, "");
    const int T = num_tokens, H = h->cfg.hidden, I = h->cfg.intermediate;
    st = check_rows("x", x, x_stride, H, 16, 8);
    if (st == EP_OK)
        st = check_rows("out", out, out_stride, H, 2, 1);
    if (st != EP_OK)
        return st;
    if (!aligned(saved, 16))
        MOE_FAIL("saved is not 16-byte aligned");
    const Span in = rows_of("x", x, T, H, x_stride, 2), y = rows_of("out", out, T, H, out_stride, 2),
               keep = whole("saved", saved, size_t(T) * 2 * I * 4);
    st = check_overlap(y, in, false);
    if (st == EP_OK)
        st = check_overlap(keep, in, false);
    if (st == EP_OK)
        st = check_overlap(keep, y, false);
    if (st == EP_OK)
        st = check_weights(y, h->cfg);
    if (st == EP_OK)
        st = check_weights(keep, h->cfg);
    if (st == EP_OK)
        st = check_workspace(workspace, workspace_bytes, FfnLayout(h->cfg, false, T).off_parts);
    if (st == EP_OK)
        st = h->flags.take();
    if (st != EP_OK)
        return st;
    unsigned long long *rec = epk::check_record();
    const epk::CheckCtx chk = epk::check_ctx(rec);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Launch first = join_of(h->cfg, T, x, x_stride, workspace, saved), second = down_of(h->cfg, T, workspace, out, out_stride);
    st = launch(h, T, first, nullptr, chk, s);
    if (st == EP_OK)
        st = launch(h, T, second, nullptr, chk, s);
    return st == EP_OK ? finish(cudaSuccess, "ep_ffn_run", rec, s) : st;
}

ep_status ep_ffn_backward(ep_ffn *h, const ep_ffn_grads *grads, int num_tokens, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    Range range("ep_ffn_backward");
    ep_status st = check_ffn_tokens(h, num_tokens);
    if (st == EP_OK)
        st = same_device(h->device);
    if (st != EP_OK)
        return st;
    if (!grads)
        MOE_FAIL("grads is NULL");
    const ep_ffn_grads &g = *grads;
    const int T = num_tokens, H = h->cfg.hidden, I = h->cfg.intermediate;
    if (g.grad_dtype != EP_DTYPE_BF16 && g.grad_dtype != EP_DTYPE_FP32)
        MOE_FAIL("grad_dtype %d: use bf16 or fp32", static_cast<int>(g.grad_dtype));
    if (g.accumulate && g.grad_dtype != EP_DTYPE_FP32)
        MOE_FAIL("accumulate needs fp32 gradients");
    if (!aligned(g.dgate_up, 16) || !aligned(g.ddown, 16))
        MOE_FAIL("dgate_up or ddown is not 16-byte aligned");
    const int size = size_of(g.grad_dtype);
    const size_t weight = size_t(H) * I * size;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Span out[3] = {rows_of("dx", g.dx, T, H, g.dx_stride, 2), whole("dgate_up", g.dgate_up, 2 * weight),
                         whole("ddown", g.ddown, weight)};
    const auto check_results = [&] {
        ep_status bad = EP_OK;
        for (int o = 0; o < 3 && bad == EP_OK; ++o) {
            for (int i = 0; i < o && bad == EP_OK; ++i)
                bad = check_overlap(out[o], out[i], false);
            if (bad == EP_OK)
                bad = check_weights(out[o], h->cfg);
        }
        return bad;
    };
    if (T == 0) {
        st = check_results();
        if (st != EP_OK)
            return st;
        cudaError_t ce = cudaSuccess;
        if (g.dgate_up && !g.accumulate)
            ce = moe::launch_ffn_zero(g.dgate_up, 2 * weight, s);
        if (ce == cudaSuccess && g.ddown && !g.accumulate)
            ce = moe::launch_ffn_zero(g.ddown, weight, s);
        return ce == cudaSuccess ? set_error(EP_OK, "") : cuda_error(ce, "ep_ffn_backward");
    }
    st = check_rows("dy", g.dy, g.dy_stride, H, 16, 8);
    if (st == EP_OK)
        st = check_rows("x", g.x, g.x_stride, H, 16, 8);
    if (st == EP_OK && g.dx)
        st = check_rows("dx", g.dx, g.dx_stride, H, 2, 1);
    if (st != EP_OK)
        return st;
    if (!g.saved || !aligned(g.saved, 16))
        MOE_FAIL("saved is NULL or not 16-byte aligned");
    const Span in[3] = {rows_of("dy", g.dy, T, H, g.dy_stride, 2), rows_of("x", g.x, T, H, g.x_stride, 2),
                        whole("saved", g.saved, size_t(T) * 2 * I * 4)};
    for (int o = 0; o < 3 && st == EP_OK; ++o)
        for (int i = 0; i < 3 && st == EP_OK; ++i)
            st = check_overlap(out[o], in[i], false);
    if (st == EP_OK)
        st = check_results();
    const FfnLayout l(h->cfg, true, T);
    if (st == EP_OK)
        st = check_workspace(workspace, workspace_bytes, l.off_parts + parts_of(h, T, g));
    if (st == EP_OK)
        st = h->flags.take();
    if (st != EP_OK)
        return st;
    if (!g.dx && !g.dgate_up && !g.ddown)
        return set_error(EP_OK, "");
    unsigned long long *rec = epk::check_record();
    const epk::CheckCtx chk = epk::check_ctx(rec);
    __nv_bfloat16 *const dgu = reinterpret_cast<__nv_bfloat16 *>(static_cast<uint8_t *>(workspace) + l.off_dgu);
    void *const parts = static_cast<uint8_t *>(workspace) + l.off_parts;
    Launch first = split_of(h->cfg, T, g, workspace, dgu), rest = gradients_of(h->cfg, T, g, workspace, dgu);
    st = launch(h, T, first, parts, chk, s);
    if (st == EP_OK)
        st = launch(h, T, rest, parts, chk, s);
    return st == EP_OK ? finish(cudaSuccess, "ep_ffn_backward", rec, s) : st;
}

ep_status ep_ffn_destroy(ep_ffn *h)
{
    if (h) {
        wait_for_device(h->device);
        cudaFree(h->parts);
        h->flags.free();
        delete h;
    }
    return set_error(EP_OK, "");
}

}  // extern "C"
