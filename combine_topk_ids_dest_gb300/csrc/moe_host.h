// moe_host.h -- what the host sides of the MoE operators share: argument
// checks, errors, tensor maps and the flags of kernels whose waits are bounded.
#pragma once

#include <new>

#include <nvtx3/nvToolsExt.h>

#include "moe_internal.h"

namespace moe_host {

using epk::set_error;

#define MOE_FAIL(...) return set_error(EP_ERR_INVALID_ARG, __VA_ARGS__)

static inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

static inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

static inline ep_status cuda_error(cudaError_t ce, const char *what)
{
    cudaGetLastError();
    return set_error(ce == cudaErrorMemoryAllocation ? EP_ERR_OOM : EP_ERR_CUDA, "%s: %s", what,
                     cudaGetErrorString(ce));
}

// The current device, which must be able to run the library.
static inline ep_status current_device(int *dev, int *sms)
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

static inline ep_status same_device(int want)
{
    int dev = -1;
    const cudaError_t ce = cudaGetDevice(&dev);
    if (ce != cudaSuccess)
        return cuda_error(ce, "cudaGetDevice");
    if (dev != want)
        MOE_FAIL("handle lives on device %d but device %d is current", want, dev);
    return EP_OK;
}

// Waits for all work of a device: before a handle's memory is freed, or is its owner's again.
static inline void wait_for_device(int device)
{
    int now = device;
    cudaGetDevice(&now);
    if (now != device)
        cudaSetDevice(device);
    if (cudaDeviceSynchronize() != cudaSuccess)
        cudaGetLastError();  // the next call reports it
    if (now != device)
        cudaSetDevice(now);
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not link libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline EncodeTiled encode_tiled()
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
// box_cols x box_rows boxes (of 64 columns: in 128-byte swizzled rows), zeros outside.
static inline ep_status encode_map(CUtensorMap *m, const char *what, int fp16, const void *base, long long cols, long long rows,
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
                          box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled of %s: error %d", what, static_cast<int>(r));
    return EP_OK;
}

// A row-major result [.., rows, cols] of bf16 or fp32 that is written through boxes of box_cols x box_rows.
static inline ep_status encode_result(CUtensorMap *m, const char *what, bool fp32, void *base, long long cols, long long rows,
                               long long mats, long long row_stride, long long mat_stride, int box_cols, int box_rows)
{
    EncodeTiled fn = encode_tiled();
    if (!fn)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const int size = fp32 ? 4 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(mats > 0 ? mats : 1)};
    const cuuint64_t strides[2] = {cuuint64_t(row_stride) * size, cuuint64_t(mat_stride) * size};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1}, step[3] = {1, 1, 1};
    const CUresult r = fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mats > 0 ? 3 : 2,
                          base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled of %s: error %d", what, static_cast<int>(r));
    return EP_OK;
}

// A 16-bit tensor [rows, 32 n] as [n][rows][32]: boxes of all its inner 32
// columns, box_rows rows and box_steps steps of 32, zeros outside.
static inline ep_status encode_steps(CUtensorMap *m, const char *what, int fp16, const void *base, long long steps, long long rows,
                       long long row_stride, int box_rows, int box_steps)
{
    EncodeTiled fn = encode_tiled();
    if (!fn)
        return set_error(EP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[3] = {32, cuuint64_t(rows), cuuint64_t(steps)}, strides[2] = {cuuint64_t(row_stride) * 2, 64};
    const cuuint32_t box[3] = {32, cuuint32_t(box_rows), cuuint32_t(box_steps)}, step[3] = {1, 1, 1};
    const CUresult r = fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                          const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

static inline ep_status finish(cudaError_t ce, const char *what, unsigned long long *rec, cudaStream_t stream)
{
    if (ce != cudaSuccess)
        return cuda_error(ce, what);
    const ep_status st = epk::check_after(rec, stream, what);
    return st == EP_OK ? set_error(EP_OK, "") : st;
}

static inline int div_up(int a, int b) { return (a + b - 1) / b; }

static inline ep_status check_rows(const char *name, const void *p, long long stride, int cols, int align, int step)
{
    if (!p || !aligned(p, align))
        MOE_FAIL("%s is NULL or not %d-byte aligned", name, align);
    if (stride < cols || stride % step)
        MOE_FAIL("%s: stride %lld must be a multiple of %d and at least %d", name, stride, step, cols);
    return EP_OK;
}

}  // namespace moe_host
