// C ABI of the weight-table operators (include/spmv.h): argument checks, the
// 4-bit matrix's handle and its teardown.
#include <memory>
#include <new>

#include "tables.h"

namespace spmv {
namespace {

struct QuantDeleter {
    void operator()(spmv_quant *q) const {
        if (!q) return;
        (void)hipFree(q->codes);
        (void)hipFree(q->scales);
        (void)hipFree(q->zeros);
        delete q;
    }
};
using QuantPtr = std::unique_ptr<spmv_quant, QuantDeleter>;

// A zeroed device array: the padding is part of the format.
template <typename T>
spmv_status zeroed(spmv_quant *q, T **p, int64_t bytes, hipStream_t s) {
    *p = nullptr;
    void *v = nullptr;
    const size_t size = static_cast<size_t>(bytes < 16 ? 16 : bytes);
    const hipError_t e = hipMalloc(&v, size);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return from_hip(e);
    }
    *p = static_cast<T *>(v);
    q->device_bytes += static_cast<int64_t>(size);
    SPMV_HIP(hipMemsetAsync(v, 0, size, s));
    return SPMV_OK;
}

bool valid_group(int32_t g) { return g == 32 || g == 64 || (g > 0 && g % 128 == 0); }

// Sizes and zeroed arrays of an R x C matrix.
spmv_status new_quant(QuantPtr &q, int32_t R, int32_t C, int32_t group, bool zeros,
                      int32_t scale_dtype, hipStream_t s) {
    // columns stay in 32 bits, and a launch's threads too
    if (C > INT32_MAX - 2 * kQuantCols || R > (1 << 28)) return SPMV_ERR_TOO_LARGE;
    q.reset(new (std::nothrow) spmv_quant);
    if (!q) return SPMV_ERR_OOM;
    SPMV_HIP(hipGetDevice(&q->device));
    q->R = R;
    q->C = C;
    q->group = group;
    q->groups = static_cast<int32_t>((static_cast<int64_t>(C) + group - 1) / group);
    q->tiles = static_cast<int32_t>((static_cast<int64_t>(R) + kQuantRows - 1) / kQuantRows);
    q->blocks = static_cast<int32_t>((static_cast<int64_t>(C) + kQuantCols - 1) / kQuantCols);
    q->set = std::max(1, kQuantCols / group);
    const int64_t reach = static_cast<int64_t>(q->blocks) * kQuantCols;
    q->sets = static_cast<int32_t>((reach + group * static_cast<int64_t>(q->set) - 1) /
                                   (group * static_cast<int64_t>(q->set)));
    q->scale_dtype = scale_dtype;
    const int64_t groups = static_cast<int64_t>(q->tiles) * q->sets * q->set * kQuantRows;
    SPMV_TRY(zeroed(q.get(), &q->codes,
                    static_cast<int64_t>(q->tiles) * q->blocks * kQuantBlockWords * 4, s));
    SPMV_TRY(zeroed(q.get(), &q->scales,
                    groups * static_cast<int64_t>(dtype_bytes(scale_dtype)), s));
    if (zeros) SPMV_TRY(zeroed(q.get(), &q->zeros, groups, s));
    return SPMV_OK;
}

// Runs fill(flag) and returns the handle if it raised no flag.
template <typename F>
spmv_status build(spmv_quant **out, int32_t R, int32_t C, int32_t group, bool zeros,
                  int32_t scale_dtype, hipStream_t s, F fill) {
    Scratch scratch(s);
    int *flag = nullptr;
    SPMV_TRY(scratch.alloc(&flag, 1));
    SPMV_HIP(hipMemsetAsync(flag, 0, sizeof(int), s));
    QuantPtr q;
    spmv_status st = new_quant(q, R, C, group, zeros, scale_dtype, s);
    if (st == SPMV_OK) st = fill(q.get(), flag);
    int bad = 0;
    if (st == SPMV_OK) {
        const hipError_t e = hipMemcpyAsync(&bad, flag, sizeof(int), hipMemcpyDeviceToHost, s);
        if (e != hipSuccess) st = from_hip(e);
    }
    // the arrays are written (or no longer touched) before anyone frees them
    const hipError_t e = hipStreamSynchronize(s);
    if (st == SPMV_OK && e != hipSuccess) st = from_hip(e);
    if (st == SPMV_OK && bad) st = SPMV_ERR_BAD_VALUE;
    if (st == SPMV_OK) *out = q.release();
    return st;
}

spmv_status check_device(const spmv_quant *q) {
    int dev = -1;
    SPMV_HIP(hipGetDevice(&dev));
    return dev == q->device ? SPMV_OK : SPMV_ERR_DEVICE;
}

size_t array_bytes(const spmv_quant *q, spmv_quant_array which) {
    const size_t items = static_cast<size_t>(q->R) * static_cast<size_t>(q->groups);
    switch (which) {
    case SPMV_Q_CODES:
        return static_cast<size_t>(q->R) *
               static_cast<size_t>((static_cast<int64_t>(q->C) + 1) / 2);
    case SPMV_Q_SCALES: return items * dtype_bytes(q->scale_dtype);
    case SPMV_Q_ZEROS: return q->zeros ? items : 0;
    default: return 0;
    }
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" {

spmv_status spmv_quant_build(spmv_quant **out, int32_t R, int32_t C, int32_t group,
                             int32_t zero_points, spmv_dtype scale_dtype, const void *weights,
                             int64_t ld, spmv_dtype weight_dtype, void *stream) {
    if (!out) return SPMV_ERR_INVALID_ARG;
    *out = nullptr;
    if (R < 0 || C < 0 || !valid_group(group) || !float_dtype(scale_dtype) ||
        !float_dtype(weight_dtype) || (R > 0 && C > 0 && !weights) || (R > 1 && ld < C))
        return SPMV_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return build(out, R, C, group, zero_points != 0, scale_dtype, s,
                 [&](spmv_quant *q, int *flag) {
                     return quant_fill_dense(q, weights, ld, weight_dtype, flag, s);
                 });
}

spmv_status spmv_quant_build_packed(spmv_quant **out, int32_t R, int32_t C, int32_t group,
                                    const uint8_t *codes, const void *scales,
                                    spmv_dtype scale_dtype, const uint8_t *zeros,
                                    int32_t validate, void *stream) {
    if (!out) return SPMV_ERR_INVALID_ARG;
    *out = nullptr;
    if (R < 0 || C < 0 || !valid_group(group) || !float_dtype(scale_dtype) ||
        (R > 0 && C > 0 && (!codes || !scales)))
        return SPMV_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return build(out, R, C, group, zeros != nullptr, scale_dtype, s,
                 [&](spmv_quant *q, int *flag) {
                     return quant_fill_packed(q, codes, scales, zeros, validate != 0, flag, s);
                 });
}

spmv_status spmv_quant_run_workspace(const spmv_quant *q, int32_t n, spmv_dtype x_dtype,
                                     size_t *bytes) {
    if (!q || !bytes || n < 0 || !float_dtype(x_dtype)) return SPMV_ERR_INVALID_ARG;
    if (n > kMostVectors) return SPMV_ERR_TOO_LARGE;
    *bytes = n == 0 || q->R == 0 ? 0 : quant_run_bytes(q, n, x_dtype);
    return SPMV_OK;
}

spmv_status spmv_quant_run(const spmv_quant *q, int32_t n, const void *x, int64_t x_ld,
                           spmv_dtype x_dtype, void *y, int64_t y_ld, spmv_dtype y_dtype,
                           int32_t accumulate, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (!q || n < 0 || !float_dtype(x_dtype) || (y_dtype != x_dtype && y_dtype != SPMV_FP32))
        return SPMV_ERR_INVALID_ARG;
    if (n > kMostVectors) return SPMV_ERR_TOO_LARGE;
    if (n == 0 || q->R == 0 || (q->C == 0 && accumulate)) return SPMV_OK;
    if ((q->C > 0 && !x) || !y || (n > 1 && (x_ld < q->C || y_ld < q->R)))
        return SPMV_ERR_INVALID_ARG;
    const size_t need = quant_run_bytes(q, n, x_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need ||
                     reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
        return SPMV_ERR_INVALID_ARG;
    SPMV_TRY(check_device(q));
    return quant_run(q, n, x, x_ld, x_dtype, y, y_ld, y_dtype, accumulate != 0, workspace,
                     static_cast<hipStream_t>(stream));
}

spmv_status spmv_quant_lookup(const spmv_quant *q, int64_t n, const void *ids,
                              spmv_dtype id_dtype, float scale, void *out, int64_t ld,
                              spmv_dtype dtype, void *stream) {
    if (!q || n < 0 || !id_dtype_ok(id_dtype) || !float_dtype(dtype)) return SPMV_ERR_INVALID_ARG;
    if (n == 0 || q->C == 0) return SPMV_OK;
    if (!ids || !out || (n > 1 && ld < q->C)) return SPMV_ERR_INVALID_ARG;
    SPMV_TRY(check_device(q));
    return quant_lookup(q, n, ids, id_dtype, scale, out, ld, dtype,
                        static_cast<hipStream_t>(stream));
}

spmv_status spmv_quant_get_info(const spmv_quant *q, spmv_quant_info *info) {
    if (!q || !info) return SPMV_ERR_INVALID_ARG;
    info->num_rows = q->R;
    info->num_cols = q->C;
    info->group_size = q->group;
    info->num_groups = q->groups;
    info->scale_dtype = q->scale_dtype;
    info->zero_points = q->zeros != nullptr;
    info->device_bytes = q->device_bytes;
    return SPMV_OK;
}

spmv_status spmv_quant_array_bytes(const spmv_quant *q, spmv_quant_array which, size_t *bytes) {
    if (!q || !bytes || which < SPMV_Q_CODES || which > SPMV_Q_ZEROS) return SPMV_ERR_INVALID_ARG;
    *bytes = array_bytes(q, which);
    return SPMV_OK;
}

spmv_status spmv_quant_export(const spmv_quant *q, spmv_quant_array which, void *dst,
                              size_t bytes) {
    if (!q || which < SPMV_Q_CODES || which > SPMV_Q_ZEROS || bytes != array_bytes(q, which) ||
        (bytes > 0 && !dst))
        return SPMV_ERR_INVALID_ARG;
    if (bytes == 0) return SPMV_OK;
    SPMV_TRY(check_device(q));
    Scratch scratch(nullptr);
    char *tmp = nullptr;
    SPMV_TRY(scratch.alloc(&tmp, bytes));
    SPMV_TRY(quant_unpack(q, which, tmp, nullptr));
    SPMV_HIP(hipMemcpy(dst, tmp, bytes, hipMemcpyDeviceToHost));
    return SPMV_OK;
}

spmv_status spmv_quant_destroy(spmv_quant *q) {
    if (!q) return SPMV_OK;
    int prev = -1;
    (void)hipGetDevice(&prev);
    if (prev != q->device) (void)hipSetDevice(q->device);
    (void)hipDeviceSynchronize();
    QuantDeleter()(q);
    if (prev >= 0 && prev != q->device) (void)hipSetDevice(prev);
    return SPMV_OK;
}

spmv_status spmv_lookup(int32_t V, int32_t D, const void *table, int64_t table_ld,
                        spmv_dtype table_dtype, int64_t n, const void *ids, spmv_dtype id_dtype,
                        float scale, void *out, int64_t out_ld, spmv_dtype out_dtype,
                        void *stream) {
    if (V < 0 || D < 0 || n < 0 || !float_dtype(table_dtype) || !id_dtype_ok(id_dtype) ||
        !float_dtype(out_dtype))
        return SPMV_ERR_INVALID_ARG;
    if (n == 0 || D == 0) return SPMV_OK;
    if ((V > 0 && !table) || !ids || !out || (V > 1 && table_ld < D) || (n > 1 && out_ld < D))
        return SPMV_ERR_INVALID_ARG;
    return lookup_rows(V, D, table, table_ld, table_dtype, n, ids, id_dtype, scale, out, out_ld,
                       out_dtype, static_cast<hipStream_t>(stream));
}

spmv_status spmv_lookup_grad_workspace(int32_t V, int32_t D, int64_t n, size_t *bytes) {
    if (!bytes || V < 0 || D < 0 || n < 0) return SPMV_ERR_INVALID_ARG;
    if (n > INT32_MAX) return SPMV_ERR_TOO_LARGE;
    *bytes = V == 0 || D == 0 ? 0 : lookup_grad_bytes(V, D, n);
    return SPMV_OK;
}

spmv_status spmv_lookup_grad(int32_t V, int32_t D, int64_t n, const void *ids,
                             spmv_dtype id_dtype, const void *grad, int64_t grad_ld,
                             spmv_dtype grad_dtype, float scale, int32_t accumulate,
                             void *dtable, int64_t ld, spmv_dtype table_dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (V < 0 || D < 0 || n < 0 || !id_dtype_ok(id_dtype) || !float_dtype(grad_dtype) ||
        !float_dtype(table_dtype))
        return SPMV_ERR_INVALID_ARG;
    if (n > INT32_MAX) return SPMV_ERR_TOO_LARGE;
    if (V == 0 || D == 0) return SPMV_OK;
    if (!dtable || (V > 1 && ld < D) || (n > 0 && (!ids || !grad)) || (n > 1 && grad_ld < D))
        return SPMV_ERR_INVALID_ARG;
    if (workspace_bytes < lookup_grad_bytes(V, D, n) ||
        (n > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)))
        return SPMV_ERR_INVALID_ARG;
    return lookup_grad(V, D, n, ids, id_dtype, grad, grad_ld, grad_dtype, scale, accumulate != 0,
                       dtable, ld, table_dtype, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
