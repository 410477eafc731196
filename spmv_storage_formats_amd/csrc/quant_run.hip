// y <- W x (+ y) with a 4-bit matrix (layout at struct spmv_quant, tables.h).
#include "tables.h"

namespace spmv {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kVecs = 4;

// A wave per row, a lane per octet, kVecs vectors at a time: fp32 throughout.
template <typename X, typename S, typename Y>
__global__ __launch_bounds__(kThreads) void k_quant_rows(
    int32_t R, int32_t C, int32_t group, int32_t groups_pad, int32_t blocks,
    const uint32_t *__restrict__ codes, const S *__restrict__ scales,
    const uint8_t *__restrict__ zeros, int32_t n, const X *__restrict__ x, int64_t x_ld,
    Y *__restrict__ y, int64_t y_ld, int accumulate, int32_t vec_groups) {
    const int lane = threadIdx.x % kWave;
    const int64_t row_groups = (static_cast<int64_t>(R) + kWaves - 1) / kWaves;
    for (int64_t i = blockIdx.x; i < row_groups * vec_groups; i += gridDim.x) {
        const int64_t r = (i % row_groups) * kWaves + threadIdx.x / kWave;
        if (r >= R) continue;
        const int32_t v0 = static_cast<int32_t>(i / row_groups) * kVecs;
        const int vecs = n - v0 < kVecs ? n - v0 : kVecs;
        const int octets = C / 8 + (C % 8 != 0);
        float sum[kVecs] = {};
        for (int o = lane; o < octets; o += kWave) {
            const int64_t block =
                (r / kQuantRows) * blocks + o / kQuantRowWords;
            const uint32_t w = codes[block * kQuantBlockWords + (r % kQuantRows) * kQuantRowWords +
                                     quant_word(o % kQuantRowWords)];
            const int64_t si =
                ((r / kQuantRows) * groups_pad + o * 8 / group) * kQuantRows +
                r % kQuantRows;
            const float s = static_cast<float>(scales[si]);
            const float z = zeros ? static_cast<float>(zeros[si]) : 8.f;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                if (v >= vecs) break;
                float xv[8];
                const X *p = x + (v0 + v) * x_ld + o * 8;
                if (o * 8 + 8 <= C)
                    load_octet(p, xv);
                else
                    load_octet_tail(p, C - o * 8, xv);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (o * 8 + e < C)
                        sum[v] = fmaf((static_cast<float>(quant_code(w, e)) - z) * s, xv[e], sum[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float t = group_sum<kWave>(sum[v]);
            if (lane == 0 && v < vecs) {
                Y *p = y + (v0 + v) * y_ld + r;
                if (accumulate) t += static_cast<float>(*p);
                *p = static_cast<Y>(t);
            }
        }
    }
}

}  // namespace

spmv_status quant_run(const spmv_quant *q, int32_t n, const void *x, int64_t x_ld,
                      int32_t x_dtype, void *y, int64_t y_ld, int32_t y_dtype, int accumulate,
                      hipStream_t s) {
    const int32_t vec_groups = n / kVecs + (n % kVecs != 0);
    const int64_t row_groups = (static_cast<int64_t>(q->R) + kWaves - 1) / kWaves;
    const unsigned grid = groups_for(row_groups * vec_groups, 1);
    with_float(x_dtype, [&](auto xt) {
        with_float(q->scale_dtype, [&](auto sc) {
            using X = decltype(xt);
            using S = decltype(sc);
            auto go = [&](auto yt) {
                using Y = decltype(yt);
                k_quant_rows<X, S, Y><<<grid, kThreads, 0, s>>>(
                    q->R, q->C, q->group, q->groups_pad, q->blocks, q->codes,
                    static_cast<const S *>(q->scales), q->zeros, n, static_cast<const X *>(x),
                    x_ld, static_cast<Y *>(y), y_ld, accumulate,
                    vec_groups);
            };
            if (y_dtype == SPMV_FP32)
                go(float{});
            else
                go(X{});
        });
    });
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

}  // namespace spmv
