// Internal declarations of the operators on a step's rows, one request's or
// sequence's each: low-rank adapters (adapt.hip, adapt_*.hip) and log
// probabilities of given tokens (logprobs.hip).  Nothing here is part of the
// public C ABI.
#pragma once

#include "tables.h"

namespace spmv {

// Vectors in registers, and in memory at the alignment of their elements: the
// compiler takes such an access apart if it is one of a struct or an array.
template <typename T, int E>
struct VecOf {
    typedef T type __attribute__((ext_vector_type(E)));
    typedef T loose __attribute__((ext_vector_type(E), aligned(sizeof(T)), may_alias));
};
template <typename T, int E>
using Vec = typename VecOf<T, E>::type;
template <typename T, int E>
using Loose = typename VecOf<T, E>::loose;
template <typename T, int E>
__device__ inline Vec<T, E> load_all(const T *p) {
    return *reinterpret_cast<const Loose<T, E> *>(p);
}
// E neighbours, the first `there` of them; the others are 0.
template <typename T, int E>
__device__ inline Vec<T, E> load_some(const T *p, int64_t there) {
    if (there >= E) return *reinterpret_cast<const Loose<T, E> *>(p);
    Vec<T, E> o = {};
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < there) o[i] = p[i];
    return o;
}

// Alternatives per row, at most: one per lane of the wave that sorts them.
constexpr int kMostTop = kWave;

// Columns of a row of logits, at most: kernels form the indexes of a whole step
// past the last column in 32 bits.
constexpr int32_t kMostVocab = INT32_MAX - (1 << 16);
// Rows of a step, at most: rows times parts or blocks of one stay in 64 bits.
constexpr int64_t kMostRows = INT32_MAX;

// logprobs.hip
size_t logprobs_bytes(int32_t V, int64_t n, int32_t top);  // of workspace
struct LogprobsArgs {
    int32_t V;
    int64_t n;
    const void *logits;
    int64_t ld;
    int32_t dtype;
    const void *ids;
    int32_t id_dtype;
    float scale;
    int32_t top;
    float *logprobs, *entropy, *stats;
    void *top_ids;
    float *top_logprobs;
    void *workspace;
};
spmv_status logprobs(const LogprobsArgs &a, hipStream_t s);

struct LogprobsGradArgs {
    int32_t V;
    int64_t n;
    const void *logits;
    int64_t ld;
    int32_t dtype;
    const void *ids;
    int32_t id_dtype;
    float scale;
    const float *stats, *grad_logprobs, *entropy, *grad_entropy;
    void *out;
    int64_t out_ld;
    int32_t out_dtype;
};
spmv_status logprobs_grad(const LogprobsGradArgs &a, hipStream_t s);

// adapt.hip
// Ranks, adapters (keys of the sort, counted in LDS), columns and rows, at most
// (blocks and tiles that one launch counts).
constexpr int32_t kMostRank = 256;
constexpr int32_t kMostAdapters = 2048;
constexpr int32_t kMostColumns = 1 << 21;
constexpr int32_t kMostAdaptRows = 1 << 24;
constexpr int64_t kMostAdaptGroups = 1 << 24;

struct AdaptArgs {
    int32_t n, adapters, rank, C, R;  // rows, adapters, their rank, columns of x and of out
    const void *x;                    // [n, C]
    int64_t x_ld;
    int32_t dtype;                    // of x, down, up, grad
    const void *down, *up;            // [adapters, rank, C], [adapters, R, rank]
    const float *scales;              // [adapters], null: ones
    const void *ids;
    int32_t id_dtype;
    const void *base;                 // [n, R] of out_dtype, null: zeros
    int64_t base_ld;
    void *out;
    int64_t out_ld;
    int32_t out_dtype;
    void *workspace;
};
size_t adapt_bytes(int32_t n, int32_t adapters, int32_t rank, int32_t C, int32_t R);
spmv_status adapt(const AdaptArgs &a, hipStream_t s);

struct AdaptGradArgs {
    int32_t n, adapters, rank, C, R;
    const void *grad;                 // [n, R]
    int64_t grad_ld;
    const void *x;                    // [n, C]
    int64_t x_ld;
    int32_t dtype;
    const void *down, *up;
    const float *scales;
    const void *ids;
    int32_t id_dtype;
    const void *base;                 // [n, C] of dtype, null: zeros
    int64_t base_ld;
    void *dx;                         // [n, C] of dtype, null: not wanted
    int64_t dx_ld;
    void *ddown, *dup;                // as down and up, of w_dtype, null: not wanted
    int32_t w_dtype, accumulate;
    void *workspace;
};
size_t adapt_grad_bytes(int32_t n, int32_t adapters, int32_t rank, int32_t C, int32_t R);
spmv_status adapt_grad(const AdaptGradArgs &a, hipStream_t s);

}  // namespace spmv
