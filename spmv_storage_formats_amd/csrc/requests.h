// Internal declarations of the operators on a step's rows, one request's or
// sequence's each: low-rank adapters (adapt.hip, adapt_*.hip) and log
// probabilities of given tokens (logprobs.hip).  Nothing here is part of the
// public C ABI.
#pragma once

#include "tables.h"

namespace spmv {

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

}  // namespace spmv
