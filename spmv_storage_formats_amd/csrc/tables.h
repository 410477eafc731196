// Internal declarations of the weight-table operators: 4-bit matrices with
// group scales (quant.hip, quant_run_*.hip), row lookups and their gradient
// (lookup.hip).  Nothing here is part of the public C ABI.
#pragma once

#include <algorithm>

#include "internal.h"

// The 4-bit matrix.  Rows are cut into tiles of kQuantRows, columns into
// blocks of kQuantCols; both are padded with code 0 and scale 0.  The codes of
// one (tile, block) are 1 KiB.  A word holds eight consecutive columns
// k0 .. k0+7 (an octet): bits rotated left by 3 of
//     sum_i code[k0 + 2i] << 4i  |  code[k0 + 2i + 1] << (16 + 4i),
// so that a shift and a mask bring two neighbouring codes to the mantissa
// bits of two 16-bit floats.  The 16 bytes that a lane of the product loads
// are octets q, q + 4, q + 8, q + 12 of a row's 16 (q = the lane's quad): four
// matrix instructions, each over 32 consecutive columns.  Four rows' 16 bytes
// lie side by side (neighbouring lanes load neighbouring bytes: 16 accesses
// of the vector cache per load instruction instead of 64), then the quads,
// then the next four rows: a row's 64 bytes are spread over 256, which is
// what a lookup of it reads.
// Scales and zero points, by tile and set of groups (the `set` groups of one
// block of columns, or one group of 128 columns and more): scales [4 quads]
// [set][4 rows], zero points [16 rows][set], so that a lane of the product has
// its rows' scales, and its row's zero points, of a whole block in one load.
struct spmv_quant {
    int device = 0;
    int32_t R = 0, C = 0, group = 0;
    int32_t groups = 0;       // ceil(C / group)
    int32_t set = 1;          // groups per block: 128 / group, at least 1
    int32_t sets = 0;         // sets that the column blocks reach
    int32_t tiles = 0;        // ceil(R / kQuantRows)
    int32_t blocks = 0;       // ceil(C / kQuantCols)
    int32_t scale_dtype = 0;
    uint32_t *codes = nullptr;
    void *scales = nullptr;
    uint8_t *zeros = nullptr;  // null: zero points of 8
    int64_t device_bytes = 0;
};

namespace spmv {

constexpr int kQuantRows = 16;
constexpr int kQuantCols = 128;
constexpr int kQuantOctets = kQuantCols / 8;                 // 16
constexpr int kQuantBlockWords = kQuantRows * kQuantOctets;  // 256

// Vectors of a product, at most: kernels take them in passes of up to kMostPass
// and form the indexes of a whole pass, past the last vector, in 32 bits.
constexpr int kMostPass = 48;
constexpr int32_t kMostVectors = INT32_MAX - kMostPass;

using bf16 = __bf16;
using f16 = _Float16;

template <typename T>
struct DTypeOf;
template <>
struct DTypeOf<float> {
    static constexpr spmv_dtype value = SPMV_FP32;
};
template <>
struct DTypeOf<f16> {
    static constexpr spmv_dtype value = SPMV_FP16;
};
template <>
struct DTypeOf<bf16> {
    static constexpr spmv_dtype value = SPMV_BF16;
};

// Workgroups for n items: at most kMostGroups (a launch counts its threads in
// 32 bits); every kernel strides over its items by the grid.
constexpr int64_t kMostGroups = 1 << 21;
inline unsigned groups_for(int64_t n, int per_group) {
    const int64_t groups = std::min(kMostGroups, (n + per_group - 1) / per_group);
    return static_cast<unsigned>(std::max<int64_t>(1, groups));
}

inline bool float_dtype(int32_t d) { return d == SPMV_FP32 || d == SPMV_FP16 || d == SPMV_BF16; }
inline bool id_dtype_ok(int32_t d) { return d == SPMV_INT32 || d == SPMV_INT64; }
inline size_t dtype_bytes(int32_t d) {
    return d == SPMV_INT64 ? 8 : d == SPMV_FP32 || d == SPMV_INT32 ? 4 : 2;
}

// f(T{}) for the type of a floating spmv_dtype
template <typename F>
auto with_float(int32_t d, F f) {
    return d == SPMV_FP32 ? f(float{}) : d == SPMV_FP16 ? f(f16{}) : f(bf16{});
}

// E consecutive elements.  Rows start at any element, so the vectors carry
// their element's alignment; gfx950 loads and stores them whole.
template <typename T, int E>
struct alignas(sizeof(T)) Piece {
    T v[E];
};

template <int E, typename T>
__device__ inline void load_piece(const T *p, float *out) {
    Piece<T, E> o;
    __builtin_memcpy(&o, p, sizeof(o));
#pragma unroll
    for (int i = 0; i < E; ++i) out[i] = static_cast<float>(o.v[i]);
}

// Elements i < count; the others are zero.
template <int E, typename T>
__device__ inline void load_piece_tail(const T *p, int count, float *out) {
#pragma unroll
    for (int i = 0; i < E; ++i) out[i] = i < count ? static_cast<float>(p[i]) : 0.f;
}

template <int E, typename T>
__device__ inline void store_piece(T *p, const float *in) {
    Piece<T, E> o;
#pragma unroll
    for (int i = 0; i < E; ++i) o.v[i] = static_cast<T>(in[i]);
    __builtin_memcpy(p, &o, sizeof(o));
}

template <int E, typename T>
__device__ inline void store_piece_tail(T *p, int count, const float *in) {
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < count) p[i] = static_cast<T>(in[i]);
}

// Word of (row r of a tile, octet o of a block) in its block, and the code of
// column k0 + e in a word (the layout above).
__host__ __device__ inline int quant_word(int r, int o) {
    return (r / 4) * 64 + (o % 4) * 16 + (r % 4) * 4 + o / 4;
}
__device__ inline uint32_t quant_code(uint32_t word, int e) {
    const int bit = ((e & 1) * 16 + (e >> 1) * 4 + 3) & 31;
    return __builtin_amdgcn_alignbit(word, word, bit) & 15u;
}

// Lanes that share a row of `octets` octets: a power of two, 4 to `most`.
inline int lanes_for(int64_t octets, int most) {
    int L = 4;
    while (L < octets && L < most) L *= 2;
    return L;
}

// Place of the scale, and of the zero point, of (row r, group g); set is 1, 2
// or 4.
__device__ inline int64_t quant_scale_at(int64_t r, int32_t g, int32_t set, int32_t sets) {
    const int32_t first = g >> (set / 2), in = g & (set - 1);
    return (r / kQuantRows * sets + first) * (kQuantRows * set) +
           ((r % kQuantRows / 4) * set + in) * 4 + r % 4;
}
__device__ inline int64_t quant_zero_at(int64_t r, int32_t g, int32_t set, int32_t sets) {
    const int32_t first = g >> (set / 2), in = g & (set - 1);
    return (r / kQuantRows * sets + first) * (kQuantRows * set) + r % kQuantRows * set + in;
}

// quant.hip: builders, export, lookup
spmv_status quant_fill_dense(spmv_quant *q, const void *w, int64_t ld, int32_t dtype, int *flag,
                             hipStream_t s);
spmv_status quant_fill_packed(spmv_quant *q, const uint8_t *codes, const void *scales,
                              const uint8_t *zeros, int validate, int *flag, hipStream_t s);
spmv_status quant_unpack(const spmv_quant *q, spmv_quant_array which, void *dev_dst,
                         hipStream_t s);
spmv_status quant_lookup(const spmv_quant *q, int64_t n, const void *ids, int32_t id_dtype,
                         float scale, void *out, int64_t ld, int32_t dtype, hipStream_t s);

// quant_run_*.hip: y <- W x (+ y)
size_t quant_run_bytes(const spmv_quant *q, int32_t n, int32_t x_dtype);  // of workspace
spmv_status quant_run(const spmv_quant *q, int32_t n, const void *x, int64_t x_ld,
                      int32_t x_dtype, void *y, int64_t y_ld, int32_t y_dtype, int accumulate,
                      void *workspace, hipStream_t s);

// lookup.hip
spmv_status lookup_rows(int32_t V, int32_t D, const void *table, int64_t table_ld, int32_t dtype,
                        int64_t n, const void *ids, int32_t id_dtype, float scale, void *out,
                        int64_t out_ld, int32_t out_dtype, hipStream_t s);
size_t lookup_grad_bytes(int32_t V, int32_t D, int64_t n);  // of workspace
spmv_status lookup_grad(int32_t V, int32_t D, int64_t n, const void *ids, int32_t id_dtype,
                        const void *grad, int64_t grad_ld, int32_t grad_dtype, float scale,
                        int accumulate, void *dtable, int64_t ld, int32_t dtype, void *workspace,
                        hipStream_t s);

}  // namespace spmv
