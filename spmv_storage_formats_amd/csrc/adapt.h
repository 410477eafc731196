// Low-rank adapters of many requests beside a shared projection: the kernels,
// included by one source per type (adapt_*.hip); adapt.hip plans and launches.
//
//   out[t] = base[t] + s[a] up[a] h[t],   h[t] = down[a] x[t],        a = ids[t]
//   dx[t]  = base[t] + down[a]^T g[t],    g[t] = s[a] up[a]^T grad[t]
//   ddown[a] = sum_t g[t] x[t]^T,         dup[a] = s[a] sum_t grad[t] h[t]^T
//
// Rows are sorted by adapter and cut into tiles of one adapter each
// (k_adapt_group, adapt.hip).  Each formula is one of three products:
//   shrink:  a tile's long rows by a matrix, to `rank` numbers per row (h, g);
//   expand:  those numbers by a matrix, to long rows (out, dx);
//   weights: sums over a chunk of rows (ddown, dup), joined in their order.
// A matrix is stored with the summed index last (down in shrink, up in expand)
// or first (up in shrink, down in expand: "across").  All sums are in fp32 on
// the matrix unit and made in an order that the sorted rows fix.
//
// The numbers between two products are fp32.  Beside bf16 matrices they are
// split into bf16 parts by their bits, from the top: two parts (16 bits) where
// the result is rounded to bf16, three (all 24) where it is fp32.  fp16 and
// fp32 operands multiply them as fp32 numbers.
#pragma once

#include <type_traits>

#include "requests.h"

namespace spmv {

constexpr int kAdaptTile = 64;     // rows of a tile, at most
constexpr int kAdaptChunk = 512;   // rows of a chunk, at most
constexpr int kAdaptThreads = 256;
constexpr int kAdaptWaves = kAdaptThreads / kWave;

// `count` rows from place `first` of the sorted list; adapter -1: no tile.
struct AdaptTile {
    int32_t adapter, first, count, pad;
};

// The rows of a workgroup's tile.  Up to kAdaptDirect rows there are no lists:
// workgroup t finds the rows of row t's adapter by itself, and takes 16 of them
// from t on if t is the first, the 17th, ... of them.
constexpr int kAdaptDirect = 256;
struct RowsArgs {
    const void *ids;
    int32_t id_dtype;
    int32_t n, adapters;
    const int32_t *order;       // rows sorted by adapter
    const AdaptTile *tiles;     // null: find them
};

struct ShrinkArgs {
    RowsArgs rows;
    const void *x;          // [n, D]
    int64_t x_ld;
    const void *w;          // adapters x [rank, D], or across [D, rank]
    int32_t D, rank, width;     // width: adapt_width(rank)
    int32_t splits, part;   // parts of D, columns of each
    float *sums;            // [splits][n][width]
};

struct ExpandArgs {
    RowsArgs rows;
    const float *sums;      // [splits][n][width]
    int32_t splits, width;
    const float *scales;
    const void *w;          // adapters x [D, rank], or across [rank, D]
    int32_t D, rank;
    const void *base;
    int64_t base_ld;
    void *out;
    int64_t out_ld;
    int32_t columns;        // of a workgroup, whole kExpandColumns
};

struct FinishArgs {         // sums of splits, scaled, rank by rank
    const float *sums;
    int32_t splits, width, n, rank, adapters;
    const float *scales;
    const int32_t *order;
    const AdaptTile *tiles;
    void *out;              // [width][stride], rows in sorted order: fp32, or three
    int32_t stride;         // such arrays of bf16 parts
};

struct WeightArgs {
    const void *x;          // [n, D]
    int64_t x_ld;
    const void *v;          // FinishArgs::out
    int32_t stride, D, rank, width;
    const int32_t *order;
    const AdaptTile *chunks;
    float *partial;         // chunks x [rank, D], or across [D, rank]
    void *out;              // where a chunk is all of its adapter: the gradients themselves
    int32_t accumulate, out_fp32;
    int32_t blocks;         // of columns
};

template <typename T>
struct Adapt {
    static void shrink(const ShrinkArgs &a, int64_t tiles, hipStream_t s);
    static void shrink_both(const ShrinkArgs &a, const ShrinkArgs &across, int64_t tiles,
                            hipStream_t s);
    static void expand(const ExpandArgs &a, bool across, bool out_fp32, int64_t tiles,
                       hipStream_t s);
    // ddown from x and dup (across) from grad; either may have no blocks
    static void weights(const WeightArgs &down, const WeightArgs &up, int32_t adapters,
                        int64_t chunks, hipStream_t s);
};

// Ranks as the kernels hold them.
inline int32_t adapt_width(int32_t rank) {
    int32_t w = 16;
    while (w < rank) w *= 2;
    return w;
}
// Ranks of a workgroup of shrink and weights; more are further workgroups.
inline int32_t adapt_slabs(int32_t rank) { return (rank + 63) / 64; }
constexpr int32_t kExpandColumns = 128;                  // of a wave, at a time
constexpr int32_t kWeightColumns = 128;                  // of a workgroup

// bf16 parts of a number: its upper 16 bits, the next ones of the rest, the rest.
__device__ inline bf16 upper(float v) {
    return __builtin_bit_cast(bf16, static_cast<uint16_t>(__builtin_bit_cast(uint32_t, v) >> 16));
}
__device__ inline float below(float v) {  // 0 where nothing is left, infinities among them
    const float u = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u);
    return v == u ? 0.f : v - u;
}

#ifdef SPMV_ADAPT_KERNELS
namespace {

using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using bf16x8 = bf16 __attribute__((ext_vector_type(8)));
using f16x8 = f16 __attribute__((ext_vector_type(8)));

// Operands: the lane's row (or column) is lane % 16, its summed indexes eight
// neighbours from 8 * (lane / 16).  Results: column lane % 16, rows
// 4 * (lane / 16) + 0..3.
__device__ inline f32x4 multiply(Piece<bf16, 8> a, Piece<bf16, 8> b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 multiply(Piece<f16, 8> a, Piece<f16, 8> b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 multiply(const Piece<float, 8> &a, const Piece<float, 8> &b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

template <typename T, int E>
__device__ inline Piece<T, E> load_some(const T *p, int64_t there) {
    Piece<T, E> o;
    if (there >= E) {
        __builtin_memcpy(&o, p, sizeof(o));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) o.v[i] = i < there ? p[i] : static_cast<T>(0.f);
    }
    return o;
}

// --------------------------------------------------------------------- rows

struct RowsShared {
    int32_t row[kAdaptTile];
    unsigned long long same[kAdaptDirect / kWave];
};

// The tile's rows to LDS; returns its adapter (`adapters`: none, -1: no tile)
// and their number.
__device__ inline int32_t find_rows(const RowsArgs &a, RowsShared &s, int32_t *count) {
    const int tid = threadIdx.x, lane = tid % kWave;
    if (a.tiles) {
        const AdaptTile tile = a.tiles[blockIdx.x];
        if (tile.adapter >= 0 && tid < tile.count) s.row[tid] = a.order[tile.first + tid];
        __syncthreads();
        *count = tile.count;
        return tile.adapter;
    }
    auto key = [&](int32_t t) -> int32_t {
        const int64_t id = a.id_dtype == SPMV_INT32 ? static_cast<const int32_t *>(a.ids)[t]
                                                    : static_cast<const int64_t *>(a.ids)[t];
        return id >= 0 && id < a.adapters ? static_cast<int32_t>(id) : a.adapters;
    };
    const int32_t t = static_cast<int32_t>(blockIdx.x), own = key(t);
    const bool same = tid < a.n && key(tid) == own;
    const unsigned long long mask = __ballot(same);
    if (lane == 0) s.same[tid / kWave] = mask;
    __syncthreads();
    int32_t before = 0, total = 0, place = 0;   // rows of the adapter before t, all, before tid
#pragma unroll
    for (int w = 0; w < kAdaptDirect / kWave; ++w) {
        const unsigned long long m = s.same[w];
        const int at = t - w * kWave, me = tid - w * kWave;
        total += __popcll(m);
        before += at >= kWave ? __popcll(m) : at > 0 ? __popcll(m & ((1ull << at) - 1)) : 0;
        place += me >= kWave ? __popcll(m) : me > 0 ? __popcll(m & ((1ull << me) - 1)) : 0;
    }
    const bool first = before % 16 == 0;
    if (first && same && place >= before && place < before + 16) s.row[place - before] = tid;
    __syncthreads();
    *count = total - before < 16 ? total - before : 16;
    return first ? own : -1;
}

// ------------------------------------------------------------------- shrink

// A workgroup takes a tile, a part of the columns and up to 64 ranks; its waves
// take every fourth 32 columns and add up in LDS.  M: row tiles of 16 that the
// tile fills.
template <typename T, int RB, bool kAcross, int M>
__device__ inline void shrink_rows(const ShrinkArgs &a, int32_t adapter, int32_t count,
                                   const int32_t *rows, int32_t split, int32_t rank0,
                                   float *lds) {
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const T *w = static_cast<const T *>(a.w) + static_cast<int64_t>(adapter) * a.rank * a.D;
    const T *xp[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int32_t k = m * 16 + i16 < count ? m * 16 + i16 : count - 1;
        xp[m] = static_cast<const T *>(a.x) + rows[k] * a.x_ld;
    }
    f32x4 sum[M][RB];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < RB; ++b) sum[m][b] = f32x4{0, 0, 0, 0};
    const T *wp[RB];  // ranks past the last repeat it: not used
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int32_t k = rank0 + b * 16 + i16;
        const int32_t row = k < a.rank ? k : a.rank - 1;
        wp[b] = w + (kAcross ? row : static_cast<int64_t>(row) * a.D);
    }
    struct Step {
        Piece<T, 8> x[M], m[RB];
    };
    auto load = [&](int64_t c, Step &s) {
        const int64_t at = c + q * 8;
#pragma unroll
        for (int u = 0; u < M; ++u) s.x[u] = load_some<T, 8>(xp[u] + at, 8);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if constexpr (kAcross) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s.m[b].v[e] = wp[b][(at + e) * a.rank];
            } else {
                s.m[b] = load_some<T, 8>(wp[b] + at, 8);
            }
        }
    };
    auto add = [&](const Step &s) {
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
            for (int b = 0; b < RB; ++b) sum[u][b] = multiply(s.x[u], s.m[b], sum[u][b]);
    };
    constexpr int kStep = kAdaptWaves * 32;
    const int64_t from = static_cast<int64_t>(split) * a.part;
    const int64_t to = from + a.part < a.D ? from + a.part : a.D;
    int64_t c = from + wave * 32;
    if (c + 32 <= to) {
        // The next columns are loaded before these are multiplied; no branch
        // around a load: the last ones are loaded again.
        Step cur, nxt;
        load(c, cur);
        for (; c + 32 <= to; c += kStep) {
            load(c + kStep + 32 <= to ? c + kStep : c, nxt);
            add(cur);
            cur = nxt;
        }
    }
    if (c < to) {
        const int64_t at = c + q * 8, there = to - at;
        Step s;
#pragma unroll
        for (int u = 0; u < M; ++u) s.x[u] = load_some<T, 8>(xp[u] + at, there);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if constexpr (kAcross) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s.m[b].v[e] = e < there ? wp[b][(at + e) * a.rank] : static_cast<T>(0.f);
            } else {
                s.m[b] = load_some<T, 8>(wp[b] + at, there);
            }
        }
        add(s);
    }
    // the waves' sums, two and two
    f32x4 *const part = reinterpret_cast<f32x4 *>(lds);
#pragma unroll
    for (int step = kAdaptWaves / 2; step >= 1; step /= 2) {
        __syncthreads();
        if (wave >= step && wave < 2 * step) {
#pragma unroll
            for (int u = 0; u < M * RB; ++u)
                part[((wave - step) * M * RB + u) * kWave + lane] = sum[u / RB][u % RB];
        }
        __syncthreads();
        if (wave < step) {
#pragma unroll
            for (int u = 0; u < M * RB; ++u)
                sum[u / RB][u % RB] += part[(wave * M * RB + u) * kWave + lane];
        }
    }
    if (wave != 0) return;
#pragma unroll
    for (int u = 0; u < M; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int32_t k = u * 16 + q * 4 + e;
            if (k >= count) continue;
            float *row = a.sums +
                         (static_cast<int64_t>(split) * a.rows.n + rows[k]) * a.width + rank0 + i16;
#pragma unroll
            for (int b = 0; b < RB; ++b) row[b * 16] = sum[u][b][e];
        }
}

template <typename T, int RB>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_shrink(ShrinkArgs a) {
    __shared__ __attribute__((aligned(16))) float lds[2 * 4 * RB * kWave * 4];
    __shared__ RowsShared s_rows;
    int32_t count;
    const int32_t adapter = find_rows(a.rows, s_rows, &count);
    if (adapter < 0 || adapter >= a.rows.adapters) return;
    const int32_t rank0 = static_cast<int32_t>(blockIdx.z) * 64;
    if (count <= 16)
        shrink_rows<T, RB, false, 1>(a, adapter, count, s_rows.row, blockIdx.y, rank0, lds);
    else
        shrink_rows<T, RB, false, 4>(a, adapter, count, s_rows.row, blockIdx.y, rank0, lds);
}

// x by down and grad by up, in one launch.
template <typename T, int RB>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_shrink_both(ShrinkArgs a, ShrinkArgs c) {
    __shared__ __attribute__((aligned(16))) float lds[2 * 4 * RB * kWave * 4];
    __shared__ RowsShared s_rows;
    int32_t count;
    const int32_t adapter = find_rows(a.rows, s_rows, &count);
    if (adapter < 0 || adapter >= a.rows.adapters) return;
    const int32_t rank0 = static_cast<int32_t>(blockIdx.z) * 64;
    const int32_t y = static_cast<int32_t>(blockIdx.y);
    if (y < a.splits)
        shrink_rows<T, RB, false, 4>(a, adapter, count, s_rows.row, y, rank0, lds);
    else
        shrink_rows<T, RB, true, 4>(c, adapter, count, s_rows.row, y - a.splits, rank0, lds);
}

// ------------------------------------------------------------------- expand

// Eight rows of eight 16-bit numbers, turned into columns.
template <typename T>
__device__ inline void turn(const Piece<T, 8> (&row)[8], Piece<T, 8> (&col)[8]) {
    u32x4 in[8], out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i] = __builtin_bit_cast(u32x4, row[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[j][i] = __builtin_amdgcn_perm(in[2 * i + 1][j / 2], in[2 * i][j / 2],
                                              j % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
    for (int j = 0; j < 8; ++j) col[j] = __builtin_bit_cast(Piece<T, 8>, out[j]);
}

// The numbers of a row, as operands beside a matrix of type T.  The ranks are
// taken in G groups of 32, eight of a lane; G = 0: one of up to 16, and the
// operand's other half takes the next part of the same ranks.
//   bf16: parts by the bits, two or (kAll) three.
//   fp16: two parts of 11 bits, of the numbers times the power of two that
//   brings the row's largest between 2^14 and 2^15: the parts lose nothing that
//   is not 2^-39 of it.  The results are multiplied by its inverse.
//   fp32: as they are.
template <typename T, int G, bool kAll>
struct Numbers;

template <int G, bool kAll>
struct Numbers<bf16, G, kAll> {
    static constexpr int kPer = 8;
    static constexpr int kGroups = G == 0 ? 1 : G;
    static constexpr int kParts = G == 0 ? (kAll ? 2 : 1) : (kAll ? 3 : 2);
    Piece<bf16, 8> p[kGroups][kParts];
    static __device__ inline int first(int g, int q) { return G == 0 ? q % 2 * 8 : g * 32 + q * 8; }
    __device__ inline float set(const float (&h)[kGroups][8], int q) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = h[g][i], next = below(v);
                const bf16 mid = kAll ? upper(next) : static_cast<bf16>(next);
                if constexpr (G == 0) {
                    p[g][0].v[i] = q < 2 ? upper(v) : mid;
                    if constexpr (kAll)
                        p[g][1].v[i] = q < 2 ? upper(below(next)) : static_cast<bf16>(0.f);
                } else {
                    p[g][0].v[i] = upper(v);
                    p[g][1].v[i] = mid;
                    if constexpr (kAll) p[g][2].v[i] = upper(below(next));
                }
            }
        return 1.f;
    }
    __device__ inline f32x4 by(int g, const Piece<bf16, 8> &w, f32x4 c) const {
#pragma unroll
        for (int k = kParts - 1; k >= 0; --k) c = multiply(p[g][k], w, c);
        return c;
    }
};

template <int G, bool kAll>
struct Numbers<f16, G, kAll> {
    static constexpr int kPer = 8;
    static constexpr int kGroups = G == 0 ? 1 : G;
    static constexpr int kParts = G == 0 ? 1 : 2;
    Piece<f16, 8> p[kGroups][kParts];
    static __device__ inline int first(int g, int q) { return G == 0 ? q % 2 * 8 : g * 32 + q * 8; }
    __device__ inline float set(const float (&h)[kGroups][8], int q) {
        float most = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(h[g][i]));
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        int e = static_cast<int>(__builtin_bit_cast(uint32_t, most) >> 23);
        e = e < 15 ? 15 : e == 255 ? 141 : e;  // infinities: as they are
        const float up = __builtin_bit_cast(float, static_cast<uint32_t>(268 - e) << 23);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = h[g][i] * up;
                const f16 lead = static_cast<f16>(v);
                const float left = v - static_cast<float>(lead);
                const f16 rest = static_cast<f16>(v == static_cast<float>(lead) ? 0.f : left);
                if constexpr (G == 0) {
                    p[g][0].v[i] = q < 2 ? lead : rest;
                } else {
                    p[g][0].v[i] = lead;
                    p[g][1].v[i] = rest;
                }
            }
        return __builtin_bit_cast(float, static_cast<uint32_t>(e - 14) << 23);
    }
    __device__ inline f32x4 by(int g, const Piece<f16, 8> &w, f32x4 c) const {
#pragma unroll
        for (int k = kParts - 1; k >= 0; --k) c = multiply(p[g][k], w, c);
        return c;
    }
};

template <int G, bool kAll>
struct Numbers<float, G, kAll> {
    static constexpr int kPer = G == 0 ? 4 : 8;
    static constexpr int kGroups = G == 0 ? 1 : G;
    Piece<float, kPer> p[kGroups];
    static __device__ inline int first(int g, int q) { return g * 32 + q * kPer; }
    __device__ inline float set(const float (&h)[kGroups][kPer], int) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int i = 0; i < kPer; ++i) p[g].v[i] = h[g][i];
        return 1.f;
    }
    __device__ inline f32x4 by(int g, const Piece<float, kPer> &w, f32x4 c) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[g].v[i], w.v[i], c, 0, 0, 0);
        return c;
    }
};

// A workgroup takes a tile and a range of columns.  A wave keeps the numbers of
// 16 rows in registers and goes over its columns, 128 at a time; the waves take
// further rows first, then further columns.  Column tile j holds columns
// i16 * 8 + j, so that a lane's results of one row are eight neighbours and 16
// lanes read the base and write 256 neighbouring bytes.
template <typename T, typename B, int G, bool kAcross>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_expand(ExpandArgs a) {
    using H = Numbers<T, G, sizeof(B) == 4>;
    constexpr int K = H::kPer, NG = H::kGroups;
    __shared__ RowsShared s_rows;
    int32_t count;
    const int32_t adapter = find_rows(a.rows, s_rows, &count);
    if (adapter < 0) return;
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool adapted = adapter < a.rows.adapters;
    if (!adapted && a.base == a.out) return;
    const int turns = count <= 16 ? 4 : count <= 32 ? 2 : 1;  // waves on the same rows
    const int row0 = wave / turns * 16;
    if (row0 >= count) return;
    const T *w = static_cast<const T *>(a.w) +
                 static_cast<int64_t>(adapted ? adapter : 0) * a.rank * a.D;
    H h;
    float back[4] = {1.f, 1.f, 1.f, 1.f};
    if (adapted) {
        const float scale = a.scales ? a.scales[adapter] : 1.f;
        const int32_t t = s_rows.row[row0 + i16 < count ? row0 + i16 : count - 1];
        float v[NG][K];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float *p = a.sums + static_cast<int64_t>(t) * a.width + H::first(g, q);
            load_piece<K>(p, v[g]);
            for (int32_t j = 1; j < a.splits; ++j) {
                float more[K];
                load_piece<K>(p + static_cast<int64_t>(j) * a.rows.n * a.width, more);
#pragma unroll
                for (int i = 0; i < K; ++i) v[g][i] += more[i];
            }
#pragma unroll
            for (int i = 0; i < K; ++i)
                v[g][i] = H::first(g, q) + i < a.rank ? v[g][i] * scale : 0.f;
        }
        const float factor = h.set(v, q);
        if constexpr (std::is_same<T, f16>::value) {
#pragma unroll
            for (int e = 0; e < 4; ++e) back[e] = __shfl(factor, q * 4 + e);
        }
    }
    const B *base[4];
    B *out[4];
    bool there[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // the rows of this lane's results
        const int32_t k = row0 + q * 4 + e;
        there[e] = k < count;
        const int64_t t = s_rows.row[there[e] ? k : 0];
        base[e] = static_cast<const B *>(a.base) + t * a.base_ld;
        out[e] = static_cast<B *>(a.out) + t * a.out_ld;
    }
    // Ranks past the last: their lanes load others, which count as 0.
    using Bits = Piece<uint32_t, K * sizeof(T) / 4>;
    Bits keep[NG];
    int32_t k0[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int32_t first = H::first(g, q);
        k0[g] = first < a.rank ? first : 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const uint32_t m = first + i < a.rank ? ~0u : 0u;
            if constexpr (sizeof(T) == 4)
                keep[g].v[i] = m;
            else
                keep[g].v[i / 2] = i % 2 ? keep[g].v[i / 2] | (m << 16) : m & 0xffffu;
        }
    }
    auto block = [&](int64_t c0, auto fast) {
        constexpr bool kFast = decltype(fast)::value;  // every load in bounds
        const int64_t col = c0 + i16 * 8;
        const int64_t left = kFast ? 8 : a.D - col;
        Piece<B, 8> o[4];
        if (a.base) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = load_some<B, 8>(base[e] + col, left);
        }
        f32x4 sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = f32x4{0, 0, 0, 0};
        if (adapted) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                Piece<T, K> m[8];
                if constexpr (kAcross) {
                    Piece<T, 8> r[K];
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int32_t row = k0[g] + k < a.rank ? k0[g] + k : a.rank - 1;
                        r[k] = load_some<T, 8>(w + static_cast<int64_t>(row) * a.D + col, left);
                    }
                    if constexpr (sizeof(T) == 2) {
                        turn(r, m);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int k = 0; k < K; ++k) m[j].v[k] = r[k].v[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        m[j] = load_some<T, K>(w + (col + j) * a.rank + k0[g],
                                               kFast ? K : j < left ? a.rank - k0[g] : 0);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    Bits bits = __builtin_bit_cast(Bits, m[j]);
#pragma unroll
                    for (unsigned i = 0; i < K * sizeof(T) / 4; ++i) bits.v[i] &= keep[g].v[i];
                    sum[j] = h.by(g, __builtin_bit_cast(std::decay_t<decltype(m[0])>, bits), sum[j]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = sum[j][e] * back[e];
                if (a.base) {
                    const float b = static_cast<float>(o[e].v[j]);
                    v[j] = adapted ? v[j] + b : b;
                }
            }
            if (!there[e]) continue;
            if (left >= 8)
                store_piece<8>(out[e] + col, v);
            else if (left > 0)
                store_piece_tail<8>(out[e] + col, static_cast<int>(left), v);
        }
    };
    const int64_t from = static_cast<int64_t>(blockIdx.y) * a.columns;
    const int64_t to = from + a.columns < a.D ? from + a.columns : a.D;
    const int32_t reach = (a.rank - 1) / K * K + K;  // numbers of a matrix row that are loaded
    for (int64_t c0 = from + wave % turns * kExpandColumns; c0 < to;
         c0 += turns * kExpandColumns) {
        const int64_t behind = a.D - c0 - kExpandColumns;  // columns
        if (behind >= 0 && (kAcross || (behind + 1) * a.rank >= reach))
            block(c0, std::true_type{});
        else
            block(c0, std::false_type{});
    }
}

// ------------------------------------------------------------------ weights

// Sums over a chunk's rows of v[k] x[c]: a workgroup takes a chunk, 128 columns
// and up to 64 ranks; its waves take 32 rows in turn and add up in LDS.  The
// lane's rows and columns, 8 x 8, are turned into operands of eight rows for
// eight column tiles (tile j: columns i16 * 8 + j).
template <typename T>
struct Columns;  // x's operands and their product with the parts of v
template <>
struct Columns<bf16> {
    Piece<bf16, 8> c[8];
    __device__ inline void set(const Piece<bf16, 8> (&x)[8]) { turn(x, c); }
    template <bool kAcross>
    __device__ inline f32x4 by(int j, const Piece<bf16, 8> (&v)[3], f32x4 s) const {
#pragma unroll
        for (int p = 2; p >= 0; --p) s = kAcross ? multiply(v[p], c[j], s) : multiply(c[j], v[p], s);
        return s;
    }
};
template <>
struct Columns<f16> {  // two bf16 parts hold the 11 bits of an fp16 number
    Piece<bf16, 8> c[8], d[8];
    __device__ inline void set(const Piece<f16, 8> (&x)[8]) {
        Piece<bf16, 8> lead[8], rest[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = static_cast<float>(x[i].v[j]);
                lead[i].v[j] = upper(f);
                rest[i].v[j] = upper(below(f));
            }
        turn(lead, c);
        turn(rest, d);
    }
    // the rest's product with the third part lies below fp32's last bit
    template <bool kAcross>
    __device__ inline f32x4 by(int j, const Piece<bf16, 8> (&v)[3], f32x4 s) const {
#pragma unroll
        for (int p = 2; p >= 0; --p) {
            if (p < 2) s = kAcross ? multiply(v[p], d[j], s) : multiply(d[j], v[p], s);
            s = kAcross ? multiply(v[p], c[j], s) : multiply(c[j], v[p], s);
        }
        return s;
    }
};
template <>
struct Columns<float> {
    Piece<float, 8> x[8];
    __device__ inline void set(const Piece<float, 8> (&r)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = r[i];
    }
    template <bool kAcross>
    __device__ inline f32x4 by(int j, const Piece<float, 8> (&v)[1], f32x4 s) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = kAcross ? __builtin_amdgcn_mfma_f32_16x16x4f32(v[0].v[i], x[i].v[j], s, 0, 0, 0)
                        : __builtin_amdgcn_mfma_f32_16x16x4f32(x[i].v[j], v[0].v[i], s, 0, 0, 0);
        return s;
    }
};

template <typename T, int RB, bool kAcross>
__device__ inline void weight_sums(const WeightArgs &a, const AdaptTile &chunk, int32_t block,
                                   int32_t rank0, f32x4 (*lds)[8][kWave]) {
    using V = std::conditional_t<sizeof(T) == 4, float, bf16>;
    constexpr int P = sizeof(T) == 4 ? 1 : 3;
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t col0 = static_cast<int64_t>(block) * kWeightColumns;
    const int64_t col = col0 + i16 * 8;  // this lane's eight columns
    f32x4 sum[8][RB];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int b = 0; b < RB; ++b) sum[j][b] = f32x4{0, 0, 0, 0};
    const int64_t part = static_cast<int64_t>(a.stride) * a.width;
    const V *vp[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
        vp[b] = static_cast<const V *>(a.v) +
                static_cast<int64_t>(rank0 + b * 16 + i16) * a.stride + chunk.first;
    const int32_t *order = a.order + chunk.first;
    const bool whole = col0 + kWeightColumns <= a.D;
    struct Step {
        Piece<T, 8> x[8];
        Piece<V, 8> v[RB][P];
    };
    // Rows past the last: their numbers count as 0, beside a row that is there.
    auto load = [&](int32_t t0, Step &s, auto fast) {
        constexpr bool kFast = decltype(fast)::value;
        const int32_t k0 = t0 + q * 8;  // this lane's eight rows of the chunk
        Piece<int32_t, 8> t;
        __builtin_memcpy(&t, order + k0, sizeof(t));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t row = k0 + i < chunk.count ? t.v[i] : order[0];
            s.x[i] = load_some<T, 8>(static_cast<const T *>(a.x) + row * a.x_ld + col,
                                     kFast ? 8 : a.D - col);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                s.v[b][p] = load_some<V, 8>(vp[b] + p * part + k0, 8);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s.v[b][p].v[i] =
                        k0 + i < chunk.count ? s.v[b][p].v[i] : static_cast<V>(0.f);
            }
    };
    auto add = [&](const Step &s) {
        Columns<T> c;
        c.set(s.x);
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j][b] = c.template by<kAcross>(j, s.v[b], sum[j][b]);
    };
    constexpr int kStep = kAdaptWaves * 32;
    int32_t t0 = wave * 32;
    if (whole) {
        if (t0 < chunk.count) {
            Step cur, nxt;
            load(t0, cur, std::true_type{});
#pragma unroll 1
            for (; t0 < chunk.count; t0 += kStep) {
                load(t0 + kStep < chunk.count ? t0 + kStep : t0, nxt, std::true_type{});
                add(cur);
                cur = nxt;
            }
        }
    } else {
#pragma unroll 1
        for (; t0 < chunk.count; t0 += kStep) {
            Step s;
            load(t0, s, std::false_type{});
            add(s);
        }
    }
    float *const to = a.partial + static_cast<int64_t>(blockIdx.x) * a.rank * a.D;
    auto put = [&](int64_t at, float s) {
        if (!a.out) {
            to[at] = s;
        } else {
            const int64_t i = static_cast<int64_t>(chunk.adapter) * a.rank * a.D + at;
            if (a.out_fp32) {
                float *o = static_cast<float *>(a.out) + i;
                *o = a.accumulate ? *o + s : s;
            } else {
                T *o = static_cast<T *>(a.out) + i;
                *o = static_cast<T>(a.accumulate ? static_cast<float>(*o) + s : s);
            }
        }
    };
    // results e of a lane: columns (q * 4 + e) * 8 + j of rank i16; across,
    // ranks q * 4 + e of column i16 * 8 + j.  Each wave adds up and stores
    // neighbours: one e, across two j.
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[wave][j][lane] = sum[j][b];
        __syncthreads();
        if constexpr (kAcross) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = wave * 2 + h;
                f32x4 s = lds[0][j][lane];
#pragma unroll
                for (int w = 1; w < kAdaptWaves; ++w) s += lds[w][j][lane];
                const int64_t c = col + j;
                const int32_t k = rank0 + b * 16 + q * 4;
                if (c >= a.D) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k + e < a.rank) put(c * a.rank + k + e, s[e]);
            }
        } else {
            const int32_t k = rank0 + b * 16 + i16;
            const int64_t c = col0 + (q * 4 + wave) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float s = lds[0][j][lane][wave];
#pragma unroll
                for (int w = 1; w < kAdaptWaves; ++w) s += lds[w][j][lane][wave];
                if (k < a.rank && c + j < a.D) put(static_cast<int64_t>(k) * a.D + c + j, s);
            }
        }
    }
}

template <typename T, int RB>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_weights(WeightArgs down, WeightArgs up,
                                                                 int32_t adapters) {
    __shared__ f32x4 lds[kAdaptWaves][8][kWave];
    const AdaptTile chunk = down.chunks[blockIdx.x];
    if (chunk.adapter < 0 || chunk.adapter >= adapters) return;
    if (chunk.count == 0 && down.accumulate) return;
    const int32_t rank0 = static_cast<int32_t>(blockIdx.z) * 64;
    const int32_t y = static_cast<int32_t>(blockIdx.y);
    if (y < down.blocks)
        weight_sums<T, RB, false>(down, chunk, y, rank0, lds);
    else
        weight_sums<T, RB, true>(up, chunk, y - down.blocks, rank0, lds);
}

}  // namespace

// f(integral_constant<rank blocks of 16 per workgroup>)
template <typename F>
void with_ranks(int32_t rank, F f) {
    if (rank <= 16)
        f(std::integral_constant<int, 1>{});
    else if (rank <= 32)
        f(std::integral_constant<int, 2>{});
    else
        f(std::integral_constant<int, 4>{});
}

// f(integral_constant<groups of 32 ranks; 0: up to 16 ranks>)
template <typename F>
void with_groups(int32_t rank, F f) {
    if (rank <= 16)
        f(std::integral_constant<int, 0>{});
    else if (rank <= 32)
        f(std::integral_constant<int, 1>{});
    else if (rank <= 64)
        f(std::integral_constant<int, 2>{});
    else if (rank <= 128)
        f(std::integral_constant<int, 4>{});
    else
        f(std::integral_constant<int, 8>{});
}

template <typename T>
void Adapt<T>::shrink(const ShrinkArgs &a, int64_t tiles, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.splits),
                    static_cast<unsigned>(adapt_slabs(a.rank)));
    with_ranks(a.rank, [&](auto rb) {
        k_adapt_shrink<T, decltype(rb)::value><<<grid, kAdaptThreads, 0, s>>>(a);
    });
}

template <typename T>
void Adapt<T>::shrink_both(const ShrinkArgs &a, const ShrinkArgs &across, int64_t tiles,
                           hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.splits + across.splits),
                    static_cast<unsigned>(adapt_slabs(a.rank)));
    with_ranks(a.rank, [&](auto rb) {
        k_adapt_shrink_both<T, decltype(rb)::value><<<grid, kAdaptThreads, 0, s>>>(a, across);
    });
}

template <typename T>
void Adapt<T>::expand(const ExpandArgs &a, bool across, bool out_fp32, int64_t tiles,
                      hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles),
                    static_cast<unsigned>((a.D - 1) / a.columns + 1));
    with_groups(a.rank, [&](auto groups) {
        constexpr int G = decltype(groups)::value;
        if (across)  // dx, of the inputs' type
            k_adapt_expand<T, T, G, true><<<grid, kAdaptThreads, 0, s>>>(a);
        else if (out_fp32)
            k_adapt_expand<T, float, G, false><<<grid, kAdaptThreads, 0, s>>>(a);
        else
            k_adapt_expand<T, T, G, false><<<grid, kAdaptThreads, 0, s>>>(a);
    });
}

template <typename T>
void Adapt<T>::weights(const WeightArgs &down, const WeightArgs &up, int32_t adapters,
                       int64_t chunks, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(down.blocks + up.blocks),
                    static_cast<unsigned>(adapt_slabs(down.rank)));
    with_ranks(down.rank, [&](auto rb) {
        k_adapt_weights<T, decltype(rb)::value>
            <<<grid, kAdaptThreads, 0, s>>>(down, up, adapters);
    });
}
#endif

}  // namespace spmv
