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

struct ShrinkArgs {
    const void *x;          // [n, D]
    int64_t x_ld;
    const void *w;          // adapters x [rank, D], or across [D, rank]
    int32_t D, rank, adapters, width;   // width: adapt_width(rank)
    int32_t splits, part;   // parts of D, columns of each
    const int32_t *order;
    const AdaptTile *tiles;
    int32_t n;
    float *sums;            // [splits][n][width], rows in sorted order
};

struct ExpandArgs {
    const float *sums;      // [splits][n][width]
    int32_t splits, width, n;
    const float *scales;
    const void *w;          // adapters x [D, rank], or across [rank, D]
    int32_t D, rank, adapters;
    const int32_t *order;
    const AdaptTile *tiles;
    const void *base;
    int64_t base_ld;
    void *out;
    int64_t out_ld;
    int32_t blocks;         // column blocks of a tile
};

struct FinishArgs {         // sums of splits, scaled, rank by rank
    const float *sums;
    int32_t splits, width, n, rank, adapters;
    const float *scales;
    const AdaptTile *tiles;
    float *out;             // [width][stride]
    int32_t stride;
};

struct WeightArgs {
    const void *x;          // [n, D]
    int64_t x_ld;
    const float *v;         // [width][stride], scaled
    int32_t stride, D, rank, adapters, width;
    const int32_t *order;
    const AdaptTile *chunks;
    float *partial;         // chunks x [rank, D], or across [D, rank]
    int32_t blocks;
};

template <typename T>
struct Adapt {
    static void shrink(const ShrinkArgs &a, bool across, int64_t tiles, hipStream_t s);
    static void expand(const ExpandArgs &a, bool across, bool out_fp32, int64_t tiles,
                       hipStream_t s);
    static void weights(const WeightArgs &a, bool across, int64_t chunks, hipStream_t s);
};

// Columns of a workgroup of expand: fewer where the matrix takes more registers.
inline int32_t expand_columns(int32_t rank) { return kAdaptWaves * (rank > 32 ? 64 : 128); }
// Ranks as the kernels hold them: 16, 32 or 64 of a workgroup.
inline int32_t adapt_width(int32_t rank) {
    return rank <= 16 ? 16 : rank <= 32 ? 32 : (rank + 63) / 64 * 64;
}
// Ranks of a workgroup; more are further workgroups (or turns, in expand).
inline int32_t adapt_slabs(int32_t rank) { return (rank + 63) / 64; }
constexpr int32_t kWeightColumns = kAdaptWaves * 128;

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

// bf16 parts of a number: its upper 16 bits, the next ones of the rest, the rest.
__device__ inline bf16 upper(float v) {
    return __builtin_bit_cast(bf16, static_cast<uint16_t>(__builtin_bit_cast(uint32_t, v) >> 16));
}
__device__ inline float below(float v) {  // 0 where nothing is left, infinities among them
    const float u = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u);
    return v == u ? 0.f : v - u;
}

// ------------------------------------------------------------------- shrink

// A workgroup takes a tile, a part of the columns and up to 64 ranks; its waves
// take every fourth 32 columns and add up in LDS.  M: row tiles of 16 that the
// tile fills.
template <typename T, int RB, bool kAcross, int M>
__device__ inline void shrink_rows(const ShrinkArgs &a, const AdaptTile &tile, int32_t split,
                                   int32_t rank0, float *lds) {
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const T *w = static_cast<const T *>(a.w) +
                 static_cast<int64_t>(tile.adapter) * a.rank * a.D;
    const T *xp[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int32_t k = m * 16 + i16 < tile.count ? m * 16 + i16 : tile.count - 1;
        xp[m] = static_cast<const T *>(a.x) + a.order[tile.first + k] * a.x_ld;
    }
    f32x4 sum[M][RB];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < RB; ++b) sum[m][b] = f32x4{0, 0, 0, 0};
    const int64_t from = static_cast<int64_t>(split) * a.part;
    const int64_t to = from + a.part < a.D ? from + a.part : a.D;
    for (int64_t c = from + wave * 32; c < to; c += kAdaptWaves * 32) {
        const int64_t at = c + q * 8;
        const int64_t there = to - at;
        Piece<T, 8> x[M], m[RB];
#pragma unroll
        for (int u = 0; u < M; ++u) x[u] = load_some<T, 8>(xp[u] + at, there);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int32_t k = rank0 + b * 16 + i16;
            const int32_t row = k < a.rank ? k : a.rank - 1;  // ranks past the last: not used
            if constexpr (kAcross) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    m[b].v[e] = e < there ? w[(at + e) * a.rank + row] : static_cast<T>(0.f);
            } else {
                m[b] = load_some<T, 8>(w + static_cast<int64_t>(row) * a.D + at, there);
            }
        }
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
            for (int b = 0; b < RB; ++b) sum[u][b] = multiply(x[u], m[b], sum[u][b]);
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
            if (k >= tile.count) continue;
            float *row = a.sums + (static_cast<int64_t>(split) * a.n + tile.first + k) * a.width +
                         rank0 + i16;
#pragma unroll
            for (int b = 0; b < RB; ++b) row[b * 16] = sum[u][b][e];
        }
}

template <typename T, int RB, bool kAcross>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_shrink(ShrinkArgs a) {
    __shared__ __attribute__((aligned(16))) float lds[2 * 4 * RB * kWave * 4];
    const AdaptTile tile = a.tiles[blockIdx.x];
    if (tile.adapter < 0 || tile.adapter >= a.adapters) return;
    const int32_t rank0 = static_cast<int32_t>(blockIdx.z) * 64;
    if (tile.count <= 16)
        shrink_rows<T, RB, kAcross, 1>(a, tile, blockIdx.y, rank0, lds);
    else
        shrink_rows<T, RB, kAcross, 4>(a, tile, blockIdx.y, rank0, lds);
}

// ------------------------------------------------------------------- expand

// How the numbers of a row meet a matrix of type T.  A block of 16 ranks is one
// or two operands: bf16 [upper part | next], and [rest | 0] for fp32 results;
// other types four operands of four ranks each.
template <typename T>
struct Meet {  // fp16, fp32
    static constexpr int kRanks = 4;  // ranks of a lane, from 4 * (lane / 16)
    float v[4];
    static __device__ inline int first(int q) { return q * 4; }
    __device__ inline void numbers(const float *h, int, bool) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = h[i];
    }
    template <bool kAll>
    static __device__ inline f32x4 product(const Piece<T, 4> &w, const Meet &h, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(static_cast<float>(w.v[i]), h.v[i], c, 0, 0,
                                                     0);
        return c;
    }
};
template <>
struct Meet<bf16> {
    static constexpr int kRanks = 8;  // lanes of the upper half repeat the lower half's
    Piece<bf16, 8> two, rest;
    static __device__ inline int first(int q) { return q % 2 * 8; }
    __device__ inline void numbers(const float *h, int q, bool all) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float next = below(h[i]);
            if (all) {
                two.v[i] = q < 2 ? upper(h[i]) : upper(next);
                rest.v[i] = q < 2 ? upper(below(next)) : static_cast<bf16>(0.f);
            } else {
                two.v[i] = q < 2 ? upper(h[i]) : static_cast<bf16>(next);
            }
        }
    }
    template <bool kAll>
    static __device__ inline f32x4 product(const Piece<bf16, 8> &w, const Meet &h, f32x4 c) {
        if constexpr (kAll) c = multiply(w, h.rest, c);
        return multiply(w, h.two, c);
    }
};

// A workgroup takes a tile and a block of columns, its waves NT * 16 columns
// each, the matrix's part in registers for all rows.  Column tiles are
// interleaved so that a lane's results are neighbours: its eight (pieces), and
// its 16-lane group's.
template <typename T, typename B, int RB, int NT, bool kAcross>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_expand(ExpandArgs a) {
    constexpr bool kAll = sizeof(B) == 4;
    using H = Meet<T>;
    constexpr int K = H::kRanks;
    constexpr int kStride = RB * 16 + 4;  // of a row in LDS
    __shared__ __attribute__((aligned(16))) float s_h[kAdaptTile * kStride];
    const AdaptTile tile = a.tiles[blockIdx.x];
    if (tile.adapter < 0) return;
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool adapted = tile.adapter < a.adapters;
    const int64_t col0 = (static_cast<int64_t>(blockIdx.y) * kAdaptWaves + wave) * (NT * 16);
    const T *w = static_cast<const T *>(a.w) +
                 static_cast<int64_t>(adapted ? tile.adapter : 0) * a.rank * a.D;
    const float scale = adapted && a.scales ? a.scales[tile.adapter] : 1.f;
    const int32_t slabs = adapted ? (a.rank + RB * 16 - 1) / (RB * 16) : 0;
    // The numbers of rows [from, to) and of this slab's ranks: sums of the splits, scaled.
    auto stage = [&](int from, int to, int32_t rank0) {
        for (int i = from * (RB * 16) + threadIdx.x; i < to * (RB * 16); i += kAdaptThreads) {
            const int row = i / (RB * 16), k = i % (RB * 16);
            float v = 0.f;
            if (row < tile.count && rank0 + k < a.rank) {
                const float *p = a.sums + (static_cast<int64_t>(tile.first) + row) * a.width +
                                 rank0 + k;
                for (int32_t j = 0; j < a.splits; ++j)
                    v += p[static_cast<int64_t>(j) * a.n * a.width];
                v *= scale;
            }
            s_h[row * kStride + k] = v;
        }
    };
    // The matrix: this lane's column of each column tile, K ranks of every block.
    Piece<T, K> m[NT][RB];
    auto load = [&](int32_t rank0) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const int32_t k0 = rank0 + b * 16 + H::first(q);
            if constexpr (kAcross) {
                // columns col0 + i16 * NT + j
                const int64_t col = col0 + i16 * NT;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const bool there = k0 + k < a.rank;
                    const Piece<T, NT> row =
                        load_some<T, NT>(w + static_cast<int64_t>(there ? k0 + k : 0) * a.D + col,
                                         there ? a.D - col : 0);
#pragma unroll
                    for (int j = 0; j < NT; ++j) m[j][b].v[k] = row.v[j];
                }
            } else {
                // columns col0 + j / 2 * 32 + i16 / 4 * 8 + j % 2 * 4 + i16 % 4
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int64_t col = col0 + j / 2 * 32 + i16 / 4 * 8 + j % 2 * 4 + i16 % 4;
                    m[j][b] = load_some<T, K>(w + col * a.rank + k0,
                                              col < a.D ? a.rank - k0 : 0);
                }
            }
        }
    };
    if (slabs == 1) {
        load(0);
        stage(0, kAdaptTile, 0);
        __syncthreads();
    }
#pragma unroll 1
    for (int u = 0; u * 16 < tile.count; ++u) {
        f32x4 sum[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) sum[j] = f32x4{0, 0, 0, 0};
#pragma unroll 1
        for (int32_t slab = 0; slab < slabs; ++slab) {
            if (slabs > 1) {
                __syncthreads();
                stage(u * 16, u * 16 + 16, slab * RB * 16);
                load(slab * RB * 16);
                __syncthreads();
            }
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                H h;
                h.numbers(&s_h[(u * 16 + i16) * kStride + b * 16 + H::first(q)], q, kAll);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    sum[j] = H::template product<kAll>(m[j][b], h, sum[j]);
            }
        }
        // Row u * 16 + i16; pieces of eight neighbouring columns.
        const int32_t k = u * 16 + i16;
        if (k >= tile.count) continue;
        const int64_t t = a.order[tile.first + k];
        const B *base = static_cast<const B *>(a.base) + t * a.base_ld;
        B *out = static_cast<B *>(a.out) + t * a.out_ld;
#pragma unroll
        for (int p = 0; p < NT / 2; ++p) {
            float v[8];
            int64_t col;
            if constexpr (kAcross) {
                // results e of tile j: column (q * 4 + e) * NT + j
                col = col0 + q * 4 * NT + p * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = sum[(p * 8 + i) % NT][(p * 8 + i) / NT];
            } else {
                col = col0 + p * 32 + q * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = sum[p * 2 + i / 4][i % 4];
            }
            if (col + 8 <= a.D) {
                if (a.base) {
                    float o[8];
                    load_piece<8>(base + col, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = adapted ? v[i] + o[i] : o[i];
                }
                store_piece<8>(out + col, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (col + i >= a.D) continue;
                    if (a.base) {
                        const float o = static_cast<float>(base[col + i]);
                        v[i] = adapted ? v[i] + o : o;
                    }
                    out[col + i] = static_cast<B>(v[i]);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ weights

// Sums over a chunk's rows of v[k] x[c]: a workgroup takes a chunk, 512 columns
// and up to 64 ranks, its waves 128 columns each; 32 rows a step.
__device__ inline void turn(const Piece<bf16, 8> (&row)[8], Piece<bf16, 8> (&col)[8]) {
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
    for (int j = 0; j < 8; ++j) col[j] = __builtin_bit_cast(Piece<bf16, 8>, out[j]);
}

template <typename T, int RB, bool kAcross>
__global__ __launch_bounds__(kAdaptThreads) void k_adapt_weights(WeightArgs a) {
    const AdaptTile chunk = a.chunks[blockIdx.x];
    if (chunk.adapter < 0 || chunk.adapter >= a.adapters) return;
    const int lane = threadIdx.x % kWave, i16 = lane % 16, q = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int32_t rank0 = static_cast<int32_t>(blockIdx.z) * 64;
    const int64_t col0 = (static_cast<int64_t>(blockIdx.y) * kAdaptWaves + wave) * 128;
    if (col0 >= a.D) return;
    const int64_t col = col0 + i16 * 8;  // this lane's eight columns
    f32x4 sum[8][RB];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int b = 0; b < RB; ++b) sum[j][b] = f32x4{0, 0, 0, 0};
    for (int32_t t0 = 0; t0 < chunk.count; t0 += 32) {
        const int32_t k0 = t0 + q * 8;  // this lane's eight rows of the chunk
        Piece<T, 8> x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool there = k0 + i < chunk.count;
            const int32_t t = there ? a.order[chunk.first + k0 + i] : 0;
            x[i] = load_some<T, 8>(static_cast<const T *>(a.x) + t * a.x_ld + col,
                                   there ? a.D - col : 0);
        }
        float v[RB][8];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            const float *p = a.v + static_cast<int64_t>(rank0 + b * 16 + i16) * a.stride +
                             chunk.first + k0;
            load_piece<8>(p, v[b]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[b][i] = k0 + i < chunk.count ? v[b][i] : 0.f;
        }
        if constexpr (sizeof(T) == 2 && !std::is_same<T, f16>::value) {
            Piece<bf16, 8> c[8];
            turn(x, c);
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                Piece<bf16, 8> part[3];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float next = below(v[b][i]);
                    part[0].v[i] = upper(v[b][i]);
                    part[1].v[i] = upper(next);
                    part[2].v[i] = upper(below(next));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int p = 2; p >= 0; --p)
                        sum[j][b] = kAcross ? multiply(part[p], c[j], sum[j][b])
                                            : multiply(c[j], part[p], sum[j][b]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c = static_cast<float>(x[i].v[j]);
#pragma unroll
                    for (int b = 0; b < RB; ++b)
                        sum[j][b] = kAcross ? __builtin_amdgcn_mfma_f32_16x16x4f32(
                                                  v[b][i], c, sum[j][b], 0, 0, 0)
                                            : __builtin_amdgcn_mfma_f32_16x16x4f32(
                                                  c, v[b][i], sum[j][b], 0, 0, 0);
                }
        }
    }
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.rank * a.D;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // results: rows are columns of x (ranks, across)
                const int32_t k = rank0 + b * 16 + (kAcross ? q * 4 + e : i16);
                const int64_t c = col0 + (kAcross ? i16 : q * 4 + e) * 8 + j;
                if (k < a.rank && c < a.D)
                    out[kAcross ? c * a.rank + k : static_cast<int64_t>(k) * a.D + c] =
                        sum[j][b][e];
            }
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

template <typename T>
void Adapt<T>::shrink(const ShrinkArgs &a, bool across, int64_t tiles, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.splits),
                    static_cast<unsigned>(adapt_slabs(a.rank)));
    with_ranks(a.rank, [&](auto rb) {
        constexpr int RB = decltype(rb)::value;
        if (across)
            k_adapt_shrink<T, RB, true><<<grid, kAdaptThreads, 0, s>>>(a);
        else
            k_adapt_shrink<T, RB, false><<<grid, kAdaptThreads, 0, s>>>(a);
    });
}

template <typename T>
void Adapt<T>::expand(const ExpandArgs &a, bool across, bool out_fp32, int64_t tiles,
                      hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.blocks));
    with_ranks(a.rank, [&](auto rb) {
        constexpr int RB = decltype(rb)::value;
        constexpr int NT = RB == 4 ? 4 : 8;
        if (across)  // dx, of the inputs' type
            k_adapt_expand<T, T, RB, NT, true><<<grid, kAdaptThreads, 0, s>>>(a);
        else if (out_fp32)
            k_adapt_expand<T, float, RB, NT, false><<<grid, kAdaptThreads, 0, s>>>(a);
        else
            k_adapt_expand<T, T, RB, NT, false><<<grid, kAdaptThreads, 0, s>>>(a);
    });
}

template <typename T>
void Adapt<T>::weights(const WeightArgs &a, bool across, int64_t chunks, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(a.blocks),
                    static_cast<unsigned>(adapt_slabs(a.rank)));
    with_ranks(a.rank, [&](auto rb) {
        constexpr int RB = decltype(rb)::value;
        if (across)
            k_adapt_weights<T, RB, true><<<grid, kAdaptThreads, 0, s>>>(a);
        else
            k_adapt_weights<T, RB, false><<<grid, kAdaptThreads, 0, s>>>(a);
    });
}
#endif

}  // namespace spmv
