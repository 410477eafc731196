// 4-bit matrices with group scales: builders, export, and rows by token.
// The layout is described at struct spmv_quant (tables.h).
#include "tables.h"

namespace spmv {
namespace {

constexpr int kThreads = 256;

#define EACH_ITEM(i, n)                                                                   \
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < (n); \
         i += static_cast<int64_t>(gridDim.x) * kThreads)

__device__ inline int64_t word_index(int32_t r, int32_t octet, int32_t blocks) {
    const int64_t block = static_cast<int64_t>(r / kQuantRows) * blocks + octet / kQuantOctets;
    return block * kQuantBlockWords + quant_word(r % kQuantRows, octet % kQuantOctets);
}

// rne(w / s) with the quotient taken exactly, s > 0.  k = rint of the rounded
// quotient is off by at most one; w - k s is exact in one fused operation
// (a multiple of both operands' last places, below s in size), so comparing
// twice its size with s settles the neighbour and the ties.
__device__ inline float rne_quotient(float w, float s) {
    float k = rintf(w / s);
    const float d = fmaf(-s, k, w);
    const float two = 2.f * fabsf(d);
    if (two > s || (two == s && (static_cast<int>(k) & 1))) k += d > 0.f ? 1.f : -1.f;
    return k;
}

// One group of one row per L lanes (L = 4..64 by the group's octets), a lane
// taking every L-th octet: the extremes first, then the codes (the second
// read of the weights comes from the cache).
template <typename T, typename S>
__global__ __launch_bounds__(kThreads) void k_quant_build(
    int32_t R, int32_t C, int32_t group, int32_t groups, int32_t set, int32_t sets, int32_t blocks,
    int L, const T *__restrict__ w, int64_t ld, uint32_t *__restrict__ codes,
    S *__restrict__ scales, uint8_t *__restrict__ zeros, int *__restrict__ flag) {
    const int per_block = kThreads / L;
    const int sub = threadIdx.x % L;
    const int64_t items = static_cast<int64_t>(R) * groups;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per_block; first < items;
         first += static_cast<int64_t>(gridDim.x) * per_block) {
        const int64_t item = first + threadIdx.x / L;
        const bool live = item < items;
        const int32_t r = live ? static_cast<int32_t>(item / groups) : 0;
        const int32_t g = live ? static_cast<int32_t>(item % groups) : 0;
        const T *row = w + static_cast<int64_t>(r) * ld;
        const int32_t c0 = g * group;
        const int32_t c1 = !live ? c0 : (C - c0 < group ? C : c0 + group);
        const int octets = (c1 - c0 + 7) / 8;

        float lo = 0.f, hi = 0.f;
        bool bad = false;
        for (int o = sub; o < octets; o += L) {
            float v[8];
            load_piece_tail<8>(row + c0 + o * 8, c1 - c0 - o * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bad |= !(fabsf(v[i]) <= 3.402823466e38f);
                lo = fminf(lo, v[i]);
                hi = fmaxf(hi, v[i]);
            }
        }
        for (int m = 1; m < L; m <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, m));
            hi = fmaxf(hi, __shfl_xor(hi, m));
        }
        float s = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
        s = static_cast<float>(static_cast<S>(s));
        bad |= !(s <= 3.402823466e38f);
        if (bad) {
            atomicOr(flag, 1);
            continue;
        }
        float z = 8.f;
        if (zeros) z = s > 0.f ? fminf(rne_quotient(-lo, s), 15.f) : 0.f;
        if (live && sub == 0) {
            scales[quant_scale_at(r, g, set, sets)] = static_cast<S>(s);
            if (zeros) zeros[quant_zero_at(r, g, set, sets)] = static_cast<uint8_t>(z);
        }
        for (int o = sub; o < octets; o += L) {
            float v[8];
            load_piece_tail<8>(row + c0 + o * 8, c1 - c0 - o * 8, v);
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float k = s > 0.f ? rne_quotient(v[i], s) : 0.f;
                const uint32_t q = static_cast<uint32_t>(fminf(fmaxf(k + z, 0.f), 15.f));
                if (o * 8 + i < c1 - c0) word |= q << ((i & 1) * 16 + (i >> 1) * 4);
            }
            codes[word_index(r, c0 / 8 + o, blocks)] = __builtin_amdgcn_alignbit(word, word, 29);
        }
    }
}

// The caller's packed codes to the handle's words: one word per thread.
__global__ __launch_bounds__(kThreads) void k_quant_pack(int32_t R, int32_t C, int32_t octets,
                                                         int32_t blocks,
                                                         const uint8_t *__restrict__ in,
                                                         uint32_t *__restrict__ codes) {
    EACH_ITEM(i, static_cast<int64_t>(R) * octets) {
        const int32_t r = static_cast<int32_t>(i / octets), o = static_cast<int32_t>(i % octets);
        const int64_t row_bytes = (static_cast<int64_t>(C) + 1) / 2;
        const uint8_t *p = in + r * row_bytes + o * 4;
        uint32_t w = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int32_t c = o * 8 + 2 * b;
            if (c < C) {
                const uint32_t v = p[b];
                w |= (v & 15u) << (4 * b);
                if (c + 1 < C) w |= (v >> 4) << (16 + 4 * b);
            }
        }
        codes[word_index(r, o, blocks)] = __builtin_amdgcn_alignbit(w, w, 29);
    }
}

template <typename S>
__global__ __launch_bounds__(kThreads) void k_quant_scales(
    int32_t R, int32_t groups, int32_t set, int32_t sets, int check,
    const S *__restrict__ scales_in, const uint8_t *__restrict__ zeros_in,
    S *__restrict__ scales, uint8_t *__restrict__ zeros, int *__restrict__ flag) {
    EACH_ITEM(i, static_cast<int64_t>(R) * groups) {
        const int32_t r = static_cast<int32_t>(i / groups), g = static_cast<int32_t>(i % groups);
        const S s = scales_in[i];
        bool bad = !(fabsf(static_cast<float>(s)) <= 3.402823466e38f);
        scales[quant_scale_at(r, g, set, sets)] = s;
        if (zeros_in) {
            const uint8_t z = zeros_in[i];
            bad |= z > 15;
            zeros[quant_zero_at(r, g, set, sets)] = z & 15;
        }
        if (check && bad) atomicOr(flag, 1);
    }
}

// Back to the caller's order.
__global__ __launch_bounds__(kThreads) void k_quant_unpack(int32_t R, int32_t C, int32_t blocks,
                                                           const uint32_t *__restrict__ codes,
                                                           uint8_t *__restrict__ out) {
    const int64_t row_bytes = (static_cast<int64_t>(C) + 1) / 2;
    EACH_ITEM(i, R * row_bytes) {
        const int32_t r = static_cast<int32_t>(i / row_bytes);
        const int32_t b = static_cast<int32_t>(i % row_bytes);
        const uint32_t w = codes[word_index(r, b / 4, blocks)];
        const int e = (b & 3) * 2;
        out[i] = static_cast<uint8_t>(quant_code(w, e) | quant_code(w, e + 1) << 4);
    }
}

template <typename S, bool Zeros>
__global__ __launch_bounds__(kThreads) void k_quant_unpack_groups(int32_t R, int32_t groups,
                                                                  int32_t set, int32_t sets,
                                                                  const S *__restrict__ in,
                                                                  S *__restrict__ out) {
    EACH_ITEM(i, static_cast<int64_t>(R) * groups) {
        const int64_t r = i / groups;
        const int32_t g = static_cast<int32_t>(i % groups);
        out[i] = in[Zeros ? quant_zero_at(r, g, set, sets) : quant_scale_at(r, g, set, sets)];
    }
}

// Rows by token: out[t] = scale * s (code - zero).  L lanes per row; a lane
// takes the 16 bytes that lie together, octets q, q + 4, q + 8 and q + 12 of a
// block of 128 columns, so that four lanes store neighbouring octets each time.
// Bound by memory, mostly writes: 8192 rows of 4096 to bf16, 67 MB written and 39
// MB read (three other rows' bytes lie in the same lines), 22 us, 4.7 TB/s, from
// memory; 19 us where the table lies in the last-level cache.
template <typename S, typename T, typename I>
__global__ __launch_bounds__(kThreads) void k_quant_lookup(
    int32_t R, int32_t C, int32_t group, int32_t set, int32_t sets, int32_t blocks, int L,
    const uint32_t *__restrict__ codes, const S *__restrict__ scales,
    const uint8_t *__restrict__ zeros, int64_t n, const I *__restrict__ ids, float scale,
    T *__restrict__ out, int64_t ld) {
    using Four = uint32_t __attribute__((ext_vector_type(4)));
    const int rows = kThreads / L;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / L; t < n;
         t += static_cast<int64_t>(gridDim.x) * rows) {
        const int64_t id = ids[t];
        const bool there = id >= 0 && id < R;
        const int32_t r = there ? static_cast<int32_t>(id) : 0;
        T *row = out + t * ld;
        for (int32_t i = threadIdx.x % L; i / 4 < blocks; i += L) {
            const int32_t c0 = i / 4 * kQuantCols + i % 4 * 8;  // columns c0 + 32 j
            Four w = {0, 0, 0, 0};
            float s[4] = {}, z[4] = {8.f, 8.f, 8.f, 8.f};
            if (there) {
                w = *reinterpret_cast<const Four *>(codes + word_index(r, c0 / 8, blocks));
                // the block's first group, and its others behind it (quant_scale_at's steps)
                const int32_t g = set > 1 ? i / 4 * set : group > kQuantCols ? c0 / group : i / 4;
                const int64_t s0 = quant_scale_at(r, g, set, sets);
                const int64_t z0 = quant_zero_at(r, g, set, sets);
                const int shift = set == 4 ? 0 : set == 2 ? 1 : 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j] = static_cast<float>(scales[s0 + (j >> shift) * 4]);
                    if (zeros) z[j] = static_cast<float>(zeros[z0 + (j >> shift)]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t c = c0 + 32 * j;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = there ? (static_cast<float>(quant_code(w[j], e)) - z[j]) * s[j] * scale
                                 : 0.f;
                if (c + 8 <= C)
                    store_piece<8>(row + c, v);
                else if (c < C)
                    store_piece_tail<8>(row + c, C - c, v);
            }
        }
    }
}

}  // namespace

spmv_status quant_fill_dense(spmv_quant *q, const void *w, int64_t ld, int32_t dtype, int *flag,
                             hipStream_t s) {
    const int64_t items = static_cast<int64_t>(q->R) * q->groups;
    if (items == 0) return SPMV_OK;
    const int L = lanes_for((std::min(q->group, q->C) + 7) / 8, kWave);
    const unsigned grid = groups_for(items, kThreads / L);
    with_float(dtype, [&](auto t) {
        with_float(q->scale_dtype, [&](auto sc) {
            using T = decltype(t);
            using S = decltype(sc);
            k_quant_build<T, S><<<grid, kThreads, 0, s>>>(
                q->R, q->C, q->group, q->groups, q->set, q->sets, q->blocks, L,
                static_cast<const T *>(w), ld, q->codes, static_cast<S *>(q->scales), q->zeros,
                flag);
        });
    });
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

spmv_status quant_fill_packed(spmv_quant *q, const uint8_t *codes, const void *scales,
                              const uint8_t *zeros, int validate, int *flag, hipStream_t s) {
    const int32_t octets = static_cast<int32_t>((static_cast<int64_t>(q->C) + 7) / 8);
    const int64_t words = static_cast<int64_t>(q->R) * octets;
    if (words == 0) return SPMV_OK;
    k_quant_pack<<<groups_for(words, kThreads), kThreads, 0, s>>>(q->R, q->C, octets, q->blocks,
                                                                codes, q->codes);
    SPMV_HIP(hipGetLastError());
    const int64_t items = static_cast<int64_t>(q->R) * q->groups;
    with_float(q->scale_dtype, [&](auto sc) {
        using S = decltype(sc);
        k_quant_scales<S><<<groups_for(items, kThreads), kThreads, 0, s>>>(
            q->R, q->groups, q->set, q->sets, validate, static_cast<const S *>(scales), zeros,
            static_cast<S *>(q->scales), q->zeros, flag);
    });
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

spmv_status quant_unpack(const spmv_quant *q, spmv_quant_array which, void *dst, hipStream_t s) {
    const int64_t items = static_cast<int64_t>(q->R) * q->groups;
    if (which == SPMV_Q_CODES) {
        const int64_t bytes = static_cast<int64_t>(q->R) * ((static_cast<int64_t>(q->C) + 1) / 2);
        k_quant_unpack<<<groups_for(bytes, kThreads), kThreads, 0, s>>>(
            q->R, q->C, q->blocks, q->codes, static_cast<uint8_t *>(dst));
    } else if (which == SPMV_Q_ZEROS) {
        k_quant_unpack_groups<uint8_t, true><<<groups_for(items, kThreads), kThreads, 0, s>>>(
            q->R, q->groups, q->set, q->sets, q->zeros, static_cast<uint8_t *>(dst));
    } else {
        with_float(q->scale_dtype, [&](auto sc) {
            using S = decltype(sc);
            k_quant_unpack_groups<S, false><<<groups_for(items, kThreads), kThreads, 0, s>>>(
                q->R, q->groups, q->set, q->sets, static_cast<const S *>(q->scales),
                static_cast<S *>(dst));
        });
    }
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

spmv_status quant_lookup(const spmv_quant *q, int64_t n, const void *ids, int32_t id_dtype,
                         float scale, void *out, int64_t ld, int32_t dtype, hipStream_t s) {
    const int L = lanes_for(static_cast<int64_t>(q->blocks) * 4, kThreads);
    const unsigned grid = groups_for(n, kThreads / L);
    with_float(q->scale_dtype, [&](auto sc) {
        with_float(dtype, [&](auto t) {
            using S = decltype(sc);
            using T = decltype(t);
            if (id_dtype == SPMV_INT64)
                k_quant_lookup<S, T, int64_t><<<grid, kThreads, 0, s>>>(
                    q->R, q->C, q->group, q->set, q->sets, q->blocks, L, q->codes,
                    static_cast<const S *>(q->scales), q->zeros, n,
                    static_cast<const int64_t *>(ids), scale, static_cast<T *>(out), ld);
            else
                k_quant_lookup<S, T, int32_t><<<grid, kThreads, 0, s>>>(
                    q->R, q->C, q->group, q->set, q->sets, q->blocks, L, q->codes,
                    static_cast<const S *>(q->scales), q->zeros, n,
                    static_cast<const int32_t *>(ids), scale, static_cast<T *>(out), ld);
        });
    });
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

}  // namespace spmv
