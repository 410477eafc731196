// y <- W x (+ y) with a 4-bit matrix (layout at struct spmv_quant, tables.h):
// the kernel, included by one source per vector type (quant_run_*.hip).
#pragma once

#include "tables.h"

namespace spmv {

struct QuantArgs {
    int32_t R, C, n, blocks, group, groups_pad;
    const uint32_t *codes;
    const void *scales;
    const uint8_t *zeros;
    const void *x;
    int64_t x_ld;
    void *y;
    int64_t y_ld;
    int32_t accumulate;
    int32_t y_fp32;
    int32_t passes;       // groups of vectors
    int32_t group_shift;  // log2 of the group, or -1
};

void quant_run_fp32(const QuantArgs &a, int32_t scale_dtype, hipStream_t s);
void quant_run_fp16(const QuantArgs &a, int32_t scale_dtype, hipStream_t s);
void quant_run_bf16(const QuantArgs &a, int32_t scale_dtype, hipStream_t s);

namespace {

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x8 = bf16 __attribute__((ext_vector_type(8)));
using f16x8 = f16 __attribute__((ext_vector_type(8)));

// How a vector type meets the matrix unit.
//
// 16-bit types: a column of the product is a vector.  A code becomes the float
// 16 + code by placing it in the mantissa's top bits (or'ed into the bits of 16).
// fp32: a vector is three columns, bf16 parts of 8 bits each (the leading bits,
// the next, the rest), which add up to x exactly.
template <typename X>
struct Unit;
template <>
struct Unit<bf16> {
    static constexpr int kParts = 1;
    static constexpr uint32_t kSixteen = 0x41804180u, kMask = 0x00780078u, kStep = 0x00080008u;
    // word bit of code pair i is 4 i + 3 and 4 i + 19 (rotated); bits 3 and 19 are wanted
    static __device__ inline uint32_t pair(uint32_t w, int i) {
        return i == 0 ? w : i == 3 ? __builtin_amdgcn_alignbit(w, w, 12) : w >> (4 * i);
    }
    static __device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Unit<float> : Unit<bf16> {
    static constexpr int kParts = 3;
};
template <>
struct Unit<f16> {
    static constexpr int kParts = 1;
    static constexpr uint32_t kSixteen = 0x4C004C00u, kMask = 0x03C003C0u, kStep = 0x00400040u;
    // bits 6 and 22 are wanted
    static __device__ inline uint32_t pair(uint32_t w, int i) {
        return i == 0 ? w << 3 : i == 3 ? __builtin_amdgcn_alignbit(w, w, 9) : w >> (4 * i - 3);
    }
    static __device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(
            __builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// Eight elements of a vector as they are loaded, and the operands they make.
template <typename X>
struct XOctet {
    u32x4 raw;
    __device__ inline void load(const X *p) { __builtin_memcpy(&raw, p, 16); }
    __device__ inline void load_tail(const X *p, int count) {
        X v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < count ? p[i] : static_cast<X>(0.f);
        __builtin_memcpy(&raw, v, 16);
    }
    __device__ inline void split(u32x4 *part) const { part[0] = raw; }
};
template <>
struct XOctet<float> {
    float v[8];
    __device__ inline void load(const float *p) { load_octet(p, v); }
    __device__ inline void load_tail(const float *p, int count) { load_octet_tail(p, count, v); }
    __device__ inline void split(u32x4 *part) const {
        uint32_t w[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = v[i] - lead(v[i]);
            w[0][i] = __builtin_bit_cast(uint32_t, v[i]);
            w[1][i] = __builtin_bit_cast(uint32_t, r);
            w[2][i] = __builtin_bit_cast(uint32_t, r - lead(r));
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[p][i] = __builtin_amdgcn_perm(w[p][2 * i + 1], w[p][2 * i], 0x07060302);
    }
    static __device__ inline float lead(float f) {
        return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) & 0xffff0000u);
    }
};

// One element of the product, in plain arithmetic.
template <typename X, typename S>
__device__ float plain_dot(const QuantArgs &a, int32_t r, int32_t v) {
    const X *x = static_cast<const X *>(a.x) + v * a.x_ld;
    const int64_t tile = r / kQuantRows;
    float sum = 0.f;
    for (int c = 0; c < a.C; ++c) {
        const int o = c / 8;
        const uint32_t w =
            a.codes[(tile * a.blocks + o / kQuantOctets) * kQuantBlockWords +
                    quant_word(r % kQuantRows, o % kQuantOctets)];
        const int64_t si = (tile * a.groups_pad + c / a.group) * kQuantRows + r % kQuantRows;
        const float s = static_cast<float>(static_cast<const S *>(a.scales)[si]);
        const float z = a.zeros ? static_cast<float>(a.zeros[si]) : 8.f;
        sum = fmaf((static_cast<float>(quant_code(w, c & 7)) - z) * s, static_cast<float>(x[c]),
                   sum);
    }
    return sum;
}

// Four scales as they are loaded (8 or 16 bytes).
template <typename S>
struct alignas(8) ScaleQuad {
    uint32_t raw[2];
    __device__ inline float get(int i) const {
        const uint32_t w = raw[i / 2];
        if constexpr (std::is_same_v<S, bf16>)
            return __builtin_bit_cast(float, i % 2 ? w & 0xffff0000u : w << 16);
        else
            return static_cast<float>(
                __builtin_bit_cast(f16, static_cast<uint16_t>(i % 2 ? w >> 16 : w)));
    }
};
template <>
struct alignas(16) ScaleQuad<float> {
    float raw[4];
    __device__ inline float get(int i) const { return raw[i]; }
};

// What a wave loads for one block of 128 columns: RT tiles' codes, scales and
// zero points, and its share of the vectors.
template <typename X, typename S, int GS, int RT, int NX>
struct Block {
    u32x4 code[RT];
    ScaleQuad<S> scale[RT][128 / GS];
    uint32_t zero[RT][128 / GS];
    XOctet<X> x[NX];
};

// Bytes between the columns of a block's vectors in LDS: 128 elements and a
// gap that spreads eight lanes' 16-byte reads over all banks.
constexpr int kColBytes = 256 + 16;

// A workgroup takes RT tiles of 16 rows and NC columns (vectors, or parts of
// fp32 vectors); its W waves take every W-th block of 128 matrix columns and
// add up at the end.  A wave keeps its block's vectors in its own part of LDS:
// loaded along their length (neighbouring lanes, neighbouring bytes), read as
// matrix operands.  GS: columns per scale, at most 128.  Z: zero points.
template <typename X, typename S, bool Z, int GS, int RT, int NC, int W>
__global__ __launch_bounds__(W *kWave) void k_quant_mfma(QuantArgs a) {
    using U = Unit<X>;
    constexpr int NT = (NC + 15) / 16;
    constexpr int kVecs = NC / U::kParts;       // vectors per pass
    constexpr int NX = (kVecs + 3) / 4;         // octets of them per lane and block
    constexpr int kScales = 128 / GS;           // scales per block and row
    constexpr int kWaveBytes = NT * 16 * kColBytes;
    static_assert(kWaveBytes >= NT * 4 * kWave * 4, "the sums reuse the vectors' part");
    __shared__ __attribute__((aligned(16))) char lds[W * kWaveBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, quad = lane / 16;
    const uint32_t code_lane = quant_word(r16, quad) * 4;
    const uint32_t scale_lane = quad * 4 * sizeof(S);
    char *const mine = lds + wave * kWaveBytes;
    const int64_t row_groups = (static_cast<int64_t>(a.R) + RT * 16 - 1) / (RT * 16);
    const int64_t last_tile = (static_cast<int64_t>(a.R) - 1) / 16;
    uint32_t sixteen = U::kSixteen, mask = U::kMask;
    asm("" : "+v"(sixteen));  // one operand of v_and_or_b32 in a VGPR, the other in an SGPR
    asm("" : "+s"(mask));
    for (int64_t item = blockIdx.x; item < row_groups * a.passes; item += gridDim.x) {
        const int64_t tile0 = (item % row_groups) * RT;
        const int32_t v0 = static_cast<int32_t>(item / row_groups) * kVecs;
        // This lane's share of the vectors.  Slots past the last repeat it: the
        // sums of their columns go nowhere.
        const X *xp[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            int32_t v = i * 4 + quad;
            v = v < kVecs ? v0 + v : v0;
            v = v < a.n ? v : a.n - 1;
            xp[i] = static_cast<const X *>(a.x) + v * a.x_ld + r16 * 8;
        }
        int64_t tile[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) tile[t] = tile0 + t < last_tile ? tile0 + t : last_tile;
        f32x4 y[RT][NT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) y[t][u] = f32x4{0, 0, 0, 0};

        using B = Block<X, S, GS, RT, NX>;
        // uniform address, then this lane's bytes
        auto at = [](const void *p, int64_t bytes, uint32_t lane_bytes) {
            return static_cast<const char *>(p) + bytes + lane_bytes;
        };
        auto load = [&](B &b, int block) {
            const int g0 = GS < 128 ? block * kScales
                           : a.group_shift >= 0 ? block >> (a.group_shift - 7)
                                                : block / (a.group >> 7);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int64_t word = (tile[t] * a.blocks + block) * kQuantBlockWords;
                b.code[t] = *reinterpret_cast<const u32x4 *>(at(a.codes, word * 4, code_lane));
                const int64_t g = (tile[t] * a.groups_pad + g0) * kQuantRows;
#pragma unroll
                for (int i = 0; i < kScales; ++i) {
                    b.scale[t][i] = *reinterpret_cast<const ScaleQuad<S> *>(
                        at(a.scales, (g + i * kQuantRows) * sizeof(S), scale_lane));
                    b.zero[t][i] = 8;
                    if constexpr (Z)
                        b.zero[t][i] = *reinterpret_cast<const uint8_t *>(
                            at(a.zeros, g + i * kQuantRows, r16));
                }
            }
        };
        // The vectors' octets to LDS: octet r16 of vector i * 4 + quad.
        auto stage = [&](const B &b) {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                if (i * 4 + quad >= kVecs) continue;
                u32x4 part[U::kParts];
                b.x[i].split(part);
#pragma unroll
                for (int p = 0; p < U::kParts; ++p)
                    *reinterpret_cast<u32x4 *>(
                        mine + ((i * 4 + quad) * U::kParts + p) * kColBytes + r16 * 16) = part[p];
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        };
        auto compute = [&](const B &s) {
#pragma unroll
            for (int g = 0; g < kScales; ++g) {
                f32x4 acc[RT][NT];
                u32x4 off[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    // -(16 + zero) in both halves
                    const uint32_t o = (s.zero[t][g] * U::kStep) | (U::kSixteen | 0x80008000u);
                    off[t] = u32x4{o, o, o, o};
                }
#pragma unroll
                for (int jj = 0; jj < GS / 32; ++jj) {
                    const int j = g * (GS / 32) + jj;
                    u32x4 b[NT];
#pragma unroll
                    for (int u = 0; u < NT; ++u)
                        b[u] = *reinterpret_cast<const u32x4 *>(
                            mine + (u * 16 + r16) * kColBytes + j * 64 + quad * 16);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        u32x4 q;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[i] = (U::pair(s.code[t][j], i) & mask) | sixteen;
#pragma unroll
                        for (int u = 0; u < NT; ++u) {
                            acc[t][u] = U::mfma(off[t], b[u],
                                                jj == 0 ? f32x4{0, 0, 0, 0} : acc[t][u]);
                            acc[t][u] = U::mfma(q, b[u], acc[t][u]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int u = 0; u < NT; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[t][u][i] = fmaf(s.scale[t][g].get(i), acc[t][u][i], y[t][u][i]);
            }
        };
        const int full = a.C / kQuantCols;  // blocks with all their columns
        const int count = wave < full ? (full - wave + W - 1) / W : 0;
        if (count > 0) {
            // No branch around a load: the last block is loaded again instead.
            B cur, nxt;
            int block = wave;
            load(cur, block);
#pragma unroll
            for (int i = 0; i < NX; ++i) cur.x[i].load(xp[i] + block * kQuantCols);
#pragma unroll 1
            for (int i = 1; i <= count; ++i) {
                stage(cur);
                block += i < count ? W : 0;
                load(nxt, block);
#pragma unroll
                for (int u = 0; u < NX; ++u) nxt.x[u].load(xp[u] + block * kQuantCols);
                __builtin_amdgcn_sched_barrier(0);
                compute(cur);
                cur = nxt;
            }
        }
        if (a.C % kQuantCols && full % W == wave) {
            int left = a.C - full * kQuantCols - r16 * 8;
            asm volatile("" : "+v"(left));  // keeps the tail's comparisons out of the item loop
            B b;
            load(b, full);
#pragma unroll
            for (int i = 0; i < NX; ++i) b.x[i].load_tail(xp[i] + full * kQuantCols, left);
            stage(b);
            compute(b);
        }

        // a row tile at a time: the waves' parts, then each element's sum
        auto part = [&](int w, int u, int i, int l) -> float & {
            return reinterpret_cast<float *>(lds + w * kWaveBytes)[(u * 4 + i) * kWave + l];
        };
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) part(wave, u, i, lane) = y[t][u][i];
            __syncthreads();
            for (int e = threadIdx.x; e < kVecs * 16; e += W * kWave) {
                const int row = e % 16, v = e / 16;
                const int64_t r = (tile0 + t) * 16 + row;
                if (r >= a.R || v0 + v >= a.n) continue;
                float sum = 0.f;
#pragma unroll
                for (int p = U::kParts - 1; p >= 0; --p) {
                    const int c = v * U::kParts + p;
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        s += part(w, c / 16, row % 4, (row / 4) * 16 + c % 16);
                    sum += s;
                }
                // Infinities among the moved codes' products cancel to NaN, and moved codes may
                // pass the range where the codes do not: such an element is computed plainly.
                if (!(fabsf(sum) <= 3.402823466e38f))
                    sum = plain_dot<X, S>(a, static_cast<int32_t>(r), v0 + v);
                const int64_t to = (v0 + v) * a.y_ld + r;
                if (a.y_fp32) {
                    float *p = static_cast<float *>(a.y) + to;
                    *p = a.accumulate ? sum + *p : sum;
                } else {
                    X *p = static_cast<X *>(a.y) + to;
                    *p = static_cast<X>(a.accumulate ? sum + static_cast<float>(*p) : sum);
                }
            }
        }
        __syncthreads();  // the next item's vectors overwrite the parts
    }
}

template <typename X, typename S, bool Z, int GS, int RT, int NC, int W>
void launch(QuantArgs a, hipStream_t s) {
    constexpr int kVecs = NC / Unit<X>::kParts;
    a.passes = a.n / kVecs + (a.n % kVecs != 0);
    const int64_t row_groups = (static_cast<int64_t>(a.R) + RT * 16 - 1) / (RT * 16);
    k_quant_mfma<X, S, Z, GS, RT, NC, W>
        <<<groups_for(row_groups * a.passes, 1), W * kWave, 0, s>>>(a);
}

// The kernel's shape by the number of vectors and of row tiles.
template <typename X, typename S, bool Z, int GS>
void launch_shape(const QuantArgs &a, hipStream_t s) {
    constexpr int P = Unit<X>::kParts;
    const int64_t passes = (static_cast<int64_t>(a.n) * P + 47) / 48;
    const int64_t cols = ((a.n + passes - 1) / passes) * P;
    const bool tall = a.R > 16 * 1024;
    if (cols <= 4) {
        if (tall)
            launch<X, S, Z, GS, 2, 4, 4>(a, s);
        else
            launch<X, S, Z, GS, 1, 4, 8>(a, s);
    } else if (cols <= 15 || (cols == 16 && P == 1)) {
        if (tall)
            launch<X, S, Z, GS, 2, 16, 4>(a, s);
        else
            launch<X, S, Z, GS, 1, 16, 8>(a, s);
    } else if (cols <= 32 && P == 1) {
        launch<X, S, Z, GS, 2, 32, 8>(a, s);
    } else {
        launch<X, S, Z, GS, 2, 48, 8>(a, s);
    }
}

template <typename X>
void launch_product(const QuantArgs &a, int32_t scale_dtype, hipStream_t s) {
    with_float(scale_dtype, [&](auto sc) {
        using S = decltype(sc);
        auto zeros = [&](auto gs) {
            constexpr int GS = decltype(gs)::value;
            if (a.zeros)
                launch_shape<X, S, true, GS>(a, s);
            else
                launch_shape<X, S, false, GS>(a, s);
        };
        if (a.group == 32)
            zeros(std::integral_constant<int, 32>{});
        else if (a.group == 64)
            zeros(std::integral_constant<int, 64>{});
        else
            zeros(std::integral_constant<int, 128>{});
    });
}

}  // namespace
}  // namespace spmv
