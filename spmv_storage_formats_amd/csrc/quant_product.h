// y <- W x (+ y) with a 4-bit matrix (layout at struct spmv_quant, tables.h):
// the kernels, included by one source per vector type (quant_run_*.hip).
//
// With q the codes, s and z the scale and zero point of row r and group g,
//   y[v, r] = sum_g s[r, g] * sum_{c in g} (q[r, c] - z[r, g]) * x[v, c]
//           = sum_g s[r, g] * (sum_c (16 + q[r, c]) x[v, c] - sum_c (16 + z[r, g]) x[v, c]).
// 16 + code is a float whose mantissa holds the code, so codes become operands
// of the matrix unit by a shift, a mask and an or for two; the second sum is a
// second matrix product, with an operand that is constant along the columns.
// Both are exact products summed in fp32; scaling is in fp32 as well.
#pragma once

#include "tables.h"

namespace spmv {

struct QuantArgs {
    int32_t R, C, n, blocks, group, set, sets;
    const uint32_t *codes;
    const void *scales;
    const uint8_t *zeros;
    const void *x;
    int64_t x_ld;
    void *y;
    int64_t y_ld;
    int32_t accumulate;
    int32_t y_fp32;
    int32_t passes;       // groups of vectors (wide products)
    int32_t splits;       // parts of the columns, each a workgroup's (wide products)
    float *partial;       // their sums [splits][n][R], where there are several
    int32_t group_shift;  // log2 of the group, or -1
};

// Matrix-unit columns of one pass over n vectors of `parts` columns each: at
// most kMostPass, the passes even.
inline int64_t wide_columns(int32_t n, int parts) {
    const int64_t vecs = kMostPass / parts;
    const int64_t passes = (n + vecs - 1) / vecs;
    return (n + passes - 1) / passes * parts;
}

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
// the next, the rest), which add up to x exactly.  The second and third are
// kept times 2^16, so that they are bf16 numbers for the smallest x, too.
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
    static constexpr float kUp = 65536.f;
    static __device__ inline float join(float lead, float next, float rest) {
        return fmaf(next + rest, 1 / kUp, lead);
    }
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
    __device__ inline void load(const float *p) { load_piece<8>(p, v); }
    __device__ inline void load_tail(const float *p, int count) { load_piece_tail<8>(p, count, v); }
    __device__ inline void split(u32x4 *part) const {
        uint32_t w[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = (v[i] - lead(v[i])) * Unit<float>::kUp;
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

// One element of the product, in plain arithmetic, an octet of codes at a time
// (groups are whole octets).
template <typename X, typename S>
__device__ float plain_dot(const QuantArgs &a, int32_t r, int32_t v) {
    const X *x = static_cast<const X *>(a.x) + v * a.x_ld;
    const uint32_t *codes =
        a.codes + static_cast<int64_t>(r / kQuantRows) * a.blocks * kQuantBlockWords;
    float sum = 0.f;
    for (int c = 0; c < a.C; c += 8) {
        const int o = c / 8;
        const uint32_t w = codes[static_cast<int64_t>(o / kQuantOctets) * kQuantBlockWords +
                                 quant_word(r % kQuantRows, o % kQuantOctets)];
        const int32_t g = c / a.group;
        const float s = static_cast<float>(
            static_cast<const S *>(a.scales)[quant_scale_at(r, g, a.set, a.sets)]);
        const float z =
            a.zeros ? static_cast<float>(a.zeros[quant_zero_at(r, g, a.set, a.sets)]) : 8.f;
        float xs[8];
        if (c + 8 <= a.C)
            load_piece<8>(x + c, xs);
        else
            load_piece_tail<8>(x + c, a.C - c, xs);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.C)
                sum = fmaf((static_cast<float>(quant_code(w, e)) - z) * s, xs[e], sum);
    }
    return sum;
}

// The scales of four rows and N groups as they are loaded.
template <typename S, int N>
struct alignas(N == 1 ? 8 : 16) Scales {
    uint32_t raw[2 * N];
    __device__ inline float get(int g, int i) const {
        const uint32_t w = raw[2 * g + i / 2];
        if constexpr (std::is_same_v<S, bf16>)
            return __builtin_bit_cast(float, i % 2 ? w & 0xffff0000u : w << 16);
        else
            return static_cast<float>(
                __builtin_bit_cast(f16, static_cast<uint16_t>(i % 2 ? w >> 16 : w)));
    }
};
template <int N>
struct alignas(16) Scales<float, N> {
    float raw[4 * N];
    __device__ inline float get(int g, int i) const { return raw[4 * g + i]; }
};

// The zero points of one row and N groups: bytes, loaded whole.
template <int N>
__device__ inline uint32_t load_zeros(const char *p) {
    if constexpr (N == 4) return *reinterpret_cast<const uint32_t *>(p);
    if constexpr (N == 2) return *reinterpret_cast<const uint16_t *>(p);
    return *reinterpret_cast<const uint8_t *>(p);
}

// What a wave loads for one block of 128 columns: RT tiles' codes, scales and
// zero points, and its share of the vectors.
template <typename X, typename S, int GS, int RT, int NX>
struct Block {
    u32x4 code[RT];
    Scales<S, 128 / GS> scale[RT];
    uint32_t zero[RT];
    XOctet<X> x[NX];
};

// Bytes between the columns of a block's vectors in LDS: 128 elements and a
// gap that spreads eight lanes' 16-byte reads over all banks.
constexpr int kColBytes = 256 + 16;

// What both kernels below do with a block, a lane at a time.
template <typename X, typename S, bool Z, int GS>
struct Lane {
    using U = Unit<X>;
    static constexpr int kScales = 128 / GS;  // scales per block and row
    int r16, quad;
    uint32_t code_at, scale_at, zero_at;  // this lane's bytes in a block's data
    uint32_t sixteen = U::kSixteen, mask = U::kMask;

    __device__ inline explicit Lane(int lane) : r16(lane % 16), quad(lane / 16) {
        code_at = quant_word(r16, quad) * 4;
        scale_at = quad * 4 * kScales * sizeof(S);
        zero_at = r16 * kScales;
        asm("" : "+v"(sixteen));  // one operand of v_and_or_b32 in a VGPR, the other in an SGPR
        asm("" : "+s"(mask));
    }

    // Codes, scales and zero points of RT tiles: a uniform address, then the lane's bytes.
    template <int RT, int NX>
    __device__ inline void load(const QuantArgs &a, const int64_t *tile, int block,
                                Block<X, S, GS, RT, NX> &b) const {
        const int set = GS < 128 ? block
                        : a.group_shift >= 0 ? block >> (a.group_shift - 7)
                                             : block / (a.group >> 7);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const char *codes = reinterpret_cast<const char *>(
                a.codes + (tile[t] * a.blocks + block) * kQuantBlockWords);
            b.code[t] = *reinterpret_cast<const u32x4 *>(codes + code_at);
            const int64_t s = (tile[t] * a.sets + set) * (kQuantRows * kScales);
            const char *scales = static_cast<const char *>(a.scales) + s * sizeof(S);
            b.scale[t] = *reinterpret_cast<const Scales<S, kScales> *>(scales + scale_at);
            b.zero[t] = 0x08080808u;
            if constexpr (Z)
                b.zero[t] =
                    load_zeros<kScales>(reinterpret_cast<const char *>(a.zeros + s) + zero_at);
        }
    }

    // y += the block's matrix times the vectors that lie in LDS at x.
    template <int RT, int NX, int NT>
    __device__ inline void multiply(const Block<X, S, GS, RT, NX> &s, const char *x,
                                    f32x4 (&y)[RT][NT]) const {
#pragma unroll
        for (int g = 0; g < kScales; ++g) {
            f32x4 acc[RT][NT];
            u32x4 off[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                // -(16 + zero) in both halves
                const uint32_t z = (s.zero[t] >> (8 * g)) & 15u;
                const uint32_t o = (z * U::kStep) | (U::kSixteen | 0x80008000u);
                off[t] = u32x4{o, o, o, o};
            }
#pragma unroll
            for (int jj = 0; jj < GS / 32; ++jj) {
                const int j = g * (GS / 32) + jj;
                u32x4 b[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u)
                    b[u] = *reinterpret_cast<const u32x4 *>(x + (u * 16 + r16) * kColBytes +
                                                            j * 64 + quad * 16);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    u32x4 q;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[i] = (U::pair(s.code[t][j], i) & mask) | sixteen;
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
                        acc[t][u] =
                            U::mfma(off[t], b[u], jj == 0 ? f32x4{0, 0, 0, 0} : acc[t][u]);
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
                        y[t][u][i] = fmaf(s.scale[t].get(g, i), acc[t][u][i], y[t][u][i]);
        }
    }
};

// The product's element (r, v) to memory.  Infinities among the moved codes'
// products cancel to NaN, and moved codes (and the lower parts of fp32 vectors)
// may pass the range where the codes do not: such an element is computed plainly.
template <typename X, typename S>
__device__ inline void put_element(const QuantArgs &a, int64_t r, int32_t v, float sum) {
    if (!(fabsf(sum) <= 3.402823466e38f)) sum = plain_dot<X, S>(a, static_cast<int32_t>(r), v);
    const int64_t to = v * a.y_ld + r;
    if (a.y_fp32) {
        float *p = static_cast<float *>(a.y) + to;
        *p = a.accumulate ? sum + *p : sum;
    } else {
        X *p = static_cast<X *>(a.y) + to;
        *p = static_cast<X>(a.accumulate ? sum + static_cast<float>(*p) : sum);
    }
}

// Elements (r .. r+3, v), as one access where they are finite and inside.
template <typename X, typename S>
__device__ inline void put_four(const QuantArgs &a, int64_t r, int32_t v, f32x4 sum) {
    const f32x4 size = __builtin_elementwise_abs(sum);
    const float most = fmaxf(fmaxf(size[0], size[1]), fmaxf(size[2], size[3]));
    // a NaN is no maximum, but makes the sum of all four one
    const bool plain = !(most <= 3.402823466e38f) || sum[0] + sum[1] + sum[2] + sum[3] !=
                                                         sum[0] + sum[1] + sum[2] + sum[3];
    if (plain || r + 4 > a.R) {
        for (int i = 0; i < 4 && r + i < a.R; ++i) put_element<X, S>(a, r + i, v, sum[i]);
        return;
    }
    auto put = [&](auto *p) {
        using Y = std::remove_pointer_t<decltype(p)>;
        struct alignas(sizeof(Y)) Four {
            Y v[4];
        } f;
        if (a.accumulate) {
            __builtin_memcpy(&f, p, sizeof(f));
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] += static_cast<float>(f.v[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f.v[i] = static_cast<Y>(sum[i]);
        __builtin_memcpy(p, &f, sizeof(f));
    };
    const int64_t to = v * a.y_ld + r;
    if (a.y_fp32)
        put(static_cast<float *>(a.y) + to);
    else
        put(static_cast<X *>(a.y) + to);
}

// A workgroup takes RT tiles of 16 rows and NC columns (vectors, or parts of
// fp32 vectors); its W waves take every W-th block of 128 matrix columns and
// add up at the end.  A wave keeps its block's vectors in its own part of LDS:
// loaded along their length (neighbouring lanes, neighbouring bytes), read as
// matrix operands.  GS: columns per scale, at most 128.  Z: zero points.
// Bound by memory where the matrix is large: 128000 x 4096, one bf16 vector, 271
// MB in 45 us, 6.0 TB/s (vector instructions busy 24 us of that, the matrix unit,
// 16 columns wide, 12).  Smaller ones have too few bytes in flight for the time
// that a load takes: 12288 x 8192, 16 vectors, 56 MB in 22 us (14 where the
// last-level cache holds the matrix), half of its waves' time waiting; 4096 x
// 4096, one vector, four blocks per wave one after another, 5.4 us, 72 %.
template <typename X, typename S, bool Z, int GS, int RT, int NC, int W>
__global__ __launch_bounds__(W *kWave) void k_quant_mfma(QuantArgs a) {
    using U = Unit<X>;
    constexpr int NT = (NC + 15) / 16;
    constexpr int kVecs = NC / U::kParts;       // vectors, at most: a.n <= kVecs
    constexpr int NX = (kVecs + 3) / 4;         // octets of them per lane and block
    constexpr int kWaveBytes = NT * 16 * kColBytes;
    static_assert(kWaveBytes >= RT * NT * 4 * kWave * 4, "the sums reuse the vectors' part");
    __shared__ __attribute__((aligned(16))) char lds[W * kWaveBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Lane<X, S, Z, GS> me(lane);
    const int r16 = me.r16, quad = me.quad;
    char *const mine = lds + wave * kWaveBytes;
    const int32_t tiles = (a.R - 1) / 16 + 1;
    const int32_t tile0 = static_cast<int32_t>(blockIdx.x) * RT;
    // This lane's share of the vectors.  Slots past the last repeat it: the
    // sums of their columns go nowhere.
    const X *xp[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        int32_t v = i * 4 + quad;
        v = v < kVecs && v < a.n ? v : a.n - 1;
        xp[i] = static_cast<const X *>(a.x) + v * a.x_ld + r16 * 8;
    }
    int64_t tile[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) tile[t] = tile0 + t < tiles ? tile0 + t : tiles - 1;
    f32x4 y[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) y[t][u] = f32x4{0, 0, 0, 0};

    using B = Block<X, S, GS, RT, NX>;
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
    const int full = a.C / kQuantCols;  // blocks with all their columns
    const int count = wave < full ? (full - wave + W - 1) / W : 0;
    if (count > 0) {
        // No branch around a load: the last block is loaded again instead.
        B cur, nxt;
        int block = wave;
        me.load(a, tile, block, cur);
#pragma unroll
        for (int i = 0; i < NX; ++i) cur.x[i].load(xp[i] + block * kQuantCols);
#pragma unroll 1
        for (int i = 1; i <= count; ++i) {
            stage(cur);
            block += i < count ? W : 0;
            me.load(a, tile, block, nxt);
#pragma unroll
            for (int u = 0; u < NX; ++u) nxt.x[u].load(xp[u] + block * kQuantCols);
            __builtin_amdgcn_sched_barrier(0);
            me.multiply(cur, mine, y);
            cur = nxt;
        }
    }
    if (a.C % kQuantCols && full % W == wave) {
        int left = a.C - full * kQuantCols - r16 * 8;
        asm volatile("" : "+v"(left));  // keeps the tail's comparisons out of the item loop
        B b;
        me.load(a, tile, full, b);
#pragma unroll
        for (int i = 0; i < NX; ++i) b.x[i].load_tail(xp[i] + full * kQuantCols, left);
        stage(b);
        me.multiply(b, mine, y);
    }

    // the waves' parts, then each element's sum
    auto part = [&](int w, int t, int u, int i, int l) -> float & {
        return reinterpret_cast<float *>(lds + w * kWaveBytes)[((t * NT + u) * 4 + i) * kWave +
                                                               l];
    };
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) part(wave, t, u, i, lane) = y[t][u][i];
    __syncthreads();
    for (int e = threadIdx.x; e < kVecs * RT * 16; e += W * kWave) {
        const int row = e % (RT * 16), v = e / (RT * 16);
        const int64_t r = static_cast<int64_t>(tile0) * 16 + row;
        if (r >= a.R || v >= a.n) continue;
        float sum[U::kParts] = {};
#pragma unroll
        for (int p = 0; p < U::kParts; ++p) {
            const int c = v * U::kParts + p;
#pragma unroll
            for (int w = 0; w < W; ++w)
                sum[p] += part(w, row / 16, c / 16, row % 4, (row % 16 / 4) * 16 + c % 16);
        }
        if constexpr (U::kParts == 3) sum[0] = U::join(sum[0], sum[1], sum[2]);
        put_element<X, S>(a, r, v, sum[0]);
    }
}

// Many columns: a workgroup's waves take RT tiles of rows each and share the
// block's vectors, which all threads bring to LDS (two buffers, one barrier per
// block): a vector is read once per kWideRows rows instead of once per 16 RT.
// Where that leaves too few workgroups, the matrix's columns are split among
// `splits` of them, whose sums meet in the workspace.  8192 x 11000, 48 bf16
// vectors: 26 us and 5 for the join, of which vector instructions are busy 8 and the
// matrix unit 7, so bound by neither: waves wait 38 % of their time for loads and at
// the block's barrier, and two waves per SIMD hide little (three passes of 16
// through the kernel above: 34 us; 32 vectors 20 + 5 against 25).  Two to four
// blocks of loads ahead in registers measured 24 to 26 us.
// Waves x tiles, 48, 32 and 96 vectors, without the join: 4 x 2 24.3, 19.5 and 38.8
// us; 8 x 1 24.0, 18.4, 42.0; 8 x 2 24.8, 18.9, 43.7; 4 x 4 27.0, 21.7, 48.7; 8 x 4
// 36.8, 27.6, 40.9.
constexpr int kWideWaves = 4;
constexpr int kWideTiles = 2;
constexpr int kWideRows = kWideWaves * kWideTiles * 16;

template <typename X, typename S, bool Z, int GS, int NT>
__global__ __launch_bounds__(kWideWaves *kWave) void k_quant_wide(QuantArgs a) {
    using U = Unit<X>;
    constexpr int RT = kWideTiles;
    constexpr int kVecs = NT * 16 / U::kParts;
    constexpr int NX = kVecs / 16;  // octets of the vectors per thread and block
    constexpr int kBufBytes = NT * 16 * kColBytes;
    static_assert(U::kParts == 1 || U::kParts == NT, "part p of a vector is column p * 16 + v");
    static_assert(kVecs <= kMostPass, "v0 + kVecs, for any n, is an int32");
    __shared__ __attribute__((aligned(16))) char lds[2 * kBufBytes];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Lane<X, S, Z, GS> me(lane);
    const int octet = threadIdx.x % 16, slot = threadIdx.x / 16;
    const int32_t tiles = (a.R - 1) / 16 + 1;
    const int full = a.C / kQuantCols;  // blocks with all their columns
    const int32_t split = blockIdx.y;
    for (int32_t pass = blockIdx.z; pass < a.passes; pass += gridDim.z) {
        const int32_t tile0 = static_cast<int32_t>(blockIdx.x) * (kWideRows / 16) + wave * RT;
        const int32_t v0 = pass * kVecs;
        const int begin = static_cast<int>(static_cast<int64_t>(a.blocks) * split / a.splits);
        const int end = static_cast<int>(static_cast<int64_t>(a.blocks) * (split + 1) / a.splits);
        const X *xp[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            int32_t v = v0 + i * 16 + slot;
            v = v < a.n ? v : a.n - 1;
            xp[i] = static_cast<const X *>(a.x) + v * a.x_ld + octet * 8;
        }
        int64_t tile[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) tile[t] = tile0 + t < tiles ? tile0 + t : tiles - 1;
        f32x4 y[RT][NT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) y[t][u] = f32x4{0, 0, 0, 0};

        using B = Block<X, S, GS, RT, NX>;
        auto stage = [&](const B &b, char *to) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                u32x4 part[U::kParts];
                b.x[i].split(part);
#pragma unroll
                for (int p = 0; p < U::kParts; ++p)
                    *reinterpret_cast<u32x4 *>(to + ((i + p) * 16 + slot) * kColBytes +
                                               octet * 16) = part[p];
            }
        };
        // Two buffers and one barrier per block: whoever writes a buffer again
        // has passed the barrier behind which nobody reads it any more.
        int turn = 0;
        const int whole = end < full ? end : full;
        if (begin < whole) {
            B cur, nxt;
            me.load(a, tile, begin, cur);
#pragma unroll
            for (int i = 0; i < NX; ++i) cur.x[i].load(xp[i] + begin * kQuantCols);
#pragma unroll 1
            for (int block = begin; block < whole; ++block) {
                char *buf = lds + turn * kBufBytes;
                stage(cur, buf);
                // no branch around a load: the last block is loaded again instead
                const int next = block + 1 < whole ? block + 1 : block;
                me.load(a, tile, next, nxt);
#pragma unroll
                for (int i = 0; i < NX; ++i) nxt.x[i].load(xp[i] + next * kQuantCols);
                __syncthreads();
                me.multiply(cur, buf, y);
                cur = nxt;
                turn ^= 1;
            }
        }
        if (whole < end) {  // the block with the last columns
            int left = a.C - full * kQuantCols - octet * 8;
            asm volatile("" : "+v"(left));  // keeps the tail's comparisons out of the item loop
            B b;
            me.load(a, tile, full, b);
#pragma unroll
            for (int i = 0; i < NX; ++i) b.x[i].load_tail(xp[i] + full * kQuantCols, left);
            char *buf = lds + turn * kBufBytes;
            stage(b, buf);
            __syncthreads();
            me.multiply(b, buf, y);
        }

        // A lane holds four neighbouring rows of one column; fp32: the parts of
        // one vector in its NT tiles.
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int64_t r = (static_cast<int64_t>(tile0) + t) * 16 + me.quad * 4;
#pragma unroll
            for (int u = 0; u < NT / U::kParts; ++u) {
                f32x4 sum = y[t][u];
                if constexpr (U::kParts == 3)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum[i] = U::join(y[t][0][i], y[t][1][i], y[t][2][i]);
                const int32_t v = v0 + u * 16 + me.r16;
                if (v >= a.n) continue;
                if (a.splits > 1) {
                    float *p = a.partial + (static_cast<int64_t>(split) * a.n + v) * a.R + r;
                    if (r + 4 <= a.R)
                        __builtin_memcpy(p, &sum, 16);
                    else
                        for (int i = 0; r + i < a.R; ++i) p[i] = sum[i];
                } else {
                    put_four<X, S>(a, r, v, sum);
                }
            }
        }
        __syncthreads();  // the next pass's vectors overwrite the last block's
    }
}

// The splits' sums in order.
template <typename X, typename S>
__global__ __launch_bounds__(256) void k_quant_join(QuantArgs a) {
    const int64_t all = static_cast<int64_t>(a.n) * a.R;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        float sum = 0.f;
        for (int s = 0; s < a.splits; ++s) sum += a.partial[s * all + i];
        put_element<X, S>(a, i % a.R, static_cast<int32_t>(i / a.R), sum);
    }
}

template <typename X, typename S, bool Z, int GS, int NT>
void launch_wide(QuantArgs a, hipStream_t s) {
    constexpr int kVecs = NT * 16 / Unit<X>::kParts;
    a.passes = a.n / kVecs + (a.n % kVecs != 0);
    const dim3 grid(grid_for(a.R, kWideRows), a.splits, std::min(a.passes, 65535));
    k_quant_wide<X, S, Z, GS, NT><<<grid, kWideWaves * kWave, 0, s>>>(a);
    if (a.splits > 1)
        k_quant_join<X, S><<<groups_for(static_cast<int64_t>(a.n) * a.R, 256), 256, 0, s>>>(a);
}

template <typename X, typename S, bool Z, int GS, int RT, int NC, int W>
void launch(const QuantArgs &a, hipStream_t s) {
    k_quant_mfma<X, S, Z, GS, RT, NC, W><<<grid_for(a.R, RT * 16), W * kWave, 0, s>>>(a);
}

// The kernel and its shape by the number of columns and of rows.  Two tiles per
// workgroup halve what is read of the vectors, one tile makes twice the
// workgroups, of which each of the 256 CUs wants one or more: up to 4096 rows
// one tile and eight waves, up to 8192 two tiles and eight waves (one workgroup
// per CU), up to 16384 one tile and four waves, beyond that two and four.
// us per call in a captured graph, from memory (tiles x waves):
//                               1 x 8  2 x 8  1 x 4  2 x 4
//   4096 x 4096   bf16,  1        5.2    5.5    7.0    7.3   vector
//                 fp16, 16        6.4    7.7    7.9    8.8
//                 fp32,  3        7.3    9.5    9.8   10.9
//   5001 x 2750   fp16, 16        9.0    8.0    8.0    8.5
//                 fp32,  3        9.4    8.8    9.5    9.9
//   8192 x 8192   bf16,  1        9.8    9.5   12.8   13.0
//                 fp16, 16       16.7   12.9   14.8   15.1
//                 fp32,  3       19.2   16.3   20.0   19.5
//   11008 x 4096  bf16,  1        7.8    8.2    9.2    8.7
//                 fp16, 16       13.3   14.0   11.7   11.7
//                 fp32,  3       15.7   17.1   15.0   15.8
//   12288 x 8192  bf16,  1       13.0   13.8   16.6   15.5
//                 fp16, 16       23.3   22.4   21.3   20.5
//                 fp32,  3       27.6   28.5   26.8   27.8
//   14336 x 5120  bf16,  1       11.8   10.4   11.6   12.1
//                 fp16, 16       21.0   18.3   20.4   16.5
//                 fp32,  3       23.2   21.0   23.1   19.9
//   16384 x 4096  bf16,  1       10.4    9.3   10.1   10.0
//                 fp16, 16       17.3   15.8   16.6   13.3
//                 fp32,  3       20.7   18.8   19.9   17.4
//   28672 x 8192  bf16,  1       27.3   27.1   28.4   25.7
//                 fp16, 16       49.8   43.6   51.4   42.4
//                 fp32,  3       59.5   55.9   56.7   53.8
// (bf16 without zero points, groups of 128; fp16 and fp32 with, of 64 and 32.)  The
// rule is the best of the four, or within 4 % of it, up to 8192 rows and from 16385
// on, in all types.  Between, no shape is best throughout: one tile and four waves are
// for several vectors up to 12288 rows (within 5 % of the best) and for matrices that
// the last-level cache holds (12288 x 8192, one vector 13.2 against 15.2 with two
// tiles); from there to 16384 rows two tiles are up to a quarter faster.
template <typename X, typename S, bool Z, int GS, int NC>
void launch_narrow(const QuantArgs &a, hipStream_t s) {
    if (a.R <= 16 * 256)
        launch<X, S, Z, GS, 1, NC, 8>(a, s);
    else if (a.R <= 16 * 512)
        launch<X, S, Z, GS, 2, NC, 8>(a, s);
    else if (a.R <= 16 * 1024)
        launch<X, S, Z, GS, 1, NC, 4>(a, s);
    else
        launch<X, S, Z, GS, 2, NC, 4>(a, s);
}

template <typename X, typename S, bool Z, int GS>
void launch_shape(const QuantArgs &a, hipStream_t s) {
    constexpr int P = Unit<X>::kParts;
    // 16 or fewer are those of one pass: where there are several, each has 25 at least
    const int64_t cols = wide_columns(a.n, P);
    if (cols <= 4) return launch_narrow<X, S, Z, GS, 4>(a, s);
    if (cols <= 16) return launch_narrow<X, S, Z, GS, 16>(a, s);
    if constexpr (P == 1)
        if (cols <= 32) return launch_wide<X, S, Z, GS, 2>(a, s);
    launch_wide<X, S, Z, GS, 3>(a, s);
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
