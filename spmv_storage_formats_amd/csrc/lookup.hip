// Rows of a dense table by token, and the gradient of that lookup by sorted
// tokens.
//
//   out[t, :]    = scale * table[ids[t], :]
//   dtable[v, :] = scale * sum over t with ids[t] = v of grad[t, :]
//
// The gradient is the product of the transposed selection matrix with the
// rows of grad.  The tokens are sorted as the COO -> CSR builder sorts row
// indices (stable radix sort), so that the tokens of one row are neighbours
// in their own order; the sorted list is cut into chunks of equal length
// whatever its rows, as a segmented sum, and the parts of a row that chunk
// borders cut are joined in order afterwards.  No atomics: the sums are the
// same from run to run.
#include "tables.h"

namespace spmv {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- lookup

// L lanes per row, an octet each per step.
template <typename A, typename B, typename I>
__global__ __launch_bounds__(kThreads) void k_lookup(int32_t V, int32_t D, int L,
                                                     const A *__restrict__ table,
                                                     int64_t table_ld, int64_t n,
                                                     const I *__restrict__ ids, float scale,
                                                     B *__restrict__ out, int64_t out_ld) {
    const int rows = kThreads / L;
    const int octets = D / 8 + (D % 8 != 0);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / L; t < n;
         t += static_cast<int64_t>(gridDim.x) * rows) {
        const int64_t id = ids[t];
        const bool there = id >= 0 && id < V;
        const A *src = table + (there ? id : 0) * table_ld;
        B *dst = out + t * out_ld;
        for (int o = threadIdx.x % L; o < octets; o += L) {
            const int left = D - o * 8;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
            if (there) {
                if (left >= 8)
                    load_octet(src + o * 8, v);
                else
                    load_octet_tail(src + o * 8, left, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= scale;
            }
            if (left >= 8)
                store_octet(dst + o * 8, v);
            else
                store_octet_tail(dst + o * 8, left, v);
        }
    }
}

// ----------------------------------------------------------- sorting tokens

// Tiles of kSortTile tokens, a workgroup each; digits of at most kSortBits.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortSteps = 4;
constexpr int kSortTile = kSortThreads * kSortSteps;
constexpr int kSortBits = 10;
constexpr int kSortDigits = 1 << kSortBits;

// A token's key: its row, or V where it names none (those sort behind all rows).
template <typename I>
__device__ inline uint32_t token_key(const I *ids, int64_t t, int32_t V) {
    const int64_t id = ids[t];
    return id >= 0 && id < V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(V);
}

// Digit counts of every tile, counts[tile][digit].
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const I *__restrict__ ids, int32_t V,
                                                             const uint32_t *__restrict__ keys,
                                                             int64_t n, int shift, int bits,
                                                             int32_t *__restrict__ counts) {
    __shared__ int h[kSortDigits];
    const int digits = 1 << bits;
    if (static_cast<int>(threadIdx.x) < digits) h[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int64_t i =
            static_cast<int64_t>(blockIdx.x) * kSortTile + j * kSortThreads + threadIdx.x;
        if (i < n) {
            const uint32_t k = keys ? keys[i] : token_key(ids, i, V);
            atomicAdd(&h[(k >> shift) & (digits - 1)], 1);
        }
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < digits)
        counts[static_cast<int64_t>(blockIdx.x) * digits + threadIdx.x] = h[threadIdx.x];
}

// Exclusive prefix of v over the workgroup's threads.
__device__ inline int sort_exclusive(int v, int *wsum) {
    const int lane = __lane_id(), w = threadIdx.x / kWave;
    int incl = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == kWave - 1) wsum[w] = incl;
    __syncthreads();
    int pre = 0;
    for (int i = 0; i < w; ++i) pre += wsum[i];
    __syncthreads();
    return pre + incl - v;
}

struct SortShared {
    int wrun[kSortWaves][kSortDigits];
    int start[kSortDigits];
    uint32_t key[kSortTile];
    uint32_t pos[kSortTile];
    int wsum[kSortWaves];
};

// One stable pass over the tile by bits [shift, shift + bits): thread-order
// entries (key, pos)[j] at tile position (wave, j, lane) move to s.key / s.pos
// by digit; s.start[d] is digit d's first place.  Ends behind a barrier.
__device__ inline void sort_tile(SortShared &s, const uint32_t *key, const uint32_t *pos,
                                 int count, int shift, int bits) {
    const int lane = __lane_id(), w = threadIdx.x / kWave, tid = threadIdx.x;
    const int digits = 1 << bits;
    for (int i = tid; i < kSortWaves * digits; i += kSortThreads)
        s.wrun[i >> bits][i & (digits - 1)] = 0;
    __syncthreads();
    const unsigned long long below = (1ull << lane) - 1ull;
    int rank[kSortSteps];
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const bool valid = (w * kSortSteps + j) * kWave + lane < count;
        const int d = (key[j] >> shift) & (digits - 1);
        unsigned long long peers = __ballot(valid);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (d >> b) & 1;
            const unsigned long long m = __ballot(bit);
            peers &= bit ? m : ~m;
        }
        const int r = __popcll(peers & below);
        const int before = valid ? s.wrun[w][d] : 0;
        rank[j] = before + r;
        if (valid && r == 0) s.wrun[w][d] = before + __popcll(peers);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    int total = 0;
    if (tid < digits) {
#pragma unroll
        for (int i = 0; i < kSortWaves; ++i) {
            const int c = s.wrun[i][tid];
            s.wrun[i][tid] = total;
            total += c;
        }
    }
    const int first = sort_exclusive(total, s.wsum);
    if (tid < digits) s.start[tid] = first;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        if ((w * kSortSteps + j) * kWave + lane < count) {
            const int d = (key[j] >> shift) & (digits - 1);
            const int p = s.start[d] + s.wrun[w][d] + rank[j];
            s.key[p] = key[j];
            s.pos[p] = pos[j];
        }
    }
    __syncthreads();
}

// All passes of at most kSortTile tokens in one workgroup.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_one(const I *__restrict__ ids, int32_t V,
                                                           int count, int passes, int bits,
                                                           uint32_t *__restrict__ keys_out,
                                                           uint32_t *__restrict__ pos_out) {
    __shared__ SortShared s;
    const int lane = __lane_id(), w = threadIdx.x / kWave;
    uint32_t key[kSortSteps], pos[kSortSteps];
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int i = (w * kSortSteps + j) * kWave + lane;
        pos[j] = i;
        key[j] = i < count ? token_key(ids, i, V) : 0u;
    }
    for (int p = 0; p < passes; ++p) {
        sort_tile(s, key, pos, count, p * bits, bits);
#pragma unroll
        for (int j = 0; j < kSortSteps; ++j) {
            const int i = (w * kSortSteps + j) * kWave + lane;
            key[j] = i < count ? s.key[i] : 0u;
            pos[j] = i < count ? s.pos[i] : 0u;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int i = (w * kSortSteps + j) * kWave + lane;
        if (i < count) {
            keys_out[i] = key[j];
            pos_out[i] = pos[j];
        }
    }
}

// One pass over many tiles.  A tile's place for digit d is the tokens of all
// smaller digits plus those of d in earlier tiles: every workgroup adds them
// up from the count table itself (thread d, one row of the table per step).
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(
    const I *__restrict__ ids, int32_t V, const uint32_t *__restrict__ keys,
    const uint32_t *__restrict__ pos_in, int64_t n, int shift, int bits, int32_t tiles,
    const int32_t *__restrict__ counts, uint32_t *__restrict__ keys_out,
    uint32_t *__restrict__ pos_out) {
    __shared__ SortShared s;
    __shared__ int goff[kSortDigits];
    const int lane = __lane_id(), w = threadIdx.x / kWave, tid = threadIdx.x;
    const int digits = 1 << bits;
    const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * kSortTile;
    const int count = static_cast<int>(n - tile0 < kSortTile ? n - tile0 : kSortTile);
    uint32_t key[kSortSteps], pos[kSortSteps];
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int i = (w * kSortSteps + j) * kWave + lane;
        key[j] = pos[j] = 0;
        if (i < count) {
            key[j] = keys ? keys[tile0 + i] : token_key(ids, tile0 + i, V);
            pos[j] = keys ? pos_in[tile0 + i] : static_cast<uint32_t>(tile0 + i);
        }
    }
    int total = 0, before = 0;
    if (tid < digits) {
        for (int t = 0; t < tiles; ++t) {
            const int c = counts[static_cast<int64_t>(t) * digits + tid];
            before += t < static_cast<int>(blockIdx.x) ? c : 0;
            total += c;
        }
    }
    const int smaller = sort_exclusive(total, s.wsum);
    if (tid < digits) goff[tid] = smaller + before;
    sort_tile(s, key, pos, count, shift, bits);
    for (int p = tid; p < count; p += kSortThreads) {
        const uint32_t k = s.key[p];
        const int d = (k >> shift) & (digits - 1);
        const int g = goff[d] + (p - s.start[d]);
        keys_out[g] = k;
        pos_out[g] = s.pos[p];
    }
}

// ----------------------------------------------------------------- gradient

// Sorted tokens per chunk, and table rows that one workgroup clears.
constexpr int kChunk = 32;
constexpr int kClearRows = 16;
constexpr int kAhead = 8;       // gradient rows in flight per lane
constexpr int kJoinParts = 16;  // waves that share a cut row's parts
constexpr int kJoinThreads = kJoinParts * kWave;

__device__ inline uint32_t first_not_below(const uint32_t *keys, uint32_t n, uint32_t v) {
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    return lo;
}

template <typename T>
__device__ inline void put_row(T *p, int left, float scale, int accumulate, const float *sum) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (accumulate) {
        if (left >= 8)
            load_octet(p, v);
        else
            load_octet_tail(p, left, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(scale, sum[i], v[i]);
    if (left >= 8)
        store_octet(p, v);
    else
        store_octet_tail(p, left, v);
}

// Items [0, chunks): the sums of one chunk of sorted tokens over one range of
// columns, an octet per lane.  A row whose tokens all lie in the chunk is
// written; the part of one that goes on from the chunk before goes to
// head[chunk], the part of one that goes on into the next to tail[chunk]
// (one that does both: head).
template <typename G, typename T>
__device__ inline void grad_chunk(int32_t V, int32_t D, int64_t n,
                                  const uint32_t *__restrict__ keys,
                                  const uint32_t *__restrict__ pos, const G *__restrict__ grad,
                                  int64_t grad_ld, float scale, int accumulate,
                                  T *__restrict__ out, int64_t ld, float *__restrict__ head,
                                  float *__restrict__ tail, int64_t chunk, int64_t col) {
    __shared__ uint32_t s_key[kChunk];
    __shared__ uint32_t s_pos[kChunk];
    const int64_t base = chunk * kChunk;
    const int count = static_cast<int>(n - base < kChunk ? n - base : kChunk);
    __syncthreads();  // the item before may still read s_key
    if (static_cast<int>(threadIdx.x) < count) {
        s_key[threadIdx.x] = keys[base + threadIdx.x];
        s_pos[threadIdx.x] = pos[base + threadIdx.x];
    }
    const uint32_t none = 0xffffffffu;
    const uint32_t prev = base > 0 ? keys[base - 1] : none;
    const uint32_t next = base + count < n ? keys[base + count] : none;
    __syncthreads();
    if (col >= D) return;
    const int left = static_cast<int>(D - col < 8 ? D - col : 8);
    float sum[8] = {};
    bool from_before = s_key[0] == prev;
    for (int k0 = 0; k0 < count; k0 += kAhead) {
        float g[kAhead][8];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j < count ? k0 + j : count - 1;
            const G *p = grad + static_cast<int64_t>(s_pos[k]) * grad_ld + col;
            if (left == 8)
                load_octet(p, g[j]);
            else
                load_octet_tail(p, left, g[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j;
            if (k >= count) break;
            const uint32_t key = s_key[k];
            if (key >= static_cast<uint32_t>(V)) return;  // tokens that name no row come last
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += g[j][i];
            const bool last = k + 1 == count;
            const uint32_t after = last ? next : s_key[k + 1];
            if (!last && after == key) continue;
            if (from_before || (last && after == key)) {
                float *p = (from_before ? head : tail) + chunk * D + col;
                if (left == 8)
                    store_octet(p, sum);
                else
                    store_octet_tail(p, left, sum);
            } else {
                put_row(out + static_cast<int64_t>(key) * ld + col, left, scale, accumulate, sum);
            }
            from_before = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = 0.f;
        }
    }
}

// Items behind the chunks: zeros into those of kClearRows table rows that no
// token names.
template <typename T>
__device__ inline void grad_clear(int32_t V, int32_t D, int64_t n,
                                  const uint32_t *__restrict__ keys, T *__restrict__ out,
                                  int64_t ld, int64_t r0, int64_t col) {
    __shared__ unsigned long long missing;
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int64_t v = r0 + threadIdx.x;
        bool none = false;
        if (threadIdx.x < kClearRows && v < V) {
            const uint32_t at =
                first_not_below(keys, static_cast<uint32_t>(n), static_cast<uint32_t>(v));
            none = at == static_cast<uint32_t>(n) || keys[at] != static_cast<uint32_t>(v);
        }
        const unsigned long long m = __ballot(none);
        if (threadIdx.x == 0) missing = m;
    }
    __syncthreads();
    if (col >= D) return;
    const int left = static_cast<int>(D - col < 8 ? D - col : 8);
    const float zero[8] = {};
    for (int i = 0; i < kClearRows; ++i) {
        if (!((missing >> i) & 1)) continue;
        T *p = out + (r0 + i) * ld + col;
        if (left == 8)
            store_octet(p, zero);
        else
            store_octet_tail(p, left, zero);
    }
}

template <typename G, typename T>
__global__ __launch_bounds__(kThreads) void k_grad_chunks(
    int32_t V, int32_t D, int64_t n, const uint32_t *__restrict__ keys,
    const uint32_t *__restrict__ pos, const G *__restrict__ grad, int64_t grad_ld, float scale,
    int accumulate, T *__restrict__ out, int64_t ld, float *__restrict__ head,
    float *__restrict__ tail, int64_t chunks, int64_t clears, int64_t parts) {
    for (int64_t i = blockIdx.x; i < (chunks + clears) * parts; i += gridDim.x) {
        const int64_t item = i / parts;
        const int64_t col = ((i % parts) * blockDim.x + threadIdx.x) * 8;
        if (item < chunks)
            grad_chunk(V, D, n, keys, pos, grad, grad_ld, scale, accumulate, out, ld, head, tail,
                       item, col);
        else
            grad_clear(V, D, n, keys, out, ld, (item - chunks) * kClearRows, col);
    }
}

// Joins the parts of the rows that chunk borders cut: the workgroup of the
// chunk where such a row begins adds that chunk's tail and the heads of the
// following chunks up to the one where the row ends.  kJoinParts waves take
// consecutive shares of the parts, which are then added in order.
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void k_grad_join(
    int32_t V, int32_t D, int64_t n, const uint32_t *__restrict__ keys, float scale,
    int accumulate, T *__restrict__ out, int64_t ld, const float *__restrict__ head,
    const float *__restrict__ tail, int64_t cuts, int64_t cols) {
    __shared__ float s[kJoinParts][kWave];
    for (int64_t item = blockIdx.x; item < cuts * cols; item += gridDim.x) {
        const int64_t c = item / cols;
        const int64_t end = (c + 1) * kChunk;  // < n: the last chunk has no workgroup
        const uint32_t key = keys[end - 1];
        if (key >= static_cast<uint32_t>(V) || keys[end] != key) continue;
        if (c > 0 && keys[c * kChunk - 1] == key) continue;  // began before: not this chunk's
        // The row's last token, by doubling and halving over [end, n).  Token
        // indices are 32-bit: with 64-bit ones clang 22 selects `hi` by the scalar
        // condition code where its compare has set the vector one.
        uint32_t lo = static_cast<uint32_t>(end), hi = lo + 1, step = kChunk;
        const uint32_t count = static_cast<uint32_t>(n);
        while (hi < count && keys[hi] == key) {
            lo = hi;
            hi = hi + step < count ? hi + step : count;
            step *= 2;
        }
        while (hi - lo > 1) {  // keys[lo] == key, keys[hi] != key or hi == n
            const uint32_t mid = lo + (hi - lo) / 2;
            if (keys[mid] == key) lo = mid; else hi = mid;
        }
        const int64_t parts = lo / kChunk - c + 1;
        const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
        const int64_t col = (item % cols) * kWave + lane;
        const int64_t from = parts * w / kJoinParts, to = parts * (w + 1) / kJoinParts;
        float sum = 0.f;
        if (col < D) {
            for (int64_t p = from; p < to; ++p)
                sum += p == 0 ? tail[c * D + col] : head[(c + p) * D + col];
        }
        __syncthreads();  // the item before may still read s
        s[w][lane] = sum;
        __syncthreads();
        if (w == 0 && col < D) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i) t += s[i][lane];
            T *p = out + static_cast<int64_t>(key) * ld + col;
            *p = static_cast<T>(fmaf(scale, t, accumulate ? static_cast<float>(*p) : 0.f));
        }
    }
}

// Parts of the gradient's workspace, each 256-byte aligned.
struct GradWorkspace {
    uint32_t *keys[2], *pos[2];
    int32_t *counts;
    float *head, *tail;
    size_t bytes;
};

GradWorkspace grad_workspace(int32_t D, int64_t n, void *base) {
    GradWorkspace w{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(base) + at;
        at += (bytes + 255) & ~size_t{255};
        return p;
    };
    const size_t tiles = static_cast<size_t>((n + kSortTile - 1) / kSortTile);
    const size_t chunks = static_cast<size_t>((n + kChunk - 1) / kChunk);
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = reinterpret_cast<uint32_t *>(take(static_cast<size_t>(n) * 4));
        w.pos[i] = reinterpret_cast<uint32_t *>(take(static_cast<size_t>(n) * 4));
    }
    w.counts = reinterpret_cast<int32_t *>(take(tiles > 1 ? tiles * kSortDigits * 4 : 0));
    const size_t part = chunks > 1 ? chunks * static_cast<size_t>(D) * 4 : 0;
    w.head = reinterpret_cast<float *>(take(part));
    w.tail = reinterpret_cast<float *>(take(part));
    w.bytes = at;
    return w;
}

template <typename I>
spmv_status sort_tokens(int32_t V, int64_t n, const I *ids, const GradWorkspace &w,
                        const uint32_t **keys, const uint32_t **pos, hipStream_t s) {
    const int need = std::max(1, bits_for(static_cast<uint64_t>(V)));
    const int passes = (need + kSortBits - 1) / kSortBits;
    const int bits = (need + passes - 1) / passes;
    const int32_t tiles = static_cast<int32_t>((n + kSortTile - 1) / kSortTile);
    if (tiles == 1) {
        k_sort_one<I><<<1, kSortThreads, 0, s>>>(ids, V, static_cast<int>(n), passes, bits,
                                                 w.keys[0], w.pos[0]);
        SPMV_HIP(hipGetLastError());
        *keys = w.keys[0];
        *pos = w.pos[0];
        return SPMV_OK;
    }
    const uint32_t *k = nullptr, *p = nullptr;
    for (int i = 0; i < passes; ++i) {
        k_sort_count<I><<<tiles, kSortThreads, 0, s>>>(ids, V, k, n, i * bits, bits, w.counts);
        SPMV_HIP(hipGetLastError());
        k_sort_scatter<I><<<tiles, kSortThreads, 0, s>>>(ids, V, k, p, n, i * bits, bits, tiles,
                                                         w.counts, w.keys[i & 1], w.pos[i & 1]);
        SPMV_HIP(hipGetLastError());
        k = w.keys[i & 1];
        p = w.pos[i & 1];
    }
    *keys = k;
    *pos = p;
    return SPMV_OK;
}

}  // namespace

spmv_status lookup_rows(int32_t V, int32_t D, const void *table, int64_t table_ld, int32_t dtype,
                        int64_t n, const void *ids, int32_t id_dtype, float scale, void *out,
                        int64_t out_ld, int32_t out_dtype, hipStream_t s) {
    const int L = lanes_for((static_cast<int64_t>(D) + 7) / 8, kThreads);
    const unsigned grid = groups_for(n, kThreads / L);
    with_float(dtype, [&](auto a) {
        with_float(out_dtype, [&](auto b) {
            using A = decltype(a);
            using B = decltype(b);
            if (id_dtype == SPMV_INT64)
                k_lookup<A, B, int64_t><<<grid, kThreads, 0, s>>>(
                    V, D, L, static_cast<const A *>(table), table_ld, n,
                    static_cast<const int64_t *>(ids), scale, static_cast<B *>(out), out_ld);
            else
                k_lookup<A, B, int32_t><<<grid, kThreads, 0, s>>>(
                    V, D, L, static_cast<const A *>(table), table_ld, n,
                    static_cast<const int32_t *>(ids), scale, static_cast<B *>(out), out_ld);
        });
    });
    SPMV_HIP(hipGetLastError());
    return SPMV_OK;
}

size_t lookup_grad_bytes(int32_t, int32_t D, int64_t n) {
    return grad_workspace(D, n, nullptr).bytes;
}

spmv_status lookup_grad(int32_t V, int32_t D, int64_t n, const void *ids, int32_t id_dtype,
                        const void *grad, int64_t grad_ld, int32_t grad_dtype, float scale,
                        int accumulate, void *dtable, int64_t ld, int32_t dtype, void *workspace,
                        hipStream_t s) {
    const GradWorkspace w = grad_workspace(D, n, workspace);
    const uint32_t *keys = nullptr, *pos = nullptr;
    if (n > 0) {
        if (id_dtype == SPMV_INT64)
            SPMV_TRY(sort_tokens(V, n, static_cast<const int64_t *>(ids), w, &keys, &pos, s));
        else
            SPMV_TRY(sort_tokens(V, n, static_cast<const int32_t *>(ids), w, &keys, &pos, s));
    }
    const int64_t octets = (static_cast<int64_t>(D) + 7) / 8;
    const int threads = std::max(kWave, lanes_for(octets, kThreads));
    const int64_t parts = (octets + threads - 1) / threads;
    const int64_t chunks = (n + kChunk - 1) / kChunk;
    const int64_t clears = accumulate ? 0 : (static_cast<int64_t>(V) + kClearRows - 1) / kClearRows;
    if (chunks + clears > 0) {
        with_float(grad_dtype, [&](auto a) {
            with_float(dtype, [&](auto b) {
                using G = decltype(a);
                using T = decltype(b);
                k_grad_chunks<G, T><<<groups_for((chunks + clears) * parts, 1), threads, 0, s>>>(
                    V, D, n, keys, pos, static_cast<const G *>(grad), grad_ld, scale, accumulate,
                    static_cast<T *>(dtable), ld, w.head, w.tail, chunks, clears, parts);
            });
        });
        SPMV_HIP(hipGetLastError());
    }
    if (chunks > 1) {
        const int64_t cols = (static_cast<int64_t>(D) + kWave - 1) / kWave;
        with_float(dtype, [&](auto b) {
            using T = decltype(b);
            k_grad_join<T><<<groups_for((chunks - 1) * cols, 1), kJoinThreads, 0, s>>>(
                V, D, n, keys, scale, accumulate, static_cast<T *>(dtable), ld, w.head, w.tail,
                chunks - 1, cols);
        });
        SPMV_HIP(hipGetLastError());
    }
    return SPMV_OK;
}

}  // namespace spmv
