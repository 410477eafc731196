// Rows of a dense table by token, and the gradient of that lookup by sorted
// tokens.
//
//   out[t, :]    = scale * table[ids[t], :]
//   dtable[v, :] = scale * sum over t with ids[t] = v of grad[t, :]
//
// The gradient is the product of the transposed selection matrix with the
// rows of grad.  The tokens are sorted stably, as the COO -> CSR builder sorts
// row indices, so that the tokens of one row are neighbours in their own order;
// the sorted list is cut into chunks of equal length whatever its rows, as a
// segmented sum, and the parts of a row that chunk borders cut are joined in
// order afterwards.  No sum is made by atomics (only the sort's counts of
// tokens are, in LDS): the sums are the same from run to run.
#include "tables.h"

namespace spmv {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- lookup

// Columns a lane handles at a time: eight, but four of them as fp32 where it
// pays.  A lane's 32 bytes are two accesses, in neither of which its
// neighbour's bytes lie beside its own (one access of the vector cache per
// lane instead of one per four), but four bf16 are only half as many bytes
// per access.  16384 rows of 4096, fp32 to fp32: 111 us by eights, 96 by fours;
// bf16 to fp32 99 and 94; fp32 to bf16 49 and 54.  Gradients of 16384 x 1024,
// fp32 to fp32: 42.5 and 41.2; 32768 x 2048, bf16 to fp32: 236 and 241.
template <typename T>
constexpr int kPiece = sizeof(T) == 4 ? 4 : 8;

// L lanes per row, kFlight pieces each per step, all loaded before the first
// is stored.  A copy: bound by memory, reads and writes mixed.  16384 rows of
// 4096 bf16 (134 MB written, 94 MB read past the caches, repeated rows once)
// take 37 us, 6.2 TB/s; with one piece in flight per lane 53 us.
constexpr int kFlight = 2;
template <typename A, typename B, typename I>
__global__ __launch_bounds__(kThreads) void k_lookup(int32_t V, int32_t D, int L,
                                                     const A *__restrict__ table,
                                                     int64_t table_ld, int64_t n,
                                                     const I *__restrict__ ids, float scale,
                                                     B *__restrict__ out, int64_t out_ld) {
    constexpr int E = kPiece<B>;
    const int rows = kThreads / L;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / L; t < n;
         t += static_cast<int64_t>(gridDim.x) * rows) {
        const int64_t id = ids[t];
        const bool there = id >= 0 && id < V;
        const A *src = table + (there ? id : 0) * table_ld;
        B *dst = out + t * out_ld;
        for (int64_t c = threadIdx.x % L * E; c < D; c += kFlight * E * L) {
            float v[kFlight][E];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int64_t at = c + u * E * L;
#pragma unroll
                for (int i = 0; i < E; ++i) v[u][i] = 0.f;
                if (there && at + E <= D)
                    load_piece<E>(src + at, v[u]);
                else if (there && at < D)
                    load_piece_tail<E>(src + at, static_cast<int>(D - at), v[u]);
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int64_t at = c + u * E * L;
                if (there) {
#pragma unroll
                    for (int i = 0; i < E; ++i) v[u][i] *= scale;
                }
                if (at + E <= D)
                    store_piece<E>(dst + at, v[u]);
                else if (at < D)
                    store_piece_tail<E>(dst + at, static_cast<int>(D - at), v[u]);
            }
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
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next step reads it
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

// Up to merge_most(V) tokens are sorted in two launches: tiles of kRankTile by
// counting, then all tiles merged by searching, whose work grows with the
// square of the tokens.  A radix pass takes two launches, and up to 2^10 rows
// one pass is enough, up to 2^20 two.  Merged, then by passes of ten bits:
// 16384 tokens 12.6 us, 14.2 per pass; 32768 18.3 and 16.7; 65536 30.0 and 17.9.
constexpr int kRankTile = kSortWaves * kWave;
inline int64_t merge_most(int32_t V) { return V < kSortDigits ? 1 << 14 : 1 << 16; }

// A token's place in its tile is the number of the tile's tokens that sort
// before it.  A workgroup ranks 64 tokens, one per lane, in all its waves;
// each wave holds 64 of the tile's keys and broadcasts them in turn.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_tiles(const I *__restrict__ ids, int32_t V,
                                                             int n,
                                                             uint32_t *__restrict__ keys_out,
                                                             uint32_t *__restrict__ pos_out) {
    __shared__ int part[kSortWaves][kWave];
    const int lane = __lane_id();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int tile = static_cast<int>(blockIdx.x) / kSortWaves * kRankTile;
    const int own = static_cast<int>(blockIdx.x) % kSortWaves;
    const int t = tile + own * kWave + lane, j = tile + w * kWave + lane;
    const uint32_t key = t < n ? token_key(ids, t, V) : 0u;
    const uint32_t k = j < n ? token_key(ids, j, V) : 0xffffffffu;  // behind every key
    int before = 0;
    if (w != own) {
        // equal keys of an earlier wave come first: k < key + 1
        const uint32_t limit = key + (w < own ? 1u : 0u);
#pragma unroll
        for (int l = 0; l < kWave; ++l)
            before += static_cast<uint32_t>(__builtin_amdgcn_readlane(k, l)) < limit;
    } else {
#pragma unroll
        for (int l = 0; l < kWave; ++l)
            before += static_cast<uint32_t>(__builtin_amdgcn_readlane(k, l)) <
                      key + (l < lane ? 1u : 0u);
    }
    part[w][lane] = before;
    __syncthreads();
    if (w == 0 && t < n) {
        int at = tile;
#pragma unroll
        for (int i = 0; i < kSortWaves; ++i) at += part[i][lane];
        keys_out[at] = key;
        pos_out[at] = t;
    }
}

// A token's place in the whole list: its place in its tile, and in every other
// tile the number of tokens before it, by binary search.  kAbreast tiles at a
// time are brought to LDS and searched side by side (searching them where they
// lie costs one access of the vector cache per lane and step: 53 us against
// the 12 of this for 32768 tokens).
__global__ __launch_bounds__(kThreads) void k_sort_merge(int n, const uint32_t *__restrict__ keys,
                                                         const uint32_t *__restrict__ pos,
                                                         uint32_t *__restrict__ keys_out,
                                                         uint32_t *__restrict__ pos_out) {
    constexpr int kAbreast = 4;
    constexpr int kPieces = kAbreast * kRankTile / (4 * kThreads);
    using Four = uint32_t __attribute__((ext_vector_type(4)));
    __shared__ __attribute__((aligned(16))) uint32_t s_key[kAbreast * kRankTile];
    const int e = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
    const uint32_t key = e < n ? keys[e] : 0u;
    const int own = e / kRankTile;
    int at = e % kRankTile;
    Four in[kPieces];
    auto load = [&](int first) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int j = first + (i * kThreads + static_cast<int>(threadIdx.x)) * 4;
            in[i] = Four{~0u, ~0u, ~0u, ~0u};  // past the end: behind every key
            if (j + 4 <= n) {
                in[i] = *reinterpret_cast<const Four *>(keys + j);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (j + q < n) in[i][q] = keys[j + q];
            }
        }
    };
    load(0);
    for (int first = 0; first < n; first += kAbreast * kRankTile) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            *reinterpret_cast<Four *>(&s_key[(i * kThreads + threadIdx.x) * 4]) = in[i];
        __syncthreads();
        load(first + kAbreast * kRankTile);
        int lo[kAbreast];
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) lo[i] = 0;
#pragma unroll
        for (int s = kRankTile / 2; s >= 0; s = s > 1 ? s / 2 : s - 1) {
            const int hop = s > 0 ? s : 1;  // the last compare is of one more key
#pragma unroll
            for (int i = 0; i < kAbreast; ++i) {
                const uint32_t limit = key + (first / kRankTile + i < own ? 1u : 0u);
                lo[i] += s_key[i * kRankTile + lo[i] + hop - 1] < limit ? hop : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kAbreast; ++i) at += first / kRankTile + i != own ? lo[i] : 0;
    }
    if (e < n) {
        keys_out[at] = key;
        pos_out[at] = pos[e];
    }
}

// A tile's place for digit d is the tokens of all smaller digits plus those of
// d in earlier tiles.  Up to kSumTiles tiles, every workgroup of the scatter
// adds them up from the count table itself (thread d, one row of the table per
// step).  More tiles are taken in segments, whose places are found first:
// segment sums, then one workgroup turns them into places.  A pass takes 22 us
// without segments and 24 with them for 35 tiles, 75 and 32 for 245 (50 with
// segments of 64).
constexpr int kSumTiles = 64;
constexpr int kSegment = 16;

// Segments that the passes over so many tiles use.
inline int32_t sort_segments(int32_t tiles) {
    return tiles > kSumTiles ? (tiles + kSegment - 1) / kSegment : 0;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_segments(int32_t tiles, int bits,
                                                                const int32_t *__restrict__ counts,
                                                                int32_t *__restrict__ places) {
    const int digits = 1 << bits, d = threadIdx.x;
    if (d >= digits) return;
    const int32_t first = static_cast<int32_t>(blockIdx.x) * kSegment;
    const int32_t last = tiles - first < kSegment ? tiles : first + kSegment;
    int32_t sum = 0;
#pragma unroll 4
    for (int32_t t = first; t < last; ++t) sum += counts[static_cast<int64_t>(t) * digits + d];
    places[static_cast<int64_t>(blockIdx.x) * digits + d] = sum;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_places(int32_t segments, int bits,
                                                              int32_t *__restrict__ places) {
    __shared__ int wsum[kSortWaves];
    const int digits = 1 << bits, d = threadIdx.x;
    int total = 0;
    if (d < digits)
#pragma unroll 4
        for (int32_t s = 0; s < segments; ++s)
            total += places[static_cast<int64_t>(s) * digits + d];
    int at = sort_exclusive(total, wsum);
    if (d < digits) {
        for (int32_t s = 0; s < segments; ++s) {
            int32_t *p = places + static_cast<int64_t>(s) * digits + d;
            const int32_t sum = *p;
            *p = at;
            at += sum;
        }
    }
}

// One pass over many tiles; `places` null: at most kSumTiles tiles.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(
    const I *__restrict__ ids, int32_t V, const uint32_t *__restrict__ keys,
    const uint32_t *__restrict__ pos_in, int64_t n, int shift, int bits, int32_t tiles,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ places,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ pos_out) {
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
    const int32_t own = static_cast<int32_t>(blockIdx.x);
    if (places) {
        if (tid < digits) {
            int at = places[static_cast<int64_t>(own / kSegment) * digits + tid];
            for (int32_t t = own / kSegment * kSegment; t < own; ++t)
                at += counts[static_cast<int64_t>(t) * digits + tid];
            goff[tid] = at;
        }
    } else {
        int total = 0, before = 0;
        if (tid < digits) {
            for (int32_t t = 0; t < tiles; ++t) {
                const int c = counts[static_cast<int64_t>(t) * digits + tid];
                before += t < own ? c : 0;
                total += c;
            }
        }
        const int smaller = sort_exclusive(total, s.wsum);
        if (tid < digits) goff[tid] = smaller + before;
    }
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

constexpr int kMaxChunk = 32;   // sorted tokens per chunk, at most
constexpr int kMinLanes = 8;    // lanes per chunk, at least
constexpr int kClearRows = 8;   // table rows that one wave clears (four: 5001 tokens into
                                // 50001 x 1000 take 1.5 us more, for the searches)
constexpr int kAhead = 8;       // gradient rows in flight per lane (four: 16384 tokens of
                                // 1024 take 25.0 us, not 24.2)
constexpr int kJoinParts = 4;   // waves that share a cut row's parts
constexpr int kJoinThreads = kJoinParts * kWave;
constexpr int kJoinCols = 4 * kWave;

// First index in [lo, n) whose key is at least v, by all lanes of a wave:
// 64 probes at a time.
__device__ inline uint32_t first_not_below(const uint32_t *keys, uint32_t lo, uint32_t n,
                                           uint32_t v) {
    const uint32_t lane = __lane_id();
    uint32_t len = n - lo;
    while (len > 0) {
        const uint32_t step = (len + kWave - 1) / kWave;
        const uint32_t i = lane * step;
        const bool below = i < len && keys[lo + i] < v;
        const uint32_t c = static_cast<uint32_t>(__popcll(__ballot(below)));
        if (c == 0) return lo;
        const uint32_t skip = (c - 1) * step + 1;  // those are below
        lo += skip;
        len = len - skip < step - 1 ? len - skip : step - 1;
    }
    return lo;
}

template <int E, typename T>
__device__ inline void put_row(T *p, int left, float scale, int accumulate, const float *sum) {
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0.f;
    if (accumulate) {
        if (left >= E)
            load_piece<E>(p, v);
        else
            load_piece_tail<E>(p, left, v);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = fmaf(scale, sum[i], v[i]);
    if (left >= E)
        store_piece<E>(p, v);
    else
        store_piece_tail<E>(p, left, v);
}

// The sums of chunks of sorted tokens over a range of columns: a group of L
// lanes per chunk, a piece of columns per lane.  A row whose tokens all lie
// in the chunk is written; the part of one that goes on from the chunk before
// goes to head[chunk], the part of one that goes on into the next to
// tail[chunk] (one that does both: head).
template <typename G, typename T>
__device__ inline void grad_chunk(int32_t V, int32_t D, int64_t n,
                                  const uint32_t *__restrict__ keys,
                                  const uint32_t *__restrict__ pos, const G *__restrict__ grad,
                                  int64_t grad_ld, float scale, int accumulate,
                                  T *__restrict__ out, int64_t ld, float *__restrict__ head,
                                  float *__restrict__ tail, int per_chunk, int L, int64_t first,
                                  int64_t part) {
    constexpr int E = kPiece<G>;
    __shared__ uint32_t lds_key[kThreads / kMinLanes][kMaxChunk];
    __shared__ uint32_t lds_pos[kThreads / kMinLanes][kMaxChunk];
    const int group = threadIdx.x / L, lane = threadIdx.x % L;
    uint32_t *const s_key = lds_key[group], *const s_pos = lds_pos[group];
    const int64_t chunk = first + group, base = chunk * per_chunk;
    const int count =
        static_cast<int>(n <= base ? 0 : n - base < per_chunk ? n - base : per_chunk);
    __syncthreads();  // the item before may still read s_key
    for (int i = lane; i < count; i += L) {
        s_key[i] = keys[base + i];
        s_pos[i] = pos[base + i];
    }
    const uint32_t none = 0xffffffffu;
    const uint32_t prev = count > 0 && base > 0 ? keys[base - 1] : none;
    const uint32_t next = base + count < n ? keys[base + count] : none;
    __syncthreads();
    const int64_t col = (part * L + lane) * E;
    if (col >= D || count == 0) return;
    const int left = static_cast<int>(D - col < E ? D - col : E);
    float sum[E] = {};
    bool from_before = s_key[0] == prev;
    for (int k0 = 0; k0 < count; k0 += kAhead) {
        Piece<G, E> g[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j < count ? k0 + j : count - 1;
            const G *p = grad + static_cast<int64_t>(s_pos[k]) * grad_ld + col;
            if (left == E) {
                __builtin_memcpy(&g[j], p, sizeof(g[j]));
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) g[j].v[i] = i < left ? p[i] : static_cast<G>(0.f);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j;
            if (k >= count) break;
            const uint32_t key = s_key[k];
            if (key >= static_cast<uint32_t>(V)) return;  // tokens that name no row come last
#pragma unroll
            for (int i = 0; i < E; ++i) sum[i] += static_cast<float>(g[j].v[i]);
            const bool last = k + 1 == count;
            const uint32_t after = last ? next : s_key[k + 1];
            if (!last && after == key) continue;
            if (from_before || (last && after == key)) {
                float *p = (from_before ? head : tail) + chunk * D + col;
                if (left == E)
                    store_piece<E>(p, sum);
                else
                    store_piece_tail<E>(p, left, sum);
            } else {
                put_row<E>(out + static_cast<int64_t>(key) * ld + col, left, scale, accumulate,
                           sum);
            }
            from_before = false;
#pragma unroll
            for (int i = 0; i < E; ++i) sum[i] = 0.f;
        }
    }
}

// Behind the chunks: a wave writes zeros into those of kClearRows table rows
// that no token names.
template <typename T>
__device__ inline void grad_clear(int32_t V, int32_t D, uint32_t n,
                                  const uint32_t *__restrict__ keys, T *__restrict__ out,
                                  int64_t ld, int64_t r0) {
    const int lane = __lane_id();
    if (r0 >= V) return;
    const uint32_t rows = static_cast<uint32_t>(V - r0 < kClearRows ? V - r0 : kClearRows);
    const uint32_t first = static_cast<uint32_t>(r0);
    uint32_t named = 0, at = first_not_below(keys, 0, n, first);
    while (at < n) {
        const uint32_t k = at + lane < n ? keys[at + lane] - first : rows;
#pragma unroll
        for (uint32_t i = 0; i < kClearRows; ++i) named |= __ballot(k == i) ? 1u << i : 0u;
        const uint32_t last = __builtin_amdgcn_readlane(k, kWave - 1);
        if (last >= rows) break;
        at = first_not_below(keys, at + kWave, n, first + last + 1);
    }
    constexpr int kPer = 16 / sizeof(T);
    using Zeros = uint32_t __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    for (uint32_t i = 0; i < rows; ++i) {
        if ((named >> i) & 1) continue;
        T *p = out + (r0 + i) * ld;
        for (int64_t c = static_cast<int64_t>(lane) * kPer; c < D; c += kWave * kPer) {
            if (c + kPer <= D) {
                *reinterpret_cast<Zeros *>(p + c) = Zeros{0, 0, 0, 0};
            } else {
                for (int64_t e = c; e < D; ++e) p[e] = static_cast<T>(0.f);
            }
        }
    }
}

// Sums and clears share a launch, the sums first: reading gradients and writing
// zeros both need memory in flight.  Bound by memory: 32768 tokens into 128000 x
// 2048 fp32 write 1.05 GB and read 134 MB in 237 us (5.0 TB/s; a fill alone
// reaches 5.7 to 6.8).
template <typename G, typename T>
__global__ __launch_bounds__(kThreads) void k_grad_chunks(
    int32_t V, int32_t D, int64_t n, const uint32_t *__restrict__ keys,
    const uint32_t *__restrict__ pos, const G *__restrict__ grad, int64_t grad_ld, float scale,
    int accumulate, T *__restrict__ out, int64_t ld, float *__restrict__ head,
    float *__restrict__ tail, int per_chunk, int L, int64_t sums, int64_t clears, int64_t parts) {
    constexpr int kWaves = kThreads / kWave;
    for (int64_t i = blockIdx.x; i < sums + clears; i += gridDim.x) {
        if (i < sums) {
            grad_chunk(V, D, n, keys, pos, grad, grad_ld, scale, accumulate, out, ld, head, tail,
                       per_chunk, L, i / parts * (kThreads / L), i % parts);
        } else {
            const int64_t w =
                (i - sums) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
            grad_clear(V, D, static_cast<uint32_t>(n), keys, out, ld, w * kClearRows);
        }
    }
}

// Joins the parts of the rows that chunk borders cut: the workgroup of the
// chunk where such a row begins adds that chunk's tail and the heads of the
// following chunks up to the one where the row ends.  kJoinParts waves take
// consecutive shares of the parts, which are then added in order.  Bound by
// the latency of a frequent token's many parts: 12 us for 32768 tokens of a
// natural-language spread, 2048 columns.  A row's parts are one workgroup's per
// 256 columns: the whole gradient of 65536 tokens of a single row, 2048
// columns, takes 138 us (126 where the tokens spread by rank over 1000 rows), of
// 2^20 such tokens 1.85 ms (1.43).
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void k_grad_join(
    int32_t V, int32_t D, int64_t n, const uint32_t *__restrict__ keys, float scale,
    int accumulate, T *__restrict__ out, int64_t ld, const float *__restrict__ head,
    const float *__restrict__ tail, int per_chunk, int64_t cuts, int64_t cols) {
    __shared__ float s[kJoinParts][kJoinCols];
    for (int64_t item = blockIdx.x; item < cuts * cols; item += gridDim.x) {
        const int64_t c = item / cols;
        const int64_t end = (c + 1) * per_chunk;  // < n: the last chunk has no workgroup
        const uint32_t key = keys[end - 1];
        if (key >= static_cast<uint32_t>(V) || keys[end] != key) continue;
        if (c > 0 && keys[c * per_chunk - 1] == key) continue;  // began before: not this chunk's
        // the row's first token behind `end` that is another's
        const uint32_t stop = first_not_below(keys, static_cast<uint32_t>(end) + 1,
                                              static_cast<uint32_t>(n), key + 1);
        const int64_t parts = (stop - 1) / per_chunk - c + 1;
        const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
        const int64_t col = (item % cols) * kJoinCols + lane * 4;
        const int left = static_cast<int>(D - col < 4 ? D - col : 4);
        const int64_t from = parts * w / kJoinParts, to = parts * (w + 1) / kJoinParts;
        float sum[4] = {};
        auto add = [&](const float *p, int count) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += e < count ? p[e] : 0.f;
        };
        if (left >= 4) {
            if (from == 0 && to > 0) add(tail + c * D + col, 4);
            const float *p = head + c * D + col;
#pragma unroll 8
            for (int64_t i = from > 1 ? from : 1; i < to; ++i) {
                float v[4];
                __builtin_memcpy(v, p + i * D, 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += v[e];
            }
        } else if (left > 0) {
            for (int64_t i = from; i < to; ++i)
                add((i == 0 ? tail : head + i * D) + c * D + col, left);
        }
        __syncthreads();  // the item before may still read s
#pragma unroll
        for (int e = 0; e < 4; ++e) s[w][lane * 4 + e] = sum[e];
        __syncthreads();
        const int64_t one = (item % cols) * kJoinCols + threadIdx.x;
        if (one < D) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i) t += s[i][threadIdx.x];
            T *p = out + static_cast<int64_t>(key) * ld + one;
            *p = static_cast<T>(fmaf(scale, t, accumulate ? static_cast<float>(*p) : 0.f));
        }
    }
}

// Lanes per chunk, a power of two, for pieces of `piece` columns.
int chunk_lanes(int32_t D, int piece) {
    return std::max(kMinLanes, lanes_for((static_cast<int64_t>(D) + piece - 1) / piece, kThreads));
}

// Sorted tokens per chunk: short chunks while there are few, so that the sums
// have 2048 waves (8 per CU); long ones leave fewer cut rows to join.  Sums and
// clear, then by chunks of 32 throughout: 512 tokens of 512 fp32 8.4 us and 18.8;
// 5001 of 1000 fp16 18.8 and 32.2; 16384 of 1024 bf16 24.2 and 32.5 (joins 0.5
// us shorter); from 32768 of 2048 on they are the same.
int chunk_length(int32_t D, int64_t n) {
    const int64_t octets = (static_cast<int64_t>(D) + 7) / 8, L = chunk_lanes(D, 8);
    const int64_t lanes = (octets + L - 1) / L * L;
    int k = 8;
    while (k < kMaxChunk && n * lanes > int64_t{2048} * kWave * k) k *= 2;
    return k;
}

// Parts of the gradient's workspace, each 256-byte aligned.
struct GradWorkspace {
    uint32_t *keys[2], *pos[2];
    int32_t *counts, *places;
    float *head, *tail;
    size_t bytes;
};

GradWorkspace grad_workspace(int32_t V, int32_t D, int64_t n, void *base) {
    GradWorkspace w{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(base) + at;
        at += (bytes + 255) & ~size_t{255};
        return p;
    };
    const int32_t tiles = static_cast<int32_t>((n + kSortTile - 1) / kSortTile);
    const int per_chunk = chunk_length(D, n);
    const size_t chunks = static_cast<size_t>((n + per_chunk - 1) / per_chunk);
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = reinterpret_cast<uint32_t *>(take(static_cast<size_t>(n) * 4));
        w.pos[i] = reinterpret_cast<uint32_t *>(take(static_cast<size_t>(n) * 4));
    }
    const size_t row = kSortDigits * 4;
    w.counts = reinterpret_cast<int32_t *>(take(n > merge_most(V) ? tiles * row : 0));
    w.places = reinterpret_cast<int32_t *>(take(sort_segments(tiles) * row));
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
    if (n <= merge_most(V)) {
        const int count = static_cast<int>(n);
        const int rank_tiles = (count + kRankTile - 1) / kRankTile;
        const int last = rank_tiles > 1 ? 1 : 0;
        k_sort_tiles<I><<<(count + kWave - 1) / kWave, kSortThreads, 0, s>>>(
            ids, V, count, w.keys[0], w.pos[0]);
        SPMV_HIP(hipGetLastError());
        if (rank_tiles > 1) {
            k_sort_merge<<<(count + kThreads - 1) / kThreads, kThreads, 0, s>>>(
                count, w.keys[0], w.pos[0], w.keys[1], w.pos[1]);
            SPMV_HIP(hipGetLastError());
        }
        *keys = w.keys[last];
        *pos = w.pos[last];
        return SPMV_OK;
    }
    const int32_t segments = sort_segments(tiles);
    int32_t *places = segments > 0 ? w.places : nullptr;
    const uint32_t *k = nullptr, *p = nullptr;
    for (int i = 0; i < passes; ++i) {
        k_sort_count<I><<<tiles, kSortThreads, 0, s>>>(ids, V, k, n, i * bits, bits, w.counts);
        SPMV_HIP(hipGetLastError());
        if (places) {
            k_sort_segments<<<segments, kSortThreads, 0, s>>>(tiles, bits, w.counts, places);
            SPMV_HIP(hipGetLastError());
            k_sort_places<<<1, kSortThreads, 0, s>>>(segments, bits, places);
            SPMV_HIP(hipGetLastError());
        }
        k_sort_scatter<I><<<tiles, kSortThreads, 0, s>>>(ids, V, k, p, n, i * bits, bits, tiles,
                                                         w.counts, places, w.keys[i & 1],
                                                         w.pos[i & 1]);
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
    const int piece = out_dtype == SPMV_FP32 ? kPiece<float> : kPiece<f16>;
    const int L = lanes_for((static_cast<int64_t>(D) + piece - 1) / piece, kThreads);
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

size_t lookup_grad_bytes(int32_t V, int32_t D, int64_t n) {
    return grad_workspace(V, D, n, nullptr).bytes;
}

spmv_status lookup_grad(int32_t V, int32_t D, int64_t n, const void *ids, int32_t id_dtype,
                        const void *grad, int64_t grad_ld, int32_t grad_dtype, float scale,
                        int accumulate, void *dtable, int64_t ld, int32_t dtype, void *workspace,
                        hipStream_t s) {
    const GradWorkspace w = grad_workspace(V, D, n, workspace);
    const uint32_t *keys = nullptr, *pos = nullptr;
    if (n > 0) {
        if (id_dtype == SPMV_INT64)
            SPMV_TRY(sort_tokens(V, n, static_cast<const int64_t *>(ids), w, &keys, &pos, s));
        else
            SPMV_TRY(sort_tokens(V, n, static_cast<const int32_t *>(ids), w, &keys, &pos, s));
    }
    const int piece = grad_dtype == SPMV_FP32 ? kPiece<float> : kPiece<f16>;
    const int L = chunk_lanes(D, piece);
    const int64_t parts = (static_cast<int64_t>(D) + L * piece - 1) / (L * piece);
    const int per_chunk = chunk_length(D, n);
    const int64_t chunks = (n + per_chunk - 1) / per_chunk;
    const int64_t sums = (chunks + kThreads / L - 1) / (kThreads / L) * parts;
    constexpr int64_t per_group = kThreads / kWave * kClearRows;
    const int64_t clears = accumulate ? 0 : (V + per_group - 1) / per_group;
    if (chunks + clears > 0) {
        with_float(grad_dtype, [&](auto a) {
            with_float(dtype, [&](auto b) {
                using G = decltype(a);
                using T = decltype(b);
                k_grad_chunks<G, T><<<groups_for(sums + clears, 1), kThreads, 0, s>>>(
                    V, D, n, keys, pos, static_cast<const G *>(grad), grad_ld, scale, accumulate,
                    static_cast<T *>(dtable), ld, w.head, w.tail, per_chunk, L, sums, clears,
                    parts);
            });
        });
        SPMV_HIP(hipGetLastError());
    }
    if (chunks > 1) {
        const int64_t cols = (static_cast<int64_t>(D) + kJoinCols - 1) / kJoinCols;
        with_float(dtype, [&](auto b) {
            using T = decltype(b);
            k_grad_join<T><<<groups_for((chunks - 1) * cols, 1), kJoinThreads, 0, s>>>(
                V, D, n, keys, scale, accumulate, static_cast<T *>(dtable), ld, w.head, w.tail,
                per_chunk, chunks - 1, cols);
        });
        SPMV_HIP(hipGetLastError());
    }
    return SPMV_OK;
}

}  // namespace spmv
