// Token embedding and its gradient (mamba_layers.h) on gfx950.
//
// Forward: one wave a token, 16 bytes a lane where rows allow it; bound by HBM (16384 tokens, 50000 x 768 bf16:
// 7.6 us for 25 MB written and at most as much read, 6.6 TB/s with repeated rows from cache).
//
// Gradient, dweight[v] = scale * sum of dy over the tokens of v: up to 2048 tokens direct_kernel; more are
// gathered into one list per id and each id's rows are added in token order, so every row of dweight is
// written exactly once, by one wave, and the sums do not depend on timing:
//   count    how many tokens each id has, and each token's place among its id's (in no order: whoever
//            adds to the count first)
//   place    each id takes a stretch of the list (any order between ids), cut into pieces of kPiece
//            tokens where it has more
//   fill     tokens into their id's stretch
//   order    stretches above kPiece tokens copied in token order: up to kRank tokens by counting the
//            smaller ones, more by walking all ids in order and keeping the id's
//   reduce   one wave an id and 64 packs of columns: the sum of its rows, sorted by the wave itself up
//            to kPiece tokens; pieces of longer stretches give partial sums (other workgroups of this
//            launch write zeros for ids without tokens)
//   join     the partial sums of the long stretches, in order
// Words are frequent unevenly, and integer atomics on one address are served one by one (1100 tokens of
// one id among 16384 made the count 14 us, now 6), so a wave adds the tokens of an id at once.
// The bytes that must move are dy read once and dweight written once: 102 MB, 22 us at the rate of a large
// copy, at 16384 tokens (a quarter of them padding), 50000 x 768 bf16. Measured there: 44 us in seven
// launches, of which sums and zeros 17, order 6, count 6, place 5; the plain index_add form takes 310.
#include <type_traits>

#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

constexpr int kPiece = 64;
constexpr int kBatch = 8;   // rows a wave loads at a time (16: 13.0 against 13.1 us at 16384 tokens, and more registers)
constexpr int kRank = 2048;
constexpr int kSlice = 256;  // tokens of a long stretch that one workgroup ranks

template <typename I>
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t t) {
    return (int64_t)static_cast<const I*>(ids)[t];
}

template <typename S, int V, typename I>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const void* ids, const S* weight, S* y, int64_t tokens, int64_t vocab,
                                                        int64_t dim, float scale) {
    using P = Pack<S, V>;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tokens; t += waves) {
        const int64_t id = id_at<I>(ids, t);
        const bool ok = id >= 0 && id < vocab;
        const S* src = weight + (ok ? id : 0) * dim;
        S* dst = y + t * dim;
        for (int64_t c = (int64_t)lane * V; c < dim; c += 64 * V) {
            P v;
            if (ok) {
                v = *reinterpret_cast<const P*>(src + c);
#pragma unroll
                for (int j = 0; j < V; ++j) v.v[j] = from_f32<S>(to_f32(v.v[j]) * scale);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v.v[j] = from_f32<S>(0.0f);
            }
            *reinterpret_cast<P*>(dst + c) = v;
        }
    }
}

// The workspace of the gradient.
struct Lists {
    int* totals;      // {list length, ids with up to kPiece tokens, ids with more, pieces}
    int* count;       // (vocab) tokens of each id
    int* start;       // (vocab) where its stretch begins
    int* place;       // (tokens) a token's place in it
    int* list;        // (tokens) the stretches
    int* sorted;      // (tokens) those of the longs in token order, at the same places
    int* shorts;      // ids with up to kPiece tokens
    int* longs;       // ids with more
    int* long_piece;  // their first piece
    int* piece_id;    // of each piece: its id, and which of the id's pieces it is
    int* piece_at;
    float* part;      // (pieces, dim)
    int64_t clear;    // ints from `totals` to zero
    int64_t max_short, max_long, max_piece, bytes;
};

Lists lists_of(void* ws, const mamba_embedding_shape& s) {
    Lists l{};
    char* p = static_cast<char*>(ws);
    int64_t o = 0;
    auto take = [&](int64_t ints) {
        int* q = reinterpret_cast<int*>(p + o);
        o = align256(o + ints * 4);
        return q;
    };
    l.max_short = s.tokens < s.vocab ? s.tokens : s.vocab;
    l.max_long = s.tokens / (kPiece + 1);
    if (l.max_long > s.vocab) l.max_long = s.vocab;
    l.max_piece = l.max_long > 0 ? s.tokens / kPiece + l.max_long : 0;
    l.totals = take(4);
    l.count = take(s.vocab);
    l.clear = o / 4;  // totals and count lie together at the start
    l.start = take(s.vocab);
    l.place = take(s.tokens);
    l.list = take(s.tokens);
    l.sorted = take(l.max_long > 0 ? s.tokens : 0);
    l.shorts = take(l.max_short);
    l.longs = take(l.max_long);
    l.long_piece = take(l.max_long);
    l.piece_id = take(l.max_piece);
    l.piece_at = take(l.max_piece);
    l.part = reinterpret_cast<float*>(take(l.max_piece * s.dim));
    l.bytes = o;
    return l;
}

__global__ __launch_bounds__(256) void zero_kernel(int* p, int64_t n) {
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) p[k] = 0;
}

// The lanes of a wave that hold the same id: how many, the first of them, and this lane's rank.
struct Mates {
    int n, first, rank;
};
__device__ __forceinline__ Mates mates_of(int id, bool ok, int bits, int lane) {  // ids below 2^bits
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(id >> b & 1);
        same &= id >> b & 1 ? set : ~set;
    }
    return Mates{(int)__popcll(same), (int)__builtin_ctzll(same | (uint64_t)1 << 63),
                 (int)__popcll(same & (((uint64_t)1 << lane) - 1))};
}

template <typename I>
__global__ __launch_bounds__(256) void count_kernel(const void* ids, int64_t tokens, int64_t vocab, int bits, Lists l) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int lane = threadIdx.x & 63;
    const int64_t id = t < tokens ? id_at<I>(ids, t) : -1;
    const bool ok = id >= 0 && id < vocab;
    const Mates m = mates_of((int)id, ok, bits, lane);
    int base = 0;
    if (ok && m.first == lane) base = atomicAdd(&l.count[id], m.n);
    base = __shfl(base, m.first, 64);
    if (ok) l.place[t] = base + m.rank;
}

// Exclusive prefix sum over a workgroup of 1024, and the total in `all`; `lds` holds 16 values of its own.
__device__ __forceinline__ int group_prefix(int v, int* lds, int& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(sum, m, 64);
        if (lane >= m) sum += o;
    }
    if (lane == 63) lds[wave] = sum;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        before += w < wave ? lds[w] : 0;
        all += lds[w];
    }
    return before + sum - v;
}

__global__ __launch_bounds__(1024) void place_kernel(int64_t vocab, Lists l) {
    __shared__ int lds[4][16], base[4];
    const int64_t v = (int64_t)blockIdx.x * 1024 + threadIdx.x;
    const int n = v < vocab ? l.count[v] : 0;
    const bool few = n > 0 && n <= kPiece, many = n > kPiece;
    const int pieces = many ? (n + kPiece - 1) / kPiece : 0;
    int all[4];
    const int at = group_prefix(n, lds[0], all[0]), sh = group_prefix(few, lds[1], all[1]);
    const int lg = group_prefix(many, lds[2], all[2]), pc = group_prefix(pieces, lds[3], all[3]);
    if (threadIdx.x < 4 && all[0] > 0) {
        const int mine = threadIdx.x == 0 ? all[0] : threadIdx.x == 1 ? all[1] : threadIdx.x == 2 ? all[2] : all[3];
        base[threadIdx.x] = mine ? atomicAdd(&l.totals[threadIdx.x], mine) : 0;
    }
    __syncthreads();
    if (all[0] == 0 || v >= vocab) return;
    l.start[v] = base[0] + at;
    if (few) l.shorts[base[1] + sh] = (int)v;
    if (many) {
        l.longs[base[2] + lg] = (int)v;
        const int first = base[3] + pc;
        l.long_piece[base[2] + lg] = first;
        for (int q = 0; q < pieces; ++q) {
            l.piece_id[first + q] = (int)v;
            l.piece_at[first + q] = q;
        }
    }
}

template <typename I>
__global__ __launch_bounds__(256) void fill_kernel(const void* ids, int64_t tokens, int64_t vocab, Lists l) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= tokens) return;
    const int64_t id = id_at<I>(ids, t);
    if (id >= 0 && id < vocab) l.list[l.start[id] + l.place[t]] = (int)t;
}

constexpr int kZeroIds = 16;  // ids a workgroup looks at for rows of zeros

// Rows of zeros for the ids without tokens among kZeroIds.
__device__ __forceinline__ void zero_rows(char* dweight, int64_t row_bytes, int64_t v0, int64_t vocab, const int* count) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k = wave; k < kZeroIds; k += 4) {
        const int64_t v = v0 + k;
        if (v >= vocab || count[v] != 0) continue;
        char* row = dweight + v * row_bytes;
        if (row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
            for (int64_t c = lane * 16; c < row_bytes; c += 64 * 16) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
        } else if (reinterpret_cast<uintptr_t>(row) % 4 == 0 && row_bytes % 4 == 0) {
            for (int64_t c = lane * 4; c < row_bytes; c += 64 * 4) *reinterpret_cast<uint32_t*>(row + c) = 0;
        } else {
            for (int64_t c = lane * 2; c < row_bytes; c += 64 * 2) *reinterpret_cast<uint16_t*>(row + c) = 0;
        }
    }
}

// Long stretches put into order, slice by slice.
template <typename I>
__global__ __launch_bounds__(1024) void order_kernel(const void* ids, int64_t tokens, Lists l) {
    __shared__ __align__(16) int s_tok[kRank + 16];
    __shared__ int s_part[4][kSlice];
    constexpr int U = 8;  // of 1024 ids walked at a time
    __shared__ int s_hits[U][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int slices = kRank / kSlice;
    const int slice = blockIdx.x % slices;
    for (int q = blockIdx.x / slices; q < l.totals[2]; q += gridDim.x / slices) {
        const int id = l.longs[q], n = l.count[id], start = l.start[id];
        if (n <= kRank) {
            const int k0 = slice * kSlice;
            if (k0 >= n) continue;
            for (int k = threadIdx.x; k < n + 15; k += 1024) s_tok[k] = k < n ? l.list[start + k] : 0x7fffffff;
            __syncthreads();
            // 4 threads count for each token of the slice, a quarter of the stretch each
            const int k = k0 + (threadIdx.x & (kSlice - 1)), part = threadIdx.x / kSlice;
            const int quarter = ((n + 3) / 4 + 3) / 4 * 4;
            const int mine = k < n ? s_tok[k] : 0;
            int rank = 0;
#pragma unroll 4
            for (int j = part * quarter; j < (part + 1) * quarter && j < n; j += 4) {
                const int4 o = *reinterpret_cast<const int4*>(&s_tok[j]);
                rank += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
            }
            s_part[part][threadIdx.x & (kSlice - 1)] = rank;
            __syncthreads();
            if (part == 0 && k < n) l.sorted[start + rank + s_part[1][threadIdx.x] + s_part[2][threadIdx.x] + s_part[3][threadIdx.x]] = mine;
            __syncthreads();
        } else if (slice == 0) {
            int base = 0;
            for (int64_t t0 = 0; t0 < tokens && base < n; t0 += 1024 * U) {
                uint64_t hits[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t t = t0 + u * 1024 + threadIdx.x;
                    hits[u] = __ballot(t < tokens && id_at<I>(ids, t < tokens ? t : 0) == id);
                    if (lane == 0) s_hits[u][wave] = (int)__popcll(hits[u]);
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    int before = 0, all = 0;
                    for (int w = 0; w < 16; ++w) {
                        before += w < wave ? s_hits[u][w] : 0;
                        all += s_hits[u][w];
                    }
                    if (hits[u] >> lane & 1)
                        l.sorted[start + base + before + __popcll(hits[u] & (((uint64_t)1 << lane) - 1))] =
                            (int)(t0 + u * 1024 + threadIdx.x);
                    base += all;
                }
                __syncthreads();
            }
        }
    }
}

// The sum of up to kPiece rows of dy at the lane's pack of columns, row k being lane k's token.
template <typename S, int V>
__device__ __forceinline__ void sum_rows(const S* dy, int64_t dim, int64_t c, int tok, int n, float (&s)[V]) {
    using P = Pack<S, V>;
    const S* at = dy + (c < dim ? c : 0);  // lanes past the row read its beginning: no branch around the loads
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.0f;
    // rows k .. k + U - 1, of which the first `left` count (the others repeat the last one)
    auto add = [&](int k, int left, auto many) __attribute__((always_inline)) {
        constexpr int U = decltype(many)::value;
        P v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = __builtin_amdgcn_readlane(tok, u < left ? k + u : k + left - 1);
            v[u] = *reinterpret_cast<const P*>(at + t * dim);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += u < left ? to_f32(v[u].v[j]) : 0.0f;
    };
    int k = 0;
    for (; k + kBatch <= n; k += kBatch) add(k, kBatch, std::integral_constant<int, kBatch>{});
    if (n - k > 4) add(k, n - k, std::integral_constant<int, kBatch>{});
    else if (n - k > 1) add(k, n - k, std::integral_constant<int, 4>{});
    else if (n - k == 1) add(k, 1, std::integral_constant<int, 1>{});
}

// What the lanes of a wave wrote to LDS before is what its lanes read after. A wave's accesses to LDS are in
// order as it is; this keeps the compiler's order too, and is no instruction.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The tokens of kGroupIds ids, from v0 up, among all: a workgroup of 16 waves looks through up to G groups of
// 64 tokens a wave, one stretch of the list each. s_sorted receives them by id and in token order, those of
// v0 + k from s_start[k] to s_start[k + 1].
constexpr int kGroupIds = 64;

template <int G, typename I>
__device__ __forceinline__ void find_tokens(const void* ids, int tokens, int64_t v0, int64_t vocab, uint16_t* s_sorted,
                                            int (&s_at)[16][kGroupIds], int (&s_start)[kGroupIds + 1]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    const int stretch = (tokens + 1023) / 1024 * 64, begin = wave * stretch;
    const int mine = tokens - begin < stretch ? tokens - begin : stretch;  // of this wave; may be negative
    const uint32_t first = (uint32_t)v0, here = (uint32_t)(vocab - v0 < kGroupIds ? vocab - v0 : kGroupIds);
    const I* from = static_cast<const I*>(ids) + (mine > 0 ? begin : 0);
    int local[G];  // the id less v0, or -1
#pragma unroll
    for (int u = 0; u < G; ++u) {
        const int k = u * 64 + lane;
        const I id = mine > 0 ? from[k < mine ? k : 0] : (I)-1;
        const uint32_t d = (uint32_t)id - first;
        bool hit = k < mine && d < here;
        if constexpr (sizeof(I) == 8) hit = hit && (uint32_t)((uint64_t)id >> 32) == 0;
        local[u] = hit ? (int)d : -1;
    }
    s_at[wave][lane] = 0;
    wave_order();
    // each token found, in order, gets the place that s_at has for its id
    auto walk = [&](auto&& to) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const int l = local[u];
            const uint64_t hits = __ballot(l >= 0);
            if (!hits) continue;
            uint64_t same = hits;  // the lanes with this lane's id
#pragma unroll
            for (int b = 0; b < 6; ++b) {
                const uint64_t set = __ballot(l >> b & 1);
                same &= l >> b & 1 ? set : ~set;
            }
            if (l >= 0) {
                const int at = s_at[wave][l], rank = (int)__popcll(same & below);
                to(at + rank, begin + u * 64 + lane);
                if (rank == 0) s_at[wave][l] = at + (int)__popcll(same);
            }
            wave_order();
        }
    };
    walk([](int, int) {});
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const int n = s_at[w][lane];
        before += w < wave ? n : 0;
        total += n;
    }
    int sum = total;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const int o = __shfl_up(sum, k, 64);
        if (lane >= k) sum += o;
    }
    __syncthreads();
    s_at[wave][lane] = sum - total + before;
    wave_order();
    if (wave == 0) {
        s_start[lane] = sum - total;
        if (lane == 63) s_start[kGroupIds] = sum;
    }
    walk([&](int at, int t) { s_sorted[at] = (uint16_t)t; });
    __syncthreads();
}

// The whole gradient of few tokens in one launch and no workspace: a workgroup takes 64 ids and 64 packs of
// columns, finds its ids' tokens among all of them, in order, and its 16 waves take an id in turn; those
// with more than kPiece tokens afterwards, a piece a wave. The sums are those of the launches above, bit
// for bit. Bound by its launch for few tokens, then by the workgroup that has the most frequent ids; with the
// call's host side, this and the launches above, at uneven frequencies: 128 tokens, 1000 x 256 bf16 12.4 and
// 34.7 us, 1500 tokens, 5000 x 1024 21.6 and 35.5, 2000 tokens, 50000 x 768 33.5 and 44.4; 1500 tokens,
// 200 x 2048 24.9 and 34.5. The same search through more tokens, with long lists left to a second launch, was
// slower than counting (16384 tokens, 50000 x 768: 57 us against 48), as each group of ids reads them all.
constexpr int kDirect = 2048, kDirectLongs = kDirect / (kPiece + 1), kDirectPieces = kDirect / kPiece + kDirectLongs;
// (65536 blocks of columns at most; 16 threads an id, whose number has to stay below 2^32)
bool direct(const mamba_embedding_shape& s) { return s.tokens <= kDirect && s.dim <= 1 << 16 && s.vocab <= 1 << 27; }

template <typename S, int V, typename I>
__global__ __launch_bounds__(1024) void direct_kernel(const void* ids, int tokens, int64_t vocab, const S* dy, S* dweight,
                                                      int64_t dim, float scale) {
    using P = Pack<S, V>;
    __shared__ uint16_t s_sorted[kDirect];
    __shared__ int s_at[16][kGroupIds], s_start[kGroupIds + 1], s_longs[kDirectLongs], s_nlong;
    __shared__ float s_part[kDirectPieces][64 * V];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t v0 = (int64_t)blockIdx.x * kGroupIds, c = (int64_t)blockIdx.y * 64 * V + lane * V;
    if (threadIdx.x == 0) s_nlong = 0;
    find_tokens<kDirect / 1024, I>(ids, tokens, v0, vocab, s_sorted, s_at, s_start);

    auto store = [&](int64_t v, const float* s) {
        if (c >= dim) return;
        P o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = from_f32<S>(s[j] * scale);
        *reinterpret_cast<P*>(dweight + v * dim + c) = o;
    };
    for (int local = wave; local < kGroupIds && v0 + local < vocab; local += 16) {
        const int from = s_start[local], n = s_start[local + 1] - from;
        if (n > kPiece) {
            if (lane == 0) s_longs[atomicAdd(&s_nlong, 1)] = local;
            continue;
        }
        float s[V];
        sum_rows<S, V>(dy, dim, c, lane < n ? s_sorted[from + lane] : 0, n, s);
        store(v0 + local, s);
    }
    __syncthreads();
    const int longs = s_nlong;
    for (int q = 0, p = 0; q < longs; ++q)
        for (int from = s_start[s_longs[q]]; from < s_start[s_longs[q] + 1]; from += kPiece, ++p) {
            if (p % 16 != wave) continue;
            const int left = s_start[s_longs[q] + 1] - from, n = left < kPiece ? left : kPiece;
            float s[V];
            sum_rows<S, V>(dy, dim, c, lane < n ? s_sorted[from + lane] : 0, n, s);
#pragma unroll
            for (int j = 0; j < V; ++j) s_part[p][j * 64 + lane] = s[j];
        }
    __syncthreads();
    for (int q = 0, p = 0; q < longs; ++q) {
        const int l = s_longs[q], pieces = (s_start[l + 1] - s_start[l] + kPiece - 1) / kPiece;
        if (q % 16 == wave) {
            float s[V];
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = 0.0f;
            for (int k = 0; k < pieces; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += s_part[p + k][j * 64 + lane];
            store(v0 + l, s);
        }
        p += pieces;
    }
}

// The pieces and the ids with up to kPiece tokens, a wave for every 64 packs of columns of each, in turns.
// `zeros` workgroups, spread among the others, write the rows of ids without tokens meanwhile: those stream,
// while the sums wait for rows from all over dy (as launches of their own 10 and 12 us, together 17).
template <typename S, int V>
__global__ __launch_bounds__(256) void reduce_kernel(const S* dy, S* dweight, int64_t dim, float scale, Lists l, int zeros,
                                                     int64_t vocab) {
    using P = Pack<S, V>;
    const int64_t id_block = grid_block(), all = grid_blocks(), zero = id_block * zeros / all;
    if ((id_block + 1) * zeros / all > zero) {
        zero_rows(reinterpret_cast<char*>(dweight), dim * (int64_t)sizeof(S), zero * kZeroIds, vocab, l.count);
        return;
    }
    const int64_t block = id_block - zero, blocks = all - zeros;
    const int lane = threadIdx.x & 63;
    const int cols = (int)((dim + 64 * V - 1) / (64 * V));
    const int pieces = l.totals[3], shorts = l.totals[1];
    const int64_t items = (int64_t)(pieces + shorts) * cols, step = blocks * 4;
    for (int64_t k = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); k < items; k += step) {
        const int64_t q = k / cols, c = (k - q * cols) * 64 * V + lane * V;
        const bool whole = q >= pieces;  // of an id's tokens
        const int id = __builtin_amdgcn_readfirstlane(whole ? l.shorts[q - pieces] : l.piece_id[q]);
        const int from = whole ? 0 : __builtin_amdgcn_readfirstlane(l.piece_at[q]) * kPiece;
        const int left = __builtin_amdgcn_readfirstlane(l.count[id]) - from, n = left < kPiece ? left : kPiece;
        int tok = lane < n ? (whole ? l.list : l.sorted)[l.start[id] + from + lane] : 0;
        if (whole && n > 1) {  // into token order: each lane's rank among the wave's tokens, then the token sent there
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += __builtin_amdgcn_readlane(tok, j) < tok;
            tok = __builtin_amdgcn_ds_permute((lane < n ? rank : lane) * 4, tok);
        }
        float s[V];
        sum_rows<S, V>(dy, dim, c, tok, n, s);
        if (c >= dim) continue;
        if (whole) {
            P o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = from_f32<S>(s[j] * scale);
            *reinterpret_cast<P*>(dweight + (int64_t)id * dim + c) = o;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) l.part[q * dim + c + j] = s[j];
        }
    }
}

template <typename S>
__global__ __launch_bounds__(256) void join_kernel(S* dweight, int64_t dim, float scale, Lists l) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= dim) return;
    for (int q = blockIdx.y; q < l.totals[2]; q += gridDim.y) {
        const int id = l.longs[q], pieces = (l.count[id] + kPiece - 1) / kPiece;
        const float* part = l.part + (int64_t)l.long_piece[q] * dim + c;
        float s = 0.0f;
#pragma unroll 8
        for (int k = 0; k < pieces; ++k) s += part[(int64_t)k * dim];
        dweight[(int64_t)id * dim + c] = from_f32<S>(s * scale);
    }
}

template <typename S, int V, typename I>
void fwd_go(const void* ids, const void* w, void* y, const mamba_embedding_shape& s, float scale, Launches& on) {
    const int64_t need = (s.tokens + 3) / 4, most = (int64_t)layers_cus() * 64;
    on(embed_fwd_kernel<S, V, I>, dim3((unsigned)(need < most ? need : most)), dim3(256), ids,
       static_cast<const S*>(w), static_cast<S*>(y), s.tokens, s.vocab, s.dim, scale);
}

// The widest pack (16 bytes and down) that rows of `dim` elements at both pointers are multiples of.
template <typename S, int V = 16 / sizeof(S), typename F>
void with_pack(int64_t dim, const void* a, const void* b, F&& f) {
    if constexpr (V == 1) {
        f(std::integral_constant<int, 1>{});
    } else {
        const bool ok = dim % V == 0 && (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % (V * sizeof(S)) == 0;
        ok ? f(std::integral_constant<int, V>{}) : with_pack<S, V / 2>(dim, a, b, f);
    }
}

template <typename S, typename I>
void fwd_typed(const void* ids, const void* w, void* y, const mamba_embedding_shape& s, float scale, Launches& on) {
    with_pack<S>(s.dim, w, y, [&](auto v) { fwd_go<S, decltype(v)::value, I>(ids, w, y, s, scale, on); });
}

template <typename S, typename I>
void bwd_typed(const void* ids, const void* dy, void* dw, void* ws, const mamba_embedding_shape& s, float scale,
               Launches& on) {
    if (direct(s)) {
        with_pack<S>(s.dim, dy, dw, [&](auto v) {
            constexpr int V = decltype(v)::value;
            const dim3 grid((unsigned)((s.vocab + kGroupIds - 1) / kGroupIds), (unsigned)((s.dim + 64 * V - 1) / (64 * V)));
            on(direct_kernel<S, V, I>, grid, dim3(1024), ids, (int)s.tokens, s.vocab,
               static_cast<const S*>(dy), static_cast<S*>(dw), s.dim, scale);
        });
        return;
    }
    const Lists l = lists_of(ws, s);
    auto grid = [](int64_t n, int64_t per) { return dim3((unsigned)((n + per - 1) / per)); };
    const int64_t zb = (l.clear + 255) / 256;
    int bits = 0;
    while ((s.vocab - 1) >> bits > 0) ++bits;
    on(zero_kernel, dim3((unsigned)(zb < 2048 ? zb : 2048)), dim3(256), l.totals, l.clear);
    if (s.tokens > 0) {  // (a wide row of no tokens comes here too)
        on(count_kernel<I>, grid(s.tokens, 256), dim3(256), ids, s.tokens, s.vocab, bits, l);
        on(place_kernel, grid(s.vocab, 1024), dim3(1024), s.vocab, l);
        on(fill_kernel<I>, grid(s.tokens, 256), dim3(256), ids, s.tokens, s.vocab, l);
    }
    const unsigned longs = (unsigned)(l.max_long < 512 ? l.max_long : 512);
    if (longs)
        on(order_kernel<I>, dim3(longs * (kRank / kSlice)), dim3(1024), ids, s.tokens, l);
    with_pack<S>(s.dim, dy, dw, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const int64_t waves = (l.max_piece + l.max_short) * ((s.dim + 64 * V - 1) / (64 * V)), most = (int64_t)layers_cus() * 64;
        const int64_t zeros = (s.vocab + kZeroIds - 1) / kZeroIds, sums = ((waves < most ? waves : most) + 3) / 4;
        on(reduce_kernel<S, V>, grid_of(zeros + sums, 256), dim3(256), static_cast<const S*>(dy),
           static_cast<S*>(dw), s.dim, scale, l, (int)zeros, s.vocab);
    });
    if (longs)
        on(join_kernel<S>, dim3((unsigned)((s.dim + 255) / 256), longs), dim3(256),
           static_cast<S*>(dw), s.dim, scale, l);
}

}  // namespace

int64_t embedding_bwd_workspace(const mamba_embedding_shape& s) { return direct(s) ? 0 : lists_of(nullptr, s).bytes; }

int launch_embedding_fwd(const void* ids, bool ids64, const void* weight, void* y, const mamba_embedding_shape& s, float scale,
                         bool bf16, hipStream_t stream) {
    Launches on(stream);
    if (bf16)
        ids64 ? fwd_typed<bf16_t, int64_t>(ids, weight, y, s, scale, on)
              : fwd_typed<bf16_t, int32_t>(ids, weight, y, s, scale, on);
    else
        ids64 ? fwd_typed<float, int64_t>(ids, weight, y, s, scale, on)
              : fwd_typed<float, int32_t>(ids, weight, y, s, scale, on);
    return on.status;
}

int launch_embedding_bwd(const void* ids, bool ids64, const void* dy, void* dweight, void* ws, const mamba_embedding_shape& s,
                         float scale, bool bf16, hipStream_t stream) {
    Launches on(stream);
    if (bf16)
        ids64 ? bwd_typed<bf16_t, int64_t>(ids, dy, dweight, ws, s, scale, on)
              : bwd_typed<bf16_t, int32_t>(ids, dy, dweight, ws, s, scale, on);
    else
        ids64 ? bwd_typed<float, int64_t>(ids, dy, dweight, ws, s, scale, on)
              : bwd_typed<float, int32_t>(ids, dy, dweight, ws, s, scale, on);
    return on.status;
}

}  // namespace mscan
