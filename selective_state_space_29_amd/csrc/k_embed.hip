// Token embedding and its gradient (mamba_layers.h) on gfx950.
//
// Forward: one wave a token, 16 bytes a lane where rows allow it; bound by HBM.
//
// Gradient: dweight[v] = scale * sum of dy over the tokens of v. The tokens are gathered into one
// list per id and each id's rows are added in token order, so every row of dweight is written exactly
// once, by one wave, and the sums do not depend on timing:
//   count    how many tokens each id has (integer atomics)
//   place    each id takes a stretch of the list (any order between ids), cut into pieces of kPiece
//            tokens where it has more
//   fill     tokens into their id's stretch, in any order (integer atomics)
//   order    stretches above kPiece tokens put into token order: up to kRank tokens by counting the
//            smaller ones, more by walking all ids in order and keeping the id's
//   reduce   one wave an id: zeros, or the sum of its rows, sorted by the wave itself up to kPiece
//            tokens; pieces of longer stretches give partial sums
//   join     the partial sums of the long stretches, in order
// The bytes that must move are dy read once and dweight written once.
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace mscan {

namespace {

constexpr int kPiece = 64;
constexpr int kRank = 2048;

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
    int* count;    // (vocab) tokens of each id
    int* start;    // (vocab) where its stretch begins
    int* cursor;   // (vocab) places taken
    int* list;     // (tokens) the stretches
    int* longs;    // ids with more than kPiece tokens
    int* long_piece;  // their first piece
    int* piece_id;    // of each piece: its id, and which of the id's pieces it is
    int* piece_at;
    int* totals;   // {list length, longs, pieces}
    float* part;   // (pieces, dim)
    int64_t clear;  // ints from `count` to zero
    int64_t max_long, max_piece, bytes;
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
    l.max_long = s.tokens / (kPiece + 1) + 1;
    l.max_piece = s.tokens / kPiece + l.max_long;
    l.totals = take(4);
    l.count = take(s.vocab);
    l.cursor = take(s.vocab);
    l.clear = o / 4;  // totals, count and cursor lie together at the start
    l.start = take(s.vocab);
    l.list = take(s.tokens);
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

template <typename I>
__global__ __launch_bounds__(256) void count_kernel(const void* ids, int64_t tokens, int64_t vocab, Lists l) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= tokens) return;
    const int64_t id = id_at<I>(ids, t);
    if (id >= 0 && id < vocab) atomicAdd(&l.count[id], 1);
}

__global__ __launch_bounds__(256) void place_kernel(int64_t vocab, Lists l) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int lane = threadIdx.x & 63;
    const int n = v < vocab ? l.count[v] : 0;
    int before = n;  // inclusive prefix sum over the wave
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(before, m, 64);
        if (lane >= m) before += o;
    }
    int base = 0;
    if (lane == 63) base = atomicAdd(&l.totals[0], before);
    base = __shfl(base, 63, 64);
    if (v < vocab) l.start[v] = base + before - n;
    if (n > kPiece) {
        const int pieces = (n + kPiece - 1) / kPiece;
        const int at = atomicAdd(&l.totals[1], 1), first = atomicAdd(&l.totals[2], pieces);
        l.longs[at] = (int)v;
        l.long_piece[at] = first;
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
    if (id >= 0 && id < vocab) l.list[l.start[id] + atomicAdd(&l.cursor[id], 1)] = (int)t;
}

template <typename I>
__global__ __launch_bounds__(1024) void order_kernel(const void* ids, int64_t tokens, Lists l) {
    __shared__ int s_tok[kRank];
    __shared__ int s_wave[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int q = blockIdx.x; q < l.totals[1]; q += gridDim.x) {
        const int id = l.longs[q], n = l.count[id];
        int* list = l.list + l.start[id];
        if (n <= kRank) {
            for (int k = threadIdx.x; k < n; k += 1024) s_tok[k] = list[k];
            __syncthreads();
            for (int k = threadIdx.x; k < n; k += 1024) {
                const int mine = s_tok[k];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += s_tok[j] < mine;
                list[rank] = mine;
            }
            __syncthreads();
        } else {
            int base = 0;
            for (int64_t t0 = 0; t0 < tokens && base < n; t0 += 1024) {
                const int64_t t = t0 + threadIdx.x;
                const bool hit = t < tokens && id_at<I>(ids, t) == id;
                const uint64_t m = __ballot(hit);
                if (lane == 0) s_wave[wave] = __popcll(m);
                __syncthreads();
                int before = 0, all = 0;
                for (int w = 0; w < 16; ++w) {
                    before += w < wave ? s_wave[w] : 0;
                    all += s_wave[w];
                }
                if (hit) list[base + before + __popcll(m & (((uint64_t)1 << lane) - 1))] = (int)t;
                base += all;
                __syncthreads();
            }
        }
    }
}

// Rows of dweight, one wave each: waves below vocab own an id, the following ones a piece.
template <typename S, int V>
__global__ __launch_bounds__(256) void reduce_kernel(const S* dy, S* dweight, int64_t vocab, int64_t dim, float scale, Lists l) {
    using P = Pack<S, V>;
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int id, n, tok = 0;
    float* part = nullptr;
    if (wave < vocab) {
        id = (int)wave;
        n = l.count[id];
        if (n > kPiece) return;
        if (lane < n) tok = l.list[l.start[id] + lane];
        // into token order: each lane's rank among the wave's tokens, then the token sent there
        int rank = lane;
        if (n > 1) {
            rank = 0;
            for (int j = 0; j < n; ++j) rank += __builtin_amdgcn_readlane(tok, j) < tok;
            if (lane >= n) rank = lane;
        }
        tok = __builtin_amdgcn_ds_permute(rank * 4, tok);
    } else {
        const int64_t q = wave - vocab;
        if (q >= l.totals[2]) return;
        id = l.piece_id[q];
        const int from = l.piece_at[q] * kPiece;
        n = l.count[id] - from < kPiece ? l.count[id] - from : kPiece;
        if (lane < n) tok = l.list[l.start[id] + from + lane];
        part = l.part + q * dim;
    }
    for (int64_t c = (int64_t)lane * V; c - (int64_t)lane * V < dim; c += 64 * V) {
        const bool in = c < dim;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.0f;
        int k = 0;
        for (; k + 4 <= n; k += 4) {
            P v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t t = __builtin_amdgcn_readlane(tok, k + u);
                if (in) v[u] = *reinterpret_cast<const P*>(dy + t * dim + c);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += to_f32(v[u].v[j]);
        }
        for (; k < n; ++k) {
            const int64_t t = __builtin_amdgcn_readlane(tok, k);
            P v;
            if (in) v = *reinterpret_cast<const P*>(dy + t * dim + c);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += to_f32(v.v[j]);
        }
        if (!in) continue;
        if (part) {
#pragma unroll
            for (int j = 0; j < V; ++j) part[c + j] = s[j];
        } else {
            P o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = from_f32<S>(s[j] * scale);
            *reinterpret_cast<P*>(dweight + (int64_t)id * dim + c) = o;
        }
    }
}

template <typename S>
__global__ __launch_bounds__(256) void join_kernel(S* dweight, int64_t dim, float scale, Lists l) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= dim) return;
    for (int q = blockIdx.y; q < l.totals[1]; q += gridDim.y) {
        const int id = l.longs[q], pieces = (l.count[id] + kPiece - 1) / kPiece;
        const float* part = l.part + (int64_t)l.long_piece[q] * dim + c;
        float s = 0.0f;
#pragma unroll 8
        for (int k = 0; k < pieces; ++k) s += part[(int64_t)k * dim];
        dweight[(int64_t)id * dim + c] = from_f32<S>(s * scale);
    }
}

template <typename S, int V, typename I>
int fwd_go(const void* ids, const void* w, void* y, const mamba_embedding_shape& s, float scale, hipStream_t stream) {
    const int64_t need = (s.tokens + 3) / 4, most = (int64_t)layers_cus() * 64;
    hipLaunchKernelGGL((embed_fwd_kernel<S, V, I>), dim3((unsigned)(need < most ? need : most)), dim3(256), 0, stream, ids,
                       static_cast<const S*>(w), static_cast<S*>(y), s.tokens, s.vocab, s.dim, scale);
    return launch_status();
}

template <typename S, typename I>
int fwd_typed(const void* ids, const void* w, void* y, const mamba_embedding_shape& s, float scale, hipStream_t stream) {
    constexpr int V = 16 / sizeof(S);
    const bool ok = s.dim % V == 0 && (reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(y)) % 16 == 0;
    return ok ? fwd_go<S, V, I>(ids, w, y, s, scale, stream) : fwd_go<S, 1, I>(ids, w, y, s, scale, stream);
}

template <typename S, typename I>
int bwd_typed(const void* ids, const void* dy, void* dw, void* ws, const mamba_embedding_shape& s, float scale,
              hipStream_t stream) {
    const Lists l = lists_of(ws, s);
    auto grid = [](int64_t n, int64_t per) { return dim3((unsigned)((n + per - 1) / per)); };
    const int64_t zb = (l.clear + 255) / 256;
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(zb < 2048 ? zb : 2048)), dim3(256), 0, stream, l.totals, l.clear);
    if (s.tokens > 0) hipLaunchKernelGGL((count_kernel<I>), grid(s.tokens, 256), dim3(256), 0, stream, ids, s.tokens, s.vocab, l);
    hipLaunchKernelGGL(place_kernel, grid(s.vocab, 256), dim3(256), 0, stream, s.vocab, l);
    if (s.tokens > 0) hipLaunchKernelGGL((fill_kernel<I>), grid(s.tokens, 256), dim3(256), 0, stream, ids, s.tokens, s.vocab, l);
    const bool longs = s.tokens > kPiece;
    if (longs)
        hipLaunchKernelGGL((order_kernel<I>), dim3((unsigned)(l.max_long < 512 ? l.max_long : 512)), dim3(1024), 0, stream, ids,
                           s.tokens, l);
    const int64_t waves = s.vocab + (longs ? l.max_piece : 0);
    constexpr int V = 16 / sizeof(S);
    const bool ok = s.dim % V == 0 && (reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dw)) % 16 == 0;
    if (ok)
        hipLaunchKernelGGL((reduce_kernel<S, V>), grid(waves, 4), dim3(256), 0, stream, static_cast<const S*>(dy),
                           static_cast<S*>(dw), s.vocab, s.dim, scale, l);
    else
        hipLaunchKernelGGL((reduce_kernel<S, 1>), grid(waves, 4), dim3(256), 0, stream, static_cast<const S*>(dy),
                           static_cast<S*>(dw), s.vocab, s.dim, scale, l);
    if (longs)
        hipLaunchKernelGGL((join_kernel<S>), dim3((unsigned)((s.dim + 255) / 256), (unsigned)(l.max_long < 512 ? l.max_long : 512)),
                           dim3(256), 0, stream, static_cast<S*>(dw), s.dim, scale, l);
    return launch_status();
}

}  // namespace

int64_t embedding_bwd_workspace(const mamba_embedding_shape& s) { return lists_of(nullptr, s).bytes; }

int launch_embedding_fwd(const void* ids, bool ids64, const void* weight, void* y, const mamba_embedding_shape& s, float scale,
                         bool bf16, hipStream_t stream) {
    if (bf16)
        return ids64 ? fwd_typed<bf16_t, int64_t>(ids, weight, y, s, scale, stream)
                     : fwd_typed<bf16_t, int32_t>(ids, weight, y, s, scale, stream);
    return ids64 ? fwd_typed<float, int64_t>(ids, weight, y, s, scale, stream)
                 : fwd_typed<float, int32_t>(ids, weight, y, s, scale, stream);
}

int launch_embedding_bwd(const void* ids, bool ids64, const void* dy, void* dweight, void* ws, const mamba_embedding_shape& s,
                         float scale, bool bf16, hipStream_t stream) {
    if (bf16)
        return ids64 ? bwd_typed<bf16_t, int64_t>(ids, dy, dweight, ws, s, scale, stream)
                     : bwd_typed<bf16_t, int32_t>(ids, dy, dweight, ws, s, scale, stream);
    return ids64 ? bwd_typed<float, int64_t>(ids, dy, dweight, ws, s, scale, stream)
                 : bwd_typed<float, int32_t>(ids, dy, dweight, ws, s, scale, stream);
}

}  // namespace mscan
