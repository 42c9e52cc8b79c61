// kernels_accept.hip -- the accepted path of a tree of drafted tokens, and the move
// of its slots.
#include <hip/hip_runtime.h>

#include "../ecmd_launch.h"
#include "ecmd_serving.h"
#include "ecmd_wave.h"

namespace ecmd {

namespace {

constexpr uint32_t kPerLane = kMaxTree / 64;

// One wave to a row, four tokens to a lane.  A step of the path is a comparison of all
// tokens' parents and names at once and the first that fits, so it takes two exchanges
// and no memory: the chain of steps is what the time goes to (128 rows of eight guesses of seven
// tokens: 3.3 us, one of four of five: 2.1; the smallest kernel takes about 2).
__global__ __launch_bounds__(64) void k_accept(const AcceptArgs A)
{
    __shared__ int32_t s_next[kMaxTree], s_path[kMaxTree];
    const uint32_t r = blockIdx.x, lane = threadIdx.x;
    int32_t token[kPerLane], parent[kPerLane];
#pragma unroll
    for (uint32_t k = 0; k < kPerLane; ++k) {
        const uint32_t i = k * 64 + lane;
        token[k] = 0;
        parent[k] = -2;
        s_path[i] = -1;
        if (i < A.t) {
            token[k] = A.tokens[(int64_t)r * A.tokens_s[0] + (int64_t)i * A.tokens_s[1]];
            parent[k] = A.parent[(int64_t)r * A.parent_s[0] + (int64_t)i * A.parent_s[1]];
            s_next[i] = A.next[(int64_t)r * A.next_s[0] + (int64_t)i * A.next_s[1]];
        }
    }
    const int32_t len = A.lens[(int64_t)r * A.lens_s];
    __syncthreads();
    uint32_t count = 0;
    int32_t last = -1;
    if (A.t && len >= 0 && __builtin_amdgcn_readfirstlane(parent[0]) == -1) {
        int32_t cur = 0;
        while (cur >= 0) {
            if (lane == 0) s_path[count] = cur;
            ++count;
            last = s_next[cur];
            int32_t to = -1;
#pragma unroll
            for (int k = kPerLane - 1; k >= 0; --k) {
                const int32_t i = k * 64 + (int32_t)lane;
                const uint64_t fits = __ballot(parent[k] == cur && token[k] == last && i > cur && (uint32_t)i < A.t);
                if (fits) to = k * 64 + __builtin_ctzll(fits);
            }
            cur = to;
        }
    }
    __syncthreads();
    for (uint32_t i = lane; i < A.t; i += 64) A.path[(int64_t)r * A.path_s[0] + (int64_t)i * A.path_s[1]] = s_path[i];
    if (lane == 0) {
        A.lens_out[(int64_t)r * A.lens_out_s] = count && (uint32_t)len + count > 0x7FFFFFFFu ? 0x7FFFFFFF : len + (int32_t)count;
        A.last[(int64_t)r * A.last_s] = last;
    }
}

template <int W>
struct Vec;
template <>
struct Vec<16> {
    typedef uint32_t T __attribute__((ext_vector_type(4)));
};
template <>
struct Vec<8> {
    typedef uint32_t T __attribute__((ext_vector_type(2)));
};
template <>
struct Vec<4> {
    typedef uint32_t T;
};
template <>
struct Vec<2> {
    typedef uint16_t T;
};

// A work-group to a row, a pool and 256 vectors of a slot.  Every work-item moves its
// own vector of one slot after the other; a path ascends with path[i] >= i, so no
// write reaches a slot that is still to be read, and eight loads may go ahead of their
// writes.  No two work-items share a byte: there is nothing to wait for.  128 rows, up to seven
// tokens each, 16 pools of 2 KB a slot: 7 us for 27 MB, two thirds of it from lengths over paths and
// pages to the first slot.
template <int W, int POOLS>
__global__ __launch_bounds__(256) void k_move(const MoveBlock<POOLS> A)
{
    typedef typename Vec<W>::T V;
    __shared__ int64_t s_from[kMaxTree], s_to[kMaxTree];
    __shared__ uint32_t s_wave[4];
    const uint32_t r = A.by_pieces.div(blockIdx.x), piece = blockIdx.x - r * A.pieces;
    const MovePool &pool = A.pool[blockIdx.y];
    const int32_t len = A.lens[(int64_t)r * A.lens_s];
    if (len < 0) return;
    const uint32_t i = threadIdx.x, held = A.cols * A.page;
    // the path's end: the first negative entry
    int32_t p = -1;
    if (i < A.t) p = A.path[(int64_t)r * A.path_s[0] + (int64_t)i * A.path_s[1]];
    const uint64_t ends = __ballot(p < 0);
    if ((i & 63) == 0) s_wave[i / 64] = ends ? (uint32_t)__builtin_ctzll(ends) : 64;
    __syncthreads();
    uint32_t count = 0;
    bool open = true;
#pragma unroll
    for (uint32_t w = 0; w < 4; ++w) {
        if (open) count += s_wave[w];
        open = open && s_wave[w] == 64;
    }
    // the moves of the path, packed, in order
    int64_t from = 0, to = 0;
    bool moves = i < count && (uint32_t)p > i;
    if (moves) {
        const uint64_t a = (uint64_t)(uint32_t)len + (uint32_t)p, b = (uint64_t)(uint32_t)len + i;
        moves = a < held && b < held;
        if (moves) {
            const uint32_t ca = A.by_page.div((uint32_t)a), cb = A.by_page.div((uint32_t)b);
            const int32_t ia = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)ca * A.pages_s[1]];
            const int32_t ib = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)cb * A.pages_s[1]];
            moves = ia >= 0 && (uint32_t)ia < pool.n && ib >= 0 && (uint32_t)ib < pool.n;
            from = (int64_t)ia * pool.page_stride + (int64_t)((uint32_t)a - ca * A.page) * pool.slot_stride;
            to = (int64_t)ib * pool.page_stride + (int64_t)((uint32_t)b - cb * A.page) * pool.slot_stride;
        }
    }
    const uint64_t these = __ballot(moves);
    __syncthreads();
    if ((i & 63) == 0) s_wave[i / 64] = (uint32_t)__popcll(these);
    __syncthreads();
    uint32_t at = (uint32_t)__popcll(these & ((uint64_t(1) << (i & 63)) - 1)), n = 0;
#pragma unroll
    for (uint32_t w = 0; w < 4; ++w) {
        if (w < i / 64) at += s_wave[w];
        n += s_wave[w];
    }
    if (moves) {
        s_from[at] = from;
        s_to[at] = to;
    }
    __syncthreads();
    const uint32_t v = piece * 256 + i;
    if (v >= A.vecs) return;
    const uint32_t head = pool.by_head.div(v);
    char *base = pool.base + (int64_t)head * pool.head_stride + (int64_t)(v - head * pool.head_vecs) * W;
    for (uint32_t k = 0; k < n; k += 8) {
        V x[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
            if (k + u < n) x[u] = *(const V *)(base + s_from[k + u]);
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
            if (k + u < n) *(V *)(base + s_to[k + u]) = x[u];
    }
}

template <int W>
int launch_move_width(const MoveArgs &A, uint32_t pools, void *stream)
{
    const dim3 grid(A.rows * A.pieces, pools);
    if (pools > (uint32_t)kMoveFew)
        return launch_kernel(reinterpret_cast<const void *>(&k_move<W, kMovePools>), grid, dim3(256), 0, stream, A);
    MoveBlock<kMoveFew> F{A.pages, A.lens, A.path, {A.pages_s[0], A.pages_s[1]}, A.lens_s, {A.path_s[0], A.path_s[1]},
                          A.rows, A.cols, A.t, A.page, A.vecs, A.pieces, A.by_page, A.by_pieces, {}};
    for (uint32_t i = 0; i < pools; ++i) F.pool[i] = A.pool[i];
    return launch_kernel(reinterpret_cast<const void *>(&k_move<W, kMoveFew>), grid, dim3(256), 0, stream, F);
}

}  // namespace

int launch_accept(const AcceptArgs &A, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_accept), dim3(A.rows), dim3(64), 0, stream, A);
}

int launch_move(int width, const MoveArgs &A, uint32_t pools, void *stream)
{
    return width == 16  ? launch_move_width<16>(A, pools, stream)
           : width == 8 ? launch_move_width<8>(A, pools, stream)
           : width == 4 ? launch_move_width<4>(A, pools, stream)
                        : launch_move_width<2>(A, pools, stream);
}

}  // namespace ecmd
