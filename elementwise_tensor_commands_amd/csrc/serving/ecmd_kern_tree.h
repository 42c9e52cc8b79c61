// ecmd_kern_tree.h -- attention for a tree of drafted tokens over a paged key-value
// cache (device code; one translation unit per element type instantiates it).
//
//   out_i = sum_x p_x v_x / sum_x p_x,   p_x = exp(scale q_i . k_x - m_i)
//
// over the row's context and the tokens above i, in one pass with the running
// maximum m_i.  The query vectors of a kv head (T tokens times its query heads)
// are columns of the matrix products, as the query heads are in one token's
// attention: a wave takes NT tiles of 16 of them, so a key's or value's piece that
// is in registers serves NT products.
//
//   scores   D[key][query] = K Q^T; lane (j = lane / 16, h = lane % 16) gets those of
//            query h at keys 16 kb + 4 j + i, i = 0..3.
//   weights  exp2 of those in place, which makes them the operand of
//   out      D[dv][query] += V^T P^T, with lane j loading the values of its keys.
//
// Two kernels.  k_tree_few takes keys and values from memory straight to registers;
// the four waves of a work-group part the positions, or the queries where there are more.
// It serves few queries or positions, where the chain from a row's length to its first key is
// what counts (one row of 777, 8 tokens of 32 heads over 8, f16: 13 us and 4 for the join),
// binary32, whose products run at a sixteenth of the 16-bit rate and hide everything else (5
// rows, 23 tokens of 12 heads of 80 and 64, a window of 1000: 19 us and 6), and rows off
// 16 bytes.  k_tree_many stages tiles of
// 32 positions in LDS, once for all queries of a work-group, by loads from memory straight to
// LDS that are up to two tiles ahead, one barrier a tile; values are read from there transposed.
// One row of 131072, 64 tokens of 32 heads over 8 of 128, bf16: 249 us.  In copies that
// leave a part out: without products 158, without reading LDS 196, without arithmetic on scores
// 206, without loads 211; products alone 134, loads alone 150, arithmetic alone 81.  So nothing
// bounds it alone: a SIMD holds two waves (256 registers: 32 queries, their sums and weights),
// too few to hide each of the parts behind the others, and the products are half as many again
// as the formula's (weights in two parts).  Four tiles in flight, tiles of 64, eight waves to a
// work-group, products of 32 queries and priorities for waves in products all took as long.
//
// Which tokens a token attends to is one bit
// mask per token, made in LDS from the parents by pointer doubling; a tile of 32
// keys takes the 32 bits of it that lie above its keys, so only the tiles at the end
// of a row (or at the start of a window) look at single keys.
//
// Rows are dealt to work-groups as in one token's attention: positions in steps,
// laid end to end and cut into equal runs, the segments of a cut row joined by a
// second launch.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>

#include "../ecmd_launch.h"
#include "ecmd_attn_tile.h"

namespace ecmd {

namespace {

// A weight is held as 2^kTreeBias exp2(score - m), m raised where a score passes it by
// more than kTreeSlack (log2).  binary16 ends at 2^16: a weight stays below 2^15 there,
// and its second part reaches down to 2^-24, 2^-35 of the weight at m.
template <int TY>
constexpr float kTreeSlack = TY == S_F16 ? 4.0f : 8.0f;
template <int TY>
constexpr float kTreeBias = TY == S_F16 ? 11.0f : 0.0f;

template <int TY>
__device__ inline float tree_log_sum(float top, float total)
{
    if (!(total > 0.0f)) return total == 0.0f || total < 0.0f ? -INFINITY : total;
    return ((top == -INFINITY ? 0.0f : top) - kTreeBias<TY> + log2f(total)) * 0.69314718055994530942f;
}

template <class T>
__device__ inline T round_to(float x);
template <>
__device__ inline float round_to<float>(float x)
{
    return x;
}
template <>
__device__ inline __bf16 round_to<__bf16>(float x)
{
    return (__bf16)x;
}
template <>
__device__ inline _Float16 round_to<_Float16>(float x)
{
    return (_Float16)x;
}

__device__ inline void store_typed(int type, void *out, int64_t at, float x)
{
    if (type == S_F32) ((float *)out)[at] = x;
    else if (type == S_BF16) ((__bf16 *)out)[at] = round_to<__bf16>(x);
    else ((_Float16 *)out)[at] = round_to<_Float16>(x);
}

// The tokens of row r's tree, in LDS: bit x of mask[i] is set if token i attends to
// token x; info[i] is how many lie above it, or -1: padding.  All work-items call it.
struct Tree {
    uint32_t *mask;   // [t][words]
    int32_t *info;    // [t]
    uint32_t *real;   // [words]: bit i is set unless token i is padding
};
constexpr uint32_t kTreeWords = kMaxTree / 32;

// A lane's token's parent, to be loaded ahead of make_tree.
__device__ inline int32_t tree_parent(const TreeArgs &A, uint32_t r)
{
    const uint32_t i = min(threadIdx.x, A.t - 1);
    return A.parent[(int64_t)r * A.parent_s[0] + (int64_t)i * A.parent_s[1]];
}

// By pointer doubling: in every turn a token takes over what the token that it points to has,
// and points where that one does.  Up to 64 tokens one wave does it, by exchanges between
// its lanes (64 tokens, 32 of them in a row: 2 us instead of 7 with barriers).
__device__ inline void make_tree(const TreeArgs &A, int32_t p, const Tree &T)
{
    const uint32_t i = threadIdx.x, words = (A.t + 31) / 32;
    const bool fine = i < A.t && p >= 0 && (uint32_t)p < i;
    int32_t jump = i >= A.t ? -1 : fine ? p : p == -1 ? -1 : -2;   // the next token up; -1: none, -2: padding
    if (A.t <= 64) {
        if (i < 64) {
            uint64_t mask = i < A.t ? uint64_t(1) << i : 0;
            while (__any(jump >= 0)) {
                const int32_t from = jump >= 0 ? jump : (int32_t)i;
                const uint64_t more = __shfl(mask, from);
                const int32_t next = __shfl(jump, from);
                if (jump >= 0) {
                    mask |= more;
                    jump = next;
                }
            }
            const bool real = i < A.t && jump == -1;
            const int32_t above = real ? (int32_t)__popcll(mask) - 1 : -1;
            const uint64_t all = __ballot(real);
            if (A.window && __any(above >= 0 && (uint32_t)above >= A.window))
                for (uint32_t x = 0; x < A.t; ++x) {
                    const int32_t at = __shfl(above, (int)x);
                    if ((uint32_t)(above - at) >= A.window) mask &= ~(uint64_t(1) << x);   // (of tokens above i)
                }
            if (i < A.t) {
                T.mask[i * words] = (uint32_t)mask;
                if (words > 1) T.mask[i * words + 1] = (uint32_t)(mask >> 32);
                T.info[i] = above;
            }
            if (i < 2) T.real[i] = (uint32_t)(all >> 32 * i);
        }
        __syncthreads();
        return;
    }
    uint32_t mask[kTreeWords];
    if (i < kTreeWords) T.real[i] = 0;
#pragma unroll
    for (uint32_t w = 0; w < kTreeWords; ++w) mask[w] = i < A.t && w == i / 32 ? 1u << (i % 32) : 0;
    for (;;) {
        if (i < A.t) {
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) T.mask[i * words + w] = mask[w];
            T.info[i] = jump;
        }
        if (!__syncthreads_or(jump >= 0)) break;
        if (jump >= 0) {
            const uint32_t up = (uint32_t)jump;
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) mask[w] |= T.mask[up * words + w];
            jump = T.info[up];
        }
        __syncthreads();
    }
    const bool real = i < A.t && jump == -1;
    int32_t above = -1;
    if (real) {
#pragma unroll
        for (uint32_t w = 0; w < kTreeWords; ++w) above += __popc(mask[w]);
    }
    __syncthreads();
    if (i < A.t) {
        T.info[i] = above;
        if (real) atomicOr(&T.real[i / 32], 1u << (i % 32));
    }
    __syncthreads();
    if (A.window && real && (uint32_t)above >= A.window) {
        for (uint32_t x = 0; x < i; ++x)
            if (T.mask[i * words + x / 32] >> (x % 32) & 1)
                if ((uint32_t)(above - T.info[x]) >= A.window) T.mask[i * words + x / 32] &= ~(1u << (x % 32));
    }
    __syncthreads();
}

// Positions of row r that a launch looks at: its context (or its window) and its tokens.
__device__ inline Span tree_span(const TreeArgs &A, uint32_t r)
{
    const int32_t len = A.lens[(int64_t)r * A.lens_s];
    const uint32_t held = A.cols * A.page;
    Span s{0, 0};
    if (len < 0) return s;
    s.hi = min((uint32_t)len + A.t, held);
    if (A.window && (uint32_t)len >= A.window) s.lo = min((uint32_t)len + 1 - A.window, s.hi);
    return s;
}

// Steps that a row's end counts for beside its positions: its tree, its tiles of single keys
// and its sums take about as long as two steps (16 rows of up to 8192, 64 tokens: the
// work-groups' ends 123 to 169 us without).
constexpr uint32_t kTreeExtra = 2;

// Steps of a run, the same in every work-group and in the join; 0: runs are rows.
__device__ inline uint32_t tree_share(const TreeArgs &A, const Rows &R)
{
    // rows of nearly one length, enough of them to use the whole chip
    if (A.b <= A.runs_whole && (uint64_t)R.all * 5 >= (uint64_t)R.longest * A.b * 4) return 0;
    const uint32_t share = A.by_runs.div(R.all + A.runs - 1);
    return R.longest <= 2 * share && A.b <= max(A.runs, A.runs_whole) ? 0 : share;
}


// What a work-group does: the run of steps, its kv head and its block of queries.
struct TreeRun {
    uint32_t group, kvh, block;
    uint32_t r, step, stop;
    Rows R;
};
__device__ inline bool tree_next_row(const TreeArgs &A, TreeRun &X)
{
    X.step = __builtin_amdgcn_readfirstlane(X.R.prefix[X.r + 1]);
    if (X.step >= X.stop) return false;
    do ++X.r;
    while (__builtin_amdgcn_readfirstlane(X.R.prefix[X.r + 1]) <= X.step);   // past empty rows
    return true;
}
__device__ inline bool tree_run(const TreeArgs &A, uint32_t *s_rows, uint32_t *s_scratch, TreeRun &X)
{
    // Work-groups go to the eight dies in turn: those of a run follow each other on one.
    const uint32_t u8 = A.by_units.div(blockIdx.x), in8 = blockIdx.x - u8 * A.by_units.d, unit = in8 / 8;
    X.group = u8 * 8 + in8 % 8;
    X.kvh = A.by_blocks.div(unit);
    X.block = unit - X.kvh * A.q_blocks;
    X.r = X.group;
    X.step = X.stop = 0;
    if (A.direct) return X.group < A.b;
    X.R = make_rows(A, s_rows, s_scratch, tree_span, kTreeExtra);
    const uint32_t share = tree_share(A, X.R);
    if (share == 0) {
        if (X.group >= A.b) return false;
        X.step = __builtin_amdgcn_readfirstlane(X.R.prefix[X.r]);
        X.stop = __builtin_amdgcn_readfirstlane(X.R.prefix[X.r + 1]);
        return X.step != X.stop;
    }
    if ((uint64_t)X.group * share >= X.R.all) return false;
    X.step = X.group * share;
    X.stop = min(X.step + share, X.R.all);
    uint32_t lo = 0, hi = A.b;   // the row with prefix[r] <= step < prefix[r + 1]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (__builtin_amdgcn_readfirstlane(X.R.prefix[mid]) <= X.step) lo = mid;
        else hi = mid;
    }
    X.r = lo;
    // a run that starts with what a row's end counts for starts with the next row
    return X.step + kTreeExtra < __builtin_amdgcn_readfirstlane(X.R.prefix[lo + 1]) || tree_next_row(A, X);
}
// On to the next row of the run.
__device__ inline bool tree_next(const TreeArgs &A, TreeRun &X, uint32_t steps)
{
    if (A.direct) return false;
    X.step += steps;
    return X.step < X.stop && tree_next_row(A, X);
}

// One row of the run.
struct Segment {
    uint32_t begin, end, steps;
    uint32_t len;                 // of the context
    bool whole_row, last_part;
};
__device__ inline Segment tree_segment(const TreeArgs &A, const TreeRun &X)
{
    Segment S;
    S.len = (uint32_t)A.lens[(int64_t)X.r * A.lens_s];   // negative: A.direct only, a row of padding
    S.steps = 0;
    S.whole_row = S.last_part = true;
    if (A.direct) {
        const Span span = tree_span(A, X.r);
        S.begin = span.lo;
        S.end = span.hi;
    } else {
        const uint32_t first = __builtin_amdgcn_readfirstlane(X.R.prefix[X.r]);
        const uint32_t last = __builtin_amdgcn_readfirstlane(X.R.prefix[X.r + 1]) - kTreeExtra;
        const uint32_t here = min(X.stop, last), hi = __builtin_amdgcn_readfirstlane(X.R.hi[X.r]);
        S.last_part = here == last;
        S.whole_row = X.step == first && S.last_part;
        S.steps = here - X.step;
        S.begin = __builtin_amdgcn_readfirstlane(X.R.lo[X.r]) + (X.step - first) * kAttnStep;
        S.end = min(S.begin + S.steps * kAttnStep, hi);
    }
    return S;
}

// The tree matters to the tiles past the context, to a window's start and to who is padding.
__device__ inline bool tree_looks(const TreeArgs &A, const Segment &S)
{
    return S.last_part || A.window != 0 || S.end > S.len;
}

// Whether every query sees all of the TILE positions from t0 on, if they hold something.
template <uint32_t TILE>
__device__ inline bool tree_whole(const TreeArgs &A, uint32_t t0, uint32_t len)
{
    return t0 + TILE <= len && (A.window == 0 || t0 + A.window >= len + A.t);
}
// Which of the TILE positions from t0 on a token sees; lo: the first that its window holds.
template <uint32_t TILE>
__device__ inline uint32_t tree_sees(const uint32_t *mask, uint32_t words, uint32_t t0, uint32_t len, uint32_t lo)
{
    uint32_t see = ~0u;
    if (t0 + TILE > len) {
        if (t0 < len) {
            see = (1u << (len - t0)) - 1 | mask[0] << (len - t0);   // len - t0 < TILE <= 32
        } else {
            const uint32_t o = t0 - len, at = o / 32;
            const uint64_t two = (at < words ? mask[at] : 0) | (uint64_t)(at + 1 < words ? mask[at + 1] : 0) << 32;
            see = (uint32_t)(two >> (o % 32));
        }
    }
    if (lo > t0) see &= lo - t0 < 32 ? ~0u << (lo - t0) : 0;
    return see;
}

// A lane's tile of queries: the token of its query and the first position of its window.
struct Query {
    uint32_t token, lo;
};
__device__ inline uint32_t tree_lo(const TreeArgs &A, uint32_t token, uint32_t len, const int32_t *s_info)
{
    if (!A.window) return 0;
    const uint32_t past = len + (uint32_t)max(s_info[token], 0) + 1;
    return past > A.window ? past - A.window : 0;
}

// Scores x of a tile to weights p: the running maximum m, its use mref, the sum l and the
// sums acc follow.  A lane has one query and keys 4 j + k % 4 of every 16; see: which of the
// tile's the query sees (unless whole).
template <int TY, int VK, int N>
__device__ inline void tree_weights(const float (&x)[VK], float (&p)[VK], f32x4 (&acc)[N], float &m, float &mref, float &l,
                                    float scale, bool whole, uint32_t see, uint32_t j)
{
    auto sees = [&](int k) { return see >> ((k / 4) * 16 + j * 4 + k % 4) & 1; };
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < VK; ++k) top = fmaxf(top, whole || sees(k) ? x[k] : -INFINITY);
    if (top != -INFINITY) top *= scale;   // (a scale of 0 times infinity)
    if (__any(top > m + kTreeSlack<TY>)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top);
        mref = mn == -INFINITY ? 0.0f : mn;
        const float a = __builtin_amdgcn_exp2f(m - mref);
        m = mn;
        l *= a;
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] *= a;
    }
    const float less = kTreeBias<TY> - mref;
#pragma unroll
    for (int k = 0; k < VK; ++k) {
        p[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[k], scale, less));
        if (!whole) p[k] = sees(k) ? p[k] : 0.0f;
        l += p[k];
    }
}

// A weight goes into the second product as the sum of two 16-bit numbers, its leading bits
// and the rest, rounded to nearest: one would add its own rounding of half a step of the
// type to the result's, and a rest cut off would make every weight a little less than what
// the sum l counts.  (bf16, 16 rows of up to 8192 and 64 tokens, against 32 bits throughout: 0.42% of
// the results in another last place with rests cut off, 0.31% rounded, both 155 us; a third
// part, all 24 bits, 0.07% and 184 us.)  Both are positive wherever the weight is, since an
// infinite value times 0 would be NaN: the rest is made 2^-23 of the weight larger, and
// binary16 has the smallest number in place of 0 (only in tiles where every weight counts).
template <int TY>
__device__ inline void split_pair(float f, float g, uint32_t &hi, uint32_t &rest, bool whole)
{
    constexpr float more = 1.0f + 0x1p-23f;
    if constexpr (TY == S_BF16) {
        const uint32_t a = __builtin_bit_cast(uint32_t, f), b = __builtin_bit_cast(uint32_t, g);
        hi = __builtin_amdgcn_perm(b, a, 0x07060302);
        const f32x2 e = {__builtin_fmaf(f, more, -as_f(a & 0xFFFF0000u)), __builtin_fmaf(g, more, -as_f(b & 0xFFFF0000u))};
        rest = __builtin_bit_cast(uint32_t, __builtin_convertvector(e, bf16x2));
    } else {
        // positive numbers order as their bits do
        const u16x2 least = __builtin_bit_cast(u16x2, whole ? 0x00010001u : 0u);
        const f16x2 h = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(f, g));
        const f32x2 r = {__builtin_fmaf(f, more, -(float)h[0]), __builtin_fmaf(g, more, -(float)h[1])};
        const u16x2 e = __builtin_bit_cast(u16x2, __builtin_convertvector(r, f16x2));
        hi = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, h), least));
        rest = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(e, least));
    }
}
template <int TY, int VK>
__device__ inline void split_weights(const float (&p)[VK], u32x4 (&hi)[VK / 8], u32x4 (&rest)[VK / 8], bool whole)
{
#pragma unroll
    for (int x = 0; x < VK; x += 2) {
        uint32_t a, b;
        split_pair<TY>(p[x], p[x + 1], a, b, whole);
        hi[x / 8][x % 8 / 2] = a;
        rest[x / 8][x % 8 / 2] = b;
    }
}

template <int TY>
constexpr uint32_t kTopExponent = TY == S_F16 ? 0x7C00u : TY == S_BF16 ? 0x7F80u : 0x7F800000u;

// In a tile where some query does not see some key: clears the values of slots that hold
// nothing (they may hold NaN), and says whether any left is no finite number.
template <int TY, int VK, int VP, int PW>
__device__ inline bool clear_values(u32x4 (&vr)[VK][VP], uint32_t now, uint32_t j)
{
    bool odd = false;
#pragma unroll
    for (int x = 0; x < VK; ++x) {
        const uint32_t keep = now >> ((x / 4) * 16 + j * 4 + x % 4) & 1 ? ~0u : 0u;
#pragma unroll
        for (int c = 0; c < VP; ++c) {
            vr[x][c] = vr[x][c] & u32x4{keep, keep, keep, keep};
#pragma unroll
            for (int w = 0; w < PW; ++w) {
                odd |= (vr[x][c][w] & kTopExponent<TY>) == kTopExponent<TY>;
                if constexpr (TY != S_F32) odd |= (vr[x][c][w] >> 16 & kTopExponent<TY>) == kTopExponent<TY>;
            }
        }
    }
    return odd;
}

// A weight of 0 times an infinity is NaN: where such values meet queries that do not see
// them, a tile's values are added one by one.  At a row's end only, and hardly ever.
template <int TY, int VK, int N, class Column>
__device__ inline void add_odd(const TreeArgs &A, uint32_t r, const char *vbase, uint32_t t0, uint32_t now, uint32_t see,
                               const float (&p)[VK], f32x4 (&acc)[N], uint32_t j, uint32_t hh, Column column)
{
    for (uint32_t key = 0; key < 4 * VK; ++key) {
        if (!(now >> key & 1)) continue;
        const uint32_t pos = t0 + key, col = A.by_page.div(pos);
        const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)col * A.pages_s[1]];
        const char *v = vbase + (int64_t)id * A.vcs[0] + (int64_t)(pos - col * A.page) * A.vcs[1];
        float w = 0.0f;
#pragma unroll
        for (int x = 0; x < VK; ++x)
            if (key / 16 * 4 + key % 4 == (uint32_t)x) w = __shfl(p[x], (int)(key % 16 / 4 * 16 + hh));   // key is uniform
        if (!(see >> key & 1)) continue;
#pragma unroll
        for (int c = 0; c < N; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = column(j * 4 + i, c);
                if (at >= A.dv) continue;
                float value;
                if constexpr (TY == S_F32) value = ((const float *)v)[at];
                else if constexpr (TY == S_BF16) value = (float)((const __bf16 *)v)[at];
                else value = (float)((const _Float16 *)v)[at];
                acc[c][i] += w * value;
            }
            asm volatile("" ::: "memory");   // not all values at once: registers
        }
    }
}

// Where a segment's sums go: out and lse, or a place of their own for the second launch
// (work-groups and rows only go forward, so group + r is no other segment's).
struct TreeOut {
    uint32_t r, kvh;
    uint64_t place;
    bool whole_row, last_part, nobody;
    const int32_t *info;
};
__device__ inline TreeOut tree_out(const TreeArgs &A, const TreeRun &X, const Segment &S, const int32_t *info)
{
    return TreeOut{X.r, X.kvh, (uint64_t)(X.group + X.r) * A.by_vectors.d + (uint64_t)X.kvh * A.m, S.whole_row, S.last_part,
                   (int32_t)S.len < 0, info};
}
// query vector x's sum of weights; -1 for padding
__device__ inline float known(const TreeArgs &A, const TreeOut &O, uint32_t x, float total)
{
    return O.last_part && (O.nobody || O.info[A.by_group.div(x)] < 0) ? -1.0f : total;
}
template <int TY>
__device__ inline void put(const TreeArgs &A, const TreeOut &O, uint32_t x, uint32_t c, float sum, float total)
{
    if (!O.whole_row) {
        A.acc[(O.place + x) * A.dv + c] = sum;
        return;
    }
    const uint32_t tok = A.by_group.div(x), head = O.kvh * A.group + x - tok * A.group;
    store_typed(TY, A.out, (int64_t)O.r * A.os[0] + (int64_t)tok * A.os[1] + (int64_t)head * A.os[2] + c,
                total > 0.0f ? sum / total : total == 0.0f || total < 0.0f ? 0.0f : total);
}
template <int TY>
__device__ inline void put_statistics(const TreeArgs &A, const TreeOut &O, uint32_t x, float top, float total)
{
    if (!O.whole_row) {
        A.ml[2 * (O.place + x)] = top;
        A.ml[2 * (O.place + x) + 1] = total;
    } else if (A.lse) {
        const uint32_t tok = A.by_group.div(x), head = O.kvh * A.group + x - tok * A.group;
        A.lse[(int64_t)O.r * A.ls[0] + (int64_t)tok * A.ls[1] + (int64_t)head * A.ls[2]] = tree_log_sum<TY>(top, total);
    }
}

// The same of four neighbouring columns from c on, in one store.
template <int TY>
__device__ inline void put4(const TreeArgs &A, const TreeOut &O, uint32_t x, uint32_t c, f32x4 sum, float total)
{
    typedef f32x4 F __attribute__((aligned(4)));
    if (!O.whole_row) {
        *(F *)&A.acc[(O.place + x) * A.dv + c] = sum;
        return;
    }
    const uint32_t tok = A.by_group.div(x), head = O.kvh * A.group + x - tok * A.group;
    const float to = total > 0.0f ? 1.0f : total == 0.0f || total < 0.0f ? 0.0f : total, by = total > 0.0f ? total : 1.0f;
    if constexpr (TY == S_F32) {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = to == 0.0f ? 0.0f : sum[i] / by * to;
        *(F *)((float *)A.out + (int64_t)O.r * A.os[0] + (int64_t)tok * A.os[1] + (int64_t)head * A.os[2] + c) = y;
        return;
    }
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef u32x2 Out __attribute__((aligned(2)));
    uint16_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = to == 0.0f ? 0.0f : sum[i] / by * to;
        if constexpr (TY == S_BF16) y[i] = __builtin_bit_cast(uint16_t, round_to<__bf16>(v));
        else y[i] = __builtin_bit_cast(uint16_t, round_to<_Float16>(v));
    }
    *(Out *)((uint16_t *)A.out + (int64_t)O.r * A.os[0] + (int64_t)tok * A.os[1] + (int64_t)head * A.os[2] + c) =
        u32x2{y[0] | (uint32_t)y[1] << 16, y[2] | (uint32_t)y[3] << 16};
}

// The sums of one tile of queries, q0 .. q0 + 15, out.  Waves with the same queries (every
// hw-th of the four) join them through LDS first: common maximum, then sums, eight queries
// at a time and four columns to a work-item.  All waves call it alike.
template <int TY, int VW, bool TINY, class Column>
__device__ inline void put_tile(const TreeArgs &A, const TreeOut &O, uint32_t q0, uint32_t hw, const f32x4 (&acc)[VW], float m,
                                float l, uint32_t wave, uint32_t lane, float *s_join, float (*s_m)[16], float (*s_l)[16],
                                Column column)
{
    constexpr uint32_t kRow = 16 * VW + 4;   // a query's row in the joining buffer (floats)
    const uint32_t j = lane >> 4, hh = lane & 15, qw = wave & (hw - 1), part = wave / hw, parts = kAttnWaves / hw;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (parts == 1) {
        const uint32_t x = q0 + hh;
        if (x < A.m) {
            const float total = known(A, O, x, l);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    const uint32_t at = column(j * 4 + i, c);
                    if (!TINY || at < A.dv) put<TY>(A, O, x, at, acc[c][i], total);
                }
            if (j == 0) put_statistics<TY>(A, O, x, m, total);
        }
        return;
    }
    __syncthreads();   // what lay in the buffer is done with
    if (j == 0) {
        s_m[wave][hh] = m;
        s_l[wave][hh] = l;
    }
    __syncthreads();
    float top = -INFINITY, total = 0.0f;
    for (uint32_t w = qw; w < kAttnWaves; w += hw) top = fmaxf(top, s_m[w][hh]);
    const float ref = top == -INFINITY ? 0.0f : top;
    for (uint32_t w = qw; w < kAttnWaves; w += hw) total += s_l[w][hh] * __builtin_amdgcn_exp2f(s_m[w][hh] - ref);
    const float factor = __builtin_amdgcn_exp2f(m - ref);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half) __syncthreads();
        if ((hh >> 3) == (uint32_t)half) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VW; ++c) s_join[(wave * 8 + (hh & 7)) * kRow + column(j * 4 + i, c)] = acc[c][i] * factor;
        }
        __syncthreads();
        for (uint32_t y = part * 64 + lane; y < 8 * 4 * VW; y += parts * 64) {
            const uint32_t g = y / (4 * VW), c = y % (4 * VW) * 4, x = q0 + half * 8 + g;
            // lane g + 8 half of every wave of these has the statistics
            const float all = __shfl(total, (int)(half * 8 + g)), best = __shfl(top, (int)(half * 8 + g));
            if (x >= A.m) continue;
            f32x4 sum = *(const f32x4 *)&s_join[(qw * 8 + g) * kRow + c];
            for (uint32_t w = qw + hw; w < kAttnWaves; w += hw) sum += *(const f32x4 *)&s_join[(w * 8 + g) * kRow + c];
            const float t = known(A, O, x, all);
            if (c + 4 <= A.dv) {
                put4<TY>(A, O, x, c, sum, t);
            } else {
                for (uint32_t k = 0; k < 4; ++k)
                    if (c + k < A.dv) put<TY>(A, O, x, c + k, sum[k], t);
            }
            if (c == 0) put_statistics<TY>(A, O, x, best, t);
        }
    }
}

// ---------------------------------------------------------------------------
// Few queries, or binary32.

template <int TY, int NK, int VW>
constexpr int few_waves()
{
    constexpr int KB = AttnType<TY>::KB, size = TY == S_F32 ? 4 : 2;
    constexpr int regs = KB * NK * 4 + KB * VW * size + NK * 4 + VW * 4 + KB * 8 + 60;
    return regs > 200 ? 1 : 2;   // (what the compiler takes is about 60 more)
}

template <int TY, int NK, int VW, AttnEdge EDGE>
__global__ __launch_bounds__(kAttnBlock, (few_waves<TY, NK, VW>())) void k_tree_few(const TreeArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, KB = AttnType<TY>::KB;
    constexpr int VK = 4 * KB;                          // keys whose values a lane holds
    constexpr int PE = VW < E ? VW : E, VP = VW / PE;   // elements of a value piece; pieces
    constexpr int PW = PE * (int)sizeof(T) / 4;         // words of a value piece
    constexpr uint32_t kTile = 16 * KB;

    __shared__ union {
        struct {
            uint64_t k[kAttnWaves][kTableKeys], v[kAttnWaves][kTableKeys];
            uint64_t valid[kAttnWaves][kTableKeys / 64];
        } table;
        __attribute__((aligned(16))) float join[kAttnWaves * 8 * (16 * VW + 4)];
    } sh;
    __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16];
    __shared__ uint32_t s_mask[kMaxTree * kTreeWords], s_real[kTreeWords];
    __shared__ int32_t s_info[kMaxTree];
    extern __shared__ uint32_t s_rows[];   // unless A.direct
    __shared__ uint32_t s_scratch[kAttnWaves];

    const uint32_t lane = threadIdx.x & 63, j = lane >> 4, hh = lane & 15;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tree tree{s_mask, s_info, s_real};
    const uint32_t words = (A.t + 31) / 32;
    TreeRun X;
    if (!tree_run(A, s_rows, s_scratch, X)) return;
    const uint32_t qw = wave & ((1u << A.q_shift) - 1), part = wave >> A.q_shift, parts = kAttnWaves >> A.q_shift;
    const uint32_t q0 = ((X.block << A.q_shift) + qw) * 16;   // the wave's first query vector

    // Element c of the value piece of product c at row m of the result.
    auto column = [&](uint32_t m, int c) {
        const uint32_t at = (c / PE * 16 + m) * PE;
        return (EDGE == kTiny ? at : min(at, A.dv - PE)) + c % PE;
    };
    auto load_row_piece = [&](const char *p, int c) {
        const int at = (c * 4 + (int)j) * E;
        if constexpr (EDGE == kTiny) return load_some<T, E>(p + at * sizeof(T), (int)A.d - at);
        return load16(p + (EDGE == kTail ? min(at, (int)A.d - E) : at) * sizeof(T));
    };
    auto masked = [&](u32x4 x, int c) {
        if (EDGE == kTail && (uint32_t)(c + 1) * 4 * E > A.d) x = only_own<E>(x, (c * 4 + (int)j) * E, (int)A.d);
        return x;
    };

    const char *kbase = (const char *)A.k + (int64_t)X.kvh * A.kcs[2];
    const char *vbase = (const char *)A.v + (int64_t)X.kvh * A.vcs[2];

    for (;;) {   // one row of the run
        const Segment S = tree_segment(A, X);
        const uint32_t r = X.r, len = S.len;
        if (tree_looks(A, S)) make_tree(A, tree_parent(A, r), tree);
        uint32_t wb = S.begin, we = S.end;
        if (parts > 1) {
            const uint32_t each = (we - wb + parts * kTile - 1) / (parts * kTile) * kTile;
            wb = min(S.begin + part * each, S.end);
            we = min(wb + each, S.end);
        }
        if (q0 >= A.m) we = wb;   // no queries of this wave's

        u32x4 q[NK];
        const uint32_t token = A.by_group.div(min(q0 + hh, A.m - 1));
        const Query Q{token, tree_lo(A, token, len, s_info)};
        {
            const uint32_t head = X.kvh * A.group + min(q0 + hh, A.m - 1) - Q.token * A.group;
            const char *p = (const char *)A.q + ((int64_t)r * A.qs[0] + (int64_t)Q.token * A.qs[1] + (int64_t)head * A.qs[2]) * sizeof(T);
#pragma unroll
            for (int c = 0; c < NK; ++c) q[c] = masked(load_row_piece(p, c), c) ^ u32x4{A.q_flip, A.q_flip, A.q_flip, A.q_flip};
        }

        f32x4 acc[VW];
#pragma unroll
        for (int c = 0; c < VW; ++c) acc[c] = f32x4{0, 0, 0, 0};
        float m = -INFINITY, mref = 0.0f, l = 0.0f;

        // Offsets of the wave's next kTableKeys positions; what is no position of
        // this row's gets slot 0 of page 0, which exists, and a clear bit.
        auto fill = [&](uint32_t at) {
            constexpr int G = kTableKeys / 64;
            int32_t id[G];
            uint32_t in[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t pos = min(at + g * 64 + lane, we - 1), col = A.by_page.div(pos);
                in[g] = pos - col * A.page;
                id[g] = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)col * A.pages_s[1]];
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t pos = at + g * 64 + lane;
                bool ok = pos < we && id[g] >= 0 && (uint32_t)id[g] < A.n;
                if (pos >= len && ok) ok = s_real[(pos - len) / 32] >> ((pos - len) % 32) & 1;   // pos < len + t
                const int64_t page = ok ? id[g] : 0, slot = ok ? in[g] : 0;
                sh.table.k[wave][g * 64 + lane] = (uint64_t)(page * A.kcs[0] + slot * A.kcs[1]);
                sh.table.v[wave][g * 64 + lane] = (uint64_t)(page * A.vcs[0] + slot * A.vcs[1]);
                const uint64_t bits = __ballot(ok);
                if (lane == 0) sh.table.valid[wave][g] = bits;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };

        u32x4 kr[KB][NK];
        u32x4 vr[VK][VP];
        uint32_t bits = 0;   // which of the tile's positions hold something
        auto load_k = [&](uint32_t t) {   // t: offset of the tile in the table
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const char *p = kbase + sh.table.k[wave][t + kb * 16 + hh];
#pragma unroll
                for (int c = 0; c < NK; ++c) kr[kb][c] = load_row_piece(p, c);
            }
            bits = (uint32_t)(sh.table.valid[wave][t / 64] >> (t % 64));
            if constexpr (KB == 1) bits &= 0xFFFFu;
            bits = __builtin_amdgcn_readfirstlane(bits);
        };
        auto load_v = [&](uint32_t t) {
#pragma unroll
            for (int x = 0; x < VK; ++x) {
                const char *p = vbase + sh.table.v[wave][t + (x / 4) * 16 + j * 4 + x % 4];
#pragma unroll
                for (int c = 0; c < VP; ++c) {
                    const uint32_t at = column(hh, c * PE);
                    if constexpr (EDGE == kTiny)
                        vr[x][c] = load_some<T, PE>(p + at * sizeof(T), (int)A.dv - (int)at);
                    else if constexpr (PE * sizeof(T) == 16)
                        vr[x][c] = load16(p + at * sizeof(T));
                    else
                        __builtin_memcpy(&vr[x][c], p + at * sizeof(T), PE * sizeof(T));
                }
            }
        };

        uint32_t tile = wb, in_table = 0;
        if (wb < we) {
            fill(wb);
            load_k(0);
            load_v(0);
        }
        while (tile < we) {
            f32x4 s[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                s[kb] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < NK; ++c) {
                    const u32x4 k = masked(kr[kb][c], c);
                    if constexpr (TY == S_F32) {
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            s[kb] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(k[f]), as_f(q[c][f]), s[kb], 0, 0, 0);
                    } else {
                        s[kb] = mma16<TY>(k, q[c], s[kb]);
                    }
                }
            }
            const uint32_t now = bits, t0 = tile;
            tile += kTile;
            in_table += kTile;
            if (tile < we) {
                if (in_table == kTableKeys) {
                    fill(tile);
                    in_table = 0;
                }
                load_k(in_table);
            }
            // Single keys matter past the context, at a window's start and at holes.
            const bool whole = now == (KB == 2 ? 0xFFFFFFFFu : 0xFFFFu) && tree_whole<kTile>(A, t0, len);
            uint32_t see = 0;
            bool odd = false;
            if (!whole) {
                see = now & tree_sees<kTile>(s_mask + Q.token * words, words, t0, len, Q.lo);
                odd = __any(clear_values<TY, VK, VP, PW>(vr, now, j));
            }
            float x[VK], p[VK];
#pragma unroll
            for (int k = 0; k < VK; ++k) x[k] = s[k / 4][k % 4];
            tree_weights<TY, VK>(x, p, acc, m, mref, l, A.scale_log2, whole, see, j);
            if (odd) {
                add_odd<TY, VK, VW>(A, r, vbase, t0, now, see, p, acc, j, hh, column);
            } else if constexpr (TY == S_F32) {
#pragma unroll
                for (int x = 0; x < VK; ++x)
#pragma unroll
                    for (int c = 0; c < VW; ++c)
                        acc[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(vr[x][c / 4][c % 4]), p[x], acc[c], 0, 0, 0);
            } else {
                u32x4 hi[1], rest[1];
                split_weights<TY, VK>(p, hi, rest, whole);
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    u32x4 a;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        a[w] = __builtin_amdgcn_perm(vr[2 * w + 1][c / 8][c % 8 / 2], vr[2 * w][c / 8][c % 8 / 2],
                                                     c & 1 ? 0x07060302 : 0x05040100);
                    acc[c] = mma16<TY>(a, rest[0], acc[c]);
                    acc[c] = mma16<TY>(a, hi[0], acc[c]);
                }
            }
            if (tile < we) load_v(in_table);
        }
        put_tile<TY, VW, EDGE == kTiny>(A, tree_out(A, X, S, s_info), q0, 1u << A.q_shift, acc, m, l, wave, lane, sh.join, s_m, s_l, column);
        if (!tree_next(A, X, S.steps)) return;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Many queries of 16 bits.

constexpr uint32_t kStageKeys = 32, kStageTable = kAttnBlock;   // positions of a tile; whose places are known ahead

// 16 bytes from each lane's p to LDS, from address lds on, in the order of the lanes.  Written
// out, for the compiler would let every later read of LDS wait for it: it does not
// know that the buffers are read in turn.  wait_loads waits.  (No register is written but m0,
// which holds the address, 16 bits of it.  The compiler keeps m0 for itself and cannot be told
// so; it uses it for nothing in these kernels, which their assembly is tested for.)
__device__ inline void load_to_lds(const char *p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory");
}

__device__ __attribute__((aligned(256))) const uint32_t g_zeros[128] = {};   // a row of a slot that holds nothing

// Where a row of PIECES 16-byte pieces has piece x, for a number that the key gives: another
// place for each of neighbouring keys, so that what is read at once lies in different banks
// (but for a little where PIECES is no power of two).
template <uint32_t PIECES>
__device__ inline uint32_t turned(uint32_t x, uint32_t turn)
{
    if constexpr ((PIECES & (PIECES - 1)) == 0) return x ^ (turn & (PIECES - 1));
    else return (x + (turn >> 2 & 3)) % PIECES;
}
template <uint32_t PIECES>
__device__ inline uint32_t turned_back(uint32_t x, uint32_t turn)
{
    if constexpr ((PIECES & (PIECES - 1)) == 0) return x ^ (turn & (PIECES - 1));
    else return (x + PIECES - (turn >> 2 & 3)) % PIECES;
}
// Keys: sixteen keys' pieces at one index.  (Rows of 128 bytes: two lie side by side.)
template <uint32_t PIECES>
__device__ inline uint32_t key_turn(uint32_t key)
{
    return PIECES == 8 ? key >> 1 : key & 15;
}
// Values: two neighbouring pieces of four keys.
__device__ inline uint32_t value_turn(uint32_t key) { return 2 * key; }

// Lane h of 16 gets element h of four rows, of which lane s reads four elements: number
// 4 (s % 4) on, of row s / 4.  Two of them are a product's first operand over its lane's keys.
__device__ inline u32x4 read_transposed(const char *low, const char *high)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 *Ptr;
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)low));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)high));
    return u32x4{a[0], a[1], b[0], b[1]};
}

// A lane's number that the compiler is to keep, not to make anew.
__device__ inline uint32_t kept(uint32_t x)
{
    asm("" : "+v"(x));
    return x;
}

// All of the LDS traffic so far is done, and all but N of the loads (to LDS too).  (The
// instruction's fields: bits 3:0 and 15:14 loads, 6:4 exports, 11:8 LDS.)
template <int N>
__device__ inline void wait_loads()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);
    asm volatile("" ::: "memory");
}
__device__ inline void group_barrier()
{
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Rows' starts are multiples of 16 bytes and so are d and dv (of 2-byte elements): see
// plan_tree.  NK: 32 elements of a key; VW: 16 of a value; NT: tiles of 16 queries of a wave.
// A lane has query lane % 16 of each and keys 4 j + i of every 16, j = lane / 16.
template <int TY, int NK, int VW, int NT>
__global__ __launch_bounds__(kAttnBlock, (NK * 64 + VW * 32 >= 640 ? 1 : 2)) void k_tree_many(const TreeArgs A)
{
    typedef uint16_t T;
    constexpr int KB = 2, VK = 8;
    constexpr uint32_t KP = 4 * NK, VPieces = 2 * VW;                 // 16-byte pieces of a key and of a value
    constexpr uint32_t kLoads = 2 * NK + VW;                          // of 1024 bytes: a tile's keys, then its values
    // A wave's; where they do not come out even, the last one more than once.
    constexpr int KU = (2 * NK + kAttnWaves - 1) / kAttnWaves, VU = (VW + kAttnWaves - 1) / kAttnWaves, PER = KU + VU;

    // Tiles' buffers: their places count 16 bits in a load to LDS, so they come first, in the one
    // object that there is (what a launch adds lies behind it), and end within 64 KiB.
    constexpr uint32_t kRing = kLoads * 3 <= 64 ? 3 : 2, kAhead = kRing - 1;
    struct Stage {
        char ring[kRing][kLoads * 1024];
        uint64_t k[2][kStageTable], v[2][kStageTable];     // where a position's key and value lie
        uint32_t valid[2][kStageTable / kStageKeys];
        uint32_t mask[kMaxTree * kTreeWords], real[kTreeWords];
        int32_t info[kMaxTree];
        uint32_t scratch[kAttnWaves];
    };
    static_assert(offsetof(Stage, ring) == 0 && sizeof(Stage::ring) <= 64 << 10);
    __shared__ __attribute__((aligned(1024))) Stage sh;
    auto &s_ring = sh.ring;
    auto &s_k = sh.k, &s_v = sh.v;
    auto &s_valid = sh.valid;
    uint32_t *const s_mask = sh.mask, *const s_real = sh.real, *const s_scratch = sh.scratch;
    int32_t *const s_info = sh.info;
    extern __shared__ uint32_t s_rows[];   // unless A.direct

    const uint32_t tid = threadIdx.x, lane = tid & 63, j = lane >> 4, hh = lane & 15;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Tree tree{s_mask, s_info, s_real};
    const uint32_t words = (A.t + 31) / 32;
    TreeRun X;
    if (!tree_run(A, s_rows, s_scratch, X)) return;
    const uint32_t q0 = (X.block * kAttnWaves + wave) * (16 * NT);   // the wave's first query vector

    const char *kbase = (const char *)A.k + (int64_t)X.kvh * A.kcs[2];
    const char *vbase = (const char *)A.v + (int64_t)X.kvh * A.vcs[2];

    // What the lane reads of a tile: pieces c * 4 + j of key hh (and 16 + hh); of the values four
    // elements of key 4 j + hh / 4 (and 16 on) for each product.
    uint32_t k_at[NK], v_at[VW];
#pragma unroll
    for (int c = 0; c < NK; ++c) k_at[c] = (hh * KP + turned<KP>(c * 4 + j, key_turn<KP>(hh))) * 16;
#pragma unroll
    for (int c = 0; c < VW; ++c) {
        const uint32_t key = j * 4 + hh / 4;
        v_at[c] = 2 * NK * 1024 + (key * VPieces + turned<VPieces>(2 * c + (hh & 3) / 2, value_turn(key))) * 16 + (hh & 1) * 8;
    }
    // What it loads: places in LDS go up with the lanes; of which key, and which of its bytes
    // (kNone: past a key's end, zeros).
    constexpr uint32_t kNone = ~0u;
    uint32_t k_key[KU], k_of[KU], v_key[VU], v_of[VU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
        const uint32_t x = min(u * kAttnWaves + wave, 2u * NK - 1) * 64 + lane, key = x / KP;
        const uint32_t piece = turned_back<KP>(x - key * KP, key_turn<KP>(key));
        k_key[u] = kept(key);
        k_of[u] = kept(piece * 8 < A.d ? piece * 16 : kNone);
    }
#pragma unroll
    for (int u = 0; u < VU; ++u) {
        const uint32_t x = min(u * kAttnWaves + wave, VW - 1u) * 64 + lane, key = x / VPieces;
        const uint32_t piece = turned_back<VPieces>(x - key * VPieces, value_turn(key));
        v_key[u] = kept(key);
        v_of[u] = kept(piece * 8 < A.dv ? piece * 16 : 0);   // (of columns past the end nothing is kept)
    }
    const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)&s_ring[0][0];

    for (;;) {   // one row of the run
        const Segment S = tree_segment(A, X);
        const uint32_t r = X.r, len = S.len;
        const uint32_t tiles = (S.end - S.begin + kStageKeys - 1) / kStageKeys;
        constexpr uint32_t kChunk = kStageTable / kStageKeys;   // tiles whose places a table holds
        // Pages of positions 256 chunk + tid of the segment: looked up a chunk ahead.
        auto look = [&](uint32_t chunk) {
            const uint32_t pos = min(S.begin + chunk * kStageTable + tid, max(S.end, 1u) - 1);
            return A.pages[(int64_t)r * A.pages_s[0] + (int64_t)A.by_page.div(pos) * A.pages_s[1]];
        };
        auto note = [&](uint32_t chunk, int32_t id) {
            const uint32_t pos = S.begin + chunk * kStageTable + tid;
            bool ok = pos < S.end && id >= 0 && (uint32_t)id < A.n;
            if (pos >= len && ok) ok = s_real[(pos - len) / 32] >> ((pos - len) % 32) & 1;   // pos < len + t
            const int64_t page = id, slot = pos - A.by_page.div(pos) * A.page;
            s_k[chunk & 1][tid] = (uint64_t)(ok ? kbase + page * A.kcs[0] + slot * A.kcs[1] : (const char *)g_zeros);
            s_v[chunk & 1][tid] = (uint64_t)(ok ? vbase + page * A.vcs[0] + slot * A.vcs[1] : (const char *)g_zeros);
            const uint64_t bits = __ballot(ok);
            if (lane == 0) {
                s_valid[chunk & 1][wave * 2] = (uint32_t)bits;
                s_valid[chunk & 1][wave * 2 + 1] = (uint32_t)(bits >> 32);
            }
        };
        // everything that the row's start waits for, asked for at once
        const bool looks = tree_looks(A, S);
        const int32_t parent = looks ? tree_parent(A, r) : -1;
        int32_t id0 = 0, id = 0;
        if (tiles) {
            id0 = look(0);
            id = look(1);
        }
        u32x4 q[NT][NK];
        Query Q[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t m = min(q0 + n * 16 + hh, A.m - 1);
            Q[n].token = A.by_group.div(m);
            const uint32_t head = X.kvh * A.group + m - Q[n].token * A.group;
            const char *p = (const char *)A.q + ((int64_t)r * A.qs[0] + (int64_t)Q[n].token * A.qs[1] + (int64_t)head * A.qs[2]) * sizeof(T);
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                const uint32_t at = (c * 4 + j) * 8;
                q[n][c] = u32x4{0, 0, 0, 0};
                if (at < A.d) q[n][c] = load16(p + at * sizeof(T)) ^ u32x4{A.q_flip, A.q_flip, A.q_flip, A.q_flip};
            }
        }
        if (looks) make_tree(A, parent, tree);
        f32x4 acc[NT][VW];
        float m[NT], mref[NT], l[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            Q[n].lo = tree_lo(A, Q[n].token, len, s_info);
            m[n] = -INFINITY;
            mref[n] = 0.0f;
            l[n] = 0.0f;
#pragma unroll
            for (int c = 0; c < VW; ++c) acc[n][c] = f32x4{0, 0, 0, 0};
        }

        // Tile t's pieces from memory into a buffer.
        auto load = [&](uint32_t t, uint32_t buffer) {
            const uint64_t *ks = s_k[t / kChunk & 1] + t % kChunk * kStageKeys, *vs = s_v[t / kChunk & 1] + t % kChunk * kStageKeys;
            const char *p[PER];
#pragma unroll
            for (int u = 0; u < KU; ++u) p[u] = (const char *)(ks[k_key[u]] + k_of[u]);
#pragma unroll
            for (int u = 0; u < VU; ++u) p[KU + u] = (const char *)(vs[v_key[u]] + v_of[u]);
            if (A.d != 32 * NK) {
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    if (k_of[u] == kNone) p[u] = (const char *)g_zeros;
            }
#pragma unroll
            for (int u = 0; u < PER; ++u)
                load_to_lds(p[u], ring0 + (buffer * kLoads + (u < KU ? min(u * kAttnWaves + wave, 2u * NK - 1)
                                                                     : 2 * NK + min((u - KU) * kAttnWaves + wave, VW - 1u))) * 1024);
        };
        // WHOLE: every query sees every key.  Otherwise (at a row's end, at holes, where a window
        // starts) slots that hold nothing have given zeros, and single keys are left out.
        auto compute = [&](auto WHOLE, uint32_t t, const char *ring, uint32_t now) {
            constexpr bool whole = decltype(WHOLE)::value;
            const uint32_t t0 = S.begin + t * kStageKeys;
            f32x4 s[NT][KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][kb] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < NK; ++c) {
                    const u32x4 k = *(const u32x4 *)(ring + k_at[c] + kb * 16 * KP * 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[n][kb] = mma16<TY>(k, q[n][c], s[n][kb]);
                }
            }
            auto value = [&](int c) { return read_transposed(ring + v_at[c], ring + v_at[c] + 16 * VPieces * 16); };
            uint32_t see[NT] = {};
            bool odd = false;
            if constexpr (!whole) {
#pragma unroll
                for (int n = 0; n < NT; ++n) see[n] = now & tree_sees<kStageKeys>(s_mask + Q[n].token * words, words, t0, len, Q[n].lo);
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    const u32x4 a = value(c);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        odd |= (a[w] & kTopExponent<TY>) == kTopExponent<TY> || (a[w] >> 16 & kTopExponent<TY>) == kTopExponent<TY>;
                }
                odd = __any(odd);
            }
            u32x4 hi[NT][1], rest[NT][1];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x[VK], p[VK];
#pragma unroll
                for (int k = 0; k < VK; ++k) x[k] = s[n][k / 4][k % 4];
                tree_weights<TY, VK>(x, p, acc[n], m[n], mref[n], l[n], A.scale_log2, whole, see[n], j);
                if (odd) add_odd<TY, VK, VW>(A, r, vbase, t0, now, see[n], p, acc[n], j, hh, [&](uint32_t m, int c) { return c * 16 + m; });
                split_weights<TY, VK>(p, hi[n], rest[n], whole);
            }
            if (odd) return;
#pragma unroll
            for (int c = 0; c < VW; ++c) {
                const u32x4 a = value(c);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][c] = mma16<TY>(a, rest[n][0], acc[n][c]);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][c] = mma16<TY>(a, hi[n][0], acc[n][c]);
            }
        };

        if (tiles) {
            note(0, id0);
            __syncthreads();
#pragma unroll
            for (uint32_t t = 0; t < kAhead; ++t)
                if (t < tiles) load(t, t);
            // what else is on its way (the query, the next table's pages) is waited for here: a
            // wait in the loop would be for the loads to LDS too
            wait_loads<0>();
        }
        auto look_ahead = [&](uint32_t t) {
            if (t % kChunk == kChunk - 1 - kAhead) {   // the next load is of the next table
                note(t / kChunk + 1, id);
                id = look(t / kChunk + 2);
            }
        };
        uint32_t t = 0, turn = 0;   // turn: t % kRing
        while (t < tiles) {
            uint32_t now = 0;
            const char *here = nullptr;
            bool whole;
            for (;;) {   // whole tiles, in a loop of their own
                // Tile t is in its buffer, and the one after it may be on its way; what was in the
                // buffer that is loaded next is done with by all, and so is the table that is written next.
                if (kAhead == 2 && t + 1 < tiles) wait_loads<PER>();
                else wait_loads<0>();
                group_barrier();
                if (t + kAhead < tiles) load(t + kAhead, turn == 0 ? kRing - 1 : turn - 1);
                here = s_ring[turn];
                turn = turn + 1 == kRing ? 0 : turn + 1;
                now = __builtin_amdgcn_readfirstlane(s_valid[t / kChunk & 1][t % kChunk]);
                whole = now == 0xFFFFFFFFu && tree_whole<kStageKeys>(A, S.begin + t * kStageKeys, len);
                if (!whole) break;
                if (q0 < A.m) compute(std::true_type(), t, here, now);
                look_ahead(t);
                if (++t == tiles) break;
            }
            if (whole) break;
            if (q0 < A.m) compute(std::false_type(), t, here, now);
            wait_loads<0>();   // its own: see above
            look_ahead(t);
            ++t;
        }
        const TreeOut O = tree_out(A, X, S, s_info);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
            const uint32_t x = q0 + n * 16 + hh;
            if (x >= A.m) continue;
            const float total = known(A, O, x, l[n]);
#pragma unroll
            for (int c = 0; c < VW; ++c)
                if (c * 16 + j * 4 < A.dv) put4<TY>(A, O, x, c * 16 + j * 4, acc[n][c], total);
            if (j == 0) put_statistics<TY>(A, O, x, m[n], total);
        }
        if (!tree_next(A, X, S.steps)) return;
        __syncthreads();
    }
}

template <int TY, int NK, int VW>
int launch_tree_many(const TreeArgs &A, void *stream)
{
    const void *fn = reinterpret_cast<const void *>(&k_tree_many<TY, NK, VW, 1>);
    if constexpr (NK <= 4) {
        if (A.tiles == 2) fn = reinterpret_cast<const void *>(&k_tree_many<TY, NK, VW, 2>);
    }
    return launch_kernel(fn, dim3(A.grid), dim3(kAttnBlock), A.direct ? 0 : rows_lds(A.b), stream, A);
}

template <int TY, int NK, int VW, AttnEdge EDGE>
int launch_tree_few(const TreeArgs &A, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_tree_few<TY, NK, VW, EDGE>), dim3(A.grid), dim3(kAttnBlock),
                         A.direct ? 0 : rows_lds(A.b), stream, A);
}

template <int TY, int NK, int VW>
int launch_tree_edge(const TreeArgs &A, void *stream)
{
    return A.d == (uint32_t)(NK * 4 * AttnType<TY>::E) ? launch_tree_few<TY, NK, VW, kExact>(A, stream)
                                                       : launch_tree_few<TY, NK, VW, kTail>(A, stream);
}

// The instance: the smallest that holds d and dv.
template <int TY>
int launch_tree_type(const TreeArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;   // 4 U pieces of 16 bytes: 32 elements
    const uint32_t d = A.d, dv = A.dv;
    if constexpr (TY != S_F32) {
        if (A.tiles) {
            if (d <= 64 && dv <= 64) return launch_tree_many<TY, 2, 4>(A, stream);
            if (dv <= 128)
                return d <= 96    ? launch_tree_many<TY, 3, 8>(A, stream)
                       : d <= 128 ? launch_tree_many<TY, 4, 8>(A, stream)
                       : d <= 192 ? launch_tree_many<TY, 6, 8>(A, stream)
                                  : launch_tree_many<TY, 8, 16>(A, stream);
            return d <= 192 ? launch_tree_many<TY, 6, 16>(A, stream) : launch_tree_many<TY, 8, 16>(A, stream);
        }
    }
    if (d < (uint32_t)E || dv < (uint32_t)E) return launch_tree_few<TY, 8 * U, 16, kTiny>(A, stream);
    // In binary32 products are what counts, so no more of them than there are: of keys in steps of 16
    // elements up to 96 (a piece of each of the four lanes), of values in steps of 64 (a piece of each
    // of the sixteen).  12 heads, 23 tokens, 5 rows in a window of 1000, by these and by the next
    // larger one that both types share: 80 and 64 25 and 38 us, 80 and 80 30 and 33, 96 and 64 25 and 31,
    // 128 and 64 27 and 33, 64 and 128 29 and 33; 8 whole rows of up to 3000, 16 tokens of 16 heads over
    // 4: 80 and 80 44 and 48, 96 and 64 40 and 47, 64 and 128 50 and 55.
    if constexpr (TY == S_F32) {
        if (dv <= 64 && d <= 128)
            return d <= 64   ? launch_tree_edge<TY, 4, 4>(A, stream)
                   : d <= 80 ? launch_tree_edge<TY, 5, 4>(A, stream)
                   : d <= 96 ? launch_tree_edge<TY, 6, 4>(A, stream)
                             : launch_tree_edge<TY, 8, 4>(A, stream);
        if (dv <= 128 && d <= 80) return d <= 64 ? launch_tree_edge<TY, 4, 8>(A, stream) : launch_tree_edge<TY, 5, 8>(A, stream);
    }
    if (d <= 64 && dv <= 64) return launch_tree_edge<TY, 2 * U, 4>(A, stream);
    if (dv <= 128) {
        if (d <= 96) return launch_tree_edge<TY, 3 * U, 8>(A, stream);
        if (d <= 128) return launch_tree_edge<TY, 4 * U, 8>(A, stream);
        if (d <= 192) return launch_tree_edge<TY, 6 * U, 8>(A, stream);
    } else if (d <= 192 && (TY != S_F32 || dv <= 192)) {
        return launch_tree_edge<TY, 6 * U, TY == S_F32 ? 12 : 16>(A, stream);
    }
    return launch_tree_edge<TY, 8 * U, 16>(A, stream);
}

}  // namespace

}  // namespace ecmd
