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
// The four waves of a work-group split the positions where there are few queries,
// and the queries where there are many.  Which tokens a token attends to is one bit
// mask per token, made in LDS from the parents by pointer doubling; a tile of 32
// keys takes the 32 bits of it that lie above its keys, so only the tiles at the end
// of a row (or at the start of a window) look at single keys.
//
// Rows are dealt to work-groups as in one token's attention: positions in steps,
// laid end to end and cut into equal runs, the segments of a cut row joined by a
// second launch.
#pragma once
#include <hip/hip_runtime.h>

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

__device__ inline void make_tree(const TreeArgs &A, uint32_t r, const Tree &T)
{
    const uint32_t i = threadIdx.x, words = (A.t + 31) / 32;
    uint32_t mask[kTreeWords];
    int32_t jump = -1;
    uint32_t bad = 0;
    if (i < kTreeWords) T.real[i] = 0;
    if (i < A.t) {
        const int32_t p = A.parent[(int64_t)r * A.parent_s[0] + (int64_t)i * A.parent_s[1]];
        const bool fine = p >= 0 && (uint32_t)p < i;
        bad = !fine && p != -1;
        jump = fine ? p : -1;
#pragma unroll
        for (uint32_t w = 0; w < kTreeWords; ++w) mask[w] = w == i / 32 ? 1u << (i % 32) : 0;
    }
    // info: the next token up that the mask does not have yet, or -1, with bit 30 for padding
    for (;;) {
        if (i < A.t) {
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) T.mask[i * words + w] = mask[w];
            T.info[i] = jump < 0 ? (bad ? -2 : -1) : jump;
        }
        if (!__syncthreads_or(jump >= 0)) break;
        if (i < A.t && jump >= 0) {
            const uint32_t up = (uint32_t)jump;
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) mask[w] |= T.mask[up * words + w];
            jump = T.info[up];
            bad = jump == -2;
        }
        __syncthreads();
    }
    int32_t above = -1;
    if (i < A.t && !bad) {
#pragma unroll
        for (uint32_t w = 0; w < kTreeWords; ++w) above += __popc(mask[w]);
    }
    __syncthreads();
    if (i < A.t) {
        T.info[i] = bad ? -1 : above;
        if (!bad) atomicOr(&T.real[i / 32], 1u << (i % 32));
    }
    __syncthreads();
    if (A.window && i < A.t && !bad && (uint32_t)above >= A.window) {
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

// Steps of a run, the same in every work-group and in the join; 0: runs are rows.
__device__ inline uint32_t tree_share(const TreeArgs &A, const Rows &R)
{
    // rows of nearly one length, enough of them to use the whole chip
    if (A.b <= A.runs_whole && (uint64_t)R.all * 5 >= (uint64_t)R.longest * A.b * 4) return 0;
    const uint32_t share = A.by_runs.div(R.all + A.runs - 1);
    return R.longest <= 2 * share && A.b <= max(A.runs, A.runs_whole) ? 0 : share;
}

template <int TY, int NK, int VW, int NT>
constexpr int tree_waves()
{
    constexpr int KB = AttnType<TY>::KB, size = TY == S_F32 ? 4 : 2;
    constexpr int regs = KB * NK * 4 + KB * VW * size + NT * (NK * 4 + VW * 4 + KB * 8) + 60;
    return regs > 236 ? 1 : 2;
}

template <int TY, int NK, int VW, AttnEdge EDGE, int NT>
__global__ __launch_bounds__(kAttnBlock, (tree_waves<TY, NK, VW, NT>())) void k_tree(const TreeArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, KB = AttnType<TY>::KB;
    constexpr int VK = 4 * KB;                          // keys whose values a lane holds
    constexpr int PE = VW < E ? VW : E, VP = VW / PE;   // elements of a value piece; pieces
    constexpr int PW = PE * (int)sizeof(T) / 4;         // words of a value piece
    constexpr uint32_t kTile = 16 * KB;
    constexpr int kRow = 16 * VW + 4;                   // a query's row in the joining buffer (floats)

    __shared__ union {
        struct {
            uint64_t k[kAttnWaves][kTableKeys], v[kAttnWaves][kTableKeys];
            uint64_t valid[kAttnWaves][kTableKeys / 64];
        } table;
        __attribute__((aligned(16))) float join[kAttnWaves][8][kRow];
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

    // Work-groups go to the eight dies in turn: those of a run follow each other on one.
    const uint32_t u8 = A.by_units.div(blockIdx.x), in8 = blockIdx.x - u8 * A.by_units.d;
    const uint32_t group = u8 * 8 + in8 % 8, unit = in8 / 8;
    const uint32_t kvh = A.by_blocks.div(unit), block = unit - kvh * A.q_blocks;
    uint32_t r, step = 0, stop = 0;
    Rows R{};
    if (A.direct) {
        if (group >= A.b) return;
        r = group;
    } else {
        R = make_rows(A, s_rows, s_scratch, tree_span);
        const uint32_t share = tree_share(A, R);
        if (share == 0) {
            if (group >= A.b) return;
            r = group;
            step = __builtin_amdgcn_readfirstlane(R.prefix[r]);
            stop = __builtin_amdgcn_readfirstlane(R.prefix[r + 1]);
            if (step == stop) return;
        } else {
            if ((uint64_t)group * share >= R.all) return;
            step = group * share;
            stop = min(step + share, R.all);
            uint32_t lo = 0, hi = A.b;   // the row with prefix[r] <= step < prefix[r + 1]
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                if (__builtin_amdgcn_readfirstlane(R.prefix[mid]) <= step) lo = mid;
                else hi = mid;
            }
            r = lo;
        }
    }
    const uint32_t qw = wave & ((1u << A.q_shift) - 1), part = wave >> A.q_shift, parts = kAttnWaves >> A.q_shift;
    const uint32_t q0 = ((block << A.q_shift) + qw) * (16 * NT);   // the wave's first query vector

    auto column = [&](uint32_t m, int piece) {
        const uint32_t at = (piece * 16 + m) * PE;
        return EDGE == kTiny ? at : min(at, A.dv - PE);
    };
    auto load_row_piece = [&](const char *p, int c) {
        const int at = (c * 4 + (int)j) * E;
        if constexpr (EDGE == kTiny) return load_some<T, E>(p + at * sizeof(T), (int)A.d - at);
        return load16(p + (EDGE == kTail ? min(at, (int)A.d - E) : at) * sizeof(T));
    };
    // clears what an earlier piece has of one that was moved back to end with the row
    auto masked = [&](u32x4 x, int c) {
        if (EDGE == kTail && (uint32_t)(c + 1) * 4 * E > A.d) {
            const int at = (c * 4 + (int)j) * E, twice = at - min(at, (int)A.d - E);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if constexpr (E == 8)
                    x[w] &= (2 * w >= twice ? 0xFFFFu : 0u) | (2 * w + 1 >= twice ? 0xFFFF0000u : 0u);
                else
                    x[w] &= w >= twice ? ~0u : 0u;
            }
        }
        return x;
    };

    const char *kbase = (const char *)A.k + (int64_t)kvh * A.kcs[2];
    const char *vbase = (const char *)A.v + (int64_t)kvh * A.vcs[2];

    for (;;) {   // one row of the run
        const uint32_t len = (uint32_t)A.lens[(int64_t)r * A.lens_s];   // negative rows have no steps
        uint32_t begin, end, steps = 0;
        bool whole_row = true, last_part = true;
        if (A.direct) {
            const Span span = tree_span(A, r);
            begin = span.lo;
            end = span.hi;
        } else {
            const uint32_t first = __builtin_amdgcn_readfirstlane(R.prefix[r]);
            const uint32_t last = __builtin_amdgcn_readfirstlane(R.prefix[r + 1]);
            const uint32_t here = min(stop, last), hi = __builtin_amdgcn_readfirstlane(R.hi[r]);
            last_part = here == last;
            whole_row = step == first && last_part;
            steps = here - step;
            begin = __builtin_amdgcn_readfirstlane(R.lo[r]) + (step - first) * kAttnStep;
            end = min(begin + steps * kAttnStep, hi);
        }
        const bool nobody = (int32_t)len < 0;   // A.direct only: a row of padding
        // the tree matters to the tiles past the context, to a window's start and to who is padding
        const bool looks = last_part || A.window != 0 || end > len;
        if (looks) make_tree(A, r, tree);

        uint32_t wb = begin, we = end;
        if (parts > 1) {
            const uint32_t each = (end - begin + parts * kTile - 1) / (parts * kTile) * kTile;
            wb = min(begin + part * each, end);
            we = min(wb + each, end);
        }
        if (q0 >= A.m) we = wb;   // no queries of this wave's

        u32x4 q[NT][NK];
        uint32_t token[NT], lo[NT];   // of the lane's queries: the token, the first position that counts
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t m = min(q0 + n * 16 + hh, A.m - 1);
            token[n] = A.by_group.div(m);
            const uint32_t head = kvh * A.group + m - token[n] * A.group;
            const char *p = (const char *)A.q + ((int64_t)r * A.qs[0] + (int64_t)token[n] * A.qs[1] + (int64_t)head * A.qs[2]) * sizeof(T);
#pragma unroll
            for (int c = 0; c < NK; ++c) q[n][c] = masked(load_row_piece(p, c), c) ^ u32x4{A.q_flip, A.q_flip, A.q_flip, A.q_flip};
            lo[n] = 0;
            if (A.window) {
                const uint32_t past = len + (uint32_t)max(s_info[token[n]], 0) + 1;
                lo[n] = past > A.window ? past - A.window : 0;
            }
        }

        f32x4 acc[NT][VW];
        float m[NT], mref[NT], l[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -INFINITY;
            mref[n] = 0.0f;
            l[n] = 0.0f;
#pragma unroll
            for (int c = 0; c < VW; ++c) acc[n][c] = f32x4{0, 0, 0, 0};
        }

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
                    const uint32_t at = column(hh, c);
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
            f32x4 s[NT][KB];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) s[n][kb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int c = 0; c < NK; ++c) {
                    const u32x4 k = masked(kr[kb][c], c);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (TY == S_F32) {
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                s[n][kb] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(k[f]), as_f(q[n][c][f]), s[n][kb], 0, 0, 0);
                        } else {
                            s[n][kb] = mma16<TY>(k, q[n][c], s[n][kb]);
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
            const bool whole = now == (KB == 2 ? 0xFFFFFFFFu : 0xFFFFu) && t0 + kTile <= len &&
                               (A.window == 0 || t0 + A.window >= len + A.t);
            uint32_t allow[NT];
            bool odd = false;   // some query leaves out a value that is no finite number
            if (!whole) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t see = ~0u;
                    if (t0 + kTile > len) {
                        const uint32_t *w = s_mask + token[n] * words;
                        if (t0 < len) {
                            see = (1u << (len - t0)) - 1 | w[0] << (len - t0);   // len - t0 < kTile <= 32
                        } else {
                            const uint32_t o = t0 - len, at = o / 32;
                            const uint64_t two = (at < words ? w[at] : 0) | (uint64_t)(at + 1 < words ? w[at + 1] : 0) << 32;
                            see = (uint32_t)(two >> (o % 32));
                        }
                    }
                    if (lo[n] > t0) see &= lo[n] - t0 < 32 ? ~0u << (lo[n] - t0) : 0;
                    allow[n] = see & now;
                }
#pragma unroll
                for (int x = 0; x < VK; ++x) {
                    // a slot that holds nothing may hold NaN: its value is cleared
                    const bool ok = now >> ((x / 4) * 16 + j * 4 + x % 4) & 1;
                    const uint32_t keep = ok ? ~0u : 0u;
#pragma unroll
                    for (int c = 0; c < VP; ++c) {
                        vr[x][c] = vr[x][c] & u32x4{keep, keep, keep, keep};
                        constexpr uint32_t top = TY == S_F16 ? 0x7C00u : TY == S_BF16 ? 0x7F80u : 0x7F800000u;
#pragma unroll
                        for (int w = 0; w < PW; ++w) {
                            odd |= (vr[x][c][w] & top) == top;
                            if constexpr (TY != S_F32) odd |= (vr[x][c][w] >> 16 & top) == top;
                        }
                    }
                }
            }

            float p[NT][VK];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < VK; ++x) {
                    p[n][x] = s[n][x / 4][x % 4] * A.scale_log2;
                    if (!whole) p[n][x] = allow[n] >> ((x / 4) * 16 + j * 4 + x % 4) & 1 ? p[n][x] : -INFINITY;
                    top = fmaxf(top, p[n][x]);
                }
                if (__any(top > m[n] + kTreeSlack<TY>)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float mn = fmaxf(m[n], top);
                    mref[n] = mn == -INFINITY ? 0.0f : mn;
                    const float a = __builtin_amdgcn_exp2f(m[n] - mref[n]);
                    m[n] = mn;
                    l[n] *= a;
#pragma unroll
                    for (int c = 0; c < VW; ++c) acc[n][c] *= a;
                }
#pragma unroll
                for (int x = 0; x < VK; ++x) {
                    p[n][x] = __builtin_amdgcn_exp2f(p[n][x] - (mref[n] - kTreeBias<TY>));
                    l[n] += p[n][x];
                }
            }

            // A weight of 0 times an infinity is NaN: where a query leaves such a value
            // out, all values of that kind are taken out of the products and added one
            // by one.  Tiles at a row's end only, and hardly ever.
            if (!whole && __any(odd)) {
                for (uint32_t key = 0; key < kTile; ++key) {
                    if (!(now >> key & 1)) continue;
                    const uint32_t pos = t0 + key, col = A.by_page.div(pos);
                    const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)col * A.pages_s[1]];
                    const char *v = vbase + (int64_t)id * A.vcs[0] + (int64_t)(pos - col * A.page) * A.vcs[1];
                    const uint32_t from = (key % 16) / 4 * 16 + hh;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float w = 0.0f;
#pragma unroll
                        for (int x = 0; x < VK; ++x) {
                            const float got = __shfl(p[n][x], (int)from);
                            if (key / 16 * 4 + key % 4 == (uint32_t)x) w = got;
                        }
                        if (!(allow[n] >> key & 1)) continue;
#pragma unroll
                        for (int c = 0; c < VW; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t at = column(j * 4 + i, c / PE) + c % PE;
                                if (at >= A.dv) continue;
                                float value;
                                if constexpr (TY == S_F32) value = ((const float *)v)[at];
                                else if constexpr (TY == S_BF16) value = (float)((const __bf16 *)v)[at];
                                else value = (float)((const _Float16 *)v)[at];
                                if (!(fabsf(value) < INFINITY)) acc[n][c][i] += w * value;
                            }
                    }
                }
#pragma unroll
                for (int x = 0; x < VK; ++x)
#pragma unroll
                    for (int c = 0; c < VP; ++c)
#pragma unroll
                        for (int w = 0; w < PW; ++w) {
                            constexpr uint32_t top = TY == S_F16 ? 0x7C00u : TY == S_BF16 ? 0x7F80u : 0x7F800000u;
                            uint32_t y = vr[x][c][w];
                            if ((y & top) == top) y &= TY == S_F32 ? 0u : 0xFFFF0000u;
                            if constexpr (TY != S_F32)
                                if ((y >> 16 & top) == top) y &= 0xFFFFu;
                            vr[x][c][w] = y;
                        }
            }

            if constexpr (TY == S_F32) {
#pragma unroll
                for (int x = 0; x < VK; ++x)
#pragma unroll
                    for (int c = 0; c < VW; ++c)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(vr[x][c / 4][c % 4]), p[n][x], acc[n][c], 0, 0, 0);
            } else {
                // A weight goes in as the sum of two 16-bit numbers, its leading bits and the
                // rest: one would add its own rounding of half a step of the type to the result's.
                // Both are positive wherever the weight is (bfloat16: the rest at least 2^-20 of the
                // leading part; binary16: the smallest number), since an infinite value times 0
                // would be NaN.
                u32x4 hi[NT], rest[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < VK; x += 2) {
                        const float f = p[n][x], g = p[n][x + 1];
                        const uint32_t a = __builtin_bit_cast(uint32_t, f), b = __builtin_bit_cast(uint32_t, g);
                        if constexpr (TY == S_BF16) {
                            const uint32_t h = __builtin_amdgcn_perm(b, a, 0x07060302);
                            const uint32_t e = __builtin_amdgcn_perm(
                                __builtin_bit_cast(uint32_t, g - as_f(b & 0xFFFF0000u)),
                                __builtin_bit_cast(uint32_t, f - as_f(a & 0xFFFF0000u)), 0x07060302);
                            const u16x2 least = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, h), u16x2{20 << 7, 20 << 7});
                            hi[n][x / 2] = h;
                            rest[n][x / 2] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, e), least));
                        } else {
                            // positive numbers order as their bits do
                            const u16x2 least = __builtin_bit_cast(u16x2, min(a, 1u) | min(b, 1u) << 16);
                            const u16x2 h = __builtin_elementwise_max(__builtin_bit_cast(u16x2, __builtin_amdgcn_cvt_pkrtz(f, g)), least);
                            const f16x2 hf = __builtin_bit_cast(f16x2, h);
                            const u16x2 e = __builtin_bit_cast(u16x2, __builtin_amdgcn_cvt_pkrtz(fmaxf(f - (float)hf[0], 0.0f), fmaxf(g - (float)hf[1], 0.0f)));
                            hi[n][x / 2] = __builtin_bit_cast(uint32_t, h);
                            rest[n][x / 2] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(e, least));
                        }
                    }
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    u32x4 a;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        a[w] = __builtin_amdgcn_perm(vr[2 * w + 1][c / 8][c % 8 / 2], vr[2 * w][c / 8][c % 8 / 2],
                                                     c & 1 ? 0x07060302 : 0x05040100);
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n][c] = mma16<TY>(a, rest[n], acc[n][c]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n][c] = mma16<TY>(a, hi[n], acc[n][c]);
                }
            }
            if (tile < we) load_v(in_table);
        }

        // The segment's sums: final, or for the second launch at a place of its own
        // (work-groups and rows only go forward).
        const uint64_t place = (uint64_t)(group + r) * A.by_vectors.d + (uint64_t)kvh * A.m;
        auto put = [&](uint32_t x, uint32_t c, float sum, float total) {   // query vector x
            if (!whole_row) {
                A.acc[(place + x) * A.dv + c] = sum;
                return;
            }
            const uint32_t tok = A.by_group.div(x), head = kvh * A.group + x - tok * A.group;
            store_typed(TY, A.out, (int64_t)r * A.os[0] + (int64_t)tok * A.os[1] + (int64_t)head * A.os[2] + c,
                        total > 0.0f ? sum / total : total == 0.0f || total < 0.0f ? 0.0f : total);
        };
        auto put_statistics = [&](uint32_t x, float top, float total) {
            if (!whole_row) {
                A.ml[2 * (place + x)] = top;
                A.ml[2 * (place + x) + 1] = total;
            } else if (A.lse) {
                const uint32_t tok = A.by_group.div(x), head = kvh * A.group + x - tok * A.group;
                A.lse[(int64_t)r * A.ls[0] + (int64_t)tok * A.ls[1] + (int64_t)head * A.ls[2]] = tree_log_sum<TY>(top, total);
            }
        };
        // the sum of weights, -1 for padding
        auto known = [&](uint32_t x, float total) {
            return last_part && (nobody || s_info[A.by_group.div(x)] < 0) ? -1.0f : total;
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
        }
        if (parts == 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t x = q0 + n * 16 + hh;
                if (x < A.m) {
                    const float total = known(x, l[n]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < VW; ++c) {
                            const uint32_t at = column(j * 4 + i, c / PE) + c % PE;
                            if (EDGE != kTiny || at < A.dv) put(x, at, acc[n][c][i], total);
                        }
                    if (j == 0) put_statistics(x, m[n], total);
                }
            }
        } else {
            // Waves with the same queries: common maximum, then sums through LDS, eight
            // queries at a time and four columns to a work-item.
            const uint32_t hw = 1u << A.q_shift;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if ((uint32_t)n * 16 >= A.m) break;   // the same for all waves: barriers follow
                __syncthreads();   // the tables, or the buffers, are done with
                if (j == 0) {
                    s_m[wave][hh] = m[n];
                    s_l[wave][hh] = l[n];
                }
                __syncthreads();
                float top = -INFINITY, total = 0.0f;
                for (uint32_t w = qw; w < kAttnWaves; w += hw) top = fmaxf(top, s_m[w][hh]);
                const float ref = top == -INFINITY ? 0.0f : top;
                for (uint32_t w = qw; w < kAttnWaves; w += hw) total += s_l[w][hh] * __builtin_amdgcn_exp2f(s_m[w][hh] - ref);
                const float factor = __builtin_amdgcn_exp2f(m[n] - ref);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half) __syncthreads();
                    if ((hh >> 3) == (uint32_t)half) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < VW; ++c)
                                sh.join[wave][hh & 7][column(j * 4 + i, c / PE) + c % PE] = acc[n][c][i] * factor;
                    }
                    __syncthreads();
                    for (uint32_t y = part * 64 + lane; y < 8 * 4 * VW; y += parts * 64) {
                        const uint32_t g = y / (4 * VW), c = y % (4 * VW) * 4, x = q0 + n * 16 + half * 8 + g;
                        // lane g + 8 half of every wave of these has the statistics
                        const float all = __shfl(total, (int)(half * 8 + g)), best = __shfl(top, (int)(half * 8 + g));
                        if (x >= A.m) continue;
                        f32x4 sum = *(const f32x4 *)&sh.join[qw][g][c];
                        for (uint32_t w = qw + hw; w < kAttnWaves; w += hw) sum += *(const f32x4 *)&sh.join[w][g][c];
                        const float t = known(x, all);
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            if (c + k < A.dv) put(x, c + k, sum[k], t);
                        if (c == 0) put_statistics(x, best, t);
                    }
                }
            }
        }
        if (A.direct) return;
        step += steps;
        if (step >= stop) return;
        do ++r;
        while (__builtin_amdgcn_readfirstlane(R.prefix[r + 1]) <= step);   // past empty rows
        __syncthreads();
    }
}

template <int TY, int NK, int VW, AttnEdge EDGE>
int launch_tree_one(const TreeArgs &A, void *stream)
{
    const void *fn = reinterpret_cast<const void *>(&k_tree<TY, NK, VW, EDGE, 1>);
    return launch_kernel(fn, dim3(A.grid), dim3(kAttnBlock), A.direct ? 0 : rows_lds(A.b), stream, A);
}

// The instance: the smallest that holds d and dv (see tree_tiles on the host for the
// number of tiles).
template <int TY>
int launch_tree_type(const TreeArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;   // 4 U pieces of 16 bytes: 32 elements
    const uint32_t d = A.d, dv = A.dv;
    if (d < (uint32_t)E || dv < (uint32_t)E) return launch_tree_one<TY, 8 * U, 16, kTiny>(A, stream);
    if (d <= 64 && dv <= 64)
        return d == 64 ? launch_tree_one<TY, 2 * U, 4, kExact>(A, stream) : launch_tree_one<TY, 2 * U, 4, kTail>(A, stream);
    if (d <= 128 && dv <= 128)
        return d == 128 ? launch_tree_one<TY, 4 * U, 8, kExact>(A, stream) : launch_tree_one<TY, 4 * U, 8, kTail>(A, stream);
    return d == 256 ? launch_tree_one<TY, 8 * U, 16, kExact>(A, stream) : launch_tree_one<TY, 8 * U, 16, kTail>(A, stream);
}

}  // namespace

}  // namespace ecmd
