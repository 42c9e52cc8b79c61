// kernels_select.hip -- the least and largest key of every page, the choice of the
// pages that a query may care for most, and the eviction of the pages of least mass.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../ecmd_launch.h"
#include "ecmd_attn_tile.h"
#include "ecmd_serving.h"
#include "ecmd_wave.h"

namespace ecmd {

namespace {

template <int TY>
__device__ inline void to_floats(u32x4 x, float *f)
{
    if constexpr (TY == S_F32) {
#pragma unroll
        for (int w = 0; w < 4; ++w) f[w] = as_f(x[w]);
    } else if constexpr (TY == S_BF16) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            f[2 * w] = as_f(x[w] << 16);
            f[2 * w + 1] = as_f(x[w] & 0xFFFF0000u);
        }
    } else {
        const f16x8 h = __builtin_bit_cast(f16x8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)h[e];
    }
}

// Floats that are numbers of the type, back to it.
template <int TY>
__device__ inline u32x4 from_floats(const float *f)
{
    u32x4 x;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if constexpr (TY == S_F32) {
            x[w] = __builtin_bit_cast(uint32_t, f[w]);
        } else if constexpr (TY == S_BF16) {
            x[w] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[2 * w + 1]), __builtin_bit_cast(uint32_t, f[2 * w]), 0x07060302);
        } else {
            const f16x2 h = {(_Float16)f[2 * w], (_Float16)f[2 * w + 1]};
            x[w] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return x;
}

// ---------------------------------------------------------------------------
// Bounds.  A work-item takes a 16-byte piece of a page's slots, one after the other,
// eight loads ahead: neighbours read neighbours, so whole slots are read where heads
// lie side by side, and nothing is exchanged.  A last piece that would reach past its
// head is moved back to end with it; what two pieces then both write is the same.
template <int TY>
__global__ __launch_bounds__(256) void k_bounds(const BoundsArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E;
    const uint32_t r = A.by_groups.div(blockIdx.x), group = blockIdx.x - r * A.groups;
    const int32_t len = A.lens[(int64_t)r * A.lens_s], since = A.since[(int64_t)r * A.since_s];
    const uint32_t held = A.cols * A.page;
    const uint32_t lo = (uint32_t)max(since, 0), hi = min((uint32_t)max(len, 0), held);
    if (lo >= hi) return;
    const uint32_t c0 = A.by_page.div(lo), c1 = A.by_page.div(hi - 1) + 1;
    // A turn of a work-group: A.many columns, or a column's A.parts-th part.
    const uint32_t turns = A.many > 1 ? A.by_many.div(c1 - c0 + A.many - 1) : (c1 - c0) * A.parts;
    for (uint32_t turn = group; turn < turns; turn += A.groups) {
        uint32_t c, i;
        if (A.many > 1) {
            const uint32_t in = A.by_items.div(threadIdx.x);
            c = c0 + turn * A.many + in;
            i = threadIdx.x - in * A.items;
            if (in >= A.many) continue;
        } else {
            const uint32_t in = A.by_parts.div(turn);
            c = c0 + in;
            i = (turn - in * A.parts) * 256 + threadIdx.x;
        }
        if (c < c1 && i < A.items) {
            const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
            if (id < 0 || (uint32_t)id >= A.n) continue;
            const uint32_t h = A.by_head.div(i), piece = i - h * A.head_items;
            const uint32_t at = A.d < (uint32_t)E ? 0 : min(piece * E, A.d - E);
            const uint32_t s0 = c * A.page < lo ? lo - c * A.page : 0, s1 = min(A.page, hi - c * A.page);
            const char *k = (const char *)A.k + (int64_t)id * A.kcs[0] + (int64_t)h * A.kcs[2] + at * sizeof(T);
            char *b = (char *)A.bounds + (int64_t)id * A.bs[0] + (int64_t)h * A.bs[1] + at * sizeof(T);
            const bool tiny = A.d < (uint32_t)E;
            auto load = [&](const char *p) { return tiny ? load_some<T, E>(p, (int)A.d) : load16(p); };
            float least[E], most[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                least[e] = INFINITY;
                most[e] = -INFINITY;
            }
            if (s0) {
                to_floats<TY>(load(b), least);
                to_floats<TY>(load(b + A.bs[2]), most);
            }
            for (uint32_t s = s0; s < s1; s += 8) {
                u32x4 x[8];
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) x[u] = load(k + (int64_t)min(s + u, s1 - 1) * A.kcs[1]);
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) {
                    float f[E];
                    to_floats<TY>(x[u], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        least[e] = fminf(least[e], f[e]);
                        most[e] = fmaxf(most[e], f[e]);
                    }
                }
            }
            const u32x4 y[2] = {from_floats<TY>(least), from_floats<TY>(most)};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                char *p = b + w * A.bs[2];
                if (tiny) {
                    for (uint32_t e = 0; e < A.d; ++e) {
                        if constexpr (TY == S_F32) ((uint32_t *)p)[e] = y[w][e];
                        else ((uint16_t *)p)[e] = (uint16_t)(y[w][e / 2] >> (16 * (e & 1)));
                    }
                } else {
                    typedef u32x4 U __attribute__((aligned(2)));
                    *(U *)p = y[w];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The `want` largest of n keys (0: no candidate), of which there are more than that:
// the keys above `key`, and of those at it the first `ties` (all of them: kAll), by radix,
// eight bits at a time from bit `top` down.  It ends as soon as a digit's keys are
// wanted altogether: two or three turns where keys differ as measured data do.
struct Cut {
    uint64_t key;
    uint32_t ties;
};
constexpr uint32_t kAll = ~0u;

template <uint32_t THREADS>
struct CutScratch {
    uint32_t bins[256];
    uint32_t digit, above, inside;
    uint32_t wave[2][THREADS / 64];
};

template <uint32_t THREADS, class Get>
__device__ inline Cut cut_largest(uint32_t n, uint32_t want, int top, Get get, CutScratch<THREADS> &S)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    uint64_t prefix = 0, mask = 0;
    for (int shift = top; shift >= 0; shift -= 8) {
        for (uint32_t b = tid; b < 256; b += THREADS) S.bins[b] = 0;
        __syncthreads();
        for (uint32_t i = tid; i < n; i += THREADS) {
            const uint64_t k = get(i);
            if (k && (k & mask) == prefix) atomicAdd(&S.bins[(uint32_t)(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid < 64) {   // lane 0 has the four largest digits
            uint32_t c[4], sum = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                c[x] = S.bins[255 - 4 * lane - x];
                sum += c[x];
            }
            const uint32_t upto = wave_prefix(sum);
            uint32_t before = upto - sum;
            if (before < want && want <= upto) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (before < want && want <= before + c[x]) {
                        S.digit = 255 - 4 * lane - x;
                        S.above = before;
                        S.inside = c[x];
                    }
                    before += c[x];
                }
            }
        }
        __syncthreads();
        prefix |= (uint64_t)S.digit << shift;
        mask |= uint64_t(255) << shift;
        want -= S.above;
        if (S.inside == want) return Cut{prefix, kAll};   // whatever the lower bits are
        // (the barriers at the start of the next turn keep S until all have read it)
    }
    return Cut{prefix, want};
}

// Whether key k of column i is on the upper side, for columns in ascending order of
// THREADS at a time (all work-items call it alike): `seen` counts the ties so far.
template <uint32_t THREADS>
__device__ inline bool chosen(uint64_t k, const Cut &C, int top, uint32_t &seen, CutScratch<THREADS> &S)
{
    const uint64_t whole = top >= 56 ? ~uint64_t(0) : (uint64_t(1) << (top + 8)) - 1;
    const uint64_t x = k & whole;
    if (C.ties == kAll) return k && x >= C.key;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const bool tie = k && x == C.key;
    const uint64_t ties = __ballot(tie);
    if (lane == 0) S.wave[0][wave] = (uint32_t)__popcll(ties);
    __syncthreads();
    uint32_t rank = seen + (uint32_t)__popcll(ties & ((uint64_t(1) << lane) - 1));
#pragma unroll
    for (uint32_t w = 0; w < THREADS / 64; ++w) {
        if (w < wave) rank += S.wave[0][w];
        seen += S.wave[0][w];
    }
    __syncthreads();
    return k && (x > C.key || (tie && rank < C.ties));
}

// Doubles as integers of the same order; NaN the least.
__device__ inline uint64_t sortable(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x == 0.0 ? 0.0 : x);
    if (x != x) return 1;
    return b >> 63 ? ~b : b | uint64_t(1) << 63;
}

// ---------------------------------------------------------------------------
// Selection.

constexpr uint32_t kSelectHeads = 8;   // query heads in LDS at a time
constexpr uint64_t kForced = ~uint64_t(0);

struct RowPages {
    uint32_t used, hi;   // columns in use; positions
};
__device__ inline RowPages row_pages(const int32_t *lens, int64_t at, uint32_t cols, uint32_t page, const Div31 &by_page)
{
    const uint32_t hi = min((uint32_t)max(lens[at], 0), cols * page);
    return RowPages{hi ? by_page.div(hi - 1) + 1 : 0, hi};
}

// Scores of columns [c0, c1) of row r and kv head h into keys[c - c0] (LDS or memory).
// Eight lanes share a page: each has NP pieces of its bounds, for up to four query
// heads at a time.  Products and sums are binary64: whole numbers come of them, so
// what another order of summing would round otherwise must not show.
template <int TY, int NP>
__device__ inline void score_columns(const SelectArgs &A, uint32_t r, uint32_t h, uint32_t used, uint32_t c0, uint32_t c1,
                                     uint64_t *keys, double *s_q)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E;
    const uint32_t tid = threadIdx.x, width = 8 * E * NP;
    const uint32_t sub = tid & 7;
    for (uint32_t g0 = 0; g0 < A.group; g0 += kSelectHeads) {
        const uint32_t heads = min(kSelectHeads, A.group - g0);
        __syncthreads();   // the heads before are done with
        for (uint32_t i = tid; i < heads * width; i += blockDim.x) {
            const uint32_t g = i / width, e = i - g * width;
            double x = 0.0;
            if (e < A.d) {
                const char *p = (const char *)A.q + (int64_t)r * A.qs[0] + (int64_t)(h * A.group + g0 + g) * A.qs[1] + e * sizeof(T);
                if constexpr (TY == S_F32) x = *(const float *)p;
                else if constexpr (TY == S_BF16) x = (double)(float)*(const __bf16 *)p;
                else x = (double)(float)*(const _Float16 *)p;
            }
            s_q[i] = x;
        }
        __syncthreads();
        for (uint32_t base = c0; base < c1; base += blockDim.x / 8) {
            const uint32_t c = base + tid / 8;
            int32_t id = -1;
            if (c < c1) id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
            const bool held = id >= 0 && (uint32_t)id < A.n;
            const bool forced = c < A.first || c + A.last >= used;
            float lo[NP][E], hi[NP][E];
            const char *b = (const char *)A.bounds + (int64_t)(held ? id : 0) * A.bs[0] + (int64_t)h * A.bs[1];
            if (held && !forced) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const uint32_t at = (p * 8 + sub) * E;
                    u32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
                    if (at + E <= A.d) {
                        x = load16(b + at * sizeof(T));
                        y = load16(b + A.bs[2] + at * sizeof(T));
                    } else if (at < A.d) {
                        x = load_some<T, E>(b + at * sizeof(T), (int)(A.d - at));
                        y = load_some<T, E>(b + A.bs[2] + at * sizeof(T), (int)(A.d - at));
                    }
                    to_floats<TY>(x, lo[p]);
                    to_floats<TY>(y, hi[p]);
                }
            }
            uint64_t best = 0;
            for (uint32_t g = 0; g < heads; g += 4) {
                double sum[4] = {0.0, 0.0, 0.0, 0.0};
                if (held && !forced) {
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (g + u >= heads) break;
                            const double *q = s_q + (g + u) * width + (p * 8 + sub) * E;
#pragma unroll
                            for (int e = 0; e < E; ++e) sum[u] = __builtin_fma(q[e], (double)(q[e] < 0.0 ? lo[p][e] : hi[p][e]), sum[u]);
                        }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (g + u >= heads) break;
                    sum[u] += __shfl_xor(sum[u], 1);
                    sum[u] += __shfl_xor(sum[u], 2);
                    sum[u] += __shfl_xor(sum[u], 4);
                    const uint64_t k = sortable(sum[u]);
                    best = k > best ? k : best;
                }
            }
            if (sub == 0 && c < c1) {
                uint64_t k = !held ? 0 : forced ? kForced : best;
                if (g0) {
                    const uint64_t old = keys[c - c0];
                    k = old > k ? old : k;
                }
                keys[c - c0] = k;
            }
        }
    }
}

// The table of row r and kv head h from the keys of its columns.
template <uint32_t THREADS, class Get>
__device__ inline void choose_columns(const SelectArgs &A, uint32_t r, uint32_t h, const RowPages &P, Get get,
                                      CutScratch<THREADS> &S)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    uint32_t held = 0;
    for (uint32_t c = tid; c < P.used; c += THREADS) held += get(c) != 0;
    held = wave_sum(held);
    if (lane == 0) S.wave[0][wave] = held;
    __syncthreads();
    held = 0;
#pragma unroll
    for (uint32_t w = 0; w < THREADS / 64; ++w) held += S.wave[0][w];
    __syncthreads();
    Cut C{0, kAll};   // all of them
    if (held > A.take) C = cut_largest<THREADS>(P.used, A.take, 56, get, S);
    int32_t *out = A.pages_out + (int64_t)r * A.pages_out_s[0] + (int64_t)h * A.pages_out_s[1];
    uint32_t count = 0, seen = 0;
    __syncthreads();
    const uint32_t all = min(held, A.take);
    if (all == 0 && tid == 0) A.lens_out[(int64_t)r * A.lens_out_s[0] + (int64_t)h * A.lens_out_s[1]] = 0;
    for (uint32_t base = 0; base < P.used && count < all; base += THREADS) {
        const uint32_t c = base + tid;
        const uint64_t k = c < P.used ? get(c) : 0;
        const bool in = chosen<THREADS>(k, C, 56, seen, S);
        const uint64_t these = __ballot(in);
        if (lane == 0) S.wave[1][wave] = (uint32_t)__popcll(these);
        __syncthreads();
        uint32_t at = count + (uint32_t)__popcll(these & ((uint64_t(1) << lane) - 1));
#pragma unroll
        for (uint32_t w = 0; w < THREADS / 64; ++w) {
            if (w < wave) at += S.wave[1][w];
            count += S.wave[1][w];
        }
        __syncthreads();
        if (in) {
            out[(int64_t)at * A.pages_out_s[2]] = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
            if (at + 1 == all)
                A.lens_out[(int64_t)r * A.lens_out_s[0] + (int64_t)h * A.lens_out_s[1]] =
                    (int32_t)(at * A.page + (c + 1 == P.used ? P.hi - c * A.page : A.page));
        }
    }
    for (uint32_t i = all + tid; i < A.take; i += THREADS) out[(int64_t)i * A.pages_out_s[2]] = -1;
}

// One work-group to a row and kv head: scores, keys in LDS, choice.
template <int TY, int NP>
__global__ __launch_bounds__(256) void k_select_alone(const SelectArgs A)
{
    extern __shared__ __attribute__((aligned(16))) uint64_t s_dynamic[];
    __shared__ CutScratch<256> S;
    const uint32_t r = A.by_hk.div(blockIdx.x), h = blockIdx.x - r * A.hk;
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    uint64_t *keys = s_dynamic;
    double *s_q = (double *)(s_dynamic + (A.cols + 1) / 2 * 2);
    if (P.used <= A.take) {   // all that are held: no scores
        for (uint32_t c = threadIdx.x; c < P.used; c += 256) {
            const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
            keys[c] = id >= 0 && (uint32_t)id < A.n ? kForced : 0;
        }
    } else {
        score_columns<TY, NP>(A, r, h, P.used, 0, P.used, keys, s_q);
    }
    __syncthreads();
    choose_columns<256>(A, r, h, P, [&](uint32_t c) { return keys[c]; }, S);
}

// Many columns and few rows: A.groups work-groups score a row and kv head, one chooses.
template <int TY, int NP>
__global__ __launch_bounds__(256) void k_select_score(const SelectArgs A)
{
    extern __shared__ __attribute__((aligned(16))) uint64_t s_dynamic[];
    const uint32_t x = A.by_groups.div(blockIdx.x), part = blockIdx.x - x * A.groups;
    const uint32_t r = A.by_hk.div(x), h = x - r * A.hk;
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    const uint32_t each = (P.used + A.groups - 1) / A.groups, c0 = min(part * each, P.used), c1 = min(c0 + each, P.used);
    if (c0 < c1) score_columns<TY, NP>(A, r, h, P.used, c0, c1, A.keys + (uint64_t)x * A.cols + c0, (double *)s_dynamic);
}

__global__ __launch_bounds__(1024) void k_select_choose(const SelectArgs A)
{
    __shared__ CutScratch<1024> S;
    const uint32_t r = A.by_hk.div(blockIdx.x), h = blockIdx.x - r * A.hk;
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    const uint64_t *keys = A.keys + (uint64_t)blockIdx.x * A.cols;
    choose_columns<1024>(A, r, h, P, [&](uint32_t c) { return keys[c]; }, S);
}

template <int TY, int NP>
int launch_select_one(const SelectArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E;
    const uint32_t q_lds = std::min(A.group, kSelectHeads) * 8 * E * NP * 8;
    if (!A.keys)
        return launch_kernel(reinterpret_cast<const void *>(&k_select_alone<TY, NP>), dim3(A.b * A.hk), dim3(256),
                             (A.cols + 1) / 2 * 16 + q_lds, stream, A);
    const int rc = launch_kernel(reinterpret_cast<const void *>(&k_select_score<TY, NP>), dim3(A.b * A.hk * A.groups), dim3(256),
                                 q_lds, stream, A);
    if (rc) return rc;
    return launch_kernel(reinterpret_cast<const void *>(&k_select_choose), dim3(A.b * A.hk), dim3(1024), 0, stream, A);
}

template <int TY>
int launch_select_type(const SelectArgs &A, void *stream)
{
    constexpr int U = 8 / AttnType<TY>::E;
    return A.d <= 64 ? launch_select_one<TY, U>(A, stream)
           : A.d <= 128 ? launch_select_one<TY, 2 * U>(A, stream)
                        : launch_select_one<TY, 4 * U>(A, stream);
}

// ---------------------------------------------------------------------------
// Eviction.  A work-group to a row.  Keys of up to kSelectAlone columns stay in LDS, those
// of longer rows are made anew from the masses in each turn.

__global__ __launch_bounds__(256) void k_evict_refs(const EvictArgs A)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < A.n) A.refs_out[(int64_t)i * A.refs_out_s] = A.refs[(int64_t)i * A.refs_s];
}

template <bool KEPT>
__global__ __launch_bounds__(256) void k_evict(const EvictArgs A)
{
    extern __shared__ uint64_t s_keys[];
    __shared__ CutScratch<256> S;
    const uint32_t r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    const int32_t *pages = A.pages + (int64_t)r * A.pages_s[0];
    const float *mass = A.mass + (int64_t)r * A.mass_s[0];
    int32_t *out = A.pages_out + (int64_t)r * A.pages_out_s[0];
    // the less mass, the larger; 0: not to be taken out
    auto make = [&](uint32_t c, int32_t id) {
        if (id < 0 || (uint32_t)id >= A.n || c < A.first || c + A.last >= P.used) return uint64_t(0);
        const float x = mass[(int64_t)c * A.mass_s[1]];
        uint32_t b = __builtin_bit_cast(uint32_t, x == 0.0f ? 0.0f : x);
        b = x != x ? ~0u : b >> 31 ? ~b : b | 1u << 31;
        return uint64_t(1) << 32 | (uint32_t)~b;
    };
    uint32_t held = 0, loose = 0;
    for (uint32_t c = tid; c < P.used; c += 256) {
        const int32_t id = pages[(int64_t)c * A.pages_s[1]];
        held += id >= 0 && (uint32_t)id < A.n;
        const uint64_t k = make(c, id);
        loose += k != 0;
        if (KEPT) s_keys[c] = k;
    }
    held = wave_sum(held);
    loose = wave_sum(loose);
    if (lane == 0) {
        S.wave[0][wave] = held;
        S.wave[1][wave] = loose;
    }
    __syncthreads();
    held = loose = 0;
#pragma unroll
    for (uint32_t w = 0; w < 4; ++w) {
        held += S.wave[0][w];
        loose += S.wave[1][w];
    }
    __syncthreads();
    const uint32_t budget = (uint32_t)max(A.budget[(int64_t)r * A.budget_s], 0);
    const uint32_t over = held > budget ? min(held - budget, loose) : 0;
    auto get = [&](uint32_t c) { return KEPT ? s_keys[c] : make(c, pages[(int64_t)c * A.pages_s[1]]); };
    Cut C{0, kAll};
    if (over && over < loose) C = cut_largest<256>(P.used, over, 24, get, S);
    __syncthreads();
    uint32_t seen = 0;
    for (uint32_t base = 0; base < A.cols; base += 256) {
        const uint32_t c = base + tid;
        const int32_t id = c < A.cols ? pages[(int64_t)c * A.pages_s[1]] : -1;
        bool gone = false;
        if (over && base < P.used) gone = chosen<256>(c < P.used ? get(c) : 0, C, 24, seen, S);
        if (gone) atomicSub(&A.refs_out[(int64_t)id * A.refs_out_s], 1);
        if (c < A.cols) out[(int64_t)c * A.pages_out_s[1]] = gone || id < 0 || (uint32_t)id >= A.n ? -1 : id;
    }
    if (tid == 0) A.count[(int64_t)r * A.count_s] = (int32_t)over;
}

}  // namespace

int launch_bounds(int type, const BoundsArgs &A, void *stream)
{
    const void *fn = type == S_F16    ? reinterpret_cast<const void *>(&k_bounds<S_F16>)
                     : type == S_BF16 ? reinterpret_cast<const void *>(&k_bounds<S_BF16>)
                                      : reinterpret_cast<const void *>(&k_bounds<S_F32>);
    return launch_kernel(fn, dim3(A.rows * A.groups), dim3(256), 0, stream, A);
}

int launch_select(int type, const SelectArgs &A, void *stream)
{
    return type == S_F16    ? launch_select_type<S_F16>(A, stream)
           : type == S_BF16 ? launch_select_type<S_BF16>(A, stream)
                            : launch_select_type<S_F32>(A, stream);
}

int launch_evict(const EvictArgs &A, void *stream)
{
    if (A.copy && A.n)
        if (const int rc = launch_kernel(reinterpret_cast<const void *>(&k_evict_refs), dim3((A.n + 255) / 256), dim3(256), 0, stream, A))
            return rc;
    if (A.rows == 0) return 0;
    if (A.cols <= kSelectAlone)
        return launch_kernel(reinterpret_cast<const void *>(&k_evict<true>), dim3(A.rows), dim3(256), A.cols * 8, stream, A);
    return launch_kernel(reinterpret_cast<const void *>(&k_evict<false>), dim3(A.rows), dim3(256), 0, stream, A);
}

}  // namespace ecmd
