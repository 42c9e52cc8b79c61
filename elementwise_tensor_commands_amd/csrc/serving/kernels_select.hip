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
// head is moved back to end with it; what two pieces then both write is the same.  16 ragged
// prompts of up to 4000 positions, 4 heads of 96, f16 (28 MB): 6.9 us, 4.0 TB/s; after a decode
// step of 64 rows 5.3: a chain from lengths over pages to slots.
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
// eight bits at a time from the highest in which two of them differ (those of kForced are
// taken out first: they would differ from all).  It ends as soon as a digit's keys are
// wanted altogether: two turns where keys differ as measured data do.
struct Cut {
    uint64_t key;
    uint32_t ties;
};
constexpr uint32_t kAll = ~0u;
constexpr uint64_t kForced = ~uint64_t(0);

struct Keys {
    uint32_t held, forced;   // candidates, and those of kForced
    uint64_t ones, zeros;    // bits that are 1 (0) in one of the others
};

// Keys' columns in work-items: column (base + k) THREADS + tid for k < PER, and all of a row's where PER
// times THREADS reaches them (in registers then); each(f): f(key) of all of the work-item's.
template <uint32_t THREADS, int PER>
struct CutScratch {
    static constexpr uint32_t N = PER * THREADS / 64;
    uint32_t bins[3][256];   // one in use, one read by those who are late, one made zero
    uint32_t wave[2][THREADS / 64];
    uint64_t bits[2][THREADS / 64];
    uint32_t ties[N], in[N];
};

template <uint32_t THREADS, int PER, class Each>
__device__ inline Keys look_over(Each each, CutScratch<THREADS, PER> &S)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    Keys K{};
    each([&](uint64_t k) {
        K.held += k != 0;
        K.forced += k == kForced;
        K.ones |= k == kForced ? 0 : k;
        K.zeros |= k == 0 ? 0 : ~k;
    });
    auto any = [](uint64_t x) {
        auto both = [](uint32_t a, uint32_t b) { return a | b; };
        return (uint64_t)last_lane(wave_scan((uint32_t)(x >> 32), 0u, both)) << 32 | last_lane(wave_scan((uint32_t)x, 0u, both));
    };
    K.held = wave_sum(K.held);
    K.forced = wave_sum(K.forced);
    K.ones = any(K.ones);
    K.zeros = any(K.zeros);
    if (lane == 0) {
        S.wave[0][wave] = K.held;
        S.wave[1][wave] = K.forced;
        S.bits[0][wave] = K.ones;
        S.bits[1][wave] = K.zeros;
    }
    for (uint32_t b = tid; b < 512; b += THREADS) S.bins[b / 256][b % 256] = 0;
    __syncthreads();
    K = Keys{};
#pragma unroll
    for (uint32_t w = 0; w < THREADS / 64; ++w) {
        K.held += S.wave[0][w];
        K.forced += S.wave[1][w];
        K.ones |= S.bits[0][w];
        K.zeros |= S.bits[1][w];
    }
    return K;
}

// After look_over.  One barrier a turn: every wave adds up the digits itself.
template <uint32_t THREADS, int PER, class Each>
__device__ inline Cut cut_largest(uint32_t want, const Keys &K, Each each, CutScratch<THREADS, PER> &S)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    if (want <= K.forced) return Cut{kForced, want};
    want -= K.forced;
    const uint64_t differ = K.ones & K.zeros;
    if (differ == 0) return Cut{K.ones, want};
    const int top = 63 - __clzll((long long)differ);
    uint64_t mask = ~((uint64_t(2) << top) - 1), prefix = K.ones & mask;
    uint32_t turn = 0;
    for (int shift = max(top - 7, 0);; shift = max(shift - 8, 0)) {
        uint32_t *bins = S.bins[turn];
        each([&](uint64_t k) {
            if (k && k != kForced && (k & mask) == prefix) atomicAdd(&bins[(uint32_t)(k >> shift) & 255], 1);
        });
        turn = turn == 2 ? 0 : turn + 1;
        if (shift < top - 7)   // (the second is zero from the start)
            for (uint32_t b = tid; b < 256; b += THREADS) S.bins[turn][b] = 0;
        __syncthreads();
        uint32_t c[4], sum = 0;   // lane 0 has the four largest digits
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            c[x] = bins[255 - 4 * lane - x];
            sum += c[x];
        }
        const uint32_t upto = wave_prefix(sum);
        uint32_t before = upto - sum;
        const uint64_t here = __ballot(before < want && want <= upto);   // one lane
        uint32_t digit = 0, above = 0, inside = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (before < want && want <= before + c[x]) {
                digit = 255 - 4 * lane - x;
                above = before;
                inside = c[x];
            }
            before += c[x];
        }
        const int who = __ffsll((unsigned long long)here) - 1;
        digit = (uint32_t)__builtin_amdgcn_readlane((int)digit, who);
        above = (uint32_t)__builtin_amdgcn_readlane((int)above, who);
        inside = (uint32_t)__builtin_amdgcn_readlane((int)inside, who);
        prefix |= (uint64_t)digit << shift;
        mask |= uint64_t(255) << shift;
        want -= above;
        if (inside == want) return Cut{prefix, kAll};   // whatever the lower bits are
        if (shift == 0) return Cut{prefix, want};
    }
}

// at[k]: how many of all before column (k, tid), in the columns' order, are in; returns how
// many there are.  `part` is not written again before the caller's next barrier.
template <uint32_t THREADS, int PER>
__device__ inline uint32_t rank_columns(const bool (&in)[PER], uint32_t (&at)[PER], uint32_t *part)
{
    constexpr uint32_t W = THREADS / 64, N = PER * W, V = (N + 63) / 64;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const uint64_t these = __ballot(in[k]);
        at[k] = (uint32_t)__popcll(these & ((uint64_t(1) << lane) - 1));
        if (lane == 0) part[k * W + wave] = (uint32_t)__popcll(these);
    }
    __syncthreads();
    uint32_t before[V], sum = 0;
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) {
        before[v] = sum;
        sum += lane * V + v < N ? part[lane * V + v] : 0;
    }
    const uint32_t upto = wave_prefix(sum);
#pragma unroll
    for (uint32_t v = 0; v < V; ++v) before[v] += upto - sum;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const uint32_t x = __builtin_amdgcn_readfirstlane(k * W + wave);
#pragma unroll
        for (uint32_t v = 0; v < V; ++v)
            if (x % V == v) at[k] += (uint32_t)__builtin_amdgcn_readlane((int)before[v], x / V);
    }
    return last_lane(upto);
}

// Which keys are on the upper side, of PER THREADS columns in ascending order (all
// work-items call it alike): `seen` counts the ties so far.
template <uint32_t THREADS, int PER>
__device__ inline void choose(const uint64_t (&key)[PER], const Cut &C, uint32_t &seen, bool (&in)[PER], CutScratch<THREADS, PER> &S)
{
    if (C.ties == kAll) {
#pragma unroll
        for (int k = 0; k < PER; ++k) in[k] = key[k] && key[k] >= C.key;
        return;
    }
    bool tie[PER];
    uint32_t at[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) tie[k] = key[k] && key[k] == C.key;
    const uint32_t all = rank_columns<THREADS, PER>(tie, at, S.ties);
#pragma unroll
    for (int k = 0; k < PER; ++k) in[k] = key[k] && (key[k] > C.key || (tie[k] && seen + at[k] < C.ties));
    seen += all;
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

struct RowPages {
    uint32_t used, hi;   // columns in use; positions
};
__device__ inline RowPages row_pages(const int32_t *lens, int64_t at, uint32_t cols, uint32_t page, const Div31 &by_page)
{
    const uint32_t hi = min((uint32_t)max(lens[at], 0), cols * page);
    return RowPages{hi ? by_page.div(hi - 1) + 1 : 0, hi};
}

template <int CTRL>
__device__ inline double moved(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Scores of a work-group's columns of a row and kv head into keys.  Eight lanes share a
// page: each has NP pieces of its bounds and of HEADS query heads at a time (in registers:
// from LDS their reading took longer than the sums).  A page's id is asked for two turns
// ahead, its bounds one.  Products and sums are binary64: whole numbers come of them, so
// what another order of summing would round otherwise must not show.  That is what bounds it:
// an element of a head takes five instructions (compare, select, two conversions, the product) of
// four cycles each, 64 rows of 8 kv heads by four query heads of 128 over up to 512 pages
// 26 us, where the bounds' bytes would take 10.  Every HEADS heads of a kv head are a pass over
// the ids and bounds of its own: one of four, two of eight (2 rows of 2 kv heads, 4096 pages: 10 us).
template <int TY, int NP, int HEADS, AttnEdge EDGE>
__global__ __launch_bounds__(256) void k_select_score(const SelectArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, W = E * NP;
    constexpr uint32_t kTurn = 256 / 8;
    const uint32_t x = A.by_groups.div(blockIdx.x), part = blockIdx.x - x * A.groups;
    const uint32_t r = A.by_hk.div(x), h = x - r * A.hk, sub = threadIdx.x & 7;
    const RowPages R = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    const uint32_t each = (R.used + A.groups - 1) / A.groups, c0 = min(part * each, R.used), c1 = min(c0 + each, R.used);
    if (c0 >= c1) return;
    uint64_t *keys = A.keys + (uint64_t)x * A.cols;
    const int32_t *pages = A.pages + (int64_t)r * A.pages_s[0];
    // Pieces that would reach past the end are moved back to end with it, and what two of them
    // then hold is 0 in the second.
    auto pieces = [&](const char *p, u32x4 (&x)[NP]) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t at = (i * 8 + sub) * E;
            if constexpr (EDGE == kTiny) x[i] = load_some<T, E>(p + at * sizeof(T), (int)A.d - (int)at);
            else x[i] = load16(p + (EDGE == kTail ? min(at, A.d - E) : at) * sizeof(T));
        }
    };
    auto masked = [&](u32x4 x, int i) {
        if (EDGE == kTail && (uint32_t)(i + 1) * 8 * E > A.d) x = only_own<E>(x, (i * 8 + (int)sub) * E, (int)A.d);
        return x;
    };
    struct Page {
        uint32_t c;
        bool held, scored;
        u32x4 lo[NP], hi[NP];
    };
    auto id_of = [&](uint32_t c) { return c < c1 ? pages[(int64_t)c * A.pages_s[1]] : -1; };
    auto ask = [&](Page &P, uint32_t c, int32_t id) {
        P.c = c;
        P.held = id >= 0 && (uint32_t)id < A.n;
        P.scored = P.held && c >= A.first && c + A.last < R.used && R.used > A.take;   // (few pages: all that are held)
        if (!P.scored) return;
        const char *b = (const char *)A.bounds + (int64_t)id * A.bs[0] + (int64_t)h * A.bs[1];
        pieces(b, P.lo);
        pieces(b + A.bs[2], P.hi);
    };
    for (uint32_t g0 = 0; g0 < A.group; g0 += HEADS) {
        Page P{}, next{};
        const uint32_t c = c0 + threadIdx.x / 8;
        int32_t id0 = id_of(c), id = id_of(c + kTurn);
        float q[HEADS][W];   // (past the last head, it once more: the largest score is the same)
#pragma unroll
        for (int u = 0; u < HEADS; ++u) {
            u32x4 x[NP];
            pieces((const char *)A.q + (int64_t)r * A.qs[0] + (int64_t)(h * A.group + min(g0 + u, A.group - 1)) * A.qs[1], x);
#pragma unroll
            for (int i = 0; i < NP; ++i) to_floats<TY>(masked(x[i], i), &q[u][i * E]);
        }
        ask(P, c, id0);
        // a key is written a turn later, before that turn's loads: the wait for them is for it too
        uint64_t ready = 0;
        auto write = [&](uint32_t c) {
            if (sub == 0 && c < c1) keys[c] = ready;
        };
        for (uint32_t base = c0; base < c1; base += kTurn) {
            if (base != c0) write(P.c - kTurn);
            const uint64_t old = g0 && P.c < c1 ? keys[P.c] : 0;   // its own
            ask(next, P.c + kTurn, id);
            id = id_of(P.c + 2 * kTurn);
            double sum[HEADS] = {};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float lo[E], hi[E];
                to_floats<TY>(masked(P.lo[i], i), lo);
                to_floats<TY>(masked(P.hi[i], i), hi);
#pragma unroll
                for (int u = 0; u < HEADS; ++u) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        asm volatile("" : "+v"(q[u][i * E + e]));   // not kept as binary64: twice the registers
                        const float x = q[u][i * E + e];
                        sum[u] = __builtin_fma((double)x, (double)(x < 0.0f ? lo[e] : hi[e]), sum[u]);
                    }
                }
            }
            uint64_t best = 0;
#pragma unroll
            for (int u = 0; u < HEADS; ++u) {
                sum[u] += moved<0xB1>(sum[u]);    // lane ^ 1
                sum[u] += moved<0x4E>(sum[u]);    // lane ^ 2
                sum[u] += moved<0x141>(sum[u]);   // 7 - lane of eight: the other four's, all alike
                const uint64_t k = sortable(sum[u]);
                best = k > best ? k : best;
            }
            ready = !P.held ? 0 : P.scored ? best : kForced;
            ready = old > ready ? old : ready;
            P = next;
        }
        write(P.c - kTurn);
    }
}

// The table of a row and kv head from the keys of its columns.  IN: all of them are in
// registers; otherwise they are read from memory in every turn.  512 tables of up to 512
// columns 5.3 us, 4 of 4097 columns 8.3: lengths and keys from memory, then two or three
// turns of a barrier each.
template <uint32_t THREADS, int PER, bool IN>
__global__ __launch_bounds__(THREADS) void k_select_choose(const SelectArgs A)
{
    __shared__ CutScratch<THREADS, PER> S;
    const uint32_t tid = threadIdx.x;
    const uint32_t r = A.by_hk.div(blockIdx.x), h = blockIdx.x - r * A.hk;
    const uint64_t *keys = A.keys + (uint64_t)blockIdx.x * A.cols;
    const int32_t *pages = A.pages + (int64_t)r * A.pages_s[0];
    uint64_t key[PER] = {};
    int32_t id[PER] = {};
    auto read = [&](uint32_t base) {   // (keys past a row's end are not written, and not used)
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t c = min(base + k * THREADS + tid, A.cols - 1);
            key[k] = keys[c];
            id[k] = pages[(int64_t)c * A.pages_s[1]];
        }
    };
    if (IN && A.cols) read(0);
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    auto end = [&](uint32_t base) {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (base + k * THREADS + tid >= P.used) key[k] = 0;
    };
    if (IN) end(0);
    auto each = [&](auto f) {
        if constexpr (IN) {
#pragma unroll
            for (int k = 0; k < PER; ++k) f(key[k]);
        } else {
            for (uint32_t c = tid; c < P.used; c += THREADS) f(keys[c]);
        }
    };
    const Keys K = look_over<THREADS, PER>(each, S);
    Cut C{0, kAll};   // all of them
    if (K.held > A.take) C = cut_largest<THREADS, PER>(A.take, K, each, S);
    int32_t *out = A.pages_out + (int64_t)r * A.pages_out_s[0] + (int64_t)h * A.pages_out_s[1];
    const uint32_t all = min(K.held, A.take);
    if (all == 0 && tid == 0) A.lens_out[(int64_t)r * A.lens_out_s[0] + (int64_t)h * A.lens_out_s[1]] = 0;
    uint32_t count = 0, seen = 0;
    for (uint32_t base = 0; base < P.used && count < all; base += PER * THREADS) {
        if (!IN) {
            __syncthreads();   // the ranks of the turn before are done with
            read(base);
            end(base);
        }
        bool in[PER];
        uint32_t at[PER];
        choose<THREADS, PER>(key, C, seen, in, S);
        const uint32_t n = rank_columns<THREADS, PER>(in, at, S.in);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (!in[k]) continue;
            const uint32_t c = base + k * THREADS + tid, to = count + at[k];
            out[(int64_t)to * A.pages_out_s[2]] = id[k];
            if (to + 1 == all)
                A.lens_out[(int64_t)r * A.lens_out_s[0] + (int64_t)h * A.lens_out_s[1]] =
                    (int32_t)(to * A.page + (c + 1 == P.used ? P.hi - c * A.page : A.page));
        }
        count += n;
    }
    for (uint32_t i = all + tid; i < A.take; i += THREADS) out[(int64_t)i * A.pages_out_s[2]] = -1;
}

template <int TY, int NP, AttnEdge EDGE>
int launch_score(const SelectArgs &A, void *stream)
{
    constexpr int HEADS = AttnType<TY>::E * NP <= 16 ? 4 : 2;
    const void *fn = A.group == 1 ? reinterpret_cast<const void *>(&k_select_score<TY, NP, 1, EDGE>)
                                  : reinterpret_cast<const void *>(&k_select_score<TY, NP, HEADS, EDGE>);
    return launch_kernel(fn, dim3(A.b * A.hk * A.groups), dim3(256), 0, stream, A);
}

template <int TY, int NP>
int launch_score_edge(const SelectArgs &A, void *stream)
{
    return A.d == (uint32_t)(NP * 8 * AttnType<TY>::E) ? launch_score<TY, NP, kExact>(A, stream) : launch_score<TY, NP, kTail>(A, stream);
}

// The instance: the smallest that holds d.
template <int TY>
int launch_select_type(const SelectArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;
    if (A.d < (uint32_t)E) return launch_score<TY, 1, kTiny>(A, stream);
    if (A.d <= 64) return launch_score_edge<TY, U>(A, stream);
    if constexpr (TY == S_F32) {
        if (A.d <= 96) return launch_score_edge<TY, 3>(A, stream);
    }
    return A.d <= 128   ? launch_score_edge<TY, 2 * U>(A, stream)
           : A.d <= 192 ? launch_score_edge<TY, 3 * U>(A, stream)
                        : launch_score_edge<TY, 4 * U>(A, stream);
}

// ---------------------------------------------------------------------------
// Eviction.  A work-group to a row, whose keys are in registers (IN) or made anew from the
// masses in each turn.  256 rows of 1024 columns: 6.2 us, and 2.0 for the copy of the counts
// before it, which other rows' subtractions may not precede.

__global__ __launch_bounds__(256) void k_evict_refs(const EvictArgs A)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < A.n) A.refs_out[(int64_t)i * A.refs_out_s] = A.refs[(int64_t)i * A.refs_s];
}

template <uint32_t THREADS, int PER, bool IN>
__global__ __launch_bounds__(THREADS) void k_evict(const EvictArgs A)
{
    __shared__ CutScratch<THREADS, PER> S;
    __shared__ uint32_t s_held[THREADS / 64];
    const uint32_t r = blockIdx.x, tid = threadIdx.x;
    const int32_t *pages = A.pages + (int64_t)r * A.pages_s[0];
    const float *mass = A.mass + (int64_t)r * A.mass_s[0];
    int32_t *out = A.pages_out + (int64_t)r * A.pages_out_s[0];
    uint64_t key[PER];
    int32_t id[PER] = {};
    float x[PER] = {};
    auto read = [&](uint32_t base) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t c = min(base + k * THREADS + tid, A.cols - 1);
            id[k] = pages[(int64_t)c * A.pages_s[1]];
            x[k] = mass[(int64_t)c * A.mass_s[1]];
        }
    };
    if (IN && A.cols) read(0);
    const uint32_t budget = (uint32_t)max(A.budget[(int64_t)r * A.budget_s], 0);
    const RowPages P = row_pages(A.lens, (int64_t)r * A.lens_s, A.cols, A.page, A.by_page);
    // the less mass, the larger; 0: not to be taken out
    auto make = [&](uint32_t c, int32_t id, float x) {
        if (c >= P.used || id < 0 || (uint32_t)id >= A.n || c < A.first || c + A.last >= P.used) return uint64_t(0);
        uint32_t b = __builtin_bit_cast(uint32_t, x == 0.0f ? 0.0f : x);
        b = x != x ? ~0u : b >> 31 ? ~b : b | 1u << 31;
        return uint64_t(1) << 32 | (uint32_t)~b;
    };
    auto end = [&](uint32_t base) {
#pragma unroll
        for (int k = 0; k < PER; ++k) key[k] = make(base + k * THREADS + tid, id[k], x[k]);
    };
    uint32_t held = 0;
    if (IN) {
        end(0);
#pragma unroll
        for (int k = 0; k < PER; ++k) held += k * THREADS + tid < P.used && id[k] >= 0 && (uint32_t)id[k] < A.n;
    } else {
        for (uint32_t c = tid; c < P.used; c += THREADS) {
            const int32_t id = pages[(int64_t)c * A.pages_s[1]];
            held += id >= 0 && (uint32_t)id < A.n;
        }
    }
    held = wave_sum(held);
    if ((tid & 63) == 0) s_held[tid / 64] = held;
    auto each = [&](auto f) {
        if constexpr (IN) {
#pragma unroll
            for (int k = 0; k < PER; ++k) f(key[k]);
        } else {
            for (uint32_t c = tid; c < P.used; c += THREADS) f(make(c, pages[(int64_t)c * A.pages_s[1]], mass[(int64_t)c * A.mass_s[1]]));
        }
    };
    const Keys K = look_over<THREADS, PER>(each, S);
    held = 0;
#pragma unroll
    for (uint32_t w = 0; w < THREADS / 64; ++w) held += s_held[w];
    const uint32_t over = held > budget ? min(held - budget, K.held) : 0;
    Cut C{0, kAll};
    if (over && over < K.held) C = cut_largest<THREADS, PER>(over, K, each, S);
    uint32_t seen = 0;
    for (uint32_t base = 0; base < A.cols; base += PER * THREADS) {
        if (!IN) {
            __syncthreads();   // the ranks of the turn before are done with
            read(base);
            end(base);
        }
        bool gone[PER] = {};
        if (over) choose<THREADS, PER>(key, C, seen, gone, S);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t c = base + k * THREADS + tid;
            if (c >= A.cols) continue;
            if (gone[k]) atomicSub(&A.refs_out[(int64_t)id[k] * A.refs_out_s], 1);
            out[(int64_t)c * A.pages_out_s[1]] = gone[k] || id[k] < 0 || (uint32_t)id[k] >= A.n ? -1 : id[k];
        }
    }
    if (tid == 0) A.count[(int64_t)r * A.count_s] = (int32_t)over;
}

// A work-group to a row of so many columns, whose keys fit the registers of 256 or 1024 work-items or none's.
template <class Args>
int launch_by_columns(uint32_t cols, uint32_t rows, void (*few)(Args), void (*many)(Args), void (*any)(Args), void *stream, const Args &A)
{
    auto *fn = cols <= 1024 ? few : cols <= 8192 ? many : any;
    return launch_kernel(reinterpret_cast<const void *>(fn), dim3(rows), dim3(cols <= 1024 ? 256 : 1024), 0, stream, A);
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
    const int rc = type == S_F16    ? launch_select_type<S_F16>(A, stream)
                   : type == S_BF16 ? launch_select_type<S_BF16>(A, stream)
                                    : launch_select_type<S_F32>(A, stream);
    if (rc) return rc;
    return launch_by_columns(A.cols, A.b * A.hk, &k_select_choose<256, 4, true>, &k_select_choose<1024, 8, true>,
                             &k_select_choose<1024, 4, false>, stream, A);
}

int launch_evict(const EvictArgs &A, void *stream)
{
    if (A.copy && A.n)
        if (const int rc = launch_kernel(reinterpret_cast<const void *>(&k_evict_refs), dim3((A.n + 255) / 256), dim3(256), 0, stream, A))
            return rc;
    if (A.rows == 0) return 0;
    return launch_by_columns(A.cols, A.rows, &k_evict<256, 4, true>, &k_evict<1024, 8, true>, &k_evict<1024, 4, false>, stream, A);
}

}  // namespace ecmd
