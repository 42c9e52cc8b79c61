// kernels_rope.hip -- rotary positions, alone and with the write into a paged
// key-value cache.
//
// Pair i of a head at position p turns by w = p * freq[i]:
//     (u, v) -> (u c - v s, v c + u s),   c = mscale cos w, s = mscale sin w
// (the inverse turns by -w).  Both kernels read and write each element once, so
// HBM bounds them; the angles are shared by all heads of a token.  A work-group
// takes a few tokens, computes their cosines and sines once into LDS, then
// streams the heads past them in 16-byte vectors, four to a work-item at once.
//
// Measured on one MI355X: 4 x 4096 tokens of 40 heads of 128, bfloat16, 336 MB: 60
// us, 5.6 TB/s (one vector at a time 71, four 66, past the caches 60); twice that, in
// pairs of neighbours, 107 us, 6.3 TB/s.  The append of 16 ragged prompts, 36 + 4
// heads, binary16, half of each head turned in pairs of neighbours, 212 MB: 45 us, 4.7
// TB/s (65 with one vector at a time; 52 with four), no faster with the pages in
// order: a token's 624 vectors leave a work-group of one token 384 of its 1024 loads
// unused.  Whole heads turned by halves, two vectors an item, take 46 us for 235 MB, 5.2
// TB/s.  One token of each of 64 sequences: 4.3 us, of which the angles' chain of
// binary64 operations overlaps the loads.  Heads of odd width, whose vectors are off
// 16 bytes and overlap at the ends: 10000 tokens of 20 heads of 101, 100 turned,
// bfloat16, 81 MB: by halves 24 us, in neighbours 20; heads of 104 20 and 17.
#include <hip/hip_runtime.h>

#include "../ecmd_launch.h"
#include "ecmd_serving.h"

namespace ecmd {

namespace {

constexpr uint32_t kBlock = 256;

template <int TY>
struct Elem;
template <>
struct Elem<S_F16> {
    typedef _Float16 T;
    static constexpr int E = 8;
};
template <>
struct Elem<S_BF16> {
    typedef __bf16 T;
    static constexpr int E = 8;
};
template <>
struct Elem<S_F32> {
    typedef float T;
    static constexpr int E = 4;
};

// cos and sin of w, both times mscale, rounded to binary32.  The position of a
// token may be in the millions, so w and its reduction are binary64: k = the
// nearest multiple of pi/2, and pi/2 as the sum of two binary64 numbers keeps
// w - k pi/2 good to 2^-80 of k.  On [-pi/4, pi/4] the Taylor series to x^13
// and x^14 are off by less than 1e-13, far below the final rounding.
__device__ inline void turn(double w, double mscale, float &c, float &s)
{
    const double k = __builtin_rint(w * 0.63661977236758134308);
    double x = __builtin_fma(-k, 1.57079632679489661923, w);
    x = __builtin_fma(-k, 6.12323399573676603587e-17, x);
    const double y = x * x;
    double sn = 1.0 / 6227020800.0;
    sn = __builtin_fma(sn, y, -1.0 / 39916800.0);
    sn = __builtin_fma(sn, y, 1.0 / 362880.0);
    sn = __builtin_fma(sn, y, -1.0 / 5040.0);
    sn = __builtin_fma(sn, y, 1.0 / 120.0);
    sn = __builtin_fma(sn, y, -1.0 / 6.0);
    sn = __builtin_fma(sn * y, x, x);
    double cs = -1.0 / 87178291200.0;
    cs = __builtin_fma(cs, y, 1.0 / 479001600.0);
    cs = __builtin_fma(cs, y, -1.0 / 3628800.0);
    cs = __builtin_fma(cs, y, 1.0 / 40320.0);
    cs = __builtin_fma(cs, y, -1.0 / 720.0);
    cs = __builtin_fma(cs, y, 1.0 / 24.0);
    cs = __builtin_fma(cs, y, -0.5);
    cs = __builtin_fma(cs, y, 1.0);
    const int quadrant = (int)__builtin_fma(-4.0, __builtin_floor(k * 0.25), k);
    const double a = quadrant & 1 ? sn : cs, b = quadrant & 1 ? cs : sn;
    c = (float)((quadrant == 1 || quadrant == 2 ? -a : a) * mscale);
    s = (float)((quadrant >= 2 ? -b : b) * mscale);
}

// E elements from p, of which the first n exist (the others are left alone).
// Rows may start at any element: the 16-byte accesses need no alignment.
// STREAM: past the caches, where a launch moves more than they hold.
template <class T, int E>
using Vec = T __attribute__((ext_vector_type(E)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 Any16 __attribute__((aligned(2)));
template <class T, int E, bool STREAM>
__device__ inline Vec<T, E> load_vec(const T *p, int n)
{
    if (n >= E) {
        if constexpr (STREAM) return __builtin_bit_cast(Vec<T, E>, __builtin_nontemporal_load((const Any16 *)p));
        else return __builtin_bit_cast(Vec<T, E>, *(const Any16 *)p);
    }
    Vec<T, E> v = (T)0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < n) v[i] = p[i];
    return v;
}
template <class T, int E, bool STREAM>
__device__ inline void store_vec(T *p, Vec<T, E> v, int n)
{
    if (n >= E) {
        if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (Any16 *)p);
        else *(Any16 *)p = __builtin_bit_cast(u32x4, v);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) p[i] = v[i];
    }
}

// Elements from `skip` on.
template <class T, int E>
__device__ inline void store_own(T *p, Vec<T, E> v, uint32_t skip)
{
#pragma unroll
    for (int i = 0; i < E; ++i)
        if ((uint32_t)i >= skip) p[i] = v[i];
}

// One item: a 16-byte vector of pairs of one head (half layout: E pairs, from
// both halves; interleaved: E / 2 pairs), or of the copied tail.  Items of a
// head: rot_items(pairs) of pairs, then the tail's.
template <int LAYOUT, int E>
__host__ __device__ constexpr uint32_t rot_items(uint32_t pairs)
{
    return LAYOUT == 0 ? (pairs + E - 1) / E : (2 * pairs + E - 1) / E;
}

// How vectors that would reach past their part of a head (the pairs of a half, the
// pairs, the tail) are read and written.
enum RopeEdge {
    kWhole,    // there are none: loads need no branch (those of a half layout's tail read one vector twice)
    kMoved,    // moved back to end with the part: what an earlier item has is read and turned twice, and
               // written twice, the same, unless it could be read in between (in place) or is no tail
    kGuarded,  // element by element: parts shorter than a vector
};

template <int TY, int LAYOUT, RopeEdge EDGE, bool STREAM>
struct Item {
    typedef typename Elem<TY>::T T;
    static constexpr int E = Elem<TY>::E;
    Vec<T, E> a, b;

    // kMoved: where an item's vector starts (from the head, or from the half), and how
    // many of its first elements are an earlier item's.
    __device__ static uint32_t start(uint32_t item, uint32_t rot, uint32_t pairs, uint32_t width, uint32_t &skip)
    {
        const uint32_t from = item < rot ? item * E : 2 * pairs + (item - rot) * E;
        const uint32_t at = min(from, (item >= rot ? width : LAYOUT == 0 ? pairs : 2 * pairs) - E);
        skip = from - at;
        return at;
    }

    __device__ void load(const T *head, uint32_t item, uint32_t pairs, uint32_t width)
    {
        const uint32_t rot = rot_items<LAYOUT, E>(pairs);
        if constexpr (EDGE != kGuarded) {
            uint32_t at, skip;
            if constexpr (EDGE == kMoved) at = start(item, rot, pairs, width, skip);
            else at = LAYOUT == 0 && item >= rot ? 2 * pairs + (item - rot) * E : item * E;
            a = load_vec<T, E, STREAM>(head + at, E);
            if constexpr (LAYOUT == 0) b = load_vec<T, E, STREAM>(head + (item < rot ? pairs + at : at), E);
            return;
        }
        if (item >= rot) {
            const int at = 2 * pairs + (item - rot) * E;
            a = load_vec<T, E, STREAM>(head + at, (int)width - at);
        } else if (LAYOUT == 0) {
            const int at = item * E;
            a = load_vec<T, E, STREAM>(head + at, (int)pairs - at);
            b = load_vec<T, E, STREAM>(head + pairs + at, (int)pairs - at);
        } else {
            const int at = item * E;
            a = load_vec<T, E, STREAM>(head + at, (int)(2 * pairs) - at);
        }
    }

    // cs and sn: the token's rows in LDS, 16-byte aligned, readable up to a
    // multiple of 8 entries.
    __device__ void finish(T *head, uint32_t item, uint32_t pairs, uint32_t width, const float *cs, const float *sn,
                           bool in_place)
    {
        const uint32_t rot = rot_items<LAYOUT, E>(pairs);
        uint32_t skip = 0, at = item < rot ? item * E : 2 * pairs + (item - rot) * E;
        if constexpr (EDGE == kMoved) at = start(item, rot, pairs, width, skip);
        // elements there are (kGuarded)
        const int n = EDGE != kGuarded ? E : (int)((item >= rot ? width : LAYOUT == 0 ? pairs : 2 * pairs) - at);
        const bool part = EDGE == kMoved && skip && (in_place || at < 2 * pairs);
        if (item >= rot) {
            if (part) store_own<T, E>(head + at, a, skip);
            else store_vec<T, E, STREAM>(head + at, a, n);
            return;
        }
        const bool own = EDGE == kMoved && skip && in_place;
        if (LAYOUT == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float u = (float)a[i], v = (float)b[i], c = cs[at + i], s = sn[at + i];
                a[i] = (T)(u * c - v * s);
                b[i] = (T)(v * c + u * s);
            }
            if (own) {
                store_own<T, E>(head + at, a, skip);
                store_own<T, E>(head + pairs + at, b, skip);
            } else {
                store_vec<T, E, STREAM>(head + at, a, n);
                store_vec<T, E, STREAM>(head + pairs + at, b, n);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float u = (float)a[i], v = (float)a[i + 1];
                const float c = cs[(at + i) / 2], s = sn[(at + i) / 2];
                a[i] = (T)(u * c - v * s);
                a[i + 1] = (T)(v * c + u * s);
            }
            if (own) store_own<T, E>(head + at, a, skip);
            else store_vec<T, E, STREAM>(head + at, a, n);
        }
    }
};

// LDS row length of a token's cosines (and sines): a multiple of 8 entries.
__host__ __device__ inline uint32_t lds_row(uint32_t pairs) { return (pairs + 7) / 8 * 8; }

extern __shared__ __attribute__((aligned(16))) float s_turn[];

// A work-group: A.tb tokens, all their heads.
template <int TY, int LAYOUT, RopeEdge EDGE, bool STREAM>
__global__ __launch_bounds__(kBlock) void k_rope(const RopeArgs A)
{
    typedef typename Elem<TY>::T T;
    const uint32_t first = blockIdx.x * A.tb;
    const uint32_t count = min(A.tb, A.tokens - first);
    const uint32_t row = lds_row(A.pairs);
    float *cs = s_turn, *sn = s_turn + A.tb * row;
    const uint32_t total = count * A.items;
    const uint32_t head_items = A.by_head_items.d;

    struct Place {
        uint32_t tok, head, item;
    };
    auto split = [&](uint32_t i) {
        const uint32_t tok = A.by_token_items.div(i), r = i - tok * A.items, head = A.by_head_items.div(r);
        return Place{tok, head, r - head * head_items};
    };
    auto offset = [&](const Place &p, const int64_t *s) {
        const uint32_t g = first + p.tok, bb = A.by_t.div(g);
        return (int64_t)bb * s[0] + (int64_t)(g - bb * A.by_t.d) * s[1] + (int64_t)p.head * s[2];
    };

    // Several items' loads are on their way before the first is stored, the first
    // ones' while the angles are computed.
    constexpr int U = 4;
    Item<TY, LAYOUT, EDGE, STREAM> it[U];
    auto load = [&](uint32_t from) {   // from: the work-group's
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = from + u * kBlock + threadIdx.x;
            if (EDGE != kGuarded ? from + u * kBlock < total : i < total) {   // the last item again, not a branch
                const Place p = split(EDGE != kGuarded ? min(i, total - 1) : i);
                it[u].load((const T *)A.x + offset(p, A.xs), p.item, A.pairs, A.width);
            }
        }
    };
    load(0);
    for (uint32_t j = threadIdx.x; j < count * A.pairs; j += kBlock) {
        const uint32_t t = j / A.pairs, p = j - t * A.pairs;
        const uint32_t g = first + t, bb = A.by_t.div(g);
        const int32_t pos = A.pos[(int64_t)bb * A.ps[0] + (int64_t)(g - bb * A.by_t.d) * A.ps[1]];
        float c, s;
        turn((double)pos * A.freq[p * A.fs], A.mscale, c, s);
        cs[t * row + p] = c;
        sn[t * row + p] = A.inverse ? -s : s;
    }
    __syncthreads();
    for (uint32_t from = 0; from < total;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = from + u * kBlock + threadIdx.x;
            if (i < total) {
                const Place p = split(i);
                it[u].finish((T *)A.out + offset(p, A.os), p.item, A.pairs, A.width, cs + p.tok * row, sn + p.tok * row,
                             A.x == A.out);
            }
        }
        from += U * kBlock;
        if (from < total) load(from);
    }
}

// A work-group: A.tb tokens, or (A.parts > 1) a part of one token's items.  The
// items are q's, k's, then v's (copied: a head without pairs), each kind's number
// rounded up to whole waves: a wave's pointers and strides are then scalars.
template <int TY, int LAYOUT, RopeEdge EDGE, bool STREAM>
__global__ __launch_bounds__(kBlock) void k_append(const AppendArgs A)
{
    typedef typename Elem<TY>::T T;
    const uint32_t group = A.by_parts.div(blockIdx.x), part = blockIdx.x - group * A.parts;
    const uint32_t first = group * A.tb;
    const uint32_t count = min(A.tb, A.tokens - first);
    const uint32_t row = lds_row(A.pairs);
    float *cs = s_turn, *sn = s_turn + A.tb * row;
    int64_t *slot = (int64_t *)(sn + A.tb * row);   // [tb][2]: element offsets into the caches, -1: padding
    auto waves = [](uint32_t n) { return (n + 63) / 64 * 64; };
    const uint32_t k_from = waves(count * A.by_q.d), v_from = k_from + waves(count * A.by_k.d);
    const uint32_t total = v_from + waves(count * A.by_v.d), step = kBlock * A.parts;

    struct Place {
        uint32_t kind, tok, head, item;   // kind: 0 q, 1 k, 2 v; the same for the wave
        bool real;
    };
    auto split = [&](uint32_t i) {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(i & ~63u);
        Place p;
        p.kind = wave >= v_from ? 2 : wave >= k_from ? 1 : 0;
        const Div31 by_token = p.kind == 2 ? A.by_v : p.kind ? A.by_k : A.by_q;
        const Div31 by_head = p.kind == 2 ? A.by_v_head : A.by_qk_head;
        uint32_t r = i - (p.kind == 2 ? v_from : p.kind ? k_from : 0);
        p.real = r < count * by_token.d;
        if (!p.real) r = 0;
        p.tok = by_token.div(r);
        r -= p.tok * by_token.d;
        p.head = by_head.div(r);
        p.item = r - p.head * by_head.d;
        return p;
    };
    constexpr int U = 4;   // as above
    Item<TY, LAYOUT, EDGE, STREAM> it[U];
    auto load = [&](uint32_t i0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * step < total) {
                const Place p = split(i0 + u * step);
                const T *from = (const T *)(p.kind == 2 ? A.v : p.kind ? A.k : A.q);
                const int64_t ts = p.kind == 2 ? A.vs[0] : p.kind ? A.ks[0] : A.qs[0];
                const int64_t hs = p.kind == 2 ? A.vs[1] : p.kind ? A.ks[1] : A.qs[1];
                it[u].load(from + (int64_t)(first + p.tok) * ts + p.head * hs, p.item, p.kind == 2 ? 0 : A.pairs,
                           p.kind == 2 ? A.dv : A.d);
            }
    };
    uint32_t i = part * kBlock + threadIdx.x;
    load(i);
    for (uint32_t t = threadIdx.x; t < count; t += kBlock) {
        const int32_t r = A.row[(first + t) * A.row_s], pos = A.pos[(first + t) * A.pos_s];
        int64_t ko = -1, vo = -1;
        if (r >= 0 && (uint32_t)r < A.rows && pos >= 0) {
            const uint32_t col = A.by_page.div((uint32_t)pos), in = (uint32_t)pos - col * A.page;
            if (col < A.cols) {
                const int32_t id = A.pages[r * A.pages_s[0] + col * A.pages_s[1]];
                if (id >= 0 && (uint32_t)id < A.n) {
                    ko = id * A.kcs[0] + in * A.kcs[1];
                    vo = id * A.vcs[0] + in * A.vcs[1];
                }
            }
        }
        slot[2 * t] = ko;
        slot[2 * t + 1] = vo;
    }
    for (uint32_t j = threadIdx.x; j < count * A.pairs; j += kBlock) {
        const uint32_t t = j / A.pairs, p = j - t * A.pairs;
        float c, s;
        turn((double)A.pos[(first + t) * A.pos_s] * A.freq[p * A.fs], A.mscale, c, s);
        cs[t * row + p] = c;
        sn[t * row + p] = s;
    }
    __syncthreads();
    while (i < total) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * step < total) {
                const Place p = split(i + u * step);
                T *to = (T *)(p.kind == 2 ? A.v_cache : p.kind ? A.k_cache : A.q_out);
                const int64_t hs = p.kind == 2 ? A.vcs[2] : p.kind ? A.kcs[2] : A.qos[1];
                const int64_t at = p.kind ? slot[2 * p.tok + p.kind - 1] : (int64_t)(first + p.tok) * A.qos[0];
                if (p.real && at >= 0)
                    it[u].finish(to + at + p.head * hs, p.item, p.kind == 2 ? 0 : A.pairs, p.kind == 2 ? A.dv : A.d,
                                 cs + p.tok * row, sn + p.tok * row, p.kind == 0 && A.q == A.q_out);
            }
        i += U * step;
        load(i);
    }
}

}  // namespace

template <int TY, int LAYOUT, RopeEdge EDGE, bool STREAM>
static int launch_one(const RopeArgs &A, uint32_t grid, uint32_t lds, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_rope<TY, LAYOUT, EDGE, STREAM>), dim3(grid), dim3(kBlock),
                         lds, stream, A);
}
template <int TY, int LAYOUT, RopeEdge EDGE, bool STREAM>
static int launch_one(const AppendArgs &A, uint32_t grid, uint32_t lds, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_append<TY, LAYOUT, EDGE, STREAM>), dim3(grid), dim3(kBlock),
                         lds, stream, A);
}
template <int TY, int LAYOUT, class Args>
static int launch_layout(int edge, bool past, const Args &A, uint32_t grid, uint32_t lds, void *stream)
{
    switch (edge) {
    case kWhole:
        return past ? launch_one<TY, LAYOUT, kWhole, true>(A, grid, lds, stream)
                    : launch_one<TY, LAYOUT, kWhole, false>(A, grid, lds, stream);
    case kMoved:
        return past ? launch_one<TY, LAYOUT, kMoved, true>(A, grid, lds, stream)
                    : launch_one<TY, LAYOUT, kMoved, false>(A, grid, lds, stream);
    default: return launch_one<TY, LAYOUT, kGuarded, false>(A, grid, lds, stream);
    }
}
template <class Args>
static int launch_any(int type, int layout, int edge, bool past, const Args &A, uint32_t grid, uint32_t lds,
                      void *stream)
{
    switch (2 * type + layout) {
    case 2 * S_F16: return launch_layout<S_F16, 0>(edge, past, A, grid, lds, stream);
    case 2 * S_F16 + 1: return launch_layout<S_F16, 1>(edge, past, A, grid, lds, stream);
    case 2 * S_BF16: return launch_layout<S_BF16, 0>(edge, past, A, grid, lds, stream);
    case 2 * S_BF16 + 1: return launch_layout<S_BF16, 1>(edge, past, A, grid, lds, stream);
    case 2 * S_F32: return launch_layout<S_F32, 0>(edge, past, A, grid, lds, stream);
    case 2 * S_F32 + 1: return launch_layout<S_F32, 1>(edge, past, A, grid, lds, stream);
    }
    return (int)hipErrorInvalidValue;
}

int launch_rope(int type, int layout, int edge, bool past, const RopeArgs &A, uint32_t grid, uint32_t lds, void *stream)
{
    return launch_any(type, layout, edge, past, A, grid, lds, stream);
}

int launch_append(int type, int layout, int edge, bool past, const AppendArgs &A, uint32_t grid, uint32_t lds,
                  void *stream)
{
    return launch_any(type, layout, edge, past, A, grid, lds, stream);
}

}  // namespace ecmd
