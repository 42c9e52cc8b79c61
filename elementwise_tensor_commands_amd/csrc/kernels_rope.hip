// kernels_rope.hip -- rotary positions, alone and with the write into a paged
// key-value cache.
//
// Pair i of a head at position p turns by w = p * freq[i]:
//     (u, v) -> (u c - v s, v c + u s),   c = mscale cos w, s = mscale sin w
// (the inverse turns by -w).  Both kernels read and write each element once, so
// HBM bounds them; the angles are shared by all heads of a token.  A work-group
// takes a few tokens, computes their cosines and sines once into LDS, then
// streams the heads past them in 16-byte vectors.
#include <hip/hip_runtime.h>

#include "ecmd_launch.h"
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
template <class T, int E>
using Vec = T __attribute__((ext_vector_type(E)));
template <class T, int E>
__device__ inline Vec<T, E> load_vec(const T *p, int n)
{
    Vec<T, E> v = (T)0.0f;
    if (n >= E) {
        __builtin_memcpy(&v, p, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) v[i] = p[i];
    }
    return v;
}
template <class T, int E>
__device__ inline void store_vec(T *p, Vec<T, E> v, int n)
{
    if (n >= E) {
        __builtin_memcpy(p, &v, sizeof v);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < n) p[i] = v[i];
    }
}

// One item: a 16-byte vector of pairs of one head (half layout: E pairs, from
// both halves; interleaved: E / 2 pairs), or of the copied tail.  Items of a
// head: rot_items(pairs) of pairs, then the tail's.
template <int LAYOUT, int E>
__host__ __device__ constexpr uint32_t rot_items(uint32_t pairs)
{
    return LAYOUT == 0 ? (pairs + E - 1) / E : (2 * pairs + E - 1) / E;
}

template <int TY, int LAYOUT>
struct Item {
    typedef typename Elem<TY>::T T;
    static constexpr int E = Elem<TY>::E;
    Vec<T, E> a, b;

    __device__ void load(const T *head, uint32_t item, uint32_t pairs, uint32_t width)
    {
        const uint32_t rot = rot_items<LAYOUT, E>(pairs);
        if (item >= rot) {
            const int at = 2 * pairs + (item - rot) * E;
            a = load_vec<T, E>(head + at, (int)width - at);
        } else if (LAYOUT == 0) {
            const int at = item * E;
            a = load_vec<T, E>(head + at, (int)pairs - at);
            b = load_vec<T, E>(head + pairs + at, (int)pairs - at);
        } else {
            const int at = item * E;
            a = load_vec<T, E>(head + at, (int)(2 * pairs) - at);
        }
    }

    // cs and sn: the token's rows in LDS, 16-byte aligned, readable up to a
    // multiple of 8 entries.
    __device__ void finish(T *head, uint32_t item, uint32_t pairs, uint32_t width, const float *cs, const float *sn)
    {
        const uint32_t rot = rot_items<LAYOUT, E>(pairs);
        if (item >= rot) {
            const int at = 2 * pairs + (item - rot) * E;
            store_vec<T, E>(head + at, a, (int)width - at);
            return;
        }
        const int at = item * E;
        if (LAYOUT == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float u = (float)a[i], v = (float)b[i], c = cs[at + i], s = sn[at + i];
                a[i] = (T)(u * c - v * s);
                b[i] = (T)(v * c + u * s);
            }
            store_vec<T, E>(head + at, a, (int)pairs - at);
            store_vec<T, E>(head + pairs + at, b, (int)pairs - at);
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float u = (float)a[i], v = (float)a[i + 1];
                const float c = cs[(at + i) / 2], s = sn[(at + i) / 2];
                a[i] = (T)(u * c - v * s);
                a[i + 1] = (T)(v * c + u * s);
            }
            store_vec<T, E>(head + at, a, (int)(2 * pairs) - at);
        }
    }
};

// LDS row length of a token's cosines (and sines): a multiple of 8 entries.
__host__ __device__ inline uint32_t lds_row(uint32_t pairs) { return (pairs + 7) / 8 * 8; }

extern __shared__ __attribute__((aligned(16))) float s_turn[];

// A work-group: A.tb tokens, all their heads.
template <int TY, int LAYOUT>
__global__ __launch_bounds__(kBlock) void k_rope(const RopeArgs A)
{
    typedef typename Elem<TY>::T T;
    const uint32_t first = blockIdx.x * A.tb;
    const uint32_t count = min(A.tb, A.tokens - first);
    const uint32_t row = lds_row(A.pairs);
    float *cs = s_turn, *sn = s_turn + A.tb * row;
    const uint32_t total = count * A.items;
    const uint32_t head_items = A.by_head_items.d;

    uint32_t tok, head, item;
    auto split = [&](uint32_t i) {
        tok = A.by_token_items.div(i);
        const uint32_t r = i - tok * A.items;
        head = A.by_head_items.div(r);
        item = r - head * head_items;
    };
    auto offset = [&](const int64_t *s) {
        const uint32_t g = first + tok, bb = A.by_t.div(g);
        return (int64_t)bb * s[0] + (int64_t)(g - bb * A.by_t.d) * s[1] + (int64_t)head * s[2];
    };

    // The first item's loads are on their way while the angles are computed.
    Item<TY, LAYOUT> it;
    uint32_t i = threadIdx.x;
    if (i < total) {
        split(i);
        it.load((const T *)A.x + offset(A.xs), item, A.pairs, A.width);
    }
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
    while (i < total) {
        it.finish((T *)A.out + offset(A.os), item, A.pairs, A.width, cs + tok * row, sn + tok * row);
        i += kBlock;
        if (i < total) {
            split(i);
            it.load((const T *)A.x + offset(A.xs), item, A.pairs, A.width);
        }
    }
}

// A work-group: A.tb tokens, or (A.parts > 1) a part of one token's items.
// Items of a token: q's, k's, then v's (copied).
template <int TY, int LAYOUT>
__global__ __launch_bounds__(kBlock) void k_append(const AppendArgs A)
{
    typedef typename Elem<TY>::T T;
    constexpr int E = Elem<TY>::E;
    const uint32_t group = A.by_parts.div(blockIdx.x), part = blockIdx.x - group * A.parts;
    const uint32_t first = group * A.tb;
    const uint32_t count = min(A.tb, A.tokens - first);
    const uint32_t row = lds_row(A.pairs);
    float *cs = s_turn, *sn = s_turn + A.tb * row;
    int64_t *slot = (int64_t *)(sn + A.tb * row);   // [tb][2]: element offsets into the caches, -1: padding
    const uint32_t total = count * A.items, step = kBlock * A.parts;

    uint32_t tok, head, item;
    int kind;   // 0 q, 1 k, 2 v
    auto split = [&](uint32_t i) {
        tok = A.by_token_items.div(i);
        uint32_t r = i - tok * A.items;
        if (r >= A.qk_items) {
            kind = 2;
            r -= A.qk_items;
            head = A.by_v.div(r);
            item = r - head * A.by_v.d;
        } else {
            kind = r >= A.q_items;
            if (kind) r -= A.q_items;
            head = A.by_qk.div(r);
            item = r - head * A.by_qk.d;
        }
    };
    Item<TY, LAYOUT> it;
    auto load = [&]() {
        const int64_t t = first + tok;
        if (kind == 2)
            it.a = load_vec<T, E>((const T *)A.v + t * A.vs[0] + head * A.vs[1] + item * E, (int)A.dv - (int)item * E);
        else
            it.load(kind ? (const T *)A.k + t * A.ks[0] + head * A.ks[1] : (const T *)A.q + t * A.qs[0] + head * A.qs[1],
                    item, A.pairs, A.d);
    };

    uint32_t i = part * kBlock + threadIdx.x;
    if (i < total) {
        split(i);
        load();
    }
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
        if (kind == 2) {
            const int64_t at = slot[2 * tok + 1];
            if (at >= 0)
                store_vec<T, E>((T *)A.v_cache + at + head * A.vcs[2] + item * E, it.a, (int)A.dv - (int)item * E);
        } else if (kind == 1) {
            const int64_t at = slot[2 * tok];
            if (at >= 0)
                it.finish((T *)A.k_cache + at + head * A.kcs[2], item, A.pairs, A.d, cs + tok * row, sn + tok * row);
        } else {
            it.finish((T *)A.q_out + (first + tok) * A.qos[0] + head * A.qos[1], item, A.pairs, A.d, cs + tok * row,
                      sn + tok * row);
        }
        i += step;
        if (i < total) {
            split(i);
            load();
        }
    }
}

}  // namespace

int launch_rope(int type, int layout, const RopeArgs &A, uint32_t grid, uint32_t lds, void *stream)
{
#define ECMD_CASE(TY, L)              \
    if (type == TY && layout == L)    \
        return launch_kernel(reinterpret_cast<const void *>(&k_rope<TY, L>), dim3(grid), dim3(kBlock), lds, stream, A);
    ECMD_CASE(S_F16, 0) ECMD_CASE(S_F16, 1) ECMD_CASE(S_BF16, 0) ECMD_CASE(S_BF16, 1) ECMD_CASE(S_F32, 0)
    ECMD_CASE(S_F32, 1)
#undef ECMD_CASE
    return (int)hipErrorInvalidValue;
}

int launch_append(int type, int layout, const AppendArgs &A, uint32_t grid, uint32_t lds, void *stream)
{
#define ECMD_CASE(TY, L)              \
    if (type == TY && layout == L)    \
        return launch_kernel(reinterpret_cast<const void *>(&k_append<TY, L>), dim3(grid), dim3(kBlock), lds, stream, A);
    ECMD_CASE(S_F16, 0) ECMD_CASE(S_F16, 1) ECMD_CASE(S_BF16, 0) ECMD_CASE(S_BF16, 1) ECMD_CASE(S_F32, 0)
    ECMD_CASE(S_F32, 1)
#undef ECMD_CASE
    return (int)hipErrorInvalidValue;
}

}  // namespace ecmd
