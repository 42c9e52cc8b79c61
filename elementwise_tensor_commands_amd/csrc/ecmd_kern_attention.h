// ecmd_kern_attention.h -- attention of one new token per sequence over a paged
// key-value cache, split over the positions (device code; one translation unit
// per element type instantiates it).
//
//   out = sum_x p_x v_x / sum_x p_x,   p_x = exp(scale q . k_x - m)
//
// in one pass over the positions with the running maximum m.  The cache is read
// once and nothing else is large, so HBM bounds it: the kernel's job is to keep
// loads in flight.  Keys and values go from HBM straight to registers in the
// operand layouts of the matrix instructions; no tile passes through LDS, and
// the waves of a work-group share nothing until the end.
//
// A wave takes tiles of 16 KB positions (KB = 2, binary32: 1) of one kv head and
// up to 16 of its query heads (fewer are padded with zeros; the matrix units
// have that to spare, by a factor of several):
//
//   scores   D[key][head] = K Q^T.  A lane holds 16-byte pieces of key lane % 16;
//            the products run over d in whatever order Q is held in too.  Lane
//            (j = lane / 16, h = lane % 16) gets the scores of head h at keys
//            16 kb + 4 j + i, i = 0..3.
//   weights  exp2 of those in place.  The contraction of the second product may
//            also run in any order of keys, so the same lane's weights are its
//            operand as they are, with lane j loading the values of keys
//            16 kb + 4 j + i.
//   out      D[dv][head] += V^T P^T.  Lane h loads VW consecutive elements of
//            its keys' values; product c takes element c of each (16-bit types:
//            two keys' elements joined by one byte permute), so its row h is
//            column VW h + c.
//
// A head's maximum and rescale factor belong to one lane column: no transposes.
#pragma once
#include <hip/hip_runtime.h>

#include "ecmd_launch.h"
#include "ecmd_serving.h"

namespace ecmd {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kAttnBlock = 256, kAttnWaves = 4;
constexpr uint32_t kTableKeys = 256;   // positions whose cache offsets a wave holds at a time

template <int TY>
struct AttnType {
    typedef uint16_t T;
    static constexpr int E = 8, KB = 2;   // elements of a 16-byte piece; key blocks of a tile
};
template <>
struct AttnType<S_F32> {
    typedef float T;
    static constexpr int E = 4, KB = 1;
};

template <int TY>
__device__ inline f32x4 mma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (TY == S_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

__device__ inline float as_f(uint32_t x) { return __builtin_bit_cast(float, x); }

// The first n elements (16-bit or 32-bit, `E` to a piece) of 16 bytes at p, the
// rest 0; nothing past them is read.
template <class T, int E, bool RAGGED>
__device__ inline u32x4 load_piece(const char *p, int n)
{
    u32x4 v = {0, 0, 0, 0};
    if (!RAGGED || n >= E) {
        __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (e < n) {
                T x;
                __builtin_memcpy(&x, p + e * sizeof(T), sizeof x);
                if constexpr (E == 8)
                    v[e / 2] |= (uint32_t)x << (16 * (e & 1));
                else
                    v[e] = __builtin_bit_cast(uint32_t, x);
            }
        }
    }
    return v;
}

// Positions of row r that a launch looks at: [lo, hi).
struct Span {
    uint32_t lo, hi;
};
__device__ inline Span row_span(const AttnArgs &A, uint32_t r)
{
    const int32_t len = A.lens[(int64_t)r * A.lens_s];
    const uint32_t held = A.cols * A.page;
    Span s{0, 0};
    if (len <= 0) return s;
    s.hi = min((uint32_t)len, held);
    if (A.window && (uint32_t)len > A.window) s.lo = min((uint32_t)len - A.window, s.hi);
    return s;
}
// Each split's share of them: equal, in whole work-group steps.
__device__ inline uint32_t split_share(const AttnArgs &A, uint32_t keys)
{
    const uint32_t each = A.by_splits.div(keys + A.splits - 1);
    return (each + kAttnShare - 1) / kAttnShare * kAttnShare;
}

template <int TY>
__device__ inline void store_out(const AttnArgs &A, uint32_t r, uint32_t h, uint32_t c, float x)
{
    const int64_t at = (int64_t)r * A.os[0] + (int64_t)h * A.os[1] + c;
    if constexpr (TY == S_F32)
        ((float *)A.out)[at] = x;
    else if constexpr (TY == S_BF16)
        ((__bf16 *)A.out)[at] = (__bf16)x;
    else
        ((_Float16 *)A.out)[at] = (_Float16)x;
}

// Weights are held as 2^kBias exp2(score - m).  m is raised only where a score
// passes it by more than kSlack (log2), which spares most tiles the exchange
// between lanes and the rescale; a weight stays below 2^(kBias + kSlack).  The
// bias keeps small binary16 weights out of its subnormals.
constexpr float kSlack = 8.0f;
template <int TY>
constexpr float kBias = TY == S_F16 ? 6.0f : 0.0f;

// VW: value columns of a lane (16 VW >= dv).  NK: 16-byte key pieces of a lane
// (4 E NK >= d).  RAGGED: d is not 4 E NK, or dv no multiple of VW.
template <int TY, int NK, int VW, bool RAGGED>
__global__ __launch_bounds__(kAttnBlock) void k_attention(const AttnArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, KB = AttnType<TY>::KB;
    constexpr int VK = 4 * KB;                        // keys whose values a lane holds
    constexpr int VP = VW * (int)sizeof(T) / 16 > 0 ? VW * (int)sizeof(T) / 16 : 1;   // 16-byte pieces of those
    constexpr uint32_t kTile = 16 * KB;
    constexpr int kRow = 16 * VW + 4;                 // a head's row in the joining buffer (floats)

    __shared__ union {
        struct {
            uint64_t k[kAttnWaves][kTableKeys], v[kAttnWaves][kTableKeys];
            uint64_t valid[kAttnWaves][kTableKeys / 64];
        } table;
        float join[kAttnWaves][8][kRow];
    } sh;
    __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16];

    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane >> 4, hh = lane & 15;
    // heads of one row and split are neighbours: together they read whole slots
    const uint32_t heads = A.hk * A.head_tiles;
    const uint32_t rs = A.by_heads.div(blockIdx.x), head = blockIdx.x - rs * heads;
    const uint32_t r = A.by_splits.div(rs), split = rs - r * A.splits;
    const uint32_t kvh = head / A.head_tiles, ht = head - kvh * A.head_tiles;
    const uint32_t q0 = kvh * A.group + ht * 16, q_n = min(16u, A.group - ht * 16);

    const Span span = row_span(A, r);
    const uint32_t share = split_share(A, span.hi - span.lo);
    const uint32_t begin = span.lo + split * share;
    // the first split of an empty row still writes its zeros
    if (split > 0 && (split * (uint64_t)share >= span.hi - span.lo)) return;
    const uint32_t end = min(begin + share, span.hi);
    const uint32_t wshare = share / kAttnWaves;
    const uint32_t wb = min(begin + wave * wshare, end), we = min(wb + wshare, end);

    u32x4 q[NK];
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        const int at = (c * 4 + j) * E;
        const char *p = (const char *)A.q + ((int64_t)r * A.qs[0] + (int64_t)(q0 + hh) * A.qs[1] + at) * sizeof(T);
        q[c] = u32x4{0, 0, 0, 0};
        if (hh < q_n) q[c] = load_piece<T, E, RAGGED>(p, (int)A.d - at);
    }

    f32x4 acc[VW];
#pragma unroll
    for (int c = 0; c < VW; ++c) acc[c] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, mref = 0.0f, l = 0.0f;

    const char *kbase = (const char *)A.k + (int64_t)kvh * A.kcs[2] + j * 16;
    const uint32_t vcol = RAGGED ? hh * VW : min(hh * VW, A.dv - VW);
    const char *vbase = (const char *)A.v + (int64_t)kvh * A.vcs[2] + vcol * sizeof(T);
    const int vleft = (int)A.dv - (int)vcol;

    // Offsets of the wave's next kTableKeys positions; what is no position of
    // this row's gets slot 0 of page 0, which exists, and a clear bit.
    auto fill = [&](uint32_t at) {
#pragma unroll
        for (uint32_t g = 0; g < kTableKeys / 64; ++g) {
            const uint32_t pos = at + g * 64 + lane;
            int32_t id = -1;
            uint32_t in = 0;
            if (pos < we) {
                const uint32_t col = A.by_page.div(pos);
                in = pos - col * A.page;
                id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)col * A.pages_s[1]];
            }
            const bool ok = id >= 0 && (uint32_t)id < A.n;
            if (!ok) id = 0, in = 0;
            sh.table.k[wave][g * 64 + lane] = (uint64_t)((int64_t)id * A.kcs[0] + (int64_t)in * A.kcs[1]);
            sh.table.v[wave][g * 64 + lane] = (uint64_t)((int64_t)id * A.vcs[0] + (int64_t)in * A.vcs[1]);
            const uint64_t bits = __ballot(ok);
            if (lane == 0) sh.table.valid[wave][g] = bits;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };

    u32x4 kr[KB][NK];
    u32x4 vr[VK][VP];
    uint32_t bits = 0;   // which of the tile's positions count
    auto load_k = [&](uint32_t t) {   // t: offset of the tile in the table
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const char *p = kbase + sh.table.k[wave][t + kb * 16 + hh];
#pragma unroll
            for (int c = 0; c < NK; ++c)
                kr[kb][c] = load_piece<T, E, RAGGED>(p + c * 64, (int)A.d - (c * 4 + (int)j) * E);
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
                if constexpr (VW * sizeof(T) >= 16) {
                    vr[x][c] = load_piece<T, E, RAGGED>(p + c * 16, vleft - c * E);
                } else {   // four 16-bit columns
                    vr[x][c] = u32x4{0, 0, 0, 0};
                    if (!RAGGED || vleft >= VW)
                        __builtin_memcpy(&vr[x][c], p, VW * sizeof(T));
                    else
                        vr[x][c] = load_piece<T, E, true>(p, vleft);
                }
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
        // scores of head hh at the lane's keys
        f32x4 s[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            s[kb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                if constexpr (TY == S_F32) {
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        s[kb] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(kr[kb][c][f]), as_f(q[c][f]), s[kb], 0, 0, 0);
                } else {
                    s[kb] = mma16<TY>(kr[kb][c], q[c], s[kb]);
                }
            }
        }
        const uint32_t now = bits;
        const uint32_t v_at = in_table;
        (void)v_at;
        tile += kTile;
        in_table += kTile;
        if (tile < we) {
            if (in_table == kTableKeys) {
                fill(tile);
                in_table = 0;
            }
            load_k(in_table);
        }

        float p[VK];
        float top = -INFINITY;
        const bool whole = now == (KB == 2 ? 0xFFFFFFFFu : 0xFFFFu);
#pragma unroll
        for (int x = 0; x < VK; ++x) {
            p[x] = s[x / 4][x % 4] * A.scale_log2;
            if (!whole) {
                const bool ok = now >> ((x / 4) * 16 + j * 4 + x % 4) & 1;
                p[x] = ok ? p[x] : -INFINITY;
                if (!ok) {   // whatever lies there may be NaN: it gets weight 0 and value 0
#pragma unroll
                    for (int c = 0; c < VP; ++c) vr[x][c] = u32x4{0, 0, 0, 0};
                }
            }
            top = fmaxf(top, p[x]);
        }
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float mn = fmaxf(m, top);
            mref = mn == -INFINITY ? 0.0f : mn;
            const float a = __builtin_amdgcn_exp2f(m - mref);
            m = mn;
            l *= a;
#pragma unroll
            for (int c = 0; c < VW; ++c) acc[c] *= a;
        }
#pragma unroll
        for (int x = 0; x < VK; ++x) {
            p[x] = __builtin_amdgcn_exp2f(p[x] - (mref - kBias<TY>));
            l += p[x];
        }

        if constexpr (TY == S_F32) {
#pragma unroll
            for (int x = 0; x < VK; ++x)
#pragma unroll
                for (int c = 0; c < VW; ++c)
                    acc[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(vr[x][c / 4][c % 4]), p[x], acc[c], 0, 0, 0);
        } else {
            // A weight goes in as the sum of two 16-bit numbers, its leading bits
            // and the rest: weights rounded to one would double the error of the
            // output's own rounding, and the matrix units are idle enough.
            u32x4 hi, lo;
#pragma unroll
            for (int x = 0; x < VK; x += 2) {
                if constexpr (TY == S_BF16) {
                    const uint32_t a = __builtin_bit_cast(uint32_t, p[x]), b = __builtin_bit_cast(uint32_t, p[x + 1]);
                    hi[x / 2] = __builtin_amdgcn_perm(b, a, 0x07060302);
                    const f32x2 rest = {p[x] - as_f(a & 0xFFFF0000u), p[x + 1] - as_f(b & 0xFFFF0000u)};
                    lo[x / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, bf16x2));
                } else {
                    const auto h = __builtin_amdgcn_cvt_pkrtz(p[x], p[x + 1]);
                    hi[x / 2] = __builtin_bit_cast(uint32_t, h);
                    lo[x / 2] = __builtin_bit_cast(
                        uint32_t, __builtin_amdgcn_cvt_pkrtz(p[x] - (float)h[0], p[x + 1] - (float)h[1]));
                }
            }
#pragma unroll
            for (int c = 0; c < VW; ++c) {
                u32x4 a;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    a[w] = __builtin_amdgcn_perm(vr[2 * w + 1][c / 8][c % 8 / 2], vr[2 * w][c / 8][c % 8 / 2],
                                                 c & 1 ? 0x07060302 : 0x05040100);
                acc[c] = mma16<TY>(a, hi, acc[c]);
                acc[c] = mma16<TY>(a, lo, acc[c]);
            }
        }
        if (tile < we) load_v(in_table);
    }

    // Join the waves: common maximum, then sums head by head through LDS, eight
    // heads at a time.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();   // the tables are done with
    if (lane < 16) {
        s_m[wave][lane] = m;
        s_l[wave][lane] = l;
    }
    __syncthreads();
    float mj = -INFINITY;
#pragma unroll
    for (int w = 0; w < (int)kAttnWaves; ++w) mj = fmaxf(mj, s_m[w][hh]);
    const float factor = __builtin_amdgcn_exp2f(m - (mj == -INFINITY ? 0.0f : mj));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half * 8 >= (int)q_n) break;
        if (half) __syncthreads();
        if ((hh >> 3) == (uint32_t)half) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < VW; ++c) sh.join[wave][hh & 7][(j * 4 + i) * VW + c] = acc[c][i] * factor;
        }
        __syncthreads();
        for (uint32_t x = threadIdx.x; x < 8 * 16 * VW; x += kAttnBlock) {
            const uint32_t g = x / (16 * VW), c = x % (16 * VW), hx = half * 8 + g;
            if (hx >= q_n || c >= A.dv) continue;
            float sum = 0.0f, total = 0.0f, mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < (int)kAttnWaves; ++w) mm = fmaxf(mm, s_m[w][hx]);
            const float ref = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
            for (int w = 0; w < (int)kAttnWaves; ++w) {
                sum += sh.join[w][g][c];
                total += s_l[w][hx] * __builtin_amdgcn_exp2f(s_m[w][hx] - ref);
            }
            const uint32_t h = q0 + hx;
            if (A.splits == 1) {
                store_out<TY>(A, r, h, c, total == 0.0f ? 0.0f : sum / total);
                if (c == 0 && A.lse)
                    A.lse[(int64_t)r * A.ls[0] + (int64_t)h * A.ls[1]] =
                        total == 0.0f ? -INFINITY : (ref - kBias<TY> + log2f(total)) * 0.69314718055994530942f;
            } else {
                const uint64_t at = ((uint64_t)r * A.hq + h) * A.splits + split;
                A.acc[at * A.dv + c] = sum;
                if (c == 0) {
                    A.ml[2 * at] = mm;
                    A.ml[2 * at + 1] = total;
                }
            }
        }
    }
}

// Joins the splits of one row and query head (a work-group).
template <int TY>
__global__ __launch_bounds__(kAttnBlock) void k_attention_join(const AttnArgs A)
{
    __shared__ float s_w[kAttnMaxSplits];
    __shared__ float s_red[2][kAttnWaves];
    __shared__ float s_sum[kAttnBlock];
    const uint32_t r = A.by_heads.div(blockIdx.x), h = blockIdx.x - r * A.hq;   // by_heads: hq here
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Span span = row_span(A, r);
    const uint32_t keys = span.hi - span.lo, share = split_share(A, keys);
    const uint32_t parts = keys ? min(A.splits, (keys + share - 1) / share) : 1;
    const uint64_t at = ((uint64_t)r * A.hq + h) * A.splits;

    float m = -INFINITY;
    for (uint32_t s = threadIdx.x; s < parts; s += kAttnBlock) m = fmaxf(m, A.ml[2 * (at + s)]);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) s_red[0][wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < (int)kAttnWaves; ++w) m = fmaxf(m, s_red[0][w]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    for (uint32_t s = threadIdx.x; s < parts; s += kAttnBlock) {
        const float w = __builtin_amdgcn_exp2f(A.ml[2 * (at + s)] - ref);
        s_w[s] = w;
        l += w * A.ml[2 * (at + s) + 1];
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) l += __shfl_xor(l, o);
    if (lane == 0) s_red[1][wave] = l;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < (int)kAttnWaves; ++w) total += s_red[1][w];

    // columns across lanes, the splits dealt to groups of lanes
    uint32_t width = 32;
    while (width < A.dv) width *= 2;   // dv <= 256
    const uint32_t c = threadIdx.x % width, g = threadIdx.x / width, groups = kAttnBlock / width;
    float sum = 0.0f;
    if (c < A.dv)
        for (uint32_t s = g; s < parts; s += groups) sum += A.acc[(at + s) * A.dv + c] * s_w[s];
    s_sum[threadIdx.x] = sum;
    __syncthreads();
    if (g == 0 && c < A.dv) {
        for (uint32_t x = 1; x < groups; ++x) sum += s_sum[x * width + c];
        store_out<TY>(A, r, h, c, total == 0.0f ? 0.0f : sum / total);
    }
    if (threadIdx.x == 0 && A.lse)
        A.lse[(int64_t)r * A.ls[0] + (int64_t)h * A.ls[1]] =
            total == 0.0f ? -INFINITY : (ref - kBias<TY> + log2f(total)) * 0.69314718055994530942f;
}

template <int TY, int NK, int VW, bool RAGGED>
int launch_attn_one(const AttnArgs &A, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_attention<TY, NK, VW, RAGGED>),
                         dim3(A.b * A.splits * A.hk * A.head_tiles), dim3(kAttnBlock), 0, stream, A);
}

// The instance: whole pieces of keys and values where d and dv have them (the
// common head widths), else the next larger one that checks each piece.
template <int TY>
int launch_attn_type(const AttnArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;   // 16-byte pieces of 32 elements: 4 U
    const uint32_t d = A.d, dv = A.dv;
    if (dv % 8 == 0 && dv <= 64 && dv % 4 == 0) {
        if (d == 64) return launch_attn_one<TY, 2 * U, 4, false>(A, stream);
        if (d == 96) return launch_attn_one<TY, 3 * U, 4, false>(A, stream);
        if (d == 128) return launch_attn_one<TY, 4 * U, 4, false>(A, stream);
    } else if (dv % 8 == 0 && dv <= 128) {
        if (d == 64) return launch_attn_one<TY, 2 * U, 8, false>(A, stream);
        if (d == 96) return launch_attn_one<TY, 3 * U, 8, false>(A, stream);
        if (d == 128) return launch_attn_one<TY, 4 * U, 8, false>(A, stream);
    }
    if (dv % 16 == 0) {
        if (d == 192) return launch_attn_one<TY, 6 * U, 16, false>(A, stream);
        if (d == 256) return launch_attn_one<TY, 8 * U, 16, false>(A, stream);
    }
    if (d <= 64 && dv <= 64) return launch_attn_one<TY, 2 * U, 4, true>(A, stream);
    if (d <= 128 && dv <= 128) return launch_attn_one<TY, 4 * U, 8, true>(A, stream);
    return launch_attn_one<TY, 8 * U, 16, true>(A, stream);
}

template <int TY>
int launch_join_type(const AttnArgs &A, void *stream)
{
    AttnArgs J = A;
    J.by_heads = Div31(A.hq);
    return launch_kernel(reinterpret_cast<const void *>(&k_attention_join<TY>), dim3(A.b * A.hq), dim3(kAttnBlock), 0,
                         stream, J);
}

}  // namespace

}  // namespace ecmd
