// ecmd_kern_mass.h -- the weight that attention gave to every page of a row (device
// code; one translation unit per element type instantiates it).
//
//   mass[j] = decay mass[j] + sum_h sum_{x in column j} exp(scale q_h . k_x - lse_h)
//
// The keys are read once and nothing else is large, so HBM bounds it.  A work-group
// takes whole columns of a row, of about 64 positions, and all heads of
// them: a column's sum is then its own business, with no atomics and in one order.
// Its waves take kv heads, or parts of the positions where there are fewer; scores come
// from the matrix units, D[key][head], keys straight from memory to registers, a tile
// ahead of the products.  64 rows of up to 8192 positions, 32 heads over 8 of 128, bf16:
// 93 us, 5.5 TB/s; what is left is work-groups' starts (lengths, then pages, then keys).
#pragma once
#include <hip/hip_runtime.h>

#include "../ecmd_launch.h"
#include "ecmd_attn_tile.h"

namespace ecmd {

namespace {

// Sum over the 16 lanes of a row of lanes, in every one of them.
__device__ inline float row_sum(float x)
{
#define ECMD_ROTATE(CTRL) x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false))
    ECMD_ROTATE(0x128);   // row_ror:8
    ECMD_ROTATE(0x124);
    ECMD_ROTATE(0x122);
    ECMD_ROTATE(0x121);
#undef ECMD_ROTATE
    return x;
}

template <int TY, int NK, AttnEdge EDGE>
__global__ __launch_bounds__(256) void k_mass(const MassArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, KB = 2;
    constexpr uint32_t kTile = 16 * KB, kTiles = kMassKeys / kTile;
    __shared__ uint64_t s_at[kMassKeys];
    __shared__ uint32_t s_valid[kTiles];
    __shared__ float s_part[kAttnWaves][kMassKeys], s_sum[kMassKeys];
    const uint32_t tid = threadIdx.x, lane = tid & 63, j = lane >> 4, hh = lane & 15;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t r = A.by_groups.div(blockIdx.x), c0 = (blockIdx.x - r * A.groups) * A.cols_group;
    const uint32_t c1 = min(c0 + A.cols_group, A.cols);
    const int32_t len = A.lens[(int64_t)r * A.lens_s];
    const uint32_t hi = min((uint32_t)max(len, 0), A.cols * A.page);
    const uint32_t lo = A.window && len > 0 && (uint32_t)len > A.window ? (uint32_t)len - A.window : 0;

    // waves to a kv head (of the positions); a wave's items: 16 heads of a kv head each
    const uint32_t hw = A.hk == 1 ? 4 : A.hk == 2 ? 2 : 1, tile0 = wave % hw;
    const uint32_t parts = (A.group + 15) / 16, items = A.hk * parts, item0 = wave / hw, item_step = kAttnWaves / hw;
    auto piece = [&](const char *p, int c) {
        const int at = (c * 4 + (int)j) * E;
        if constexpr (EDGE == kTiny) return load_some<T, E>(p + at * sizeof(T), (int)A.d - at);
        return load16(p + (EDGE == kTail ? min(at, (int)A.d - E) : at) * sizeof(T));
    };
    auto masked = [&](u32x4 x, int c) {
        if (EDGE == kTail && (uint32_t)(c + 1) * 4 * E > A.d) x = only_own<E>(x, (c * 4 + (int)j) * E, (int)A.d);
        return x;
    };
    auto kv_head = [&](uint32_t item) { return parts == 1 ? item : item / parts; };
    // An item's query vectors and their log-sums: asked for an item ahead.
    u32x4 qn[NK];
    float lse_n = 0.0f;
    auto load_q = [&](uint32_t item) {
        const uint32_t kvh = kv_head(item), g0 = (item - kvh * parts) * 16;
        const uint32_t head = kvh * A.group + min(g0 + hh, A.group - 1);
        const char *qp = (const char *)A.q + (int64_t)r * A.qs[0] + (int64_t)head * A.qs[1];
#pragma unroll
        for (int c = 0; c < NK; ++c) qn[c] = piece(qp, c);
        lse_n = A.lse[(int64_t)r * A.lse_s[0] + (int64_t)head * A.lse_s[1]];
        if (g0 + hh >= A.group) lse_n = -INFINITY;
    };
    float mine = 0.0f;   // column c0 + tid's sum
    bool asked = false;
    const uint32_t begin = c0 * A.page, end = min(c1 * A.page, hi);
    // (a page of more than 256 slots takes turns)
    for (uint32_t base = begin; base < end; base += kMassKeys) {
        if (base + kMassKeys <= lo) continue;
        const uint32_t n = min(kMassKeys, end - base);
        {
            if (!asked && item0 < items) load_q(item0);
            asked = true;
            const uint32_t pos = min(base + tid, end - 1), col = A.by_page.div(pos);
            const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)col * A.pages_s[1]];
            const bool ok = tid < n && base + tid >= lo && id >= 0 && (uint32_t)id < A.n;
            s_at[tid] = ok ? (uint64_t)((int64_t)id * A.kcs[0] + (int64_t)(pos - col * A.page) * A.kcs[1]) : 0;
            const uint64_t bits = __ballot(ok);
            if (lane == 0) {
                s_valid[wave * 2] = (uint32_t)bits;
                s_valid[wave * 2 + 1] = (uint32_t)(bits >> 32);
            }
#pragma unroll
            for (uint32_t k = 0; k < kMassKeys / 64; ++k) s_part[wave][k * 64 + lane] = 0.0f;
        }
        __syncthreads();
        const uint32_t tiles = (n + kTile - 1) / kTile;
        u32x4 kr[KB][NK];
        auto load = [&](uint32_t item, uint32_t t) {
            const char *kbase = (const char *)A.k + (int64_t)kv_head(item) * A.kcs[2];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const char *p = kbase + s_at[t * kTile + kb * 16 + hh];
#pragma unroll
                for (int c = 0; c < NK; ++c) kr[kb][c] = piece(p, c);
            }
        };
        if (tile0 < tiles && item0 < items) {
            load(item0, tile0);
            for (uint32_t item = item0; item < items; item += item_step) {
                u32x4 q[NK];
#pragma unroll
                for (int c = 0; c < NK; ++c) q[c] = masked(qn[c], c);
                const bool on = lse_n != -INFINITY;
                const float lse = lse_n;
                load_q(item + item_step < items ? item + item_step : item0);   // (or of the next turn)
                for (uint32_t t = tile0; t < tiles; t += hw) {
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
                    if (t + hw < tiles) load(item, t + hw);
                    else if (item + item_step < items) load(item + item_step, tile0);
                    const uint32_t valid = s_valid[t];
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        f32x4 w;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool ok = on && valid >> (kb * 16 + j * 4 + i) & 1;
                            // the difference first, then base 2: it is small where a weight counts,
                            // scores and log-sums need not be
                            const float below = __builtin_fmaf(s[kb][i], A.scale, -lse);
                            w[i] = row_sum(ok ? __builtin_amdgcn_exp2f(below * 1.44269504088896340736f) : 0.0f);
                        }
                        if (hh < 4) {
                            const float v = hh == 0 ? w[0] : hh == 1 ? w[1] : hh == 2 ? w[2] : w[3];
                            s_part[wave][t * kTile + kb * 16 + j * 4 + hh] += v;
                        }
                    }
                }
            }
        }
        __syncthreads();
        float sum = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < kAttnWaves; ++w) sum += s_part[w][tid];
        s_sum[tid] = sum;
        __syncthreads();
        if (A.page > kMassKeys) {   // one column: all of them are its
            if (wave == 0) {
                float all = s_sum[lane];
#pragma unroll
                for (uint32_t k = 1; k < kMassKeys / 64; ++k) all += s_sum[k * 64 + lane];
                mine += wave_sum(all);
            }
        } else if (tid < c1 - c0) {
            for (uint32_t k = 0; k < A.page; ++k) {
                const uint32_t x = tid * A.page + k;
                if (x < n) mine += s_sum[x];
            }
        }
        __syncthreads();
    }
    if (tid < c1 - c0) {
        const uint32_t c = c0 + tid;
        const float was = A.mass[(int64_t)r * A.mass_s[0] + (int64_t)c * A.mass_s[1]];
        A.out[(int64_t)r * A.out_s[0] + (int64_t)c * A.out_s[1]] = A.decay * was + mine;
    }
}

template <int TY, int NK, AttnEdge EDGE>
int launch_mass_one(const MassArgs &A, void *stream)
{
    return launch_kernel(reinterpret_cast<const void *>(&k_mass<TY, NK, EDGE>), dim3(A.b * A.groups), dim3(256), 0, stream, A);
}
template <int TY, int NK>
int launch_mass_edge(const MassArgs &A, void *stream)
{
    return A.d == (uint32_t)(NK * 4 * AttnType<TY>::E) ? launch_mass_one<TY, NK, kExact>(A, stream)
                                                       : launch_mass_one<TY, NK, kTail>(A, stream);
}

template <int TY>
int launch_mass_type(const MassArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;
    const uint32_t d = A.d;
    // The smallest that holds d: in steps of 32 elements, in binary32, whose products cost sixteen times
    // as much, of 16 up to 96 (heads of 80 and of 72 by the instances for 80 and for 96: 3 rows in a
    // window of 1000, 12 heads, 9.1 and 12.3 us, 11.3 and 12.3; 16 rows of up to 4096, 16 heads over 4, 16.0 and
    // 17.9, 15.7 and 17.2).
    if (d < (uint32_t)E) return launch_mass_one<TY, U, kTiny>(A, stream);
    if (d <= 64) return launch_mass_edge<TY, 2 * U>(A, stream);
    if constexpr (TY == S_F32) {
        if (d <= 80) return launch_mass_edge<TY, 5>(A, stream);
    }
    return d <= 96    ? launch_mass_edge<TY, 3 * U>(A, stream)
           : d <= 128 ? launch_mass_edge<TY, 4 * U>(A, stream)
           : d <= 192 ? launch_mass_edge<TY, 6 * U>(A, stream)
                      : launch_mass_edge<TY, 8 * U>(A, stream);
}

}  // namespace

}  // namespace ecmd
