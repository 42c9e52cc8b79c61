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
//   out      D[dv][head] += V^T P^T.  Lane h loads the h-th 16 bytes of its keys'
//            values (of each 256); product c takes element c of each (16-bit
//            types: two keys' elements joined by one byte permute), so its row h
//            is column 8 h + c (binary32: 4 h + c).
//
// A head's maximum and rescale factor belong to one lane column: no transposes.
//
// Rows differ in length (some are empty, the table says how long they could be,
// not how long they are), so positions are dealt out by what the lengths say on
// the device: the rows' positions in steps, laid end to end, are cut into equal
// runs.  A run may span rows; each row in it is a segment with a start and an
// end of its own.  Segments of a row that is cut are joined by a second launch.
//
// The four waves of a work-group split its positions and join their sums through
// LDS, or, where there is much to read and the heads allow it, take four kv heads
// of the same positions: together they then read whole slots and exchange nothing.
//
// Measured on one MI355X (a stream of independent reads reaches 6.2 TB/s there, a
// copy 4.9): 64 rows of up to 8192 positions, 8 kv heads of 128, bfloat16, 987 MB:
// 168 us, 5.9 TB/s, the join 6.5 us; two rows of up to 262143, binary16, 289 MB: 52
// and 5.7 us.  One row of 777: 7.4 and 4.7 us, nearly all of it the chain of dependent
// loads (length, page, key) and of barriers; 0.3 us are the weights' further parts
// and the bounding of their sums, which larger calls do not show.  Tried and dropped: as many splits for every
// row (205 us on the first; equal runs 199), half of the registers as accumulation
// registers, which the compiler prefers (32 moves there and back in every tile),
// eight waves to a work-group (a compute unit alone reads no more than 55 to 70
// GB/s either way).
#pragma once
#include <hip/hip_runtime.h>

#include "../ecmd_launch.h"
#include "ecmd_attn_tile.h"

namespace ecmd {

namespace {

// How the steps are dealt out, the same in every work-group and in the join.
// Waves by heads or by positions: 1138 MB in 64 ragged rows take 209 us by heads
// and 228 by positions (streaming loads), 262 MB in 64 rows of 1000 (4096 steps of
// 8 heads) 55 and 45.  Rows whole or cut: 16 rows of 2500, 16 heads, 33 us whole
// and 43 cut; 64 ragged rows of up to 8192, 295 whole and 204 cut.
struct Deal {
    uint32_t head_shift;   // 2^head_shift waves of a work-group take a head each
    uint32_t share;        // steps of a run; 0: a run is a row
};
__device__ inline Deal deal_steps(const AttnArgs &A, const Rows &R)
{
    Deal D;
    const uint32_t heads = A.hk * A.head_tiles;
    // Rows of nearly one length (none a quarter above the mean), enough of them to
    // use the whole memory: cutting them would only add segments.
    if (A.b <= A.runs_whole && (uint64_t)R.all * 5 >= (uint64_t)R.longest * A.b * 4) return Deal{0, 0};
    const bool much = (uint64_t)R.all * heads >= kAttnMuch;
    D.head_shift = much ? A.head_shift : 0;
    const uint32_t runs = much ? A.runs_much : A.runs;
    D.share = (much ? A.by_runs_much : A.by_runs).div(R.all + runs - 1);
    // Rows of about one run's length are not cut at all.
    if (R.longest <= 2 * D.share && A.b <= runs) D.share = 0;
    return D;
}

template <int TY, bool APART = true>
__device__ inline void store_out(const AttnArgs &A, uint32_t r, uint32_t h, uint32_t c, float x)
{
    const Whose w = row_whose<APART>(A, r);
    const int64_t at = (int64_t)w.b * A.os[0] + (int64_t)(w.h * A.hq + h) * A.os[1] + c;
    if constexpr (TY == S_F32)
        ((float *)A.out)[at] = x;
    else if constexpr (TY == S_BF16)
        ((__bf16 *)A.out)[at] = (__bf16)x;
    else
        ((_Float16 *)A.out)[at] = (_Float16)x;
}

template <bool APART = true>
__device__ inline void store_lse(const AttnArgs &A, uint32_t r, uint32_t h, float x)
{
    const Whose w = row_whose<APART>(A, r);
    A.lse[(int64_t)w.b * A.ls[0] + (int64_t)(w.h * A.hq + h) * A.ls[1]] = x;
}

// Weights are held as 2^kBias exp2(score - m).  m is raised only where a score
// passes it by more than kSlack (log2), which spares most tiles the exchange
// between lanes and the rescale; a weight stays below 2^(kBias + kSlack).  With
// binary16, whose numbers end at 2^16 and 2^-24, both leave most of the range to
// the weights below m, and the second part of a weight is held kRests times as
// large: with leading bits of 2^-24 or more and 11 bits below them a weight is off
// by at most 2^-22 of itself or 2^-47 of the one at m, whichever is more.
template <int TY>
constexpr float kSlack = TY == S_F16 ? 4.0f : 8.0f;
template <int TY>
constexpr float kBias = TY == S_F16 ? 11.0f : 0.0f;
template <int TY>
constexpr float kRests = TY == S_F16 ? 2048.0f : 1.0f;

// The natural logarithm of the softmax's sum from a maximum (log2) and the sum
// of the weights against it.
template <int TY>
__device__ inline float log_sum(float top, float total)
{
    if (total == 0.0f) return -INFINITY;
    return ((top == -INFINITY ? 0.0f : top) - kBias<TY> + log2f(total)) * 0.69314718055994530942f;
}

// Waves of a SIMD that an instance asks for: what its registers (keys, values,
// query, sums and the rest, about) leave room for without spills in the loop.
template <int TY, int NK, int VW, AttnEdge EDGE, bool APART>
constexpr int attn_waves()
{
    constexpr int KB = AttnType<TY>::KB, size = TY == S_F32 ? 4 : 2;
    constexpr int regs = KB * NK * 4 + KB * VW * size + NK * 4 + VW * 4 + (TY == S_F32 ? 52 : 60) + (EDGE == kTail ? 10 : 0) + (APART ? 10 : 0);
    return regs > 268 ? 1 : regs > 172 ? 2 : regs > (TY == S_F32 ? 128 : 112) ? 3 : 4;
}

// VW: value columns of a lane (16 VW >= dv).  NK: 16-byte key pieces of a lane
// (4 E NK >= d).  STREAM: the cache is larger than the last-level cache.
// APART: the tables are the kv heads' own.
template <int TY, int NK, int VW, AttnEdge EDGE, bool STREAM, bool APART>
__global__ __launch_bounds__(kAttnBlock, (attn_waves<TY, NK, VW, EDGE, APART>())) void k_attention(const AttnArgs A)
{
    typedef typename AttnType<TY>::T T;
    constexpr int E = AttnType<TY>::E, KB = AttnType<TY>::KB;
    constexpr int VK = 4 * KB;                          // keys whose values a lane holds
    constexpr int PE = VW < E ? VW : E, VP = VW / PE;   // elements of a value piece; pieces
    constexpr uint32_t kTile = 16 * KB;
    constexpr int kRow = 16 * VW + 4;                   // a head's row in the joining buffer (floats)

    __shared__ union {
        struct {
            uint64_t k[kAttnWaves][kTableKeys], v[kAttnWaves][kTableKeys];
            uint64_t valid[kAttnWaves][kTableKeys / 64];
        } table;
        __attribute__((aligned(16))) float join[kAttnWaves][8][kRow];
    } sh;
    __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16], s_top[kAttnWaves][16], s_total[kAttnWaves][16];
    extern __shared__ uint32_t s_rows[];   // unless A.direct
    __shared__ uint32_t s_scratch[kAttnWaves];

    const uint32_t lane = threadIdx.x & 63, j = lane >> 4, hh = lane & 15;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The run of this work-group: steps [step, stop) of all rows', from row r on.
    uint32_t head_shift = 0, group, r, step = 0, stop = 0, bh;
    Rows R{};
    // Work-groups go to the eight dies in turn: the heads of a run follow each other
    // on one, a slot's heads together use all of its cache's channels.
    auto place = [&](const Div31 &by) {   // by: eight runs' work-groups
        const uint32_t u = by.div(blockIdx.x), x = blockIdx.x - u * by.d;
        group = u * 8 + x % 8;
        bh = x / 8;
    };
    if (A.direct) {
        place(A.by_heads);
        if (group >= A.b) return;
        r = group;
    } else {
        R = make_rows(A, s_rows, s_scratch, row_span<APART>);
        const Deal D = deal_steps(A, R);
        head_shift = D.head_shift;
        place(head_shift ? A.by_heads_much : A.by_heads);
        if (D.share == 0) {
            if (group >= A.b) return;
            r = group;
            step = __builtin_amdgcn_readfirstlane(R.prefix[r]);
            stop = __builtin_amdgcn_readfirstlane(R.prefix[r + 1]);
            if (step == stop) return;
        } else {
            step = group * D.share;
            stop = min(step + D.share, R.all);
            if (step >= stop) return;
            uint32_t lo = 0, hi = A.b;   // the row with prefix[r] <= step < prefix[r + 1]
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                if (__builtin_amdgcn_readfirstlane(R.prefix[mid]) <= step) lo = mid;
                else hi = mid;
            }
            r = lo;
        }
    }
    // hw waves side by side take a head each, the others a part of the positions
    const uint32_t hw = 1u << head_shift, part = wave >> head_shift, parts = kAttnWaves >> head_shift;
    const uint32_t sub = wave & (hw - 1), head = bh * hw + sub;
    const uint32_t kvh = A.by_tiles.div(head), ht = head - kvh * A.head_tiles;
    const uint32_t q0 = kvh * A.group + ht * 16, q_n = min(16u, A.group - ht * 16);

    // Where a lane's value pieces start: neighbours to neighbours.  The last ones
    // end with the row.
    auto column = [&](uint32_t m, int piece) {
        const uint32_t at = (piece * 16 + m) * PE;
        return EDGE == kTiny ? at : min(at, A.dv - PE);
    };
    // Piece c of a row of d elements at p.  One that would reach past the end is
    // moved back to end with the row; masked() clears what earlier ones have, all
    // of it where the piece lies past the end altogether.
    auto load_row_piece = [&](const char *p, int c, uint32_t quarter, auto stream) {   // quarter: j
        const int at = (c * 4 + (int)quarter) * E;
        if constexpr (EDGE == kTiny) return load_some<T, E>(p + at * sizeof(T), (int)A.d - at);
        return load16<stream>(p + (EDGE == kTail ? min(at, (int)A.d - E) : at) * sizeof(T));
    };
    auto masked = [&](u32x4 x, int c, uint32_t now) {
        if (EDGE == kTail && (uint32_t)(c + 1) * 4 * E > A.d)   // the same for the whole launch
            x = only_own<E>(x, (c * 4 + (int)fresh(j, now)) * E, (int)A.d);
        return x;
    };

    for (;;) {   // one row of the run
        const Whose whose = row_whose<APART>(A, r);
        const char *kbase = (const char *)A.k + (int64_t)(kvh + whose.h) * A.kcs[2];
        const char *vbase = (const char *)A.v + (int64_t)(kvh + whose.h) * A.vcs[2];
        uint32_t begin, end, steps = 0;
        bool whole_row = true;
        if (A.direct) {
            const Span span = row_span<APART>(A, r);
            begin = span.lo;
            end = span.hi;
        } else {
            const uint32_t first = __builtin_amdgcn_readfirstlane(R.prefix[r]);
            const uint32_t last = __builtin_amdgcn_readfirstlane(R.prefix[r + 1]);
            const uint32_t here = min(stop, last), hi = __builtin_amdgcn_readfirstlane(R.hi[r]);
            whole_row = step == first && here == last;
            steps = here - step;
            begin = __builtin_amdgcn_readfirstlane(R.lo[r]) + (step - first) * kAttnStep;
            end = min(begin + steps * kAttnStep, hi);
        }
        uint32_t wb = begin, we = end;
        if (fresh_uniform(parts, r) > 1) {
            const uint32_t each = (end - begin + parts * kTile - 1) / kTile >> (2 - head_shift) << (KB == 2 ? 5 : 4);
            wb = min(begin + part * each, end);
            we = min(wb + each, end);
        }

        u32x4 q[NK];
        // The query's addresses need not wait for the run's, except where they would
        // take registers of the loop (one row of 777: 11.1 us, or 11.2).
        constexpr bool kLate = TY != S_F32 && VW == 16;
        const uint32_t qh = q0 + min(kLate ? fresh(hh, r) : hh, q_n - 1), qj = kLate ? fresh(j, r) : j;
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const char *p = (const char *)A.q + ((int64_t)whose.b * A.qs[0] + (int64_t)(whose.h * A.hq + qh) * A.qs[1]) * sizeof(T);
            q[c] = masked(load_row_piece(p, c, qj, std::false_type()), c, r);
            if (hh >= q_n) q[c] = u32x4{0, 0, 0, 0};
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
                id[g] = A.pages[(int64_t)whose.b * A.pages_s[0] + (int64_t)whose.h * A.pages_s[2] + (int64_t)col * A.pages_s[1]];
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const bool ok = at + g * 64 + lane < we && id[g] >= 0 && (uint32_t)id[g] < A.n;
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
        uint32_t bits = 0;   // which of the tile's positions count
        auto load_k = [&](uint32_t t) {   // t: offset of the tile in the table
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const char *p = kbase + sh.table.k[wave][t + kb * 16 + hh];
#pragma unroll
                for (int c = 0; c < NK; ++c) kr[kb][c] = load_row_piece(p, c, j, std::bool_constant<STREAM>());
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
                        vr[x][c] = load16<STREAM>(p + at * sizeof(T));
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
            // scores of head hh at the lane's keys
            f32x4 s[KB];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                s[kb] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < NK; ++c) {
                    const u32x4 k = masked(kr[kb][c], c, tile);
                    if constexpr (TY == S_F32) {
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            s[kb] = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(k[f]), as_f(q[c][f]), s[kb], 0, 0, 0);
                    } else {
                        s[kb] = mma16<TY>(k, q[c], s[kb]);
                    }
                }
            }
            const uint32_t now = bits;
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
            for (int x = 0; x < VK; ++x) p[x] = s[x / 4][x % 4] * A.scale_log2;
            if (!whole) {
                // whatever lies in other slots may be NaN: it gets weight 0 and value 0
#pragma unroll
                for (int x = 0; x < VK; ++x) {
                    const bool ok = now >> ((x / 4) * 16 + j * 4 + x % 4) & 1;
                    p[x] = ok ? p[x] : -INFINITY;
                    const uint32_t keep = ok ? ~0u : 0u;
#pragma unroll
                    for (int c = 0; c < VP; ++c) vr[x][c] = vr[x][c] & u32x4{keep, keep, keep, keep};
                }
            }
#pragma unroll
            for (int x = 0; x < VK; ++x) top = fmaxf(top, p[x]);
            if (__any(top > m + kSlack<TY>)) {
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
                // A weight goes in as the sum of 16-bit numbers, its leading bits and
                // the rest: bfloat16 in three parts, which are all of its 24 bits, binary16
                // in two (see kBias).  Fewer would show where values cancel, and the
                // matrix units are idle enough.  The leading part is 0 only if the weight
                // is: an infinite value gives an infinity there, and what the rest (0, or
                // of the other sign) makes of it is no number or the wrong one, so the
                // rests' sums are kept apart and bounded before they are added.
                u32x4 hi, lo, last;
#pragma unroll
                for (int x = 0; x < VK; x += 2) {
                    if constexpr (TY == S_BF16) {
                        // the leading halves of both numbers, which keep the rest
                        auto split = [](float &f, float &g) {
                            const uint32_t a = __builtin_bit_cast(uint32_t, f), b = __builtin_bit_cast(uint32_t, g);
                            f -= as_f(a & 0xFFFF0000u);
                            g -= as_f(b & 0xFFFF0000u);
                            return __builtin_amdgcn_perm(b, a, 0x07060302);
                        };
                        hi[x / 2] = split(p[x], p[x + 1]);
                        lo[x / 2] = split(p[x], p[x + 1]);
                        last[x / 2] = split(p[x], p[x + 1]);
                    } else {
                        const uint32_t a = __builtin_bit_cast(uint32_t, p[x]), b = __builtin_bit_cast(uint32_t, p[x + 1]);
                        // positive numbers order as their bits do; the smallest stands for less
                        const u16x2 least = __builtin_bit_cast(u16x2, min(a, 1u) | min(b, 1u) << 16);
                        const u16x2 bits = __builtin_elementwise_max(
                            __builtin_bit_cast(u16x2, __builtin_amdgcn_cvt_pkrtz(p[x], p[x + 1])), least);
                        const f16x2 h = __builtin_bit_cast(f16x2, bits);
                        hi[x / 2] = __builtin_bit_cast(uint32_t, bits);
                        const f32x2 rest = {(p[x] - (float)h[0]) * kRests<TY>, (p[x + 1] - (float)h[1]) * kRests<TY>};
                        lo[x / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
                    }
                }
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    u32x4 a;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        a[w] = __builtin_amdgcn_perm(vr[2 * w + 1][c / 8][c % 8 / 2], vr[2 * w][c / 8][c % 8 / 2],
                                                     c & 1 ? 0x07060302 : 0x05040100);
                    f32x4 rest = {0, 0, 0, 0};
                    if constexpr (TY == S_BF16) rest = mma16<TY>(a, last, rest);
                    rest = mma16<TY>(a, lo, rest);
                    acc[c] = mma16<TY>(a, hi, acc[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[c][i] = __builtin_fmaf(finite(rest[i]), 1.0f / kRests<TY>, acc[c][i]);
                    asm volatile("" : "+v"(acc[c]));   // added here: all rests at once would not fit the registers
                }
            }
            if (tile < we) load_v(in_table);
        }

        // The segment's sums: final, or for the second launch at a place of its
        // own (work-groups and rows only go forward).
        const uint32_t tid = fresh(wave * 64 + __lane_id(), r), eh = tid & 15, ej = tid >> 4 & 3;
        const uint64_t place = (uint64_t)(group + r) * A.hq + q0;
        auto put = [&](uint32_t hx, uint32_t c, float sum, float total) {
            if (whole_row) store_out<TY, APART>(A, r, q0 + hx, c, total == 0.0f ? 0.0f : sum / total);
            else A.acc[(place + hx) * A.dv + c] = sum;
        };
        auto put_statistics = [&](uint32_t hx, float top, float total) {
            if (!whole_row) {
                A.ml[2 * (place + hx)] = top;
                A.ml[2 * (place + hx) + 1] = total;
            } else if (A.lse) {
                store_lse<APART>(A, r, q0 + hx, log_sum<TY>(top, total));
            }
        };
        // Of `PARTS` waves with the same heads: common maximum, then sums through
        // LDS, eight heads at a time and four columns to a work-item.
        auto join_waves = [&](auto PARTS) {
            constexpr uint32_t P = decltype(PARTS)::value, HW = kAttnWaves / P;
            if (ej == 0) {
                s_m[wave][eh] = m;
                s_l[wave][eh] = l;
            }
            __syncthreads();   // also: the tables are done with
            float top = -INFINITY, total = 0.0f, ms[P];
#pragma unroll
            for (uint32_t w = 0; w < P; ++w) {
                ms[w] = s_m[sub + w * HW][eh];
                top = fmaxf(top, ms[w]);
            }
            const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (uint32_t w = 0; w < P; ++w) total += s_l[sub + w * HW][eh] * __builtin_amdgcn_exp2f(ms[w] - ref);
            if (ej == 0) {   // read after the next barrier
                s_top[wave][eh] = top;
                s_total[wave][eh] = total;
            }
            const float factor = __builtin_amdgcn_exp2f(m - ref);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half * 8 >= (int)min(16u, A.group)) break;   // the same for all waves: barriers follow
                if (half) __syncthreads();
                if ((eh >> 3) == (uint32_t)half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < VW; ++c)
                            sh.join[wave][eh & 7][column(ej * 4 + i, c / PE) + c % PE] = acc[c][i] * factor;
                }
                __syncthreads();
                const uint32_t heads_here = min(8u, q_n > half * 8u ? q_n - half * 8u : 0u);
                for (uint32_t x = part * 64 + (tid & 63); x < heads_here * 4 * VW; x += P * 64) {
                    const uint32_t g = x / (4 * VW), c = x % (4 * VW) * 4, hx = half * 8 + g;
                    f32x4 sum = *(const f32x4 *)&sh.join[sub][g][c];
#pragma unroll
                    for (uint32_t w = 1; w < P; ++w) sum += *(const f32x4 *)&sh.join[sub + w * HW][g][c];
                    const float all = s_total[wave][hx];
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        if (c + k < A.dv) put(hx, c + k, sum[k], all);
                    if (c == 0) put_statistics(hx, s_top[wave][hx], all);
                }
            }
        };
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (parts == 1) {
            if (eh < q_n) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < VW; ++c) {
                        const uint32_t at = column(ej * 4 + i, c / PE) + c % PE;
                        if (EDGE != kTiny || at < A.dv) put(eh, at, acc[c][i], l);
                    }
                if (ej == 0) put_statistics(eh, m, l);
            }
        } else if (parts == 4) {
            join_waves(std::integral_constant<uint32_t, 4>());
        } else {
            join_waves(std::integral_constant<uint32_t, 2>());
        }
        if (A.direct) return;
        step += steps;
        if (step >= stop) return;
        do ++r;
        while (__builtin_amdgcn_readfirstlane(R.prefix[r + 1]) <= step);   // past empty rows
        if (parts > 1) __syncthreads();
    }
}

// The segments of row r, from the work-group `first` on; none: the row is empty.
struct Segments {
    uint32_t first, count;
};
__device__ inline Segments row_segments(const AttnArgs &A, const Rows &R, uint32_t r)
{
    const uint32_t from = R.prefix[r], to = R.prefix[r + 1], share = deal_steps(A, R).share;
    if (from == to) return Segments{0, 0};
    if (share == 0) return Segments{r, 1};
    return Segments{from / share, (to - 1) / share - from / share + 1};
}

// Joins the segments of rows that were cut into few, or writes an empty row's
// zeros: a wave to a row and query head, a segment to a lane and then columns.
template <int TY>
__global__ __launch_bounds__(kAttnBlock) void k_attention_join_few(const AttnArgs A)
{
    extern __shared__ uint32_t s_rows[];
    __shared__ uint32_t s_scratch[kAttnWaves];
    const uint32_t lane = threadIdx.x & 63;
    const Rows R = make_rows(A, s_rows, s_scratch, row_span<true>);
    const uint32_t x = __builtin_amdgcn_readfirstlane(blockIdx.x * kAttnWaves + threadIdx.x / 64);
    if (x >= A.b * A.hq) return;
    const uint32_t r = A.by_heads.div(x), h = x - r * A.hq;   // by_heads: hq here
    const Segments S = row_segments(A, R, r);
    if (S.count == 0) {
        for (uint32_t c = lane; c < A.dv; c += 64) store_out<TY>(A, r, h, c, 0.0f);
        if (lane == 0 && A.lse) store_lse(A, r, h, -INFINITY);
        return;
    }
    if (S.count == 1) return;   // written by its work-group
    const uint64_t at = (uint64_t)(S.first + r) * A.hq + h;   // segment s: at + s * hq
    float v[4][4];   // columns lane, lane + 64, ... of four segments
    auto load = [&](uint32_t s) {
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) {
            const float *p = A.acc + (at + (uint64_t)min(s + u, S.count - 1) * A.hq) * A.dv;
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
                if (c == 0 || c * 64 < A.dv) v[u][c] = p[min(c * 64 + lane, A.dv - 1)];
        }
    };
    load(0);   // on their way while the weights are made
    float m = -INFINITY;
    for (uint32_t s = lane; s < S.count; s += 64) m = fmaxf(m, A.ml[2 * (at + (uint64_t)s * A.hq)]);
    m = wave_max(m);
    const float ref = m == -INFINITY ? 0.0f : m;
    float total = 0.0f, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t s0 = 0; s0 < S.count; s0 += 64) {
        const uint32_t s = s0 + lane;
        float w = 0.0f;
        if (s < S.count) {
            const uint64_t y = 2 * (at + (uint64_t)s * A.hq);
            w = __builtin_amdgcn_exp2f(A.ml[y] - ref);
            total += w * A.ml[y + 1];
        }
        const uint32_t n = min(64u, S.count - s0);
        for (uint32_t k = 0; k < n; k += 4) {
            if (s0 + k) load(s0 + k);
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                if (k + u < n) {
                    const float wu = as_f(__builtin_amdgcn_readlane(__builtin_bit_cast(uint32_t, w), k + u));
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c)
                        if (c == 0 || c * 64 < A.dv) sum[c] += v[u][c] * wu;
                }
        }
    }
    total = wave_sum(total);
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
        if (c * 64 + lane < A.dv) store_out<TY>(A, r, h, c * 64 + lane, total == 0.0f ? 0.0f : sum[c] / total);
    if (lane == 0 && A.lse) store_lse(A, r, h, log_sum<TY>(m, total));
}

// The same for rows cut into many.
// A work-group takes COLS columns: groups of COLS work-items take every so many
// segments, eight loads in flight each.
template <int TY, int THREADS, int COLS>
__global__ __launch_bounds__(THREADS) void k_attention_join(const AttnArgs A)
{
    constexpr uint32_t kGroups = THREADS / COLS, kW = THREADS / 64;
    extern __shared__ uint32_t s_rows[];
    __shared__ uint32_t s_scratch[kAttnWaves];
    __shared__ float s_w[kAttnMaxRuns];
    __shared__ float s_red[2][kW];
    __shared__ float s_sum[THREADS];
    const uint32_t r = A.by_heads.div(blockIdx.x), h = blockIdx.x - r * A.hq;   // by_heads: hq here
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t c0 = blockIdx.y * COLS, c = c0 + threadIdx.x % COLS, g = threadIdx.x / COLS;
    const Rows R = make_rows(A, s_rows, s_scratch, row_span<true>);
    const Segments S = row_segments(A, R, r);
    const bool first_cols = blockIdx.y == 0 && threadIdx.x == 0;
    if (S.count == 0) {
        if (g == 0 && c < A.dv) store_out<TY>(A, r, h, c, 0.0f);
        if (first_cols && A.lse) store_lse(A, r, h, -INFINITY);
        return;
    }
    const uint32_t first = S.first, parts = S.count;
    if (parts == 1) return;   // written by its work-group
    const uint64_t at = (uint64_t)(first + r) * A.hq + h;   // segment s: at + s * hq

    float m = -INFINITY;
    for (uint32_t s = threadIdx.x; s < parts; s += THREADS) m = fmaxf(m, A.ml[2 * (at + (uint64_t)s * A.hq)]);
    m = wave_max(m);
    if (lane == 0) s_red[0][wave] = m;
    __syncthreads();
#pragma unroll
    for (uint32_t w = 0; w < kW; ++w) m = fmaxf(m, s_red[0][w]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    for (uint32_t s = threadIdx.x; s < parts; s += THREADS) {
        const uint64_t x = 2 * (at + (uint64_t)s * A.hq);
        const float w = __builtin_amdgcn_exp2f(A.ml[x] - ref);
        s_w[s] = w;
        l += w * A.ml[x + 1];
    }
    l = wave_sum(l);
    if (lane == 0) s_red[1][wave] = l;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < kW; ++w) total += s_red[1][w];

    float sum = 0.0f;
    if (c < A.dv) {
        const float *p = A.acc + at * A.dv + c;
        const uint64_t stride = (uint64_t)A.hq * A.dv;
        for (uint32_t s = g; s < parts; s += 8 * kGroups) {
            float x[8];
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u) x[u] = s + u * kGroups < parts ? p[(s + u * kGroups) * stride] : 0.0f;
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u)
                if (s + u * kGroups < parts) sum += x[u] * s_w[s + u * kGroups];
        }
    }
    s_sum[threadIdx.x] = sum;
    __syncthreads();
    if (g == 0 && c < A.dv) {
        for (uint32_t x = 1; x < kGroups; ++x) sum += s_sum[x * COLS + c - c0];
        store_out<TY>(A, r, h, c, total == 0.0f ? 0.0f : sum / total);
    }
    if (first_cols && A.lse) store_lse(A, r, h, log_sum<TY>(m, total));
}

template <int TY, int NK, int VW, AttnEdge EDGE>
int launch_attn_one(const AttnArgs &A, void *stream)
{
    // (what a table of a head's own names is little of a large cache, and kept)
    const void *fn = A.apart_tables ? reinterpret_cast<const void *>(&k_attention<TY, NK, VW, EDGE, false, true>)
                     : EDGE != kTiny && A.stream
                         ? reinterpret_cast<const void *>(&k_attention<TY, NK, VW, EDGE, EDGE != kTiny, false>)
                         : reinterpret_cast<const void *>(&k_attention<TY, NK, VW, EDGE, false, false>);
    return launch_kernel(fn, dim3(A.grid), dim3(kAttnBlock), A.direct ? 0 : rows_lds(A.b), stream, A);
}

// The instance: the smallest that holds d and dv; whole key pieces where d is one
// of the common head widths.  Others have pieces moved back: binary32 heads of 80 take
// 18.0 us with an instance of their own and 19.1 without (9 rows, windows of 1000), so
// widths that have none, 112 or 144 among them, give up about that.
template <int TY>
int launch_attn_type(const AttnArgs &A, void *stream)
{
    constexpr int E = AttnType<TY>::E, U = 8 / E;   // 4 U pieces of 16 bytes: 32 elements
    const uint32_t d = A.d, dv = A.dv;
    if (d < (uint32_t)E || dv < (uint32_t)E)
        return d <= 64 && dv <= 64 ? launch_attn_one<TY, 2 * U, 4, kTiny>(A, stream)
                                   : launch_attn_one<TY, 8 * U, 16, kTiny>(A, stream);
    if (dv <= 64) {
        if (d == 64) return launch_attn_one<TY, 2 * U, 4, kExact>(A, stream);
        if (d == 96) return launch_attn_one<TY, 3 * U, 4, kExact>(A, stream);
        if (d == 128) return launch_attn_one<TY, 4 * U, 4, kExact>(A, stream);
        if (TY == S_F32 && d == 80) return launch_attn_one<TY, 5 * U / 2, 4, TY == S_F32 ? kExact : kTail>(A, stream);
        if (d <= 64) return launch_attn_one<TY, 2 * U, 4, kTail>(A, stream);
        if (d <= 96) return launch_attn_one<TY, 3 * U, 4, kTail>(A, stream);
    }
    if (dv <= 128) {
        if (d == 64) return launch_attn_one<TY, 2 * U, 8, kExact>(A, stream);
        if (d == 96) return launch_attn_one<TY, 3 * U, 8, kExact>(A, stream);
        if (d == 128) return launch_attn_one<TY, 4 * U, 8, kExact>(A, stream);
        if (d == 192) return launch_attn_one<TY, 6 * U, 8, kExact>(A, stream);
        if (TY == S_F32 && d == 80) return launch_attn_one<TY, 5 * U / 2, 8, TY == S_F32 ? kExact : kTail>(A, stream);
        if (d <= 96) return launch_attn_one<TY, 3 * U, 8, kTail>(A, stream);
        if (d <= 128) return launch_attn_one<TY, 4 * U, 8, kTail>(A, stream);
    }
    if (d == 192) return launch_attn_one<TY, 6 * U, 16, kExact>(A, stream);
    if (d == 256) return launch_attn_one<TY, 8 * U, 16, kExact>(A, stream);
    if (d <= 192) return launch_attn_one<TY, 6 * U, 16, kTail>(A, stream);
    return launch_attn_one<TY, 8 * U, 16, kTail>(A, stream);
}

template <int TY>
int launch_join_type(const AttnArgs &A, void *stream)
{
    AttnArgs J = A;
    J.by_heads = Div31(A.hq);
    const dim3 grid(A.b * A.hq, (A.dv + 31) / 32);
    if (A.join == 2)
        return launch_kernel(reinterpret_cast<const void *>(&k_attention_join<TY, 1024, 32>), grid, dim3(1024),
                             rows_lds(A.b), stream, J);
    if (A.join == 1)
        return launch_kernel(reinterpret_cast<const void *>(&k_attention_join<TY, 256, 32>), grid, dim3(256),
                             rows_lds(A.b), stream, J);
    return launch_kernel(reinterpret_cast<const void *>(&k_attention_join_few<TY>),
                         dim3((A.b * A.hq + kAttnWaves - 1) / kAttnWaves), dim3(kAttnBlock), rows_lds(A.b), stream, J);
}

}  // namespace

}  // namespace ecmd
