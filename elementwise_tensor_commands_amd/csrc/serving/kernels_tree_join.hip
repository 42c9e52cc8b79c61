// kernels_tree_join.hip -- the second launch of attention for trees: joins the
// segments of rows that were cut.
#include "ecmd_kern_tree.h"

namespace ecmd {

namespace {

// 2^A.join_shift work-items to a query vector, four columns to each, four segments at a
// time: (m, l, sums) of the four and of those before are brought to their common maximum.
// FEW: all of a work-group's work-items share one vector's segments, and are joined in LDS;
// else each takes its part of A.join_turn vectors a work-group one after another (where the
// rows lie is worked out once for them).  Empty rows get their zeros here.
template <int TY, bool FEW>
__global__ __launch_bounds__(kAttnBlock) void k_tree_join(const TreeArgs A)
{
    extern __shared__ uint32_t s_rows[];
    __shared__ uint32_t s_scratch[kAttnWaves];
    __shared__ f32x4 s_sum[FEW ? kAttnBlock : 1];
    __shared__ float s_m[FEW ? kAttnBlock : 1], s_l[FEW ? kAttnBlock : 1];
    const uint32_t tid = threadIdx.x;
    const Rows R = make_rows(A, s_rows, s_scratch, tree_span, kTreeExtra);
    const uint32_t all = A.by_vectors.d, share = tree_share(A, R);
    const uint32_t place = tid >> A.join_shift, places = kAttnBlock >> A.join_shift;
    const uint32_t column = (tid - (place << A.join_shift)) * 4;
    const bool wide = A.dv % 4 == 0;
    const uint32_t step = FEW ? places : 1;
    for (uint32_t turn = FEW ? 0 : place; turn < A.join_turn; turn += places) {
        const uint32_t x = blockIdx.x * A.join_turn + turn;
        if (x >= A.b * all) return;
        const uint32_t r = A.by_vectors.div(x), y = x - r * all;
        const uint32_t from = R.prefix[r], upto = R.prefix[r + 1];
        if (from != upto && share == 0) continue;   // a run, written by its work-groups
        const uint32_t first = from == upto ? 0 : from / share;
        const uint32_t count = from == upto ? 0 : (upto - kTreeExtra - 1) / share - first + 1;
        if (count == 1) continue;
        const uint64_t at = (uint64_t)(first + r) * all + y;   // segment s: at + s * all
        float m = -INFINITY, total = 0.0f;
        f32x4 sum = {0, 0, 0, 0};
        for (uint32_t s0 = FEW ? place : 0; s0 < count; s0 += 4 * step) {
            float sm[4], sl[4];
            f32x4 v[4];
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const uint64_t z = at + (uint64_t)min(s0 + u * step, count - 1) * all;
                sm[u] = s0 + u * step < count ? A.ml[2 * z] : -INFINITY;
                sl[u] = A.ml[2 * z + 1];
                const float *p = A.acc + z * A.dv;
                if (wide) v[u] = *(const f32x4 *)(p + min(column, A.dv - 4));
                else
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) v[u][i] = p[min(column + i, A.dv - 1)];
            }
            const float top = fmaxf(fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), m), ref = top == -INFINITY ? 0.0f : top;
            const float a = __builtin_amdgcn_exp2f(m - ref);
            sum *= a;
            total *= a;
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const float w = __builtin_amdgcn_exp2f(sm[u] - ref);   // 0 past the last segment, and where none is seen
                total += w * sl[u];
                if (w != 0.0f) sum += v[u] * w;
            }
            m = top;
        }
        if constexpr (FEW) {
            s_sum[tid] = sum;
            s_m[tid] = m;
            s_l[tid] = total;
            __syncthreads();
            if (place == 0) {
                for (uint32_t o = 1; o < places; ++o) m = fmaxf(m, s_m[o << A.join_shift]);
                const float ref = m == -INFINITY ? 0.0f : m;
                total = 0.0f;
                sum = f32x4{0, 0, 0, 0};
                for (uint32_t o = 0; o < places; ++o) {
                    const uint32_t from = (o << A.join_shift) + tid;
                    const float w = __builtin_amdgcn_exp2f(s_m[from] - ref);
                    total += w * s_l[from];
                    if (w != 0.0f) sum += s_sum[from] * w;
                }
            }
            if (place) return;   // join_turn is 1
        }
        const uint32_t kvh = y / A.m, in = y - kvh * A.m, token = A.by_group.div(in), head = kvh * A.group + in - token * A.group;
        const bool padding = count != 0 && A.ml[2 * (at + (uint64_t)(count - 1) * all) + 1] < 0.0f;
        const bool none = padding || total == 0.0f;
        const int64_t to = (int64_t)r * A.os[0] + (int64_t)token * A.os[1] + (int64_t)head * A.os[2];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (column + i < A.dv) store_typed(TY, A.out, to + column + i, none ? 0.0f : sum[i] / total);
        if (column == 0 && A.lse)
            A.lse[(int64_t)r * A.ls[0] + (int64_t)token * A.ls[1] + (int64_t)head * A.ls[2]] = none ? -INFINITY : tree_log_sum<TY>(m, total);
    }
}

template <int TY>
int launch_join(const TreeArgs &A, void *stream)
{
    const void *fn = A.join_turn == 1 ? reinterpret_cast<const void *>(&k_tree_join<TY, true>)
                                      : reinterpret_cast<const void *>(&k_tree_join<TY, false>);
    return launch_kernel(fn, dim3((A.b * A.by_vectors.d + A.join_turn - 1) / A.join_turn), dim3(kAttnBlock), rows_lds(A.b), stream, A);
}

}  // namespace

int launch_tree_join(int type, const TreeArgs &A, void *stream)
{
    return type == S_F16    ? launch_join<S_F16>(A, stream)
           : type == S_BF16 ? launch_join<S_BF16>(A, stream)
                            : launch_join<S_F32>(A, stream);
}

}  // namespace ecmd
