// kernels_tree_join.hip -- the second launch of attention for trees: joins the
// segments of rows that were cut.
#include "ecmd_kern_tree.h"

namespace ecmd {

namespace {

// A wave to a row and query vector: a segment to a lane for the weights, then its
// columns.  Empty rows get their zeros here.
template <int TY>
__global__ __launch_bounds__(kAttnBlock) void k_tree_join(const TreeArgs A)
{
    extern __shared__ uint32_t s_rows[];
    __shared__ uint32_t s_scratch[kAttnWaves];
    const uint32_t lane = threadIdx.x & 63;
    const Rows R = make_rows(A, s_rows, s_scratch, tree_span);
    const uint32_t x = __builtin_amdgcn_readfirstlane(blockIdx.x * kAttnWaves + threadIdx.x / 64);
    const uint32_t all = A.by_vectors.d;
    if (x >= A.b * all) return;
    const uint32_t r = A.by_vectors.div(x), y = x - r * all;
    const uint32_t kvh = y / A.m, in = y - kvh * A.m, token = A.by_group.div(in), head = kvh * A.group + in - token * A.group;
    const int64_t to = (int64_t)r * A.os[0] + (int64_t)token * A.os[1] + (int64_t)head * A.os[2];
    auto put_lse = [&](float v) {
        if (lane == 0 && A.lse) A.lse[(int64_t)r * A.ls[0] + (int64_t)token * A.ls[1] + (int64_t)head * A.ls[2]] = v;
    };
    const uint32_t from = R.prefix[r], upto = R.prefix[r + 1], share = tree_share(A, R);
    if (from == upto) {
        for (uint32_t c = lane; c < A.dv; c += 64) store_typed(TY, A.out, to + c, 0.0f);
        put_lse(-INFINITY);
        return;
    }
    if (share == 0) return;   // a run, written by its work-groups
    const uint32_t first = from / share, count = (upto - 1) / share - first + 1;
    if (count == 1) return;
    const uint64_t at = (uint64_t)(first + r) * all + y;   // segment s: at + s * all
    float m = -INFINITY;
    for (uint32_t s = lane; s < count; s += 64) m = fmaxf(m, A.ml[2 * (at + (uint64_t)s * all)]);
    m = wave_max(m);
    const float ref = m == -INFINITY ? 0.0f : m;
    const bool padding = A.ml[2 * (at + (uint64_t)(count - 1) * all) + 1] < 0.0f;
    float total = 0.0f, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t s0 = 0; s0 < count; s0 += 64) {
        const uint32_t s = s0 + lane;
        float w = 0.0f;
        if (s < count) {
            const uint64_t z = 2 * (at + (uint64_t)s * all);
            w = __builtin_amdgcn_exp2f(A.ml[z] - ref);
            total += w * A.ml[z + 1];
        }
        const uint32_t n = min(64u, count - s0);
        for (uint32_t k = 0; k < n; k += 4) {
            float v[4][4];   // columns lane, lane + 64, ... of four segments
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const float *p = A.acc + (at + (uint64_t)min(s0 + k + u, count - 1) * all) * A.dv;
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
                    if (c == 0 || c * 64 < A.dv) v[u][c] = p[min(c * 64 + lane, A.dv - 1)];
            }
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
    const bool none = padding || total == 0.0f;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
        if (c * 64 + lane < A.dv) store_typed(TY, A.out, to + c * 64 + lane, none ? 0.0f : sum[c] / total);
    put_lse(none ? -INFINITY : tree_log_sum<TY>(m, total));
}

}  // namespace

int launch_tree_join(int type, const TreeArgs &A, void *stream)
{
    const void *fn = type == S_F16    ? reinterpret_cast<const void *>(&k_tree_join<S_F16>)
                     : type == S_BF16 ? reinterpret_cast<const void *>(&k_tree_join<S_BF16>)
                                      : reinterpret_cast<const void *>(&k_tree_join<S_F32>);
    return launch_kernel(fn, dim3((A.b * A.by_vectors.d + kAttnWaves - 1) / kAttnWaves), dim3(kAttnBlock), rows_lds(A.b),
                         stream, A);
}

}  // namespace ecmd
