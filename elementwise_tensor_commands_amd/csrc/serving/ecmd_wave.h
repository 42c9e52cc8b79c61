// ecmd_wave.h -- prefixes, sums and maxima over the 64 lanes of a wave (device
// code), by moves between neighbouring lanes within vector instructions: six of
// them, where an exchange through LDS waits about 100 cycles in every step.
#pragma once
#include <hip/hip_runtime.h>

namespace ecmd {

// Lane i's op over lanes 0 .. i: within rows of 16 lanes by shifts of 1, 2, 4 and
// 8, then the last lane of rows 0 and 2 into rows 1 and 3, then lane 31's into rows
// 2 and 3.  A lane without a source takes `none`, which changes nothing.
template <class T, class Op>
__device__ inline T wave_scan(T x, T none, Op op)
{
    static_assert(sizeof(T) == 4);
#define ECMD_STEP(CTRL, ROWS)                                                                                        \
    x = op(x, __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),                      \
                                                                __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false)))
    ECMD_STEP(0x111, 0xf);   // row_shr:1
    ECMD_STEP(0x112, 0xf);
    ECMD_STEP(0x114, 0xf);
    ECMD_STEP(0x118, 0xf);
    ECMD_STEP(0x142, 0xa);   // row_bcast:15
    ECMD_STEP(0x143, 0xc);   // row_bcast:31
#undef ECMD_STEP
    return x;
}

template <class T>
__device__ inline T last_lane(T x)
{
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

__device__ inline uint32_t wave_prefix(uint32_t x)
{
    return wave_scan(x, 0u, [](uint32_t a, uint32_t b) { return a + b; });
}
// Over all lanes, in every lane.
__device__ inline uint32_t wave_sum(uint32_t x) { return last_lane(wave_prefix(x)); }
__device__ inline float wave_sum(float x)
{
    return last_lane(wave_scan(x, 0.0f, [](float a, float b) { return a + b; }));
}
__device__ inline uint32_t wave_max(uint32_t x)
{
    return last_lane(wave_scan(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
}
__device__ inline float wave_max(float x)   // NaN counts as nothing
{
    return last_lane(wave_scan(x, -INFINITY, [](float a, float b) { return fmaxf(a, b); }));
}

}  // namespace ecmd
