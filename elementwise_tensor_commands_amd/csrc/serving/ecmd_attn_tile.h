// ecmd_attn_tile.h -- what the attention kernels share (device code): matrix
// products, loads of 16-byte pieces, and the dealing of the rows' positions to
// work-groups.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ecmd_serving.h"
#include "ecmd_wave.h"

namespace ecmd {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

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

// x if it is finite, else some finite number.
__device__ inline float finite(float x)
{
    float most = 3.40282346638528859812e38f;
    asm("" : "+s"(most));   // one register and its negative, not two
    return __builtin_amdgcn_fmed3f(x, -most, most);
}

// x, as far as the compiler knows another one for every `now`: what depends on it is
// computed where `now` is known, not moved out of a loop into registers that the
// loop needs.
__device__ inline uint32_t fresh(uint32_t x, uint32_t now)
{
    asm("" : "+v"(x) : "s"(now));
    return x;
}
__device__ inline uint32_t fresh_uniform(uint32_t x, uint32_t now)
{
    asm("" : "+s"(x) : "s"(now));
    return x;
}

// 16 bytes at p, wherever that is.  STREAM: not to be kept in the caches.
template <bool STREAM = false>
__device__ inline u32x4 load16(const char *p)
{
    typedef u32x4 U __attribute__((aligned(2)));
    if constexpr (STREAM) return __builtin_nontemporal_load((const U *)p);
    else return *(const U *)p;
}

// The first n of N elements at p, the rest 0; nothing past them is read.
template <class T, int N>
__device__ inline u32x4 load_some(const char *p, int n)
{
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (e < n) {
            T x;
            __builtin_memcpy(&x, p + e * sizeof(T), sizeof x);
            if constexpr (sizeof(T) == 2)
                v[e / 2] |= (uint32_t)x << (16 * (e & 1));
            else
                v[e] = __builtin_bit_cast(uint32_t, x);
        }
    }
    return v;
}

// How pieces that reach past the end of a row of d or dv elements are read.
enum AttnEdge {
    kExact,   // there are none: d = 4 E NK
    kTail,    // moved back to end with the row; keys' elements read twice are masked off
    kTiny,    // element by element: rows shorter than a piece
};

// Clears what an earlier piece has of the piece from element `at` on of a row of d elements,
// which was moved back to end with the row.
template <int E>
__device__ inline u32x4 only_own(u32x4 x, int at, int d)
{
    const int twice = at - min(at, d - E);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if constexpr (E == 8)
            x[w] &= (2 * w >= twice ? 0xFFFFu : 0u) | (2 * w + 1 >= twice ? 0xFFFF0000u : 0u);
        else
            x[w] &= w >= twice ? ~0u : 0u;
    }
    return x;
}

// Positions of row r that a launch looks at: [lo, hi).
struct Span {
    uint32_t lo, hi;
};
// A row's sequence and kv head (0 unless the tables are the heads' own).
struct Whose {
    uint32_t b, h;
};
template <bool APART = true>
__device__ inline Whose row_whose(const AttnArgs &A, uint32_t r)
{
    if (!APART) return Whose{r, 0};
    const uint32_t b = A.by_apart.div(r);
    return Whose{b, r - b * A.apart};
}
template <bool APART = true>
__device__ inline Span row_span(const AttnArgs &A, uint32_t r)
{
    const Whose w = row_whose<APART>(A, r);
    const int32_t len = A.lens[(int64_t)w.b * A.lens_s[0] + (int64_t)w.h * A.lens_s[1]];
    const uint32_t held = A.cols * A.page;
    Span s{0, 0};
    if (len <= 0) return s;
    s.hi = min((uint32_t)len, held);
    if (A.window && (uint32_t)len > A.window) s.lo = min((uint32_t)len - A.window, s.hi);
    return s;
}

// The rows' spans and the steps before each row, in LDS.
struct Rows {
    uint32_t *prefix;    // [b + 1]
    uint32_t *lo, *hi;   // [b]
    uint32_t all, longest;
};
__host__ __device__ inline uint32_t rows_lds(uint32_t b) { return (3 * b + 1) * 4; }

// A row that holds something counts for `extra` steps more.
// Up to 64 rows every wave makes the whole of it, the same values in the same
// places, and waits for nobody; more rows are the first kAttnBlock work-items'
// and end with a barrier.
template <class Args, class SpanOf>
__device__ inline Rows make_rows(const Args &A, uint32_t *lds, uint32_t *scratch, SpanOf span_of, uint32_t extra = 0)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Rows R{lds, lds + A.b + 1, lds + 2 * A.b + 1, 0, 0};
    const bool alone = A.b <= 64;
    uint32_t run = 0, most = 0;
    for (uint32_t r0 = 0; r0 < A.b; r0 += kAttnBlock) {
        const uint32_t r = alone ? lane : threadIdx.x < kAttnBlock ? r0 + threadIdx.x : A.b;
        uint32_t x = 0;
        if (r < A.b) {
            const Span s = span_of(A, r);
            R.lo[r] = s.lo;
            R.hi[r] = s.hi;
            x = (s.hi - s.lo + kAttnStep - 1) / kAttnStep;
            if (x) x += extra;
            most = max(most, x);
        }
        const uint32_t inc = wave_prefix(x);
        uint32_t before = run;
        if (alone) {
            run = last_lane(inc);
        } else {
            if (lane == 63 && wave < kAttnWaves) scratch[wave] = inc;
            __syncthreads();
#pragma unroll
            for (uint32_t w = 0; w < kAttnWaves; ++w) {
                if (w < wave) before += scratch[w];
                run += scratch[w];
            }
            __syncthreads();
        }
        if (r < A.b) R.prefix[r] = before + inc - x;
    }
    if (alone ? lane == 0 : threadIdx.x == 0) R.prefix[A.b] = run;
    most = wave_max(most);
    if (alone) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        if (lane == 0 && wave < kAttnWaves) scratch[wave] = most;
        __syncthreads();
#pragma unroll
        for (uint32_t w = 0; w < kAttnWaves; ++w) most = max(most, scratch[w]);
    }
    R.all = __builtin_amdgcn_readfirstlane(run);
    R.longest = __builtin_amdgcn_readfirstlane(most);
    return R;
}

}  // namespace

}  // namespace ecmd
