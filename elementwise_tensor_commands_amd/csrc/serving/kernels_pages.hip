// kernels_pages.hip -- the page bookkeeping of a paged key-value cache: assign,
// compact, copy.
//
// Assigning and compacting need the rank of a page among the free (or live)
// ones, and the page of a given rank.  Both come from one bit per page: a ballot
// makes a wave's 64 bits, each word keeps the count of set bits before it
// within its tile, each tile its total.  A rank is then two prefixes and a
// population count, a selection two binary searches and one within a word.
// What is left is integer reads and writes of the tables, a few microseconds of
// dependent accesses and launches at any size met in practice, so the number of
// launches is kept small: two to assign and two to compact, one where little is to do.
//
// Only integer atomics (reference counts) are used: results do not depend on
// their order.
//
// Measured on one MI355X: 512 rows of 1024 entries and 131072 pages are assigned in
// 3.3 + 6.2 us; 32768 pages compacted in 4.8 + 4.8 us, and 8192 of them, 16 KB in
// each of two pools, copied in 96, 5.6 TB/s (104 without streaming accesses).
#include <hip/hip_runtime.h>

#include "../ecmd_launch.h"
#include "ecmd_serving.h"
#include "ecmd_wave.h"

namespace ecmd {

namespace {

constexpr uint32_t kBlock = 256, kWaves = kBlock / 64;

__device__ inline uint32_t popc(uint64_t x) { return (uint32_t)__popcll(x); }

// Exclusive prefix of x over the work-group of NW waves (all threads call it);
// total gets the sum.  scratch: NW entries, free again when it returns.
template <uint32_t NW = kWaves>
__device__ inline uint32_t block_prefix(uint32_t x, uint32_t *scratch, uint32_t &total)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t inc = wave_prefix(x);
    if (lane == 63) scratch[wave] = inc;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (uint32_t w = 0; w < NW; ++w) {
        if (w < wave) before += scratch[w];
        total += scratch[w];
    }
    __syncthreads();
    return before + inc - x;
}

// The bits, word prefixes and count of tile `tile`: set where pick(id).
template <class F>
__device__ inline void mark_tile(const PageBits &B, uint32_t tile, uint32_t *scratch, F pick)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t run = 0;
    // 256 words at a time: the waves make their words' bits, then one prefix
    for (uint32_t w0 = 0; w0 < B.tile_words; w0 += kBlock) {
        const uint32_t words = min(kBlock, B.tile_words - w0);
        __shared__ uint32_t s_count[kBlock];
        for (uint32_t w = wave; w < words; w += kWaves) {
            const uint64_t word = (uint64_t)tile * B.tile_words + w0 + w, id = word * 64 + lane;
            const uint64_t bits = __ballot(id < B.n && pick((uint32_t)id));
            if (lane == 0) {
                B.word[word] = bits;
                s_count[w] = popc(bits);
            }
        }
        __syncthreads();
        const uint32_t mine = threadIdx.x < words ? s_count[threadIdx.x] : 0;
        uint32_t total;
        const uint32_t before = block_prefix(mine, scratch, total);
        if (threadIdx.x < words) B.word_prefix[(uint64_t)tile * B.tile_words + w0 + threadIdx.x] = run + before;
        run += total;
    }
    if (threadIdx.x == 0) B.tile_count[tile] = run;
}

// Prefixes of the tile counts into LDS: prefix[t] set bits before tile t,
// prefix[tiles] all of them.  mine: the count of tile threadIdx.x (or 0), read
// early.  Ends with a barrier.
__device__ inline void tile_prefixes(const PageBits &B, uint32_t *prefix, uint32_t *scratch, uint32_t mine)
{
    uint32_t run = 0;
    for (uint32_t t0 = 0; t0 < B.tiles; t0 += kBlock) {
        const uint32_t t = t0 + threadIdx.x;
        uint32_t total;
        const uint32_t before = block_prefix(t0 == 0 ? mine : t < B.tiles ? B.tile_count[t] : 0, scratch, total);
        if (t < B.tiles) prefix[t] = run + before;
        run += total;
    }
    if (threadIdx.x == 0) prefix[B.tiles] = run;
    __syncthreads();
}

// The id of the set (SET) or clear bit with this rank, which has to exist.
// Sixteen word prefixes are read at once: one wait instead of four.
template <bool SET>
__device__ inline uint32_t select_bit(const PageBits &B, const uint32_t *prefix, uint32_t rank)
{
    // bits of the kind before a place, from the set ones before it
    auto kind = [](uint32_t set, uint64_t places) { return SET ? set : (uint32_t)places - set; };
    uint32_t lo = 0, hi = B.tiles;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (kind(prefix[mid], (uint64_t)mid * B.tile_words * 64) <= rank) lo = mid;
        else hi = mid;
    }
    const uint64_t w0 = (uint64_t)lo * B.tile_words;
    rank -= kind(prefix[lo], w0 * 64);
    uint32_t a = 0, b = B.tile_words;   // tile_words: 16 times a power of two
    while (b - a > 16) {
        const uint32_t mid = (a + b) / 2;
        if (kind(B.word_prefix[w0 + mid], mid * 64) <= rank) a = mid;
        else b = mid;
    }
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = ((const u32x4 *)(B.word_prefix + w0 + a))[k];
    uint32_t in = 0, before = kind(p[0][0], a * 64);
#pragma unroll
    for (int k = 1; k < 16; ++k) {
        const uint32_t x = kind(p[k / 4][k % 4], (a + k) * 64);
        if (x <= rank) {
            in = k;
            before = x;
        }
    }
    rank -= before;
    a += in;
    const uint64_t word = SET ? B.word[w0 + a] : ~B.word[w0 + a];
    uint32_t at = 0;
#pragma unroll
    for (uint32_t half = 32; half; half /= 2) {
        const uint32_t low = popc((word >> at) & ((uint64_t(1) << half) - 1));
        if (rank >= low) {
            rank -= low;
            at += half;
        }
    }
    return (uint32_t)(w0 + a) * 64 + at;
}

// ---------------------------------------------------------------------------
// Assign.

struct RowPlan {
    bool has;
    uint32_t parent, old, length, len_new, keep, total;
};
__device__ inline RowPlan plan_row(const AssignArgs &A, uint32_t r)
{
    RowPlan p;
    const uint32_t most = A.cols * A.page;
    const int32_t parent = A.parent[r * A.parent_s];
    p.has = parent >= 0 && (uint32_t)parent < A.rows;
    p.parent = p.has ? (uint32_t)parent : r;
    p.old = min((uint32_t)max(A.lens[r * A.lens_s], 0), most);
    p.length = !p.has ? 0 : min((uint32_t)max(A.lens[p.parent * A.lens_s], 0), most);
    p.len_new = min(p.length + (uint32_t)max(A.add[r * A.add_s], 0), most);   // both below 2^31
    p.keep = p.has && p.parent == r ? A.by_page.div(p.length + A.page - 1) : A.by_page.div(p.length);
    p.total = A.by_page.div(p.len_new + A.page - 1);
    return p;
}

// First launch: a work-group per tile of pages (the free ones' bits, the copy of
// the counts), then one per 256 rows (pages wanted).
__global__ __launch_bounds__(kBlock) void k_assign_count(const AssignArgs A)
{
    __shared__ uint32_t scratch[kWaves];
    if (blockIdx.x < A.bits.tiles) {
        mark_tile(A.bits, blockIdx.x, scratch, [&](uint32_t id) {
            const int32_t c = A.refs[id * A.refs_s];
            A.refs_out[id * A.refs_out_s] = c;
            return c == 0;
        });
        return;
    }
    const uint32_t g = blockIdx.x - A.bits.tiles, r = g * kBlock + threadIdx.x;
    uint32_t want = 0, total;
    if (r < A.rows) {
        const RowPlan p = plan_row(A, r);
        want = p.total - p.keep;
    }
    const uint32_t before = block_prefix(want, scratch, total);
    if (r < A.rows) A.want[r] = before;
    if (threadIdx.x == 0) A.want_group[g] = total;
}

// Column c of row r: its page, what that changes in the counts (add(id, by)), and
// the copy of a parent's partial page.
template <class F>
__device__ inline void assign_entry(const AssignArgs &A, const PageBits &B, const uint32_t *prefix, const RowPlan &p,
                                    uint32_t r, uint32_t c, uint32_t base, uint32_t have, F add)
{
    const uint32_t held = A.by_page.div(p.old + A.page - 1), last = A.by_page.div(p.length);
    const int32_t *own = A.pages + (int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1];
    const int32_t *from = A.pages + (int64_t)p.parent * A.pages_s[0] + (int64_t)c * A.pages_s[1];
    int32_t was = -1, now = -1;
    if (c < held) was = *own;
    if (was < 0 || (uint32_t)was >= B.n) was = -1;
    if (c < p.keep) {
        now = *from;
        if (now < 0 || (uint32_t)now >= B.n) now = -1;
    } else if (c < p.total) {
        const uint32_t rank = base + (c - p.keep);
        if (rank < have) now = (int32_t)select_bit<true>(B, prefix, rank);
    }
    A.pages_out[(int64_t)r * A.pages_out_s[0] + (int64_t)c * A.pages_out_s[1]] = now;
    if (was != now) {
        if (was >= 0) add(was, -1);
        if (now >= 0) add(now, 1);
    }
    if (c == last && p.has && p.parent != r && p.length != last * A.page) {
        const int32_t a = *from;
        const bool copy = a >= 0 && (uint32_t)a < B.n && now >= 0;
        A.src[r * A.src_s] = copy ? a : -1;
        A.dst[r * A.dst_s] = copy ? now : -1;
    }
}

// Sums over the work-group; scratch: 2 kWaves entries.
__device__ inline void block_sums(uint32_t &x, uint32_t &y, uint32_t *scratch)
{
    x = wave_sum(x);
    y = wave_sum(y);
    if ((threadIdx.x & 63) == 0) {
        scratch[threadIdx.x >> 6] = x;
        scratch[kWaves + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = y = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
        x += scratch[w];
        y += scratch[kWaves + w];
    }
}

// Second launch: a work-group per row.  What it waits for is the chain of
// loads, so the first launch's counts are asked for before the row's own plan is
// made of three dependent loads.
__global__ __launch_bounds__(kBlock) void k_assign(const AssignArgs A)
{
    __shared__ uint32_t prefix[kMaxPageTiles + 1], scratch[kWaves], scratch2[2 * kWaves];
    const uint32_t r = blockIdx.x;
    uint32_t count = threadIdx.x < A.bits.tiles ? A.bits.tile_count[threadIdx.x] : 0;
    uint32_t mine = 0, all = 0;
    for (uint32_t g = threadIdx.x; g < A.row_groups; g += kBlock) {
        const uint32_t w = A.want_group[g];
        all += w;
        if (g < r / kBlock) mine += w;
    }
    RowPlan p{};
    uint32_t base = 0;
    if (r < A.rows) {
        base = A.want[r];
        p = plan_row(A, r);
    }
    const uint32_t fresh = p.total - p.keep;
    uint32_t have = 0;
    if (fresh || r == 0) {   // the same for the whole work-group
        tile_prefixes(A.bits, prefix, scratch, count);
        have = prefix[A.bits.tiles];
        block_sums(mine, all, scratch2);
        base += mine;
        if (r == 0 && threadIdx.x == 0) {
            A.stats[0] = (int32_t)all;
            A.stats[A.stats_s] = (int32_t)min(all, have);
        }
    }
    if (r >= A.rows) return;   // no rows at all
    const bool partial = p.has && p.parent != r && p.length != A.by_page.div(p.length) * A.page;
    if (threadIdx.x == 0) {
        A.lens_out[r * A.lens_out_s] = (int32_t)p.len_new;
        if (!partial) A.src[r * A.src_s] = A.dst[r * A.dst_s] = -1;
    }
    for (uint32_t c = threadIdx.x; c < A.cols; c += kBlock)
        assign_entry(A, A.bits, prefix, p, r, c, base, have,
                     [&](int32_t id, int32_t by) { atomicAdd(&A.refs_out[id * A.refs_out_s], by); });
}

// ---------------------------------------------------------------------------
// Compact.

__global__ __launch_bounds__(kBlock) void k_compact_mark(const CompactArgs A)
{
    __shared__ uint32_t scratch[kWaves];
    mark_tile(A.bits, blockIdx.x, scratch, [&](uint32_t id) { return A.refs[id * A.refs_s] > 0; });
}

// Set bits before id (id <= n).
__device__ inline uint32_t rank_bit(const PageBits &B, const uint32_t *prefix, uint32_t id)
{
    const uint32_t w = id / 64, tile = w >> B.tile_shift;
    if (tile >= B.tiles) return prefix[B.tiles];
    return prefix[tile] + B.word_prefix[w] + popc(B.word[w] & ((uint64_t(1) << (id % 64)) - 1));
}

// Second launch, all of the rest from the bits: work-groups for the ids, then for
// the table's entries.  With `live` set bits in all, `kept` of them before id live,
// the i-th move goes from the set bit of rank kept + i to the clear bit of rank i.
__global__ __launch_bounds__(kBlock) void k_compact(const CompactArgs A, uint32_t id_groups)
{
    __shared__ uint32_t prefix[kMaxPageTiles + 1], scratch[kWaves];
    const uint32_t count = threadIdx.x < A.bits.tiles ? A.bits.tile_count[threadIdx.x] : 0;
    const bool entries = blockIdx.x >= id_groups;
    const uint32_t i = (blockIdx.x - (entries ? id_groups : 0)) * kBlock + threadIdx.x;
    // what the bits are asked for, read before they are
    const bool here = entries ? i < A.rows * A.cols : i < A.bits.n;
    const uint32_t r = entries ? A.by_cols.div(i) : 0, c = i - r * A.cols;
    int32_t id = (int32_t)i, refs = 0;
    if (entries && here) id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
    if (!entries && here) refs = A.refs[i * A.refs_s];
    const bool valid = here && id >= 0 && (uint32_t)id < A.bits.n;
    const uint64_t word = valid ? A.bits.word[id / 64] : 0;
    const uint32_t word_prefix = valid ? A.bits.word_prefix[id / 64] : 0;
    tile_prefixes(A.bits, prefix, scratch, count);
    const uint32_t live = prefix[A.bits.tiles], kept = rank_bit(A.bits, prefix, live), moves = live - kept;
    const bool set = valid && (word >> (id % 64) & 1);
    const uint32_t rank = valid ? prefix[id / 64 >> A.bits.tile_shift] + word_prefix +
                                      popc(word & ((uint64_t(1) << (id % 64)) - 1))
                                : 0;
    if (entries) {
        if (!here) return;
        int32_t now = -1;
        if (set) now = (uint32_t)id < live ? id : (int32_t)select_bit<false>(A.bits, prefix, rank - kept);
        A.pages_out[(int64_t)r * A.pages_out_s[0] + (int64_t)c * A.pages_out_s[1]] = now;
        return;
    }
    if (i >= moves && i < A.capacity) {
        A.src[i * A.src_s] = -1;
        A.dst[i * A.dst_s] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        A.stats[0] = (int32_t)live;
        A.stats[A.stats_s] = (int32_t)moves;
    }
    if (!here) return;
    if (i >= live) {
        refs = 0;
    } else if (!set) {   // a page comes here
        const uint32_t move = i - rank, from = select_bit<true>(A.bits, prefix, kept + move);
        A.src[move * A.src_s] = (int32_t)from;
        A.dst[move * A.dst_s] = (int32_t)i;
        refs = A.refs[from * A.refs_s];
    }
    A.refs_out[i * A.refs_out_s] = refs;
}

// ---------------------------------------------------------------------------
// Small problems in one launch: one work-group, bits and counts in LDS.  Its time
// grows with the entries and, less, the pages; two launches and their workspace are
// the caller's 9.8 us to assign and 9.2 to compact at every such size.  Measured, a
// call among others, 1000 pages and 4096: 2560 entries 8.0 and 8.3 us to assign, 6.4
// and 8.1 to compact; 3200 entries 8.0 and 8.7, 7.9 and 9.2; 4096 entries 9.1 and
// 10.4, 8.7 and 10.5; 12800 entries 18.5 and 20.4, 22.3 and 23.5.  So the limit is
// 3200 entries, where neither is slower.

constexpr uint32_t kSmallBlock = kSmallRows, kSmallWords = kSmallPages / 64;

struct SmallBits {
    uint64_t word[kSmallWords];
    __attribute__((aligned(16))) uint32_t word_prefix[kSmallWords];
    uint32_t prefix[2], scratch[kSmallBlock / 64];
};

// The counts into LDS and the bits of those that pick(count) says.
template <class F>
__device__ inline PageBits small_bits(SmallBits &S, int32_t *counts, const int32_t *refs, int64_t stride, uint32_t n, F pick)
{
    for (uint32_t id = threadIdx.x; id < kSmallPages; id += kSmallBlock) {   // whole waves
        int32_t c = 0;
        if (id < n) counts[id] = c = refs[id * stride];
        const uint64_t bits = __ballot(id < n && pick(c));
        if (threadIdx.x % 64 == 0) S.word[id / 64] = bits;
    }
    __syncthreads();
    const uint32_t w = threadIdx.x;
    uint32_t total;
    const uint32_t before = block_prefix<kSmallBlock / 64>(w < kSmallWords ? popc(S.word[w]) : 0, S.scratch, total);
    if (w < kSmallWords) S.word_prefix[w] = before;
    if (w == 0) {
        S.prefix[0] = 0;
        S.prefix[1] = total;
    }
    __syncthreads();
    PageBits B{};
    B.word = S.word;
    B.word_prefix = S.word_prefix;
    B.n = n;
    B.tiles = 1;
    B.tile_words = kSmallWords;
    while ((1u << B.tile_shift) < kSmallWords) ++B.tile_shift;
    return B;
}

__global__ __launch_bounds__(kSmallBlock) void k_assign_small(const AssignArgs A)
{
    __shared__ SmallBits S;
    __shared__ int32_t counts[kSmallPages];
    __shared__ uint32_t s_base[kSmallBlock];
    __shared__ RowPlan s_plan[kSmallBlock];
    const uint32_t n = A.bits.n, tid = threadIdx.x;
    RowPlan p{};
    if (tid < A.rows) p = plan_row(A, tid);
    const PageBits B = small_bits(S, counts, A.refs, A.refs_s, n, [](int32_t c) { return c == 0; });
    const uint32_t have = S.prefix[1];
    uint32_t wanted;
    const uint32_t base = block_prefix<kSmallBlock / 64>(p.total - p.keep, S.scratch, wanted);
    if (tid < A.rows) {
        s_plan[tid] = p;
        s_base[tid] = base;
        A.lens_out[tid * A.lens_out_s] = (int32_t)p.len_new;
        const bool partial = p.has && p.parent != tid && p.length != A.by_page.div(p.length) * A.page;
        if (!partial) A.src[tid * A.src_s] = A.dst[tid * A.dst_s] = -1;
    }
    if (tid == 0) {
        A.stats[0] = (int32_t)wanted;
        A.stats[A.stats_s] = (int32_t)min(wanted, have);
    }
    __syncthreads();
#pragma unroll 4
    for (uint32_t i = tid; i < A.rows * A.cols; i += kSmallBlock) {
        const uint32_t r = A.by_cols.div(i), c = i - r * A.cols;
        const RowPlan &P = s_plan[r];
        assign_entry(A, B, S.prefix, P, r, c, s_base[r], have, [&](int32_t id, int32_t by) { atomicAdd(&counts[id], by); });
    }
    __syncthreads();
    for (uint32_t id = tid; id < n; id += kSmallBlock) A.refs_out[id * A.refs_out_s] = counts[id];
}

__global__ __launch_bounds__(kSmallBlock) void k_compact_small(const CompactArgs A)
{
    __shared__ SmallBits S;
    __shared__ int32_t counts[kSmallPages];
    const uint32_t n = A.bits.n, tid = threadIdx.x;
    const PageBits B = small_bits(S, counts, A.refs, A.refs_s, n, [](int32_t c) { return c > 0; });
    const uint32_t live = S.prefix[1], kept = rank_bit(B, S.prefix, live), moves = live - kept;
    if (tid == 0) {
        A.stats[0] = (int32_t)live;
        A.stats[A.stats_s] = (int32_t)moves;
    }
    for (uint32_t i = tid; i < max(n, A.capacity); i += kSmallBlock) {
        if (i >= moves && i < A.capacity) {
            A.src[i * A.src_s] = -1;
            A.dst[i * A.dst_s] = -1;
        }
        if (i >= n) continue;
        int32_t refs = i < live ? counts[i] : 0;
        if (i < live && !(B.word[i / 64] >> (i % 64) & 1)) {   // a page comes here
            const uint32_t move = i - rank_bit(B, S.prefix, i), from = select_bit<true>(B, S.prefix, kept + move);
            A.src[move * A.src_s] = (int32_t)from;
            A.dst[move * A.dst_s] = (int32_t)i;
            refs = counts[from];
        }
        A.refs_out[i * A.refs_out_s] = refs;
    }
#pragma unroll 4
    for (uint32_t i = tid; i < A.rows * A.cols; i += kSmallBlock) {
        const uint32_t r = A.by_cols.div(i), c = i - r * A.cols;
        const int32_t id = A.pages[(int64_t)r * A.pages_s[0] + (int64_t)c * A.pages_s[1]];
        int32_t now = -1;
        if (id >= 0 && (uint32_t)id < n && (B.word[id / 64] >> (id % 64) & 1))
            now = (uint32_t)id < live ? id : (int32_t)select_bit<false>(B, S.prefix, rank_bit(B, S.prefix, id) - kept);
        A.pages_out[(int64_t)r * A.pages_out_s[0] + (int64_t)c * A.pages_out_s[1]] = now;
    }
}

// ---------------------------------------------------------------------------
// Copy: a work-group takes one piece of one page (four vectors per work-item,
// all loaded before the first store), or several whole small pages.  HBM bounds
// it.

template <int W>
struct CopyVec;
template <>
struct CopyVec<16> {
    typedef uint32_t V __attribute__((ext_vector_type(4)));
};
template <>
struct CopyVec<8> {
    typedef uint32_t V __attribute__((ext_vector_type(2)));
};
template <>
struct CopyVec<4> {
    typedef uint32_t V;
};
template <>
struct CopyVec<2> {
    typedef uint16_t V;
};

template <int W, bool STREAM, int POOLS>
__global__ __launch_bounds__(kBlock) void k_copy(const CopyBlock<POOLS> A)
{
    typedef typename CopyVec<W>::V V;
    const CopyPool &P = A.pool[blockIdx.y];
    uint32_t pair, first, step;
    if (A.per_group > 1) {
        const uint32_t in = A.by_vecs.div(threadIdx.x);
        if (in >= A.per_group) return;
        pair = blockIdx.x * A.per_group + in;
        first = threadIdx.x - in * A.by_vecs.d;
        step = A.by_vecs.d;
        if (pair >= A.count) return;
    } else {
        pair = A.by_pieces.div(blockIdx.x);
        first = (blockIdx.x - pair * A.pieces) * (4 * kBlock) + threadIdx.x;
        step = kBlock;
    }
    const int32_t a = A.src[pair * A.src_s], b = A.dst[pair * A.dst_s];
    if (a < 0 || b < 0 || (uint32_t)a >= P.n || (uint32_t)b >= P.n) return;
    const char *from = P.base + a * P.page_stride;
    char *to = P.base + b * P.page_stride;
    auto at = [&](uint32_t v) {
        const uint32_t row = P.by_row.div(v);
        return (int64_t)row * P.row_stride + (int64_t)(v - row * P.row_vecs) * W;
    };
    V x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (first + k * step < P.vecs) {
            const V *p = (const V *)(from + at(first + k * step));
            if constexpr (STREAM) x[k] = __builtin_nontemporal_load(p);
            else x[k] = *p;
        }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (first + k * step < P.vecs) {
            V *p = (V *)(to + at(first + k * step));
            if constexpr (STREAM) __builtin_nontemporal_store(x[k], p);
            else *p = x[k];
        }
}

}  // namespace

int launch_assign(const AssignArgs &A, void *stream)
{
    if (A.small)
        return launch_kernel(reinterpret_cast<const void *>(&k_assign_small), dim3(1), dim3(kSmallBlock), 0, stream, A);
    const uint32_t first = A.bits.tiles + A.row_groups;
    if (first) {
        const int rc = launch_kernel(reinterpret_cast<const void *>(&k_assign_count), dim3(first), dim3(kBlock), 0,
                                     stream, A);
        if (rc) return rc;
    }
    return launch_kernel(reinterpret_cast<const void *>(&k_assign), dim3(A.rows ? A.rows : 1), dim3(kBlock), 0, stream,
                         A);
}

int launch_compact(const CompactArgs &A, void *stream)
{
    if (A.small)
        return launch_kernel(reinterpret_cast<const void *>(&k_compact_small), dim3(1), dim3(kSmallBlock), 0, stream, A);
    int rc = 0;
    if (A.bits.tiles)
        rc = launch_kernel(reinterpret_cast<const void *>(&k_compact_mark), dim3(A.bits.tiles), dim3(kBlock), 0, stream,
                           A);
    if (rc) return rc;
    const uint32_t entries = (uint32_t)(((uint64_t)A.rows * A.cols + kBlock - 1) / kBlock);
    const uint64_t ids = A.bits.n > A.capacity ? A.bits.n : A.capacity;
    const uint32_t id_groups = ids ? (uint32_t)((ids + kBlock - 1) / kBlock) : 1;   // one at least, for the counts
    return launch_kernel(reinterpret_cast<const void *>(&k_compact), dim3(id_groups + entries), dim3(kBlock), 0, stream,
                         A, id_groups);
}

template <int POOLS>
static int launch_copy_block(int width, bool past, const CopyBlock<POOLS> &A, uint32_t pools, uint32_t grid, void *stream)
{
    const void *fn = width == 16  ? past ? reinterpret_cast<const void *>(&k_copy<16, true, POOLS>)
                                         : reinterpret_cast<const void *>(&k_copy<16, false, POOLS>)
                     : width == 8 ? reinterpret_cast<const void *>(&k_copy<8, false, POOLS>)
                     : width == 4 ? reinterpret_cast<const void *>(&k_copy<4, false, POOLS>)
                                  : reinterpret_cast<const void *>(&k_copy<2, false, POOLS>);
    return launch_kernel(fn, dim3(grid, pools), dim3(kBlock), 0, stream, A);
}

int launch_copy(int width, bool past, const CopyArgs &A, uint32_t pools, uint32_t grid, void *stream)
{
    if (pools > (uint32_t)kFewPools) return launch_copy_block(width, past, A, pools, grid, stream);
    CopyBlock<kFewPools> B{A.src, A.dst, A.src_s, A.dst_s, A.count, A.per_group, A.pieces, A.by_pieces, A.by_vecs, {}};
    for (uint32_t k = 0; k < pools; ++k) B.pool[k] = A.pool[k];
    return launch_copy_block(width, past, B, pools, grid, stream);
}

}  // namespace ecmd
