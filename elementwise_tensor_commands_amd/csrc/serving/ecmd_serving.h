// ecmd_serving.h -- kernel argument blocks of the serving operators and the
// functions that launch them (internal to the library).
//
// The host (ecmd_serving.cpp, ecmd_serving_cache.cpp) checks every argument and fills a block; a
// launcher picks the kernel instance and enqueues it.  Offsets within a tensor
// are 64-bit throughout.
#pragma once
#include <stdint.h>

namespace ecmd {

// Quotients by a divisor known on the host: n / d for n < 2^31 as
// (mulhi(n, mul) + n) >> shift, the round-up method.  (The Commands' FastDiv
// takes every 32-bit n for one more shift; here the sum stays below 2^32.)
struct Div31 {
    uint32_t mul = 0, shift = 0, d = 1;
    Div31() = default;
    explicit Div31(uint32_t div) : d(div)
    {
        if (div == 0) return;   // the size of something empty: nothing asks for a quotient
        while ((uint64_t(1) << shift) < div) ++shift;
        mul = (uint32_t)((((uint64_t(1) << shift) - div) << 32) / div + 1);
    }
#ifdef __HIPCC__
    __host__ __device__ uint32_t div(uint32_t n) const
    {
        return (uint32_t)(((uint64_t(n) * mul >> 32) + n) >> shift);
    }
#endif
};

enum ServingType { S_F16 = 0, S_BF16 = 1, S_F32 = 2 };

// --- rotary positions ------------------------------------------------------

struct RopeArgs {
    const void *x;
    void *out;
    const int32_t *pos;
    const double *freq;
    int64_t xs[3], os[3];            // element strides of batch, token, head
    int64_t ps[2], fs;               // of pos (batch, token) and freq
    uint32_t tokens, pairs, width;   // b * t, m, d
    uint32_t tb;                     // tokens per work-group
    double mscale;
    int32_t inverse;
    Div31 by_t;                    // token index -> batch
    Div31 by_head_items, by_token_items;
    uint32_t items;                  // per token: heads * head_items
};

struct AppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const int32_t *pos, *row, *pages;
    const double *freq;
    int64_t qs[2], ks[2], vs[2], qos[2];   // token, head
    int64_t kcs[3], vcs[3];                // page, slot, head
    int64_t pos_s, row_s, pages_s[2], fs;
    uint32_t tokens, pairs, d, dv, hq, hk;
    uint32_t rows, cols, n, page;
    uint32_t tb, parts;                    // tokens per work-group; work-groups per token group
    double mscale;
    Div31 by_page, by_parts;
    Div31 by_q, by_k, by_v;                // items of a token
    Div31 by_qk_head, by_v_head;           // items of a head
};

// edge: 0 pairs, tails and value rows are whole 16-byte vectors, 1 they are no shorter
// than one, 2 some are; past: go past the caches
int launch_rope(int type, int layout, int edge, bool past, const RopeArgs &A, uint32_t grid, uint32_t lds, void *stream);
int launch_append(int type, int layout, int edge, bool past, const AppendArgs &A, uint32_t grid, uint32_t lds, void *stream);

// --- paged attention -------------------------------------------------------

struct AttnArgs {
    const void *q, *k, *v;
    const int32_t *pages, *lens;
    void *out;
    float *lse;                            // may be null
    float *acc;                            // workspace: [runs + b, hq, dv] sums
    float *ml;                             // workspace: [runs + b, hq] (maximum, sum) pairs
    int64_t qs[2], os[2], ls[2];           // batch, head
    int64_t kcs[3], vcs[3];                // BYTE strides of page, slot, head
    int64_t pages_s[3], lens_s[2];         // batch, column, kv head; batch, kv head
    // Tables of every kv head: each of a sequence's `apart` kv heads is a row of its
    // own, with one kv head (b = sequences * apart, hq = group, hk = 1).  Otherwise 1.
    uint32_t apart, apart_tables;
    uint32_t b, hq, hk, d, dv, group, head_tiles;
    uint32_t n, page, cols;
    uint32_t window;
    uint32_t direct;                       // 1: a work-group to a row and head, no join
    uint32_t head_shift;                   // with much to read, 2^this waves of a work-group take a head each
    uint32_t runs, runs_much, runs_most;   // runs of positions for each head; the larger one
    uint32_t runs_whole;                   // rows up to which they may all be runs (0: too few work-groups)
    uint32_t grid;
    uint32_t stream;                       // 1: larger than the last-level cache
    uint32_t join;                         // 0, 1, 2: few, many, very many segments to a row
    float scale_log2;                      // scale * log2(e)
    Div31 by_page;
    Div31 by_heads, by_heads_much;         // work-groups of eight runs: 8 heads; 8 heads >> head_shift
    Div31 by_tiles;                        // head_tiles
    Div31 by_runs, by_runs_much;
    Div31 by_apart;
};

// Positions are dealt to work-groups in steps of this many: a tile for each of
// four waves, at 16 bits.  (Half of it for binary32: one row of 19296 positions 26
// us instead of 29, nine rows of up to 1000 20 instead of 18, as runs then end
// within rows.)
constexpr uint32_t kAttnStep = 128;
// Steps of all heads that count as much to read (see deal_steps).
constexpr uint32_t kAttnMuch = 6144;

constexpr uint32_t kAttnMaxRuns = 1024;
constexpr uint32_t kAttnMaxRows = 2048;    // rows whose prefixes fit LDS; more go direct

int launch_attention_f16(const AttnArgs &A, void *stream);
int launch_attention_bf16(const AttnArgs &A, void *stream);
int launch_attention_f32(const AttnArgs &A, void *stream);
int launch_attention_join_f16(const AttnArgs &A, void *stream);
int launch_attention_join_bf16(const AttnArgs &A, void *stream);
int launch_attention_join_f32(const AttnArgs &A, void *stream);

// --- pages -----------------------------------------------------------------

// One bit per page id (free, or live), 64 ids a word, words grouped into at
// most kMaxPageTiles tiles: a bit's rank is its tile's prefix, its word's
// prefix within the tile and a population count.
constexpr uint32_t kMaxPageTiles = 1024;
struct PageBits {
    uint64_t *word;          // [tiles * tile_words]
    uint32_t *word_prefix;   // [tiles * tile_words] set bits before the word within its tile
    uint32_t *tile_count;    // [tiles]
    uint32_t n, tiles, tile_words, tile_shift;   // tile_words = 1 << tile_shift
};

// What one work-group does alone, in one launch and without a workspace.
constexpr uint32_t kSmallPages = 4096, kSmallRows = 1024, kSmallEntries = 3200;

struct AssignArgs {
    const int32_t *pages, *lens, *refs, *parent, *add;
    int32_t *pages_out, *lens_out, *refs_out, *src, *dst, *stats;
    int64_t pages_s[2], pages_out_s[2];
    int64_t lens_s, refs_s, parent_s, add_s, lens_out_s, refs_out_s, src_s, dst_s, stats_s;
    uint32_t rows, cols, page;
    PageBits bits;
    uint32_t *want;          // workspace: [rows] pages wanted before the row within its group of 256
    uint32_t *want_group;    // workspace: [groups] pages wanted by the group
    uint32_t row_groups, small;
    Div31 by_page, by_cols;
};

struct CompactArgs {
    const int32_t *pages, *refs;
    int32_t *pages_out, *refs_out, *src, *dst, *stats;
    int64_t pages_s[2], pages_out_s[2];
    int64_t refs_s, refs_out_s, src_s, dst_s, stats_s;
    uint32_t rows, cols, capacity, small;
    PageBits bits;
    Div31 by_cols;
};

constexpr int kCopyPools = 24;   // of one launch
constexpr int kFewPools = 4;
struct CopyPool {
    char *base;
    int64_t page_stride, row_stride;   // bytes
    uint32_t n, vecs, row_vecs;        // pages; vectors per page and per row of a page
    uint32_t pad;
    Div31 by_row;
};
// One launch's argument block is copied for the device each time: the few pools of
// one layer take a short one (a call 4.1 us instead of 5.1).
template <int POOLS>
struct CopyBlock {
    const int32_t *src, *dst;
    int64_t src_s, dst_s;
    uint32_t count, per_group;         // pairs; pairs per work-group (small pages) or 1
    uint32_t pieces;                   // work-groups per pair
    Div31 by_pieces, by_vecs;          // by_vecs: vectors per page, where per_group > 1
    CopyPool pool[POOLS];
};
typedef CopyBlock<kCopyPools> CopyArgs;

int launch_assign(const AssignArgs &A, void *stream);
int launch_compact(const CompactArgs &A, void *stream);
// width: bytes of one vector (16, 8, 4 or 2); past: go past the caches
int launch_copy(int width, bool past, const CopyArgs &A, uint32_t pools, uint32_t grid, void *stream);

// --- trees of drafted tokens -------------------------------------------------

constexpr uint32_t kMaxTree = 256;   // tokens of a tree
constexpr uint32_t kTreeMaxRows = 1024;   // rows whose prefixes fit LDS beside the tree; more go direct

struct TreeArgs {
    const void *q, *k, *v;
    const int32_t *pages, *lens, *parent;
    void *out;
    float *lse;                            // may be null
    float *acc;                            // workspace: [runs + b, hk * m, dv] sums
    float *ml;                             // workspace: [runs + b, hk * m] (maximum, sum) pairs; sum < 0: padding
    int64_t qs[3], os[3], ls[3];           // batch, token, head
    int64_t kcs[3], vcs[3];                // BYTE strides of page, slot, head
    int64_t pages_s[2], lens_s, parent_s[2];
    uint32_t b, t, hq, hk, d, dv, group;
    uint32_t m;                            // query vectors of a kv head: t * group, token by token
    uint32_t tiles;                        // 16 query vectors of a wave where tiles are staged (1 or 2); 0: they are not
    uint32_t join_shift, join_turn;        // the join: 2^shift work-items to a query vector; vectors of a work-group
    uint32_t q_blocks, q_shift;            // work-groups that share them; 2^q_shift waves of one take apart (not staged)
    uint32_t n, page, cols, window;
    uint32_t direct;                       // 1: a work-group to a row, kv head and block, no join
    uint32_t runs, runs_whole, grid;       // as in AttnArgs
    float scale_log2;                      // |scale| * log2(e)
    uint32_t q_flip;                       // sign bits to flip in q: the scale is negative
    Div31 by_page, by_units, by_blocks, by_group, by_runs, by_vectors;   // by_units: 8 * hk * q_blocks
};

int launch_tree_f16(const TreeArgs &A, void *stream);
int launch_tree_bf16(const TreeArgs &A, void *stream);
int launch_tree_f32(const TreeArgs &A, void *stream);
int launch_tree_join(int type, const TreeArgs &A, void *stream);

struct AcceptArgs {
    const int32_t *tokens, *parent, *next, *lens;
    int32_t *path, *lens_out, *last;
    int64_t tokens_s[2], parent_s[2], next_s[2], path_s[2];
    int64_t lens_s, lens_out_s, last_s;
    uint32_t rows, t;
};
int launch_accept(const AcceptArgs &A, void *stream);

constexpr int kMovePools = 24, kMoveFew = 4;   // of one launch
struct MovePool {
    char *base;
    int64_t page_stride, slot_stride, head_stride;   // bytes
    uint32_t n, head_vecs;
    Div31 by_head;                                   // vectors of a head
};
template <int POOLS>
struct MoveBlock {
    const int32_t *pages, *lens, *path;
    int64_t pages_s[2], lens_s, path_s[2];
    uint32_t rows, cols, t, page;
    uint32_t vecs, pieces;                           // vectors of a slot; work-groups that share them
    Div31 by_page, by_pieces;
    MovePool pool[POOLS];
};
typedef MoveBlock<kMovePools> MoveArgs;
// width: bytes of one vector (16, 8, 4 or 2)
int launch_move(int width, const MoveArgs &A, uint32_t pools, void *stream);

// --- pages worth reading or keeping ----------------------------------------

struct BoundsArgs {
    const void *k;
    void *bounds;
    const int32_t *pages, *lens, *since;
    int64_t kcs[3];                        // BYTE strides of page, slot, head
    int64_t bs[3];                         // BYTE strides of page, head, least/largest
    int64_t pages_s[2], lens_s, since_s;
    uint32_t rows, cols, n, page, hk, d;
    uint32_t head_items, items;            // 16-byte pieces of a head and of a slot
    uint32_t many, parts;                  // columns of a work-group's turn; or its turns of a column (many = 1)
    uint32_t groups;                       // work-groups of a row
    Div31 by_page, by_items, by_head, by_many, by_parts, by_groups;
};
int launch_bounds(int type, const BoundsArgs &A, void *stream);

struct SelectArgs {
    const void *q, *bounds;
    const int32_t *pages, *lens;
    int32_t *pages_out, *lens_out;
    uint64_t *keys;                        // workspace: [b, hk, cols]
    int64_t qs[2];                         // BYTE strides of batch, head
    int64_t bs[3];                         // BYTE strides of page, head, least/largest
    int64_t pages_s[2], lens_s, pages_out_s[3], lens_out_s[2];
    uint32_t b, hk, group, d, n, cols, page, take, first, last;
    uint32_t groups;                       // work-groups that score a row and kv head
    Div31 by_page, by_hk, by_groups;
};
int launch_select(int type, const SelectArgs &A, void *stream);

struct MassArgs {
    const void *q, *k;
    const int32_t *pages, *lens;
    const float *lse, *mass;
    float *out;
    int64_t qs[2], kcs[3];                 // BYTE strides of batch, head; of page, slot, head
    int64_t pages_s[2], lens_s, lse_s[2], mass_s[2], out_s[2];
    uint32_t b, hk, group, d, n, cols, page, window;
    uint32_t cols_group, groups;           // columns of a work-group; work-groups of a row
    float scale, decay;
    Div31 by_page, by_groups;
};
int launch_mass_f16(const MassArgs &A, void *stream);
int launch_mass_bf16(const MassArgs &A, void *stream);
int launch_mass_f32(const MassArgs &A, void *stream);
constexpr uint32_t kMassKeys = 256;        // positions of a work-group at a time

struct EvictArgs {
    const int32_t *pages, *lens, *refs, *budget;
    const float *mass;
    int32_t *pages_out, *refs_out, *count;
    int64_t pages_s[2], mass_s[2], pages_out_s[2];
    int64_t lens_s, refs_s, budget_s, refs_out_s, count_s;
    uint32_t rows, cols, n, page, first, last;
    uint32_t copy;                         // 1: refs_out is not refs
    Div31 by_page;
};
int launch_evict(const EvictArgs &A, void *stream);

}  // namespace ecmd
