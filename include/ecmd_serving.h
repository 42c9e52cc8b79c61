/*
 * ecmd_serving.h -- C ABI of the serving operators on AMD Instinct MI355X
 * (gfx950): rotary positions, rotary positions with the write into a paged
 * key-value cache, attention of one new token over that cache, and the
 * bookkeeping of the cache's pages.  They run beside Commands (ecmd.h) on the
 * caller's stream and share the library's conventions:
 *
 *   - a tensor is a cmd_arg: kind CMD_ARG_TENSOR, dtype, device pointer, sizes
 *     and element strides of its rank (the unused entries are not read);
 *   - every status except CMD_E_LAUNCH is returned before any HIP call, and no
 *     GPU work is submitted after a failed check; calls are asynchronous;
 *   - strides are >= 0; an input may have stride 0 (broadcast); an output must
 *     be one-to-one, each of its dimensions, by ascending stride, stepping past
 *     the smaller ones; an output overlaps no other argument unless the call
 *     says so (then: the identical view);
 *   - the elements of a head (the last dimension of x, q, k, v, the caches and
 *     their outputs, where it has more than one) are neighbours: stride 1, else
 *     CMD_E_STRIDE.  Every other dimension, and all of the tables, lse and the
 *     pools of cmd_page_copy, may have any strides that the call does not exclude;
 *   - the library allocates no device memory: calls that need scratch memory
 *     take a workspace (16-byte aligned, apart from every argument; its contents
 *     need no preparation and mean nothing afterwards), sized by the matching
 *     *_workspace call;
 *   - what one launch cannot hold is refused with CMD_E_LIMIT: 2^24 work-groups, of
 *     a row and 16 query heads in attention, of a row in cmd_page_assign, of 256
 *     entries and ids in cmd_page_compact, of 16 KiB of a page in cmd_page_copy;
 *   - cmd_last_error(NULL) describes the last failure on this thread.
 *
 * What the data say -- positions, row numbers, page ids, lengths, reference
 * counts -- cannot be checked on the host; every kernel checks it and treats
 * what lies outside its range as documented below, so no value of theirs makes
 * a kernel read or write outside the tensors.
 *
 * The cache: k_cache [N, page, kv heads, d] and v_cache [N, page, kv heads, dv]
 * are N pages of `page` slots.  A page table row pages[r, 0..P) names the pages
 * of sequence r: position p lies in slot p % page of page pages[r, p / page].
 * An id outside 0 .. N - 1 is a hole.  Any strides but the last: a cache laid
 * out [N, kv heads, page, d] is passed as its permuted view.
 */
#ifndef ECMD_SERVING_H
#define ECMD_SERVING_H

#include "ecmd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* binary64, the type of the rotary frequency table only (no Command dtype). */
#define CMD_F64 5

/* Which elements of a head form the pairs of a rotary part of width r = 2 m. */
#define CMD_ROPE_HALF 0        /* pair i: elements i and m + i */
#define CMD_ROPE_INTERLEAVED 1 /* pair i: elements 2 i and 2 i + 1 */

/* flags of every call below */
#define CMD_CHECK_ONLY 1 /* check the arguments and return; makes no HIP call */

/* Rotary positions.  args: x [b, t, h, d], pos [b, t] int32, freq [m] binary64
 * (2 m <= d), out [b, t, h, d]; x and out of one dtype f16, bf16 or f32; out
 * may be the identical view as x.  With the angle w = pos[b, t] * freq[i]
 * (rounded once to binary64, |w| < 2^40), c = mscale cos w, s = mscale sin w,
 * pair i (u, v) of every head becomes
 *      forward  (u c - v s,  v c + u s)
 *      inverse  (u c + v s,  v c - u s)     the transpose: the gradient's map
 * c and s are rounded to binary32, products and sums are binary32 (each rounds
 * on its own), the result rounds once to the dtype.  Elements 2 m .. d - 1 are
 * copied. */
int cmd_rope(const cmd_arg args[4], int32_t layout, double mscale, int32_t inverse, int32_t flags, void *hip_stream);

/* Rotary positions of T packed tokens and the write into the cache.  args:
 *   0 q [T, hq, d]   1 k [T, hk, d]   2 v [T, hk, dv]   3 pos [T] int32   4 row [T] int32
 *   5 pages [R, P] int32   6 freq [m] binary64   7 q_out [T, hq, d]
 *   8 k_cache [N, page, hk, d]   9 v_cache [N, page, hk, dv]
 * All but pos, row, pages and freq of one dtype f16, bf16 or f32; q_out may be
 * the identical view as q.  Every token's q is rotated into q_out; k rotated
 * and v as it is go to position pos[t] of sequence row[t].  A token whose row
 * or position is outside the table, or whose page is a hole, is padding: its
 * q_out is written, the cache is not.  After two tokens of one call at one slot
 * each element there is one or the other's. */
int cmd_rope_append(const cmd_arg args[10], int32_t layout, double mscale, int32_t flags, void *hip_stream);

/* Attention of one new token per sequence over the paged cache.  args:
 *   0 q [B, hq, d]   1 k_cache [N, page, hk, d]   2 v_cache [N, page, hk, dv]
 *   3 pages [B, P] int32   4 lens [B] int32   5 out [B, hq, dv]
 *   6 lse [B, hq] f32, or kind 0: not wanted
 * q, the caches and out of one dtype f16, bf16 or f32; hq a multiple of hk
 * (query head h reads kv head h / (hq / hk)); d, dv <= 256.  Row r attends to
 * the positions x with  x < min(lens[r], P * page),  x >= lens[r] - window if
 * window > 0, and no hole under them:
 *      out = sum_x softmax_x(scale q . k_x) v_x,   lse = log sum_x exp(scale q . k_x)
 * Scores, weights, sums and softmax statistics are binary32, but for f16 a weight
 * meets the values held to within 2^-22 of itself or 2^-47 of its row's largest.
 * A row that attends to nothing gets out 0 and lse -inf.  What slots hold that no
 * row attends to is of no account (NaN included); an infinite value that is
 * attended to with a weight that is not 0 in binary32 makes its column infinite. */
int cmd_paged_attention(const cmd_arg args[7], float scale, int32_t window, void *workspace,
                        int64_t workspace_bytes, int32_t flags, void *hip_stream);
/* Bytes of workspace that call needs (0: none), or a negative status. */
int64_t cmd_paged_attention_workspace(const cmd_arg args[7], int32_t window);

/* One step of a decode loop in the page tables: every sequence takes over its
 * parent's state (itself, another sequence: a fork, or none: it starts empty)
 * and grows.  args:
 *   0 pages [R, P] int32   1 lens [R] int32   2 refs [N] int32   3 parent [R] int32   4 add [R] int32
 *   5 pages_out [R, P]   6 lens_out [R]   7 refs_out [N]   8 src [R]   9 dst [R]   10 stats [2]   (all int32)
 * refs[i] counts the table entries that name page i; a page with count 0 is
 * free.  refs_out may be the identical view as refs.  For row r with parent p:
 * length = lens[p] (0 without a parent, i.e. p outside 0 .. R - 1), new length
 * lens_out = min(length + max(add, 0), P * page).  The parent's full pages are
 * kept (shared); its partial last page too if p = r, else the row gets a page
 * of its own and (src[r], dst[r]) = (the parent's page, the own page) asks for
 * the copy that cmd_page_copy makes; src and dst are -1 where there is none.
 * New pages are the free ones in ascending order, given row by row and column by
 * column; when they run out the entries are -1.  A page that loses its last
 * reference in this call is free for the next one.  Columns past the new length
 * are -1.  stats = (pages wanted, pages given). */
int cmd_page_assign(const cmd_arg args[11], int32_t page, void *workspace, int64_t workspace_bytes, int32_t flags,
                    void *hip_stream);
int64_t cmd_page_assign_workspace(const cmd_arg args[11], int32_t page);

/* Pack the live pages (refs > 0) into ids 0 .. live - 1.  args:
 *   0 pages [R, P]   1 refs [N]   2 pages_out [R, P]   3 refs_out [N]   4 src [C]   5 dst [C]   6 stats [2]
 * all int32, C >= N / 2 (rounded down); pages_out may be the identical view as
 * pages.  The live pages with ids >= live move, in ascending order, to the free ids below live, in
 * ascending order: pairs (src[i], dst[i]) for cmd_page_copy, then -1.  pages_out
 * and refs_out are the table and counts after the move (entries that name no
 * live page become -1; the counts past live are 0).  stats = (live, moves). */
int cmd_page_compact(const cmd_arg args[7], void *workspace, int64_t workspace_bytes, int32_t flags,
                     void *hip_stream);
int64_t cmd_page_compact_workspace(const cmd_arg args[7]);

/* Copy page src[i] to page dst[i] in each of npools pools [N_k, page, heads, d] (rank 4,
 * any dtype of 2 or 4 bytes; each pool its own sizes), i = 0 .. C - 1.  Pairs with
 * either id outside a pool are skipped there.  No dst may appear twice or as
 * a src.  A page's elements lie one-to-one, in any order of strides, as rows of
 * neighbours at one distance, as a slice of one of a dense page's dimensions
 * has them; else CMD_E_STRIDE. */
int cmd_page_copy(const cmd_arg *pools, int32_t npools, const cmd_arg *src, const cmd_arg *dst, int32_t flags,
                  void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* ECMD_SERVING_H */
