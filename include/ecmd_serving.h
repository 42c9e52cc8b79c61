/*
 * ecmd_serving.h -- C ABI of the serving operators on AMD Instinct MI355X
 * (gfx950): rotary positions, rotary positions with the write into a paged
 * key-value cache, attention of one new token or of a tree of drafted tokens over
 * that cache, the choice of pages worth reading or worth keeping, and the
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
 *     a row and 16 query heads in attention, of four query vectors (a token's head)
 *     in cmd_tree_attention, of a row in cmd_page_assign, cmd_tree_accept and
 *     cmd_page_evict, of a row and kv head in cmd_page_select, of 256 entries and ids
 *     in cmd_page_compact, of 16 KiB of a page in cmd_page_copy, of a row and 256
 *     vectors of a slot in cmd_slot_move, of a row and up to 256 positions in
 *     cmd_page_mass;
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

/* The same over a page table of its own for every kv head: pages [B, hk, P] and
 * lens [B, hk] in place of args 3 and 4, as cmd_page_select makes them.  Position x
 * of kv head h is slot x % page of page pages[r, h, x / page]. */
int cmd_paged_attention_heads(const cmd_arg args[7], float scale, int32_t window, void *workspace,
                              int64_t workspace_bytes, int32_t flags, void *hip_stream);
int64_t cmd_paged_attention_heads_workspace(const cmd_arg args[7], int32_t window);

/* Attention for a tree of drafted tokens over the paged cache.  args:
 *   0 q [B, T, hq, d]   1 k_cache [N, page, hk, d]   2 v_cache [N, page, hk, dv]
 *   3 pages [B, P] int32   4 lens [B] int32   5 parent [B, T] int32
 *   6 out [B, T, hq, dv]   7 lse [B, T, hq] f32, or kind 0: not wanted
 * T <= 256; dtypes, heads and widths as in cmd_paged_attention.  lens[r] positions
 * of row r are its context; its token i's key and value lie at position lens[r] + i
 * (see cmd_rope_append), and the token follows token parent[r, i] < i, or the
 * context itself if that is -1.  A token with another parent, or below such a one,
 * is padding, and so are all of a row with a negative length: out 0, lse -inf.  A
 * token attends to the context, to the tokens above it and to itself, of these to
 * the `window` nearest (by steps up the tree, then back in the context) if window >
 * 0; never to holes or to positions past the table:
 *      out = sum_x softmax_x(scale q . k_x) v_x,   lse = log sum_x exp(scale q . k_x)
 * T = 1, or parent[r, i] = i - 1, is attention of the next tokens of a sequence.
 * Scores, weights, sums and softmax statistics are binary32, but with 16-bit types a
 * weight meets the values as the sum of two numbers of the type, which hold it to
 * within 1.01 x 2^-16 (bf16) or 2^-21 (f16) of itself, f16 to no better than 2^-34 of
 * its row's largest.  A token that attends to nothing gets out 0 and lse -inf.  What a
 * token does not attend to is of no account to it (NaN included); an infinite value
 * that it does attend to makes its column infinite, where the weight is at least
 * 2^-90 of the row's largest. */
int cmd_tree_attention(const cmd_arg args[8], float scale, int32_t window, void *workspace, int64_t workspace_bytes,
                       int32_t flags, void *hip_stream);
int64_t cmd_tree_attention_workspace(const cmd_arg args[8], int32_t window);

/* The accepted path of a tree of drafted tokens.  args, all int32:
 *   0 tokens [B, T]   1 parent [B, T]   2 next [B, T]   3 lens [B]
 *   4 path [B, T]   5 lens_out [B]   6 last [B]
 * T <= 256.  Token 0, whose parent is -1, is the sequence's newest and stands; after
 * token i the model goes on with next[r, i].  From token 0 on the path goes to the
 * first token c with parent[r, c] = i < c and tokens[r, c] = next[r, i], until there
 * is none.  path[r] holds the tokens of the path, ascending, then -1; lens_out =
 * lens + how many they are (at most 2^31 - 1); last = next of the path's last.  A row
 * whose token 0 has another parent, or whose length is negative, has an empty path:
 * lens_out = lens, last -1.  lens_out may be the identical view as lens. */
int cmd_tree_accept(const cmd_arg args[7], int32_t flags, void *hip_stream);

/* Move the slots of a path's tokens to the end of their rows: in each of npools pools
 * [N_k, page, heads, d] (rank 4, any dtype of 2 or 4 bytes, page alike), for row r and
 * i = 0, 1, ... until path[r, i] is negative, what position lens[r] + path[r, i] holds
 * goes to position lens[r] + i, one i after the other.  args: 0 pages [R, P]   1 lens
 * [R]   2 path [R, T], all int32.  Entries path[r, i] <= i, positions past the table
 * and holes (ids outside a pool are its holes) move nothing, nor do rows with a
 * negative length.  T <= 256.  No slot that is written may lie in another row or column too.
 * The elements of a slot's head are neighbours. */
int cmd_slot_move(const cmd_arg *pools, int32_t npools, const cmd_arg args[3], int32_t flags, void *hip_stream);

/* Keep up the least and largest key of every page.  args:
 *   0 k_cache [N, page, hk, d]   1 pages [R, P] int32   2 lens [R] int32   3 since [R] int32
 *   4 bounds [N, hk, 2, d]       (of the cache's dtype f16, bf16 or f32; bounds[i, h, 0]
 *     the least, bounds[i, h, 1] the largest of what page i's slots hold, by element)
 * Positions max(since, 0) .. min(lens, P * page) - 1 of every row are new: the bounds
 * of a page whose first position is one of them are made from them, those of a page
 * that held earlier ones are widened by them.  Other pages' bounds stay.  NaN counts
 * as nothing (of NaN alone: least +inf, largest -inf).  No page with new positions may
 * stand in two rows or columns.  Bounds are a pool to cmd_page_copy: copied pages take theirs along. */
int cmd_page_bounds(const cmd_arg args[5], int32_t flags, void *hip_stream);

/* Choose for every sequence and kv head the pages that its query tokens may care for
 * most.  args:
 *   0 q [B, hq, d]   1 bounds [N, hk, 2, d]   2 pages [B, P] int32   3 lens [B] int32
 *   4 pages_out [B, hk, C] int32   5 lens_out [B, hk] int32
 * Candidates are the columns j < U = ceil(min(lens[r], P * page) / page) that are no
 * holes, in all if they are at most C.  Else those among the first `first` and the last
 * `last` of the U columns (first + last <= C), then the others by descending
 *      score[h, j] = max over kv head h's query heads of sum_e q_e (q_e < 0 ? least_e : largest_e)
 * (what no key of the page can pass; sums of binary64, NaN the least) until they
 * are C; the lower column wins a tie.  Bounds of NaN alone (least +inf, largest -inf)
 * make a score -inf or NaN, and so does 0 times an infinity: such pages come last.  pages_out[r, h] names them by ascending column, then
 * -1; lens_out is how many positions they hold: a table for cmd_paged_attention_heads.
 * P <= 2^20. */
int cmd_page_select(const cmd_arg args[6], int32_t page, int32_t first, int32_t last, void *workspace,
                    int64_t workspace_bytes, int32_t flags, void *hip_stream);
int64_t cmd_page_select_workspace(const cmd_arg args[6], int32_t page, int32_t first, int32_t last);

/* The weight that attention gave to every page, added up.  args:
 *   0 q [B, hq, d]   1 k_cache [N, page, hk, d]   2 pages [B, P] int32   3 lens [B] int32
 *   4 lse [B, hq] f32   5 mass [B, P] f32   6 mass_out [B, P] f32 (may be the identical view as mass)
 * with cmd_paged_attention's dtypes, positions and lse:
 *      mass_out[r, j] = decay mass[r, j] + sum_h sum_x exp(scale q_h . k_x - lse[r, h])
 * over the positions x of column j that row r attends to; heads whose lse is -inf add
 * nothing.  Products and sums are binary32. */
int cmd_page_mass(const cmd_arg args[7], float scale, float decay, int32_t window, int32_t flags, void *hip_stream);

/* Take the pages of least mass out of rows that hold more than their budgets.  args:
 *   0 pages [R, P] int32   1 lens [R] int32   2 refs [N] int32   3 mass [R, P] f32   4 budget [R] int32
 *   5 pages_out [R, P] int32   6 refs_out [N] int32   7 count [R] int32
 * Row r holds the columns j < U = ceil(min(lens[r], P * page) / page) that are no holes.
 * While they are more than max(budget[r], 0), the one of least mass is taken out (the
 * lower column wins a tie, NaN counts as more than any number), but for the first
 * `first` and the last `last` of the U columns.  pages_out is the table with holes (-1) in
 * their places (and where entries name no page), refs_out the counts less the entries
 * taken out, count how many each row lost.  pages_out may be the identical view as
 * pages, refs_out as refs.  P <= 2^20. */
int cmd_page_evict(const cmd_arg args[8], int32_t page, int32_t first, int32_t last, int32_t flags, void *hip_stream);

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
