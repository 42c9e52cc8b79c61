// ecmd_serving_cache.cpp -- argument checks, workspace sizes and launch geometry of
// the operators on trees of drafted tokens and on pages worth reading or keeping
// (include/ecmd_serving.h).  Host code; every check comes before the first HIP
// call, nothing here allocates or throws.
#include "ecmd_serving_check.h"

using namespace ecmd;

namespace {

// ---------------------------------------------------------------------------
// Attention for trees.

struct TreePlan {
    Tensor t[8];
    TreeArgs A;
    int type;
    int64_t workspace;
    bool nothing;
};

int plan_tree(const cmd_arg *args, int32_t window, TreePlan &P)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    Tensor *t = P.t;
    const int dt = args[0].dtype;
    TRY(check_float(dt, "q"));
    TRY(check(t[0], args[0], 4, dt, "q"));
    TRY(check(t[1], args[1], 4, dt, "k_cache"));
    TRY(check(t[2], args[2], 4, dt, "v_cache"));
    TRY(check(t[3], args[3], 2, CMD_I32, "pages"));
    TRY(check(t[4], args[4], 1, CMD_I32, "lens"));
    TRY(check(t[5], args[5], 2, CMD_I32, "parent"));
    TRY(check(t[6], args[6], 4, dt, "out"));
    if (args[7].kind != 0) TRY(check(t[7], args[7], 3, CMD_F32, "lse"));
    const int64_t b = t[0].size(0), tokens = t[0].size(1), hq = t[0].size(2), d = t[0].size(3);
    const int64_t n = t[1].size(0), page = t[1].size(1), hk = t[1].size(2), dv = t[2].size(3), cols = t[3].size(1);
    TRY(check_size(t[1], 3, d, "q"));
    for (int i = 0; i < 3; ++i) TRY(check_size(t[2], i, t[1].size(i), "k_cache"));
    for (int i : {3, 4, 5}) TRY(check_size(t[i], 0, b, "q"));
    TRY(check_size(t[5], 1, tokens, "q"));
    for (int i = 0; i < 3; ++i) {
        TRY(check_size(t[6], i, t[0].size(i), "q"));
        if (t[7].a) TRY(check_size(t[7], i, t[0].size(i), "q"));
    }
    TRY(check_size(t[6], 3, dv, "v_cache"));
    if (tokens > (int64_t)kMaxTree)
        return refuse(CMD_E_LIMIT, "a tree of %lld tokens, at most %u expected", (long long)tokens, kMaxTree);
    if (hk == 0 ? hq != 0 : hq % hk != 0)
        return refuse(CMD_E_SHAPE, "%lld query heads are no multiple of %lld kv heads", (long long)hq, (long long)hk);
    if (d < 1 || dv < 1) return refuse(CMD_E_SHAPE, "heads of width 0");
    if (d > 256 || dv > 256) return refuse(CMD_E_LIMIT, "heads wider than 256");
    if (window < 0) return refuse(CMD_E_ARG, "negative window");
    for (int i : {0, 1, 2, 6}) TRY(check_unit(t[i]));
    TRY(check_outputs(t, 8, 6, nullptr));
    if (cols * std::max<int64_t>(page, 1) > (int64_t(1) << 30))
        return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    TreeArgs &A = P.A;
    A = TreeArgs{};
    P.type = serving_type(dt);
    P.workspace = 0;
    P.nothing = b == 0 || hq == 0 || tokens == 0;
    if (P.nothing) return CMD_OK;
    const int64_t esize = type_size(dt);
    A.q = args[0].ptr;
    A.k = args[1].ptr;
    A.v = args[2].ptr;
    A.pages = (const int32_t *)args[3].ptr;
    A.lens = (const int32_t *)args[4].ptr;
    A.parent = (const int32_t *)args[5].ptr;
    A.out = args[6].ptr;
    A.lse = t[7].a ? (float *)args[7].ptr : nullptr;
    for (int i = 0; i < 3; ++i) {
        A.qs[i] = t[0].stride(i);
        A.os[i] = t[6].stride(i);
        A.ls[i] = t[7].a ? t[7].stride(i) : 0;
        A.kcs[i] = t[1].stride(i) * esize;
        A.vcs[i] = t[2].stride(i) * esize;
    }
    for (int i = 0; i < 2; ++i) {
        A.pages_s[i] = t[3].stride(i);
        A.parent_s[i] = t[5].stride(i);
    }
    A.lens_s = t[4].stride(0);
    if ((uint64_t)b * tokens * hq > (uint64_t)kMaxCount || ((uint64_t)b * tokens * hq + 3) / 4 > kMaxGroups)
        return refuse(CMD_E_LIMIT, "too many query vectors for one launch");
    A.b = (uint32_t)b;
    A.t = (uint32_t)tokens;
    A.hq = (uint32_t)hq;
    A.hk = (uint32_t)hk;
    A.d = (uint32_t)d;
    A.dv = (uint32_t)dv;
    A.group = (uint32_t)(hq / hk);
    A.m = A.t * A.group;
    A.n = (uint32_t)n;
    A.page = (uint32_t)std::max<int64_t>(1, page);
    A.cols = n > 0 && page > 0 ? (uint32_t)cols : 0;   // a cache without slots: every row is empty
    A.window = (uint32_t)window;
    uint64_t keys = (uint64_t)A.cols * A.page;
    if (window) keys = std::min<uint64_t>(keys, (uint64_t)window + 2 * kMaxTree);
    const uint64_t steps = (keys + kAttnStep - 1) / kAttnStep, most = std::max<uint64_t>(1, steps * (uint64_t)b);
    const uint64_t row_bytes = keys * (uint64_t)((d + dv) * esize);
    // Tiles of 16-bit keys and values are staged for all query vectors of a work-group, if every
    // row of the caches starts at a multiple of 16 bytes and is one: from 65 vectors on, and from
    // 17 on where steps and heads are more than the compute units.  (8 tokens of 32 heads over 8, us
    // not staged and staged: 16 rows of up to 8192 positions 76 and 62, one of 6000 23.0 and
    // 22.6, one of 3000 19.7 and 21.1; 16 tokens: 123 and 74, one row of 777 18.3 and 21.0; 4
    // tokens, 16 rows: 66 and 66; 64 tokens, two rows of 60: 27 and 20.)  A wave takes 32 vectors from
    // 65 on, as far as the registers go (17 tokens: 83, with 16 97; 9 tokens: 73, with 16 68).
    // Otherwise the waves part the positions of up to 16 (32) vectors, the vectors of more.
    bool even = P.type != S_F32 && (d * esize) % 16 == 0 && (dv * esize) % 16 == 0 && (uintptr_t)A.k % 16 == 0 && (uintptr_t)A.v % 16 == 0;
    for (int i = 0; i < 3; ++i) even = even && A.kcs[i] % 16 == 0 && A.vcs[i] % 16 == 0;
    if (A.m <= 64) even = even && A.m > 16 && most * A.hk > 256;
    A.tiles = !even ? 0 : A.m > 64 && d <= 128 && dv <= 128 ? 2 : 1;
    A.direct = (steps <= 6 && row_bytes <= (256 << 10)) || b > kTreeMaxRows || most > (uint64_t(1) << 30);
    // While less than a work-group for each compute unit comes of it, waves part
    // positions rather than vectors (12 rows of 4 tokens, 32 heads over 2, up to 164 positions, f32:
    // 55 to 32 us; past that, a tile read for fewer vectors costs more: 16 rows of 28 tokens, 24
    // heads over 8, 60 positions, f32: 25 to 32 us).
    const uint32_t need = ceil_div(A.m, 16);
    auto blocks = [&] { return A.tiles ? ceil_div(A.m, 64 * A.tiles) : ceil_div(need, 1u << A.q_shift); };
    A.q_shift = need >= 3 ? 2 : need - 1;
    while (!A.tiles && A.q_shift && (A.direct ? (uint64_t)b : most) * A.hk * blocks() < 256) --A.q_shift;
    A.q_blocks = blocks();
    const uint64_t units = (uint64_t)A.hk * A.q_blocks;
    if ((uint64_t)(b + 8) * units > kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
    // Work-groups at once (2 rows of 27 tokens, 4 heads of 192 over 1, up to 56404 positions, bf16:
    // 512 runs take 71 us, 256 54).
    const uint64_t fit = A.tiles && (d > 128 || dv > 128) ? 256 : 512;
    A.runs = (uint32_t)std::min(std::max<uint64_t>(1, fit / units), std::min<uint64_t>(most, kAttnMaxRuns));
    A.runs_whole = (uint64_t)b * units >= 128 && (uint64_t)b * units <= 2048 ? A.b : 0;
    auto eight = [](uint64_t x) { return (x + 7) / 8 * 8; };
    A.grid = (uint32_t)((A.direct ? eight(b) : eight(std::max(A.runs, std::max(A.runs_whole, A.b <= A.runs ? A.b : 0)))) * units);
    A.by_page = Div31(A.page);
    A.by_units = Div31((uint32_t)(8 * units));
    A.by_blocks = Div31(A.q_blocks);
    A.by_group = Div31(A.group);
    A.by_runs = Div31(A.runs);
    A.by_vectors = Div31(A.hk * A.m);
    // The join: a vector to a work-group where there are at most 2048 and a row may be in more
    // than a dozen segments (8 heads, one row of 60000 positions 33 us, several 91; 4 rows of
    // 8192, 16 segments each, 29 and 33; 5 rows, 8 each, 27.3 and 25.5); else as many as make 2048
    // work-groups (32768 vectors, with the attention before it: 512 178 us, 1024 177, 2048 174, 4096 177).
    while (4u << A.join_shift < A.dv) ++A.join_shift;
    const uint32_t vectors = A.b * A.hk * A.m, places = 256 >> A.join_shift;
    A.join_turn = vectors <= 2048 && A.runs > 12 * A.b ? 1 : ceil_div(ceil_div(vectors, 2048), places) * places;
    if (!A.direct) P.workspace = (int64_t)((((uint64_t)A.runs + b) * A.hk * A.m * (dv + 2)) * 4 + 16);
    return CMD_OK;
}

}  // namespace

extern "C" {

int64_t cmd_tree_attention_workspace(const cmd_arg args[8], int32_t window)
{
    TreePlan P;
    const int rc = plan_tree(args, window, P);
    return rc ? rc : P.workspace;
}

int cmd_tree_attention(const cmd_arg args[8], float scale, int32_t window, void *workspace, int64_t workspace_bytes,
                       int32_t flags, void *hip_stream)
{
    TRY(check_flags(flags));
    TreePlan P;
    TRY(plan_tree(args, window, P));
    const float scale_log2 = (float)((double)scale * 1.44269504088896340736);
    if (!std::isfinite(scale_log2)) return refuse(CMD_E_ARG, "scale is not finite, or too large for binary32 in base 2");
    if ((flags & CMD_CHECK_ONLY) || P.nothing) return CMD_OK;
    TRY(check_workspace(workspace, workspace_bytes, P.workspace));
    TreeArgs &A = P.A;
    A.scale_log2 = std::fabs(scale_log2);
    A.q_flip = std::signbit(scale_log2) ? (P.type == S_F32 ? 0x80000000u : 0x80008000u) : 0;
    if (!A.direct) {
        A.ml = (float *)workspace;
        A.acc = A.ml + ((((uint64_t)A.runs + A.b) * A.hk * A.m * 2 + 3) & ~uint64_t(3));
    }
    TRY(launched(P.type == S_F16    ? launch_tree_f16(A, hip_stream)
                 : P.type == S_BF16 ? launch_tree_bf16(A, hip_stream)
                                    : launch_tree_f32(A, hip_stream),
                 "tree_attention"));
    if (A.direct) return CMD_OK;
    return launched(launch_tree_join(P.type, A, hip_stream), "tree_attention join");
}

// ---------------------------------------------------------------------------
// The accepted path.

int cmd_tree_accept(const cmd_arg args[7], int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    static const char *const names[7] = {"tokens", "parent", "next", "lens", "path", "lens_out", "last"};
    Tensor t[7];
    for (int i = 0; i < 7; ++i) TRY(check(t[i], args[i], i == 3 || i >= 5 ? 1 : 2, CMD_I32, names[i]));
    const int64_t rows = t[0].size(0), tokens = t[0].size(1);
    for (int i = 1; i < 7; ++i) TRY(check_size(t[i], 0, rows, "tokens"));
    for (int i : {1, 2, 4}) TRY(check_size(t[i], 1, tokens, "tokens"));
    if (tokens > (int64_t)kMaxTree)
        return refuse(CMD_E_LIMIT, "a tree of %lld tokens, at most %u expected", (long long)tokens, kMaxTree);
    if (rows > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "too many rows for one launch");
    static const int share[7] = {-1, -1, -1, -1, -1, 3, -1};
    TRY(check_outputs(t, 7, 4, share));
    if ((flags & CMD_CHECK_ONLY) || rows == 0) return CMD_OK;
    AcceptArgs A{};
    A.tokens = (const int32_t *)args[0].ptr;
    A.parent = (const int32_t *)args[1].ptr;
    A.next = (const int32_t *)args[2].ptr;
    A.lens = (const int32_t *)args[3].ptr;
    A.path = (int32_t *)args[4].ptr;
    A.lens_out = (int32_t *)args[5].ptr;
    A.last = (int32_t *)args[6].ptr;
    for (int i = 0; i < 2; ++i) {
        A.tokens_s[i] = t[0].stride(i);
        A.parent_s[i] = t[1].stride(i);
        A.next_s[i] = t[2].stride(i);
        A.path_s[i] = t[4].stride(i);
    }
    A.lens_s = t[3].stride(0);
    A.lens_out_s = t[5].stride(0);
    A.last_s = t[6].stride(0);
    A.rows = (uint32_t)rows;
    A.t = (uint32_t)tokens;
    return launched(launch_accept(A, hip_stream), "tree_accept");
}

int cmd_slot_move(const cmd_arg *pools, int32_t npools, const cmd_arg args[3], int32_t flags, void *hip_stream)
{
    TRY(check_flags(flags));
    if (npools < 0 || (npools && !pools) || !args) return refuse(CMD_E_ARG, "pools or args is NULL");
    Tensor pages, lens, path;
    TRY(check(pages, args[0], 2, CMD_I32, "pages"));
    TRY(check(lens, args[1], 1, CMD_I32, "lens"));
    TRY(check(path, args[2], 2, CMD_I32, "path"));
    const int64_t rows = pages.size(0), cols = pages.size(1), tokens = path.size(1);
    TRY(check_size(lens, 0, rows, "pages"));
    TRY(check_size(path, 0, rows, "pages"));
    if (tokens > (int64_t)kMaxTree)
        return refuse(CMD_E_LIMIT, "paths of %lld tokens, at most %u expected", (long long)tokens, kMaxTree);
    // Two passes: everything is checked before the first launch.
    for (int pass = 0; pass < 2; ++pass) {
        MoveArgs A{};
        int held = 0, width = 0;
        uint32_t vecs = 0;
        int64_t page = -1;
        auto flush = [&]() -> int {
            if (!held) return CMD_OK;
            A.pages = (const int32_t *)args[0].ptr;
            A.lens = (const int32_t *)args[1].ptr;
            A.path = (const int32_t *)args[2].ptr;
            for (int i = 0; i < 2; ++i) A.pages_s[i] = pages.stride(i), A.path_s[i] = path.stride(i);
            A.lens_s = lens.stride(0);
            A.rows = (uint32_t)rows;
            A.cols = (uint32_t)cols;
            A.t = (uint32_t)tokens;
            A.page = (uint32_t)page;
            A.vecs = vecs;
            A.pieces = ceil_div(vecs, 256);
            A.by_page = Div31(A.page);
            A.by_pieces = Div31(A.pieces);
            if ((uint64_t)rows * A.pieces * held > kMaxGroups) return refuse(CMD_E_LIMIT, "too many rows for slots of this size");
            const uint32_t n = (uint32_t)held;
            held = 0;
            if (pass == 0) return CMD_OK;
            return launched(launch_move(width, A, n, hip_stream), "slot_move");
        };
        for (int i = 0; i < npools; ++i) {
            Tensor t;
            char name[32];
            snprintf(name, sizeof name, "pool %d", i);
            const int dt = pools[i].dtype;
            if (dt != CMD_F16 && dt != CMD_BF16 && dt != CMD_F32 && dt != CMD_I32)
                return refuse(CMD_E_DTYPE, "%s has an unknown dtype %d", name, dt);
            TRY(check(t, pools[i], 4, dt, name));
            TRY(check_unit(t));
            if (pass == 0) {
                TRY(check_one_to_one(t));
                for (const Tensor *x : {&pages, &lens, &path})
                    if (!disjoint(*x, t)) return refuse(CMD_E_ALIAS, "%s overlaps %s", name, x->name);
                for (int k = 0; k < i; ++k) {
                    const Tensor other{&pools[k], 4, ""};
                    if (!disjoint(other, t)) return refuse(CMD_E_ALIAS, "%s overlaps pool %d", name, k);
                }
            }
            if (page >= 0 && t.size(1) != page)
                return refuse(CMD_E_SHAPE, "%s: dimension 1 is %lld, %lld expected (pool 0)", name, (long long)t.size(1), (long long)page);
            page = t.size(1);
            if (page * cols > (int64_t(1) << 30)) return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
            if (t.empty() || rows == 0 || cols == 0 || tokens == 0) continue;
            const int e = type_size(dt);
            const uint64_t inner = (uint64_t)t.size(3) * e;
            const uint64_t page_stride = (uint64_t)t.stride(0) * e, slot_stride = (uint64_t)t.stride(1) * e, head_stride = (uint64_t)t.stride(2) * e;
            // the widest vector that divides the heads and starts aligned in every one
            int w = 16;
            const uint64_t all = (uint64_t)t.begin() | page_stride | slot_stride | head_stride | inner;
            while (w > e && all % w) w /= 2;
            if (t.size(2) * (int64_t)(inner / w) > kMaxCount / 2) return refuse(CMD_E_LIMIT, "%s: a slot is too large", name);
            const uint32_t v = (uint32_t)(t.size(2) * (inner / w));
            if (held && (w != width || v != vecs || held == kMovePools)) TRY(flush());
            width = w;
            vecs = v;
            MovePool &p = A.pool[held++];
            p.base = (char *)t.a->ptr;
            p.page_stride = (int64_t)page_stride;
            p.slot_stride = (int64_t)slot_stride;
            p.head_stride = (int64_t)head_stride;
            p.n = (uint32_t)t.size(0);
            p.head_vecs = (uint32_t)(inner / w);
            p.by_head = Div31(p.head_vecs);
        }
        TRY(flush());
        if (flags & CMD_CHECK_ONLY) return CMD_OK;
    }
    return CMD_OK;
}

// ---------------------------------------------------------------------------
// Pages worth reading or keeping.

int cmd_page_bounds(const cmd_arg args[5], int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    const int dt = args[0].dtype;
    TRY(check_float(dt, "k_cache"));
    Tensor t[5];
    TRY(check(t[0], args[0], 4, dt, "k_cache"));
    TRY(check(t[1], args[1], 2, CMD_I32, "pages"));
    TRY(check(t[2], args[2], 1, CMD_I32, "lens"));
    TRY(check(t[3], args[3], 1, CMD_I32, "since"));
    TRY(check(t[4], args[4], 4, dt, "bounds"));
    const int64_t n = t[0].size(0), page = t[0].size(1), hk = t[0].size(2), d = t[0].size(3);
    const int64_t rows = t[1].size(0), cols = t[1].size(1);
    TRY(check_size(t[2], 0, rows, "pages"));
    TRY(check_size(t[3], 0, rows, "pages"));
    TRY(check_size(t[4], 0, n, "k_cache"));
    TRY(check_size(t[4], 1, hk, "k_cache"));
    TRY(check_size(t[4], 2, 2, "the least and the largest"));
    TRY(check_size(t[4], 3, d, "k_cache"));
    TRY(check_unit(t[0]));
    TRY(check_unit(t[4]));
    TRY(check_outputs(t, 5, 4, nullptr));
    if (cols * std::max<int64_t>(page, 1) > (int64_t(1) << 30))
        return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    if (rows > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "too many rows for one launch");
    const int64_t e = type_size(dt), head_items = (d * e + 15) / 16, items = head_items * hk, parts = (items + 255) / 256;
    if (parts * std::max<int64_t>(cols, 1) > kMaxCount) return refuse(CMD_E_LIMIT, "k_cache: slots too large for tables this long");
    if ((flags & CMD_CHECK_ONLY) || rows == 0 || cols == 0 || t[0].empty()) return CMD_OK;
    BoundsArgs A{};
    A.k = args[0].ptr;
    A.pages = (const int32_t *)args[1].ptr;
    A.lens = (const int32_t *)args[2].ptr;
    A.since = (const int32_t *)args[3].ptr;
    A.bounds = args[4].ptr;
    for (int i = 0; i < 3; ++i) A.kcs[i] = t[0].stride(i) * e, A.bs[i] = t[4].stride(i) * e;
    for (int i = 0; i < 2; ++i) A.pages_s[i] = t[1].stride(i);
    A.lens_s = t[2].stride(0);
    A.since_s = t[3].stride(0);
    A.rows = (uint32_t)rows;
    A.cols = (uint32_t)cols;
    A.n = (uint32_t)n;
    A.page = (uint32_t)page;
    A.hk = (uint32_t)hk;
    A.d = (uint32_t)d;
    A.head_items = (uint32_t)head_items;
    A.items = (uint32_t)items;
    A.many = items <= 128 ? (uint32_t)(256 / items) : 1;
    A.parts = (uint32_t)parts;
    // as many work-groups as all of a row's columns make, 2048 in all at most (a decode
    // step needs one a row)
    const uint64_t turns = A.many > 1 ? ceil_div(cols, A.many) : (uint64_t)cols * A.parts;
    A.groups = (uint32_t)std::min<uint64_t>(turns, std::max<uint64_t>(1, 2048 / (uint64_t)rows));
    A.by_page = Div31(A.page);
    A.by_items = Div31(A.items);
    A.by_head = Div31(A.head_items);
    A.by_many = Div31(A.many);
    A.by_parts = Div31(A.parts);
    A.by_groups = Div31(A.groups);
    return launched(launch_bounds(serving_type(dt), A, hip_stream), "page_bounds");
}

}  // extern "C"

namespace {

struct SelectPlan {
    SelectArgs A;
    int type;
    int64_t workspace;
    bool nothing;
};

int plan_select(const cmd_arg *args, int32_t page, int32_t first, int32_t last, SelectPlan &P)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    const int dt = args[0].dtype;
    TRY(check_float(dt, "q"));
    Tensor t[6];
    TRY(check(t[0], args[0], 3, dt, "q"));
    TRY(check(t[1], args[1], 4, dt, "bounds"));
    TRY(check(t[2], args[2], 2, CMD_I32, "pages"));
    TRY(check(t[3], args[3], 1, CMD_I32, "lens"));
    TRY(check(t[4], args[4], 3, CMD_I32, "pages_out"));
    TRY(check(t[5], args[5], 2, CMD_I32, "lens_out"));
    const int64_t b = t[0].size(0), hq = t[0].size(1), d = t[0].size(2), n = t[1].size(0), hk = t[1].size(1);
    const int64_t cols = t[2].size(1), take = t[4].size(2);
    TRY(check_size(t[1], 2, 2, "the least and the largest"));
    TRY(check_size(t[1], 3, d, "q"));
    for (int i : {2, 3, 4, 5}) TRY(check_size(t[i], 0, b, "q"));
    TRY(check_size(t[4], 1, hk, "bounds"));
    TRY(check_size(t[5], 1, hk, "bounds"));
    if (hk == 0 ? hq != 0 : hq % hk != 0 || hq == 0)
        return refuse(CMD_E_SHAPE, "%lld query heads are no multiple of %lld kv heads", (long long)hq, (long long)hk);
    if (d < 1) return refuse(CMD_E_SHAPE, "heads of width 0");
    if (d > 256) return refuse(CMD_E_LIMIT, "heads wider than 256");
    if (page < 1) return refuse(CMD_E_ARG, "pages of %d slots", page);
    if (first < 0 || last < 0 || (int64_t)first + last > take || take < 1)
        return refuse(CMD_E_ARG, "%d first and %d last pages of %lld", first, last, (long long)take);
    TRY(check_unit(t[0]));
    TRY(check_unit(t[1]));
    TRY(check_outputs(t, 6, 4, nullptr));
    if (cols * (int64_t)page > (int64_t(1) << 30)) return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    if (cols > (int64_t(1) << 20)) return refuse(CMD_E_LIMIT, "a table of more than 2^20 columns");
    if (b * hk > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
    SelectArgs &A = P.A;
    A = SelectArgs{};
    P.type = serving_type(dt);
    P.workspace = 0;
    P.nothing = b == 0 || hk == 0;
    if (P.nothing) return CMD_OK;
    const int64_t e = type_size(dt);
    A.q = args[0].ptr;
    A.bounds = args[1].ptr;
    A.pages = (const int32_t *)args[2].ptr;
    A.lens = (const int32_t *)args[3].ptr;
    A.pages_out = (int32_t *)args[4].ptr;
    A.lens_out = (int32_t *)args[5].ptr;
    for (int i = 0; i < 2; ++i) {
        A.qs[i] = t[0].stride(i) * e;
        A.pages_s[i] = t[2].stride(i);
        A.lens_out_s[i] = t[5].stride(i);
    }
    for (int i = 0; i < 3; ++i) A.bs[i] = t[1].stride(i) * e, A.pages_out_s[i] = t[4].stride(i);
    A.lens_s = t[3].stride(0);
    A.b = (uint32_t)b;
    A.hk = (uint32_t)hk;
    A.group = (uint32_t)(hq / hk);
    A.d = (uint32_t)d;
    A.n = (uint32_t)n;
    A.cols = (uint32_t)cols;
    A.page = (uint32_t)page;
    A.take = (uint32_t)std::min<int64_t>(take, kMaxCount);
    A.first = (uint32_t)first;
    A.last = (uint32_t)last;
    A.by_page = Div31(A.page);
    A.by_hk = Div31(A.hk);
    const uint64_t rows = (uint64_t)b * hk;
    // A turn of columns to a work-group at least, and about 2048 work-groups (64 rows of 8 heads and
    // up to 512 columns: 512 take 95 us with the attention after it, 1024 92, 2048 89, 4096 93).
    A.groups = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(ceil_div(cols, 32), ceil_div(2048, rows)));
    A.by_groups = Div31(A.groups);
    if (rows * A.groups > kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
    P.workspace = (int64_t)(rows * cols * 8);
    return CMD_OK;
}

}  // namespace

extern "C" {

int64_t cmd_page_select_workspace(const cmd_arg args[6], int32_t page, int32_t first, int32_t last)
{
    SelectPlan P;
    const int rc = plan_select(args, page, first, last, P);
    return rc ? rc : P.workspace;
}

int cmd_page_select(const cmd_arg args[6], int32_t page, int32_t first, int32_t last, void *workspace,
                    int64_t workspace_bytes, int32_t flags, void *hip_stream)
{
    TRY(check_flags(flags));
    SelectPlan P;
    TRY(plan_select(args, page, first, last, P));
    if ((flags & CMD_CHECK_ONLY) || P.nothing) return CMD_OK;
    TRY(check_workspace(workspace, workspace_bytes, P.workspace));
    P.A.keys = P.workspace ? (uint64_t *)workspace : nullptr;
    return launched(launch_select(P.type, P.A, hip_stream), "page_select");
}

int cmd_page_mass(const cmd_arg args[7], float scale, float decay, int32_t window, int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    const int dt = args[0].dtype;
    TRY(check_float(dt, "q"));
    Tensor t[7];
    TRY(check(t[0], args[0], 3, dt, "q"));
    TRY(check(t[1], args[1], 4, dt, "k_cache"));
    TRY(check(t[2], args[2], 2, CMD_I32, "pages"));
    TRY(check(t[3], args[3], 1, CMD_I32, "lens"));
    TRY(check(t[4], args[4], 2, CMD_F32, "lse"));
    TRY(check(t[5], args[5], 2, CMD_F32, "mass"));
    TRY(check(t[6], args[6], 2, CMD_F32, "mass_out"));
    const int64_t b = t[0].size(0), hq = t[0].size(1), d = t[0].size(2);
    const int64_t n = t[1].size(0), page = t[1].size(1), hk = t[1].size(2), cols = t[2].size(1);
    TRY(check_size(t[1], 3, d, "q"));
    for (int i : {2, 3, 4, 5, 6}) TRY(check_size(t[i], 0, b, "q"));
    TRY(check_size(t[4], 1, hq, "q"));
    TRY(check_size(t[5], 1, cols, "pages"));
    TRY(check_size(t[6], 1, cols, "pages"));
    if (hk == 0 ? hq != 0 : hq % hk != 0)
        return refuse(CMD_E_SHAPE, "%lld query heads are no multiple of %lld kv heads", (long long)hq, (long long)hk);
    if (d < 1) return refuse(CMD_E_SHAPE, "heads of width 0");
    if (d > 256) return refuse(CMD_E_LIMIT, "heads wider than 256");
    if (window < 0) return refuse(CMD_E_ARG, "negative window");
    if (!std::isfinite((float)((double)scale * 1.44269504088896340736)))   // as attention does
        return refuse(CMD_E_ARG, "scale is not finite, or too large for binary32 in base 2");
    if (!std::isfinite(decay)) return refuse(CMD_E_ARG, "decay is not finite");
    TRY(check_unit(t[0]));
    TRY(check_unit(t[1]));
    static const int share[7] = {-1, -1, -1, -1, -1, -1, 5};
    TRY(check_outputs(t, 7, 6, share));
    if (cols * std::max<int64_t>(page, 1) > (int64_t(1) << 30))
        return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    MassArgs A{};
    A.page = (uint32_t)std::max<int64_t>(1, page);
    // Columns of a work-group: of about 64 positions (64 rows of up to 8192, bf16: 256 take 102
    // us, 128 96, 64 93 and 32 104), and of 32 where that leaves less than two work-groups for
    // each compute unit (3 rows of up to 1500, f32: 58 us at 256, 14.6 at 32, 8.7 with d's own products).
    A.cols_group = std::max(1u, 64 / A.page);
    if ((uint64_t)b * ceil_div(cols, A.cols_group) < 512) A.cols_group = std::max(1u, 32 / A.page);
    A.groups = ceil_div(cols, A.cols_group);
    if ((uint64_t)b * A.groups > kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times pages for one launch");
    if ((flags & CMD_CHECK_ONLY) || b == 0 || cols == 0) return CMD_OK;
    const int64_t e = type_size(dt);
    A.q = args[0].ptr;
    A.k = args[1].ptr;
    A.pages = (const int32_t *)args[2].ptr;
    A.lens = (const int32_t *)args[3].ptr;
    A.lse = (const float *)args[4].ptr;
    A.mass = (const float *)args[5].ptr;
    A.out = (float *)args[6].ptr;
    for (int i = 0; i < 2; ++i) {
        A.qs[i] = t[0].stride(i) * e;
        A.pages_s[i] = t[2].stride(i);
        A.lse_s[i] = t[4].stride(i);
        A.mass_s[i] = t[5].stride(i);
        A.out_s[i] = t[6].stride(i);
    }
    for (int i = 0; i < 3; ++i) A.kcs[i] = t[1].stride(i) * e;
    A.lens_s = t[3].stride(0);
    A.b = (uint32_t)b;
    A.hk = t[1].empty() ? 0 : (uint32_t)hk;   // a cache without slots: nothing is read
    A.group = hk ? (uint32_t)(hq / hk) : 0;
    A.d = (uint32_t)d;
    A.n = (uint32_t)n;
    A.cols = (uint32_t)cols;
    A.window = (uint32_t)window;
    A.scale = scale;
    A.decay = decay;
    A.by_page = Div31(A.page);
    A.by_groups = Div31(A.groups);
    const int type = serving_type(dt);
    return launched(type == S_F16    ? launch_mass_f16(A, hip_stream)
                    : type == S_BF16 ? launch_mass_bf16(A, hip_stream)
                                     : launch_mass_f32(A, hip_stream),
                    "page_mass");
}

int cmd_page_evict(const cmd_arg args[8], int32_t page, int32_t first, int32_t last, int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    static const char *const names[8] = {"pages", "lens", "refs", "mass", "budget", "pages_out", "refs_out", "count"};
    Tensor t[8];
    for (int i = 0; i < 8; ++i) TRY(check(t[i], args[i], i == 0 || i == 3 || i == 5 ? 2 : 1, i == 3 ? CMD_F32 : CMD_I32, names[i]));
    const int64_t rows = t[0].size(0), cols = t[0].size(1), n = t[2].size(0);
    for (int i : {1, 3, 4, 5, 7}) TRY(check_size(t[i], 0, rows, "pages"));
    TRY(check_size(t[3], 1, cols, "pages"));
    TRY(check_size(t[5], 1, cols, "pages"));
    TRY(check_size(t[6], 0, n, "refs"));
    if (page < 1) return refuse(CMD_E_ARG, "pages of %d slots", page);
    if (first < 0 || last < 0) return refuse(CMD_E_ARG, "%d first and %d last pages", first, last);
    static const int share[8] = {-1, -1, -1, -1, -1, 0, 2, -1};
    TRY(check_outputs(t, 8, 5, share));
    if (cols * (int64_t)page > (int64_t(1) << 30)) return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    if (cols > (int64_t(1) << 20)) return refuse(CMD_E_LIMIT, "a table of more than 2^20 columns");
    if (rows > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "too many rows for one launch");
    if ((flags & CMD_CHECK_ONLY)) return CMD_OK;
    EvictArgs A{};
    A.pages = (const int32_t *)args[0].ptr;
    A.lens = (const int32_t *)args[1].ptr;
    A.refs = (const int32_t *)args[2].ptr;
    A.mass = (const float *)args[3].ptr;
    A.budget = (const int32_t *)args[4].ptr;
    A.pages_out = (int32_t *)args[5].ptr;
    A.refs_out = (int32_t *)args[6].ptr;
    A.count = (int32_t *)args[7].ptr;
    for (int i = 0; i < 2; ++i) {
        A.pages_s[i] = t[0].stride(i);
        A.mass_s[i] = t[3].stride(i);
        A.pages_out_s[i] = t[5].stride(i);
    }
    A.lens_s = t[1].stride(0);
    A.refs_s = t[2].stride(0);
    A.budget_s = t[4].stride(0);
    A.refs_out_s = t[6].stride(0);
    A.count_s = t[7].stride(0);
    A.rows = (uint32_t)rows;
    A.cols = (uint32_t)cols;
    A.n = (uint32_t)n;
    A.page = (uint32_t)page;
    A.first = (uint32_t)first;
    A.last = (uint32_t)last;
    A.copy = !identical(t[2], t[6]);
    A.by_page = Div31(A.page);
    return launched(launch_evict(A, hip_stream), "page_evict");
}

}  // extern "C"
