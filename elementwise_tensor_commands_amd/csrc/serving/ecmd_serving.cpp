// ecmd_serving.cpp -- the serving operators' C ABI (include/ecmd_serving.h):
// argument checks, workspace sizes, launch geometry of rope, paged attention and
// the pages' bookkeeping.  Host code; every check comes before the first HIP call,
// nothing here allocates or throws.
#include "ecmd_serving_check.h"

using namespace ecmd;

namespace {

int check_layout(int32_t layout, double mscale)
{
    if (layout != CMD_ROPE_HALF && layout != CMD_ROPE_INTERLEAVED)
        return refuse(CMD_E_ARG, "layout %d is neither CMD_ROPE_HALF nor CMD_ROPE_INTERLEAVED", layout);
    if (!std::isfinite(mscale)) return refuse(CMD_E_ARG, "mscale is not finite");
    return CMD_OK;
}

constexpr int64_t kMaxPairs = 2048;

// 16-byte items of a head (see the rope kernels): pairs, then the copied tail.
uint32_t head_items(int type, int layout, uint32_t pairs, uint32_t width)
{
    const uint32_t e = type == S_F32 ? 4 : 8;
    const uint32_t rot = layout == CMD_ROPE_HALF ? ceil_div(pairs, e) : ceil_div(2 * pairs, e);
    return rot + ceil_div(width - 2 * pairs, e);
}

// The kernels' edge for heads of this kind: 0, no vector is cut short; 1, none is
// longer than what it is cut from; 2.
int head_edge(int type, int layout, uint32_t pairs, uint32_t width)
{
    const uint32_t e = type == S_F32 ? 4 : 8, part = layout == CMD_ROPE_HALF ? pairs : 2 * pairs;
    if (part % e == 0 && (width - 2 * pairs) % e == 0) return 0;
    return (part == 0 || part >= e) && width >= e ? 1 : 2;
}

// Tokens of a work-group: about 1024 items (the four that each work-item loads at
// once), while there remain enough groups for 256 compute units four times over
// and the cosines stay within 16 KiB of LDS.  More where a launch cannot have so many
// groups: the 288 GB of tokens that fill the memory then still take less than 64 KiB.
uint32_t tokens_per_group(uint64_t tokens, uint64_t items, uint64_t pairs)
{
    uint64_t tb = std::max<uint64_t>(1, 1024 / std::max<uint64_t>(1, items));
    tb = std::min(tb, std::max<uint64_t>(1, tokens / 1024));
    tb = std::min(tb, std::max<uint64_t>(1, 16384 / (8 * ((pairs + 7) / 8 * 8) + 16)));
    return (uint32_t)std::max<uint64_t>(tb, ceil_div(tokens, kMaxGroups));
}

uint32_t turn_lds(uint32_t tb, uint32_t pairs) { return tb * ((pairs + 7) / 8 * 8) * 8; }

}  // namespace

extern "C" {

int cmd_rope(const cmd_arg args[4], int32_t layout, double mscale, int32_t inverse, int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    TRY(check_layout(layout, mscale));
    const int dt = args[0].dtype;
    TRY(check_float(dt, "x"));
    Tensor t[4];
    TRY(check(t[0], args[0], 4, dt, "x"));
    TRY(check(t[1], args[1], 2, CMD_I32, "pos"));
    TRY(check(t[2], args[2], 1, CMD_F64, "freq"));
    TRY(check(t[3], args[3], 4, dt, "out"));
    for (int i = 0; i < 4; ++i) TRY(check_size(t[3], i, t[0].size(i), "x"));
    for (int i = 0; i < 2; ++i) TRY(check_size(t[1], i, t[0].size(i), "x"));
    const int64_t b = t[0].size(0), n = t[0].size(1), h = t[0].size(2), d = t[0].size(3), m = t[2].size(0);
    if (2 * m > d)
        return refuse(CMD_E_SHAPE, "%lld frequencies turn %lld elements of a head of %lld", (long long)m,
                      (long long)(2 * m), (long long)d);
    if (m > kMaxPairs) return refuse(CMD_E_LIMIT, "more than %lld frequencies", (long long)kMaxPairs);
    TRY(check_unit(t[0]));
    TRY(check_unit(t[3]));
    static const int share[4] = {-1, -1, -1, 0};
    TRY(check_outputs(t, 4, 3, share));
    if (b * n > kMaxCount) return refuse(CMD_E_LIMIT, "more than 2^31 - 1 tokens");
    const int type = serving_type(dt);
    RopeArgs A{};
    A.pairs = (uint32_t)m;
    A.width = (uint32_t)d;
    const uint64_t per_head = head_items(type, layout, A.pairs, A.width), items = per_head * (uint64_t)h;
    if (items > (uint64_t)kMaxCount / 2) return refuse(CMD_E_LIMIT, "x: a token has too many elements");
    if ((flags & CMD_CHECK_ONLY) || t[0].empty()) return CMD_OK;
    A.x = args[0].ptr;
    A.pos = (const int32_t *)args[1].ptr;
    A.freq = (const double *)args[2].ptr;
    A.out = args[3].ptr;
    for (int i = 0; i < 3; ++i) A.xs[i] = t[0].stride(i), A.os[i] = t[3].stride(i);
    for (int i = 0; i < 2; ++i) A.ps[i] = t[1].stride(i);
    A.fs = t[2].stride(0);
    A.tokens = (uint32_t)(b * n);
    A.items = (uint32_t)items;
    A.tb = tokens_per_group(A.tokens, items, m);
    A.mscale = mscale;
    A.inverse = inverse != 0;
    A.by_t = Div31((uint32_t)n);
    A.by_head_items = Div31((uint32_t)per_head);
    A.by_token_items = Div31(A.items);
    return launched(launch_rope(type, layout, head_edge(type, layout, A.pairs, A.width),
                                (uint64_t)A.tokens * 2 * (h * d) * type_size(dt) > kPastCaches, A,
                                ceil_div(A.tokens, A.tb), turn_lds(A.tb, A.pairs), hip_stream),
                    "rope");
}

int cmd_rope_append(const cmd_arg args[10], int32_t layout, double mscale, int32_t flags, void *hip_stream)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    TRY(check_flags(flags));
    TRY(check_layout(layout, mscale));
    const int dt = args[0].dtype;
    TRY(check_float(dt, "q"));
    Tensor t[10];
    static const char *const names[10] = {"q", "k", "v", "pos", "row", "pages", "freq", "q_out", "k_cache", "v_cache"};
    static const int ranks[10] = {3, 3, 3, 1, 1, 2, 1, 3, 4, 4};
    for (int i = 0; i < 10; ++i)
        TRY(check(t[i], args[i], ranks[i], i >= 3 && i <= 5 ? CMD_I32 : i == 6 ? CMD_F64 : dt, names[i]));
    const int64_t tokens = t[0].size(0), hq = t[0].size(1), d = t[0].size(2), hk = t[1].size(1), dv = t[2].size(2);
    const int64_t m = t[6].size(0), pages = t[8].size(0), page = t[8].size(1);
    for (int i = 1; i <= 4; ++i) TRY(check_size(t[i], 0, tokens, "q"));
    TRY(check_size(t[1], 2, d, "q"));
    TRY(check_size(t[2], 1, hk, "k"));
    for (int i = 0; i < 3; ++i) TRY(check_size(t[7], i, t[0].size(i), "q"));
    TRY(check_size(t[8], 2, hk, "k"));
    TRY(check_size(t[8], 3, d, "k"));
    TRY(check_size(t[9], 0, pages, "k_cache"));
    TRY(check_size(t[9], 1, page, "k_cache"));
    TRY(check_size(t[9], 2, hk, "v"));
    TRY(check_size(t[9], 3, dv, "v"));
    if (2 * m > d)
        return refuse(CMD_E_SHAPE, "%lld frequencies turn %lld elements of a head of %lld", (long long)m,
                      (long long)(2 * m), (long long)d);
    if (m > kMaxPairs) return refuse(CMD_E_LIMIT, "more than %lld frequencies", (long long)kMaxPairs);
    for (int i : {0, 1, 2, 7, 8, 9}) TRY(check_unit(t[i]));
    static const int share[10] = {-1, -1, -1, -1, -1, -1, -1, 0, -1, -1};
    TRY(check_outputs(t, 10, 7, share));
    const int type = serving_type(dt);
    AppendArgs A{};
    const uint32_t e = type == S_F32 ? 4 : 8;
    const uint64_t per_qk = head_items(type, layout, (uint32_t)m, (uint32_t)d), per_v = ceil_div(dv, e);
    const uint64_t items = per_qk * (uint64_t)(hq + hk) + per_v * (uint64_t)hk;
    if (items > (uint64_t)kMaxCount / 2) return refuse(CMD_E_LIMIT, "q, k and v: a token has too many elements");
    if ((flags & CMD_CHECK_ONLY) || tokens == 0 || items == 0) return CMD_OK;
    A.q = args[0].ptr;
    A.k = args[1].ptr;
    A.v = args[2].ptr;
    A.pos = (const int32_t *)args[3].ptr;
    A.row = (const int32_t *)args[4].ptr;
    A.pages = (const int32_t *)args[5].ptr;
    A.freq = (const double *)args[6].ptr;
    A.q_out = args[7].ptr;
    A.k_cache = args[8].ptr;
    A.v_cache = args[9].ptr;
    for (int i = 0; i < 2; ++i) {
        A.qs[i] = t[0].stride(i);
        A.ks[i] = t[1].stride(i);
        A.vs[i] = t[2].stride(i);
        A.qos[i] = t[7].stride(i);
        A.pages_s[i] = t[5].stride(i);
    }
    for (int i = 0; i < 3; ++i) A.kcs[i] = t[8].stride(i), A.vcs[i] = t[9].stride(i);
    A.pos_s = t[3].stride(0);
    A.row_s = t[4].stride(0);
    A.fs = t[6].stride(0);
    A.tokens = (uint32_t)tokens;
    A.pairs = (uint32_t)m;
    A.d = (uint32_t)d;
    A.dv = (uint32_t)dv;
    A.hq = (uint32_t)hq;
    A.hk = (uint32_t)hk;
    A.n = page ? (uint32_t)pages : 0;
    A.page = (uint32_t)std::max<int64_t>(1, page);
    A.rows = (uint32_t)t[5].size(0);
    A.cols = (uint32_t)t[5].size(1);
    A.mscale = mscale;
    A.tb = tokens_per_group(A.tokens, items, m);
    // few tokens: several work-groups to a token
    A.parts = A.tb > 1 ? 1 : std::max(1u, std::min(ceil_div(items, 256), 1024 / A.tokens));
    A.by_page = Div31(A.page);
    auto div = [](uint64_t n) { return Div31((uint32_t)n); };
    A.by_q = div(per_qk * hq);
    A.by_k = div(per_qk * hk);
    A.by_v = div(per_v * hk);
    A.by_qk_head = div(per_qk);
    A.by_v_head = div(per_v);
    A.by_parts = Div31(A.parts);
    const uint64_t grid = (uint64_t)ceil_div(A.tokens, A.tb) * A.parts;
    const int edge = std::max(head_edge(type, layout, A.pairs, A.d), A.dv % e == 0 ? 0 : A.dv >= e ? 1 : 2);
    const bool past = (uint64_t)A.tokens * 2 * ((hq + hk) * d + hk * dv) * type_size(dt) > kPastCaches;
    return launched(launch_append(type, layout, edge, past, A, (uint32_t)grid, turn_lds(A.tb, A.pairs) + A.tb * 16,
                                  hip_stream),
                    "rope_append");
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Paged attention.

namespace {

struct AttnPlan {
    Tensor t[7];
    AttnArgs A;
    int type;
    int64_t workspace;
    bool nothing;
};

// apart: pages [B, hk, P] and lens [B, hk], a table for every kv head.
int plan_attention(const cmd_arg *args, int32_t window, bool apart, AttnPlan &P)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    Tensor *t = P.t;
    const int dt = args[0].dtype;
    TRY(check_float(dt, "q"));
    TRY(check(t[0], args[0], 3, dt, "q"));
    TRY(check(t[1], args[1], 4, dt, "k_cache"));
    TRY(check(t[2], args[2], 4, dt, "v_cache"));
    TRY(check(t[3], args[3], apart ? 3 : 2, CMD_I32, "pages"));
    TRY(check(t[4], args[4], apart ? 2 : 1, CMD_I32, "lens"));
    TRY(check(t[5], args[5], 3, dt, "out"));
    if (args[6].kind != 0) TRY(check(t[6], args[6], 2, CMD_F32, "lse"));
    const int64_t sequences = t[0].size(0), d = t[0].size(2), dv = t[2].size(3);
    const int64_t n = t[1].size(0), page = t[1].size(1), cols = t[3].size(apart ? 2 : 1);
    int64_t b = sequences, hq = t[0].size(1), hk = t[1].size(2);
    TRY(check_size(t[1], 3, d, "q"));
    for (int i = 0; i < 3; ++i) TRY(check_size(t[2], i, t[1].size(i), "k_cache"));
    TRY(check_size(t[3], 0, b, "q"));
    TRY(check_size(t[4], 0, b, "q"));
    if (apart) {
        TRY(check_size(t[3], 1, hk, "k_cache"));
        TRY(check_size(t[4], 1, hk, "k_cache"));
    }
    TRY(check_size(t[5], 0, b, "q"));
    TRY(check_size(t[5], 1, hq, "q"));
    TRY(check_size(t[5], 2, dv, "v_cache"));
    if (t[6].a) {
        TRY(check_size(t[6], 0, b, "q"));
        TRY(check_size(t[6], 1, hq, "q"));
    }
    if (hk == 0 ? hq != 0 : hq % hk != 0)
        return refuse(CMD_E_SHAPE, "%lld query heads are no multiple of %lld kv heads", (long long)hq, (long long)hk);
    if (d < 1 || dv < 1) return refuse(CMD_E_SHAPE, "heads of width 0");
    if (d > 256 || dv > 256) return refuse(CMD_E_LIMIT, "heads wider than 256");
    if (window < 0) return refuse(CMD_E_ARG, "negative window");
    for (int i : {0, 1, 2, 5}) TRY(check_unit(t[i]));
    TRY(check_outputs(t, 7, 5, nullptr));
    if (cols * std::max<int64_t>(page, 1) > (int64_t(1) << 30))
        return refuse(CMD_E_LIMIT, "the table holds more than 2^30 positions");
    AttnArgs &A = P.A;
    A = AttnArgs{};
    P.type = serving_type(dt);
    P.workspace = 0;
    P.nothing = b == 0 || hq == 0;
    if (P.nothing) return CMD_OK;
    const int64_t esize = type_size(dt);
    A.q = args[0].ptr;
    A.k = args[1].ptr;
    A.v = args[2].ptr;
    A.pages = (const int32_t *)args[3].ptr;
    A.lens = (const int32_t *)args[4].ptr;
    A.out = args[5].ptr;
    A.lse = t[6].a ? (float *)args[6].ptr : nullptr;
    for (int i = 0; i < 2; ++i) {
        A.qs[i] = t[0].stride(i);
        A.os[i] = t[5].stride(i);
        A.ls[i] = t[6].a ? t[6].stride(i) : 0;
    }
    A.pages_s[0] = t[3].stride(0);
    A.pages_s[1] = t[3].stride(apart ? 2 : 1);
    A.pages_s[2] = apart ? t[3].stride(1) : 0;
    A.lens_s[0] = t[4].stride(0);
    A.lens_s[1] = apart ? t[4].stride(1) : 0;
    A.apart = 1;
    A.apart_tables = apart;
    if (apart) {   // from here on each kv head of a sequence is a row
        if (b * hk > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
        A.apart = (uint32_t)hk;
        b *= hk;
        hq /= hk;
        hk = 1;
    }
    A.by_apart = Div31(A.apart);
    for (int i = 0; i < 3; ++i) {
        A.kcs[i] = t[1].stride(i) * esize;
        A.vcs[i] = t[2].stride(i) * esize;
    }
    A.b = (uint32_t)b;
    A.hq = (uint32_t)hq;
    A.hk = (uint32_t)hk;
    A.d = (uint32_t)d;
    A.dv = (uint32_t)dv;
    A.group = (uint32_t)(hq / hk);
    A.head_tiles = ceil_div(A.group, 16);
    A.n = (uint32_t)n;
    A.page = (uint32_t)std::max<int64_t>(1, page);
    A.cols = n > 0 && page > 0 ? (uint32_t)cols : 0;   // a cache without slots: every row is empty
    A.window = (uint32_t)window;
    A.by_page = Div31(A.page);
    const uint64_t heads = (uint64_t)A.hk * A.head_tiles;
    if ((uint64_t)(b + 8) * heads > kMaxGroups || (uint64_t)b * hq > (uint64_t)kMaxCount)
        return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
    uint64_t keys = (uint64_t)A.cols * A.page;
    if (window) keys = std::min<uint64_t>(keys, (uint64_t)window);
    const uint64_t steps = (keys + kAttnStep - 1) / kAttnStep, most = std::max<uint64_t>(1, steps * (uint64_t)b);
    // One work-group to a row and head, without a join, where the longest row that
    // the table can hold takes one no longer than cutting it does with the second
    // launch: 600 positions of 512 bytes 10.2 us against 11.0, 777 12.8 against
    // 12.0, binary32's 300 of 1024 bytes 12.7 against 13.2; with many rows twice that.
    const uint64_t row_bytes = keys * (uint64_t)((d + dv) * esize);
    A.direct = (steps <= 6 && row_bytes <= (256 << 10)) ||
               (steps <= 8 && row_bytes <= (512 << 10) && (uint64_t)b * heads >= 512) || b > kAttnMaxRows ||
               most > (uint64_t(1) << 30);
    // Runs for three work-groups on each of 256 compute units (what registers
    // allow at the common widths), but no more than there can be steps.  64 ragged
    // rows: 191 us with 512 or 768 work-groups, 196 with 1024, 209 with 2304.
    A.head_shift = heads % 4 == 0 ? 2 : heads % 2 == 0 ? 1 : 0;
    const uint64_t much = heads >> A.head_shift;
    auto runs = [&](uint64_t work_groups, uint64_t per_run) {
        return (uint32_t)std::min(std::max<uint64_t>(1, work_groups / per_run), std::min<uint64_t>(most, kAttnMaxRuns));
    };
    A.runs = runs(768, heads);
    A.runs_much = runs(768, much);
    A.runs_most = std::max(A.runs, A.runs_much);
    A.by_heads = Div31((uint32_t)(8 * heads));
    A.by_heads_much = Div31((uint32_t)(8 * much));
    A.by_tiles = Div31(A.head_tiles);
    A.by_runs = Div31(A.runs);
    A.by_runs_much = Div31(A.runs_much);
    // With 128 work-groups or more (a compute unit alone reads 55 to 70 GB/s of 6
    // TB/s) rows may be taken whole; many more than needed would only start and end.
    A.runs_whole = (uint64_t)b * heads >= 128 && (uint64_t)b * heads <= 2048 ? (uint32_t)b : 0;
    auto eight = [](uint64_t n) { return (n + 7) / 8 * 8; };
    A.grid = (uint32_t)(A.direct ? eight(b) * heads : std::max(eight(std::max(A.runs, A.runs_whole)) * heads, eight(A.runs_much) * much));
    // Reads that nothing can find in a 256 MiB cache again pass it by: 1138 MB in
    // 64 ragged rows 206 us against 218; 262 MB that it can hold 56 against 48.
    A.stream = (t[1].span() + t[2].span()) > (int64_t(1) << 28);
    // Many segments to few rows: two rows of 262143 positions are joined by 1024
    // work-items to 32 columns in 5.7 us, by 256 to a row in 14.8; 8 rows of 2000 take
    // 28.7 us with the former and 21.3 with a wave to a row; 8 ragged rows of up to
    // 6263, 3 kv heads, 22 us with a wave to a row and 16 with 256 work-items
    // to 32 columns.
    const uint64_t segments = std::min<uint64_t>(A.runs_most, steps);   // of a row, at most
    A.join = segments <= 16 ? 0 : (uint64_t)b * hq * ((dv + 31) / 32) <= 512 ? 2 : A.runs_most > 12 * (uint64_t)b ? 1 : 0;
    // (work-groups of 1024 join only what is little)
    if (!A.direct && (uint64_t)b * hq > kMaxGroups) return refuse(CMD_E_LIMIT, "too many sequences times heads for one launch");
    if (!A.direct) P.workspace = (int64_t)(((uint64_t)A.runs_most + b) * hq * (dv + 2) * 4 + 16);
    return CMD_OK;
}

}  // namespace

extern "C" {

static int64_t attention_workspace(const cmd_arg *args, int32_t window, bool apart)
{
    AttnPlan P;
    const int rc = plan_attention(args, window, apart, P);
    return rc ? rc : P.workspace;
}

static int attention(const cmd_arg *args, float scale, int32_t window, bool apart, void *workspace,
                     int64_t workspace_bytes, int32_t flags, void *hip_stream)
{
    TRY(check_flags(flags));
    AttnPlan P;
    TRY(plan_attention(args, window, apart, P));
    const float scale_log2 = (float)((double)scale * 1.44269504088896340736);
    if (!std::isfinite(scale_log2)) return refuse(CMD_E_ARG, "scale is not finite, or too large for binary32 in base 2");
    if (flags & CMD_CHECK_ONLY) return CMD_OK;
    if (P.nothing) return CMD_OK;
    TRY(check_workspace(workspace, workspace_bytes, P.workspace));
    AttnArgs &A = P.A;
    A.scale_log2 = scale_log2;
    if (!A.direct) {
        A.ml = (float *)workspace;
        A.acc = A.ml + ((((uint64_t)A.runs_most + A.b) * A.hq * 2 + 3) & ~uint64_t(3));
    }
    const int rc = P.type == S_F16    ? launch_attention_f16(A, hip_stream)
                   : P.type == S_BF16 ? launch_attention_bf16(A, hip_stream)
                                      : launch_attention_f32(A, hip_stream);
    TRY(launched(rc, "paged_attention"));
    if (A.direct) return CMD_OK;
    return launched(P.type == S_F16    ? launch_attention_join_f16(A, hip_stream)
                    : P.type == S_BF16 ? launch_attention_join_bf16(A, hip_stream)
                                       : launch_attention_join_f32(A, hip_stream),
                    "paged_attention join");
}

int64_t cmd_paged_attention_workspace(const cmd_arg args[7], int32_t window)
{
    return attention_workspace(args, window, false);
}

int cmd_paged_attention(const cmd_arg args[7], float scale, int32_t window, void *workspace, int64_t workspace_bytes,
                        int32_t flags, void *hip_stream)
{
    return attention(args, scale, window, false, workspace, workspace_bytes, flags, hip_stream);
}

int64_t cmd_paged_attention_heads_workspace(const cmd_arg args[7], int32_t window)
{
    return attention_workspace(args, window, true);
}

int cmd_paged_attention_heads(const cmd_arg args[7], float scale, int32_t window, void *workspace,
                              int64_t workspace_bytes, int32_t flags, void *hip_stream)
{
    return attention(args, scale, window, true, workspace, workspace_bytes, flags, hip_stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Pages.

namespace {

// Tiles of at least 16 words, at most kMaxPageTiles of them.  Returns the bytes
// of the bits, prefixes and counts.
int64_t plan_bits(PageBits &B, int64_t n)
{
    B = PageBits{};
    B.n = (uint32_t)n;
    if (n == 0) return 0;
    B.tile_shift = 4;
    while (ceil_div((uint64_t)n, uint64_t(64) << B.tile_shift) > kMaxPageTiles) ++B.tile_shift;
    B.tile_words = 1u << B.tile_shift;
    B.tiles = ceil_div((uint64_t)n, uint64_t(64) << B.tile_shift);
    return (int64_t)B.tiles * B.tile_words * 12 + (int64_t)B.tiles * 4;
}

char *place_bits(PageBits &B, char *ws)
{
    const uint64_t words = (uint64_t)B.tiles * B.tile_words;
    B.word = (uint64_t *)ws;
    B.word_prefix = (uint32_t *)(ws + words * 8);
    B.tile_count = (uint32_t *)(ws + words * 12);
    return ws + words * 12 + (uint64_t)B.tiles * 4;
}

struct AssignPlan {
    AssignArgs A;
    int64_t workspace;
};

int plan_assign(const cmd_arg *args, int32_t page, AssignPlan &P)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    static const char *const names[11] = {"pages", "lens", "refs", "parent", "add", "pages_out",
                                          "lens_out", "refs_out", "src", "dst", "stats"};
    Tensor t[11];
    for (int i = 0; i < 11; ++i) TRY(check(t[i], args[i], i == 0 || i == 5 ? 2 : 1, CMD_I32, names[i]));
    const int64_t rows = t[0].size(0), cols = t[0].size(1), n = t[2].size(0);
    for (int i : {1, 3, 4, 6, 8, 9}) TRY(check_size(t[i], 0, rows, "pages"));
    TRY(check_size(t[5], 0, rows, "pages"));
    TRY(check_size(t[5], 1, cols, "pages"));
    TRY(check_size(t[7], 0, n, "refs"));
    TRY(check_size(t[10], 0, 2, "the two counts"));
    if (page < 1) return refuse(CMD_E_ARG, "pages of %d slots", page);
    if ((cols + 1) * (int64_t)page > kMaxCount) return refuse(CMD_E_LIMIT, "the table holds more than 2^31 positions");
    if (rows * cols > kMaxCount) return refuse(CMD_E_LIMIT, "the table has more than 2^31 - 1 entries");
    if (rows > (int64_t)kMaxGroups) return refuse(CMD_E_LIMIT, "the table has too many rows for one launch");
    static const int share[11] = {-1, -1, -1, -1, -1, -1, -1, 2, -1, -1, -1};
    TRY(check_outputs(t, 11, 5, share));
    AssignArgs &A = P.A;
    A = AssignArgs{};
    A.pages = (const int32_t *)args[0].ptr;
    A.lens = (const int32_t *)args[1].ptr;
    A.refs = (const int32_t *)args[2].ptr;
    A.parent = (const int32_t *)args[3].ptr;
    A.add = (const int32_t *)args[4].ptr;
    A.pages_out = (int32_t *)args[5].ptr;
    A.lens_out = (int32_t *)args[6].ptr;
    A.refs_out = (int32_t *)args[7].ptr;
    A.src = (int32_t *)args[8].ptr;
    A.dst = (int32_t *)args[9].ptr;
    A.stats = (int32_t *)args[10].ptr;
    for (int i = 0; i < 2; ++i) A.pages_s[i] = t[0].stride(i), A.pages_out_s[i] = t[5].stride(i);
    A.lens_s = t[1].stride(0);
    A.refs_s = t[2].stride(0);
    A.parent_s = t[3].stride(0);
    A.add_s = t[4].stride(0);
    A.lens_out_s = t[6].stride(0);
    A.refs_out_s = t[7].stride(0);
    A.src_s = t[8].stride(0);
    A.dst_s = t[9].stride(0);
    A.stats_s = t[10].stride(0);
    A.rows = (uint32_t)rows;
    A.cols = (uint32_t)cols;
    A.page = (uint32_t)page;
    A.by_page = Div31(A.page);
    A.by_cols = Div31(std::max(1u, A.cols));
    A.row_groups = ceil_div(A.rows, 256);
    P.workspace = plan_bits(A.bits, n) + (int64_t)A.rows * 4 + (int64_t)A.row_groups * 4;
    A.small = n <= kSmallPages && rows <= kSmallRows && rows * cols <= kSmallEntries;
    if (A.small) P.workspace = 0;
    return CMD_OK;
}

struct CompactPlan {
    CompactArgs A;
    int64_t workspace;
};

int plan_compact(const cmd_arg *args, CompactPlan &P)
{
    if (!args) return refuse(CMD_E_ARG, "args is NULL");
    static const char *const names[7] = {"pages", "refs", "pages_out", "refs_out", "src", "dst", "stats"};
    Tensor t[7];
    for (int i = 0; i < 7; ++i) TRY(check(t[i], args[i], i == 0 || i == 2 ? 2 : 1, CMD_I32, names[i]));
    const int64_t rows = t[0].size(0), cols = t[0].size(1), n = t[1].size(0);
    for (int i = 0; i < 2; ++i) TRY(check_size(t[2], i, t[0].size(i), "pages"));
    TRY(check_size(t[3], 0, n, "refs"));
    if (t[4].size(0) < n / 2)
        return refuse(CMD_E_SHAPE, "src has %lld entries, at least %lld needed", (long long)t[4].size(0),
                      (long long)(n / 2));
    TRY(check_size(t[5], 0, t[4].size(0), "src"));
    TRY(check_size(t[6], 0, 2, "the two counts"));
    if (rows * cols > kMaxCount) return refuse(CMD_E_LIMIT, "the table has more than 2^31 - 1 entries");
    if ((uint64_t)ceil_div(rows * cols, 256) + ceil_div(std::max(n, t[4].size(0)), 256) > kMaxGroups)
        return refuse(CMD_E_LIMIT, "too many pages and entries for one launch");
    static const int share[7] = {-1, -1, 0, -1, -1, -1, -1};
    TRY(check_outputs(t, 7, 2, share));
    CompactArgs &A = P.A;
    A = CompactArgs{};
    A.pages = (const int32_t *)args[0].ptr;
    A.refs = (const int32_t *)args[1].ptr;
    A.pages_out = (int32_t *)args[2].ptr;
    A.refs_out = (int32_t *)args[3].ptr;
    A.src = (int32_t *)args[4].ptr;
    A.dst = (int32_t *)args[5].ptr;
    A.stats = (int32_t *)args[6].ptr;
    for (int i = 0; i < 2; ++i) A.pages_s[i] = t[0].stride(i), A.pages_out_s[i] = t[2].stride(i);
    A.refs_s = t[1].stride(0);
    A.refs_out_s = t[3].stride(0);
    A.src_s = t[4].stride(0);
    A.dst_s = t[5].stride(0);
    A.stats_s = t[6].stride(0);
    A.rows = (uint32_t)rows;
    A.cols = (uint32_t)cols;
    A.capacity = (uint32_t)t[4].size(0);
    A.by_cols = Div31(std::max(1u, A.cols));
    P.workspace = plan_bits(A.bits, n);
    A.small = n <= kSmallPages && A.capacity <= kSmallPages && rows * cols <= kSmallEntries;
    if (A.small) P.workspace = 0;
    return CMD_OK;
}

// How a page of a pool is copied: rows of `inner` bytes, `row_stride` apart.
struct PageShape {
    int64_t rows = 1, inner = 0, row_stride = 0;
};

int page_shape(const Tensor &t, PageShape &S)
{
    int order[3], n = 0;
    for (int i = 1; i < 4; ++i)
        if (t.size(i) > 1) order[n++] = i;
    std::sort(order, order + n, [&](int x, int y) { return t.stride(x) < t.stride(y); });
    int64_t run = 1;   // elements of the innermost dense run
    int k = 0;
    for (; k < n && t.stride(order[k]) == run; ++k) run *= t.size(order[k]);
    const int e = type_size(t.a->dtype);
    S.inner = run * e;
    S.rows = 1;
    S.row_stride = 0;
    if (k < n) {
        S.row_stride = t.stride(order[k]) * e;
        S.rows = t.size(order[k]);
        for (++k; k < n; ++k) {
            if (t.stride(order[k]) * e != S.row_stride * S.rows)
                return refuse(CMD_E_STRIDE, "%s: a page is more than rows at one distance", t.name);
            S.rows *= t.size(order[k]);
        }
    }
    return CMD_OK;
}

}  // namespace

extern "C" {

int64_t cmd_page_assign_workspace(const cmd_arg args[11], int32_t page)
{
    AssignPlan P;
    const int rc = plan_assign(args, page, P);
    return rc ? rc : P.workspace;
}

int cmd_page_assign(const cmd_arg args[11], int32_t page, void *workspace, int64_t workspace_bytes, int32_t flags,
                    void *hip_stream)
{
    TRY(check_flags(flags));
    AssignPlan P;
    TRY(plan_assign(args, page, P));
    if (flags & CMD_CHECK_ONLY) return CMD_OK;
    TRY(check_workspace(workspace, workspace_bytes, P.workspace));
    char *at = place_bits(P.A.bits, (char *)workspace);
    P.A.want = (uint32_t *)at;
    P.A.want_group = P.A.want + P.A.rows;
    return launched(launch_assign(P.A, hip_stream), "page_assign");
}

int64_t cmd_page_compact_workspace(const cmd_arg args[7])
{
    CompactPlan P;
    const int rc = plan_compact(args, P);
    return rc ? rc : P.workspace;
}

int cmd_page_compact(const cmd_arg args[7], void *workspace, int64_t workspace_bytes, int32_t flags, void *hip_stream)
{
    TRY(check_flags(flags));
    CompactPlan P;
    TRY(plan_compact(args, P));
    if (flags & CMD_CHECK_ONLY) return CMD_OK;
    TRY(check_workspace(workspace, workspace_bytes, P.workspace));
    place_bits(P.A.bits, (char *)workspace);
    return launched(launch_compact(P.A, hip_stream), "page_compact");
}

int cmd_page_copy(const cmd_arg *pools, int32_t npools, const cmd_arg *src, const cmd_arg *dst, int32_t flags,
                  void *hip_stream)
{
    TRY(check_flags(flags));
    if (npools < 0 || (npools && !pools) || !src || !dst) return refuse(CMD_E_ARG, "pools, src or dst is NULL");
    Tensor s, d;
    TRY(check(s, *src, 1, CMD_I32, "src"));
    TRY(check(d, *dst, 1, CMD_I32, "dst"));
    TRY(check_size(d, 0, s.size(0), "src"));
    const int64_t count = s.size(0);
    // Two passes: everything is checked before the first launch.
    for (int pass = 0; pass < 2; ++pass) {
        CopyArgs A{};
        int held = 0, width = 0;
        uint32_t vecs = 0;
        auto flush = [&]() -> int {
            if (!held) return CMD_OK;
            A.src = (const int32_t *)src->ptr;
            A.dst = (const int32_t *)dst->ptr;
            A.src_s = s.stride(0);
            A.dst_s = d.stride(0);
            A.count = (uint32_t)count;
            A.per_group = vecs < 256 ? 256 / vecs : 1;
            A.pieces = A.per_group > 1 ? 1 : ceil_div(vecs, 1024);
            A.by_pieces = Div31(A.pieces);
            A.by_vecs = Div31(vecs);
            const uint64_t grid = A.per_group > 1 ? ceil_div(A.count, A.per_group) : (uint64_t)A.count * A.pieces;
            if (grid > kMaxGroups) return refuse(CMD_E_LIMIT, "too many pairs for pages of this size");
            const int n = held;
            held = 0;
            const bool past = (uint64_t)count * n * 2 * vecs * width > kPastCaches;
            if (pass == 0) return CMD_OK;
            return launched(launch_copy(width, past, A, (uint32_t)n, (uint32_t)grid, hip_stream), "page_copy");
        };
        for (int i = 0; i < npools; ++i) {
            Tensor t;
            char name[32];
            snprintf(name, sizeof name, "pool %d", i);
            const int dt = pools[i].dtype;
            if (dt != CMD_F16 && dt != CMD_BF16 && dt != CMD_F32 && dt != CMD_I32)
                return refuse(CMD_E_DTYPE, "%s has an unknown dtype %d", name, dt);
            TRY(check(t, pools[i], 4, dt, name));
            if (pass == 0) {
                TRY(check_one_to_one(t));
                if (!disjoint(s, t)) return refuse(CMD_E_ALIAS, "%s overlaps src", name);
                if (!disjoint(d, t)) return refuse(CMD_E_ALIAS, "%s overlaps dst", name);
            }
            PageShape S;
            TRY(page_shape(t, S));
            if (t.empty() || count == 0) continue;
            const int e = type_size(dt);
            const uint64_t page_stride = (uint64_t)t.stride(0) * e;
            // the widest vector that divides the rows and starts aligned in every page
            int w = 16;
            const uint64_t all = (uint64_t)t.begin() | page_stride | (uint64_t)S.inner | (uint64_t)S.row_stride;
            while (w > e && all % w) w /= 2;
            if (S.rows * (S.inner / w) > kMaxCount / 2) return refuse(CMD_E_LIMIT, "%s: a page is too large", name);
            const uint32_t v = (uint32_t)(S.rows * (S.inner / w));
            if (held && (w != width || v != vecs || held == kCopyPools)) TRY(flush());
            width = w;
            vecs = v;
            CopyPool &p = A.pool[held++];
            p.base = (char *)t.a->ptr;
            p.page_stride = (int64_t)page_stride;
            p.row_stride = S.row_stride;
            p.n = (uint32_t)t.size(0);
            p.vecs = v;
            p.row_vecs = (uint32_t)(S.inner / w);
            p.by_row = Div31(p.row_vecs);
        }
        TRY(flush());
        if (flags & CMD_CHECK_ONLY) return CMD_OK;
    }
    return CMD_OK;
}

}  // extern "C"
