// ecmd_serving_check.h -- the serving operators' argument checks (host code; each
// of their translation units has its own copy).  Nothing here makes a HIP call,
// allocates or throws.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../../include/ecmd_serving.h"
#include "../ecmd_command.h"
#include "../ecmd_launch.h"
#include "ecmd_serving.h"

namespace ecmd {

namespace {

int refuse(int code, const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    try {
        set_create_error(buf);
    } catch (...) {   // no memory for the message: the status stands alone
    }
    return code;
}

int launched(int herr, const char *what)
{
    if (herr == 0) return CMD_OK;
    return refuse(CMD_E_LAUNCH, "%s launch failed: %s", what, hipGetErrorString((hipError_t)herr));
}

const char *type_name(int d)
{
    return d == CMD_F16 ? "f16" : d == CMD_F32 ? "f32" : d == CMD_I32 ? "i32" : d == CMD_BF16 ? "bf16"
           : d == CMD_F64 ? "f64" : "?";
}
int type_size(int d) { return d == CMD_F64 ? 8 : d == CMD_F16 || d == CMD_BF16 ? 2 : 4; }

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;   // sizes and counts that kernels hold in 32 bits

// One tensor argument.
struct Tensor {
    const cmd_arg *a = nullptr;
    int rank = 0;
    const char *name = "";

    int64_t size(int i) const { return a->size[i]; }
    int64_t stride(int i) const { return a->size[i] == 1 ? 0 : a->stride[i]; }
    bool empty() const
    {
        for (int i = 0; i < rank; ++i)
            if (a->size[i] == 0) return true;
        return false;
    }
    // bytes from the first element's start to the last one's end
    int64_t span() const
    {
        if (empty()) return 0;
        int64_t e = 0;
        for (int i = 0; i < rank; ++i) e += (a->size[i] - 1) * a->stride[i];
        return (e + 1) * type_size(a->dtype);
    }
    uintptr_t begin() const { return (uintptr_t)a->ptr; }
    uintptr_t end() const { return begin() + (uintptr_t)span(); }
};

int check(Tensor &t, const cmd_arg &a, int rank, int dtype, const char *name)
{
    t = Tensor{&a, rank, name};
    if (a.kind != CMD_ARG_TENSOR) return refuse(CMD_E_ARG, "%s is not a tensor argument", name);
    if (a.dtype != dtype)
        return refuse(CMD_E_DTYPE, "%s has dtype %s, %s expected", name, type_name(a.dtype), type_name(dtype));
    int64_t reach = 1;
    for (int i = 0; i < rank; ++i) {
        if (a.size[i] < 0) return refuse(CMD_E_SHAPE, "%s does not have %d dimensions", name, rank);
        if (a.size[i] > kMaxCount)
            return refuse(CMD_E_LIMIT, "%s: dimension %d has %lld elements", name, i, (long long)a.size[i]);
    }
    if (!t.empty())
        for (int i = 0; i < rank; ++i) {
            if (a.size[i] <= 1) continue;
            if (a.stride[i] < 0) return refuse(CMD_E_STRIDE, "%s: negative stride in dimension %d", name, i);
            // 2^56 elements: keeps every later sum of products within 64 bits
            if (a.stride[i] > ((int64_t(1) << 56) - reach) / a.size[i])
                return refuse(CMD_E_LIMIT, "%s spans more than 2^56 elements", name);
            reach += (a.size[i] - 1) * a.stride[i];
        }
    if (!t.empty() && !a.ptr) return refuse(CMD_E_ARG, "%s is NULL", name);
    if (!t.empty() && (uintptr_t)a.ptr % type_size(dtype))
        return refuse(CMD_E_ARG, "%s is not aligned to its elements", name);
    return CMD_OK;
}

int check_float(int dtype, const char *name)
{
    if (dtype == CMD_F16 || dtype == CMD_BF16 || dtype == CMD_F32) return CMD_OK;
    return refuse(CMD_E_DTYPE, "%s has dtype %s; f16, bf16 or f32 expected", name, type_name(dtype));
}
int serving_type(int dtype) { return dtype == CMD_F16 ? S_F16 : dtype == CMD_BF16 ? S_BF16 : S_F32; }

// The last dimension's elements are neighbours.
int check_unit(const Tensor &t)
{
    if (t.size(t.rank - 1) > 1 && t.stride(t.rank - 1) != 1)
        return refuse(CMD_E_STRIDE, "%s: the last dimension's stride is %lld, 1 expected", t.name,
                      (long long)t.stride(t.rank - 1));
    return CMD_OK;
}

int check_size(const Tensor &t, int dim, int64_t want, const char *like)
{
    if (t.size(dim) == want) return CMD_OK;
    return refuse(CMD_E_SHAPE, "%s: dimension %d is %lld, %lld expected (%s)", t.name, dim, (long long)t.size(dim),
                  (long long)want, like);
}

// An output maps no two indexes to one element: each dimension, by ascending
// stride, steps past all the smaller ones.
int check_one_to_one(const Tensor &t)
{
    if (t.empty()) return CMD_OK;
    int order[4], n = 0;
    for (int i = 0; i < t.rank; ++i)
        if (t.size(i) > 1) order[n++] = i;
    std::sort(order, order + n, [&](int x, int y) { return t.stride(x) < t.stride(y); });
    int64_t reach = 0;
    for (int k = 0; k < n; ++k) {
        const int i = order[k];
        if (t.stride(i) <= reach)
            return refuse(CMD_E_STRIDE, "%s: an output view with overlapping elements (dimension %d, stride %lld)",
                          t.name, i, (long long)t.stride(i));
        reach += (t.size(i) - 1) * t.stride(i);
    }
    return CMD_OK;
}

bool identical(const Tensor &a, const Tensor &b)
{
    if (a.a->ptr != b.a->ptr || a.a->dtype != b.a->dtype || a.rank != b.rank) return false;
    for (int i = 0; i < a.rank; ++i)
        if (a.size(i) != b.size(i) || a.stride(i) != b.stride(i)) return false;
    return true;
}

// True if no byte belongs to both.  Beyond disjoint ranges, two views that step
// through memory in lockstep (slices of one packed tensor) are recognised: if
// for some period S every stride of both is either a multiple of S or, together
// with the other small ones, stays inside one period, the views compare modulo S.
bool disjoint(const Tensor &a, const Tensor &b)
{
    if (a.empty() || b.empty()) return true;
    if (a.end() <= b.begin() || b.end() <= a.begin()) return true;
    const int ea = type_size(a.a->dtype), eb = type_size(b.a->dtype);
    for (int k = 0; k < a.rank; ++k) {
        const int64_t S = a.stride(k) * ea;
        if (a.size(k) <= 1 || S <= 0) continue;
        int64_t small[2] = {ea, eb};
        bool ok = true;
        for (int w = 0; w < 2 && ok; ++w) {
            const Tensor &t = w ? b : a;
            const int e = w ? eb : ea;
            for (int i = 0; i < t.rank; ++i) {
                if (t.size(i) <= 1) continue;
                const int64_t s = t.stride(i) * e;
                if (s % S == 0) continue;
                if (s > S) {
                    ok = false;
                    break;
                }
                small[w] += (t.size(i) - 1) * s;
            }
        }
        if (!ok || small[0] > S || small[1] > S) continue;
        const int64_t delta = (int64_t)(((uintptr_t)b.begin() - a.begin()) % (uint64_t)S);
        const int64_t d = b.begin() >= a.begin()
                              ? delta
                              : (S - (int64_t)((a.begin() - b.begin()) % (uint64_t)S)) % S;
        if (d >= small[0] && d + small[1] <= S) return true;
    }
    return false;
}

// Outputs overlap nothing; may_share names the one input an output may be
// identical to (index into all, or -1).
int check_outputs(const Tensor *all, int n, int first_out, const int *may_share)
{
    for (int o = first_out; o < n; ++o) {
        if (!all[o].a) continue;
        if (int rc = check_one_to_one(all[o])) return rc;
        for (int i = 0; i < n; ++i) {
            if (i == o || !all[i].a || (i > o)) continue;
            if (may_share && may_share[o] == i && identical(all[i], all[o])) continue;
            if (!disjoint(all[i], all[o]))
                return refuse(CMD_E_ALIAS, "%s overlaps %s", all[o].name, all[i].name);
        }
    }
    return CMD_OK;
}

int check_flags(int32_t flags)
{
    if (flags & ~CMD_CHECK_ONLY) return refuse(CMD_E_ARG, "unknown flags %d", flags);
    return CMD_OK;
}

int check_workspace(void *ws, int64_t given, int64_t need)
{
    if (need == 0) return CMD_OK;
    if (!ws || given < need)
        return refuse(CMD_E_ARG, "the workspace has %lld bytes, %lld needed", (long long)(ws ? given : 0),
                      (long long)need);
    if ((uintptr_t)ws % 16) return refuse(CMD_E_ARG, "the workspace is not 16-byte aligned");
    return CMD_OK;
}

#define TRY(x)                \
    do {                      \
        if (int rc_ = (x)) return rc_; \
    } while (0)

uint32_t ceil_div(uint64_t a, uint64_t b) { return (uint32_t)((a + b - 1) / b); }

// Work-groups of 256 in one launch: a grid's work-items are a 32-bit count.
constexpr uint64_t kMaxGroups = (uint64_t(1) << 24) - 1;

// Reads and writes that displace more than the L2 caches' 32 MiB twice over go
// past the caches: 335 MB of a prompt's rope 66 -> 60 us, 212 MB of an append 52 ->
// 45 us; smaller ones leave their output where the next kernel finds it.
constexpr uint64_t kPastCaches = 64 << 20;

}  // namespace

}  // namespace ecmd
