"""Serving operators beside Commands: rotary positions, a paged key-value
cache, attention of one new token or of a tree of drafted tokens over it, the
pages worth reading or keeping, and the bookkeeping of its pages.

A thin layer over ``include/ecmd_serving.h``, which defines every
operator; outputs are the caller's tensors, work goes to torch's current stream
or ``stream``, errors are ``Error`` with the library's status and message, and
nothing is launched after a failed check.  Scratch memory is the caller's
``workspace`` (a contiguous GPU tensor of at least the matching
``*_workspace`` bytes) or, without one, taken from torch's allocator on the
launch's stream.  The version counters of what was written advance, as after
torch's in-place operations, so a backward pass does not take a tensor that was
saved before for what it was; no call records a gradient (``rope`` says how to
take its own).

A decode step of a model's attention:

    ecmd.page_assign(pages, lens, refs, parent, add, page, pages2, lens2, refs2, src, dst, stats)
    ecmd.page_copy([k_cache, v_cache], src, dst)                  # forked rows get their own last page
    ecmd.rope_append(q, k, v, pos, row, pages2, freq, q, k_cache, v_cache)
    ecmd.paged_attention(q, k_cache, v_cache, pages2, lens2, out)

The same that reads only the pages a cheap score selects for each kv head:

    ecmd.page_bounds(k_cache, pages2, lens2, lens, bounds)        # after the append: the new positions' keys
    ecmd.page_select(q, bounds, pages2, lens2, page, picked, picked_lens)
    ecmd.paged_attention(q, k_cache, v_cache, picked, picked_lens, out)

that keeps rows within a budget of pages, by the weight attention gave them:

    ecmd.page_mass(q, k_cache, pages2, lens2, lse, mass, mass, decay=0.95)
    ecmd.page_evict(pages2, lens2, refs2, mass, budget, page, pages2, refs2, count)

and that checks a tree of drafted tokens in one step (their keys and values appended
at positions lens + i):

    ecmd.tree_attention(q, k_cache, v_cache, pages, lens, parent, out)
    ecmd.tree_accept(tokens, parent, next, lens, path, lens2, last)
    ecmd.slot_move([k_cache, v_cache], pages, lens, path)         # the accepted ones to lens, lens + 1, ...

``decode.py`` in this package runs them end to end.
"""
from __future__ import annotations

import ctypes
import math

from . import Error, cmd_arg, lib

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
CHECK_ONLY = 1

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_args = ctypes.c_char_p      # packed cmd_arg structures
for _name, _res, _sig in [
        ("cmd_rope", ctypes.c_int, [_args, _i32, ctypes.c_double, _i32, _i32, _vp]),
        ("cmd_rope_append", ctypes.c_int, [_args, _i32, ctypes.c_double, _i32, _vp]),
        ("cmd_paged_attention", ctypes.c_int, [_args, ctypes.c_float, _i32, _vp, _i64, _i32, _vp]),
        ("cmd_paged_attention_workspace", _i64, [_args, _i32]),
        ("cmd_page_assign", ctypes.c_int, [_args, _i32, _vp, _i64, _i32, _vp]),
        ("cmd_page_assign_workspace", _i64, [_args, _i32]),
        ("cmd_page_compact", ctypes.c_int, [_args, _vp, _i64, _i32, _vp]),
        ("cmd_page_compact_workspace", _i64, [_args]),
        ("cmd_page_copy", ctypes.c_int, [_args, _i32, _args, _args, _i32, _vp]),
        ("cmd_paged_attention_heads", ctypes.c_int, [_args, ctypes.c_float, _i32, _vp, _i64, _i32, _vp]),
        ("cmd_paged_attention_heads_workspace", _i64, [_args, _i32]),
        ("cmd_tree_attention", ctypes.c_int, [_args, ctypes.c_float, _i32, _vp, _i64, _i32, _vp]),
        ("cmd_tree_attention_workspace", _i64, [_args, _i32]),
        ("cmd_tree_accept", ctypes.c_int, [_args, _i32, _vp]),
        ("cmd_slot_move", ctypes.c_int, [_args, _i32, _args, _i32, _vp]),
        ("cmd_page_bounds", ctypes.c_int, [_args, _i32, _vp]),
        ("cmd_page_select", ctypes.c_int, [_args, _i32, _i32, _i32, _vp, _i64, _i32, _vp]),
        ("cmd_page_select_workspace", _i64, [_args, _i32, _i32, _i32]),
        ("cmd_page_mass", ctypes.c_int, [_args, ctypes.c_float, ctypes.c_float, _i32, _i32, _vp]),
        ("cmd_page_evict", ctypes.c_int, [_args, _i32, _i32, _i32, _i32, _vp])]:
    getattr(lib, _name).restype = _res
    getattr(lib, _name).argtypes = _sig

_SIZE = ctypes.sizeof(cmd_arg)
_binding = None


def _pack(ranks: bytes, *tensors):
    """(cmd_arg structures of the tensors, their GPU if it is the current one or
    -1, its current stream's handle); see ecmd_binding.cpp."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401  (first: the module links against its libraries)
        try:
            from . import _binding as module
        except ImportError as e:
            raise ImportError("the binding of the serving operators is not built for this interpreter and torch (%s); "
                              "build it with `python elementwise_tensor_commands_amd/build.py`" % e) from e
        _binding = module
    return _binding.pack(ranks, *tensors)


def _check(rc: int):
    if rc < 0:
        raise Error(int(rc), lib.cmd_last_error(None).decode())


def _refuse(rc: int):
    """Tensors that are not all on the current GPU are an error, after the errors
    that the library found in them (its status rc with CHECK_ONLY)."""
    _check(rc)
    raise Error(-1, "every tensor must be on the current GPU")


def _handle(stream, device: int) -> int:
    if isinstance(stream, int):
        return stream
    at = getattr(stream, "device", None)
    if at is not None and at.index != device:
        raise Error(-1, "the stream belongs to another GPU")
    return getattr(stream, "cuda_stream", stream)


def _scratch(workspace, size: int, stream, device: int):
    """(pointer, bytes, owner) of the workspace: the caller's, or from the
    allocator of the launch's stream, which may hand the memory on once that
    stream is done with it."""
    _check(size)
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise Error(-1, "the workspace must be contiguous and on the current GPU")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if size == 0:
        return None, 0, None
    if stream is None:
        ptr, owner = _binding.scratch(size, device)
    else:
        import torch
        if isinstance(stream, int):   # of handle 0 ExternalStream would make a new stream
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            ptr, owner = _binding.scratch(size, device)
    return ptr, size, owner


def _layout(layout) -> int:
    return ROPE_LAYOUTS.get(layout, -1)


def _int32(x) -> int:
    """x for a C int32 argument; what does not fit becomes the nearest number that
    does, which the library refuses or which means the same."""
    return max(-1, min(int(x), 2 ** 31 - 1))


def rope(x, pos, freq, out, *, layout="half", mscale=1.0, inverse=False, stream=None):
    """Rotary positions (cmd_rope): x [b, t, h, d] turned by pos [b, t] (int32)
    into out, pair i by pos * freq[i] (freq: float64, on the GPU).  out may be
    x.  ``inverse`` is the transposed map: applied to the gradient of out it
    gives the gradient of x."""
    args, dev, current = _pack(b"\4\2\1\4", x, pos, freq, out)
    if dev < 0:
        _refuse(lib.cmd_rope(args, _layout(layout), mscale, bool(inverse), CHECK_ONLY, None))
    _check(lib.cmd_rope(args, _layout(layout), mscale, bool(inverse), 0,
                        current if stream is None else _handle(stream, dev)))
    _binding.wrote(out)


def rope_append(q, k, v, pos, row, pages, freq, q_out, k_cache, v_cache, *, layout="half", mscale=1.0, stream=None):
    """Rotary positions of packed tokens and the write into the cache
    (cmd_rope_append): q [T, hq, d] turned into q_out (which may be q), k [T,
    hk, d] turned and v [T, hk, dv] as it is into the slots of positions pos [T]
    of sequences row [T].  Tokens whose row, position or page is out of range
    are padding."""
    args, dev, current = _pack(b"\3\3\3\1\1\2\1\3\4\4", q, k, v, pos, row, pages, freq, q_out, k_cache, v_cache)
    if dev < 0:
        _refuse(lib.cmd_rope_append(args, _layout(layout), mscale, CHECK_ONLY, None))
    _check(lib.cmd_rope_append(args, _layout(layout), mscale, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(q_out, k_cache, v_cache)


_ATTENTION = b"\3\4\4\2\1\3\2"
_ATTENTION_HEADS = b"\3\4\4\3\2\3\2"


def _attention(pages):
    """(ranks, the call and its workspace's) for tables of rows, or of rows and kv heads."""
    if getattr(pages, "ndim", 2) == 3:
        return _ATTENTION_HEADS, lib.cmd_paged_attention_heads, lib.cmd_paged_attention_heads_workspace
    return _ATTENTION, lib.cmd_paged_attention, lib.cmd_paged_attention_workspace


def _scale(scale, q) -> float:
    if scale is None:
        return 1.0 / math.sqrt(max(1, q.shape[-1])) if q.dim() else 1.0
    return scale


def paged_attention(q, k_cache, v_cache, pages, lens, out, *, lse=None, scale=None, window=0, workspace=None,
                    stream=None):
    """Attention of one new token per sequence over the paged cache
    (cmd_paged_attention): q [B, hq, d] over the first lens[r] positions of row
    r -- the last ``window`` of them if that is not 0 -- into out [B, hq, dv],
    the log of the softmax's sum into lse [B, hq] (float32) if given.  scale:
    1 / sqrt(d) by default.  pages [B, P] and lens [B] are the rows' tables, or pages
    [B, hk, P] and lens [B, hk] one for every kv head, as ``page_select`` makes them
    (cmd_paged_attention_heads)."""
    ranks, call, size_of = _attention(pages)
    args, dev, current = _pack(ranks, q, k_cache, v_cache, pages, lens, out, lse)
    scale = _scale(scale, q)
    window = _int32(window)
    if dev < 0:
        _refuse(call(args, scale, window, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, size_of(args, window), stream, dev)
    _check(call(args, scale, window, ptr, size, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(out, lse)


def paged_attention_workspace(q, k_cache, v_cache, pages, lens, out, *, window=0) -> int:
    """Bytes of workspace that paged_attention needs for these tensors."""
    ranks, _, size_of = _attention(pages)
    n = size_of(_pack(ranks, q, k_cache, v_cache, pages, lens, out, None)[0], _int32(window))
    _check(n)
    return n


_TREE = b"\4\4\4\2\1\2\4\3"


def tree_attention(q, k_cache, v_cache, pages, lens, parent, out, *, lse=None, scale=None, window=0, workspace=None,
                   stream=None):
    """Attention for a tree of drafted tokens over the paged cache
    (cmd_tree_attention): token i of row r, q [B, T, hq, d], follows token parent[r,
    i] < i (-1: the context; others: padding) and attends to the row's first lens[r]
    positions, to the tokens above it and to itself, whose keys and values lie at
    positions lens[r] + i.  out [B, T, hq, dv], lse [B, T, hq] (float32) if given."""
    args, dev, current = _pack(_TREE, q, k_cache, v_cache, pages, lens, parent, out, lse)
    scale = _scale(scale, q)
    window = _int32(window)
    if dev < 0:
        _refuse(lib.cmd_tree_attention(args, scale, window, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, lib.cmd_tree_attention_workspace(args, window), stream, dev)
    _check(lib.cmd_tree_attention(args, scale, window, ptr, size, 0,
                                  current if stream is None else _handle(stream, dev)))
    _binding.wrote(out, lse)


def tree_attention_workspace(q, k_cache, v_cache, pages, lens, parent, out, *, window=0) -> int:
    """Bytes of workspace that tree_attention needs for these tensors."""
    n = lib.cmd_tree_attention_workspace(_pack(_TREE, q, k_cache, v_cache, pages, lens, parent, out, None)[0],
                                         _int32(window))
    _check(n)
    return n


def tree_accept(tokens, parent, next, lens, path, lens_out, last, *, stream=None):
    """The accepted path of a tree of drafted tokens (cmd_tree_accept): from token 0
    on to the first child that is what the model went on with, next [B, T]; all
    int32.  path [B, T]: its tokens, then -1; lens_out (which may be lens) = lens +
    how many they are; last [B]: what follows the last of them."""
    args, dev, current = _pack(b"\2\2\2\1\2\1\1", tokens, parent, next, lens, path, lens_out, last)
    if dev < 0:
        _refuse(lib.cmd_tree_accept(args, CHECK_ONLY, None))
    _check(lib.cmd_tree_accept(args, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(path, lens_out, last)


def slot_move(pools, pages, lens, path, *, stream=None):
    """Move what position lens[r] + path[r, i] of row r holds to position lens[r] + i
    in every pool [N, page, heads, d] (cmd_slot_move), in order, up to the first
    negative entry.  lens: from before the path was accepted."""
    pools = list(pools)
    n = len(pools)
    args, dev, current = _pack(b"\2\1\2" + b"\4" * n, pages, lens, path, *pools)
    both = (args[3 * _SIZE:], n, args[:3 * _SIZE])
    if dev < 0:
        _refuse(lib.cmd_slot_move(*both, CHECK_ONLY, None))
    _check(lib.cmd_slot_move(*both, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(*pools)


def page_bounds(k_cache, pages, lens, since, bounds, *, stream=None):
    """Keep up the least and largest key of every page (cmd_page_bounds) with
    positions since[r] .. lens[r] - 1 of every row: bounds [N, hk, 2, d] of
    k_cache's dtype.  Call it after the append of those positions."""
    args, dev, current = _pack(b"\4\2\1\1\4", k_cache, pages, lens, since, bounds)
    if dev < 0:
        _refuse(lib.cmd_page_bounds(args, CHECK_ONLY, None))
    _check(lib.cmd_page_bounds(args, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(bounds)


_SELECT = b"\3\4\2\1\3\2"


def page_select(q, bounds, pages, lens, page, pages_out, lens_out, *, first=1, last=2, workspace=None, stream=None):
    """Choose the pages that q [B, hq, d] may care for most, for every sequence and kv
    head (cmd_page_select): pages_out [B, hk, C] and lens_out [B, hk], tables for
    ``paged_attention``.  The row's ``first`` first and ``last`` last pages are
    always among them."""
    page, first, last = _int32(page), _int32(first), _int32(last)
    args, dev, current = _pack(_SELECT, q, bounds, pages, lens, pages_out, lens_out)
    if dev < 0:
        _refuse(lib.cmd_page_select(args, page, first, last, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, lib.cmd_page_select_workspace(args, page, first, last), stream, dev)
    _check(lib.cmd_page_select(args, page, first, last, ptr, size, 0,
                               current if stream is None else _handle(stream, dev)))
    _binding.wrote(pages_out, lens_out)


def page_select_workspace(q, bounds, pages, lens, page, pages_out, lens_out, *, first=1, last=2) -> int:
    """Bytes of workspace that page_select needs for these tensors."""
    n = lib.cmd_page_select_workspace(_pack(_SELECT, q, bounds, pages, lens, pages_out, lens_out)[0], _int32(page),
                                      _int32(first), _int32(last))
    _check(n)
    return n


def page_mass(q, k_cache, pages, lens, lse, mass, mass_out, *, scale=None, decay=1.0, window=0, stream=None):
    """Add the weight that attention gave to every page (cmd_page_mass): mass_out [B,
    P] (float32; it may be mass) = decay * mass + the softmax weights of
    ``paged_attention``, with its lse, over column j's positions and all heads."""
    args, dev, current = _pack(b"\3\4\2\1\2\2\2", q, k_cache, pages, lens, lse, mass, mass_out)
    scale = _scale(scale, q)
    window = _int32(window)
    if dev < 0:
        _refuse(lib.cmd_page_mass(args, scale, decay, window, CHECK_ONLY, None))
    _check(lib.cmd_page_mass(args, scale, decay, window, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(mass_out)


def page_evict(pages, lens, refs, mass, budget, page, pages_out, refs_out, count, *, first=0, last=1, stream=None):
    """Take the pages of least mass out of rows that hold more than budget [R] of them
    (cmd_page_evict), but for the ``first`` first and ``last`` last: pages_out with
    holes there (it may be pages), refs_out without their entries (it may be refs),
    count [R] how many each row lost."""
    page, first, last = _int32(page), _int32(first), _int32(last)
    args, dev, current = _pack(b"\2\1\1\2\1\2\1\1", pages, lens, refs, mass, budget, pages_out, refs_out, count)
    if dev < 0:
        _refuse(lib.cmd_page_evict(args, page, first, last, CHECK_ONLY, None))
    _check(lib.cmd_page_evict(args, page, first, last, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(pages_out, refs_out, count)


_ASSIGN = b"\2\1\1\1\1\2\1\1\1\1\1"


def page_assign(pages, lens, refs, parent, add, page, pages_out, lens_out, refs_out, src, dst, stats, *,
                workspace=None, stream=None):
    """One step in the page tables (cmd_page_assign): every sequence takes over
    the state of sequence parent[r] (its own, another's: a fork, or -1: none)
    and grows by add[r] positions.  Fills pages_out, lens_out, refs_out, the
    page copies src -> dst that forks need (-1: none) and stats = (pages wanted,
    pages given).  refs_out may be refs."""
    page = _int32(page)
    args, dev, current = _pack(_ASSIGN, pages, lens, refs, parent, add, pages_out, lens_out, refs_out, src, dst, stats)
    if dev < 0:
        _refuse(lib.cmd_page_assign(args, page, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, lib.cmd_page_assign_workspace(args, page), stream, dev)
    _check(lib.cmd_page_assign(args, page, ptr, size, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(pages_out, lens_out, refs_out, src, dst, stats)


def page_assign_workspace(pages, lens, refs, parent, add, page, pages_out, lens_out, refs_out, src, dst, stats) -> int:
    """Bytes of workspace that page_assign needs for these tensors."""
    args = _pack(_ASSIGN, pages, lens, refs, parent, add, pages_out, lens_out, refs_out, src, dst, stats)[0]
    n = lib.cmd_page_assign_workspace(args, _int32(page))
    _check(n)
    return n


_COMPACT = b"\2\1\2\1\1\1\1"


def page_compact(pages, refs, pages_out, refs_out, src, dst, stats, *, workspace=None, stream=None):
    """Pack the live pages (refs > 0) into the lowest ids (cmd_page_compact):
    the table and counts after it, the copies src -> dst it takes (then -1) and
    stats = (live pages, moves).  src and dst hold refs.numel() // 2 entries or
    more; pages_out may be pages."""
    args, dev, current = _pack(_COMPACT, pages, refs, pages_out, refs_out, src, dst, stats)
    if dev < 0:
        _refuse(lib.cmd_page_compact(args, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, lib.cmd_page_compact_workspace(args), stream, dev)
    _check(lib.cmd_page_compact(args, ptr, size, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(pages_out, refs_out, src, dst, stats)


def page_compact_workspace(pages, refs, pages_out, refs_out, src, dst, stats) -> int:
    """Bytes of workspace that page_compact needs for these tensors."""
    n = lib.cmd_page_compact_workspace(_pack(_COMPACT, pages, refs, pages_out, refs_out, src, dst, stats)[0])
    _check(n)
    return n


def page_copy(pools, src, dst, *, stream=None):
    """Copy page src[i] to page dst[i] in every pool [N, page, heads, d]
    (cmd_page_copy); pairs with an id outside the pool are skipped."""
    pools = list(pools)
    n = len(pools)
    args, dev, current = _pack(b"\1\1" + b"\4" * n, src, dst, *pools)
    pairs = (args[2 * _SIZE:], n, args[:_SIZE], args[_SIZE:2 * _SIZE])
    if dev < 0:
        _refuse(lib.cmd_page_copy(*pairs, CHECK_ONLY, None))
    _check(lib.cmd_page_copy(*pairs, 0, current if stream is None else _handle(stream, dev)))
    _binding.wrote(*pools)


def rope_frequencies(width, *, base=10000.0, factor=1.0, scaling="linear", trained=0, slow=1.0, fast=32.0):
    """The frequency table of a rotary part of this (even) width, float64 on the
    CPU: base ** (-2 i / width), for contexts ``factor`` times as long as the
    trained ones changed by ``scaling``:

      "linear"  every frequency divided by factor (positions interpolated);
      "base"    the base raised so that the slowest pair is divided by factor
                and the fastest keeps its frequency;
      "parts"   by how often a pair turns within ``trained`` positions: pairs
                that turn more than ``fast`` times keep their frequency, those
                that turn less than ``slow`` times are divided by factor, a
                linear ramp between (usually with mscale = 0.1 ln factor + 1).
    """
    import torch
    if width < 0 or width % 2:
        raise ValueError("width must be even, got %d" % width)
    if factor < 1.0 or scaling not in ("linear", "base", "parts"):
        raise ValueError("factor must be at least 1 and scaling one of linear, base, parts")
    if scaling == "base" and width > 2:
        base = base * factor ** (width / (width - 2.0))
    f = torch.tensor([base ** (-2.0 * i / width) for i in range(width // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if trained <= 0 or fast <= slow:
            raise ValueError("scaling by parts needs the trained length and slow < fast")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f
