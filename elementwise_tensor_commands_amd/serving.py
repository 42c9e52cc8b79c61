"""Serving operators beside Commands: rotary positions, a paged key-value
cache, attention of one new token over it, and the bookkeeping of its pages.

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

``decode.py`` in this package runs it end to end.
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
        ("cmd_page_copy", ctypes.c_int, [_args, _i32, _args, _args, _i32, _vp])]:
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


def paged_attention(q, k_cache, v_cache, pages, lens, out, *, lse=None, scale=None, window=0, workspace=None,
                    stream=None):
    """Attention of one new token per sequence over the paged cache
    (cmd_paged_attention): q [B, hq, d] over the first lens[r] positions of row
    r -- the last ``window`` of them if that is not 0 -- into out [B, hq, dv],
    the log of the softmax's sum into lse [B, hq] (float32) if given.  scale:
    1 / sqrt(d) by default."""
    args, dev, current = _pack(_ATTENTION, q, k_cache, v_cache, pages, lens, out, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(max(1, q.shape[-1])) if q.dim() else 1.0
    window = _int32(window)
    if dev < 0:
        _refuse(lib.cmd_paged_attention(args, scale, window, None, 0, CHECK_ONLY, None))
    ptr, size, _owner = _scratch(workspace, lib.cmd_paged_attention_workspace(args, window), stream, dev)
    _check(lib.cmd_paged_attention(args, scale, window, ptr, size, 0,
                                   current if stream is None else _handle(stream, dev)))
    _binding.wrote(out, lse)


def paged_attention_workspace(q, k_cache, v_cache, pages, lens, out, *, window=0) -> int:
    """Bytes of workspace that paged_attention needs for these tensors."""
    n = lib.cmd_paged_attention_workspace(_pack(_ATTENTION, q, k_cache, v_cache, pages, lens, out, None)[0],
                                          _int32(window))
    _check(n)
    return n


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
