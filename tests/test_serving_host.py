"""The serving operators on the host: argument checks (every refusal comes
before any HIP call, so CPU tensors do), workspace sizes, frequency tables, and
the oracle against hand-worked cases."""
import math
import os
import re

import pytest
import torch

import elementwise_tensor_commands_amd as E
import serving_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32 = torch.int32


def _refused(name, fn, *args, **kw):
    with pytest.raises(E.Error) as e:
        fn(*args, **kw)
    assert e.value.name == name, str(e.value)
    assert len(str(e.value)) > len(name) + 8      # a message that says what is wrong
    return str(e.value)


def i32(*shape):
    return torch.zeros(shape, dtype=I32)


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "ecmd_serving.h")).read()
    declared = set(re.findall(r"^\s*(?:int|int64_t)\s+(cmd_\w+)\s*\(", text, re.M))
    assert declared >= {"cmd_rope", "cmd_rope_append", "cmd_paged_attention", "cmd_page_assign", "cmd_page_compact",
                        "cmd_page_copy"}
    for name in declared:
        assert hasattr(E.lib, name), name


# ---------------------------------------------------------------------------
# Rotary positions.

def rope_args(**kw):
    a = dict(x=torch.zeros(2, 3, 4, 10), pos=i32(2, 3), freq=torch.zeros(4, dtype=torch.float64),
             out=torch.zeros(2, 3, 4, 10))
    a.update(kw)
    return [a[k] for k in ("x", "pos", "freq", "out")]


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(x=torch.zeros(2, 3, 4, 10, dtype=torch.float64))),
    ("CMD_E_DTYPE", dict(out=torch.zeros(2, 3, 4, 10, dtype=torch.float16))),
    ("CMD_E_DTYPE", dict(pos=torch.zeros(2, 3, dtype=torch.int64))),
    ("CMD_E_DTYPE", dict(freq=torch.zeros(4))),
    ("CMD_E_SHAPE", dict(x=torch.zeros(2, 3, 40))),
    ("CMD_E_SHAPE", dict(out=torch.zeros(2, 3, 4, 9))),
    ("CMD_E_SHAPE", dict(pos=i32(3, 2))),
    ("CMD_E_SHAPE", dict(freq=torch.zeros(6, dtype=torch.float64))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(2, 3, 10, 4).transpose(2, 3))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(2, 1, 4, 10).expand(2, 3, 4, 10))),
])
def test_rope_refusals(name, kw):
    _refused(name, E.rope, *rope_args(**kw))


def test_rope_refusals_of_options_and_aliases():
    _refused("CMD_E_ARG", E.rope, *rope_args(), layout="thirds")
    _refused("CMD_E_ARG", E.rope, *rope_args(), mscale=math.inf)
    big = torch.zeros(2, 3, 4, 20)
    _refused("CMD_E_ALIAS", E.rope, *rope_args(x=big[..., :10], out=big[..., 5:15]))
    _refused("CMD_E_LIMIT", E.rope, *rope_args(x=torch.zeros(1, 1, 1, 5000), out=torch.zeros(1, 1, 1, 5000), pos=i32(1, 1),
                                               freq=torch.zeros(2049, dtype=torch.float64)))
    # what is right but on the CPU is refused last, with in-place and packed views
    x = torch.zeros(2, 3, 4, 10)
    for args in (rope_args(), rope_args(x=x, out=x), rope_args(x=big[..., :10], out=big[..., 10:])):
        assert "GPU" in _refused("CMD_E_ARG", E.rope, *args)


def test_views_with_the_negative_bit_are_refused():
    """Such a view's memory holds the opposite of its numbers."""
    freq = torch.complex(torch.ones(4, dtype=torch.float64), torch.ones(4, dtype=torch.float64)).conj().imag
    assert freq.is_neg()
    with pytest.raises(TypeError, match="negative bit"):
        E.rope(*rope_args(freq=freq))
    assert "GPU" in _refused("CMD_E_ARG", E.rope, *rope_args(freq=freq.resolve_neg()))


def test_version_counters():
    """Advanced for what a call wrote, shared with views; not by a refused call, not of inference tensors."""
    from elementwise_tensor_commands_amd import serving as S
    args = rope_args()
    before = [t._version for t in args]
    _refused("CMD_E_ARG", E.rope, *args)
    assert [t._version for t in args] == before
    with torch.inference_mode():
        none = torch.zeros(3)
    x = torch.zeros(4, 4)
    view = x[1:]
    S._binding.wrote(view, None, none, args[0])
    assert x._version == view._version == 1 and args[0]._version == before[0] + 1
    with pytest.raises(TypeError):
        S._binding.wrote(3)


# ---------------------------------------------------------------------------
# The append.

def append_args(**kw):
    kc = torch.zeros(7, 16, 2, 8)
    a = dict(q=torch.zeros(5, 4, 8), k=torch.zeros(5, 2, 8), v=torch.zeros(5, 2, 6), pos=i32(5), row=i32(5),
             pages=i32(3, 2), freq=torch.zeros(4, dtype=torch.float64), q_out=torch.zeros(5, 4, 8), k_cache=kc,
             v_cache=torch.zeros(7, 16, 2, 6))
    a.update(kw)
    return [a[k] for k in ("q", "k", "v", "pos", "row", "pages", "freq", "q_out", "k_cache", "v_cache")]


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(k=torch.zeros(5, 2, 8, dtype=torch.bfloat16))),
    ("CMD_E_DTYPE", dict(row=torch.zeros(5))),
    ("CMD_E_SHAPE", dict(k=torch.zeros(4, 2, 8))),
    ("CMD_E_SHAPE", dict(v=torch.zeros(5, 3, 6))),
    ("CMD_E_SHAPE", dict(pos=i32(4))),
    ("CMD_E_SHAPE", dict(k_cache=torch.zeros(7, 16, 3, 8))),
    ("CMD_E_SHAPE", dict(v_cache=torch.zeros(6, 16, 2, 6))),
    ("CMD_E_SHAPE", dict(v_cache=torch.zeros(7, 8, 2, 6))),
    ("CMD_E_SHAPE", dict(freq=torch.zeros(5, dtype=torch.float64))),
    ("CMD_E_STRIDE", dict(k_cache=torch.zeros(7, 16, 8, 2).transpose(2, 3))),
    ("CMD_E_STRIDE", dict(v_cache=torch.zeros(1, 16, 2, 6).expand(7, 16, 2, 6))),
])
def test_append_refusals(name, kw):
    _refused(name, E.rope_append, *append_args(**kw))


def test_append_accepts_packed_and_refuses_overlapping():
    qkv = torch.zeros(5, 8, 8)
    packed = dict(q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:8], q_out=qkv[:, :4], v_cache=torch.zeros(7, 16, 2, 8))
    assert "GPU" in _refused("CMD_E_ARG", E.rope_append, *append_args(**packed))       # q turned in place
    kv = torch.zeros(7, 2, 16, 2, 8)
    both = dict(v=torch.zeros(5, 2, 8), k_cache=kv[:, 0], v_cache=kv[:, 1])
    assert "GPU" in _refused("CMD_E_ARG", E.rope_append, *append_args(**both))
    kv = torch.zeros(7, 16, 2, 2, 8)
    both.update(k_cache=kv[:, :, 0], v_cache=kv[:, :, 1])
    assert "GPU" in _refused("CMD_E_ARG", E.rope_append, *append_args(**both))
    both.update(v_cache=kv[:, :, 0])
    _refused("CMD_E_ALIAS", E.rope_append, *append_args(**both))
    packed["q_out"] = qkv[:, 1:5]
    _refused("CMD_E_ALIAS", E.rope_append, *append_args(**packed))


# ---------------------------------------------------------------------------
# Attention.

def attention_args(**kw):
    a = dict(q=torch.zeros(3, 4, 8), k=torch.zeros(7, 16, 2, 8), v=torch.zeros(7, 16, 2, 6), pages=i32(3, 2),
             lens=i32(3), out=torch.zeros(3, 4, 6))
    a.update(kw)
    return [a[k] for k in ("q", "k", "v", "pages", "lens", "out")]


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(k=torch.zeros(7, 16, 2, 8, dtype=torch.float16))),
    ("CMD_E_DTYPE", dict(lens=torch.zeros(3, dtype=torch.int64))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 4, 9))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 8), out=torch.zeros(3, 5, 6))),
    ("CMD_E_SHAPE", dict(v=torch.zeros(7, 15, 2, 6))),
    ("CMD_E_SHAPE", dict(pages=i32(2, 2))),
    ("CMD_E_SHAPE", dict(lens=i32(4))),
    ("CMD_E_SHAPE", dict(out=torch.zeros(3, 4, 8))),
    ("CMD_E_LIMIT", dict(q=torch.zeros(3, 4, 257), k=torch.zeros(7, 16, 2, 257))),
    ("CMD_E_LIMIT", dict(pages=torch.zeros(3, 1, dtype=I32).expand(3, 1 << 27))),
    ("CMD_E_STRIDE", dict(q=torch.zeros(3, 8, 4).transpose(1, 2))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(3, 1, 6).expand(3, 4, 6))),
])
def test_attention_refusals(name, kw):
    _refused(name, E.paged_attention, *attention_args(**kw))
    _refused(name, E.paged_attention_workspace, *attention_args(**kw))


def test_attention_out_has_neighbouring_columns():
    """An out whose last dimension has another stride is refused, as the inputs are."""
    for out in (torch.zeros(3, 6, 4).transpose(1, 2), torch.zeros(3, 4, 12)[..., ::2]):
        assert tuple(out.shape) == (3, 4, 6)
        for fn in (E.paged_attention, E.paged_attention_workspace):
            assert "last dimension" in _refused("CMD_E_STRIDE", fn, *attention_args(out=out))
    # any strides of the other dimensions, a last dimension of one element, and lse of any strides
    for kw in (dict(out=torch.zeros(4, 3, 9)[..., 2:8].transpose(0, 1)),
               dict(v=torch.zeros(7, 16, 2, 1), out=torch.zeros(3, 4, 5)[..., 3:4])):
        assert "GPU" in _refused("CMD_E_ARG", E.paged_attention, *attention_args(**kw), lse=torch.zeros(4, 6).t()[::2])


def test_attention_refusals_of_options():
    _refused("CMD_E_ARG", E.paged_attention, *attention_args(), window=-1)
    _refused("CMD_E_ARG", E.paged_attention, *attention_args(), window=5 - (1 << 32))
    _refused("CMD_E_ARG", E.paged_attention, *attention_args(), scale=math.nan)
    _refused("CMD_E_SHAPE", E.paged_attention, *attention_args(), lse=torch.zeros(3, 5))
    _refused("CMD_E_DTYPE", E.paged_attention, *attention_args(), lse=torch.zeros(3, 4, dtype=torch.float64))
    a = attention_args(q=torch.zeros(3, 4, 6), k=torch.zeros(7, 16, 2, 6))
    a[5] = a[0]
    _refused("CMD_E_ALIAS", E.paged_attention, *a)
    assert "GPU" in _refused("CMD_E_ARG", E.paged_attention, *attention_args(), lse=torch.zeros(3, 4))


def test_attention_scale_in_base_2():
    """Scores are taken to base 2 in binary32: a scale that has no number there would make 0 * inf of a score of 0."""
    for scale in (3.0e38, -2.4e38, math.inf, 1e300):
        assert "scale" in _refused("CMD_E_ARG", E.paged_attention, *attention_args(), scale=scale)
    for scale in (2.3e38, -1e30, 0.0, 1e-45):
        assert "GPU" in _refused("CMD_E_ARG", E.paged_attention, *attention_args(), scale=scale)


def test_attention_workspace():
    assert E.paged_attention_workspace(*attention_args(pages=i32(3, 1))) == 0           # too few keys to cut
    a = attention_args(pages=i32(3, 4096))
    need = E.paged_attention_workspace(*a)
    assert need > 0 and E.paged_attention_workspace(*a, window=100) == 0
    # a workspace too small is refused without a HIP call (from C, as a caller would)
    from elementwise_tensor_commands_amd import serving as S
    args = S._pack(S._ATTENTION, *a, None)[0]
    buf = torch.zeros(need, dtype=torch.uint8)
    assert E.lib.cmd_paged_attention(args, 1.0, 0, None, 0, 0, None) == -1
    assert E.lib.cmd_paged_attention(args, 1.0, 0, buf.data_ptr(), need - 1, 0, None) == -1
    assert b"workspace" in E.lib.cmd_last_error(None)
    assert E.lib.cmd_paged_attention(None, 1.0, 0, None, 0, 0, None) == -1
    assert E.lib.cmd_paged_attention(args, 1.0, 0, None, 0, 2, None) == -1              # unknown flag
    assert E.lib.cmd_paged_attention(args, 1.0, 0, None, 0, S.CHECK_ONLY, None) == 0


def test_scratch_memory_is_the_launch_stream_s(monkeypatch):
    """Of a handle, its stream's; of handle 0, the default stream's (which torch wraps in no ExternalStream)."""
    import contextlib
    import types

    from elementwise_tensor_commands_amd import serving as S
    entered = []

    @contextlib.contextmanager
    def enter(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(S, "_binding", types.SimpleNamespace(scratch=lambda size, device: (4096, "owner")))
    other = object()
    for stream, want in ((0, ("default", 3)), (77, ("external", 77)), (other, other)):
        assert S._scratch(None, 64, stream, 3) == (4096, 64, "owner")
        assert entered.pop() == want
    assert S._scratch(None, 64, None, 3) == (4096, 64, "owner") and not entered      # torch's current stream


# ---------------------------------------------------------------------------
# Pages.

def assign_args(**kw):
    a = dict(pages=i32(3, 4), lens=i32(3), refs=i32(9), parent=i32(3), add=i32(3), page=16, pages_out=i32(3, 4),
             lens_out=i32(3), refs_out=i32(9), src=i32(3), dst=i32(3), stats=i32(2))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(pages=torch.zeros(3, 4, dtype=torch.int64))),
    ("CMD_E_SHAPE", dict(lens=i32(4))),
    ("CMD_E_SHAPE", dict(pages_out=i32(3, 5))),
    ("CMD_E_SHAPE", dict(refs_out=i32(8))),
    ("CMD_E_SHAPE", dict(src=i32(2))),
    ("CMD_E_SHAPE", dict(stats=i32(3))),
    ("CMD_E_ARG", dict(page=0)),
    ("CMD_E_LIMIT", dict(page=1 << 30)),
    ("CMD_E_LIMIT", dict(page=(1 << 32) + 16)),                      # not 16, as 32 bits would have it
    ("CMD_E_ARG", dict(page=16 - (1 << 32))),
    ("CMD_E_STRIDE", dict(lens_out=i32(1).expand(3))),
])
def test_assign_refusals(name, kw):
    _refused(name, E.page_assign, *assign_args(**kw))


def test_assign_aliases():
    p, l, r = i32(3, 4), i32(3), i32(9)
    _refused("CMD_E_ALIAS", E.page_assign, *assign_args(pages=p, pages_out=p))
    _refused("CMD_E_ALIAS", E.page_assign, *assign_args(lens=l, lens_out=l))
    _refused("CMD_E_ALIAS", E.page_assign, *assign_args(src=l, dst=l))
    assert "GPU" in _refused("CMD_E_ARG", E.page_assign, *assign_args(refs=r, refs_out=r))


def compact_args(**kw):
    a = dict(pages=i32(3, 4), refs=i32(9), pages_out=i32(3, 4), refs_out=i32(9), src=i32(4), dst=i32(4), stats=i32(2))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(refs=torch.zeros(9))),
    ("CMD_E_SHAPE", dict(src=i32(3), dst=i32(3))),
    ("CMD_E_SHAPE", dict(dst=i32(5))),
    ("CMD_E_SHAPE", dict(pages_out=i32(4, 3))),
    ("CMD_E_STRIDE", dict(refs_out=i32(1).expand(9))),
])
def test_compact_refusals(name, kw):
    _refused(name, E.page_compact, *compact_args(**kw))


def test_compact_aliases():
    p, r = i32(3, 4), i32(9)
    _refused("CMD_E_ALIAS", E.page_compact, *compact_args(refs=r, refs_out=r))
    assert "GPU" in _refused("CMD_E_ARG", E.page_compact, *compact_args(pages=p, pages_out=p))


def test_copy_refusals():
    pool, s, d = torch.zeros(5, 4, 2, 8), i32(3), i32(3)
    _refused("CMD_E_SHAPE", E.page_copy, [pool], s, i32(4))
    _refused("CMD_E_SHAPE", E.page_copy, [pool[0]], s, d)
    _refused("CMD_E_DTYPE", E.page_copy, [pool.to(torch.int8)], s, d)
    _refused("CMD_E_STRIDE", E.page_copy, [pool[:1].expand(5, 4, 2, 8)], s, d)
    _refused("CMD_E_STRIDE", E.page_copy, [torch.zeros(5, 8, 4, 16)[:, ::2, ::2, ::2]], s, d)
    _refused("CMD_E_ALIAS", E.page_copy, [s.view(3, 1, 1, 1)], s, d)
    assert "GPU" in _refused("CMD_E_ARG", E.page_copy, [pool, pool.transpose(1, 2)], s, d)


# ---------------------------------------------------------------------------
# What one launch holds: 2^24 - 1 work-groups.

def made_up(dtype, shape, at, strides=None):
    """A cmd_arg of a tensor that nothing reads: dense unless strides are given, `at` TB in."""
    a = E.cmd_arg()
    a.kind, a.dtype, a.ptr = 1, {"f16": 1, "f32": 2, "i32": 3, "bf16": 4, "f64": 5}[dtype], at << 40
    step = 1
    for i in reversed(range(len(shape))):
        a.size[i], a.stride[i] = shape[i], step if strides is None else strides[i]
        step *= max(1, shape[i])
    return a


def check_only(fn, args, *rest):
    return getattr(E.lib, fn)(b"".join(bytes(a) for a in args), *rest, 1, None)


def test_calls_larger_than_a_launch():
    """Refused before any HIP call, as the header says, where no launch could hold them."""
    from elementwise_tensor_commands_amd import serving as S  # noqa: F401  (argument types)
    limit = -next(k for k in range(1, 40) if E.Error(-k, "").name == "CMD_E_LIMIT")

    def attend(b, hk, group, cols):
        q = made_up("f16", (b, hk * group, 8), 1)
        cache = [made_up("f16", (4, 16, hk, 8), 2 + i) for i in range(2)]
        none = E.cmd_arg()
        return check_only("cmd_paged_attention", [q, *cache, made_up("i32", (b, cols), 4, (0, 0)), made_up("i32", (b,), 5),
                                                  made_up("f16", (b, hk * group, 8), 6), none], 1.0, 0, None, 0)

    assert attend(131000, 128, 1, 8) == 0
    assert attend(131072, 128, 1, 8) == limit
    assert attend(2048, 16, 500, 4096) == 0
    assert attend(2048, 16, 520, 4096) == limit                    # the second launch

    def assign(rows):
        i = lambda at, *shape: made_up("i32", shape, at)
        return check_only("cmd_page_assign", [i(1, rows, 2), i(2, rows), i(3, 9), i(4, rows), i(5, rows), i(6, rows, 2), i(7, rows),
                                              i(8, 9), i(9, rows), i(10, rows), i(11, 2)], 4, None, 0)

    assert assign((1 << 24) - 1) == 0
    assert assign(1 << 24) == limit

    def compact(rows, n):
        i = lambda at, *shape: made_up("i32", shape, at)
        return check_only("cmd_page_compact", [i(1, rows, 1), i(2, n), i(3, rows, 1), i(4, n), i(5, n // 2), i(6, n // 2), i(7, 2)], None, 0)

    assert compact((1 << 31) - 1024, (1 << 31) - 1024) == 0
    assert compact((1 << 31) - 1, (1 << 31) - 1) == limit

    def copy(pairs):
        src, dst, pool = made_up("i32", (pairs,), 1), made_up("i32", (pairs,), 2), made_up("f16", (9, 16, 8, 128), 3)
        return E.lib.cmd_page_copy(bytes(pool), 1, bytes(src), bytes(dst), 1, None)

    assert copy((1 << 23) - 1) == 0
    assert copy(1 << 23) == limit

    # rope and the append give their groups more tokens instead
    for tokens in ((1 << 24) - 1, 1 << 24, (1 << 31) - 1):
        x = made_up("f16", (1, tokens, 1, 4104), 3)
        assert check_only("cmd_rope", [x, made_up("i32", (1, tokens), 1, (0, 0)), made_up("f64", (2048,), 2), x], 0, 1.0, 0) == 0


# ---------------------------------------------------------------------------
# The oracle and the tables of frequencies.

def test_oracle_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = torch.tensor([math.pi / 2, 0.0], dtype=torch.float64)
    y, _ = O.rope(x, torch.tensor([1]), quarter, "half")           # pairs (1, 3) and (2, 4), the first a quarter turn
    assert torch.allclose(y, torch.tensor([[[-3.0, 2.0, 1.0, 4.0, 5.0]]]).double(), atol=1e-15)
    y, _ = O.rope(x, torch.tensor([1]), quarter, "interleaved", mscale=2.0, inverse=True)
    assert torch.allclose(y, torch.tensor([[[4.0, -2.0, 6.0, 8.0, 5.0]]]).double(), atol=1e-15)

    k = torch.zeros(2, 2, 1, 1)
    v = torch.tensor([1.0, 2.0, 4.0, 8.0]).view(2, 2, 1, 1)
    k[1, 0] = math.log(3.0)
    q = torch.ones(1, 1, 1)
    pages = torch.tensor([[1, 0, -1]])
    out, lse, _, _ = O.attention(q, k, v, pages, [3], 1.0)         # keys: 1.0 -> 4 (weight 3), 8, then 1
    assert abs(out.item() - (3 * 4 + 8 + 1) / 5) < 1e-6 and abs(lse.item() - math.log(5)) < 1e-6
    out, lse, _, _ = O.attention(q, k, v, pages, [3], 1.0, window=1)
    assert out.item() == 1.0
    out, lse, _, _ = O.attention(q, k, v, pages, [0], 1.0)
    assert out.item() == 0.0 and lse.item() == -math.inf
    out, lse, _, _ = O.attention(q, k, v, pages, [6], 1.0, window=2)   # only the hole's positions
    assert out.item() == 0.0 and lse.item() == -math.inf

    # rows: 0 goes on, 1 forks from 0 (shares page 3, copies page 1), 2 ends and starts anew with 5
    out = O.assign([[3, 1, -1], [4, -1, -1], [0, -1, -1]], [6, 2, 4], [1, 1, 0, 1, 1, 0, 0], [0, 0, -1], [1, 3, 5], 4)
    assert out[0] == [[3, 1, -1], [3, 2, 5], [6, -1, -1]]
    assert out[1:] == ([7, 9, 5], [0, 1, 1, 2, 0, 1, 1], [-1, 1, -1], [-1, 2, -1], [4, 3])
    assert O.compact([[5, 2], [3, 9]], [0, 0, 1, 1, 0, 2], 3) == (
        [[1, 2], [0, -1]], [1, 2, 1, 0, 0, 0], [3, 5, -1], [0, 1, -1], [3, 2])


def test_rope_gradient_is_the_inverse():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 3, 9, generator=g, dtype=torch.float64)
    dy = torch.randn(2, 3, 9, generator=g, dtype=torch.float64)
    pos, freq = torch.tensor([3, 7]), E.rope_frequencies(8)
    for layout in ("half", "interleaved"):
        dx, _ = O.rope(dy, pos, freq, layout, 1.3, inverse=True)
        leaf = x.clone().requires_grad_()
        u, v = O.pairs(leaf, 4, layout)
        w = pos.double()[:, None, None] * freq
        turned = torch.cat([u * w.cos() - v * w.sin(), v * w.cos() + u * w.sin()], -1) * 1.3
        want = torch.cat([*O.pairs(dy, 4, layout)], -1)
        ((turned * want).sum() + (leaf[..., 8:] * dy[..., 8:]).sum()).backward()
        assert torch.allclose(leaf.grad, dx, atol=1e-12)
        for i in (0, 4, 8):                                        # and against differences
            h = 1e-4
            e = torch.zeros_like(x)
            e[1, 2, i] = h
            d = ((O.rope(x + e, pos, freq, layout, 1.3)[0] - O.rope(x - e, pos, freq, layout, 1.3)[0]) * dy).sum() / (2 * h)
            assert abs(float(d) - float(dx[1, 2, i])) < 1e-9


def test_frequencies():
    f = E.rope_frequencies(8)
    assert f.dtype == torch.float64 and torch.allclose(f, 10000.0 ** (-torch.arange(4).double() / 4))
    assert torch.allclose(E.rope_frequencies(8, factor=4.0), f / 4)
    b = E.rope_frequencies(8, factor=4.0, scaling="base")
    assert b[0] == 1 and abs(float(b[3] * 4 / f[3]) - 1) < 1e-12
    p = E.rope_frequencies(128, factor=8.0, scaling="parts", trained=4096)
    q = E.rope_frequencies(128)
    assert p[0] == q[0] and abs(float(p[-1] * 8 / q[-1]) - 1) < 1e-12
    assert bool(((p <= q) & (p >= q / 8 * (1 - 1e-12))).all())
    assert E.rope_frequencies(0).numel() == 0 and E.rope_frequencies(2, factor=2.0, scaling="base").tolist() == [1.0]
    for bad in (dict(width=7), dict(width=8, factor=0.5), dict(width=8, scaling="x"), dict(width=8, factor=2.0, scaling="parts")):
        with pytest.raises(ValueError):
            E.rope_frequencies(**bad)


# ---------------------------------------------------------------------------
# The small decoder's host part.

def test_beams_go_on_from_a_living_row_with_its_tokens():
    from elementwise_tensor_commands_amd.decode import next_beams
    logits = torch.full((6, 9), -20.0)
    logits[0, 4], logits[0, 2], logits[0, 8] = 5.0, 4.0, 3.0
    logits[1, 1] = 9.0                                             # the highest, of a row that has ended
    logits[2, 3] = 4.5
    logits[3, 0], logits[3, 5], logits[3, 7] = -9.0, -8.0, -10.0   # the only one alive of its group
    logits[4, 1], logits[5, 1] = 7.0, 8.0
    parent, tokens = next_beams(logits, torch.tensor([1, 0, 1, 1, 0, 0], dtype=I32), 3)
    assert parent.dtype == I32 and parent.tolist() == [0, 0, 0, 3, 3, 3]
    assert tokens.dtype == torch.int64 and tokens.tolist() == [4, 2, 8, 5, 0, 7]
    parent, tokens = next_beams(logits.half(), torch.ones(6, dtype=I32), 1)
    assert parent.tolist() == list(range(6)) and tokens.tolist() == logits.argmax(-1).tolist()


def test_arguments_of_the_decoder(capsys):
    from elementwise_tensor_commands_amd.decode import PROMPTS, arguments
    assert arguments([]) == (32, 4, 32)
    assert arguments(["--steps", "4", "--beams", "2"]) == (2, 2, 32)
    for steps in (1, 2, 391, 392, 1000, 4097):
        half, _, cols = arguments(["--steps", str(steps)])
        assert half >= 1 and 2 * half >= steps
        assert max(PROMPTS) + 1 + 2 * half <= 16 * cols              # no sequence outgrows its table
    for bad in (["--steps"], ["--steps", "0"], ["--beams", "0"], ["--steps", "x"], ["--beams", "-3"], ["5"]):
        with pytest.raises(SystemExit) as e:
            arguments(bad)
        assert e.value.code == 2 and "usage" in capsys.readouterr().err


# ---------------------------------------------------------------------------
# The build.

def build_module():
    import importlib.util
    spec = importlib.util.spec_from_file_location("ecmd_build", os.path.join(ROOT, "elementwise_tensor_commands_amd", "build.py"))
    B = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(B)
    return B


@pytest.mark.parametrize("with_torch", [True, False])
def test_the_library_is_built_without_torch_too(monkeypatch, tmp_path, with_torch):
    """Only the Python binding needs torch's headers; the C library does not."""
    import importlib.util
    B = build_module()
    ran, moved = [], []
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" and not with_torch else find(name, *a))
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "_run_all", ran.extend)
    monkeypatch.setattr(B.os, "replace", lambda a, b: moved.append(b))
    assert B.build(asm=False) == B.LIB
    sources = [os.path.basename(x) for c in ran for x in c if x.endswith((".cpp", ".hip"))]
    assert all(os.path.basename(s) in sources for s in B.SOURCES)
    assert ("ecmd_binding.cpp" in sources) == with_torch
    assert moved == [B.LIB] + [B.BINDING] * with_torch


def test_the_binding_is_this_interpreter_s():
    """Its name has the interpreter's tag, so no other one loads it; without it the error says what to do."""
    import subprocess
    import sys
    import sysconfig
    B = build_module()
    assert os.path.basename(B.BINDING) == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(B.BINDING) and not os.path.exists(os.path.join(B.PKG, "_binding.so"))
    code = ("import sys; sys.modules['elementwise_tensor_commands_amd._binding'] = None\n"
            "import torch, elementwise_tensor_commands_amd as E\n"
            "try:\n    E.page_copy([], torch.zeros(1), torch.zeros(1))\n"
            "except ImportError as e:\n    print('said:', e)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=200)
    assert "said:" in r.stdout and "build.py" in r.stdout and "torch" in r.stdout, r.stdout + r.stderr


# ---------------------------------------------------------------------------
# The kernels' own assembly.

@pytest.mark.parametrize("name", ["kernels_rope", "kernels_pages", "kernels_attention_f16", "kernels_attention_bf16",
                                  "kernels_attention_f32"])
def test_own_assembly(name):
    """No scratch memory, no packed binary32 arithmetic; attention on matrix instructions."""
    import importlib.util
    import subprocess
    spec = importlib.util.spec_from_file_location("ecmd_build", os.path.join(ROOT, "elementwise_tensor_commands_amd", "build.py"))
    B = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(B)
    src, path = "serving/%s.hip" % name, os.path.join(B.BUILD, name + ".s")
    folder = os.path.join(B.CSRC, "serving")
    newest = max(os.path.getmtime(os.path.join(folder, f)) for f in os.listdir(folder))
    if not os.path.exists(path) or os.path.getmtime(path) < newest:
        os.makedirs(B.BUILD, exist_ok=True)
        subprocess.run([B.HIPCC, *B.FLAGS, *B.FILE_FLAGS.get(src, []), "-x", "hip", "--offload-device-only", "-S",
                        os.path.join(B.CSRC, src), "-o", path], check=True, capture_output=True)
    text = open(path).read()
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)
    assert sizes and all(s == "0" for s in sizes)
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)
    if "attention" in name:
        kind = {"f16": "16x16x32_f16", "bf16": "16x16x32_bf16", "f32": "16x16x4_f32"}[name.rsplit("_", 1)[1]]
        assert text.count("v_mfma_f32_" + kind) > 100


def test_copy_of_sliced_pages():
    """Slices of one dimension of a dense page, keys beside values among them, are taken; of two, refused."""
    s, d = i32(3), i32(3)
    dense = torch.zeros(5, 16, 4, 64)
    for pool in (dense[:, 2:9], dense[:, :, 1:3], dense[..., :40], dense[..., 5:6], dense.transpose(1, 2)[:, 1:3], dense[::2],
                 torch.zeros(5, 16, 2, 4, 64)[:, :, 1], torch.zeros(5, 16, 4, 2, 64)[:, :, :, 0], torch.zeros(5, 2, 16, 4, 64)[:, 1]):
        assert "GPU" in _refused("CMD_E_ARG", E.page_copy, [pool], s, d)
    _refused("CMD_E_STRIDE", E.page_copy, [dense[:, :, 1:3, :40]], s, d)
