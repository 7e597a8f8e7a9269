"""The operators of policies over token sequences without a GPU: refusals of the C ABI and of
the Python binding, and workspace sizes.

Every call below is refused (or has nothing to do) before any HIP call.
"""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import linear_recurrence_scan_reverse_amd as rl
from linear_recurrence_scan_reverse_amd.policy import _Heads

OK, ERR_NULL, ERR_SHAPE, ERR_PARAM, ERR_HIP, ERR_ALIGN, ERR_ALIAS, ERR_WORKSPACE = range(8)
F32, BF16, F16 = 0, 1, 2
BASE = 0x7F0000000000  # fake device addresses, never dereferenced
GIB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rl.library_path()):
        from linear_recurrence_scan_reverse_amd import build
        build.build(verbose=False)
    return rl.lib()


def addr(i):
    return BASE + i * 64 * GIB


def rows(i, T, D, offset=0, env=None, step=None):
    return _Heads(addr(i) + offset, T * D if env is None else env, D if step is None else step, 0)


def by_reference(x):
    return ctypes.byref(x) if isinstance(x, _Heads) else x


def recurrence(lib, E=2, T=100, D=70, fmt=BF16, layout=0, **kw):
    a = {"x": rows(0, T, D), "ig": rows(1, T, D), "dg": rows(2, T, D), "rate": addr(3), "done": addr(4),
         "reset": addr(17), "init": addr(5), "out": rows(6, T, D), "final": addr(7), "marks": addr(8), "ws": addr(9)}
    a["bytes"] = max(0, lib.rlscan_gated_recurrence_workspace(fmt, E, T, D, 0))
    a.update(kw)
    p = by_reference
    return lib.rlscan_gated_recurrence(fmt, layout, p(a["x"]), p(a["ig"]), p(a["dg"]), a["rate"], a["done"],
                                       a["reset"], a["init"], p(a["out"]), a["final"], a["marks"], a["ws"], a["bytes"], E, T, D, None)


def recurrence_backward(lib, E=2, T=100, D=70, fmt=BF16, layout=0, **kw):
    a = {"do": rows(10, T, D), "x": rows(0, T, D), "ig": rows(1, T, D), "dg": rows(2, T, D), "rate": addr(3),
         "marks": addr(8), "done": addr(4), "reset": addr(17), "d_final": addr(5), "dx": rows(11, T, D), "di": rows(12, T, D),
         "dr": rows(13, T, D), "d_rate": addr(14), "d_init": addr(15), "ws": addr(9)}
    a["bytes"] = max(0, lib.rlscan_gated_recurrence_workspace(fmt, E, T, D, 1))
    a.update(kw)
    p = by_reference
    return lib.rlscan_gated_recurrence_backward(
        fmt, layout, p(a["do"]), p(a["x"]), p(a["ig"]), p(a["dg"]), a["rate"], a["marks"], a["done"], a["reset"], a["d_final"],
        p(a["dx"]), p(a["di"]), p(a["dr"]), a["d_rate"], a["d_init"], a["ws"], a["bytes"], E, T, D, None)


def recurrence_step(lib, E=3, S=5, D=70, fmt=BF16, **kw):
    a = {"x": rows(0, 1, D), "ig": rows(1, 1, D), "dg": rows(2, 1, D), "rate": addr(3), "reset": addr(4),
         "slots": addr(5), "state": addr(6), "out": rows(7, 1, D)}
    a.update(kw)
    p = by_reference
    return lib.rlscan_gated_recurrence_step(fmt, p(a["x"]), p(a["ig"]), p(a["dg"]), a["rate"], a["reset"], a["slots"],
                                            a["state"], p(a["out"]), E, S, D, None)


@pytest.mark.parametrize("call", [recurrence, recurrence_backward])
def test_recurrence_sizes(lib, call):
    assert call(lib, E=-1) == ERR_SHAPE
    assert call(lib, T=-1) == ERR_SHAPE
    assert call(lib, T=2 ** 30) == ERR_SHAPE
    assert call(lib, D=-1) == ERR_SHAPE
    assert call(lib, E=2 ** 20, T=2 ** 20, D=2 ** 10) == ERR_SHAPE
    assert call(lib, E=2 ** 22, T=1) == ERR_SHAPE  # more blocks than a launch takes
    assert call(lib, D=2 ** 30) == ERR_SHAPE
    assert call(lib, fmt=3) == ERR_PARAM
    assert call(lib, layout=2) == ERR_PARAM
    assert call(lib, E=1, T=4000, bytes=0) == ERR_WORKSPACE
    assert call(lib, E=1, T=4000, ws=None) == ERR_NULL
    assert call(lib, E=1, T=4000, ws=addr(9) + 4) == ERR_ALIGN
    assert call(lib, D=0) == OK


def test_recurrence_pointers(lib):
    for name in ("x", "ig", "dg", "rate", "out"):
        assert recurrence(lib, **{name: None}) == ERR_NULL, name
    for name in ("do", "x", "ig", "dg", "rate", "marks", "dx", "di", "dr", "d_rate"):
        assert recurrence_backward(lib, **{name: None}) == ERR_NULL, name
    assert recurrence(lib, x=rows(0, 100, 70, offset=1)) == ERR_ALIGN
    assert recurrence(lib, fmt=F32, out=rows(6, 100, 70, offset=2)) == ERR_ALIGN
    for name, i in (("rate", 3), ("init", 5), ("final", 7), ("marks", 8)):
        assert recurrence(lib, **{name: addr(i) + 2}) == ERR_ALIGN, name
    for name, i in (("rate", 3), ("marks", 8), ("d_final", 5), ("d_rate", 14), ("d_init", 15)):
        assert recurrence_backward(lib, **{name: addr(i) + 2}) == ERR_ALIGN, name


def test_recurrence_strides_and_overlap(lib):
    assert recurrence(lib, x=rows(0, 100, 70, step=-70)) == ERR_SHAPE
    assert recurrence(lib, x=rows(0, 100, 70, env=2 ** 60)) == ERR_SHAPE
    # an output that holds an element twice
    assert recurrence(lib, out=rows(6, 100, 70, env=0)) == ERR_ALIAS
    assert recurrence(lib, out=rows(6, 100, 70, step=69)) == ERR_ALIAS
    # outputs on inputs, on each other and on the workspace
    for name in ("x", "ig", "dg"):
        assert recurrence(lib, out=rows({"x": 0, "ig": 1, "dg": 2}[name], 100, 70)) == ERR_ALIAS, name
    assert recurrence(lib, final=addr(5)) == ERR_ALIAS
    assert recurrence(lib, marks=addr(4)) == ERR_ALIAS
    assert recurrence(lib, marks=addr(17)) == ERR_ALIAS
    assert recurrence(lib, marks=addr(7)) == ERR_ALIAS
    assert recurrence(lib, E=1, T=4000, marks=addr(9)) == ERR_ALIAS
    assert recurrence_backward(lib, dx=rows(11, 100, 70), di=rows(11, 100, 70)) == ERR_ALIAS
    assert recurrence_backward(lib, dx=rows(10, 100, 70)) == ERR_ALIAS
    assert recurrence_backward(lib, d_rate=addr(3)) == ERR_ALIAS
    assert recurrence_backward(lib, d_init=addr(5)) == ERR_ALIAS
    assert recurrence_backward(lib, d_init=addr(8)) == ERR_ALIAS
    assert recurrence_backward(lib, d_rate=addr(17)) == ERR_ALIAS


def test_recurrence_workspace(lib):
    size = lib.rlscan_gated_recurrence_workspace
    assert size(BF16, 4096, 256, 64, 0) == 0  # enough rows: no segments
    assert size(BF16, 1, 32768, 1280, 0) > 0
    assert size(BF16, 2, 10, 64, 1) > 0  # shares of d_rate
    assert size(BF16, 1, 10, 64, 1) == 0
    assert size(BF16, 0, 10, 64, 1) == 0
    assert size(BF16, -1, 10, 64, 0) == -1
    assert size(5, 1, 10, 64, 0) == -1
    # shares of d_rate stay small however many rows there are
    assert size(F32, 2 ** 20, 4, 64, 1) < 16 << 20


def test_step_refusals(lib):
    call = recurrence_step
    assert call(lib, E=-1) == ERR_SHAPE
    assert call(lib, S=-1) == ERR_SHAPE
    assert call(lib, S=2, slots=None) == ERR_SHAPE
    assert call(lib, D=-5) == ERR_SHAPE
    assert call(lib, fmt=7) == ERR_PARAM
    assert call(lib, E=0) == OK
    for name in ("x", "ig", "dg", "rate", "state", "out"):
        assert call(lib, **{name: None}) == ERR_NULL, name
    for name, i in (("rate", 3), ("slots", 5), ("state", 6)):
        assert call(lib, **{name: addr(i) + 2}) == ERR_ALIGN, name
    assert call(lib, out=rows(0, 1, 70)) == ERR_ALIAS
    assert call(lib, state=addr(3)) == ERR_ALIAS
    assert call(lib, out=rows(7, 1, 70, env=3)) == ERR_ALIAS


def test_binding_refuses_other_tensors():
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="GPU"):
        rl.gated_recurrence(x, x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="3 dimensions"):
        rl.gated_recurrence(x[0], x, x, torch.zeros(4))
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        rl.gated_recurrence(x.double(), x, x, torch.zeros(4))
    with pytest.raises(TypeError):
        rl.gated_recurrence([1.0], x, x, torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        rl.gated_recurrence_step(x[0], x[0], x[0], torch.zeros(4), torch.zeros(2, 4))


# ------------------------------------------------------------------ heads
def heads(i, T, H, D, offset=0, env=None, step=None, head=None):
    return _Heads(addr(i) + offset, T * H * D if env is None else env, H * D if step is None else step,
                  D if head is None else head)


def norm_rotate(lib, E=2, T=10, H=4, Hk=2, D=64, rotate=64, base=10000.0, inter=0, eps=1e-6, fmt=BF16, layout=0, **kw):
    a = {"q": heads(0, T, H, D), "k": heads(1, T, Hk, D), "qw": addr(2), "kw": addr(3), "pos": addr(4),
         "qo": heads(5, T, H, D), "ko": heads(6, T, Hk, D)}
    a.update(kw)
    p = by_reference
    return lib.rlscan_norm_rotate_heads(fmt, layout, p(a["q"]), p(a["k"]), a["qw"], a["kw"], a["pos"], p(a["qo"]),
                                        p(a["ko"]), E, T, H, Hk, D, rotate, base, inter, eps, None)


def norm_rotate_backward(lib, E=2, T=10, H=4, Hk=2, D=64, rotate=64, base=10000.0, inter=0, eps=1e-6, fmt=BF16,
                         layout=0, **kw):
    a = {"q": heads(0, T, H, D), "k": heads(1, T, Hk, D), "qw": addr(2), "kw": addr(3), "pos": addr(4),
         "gq": heads(5, T, H, D), "gk": heads(6, T, Hk, D), "dq": heads(7, T, H, D), "dk": heads(8, T, Hk, D),
         "dqw": addr(9), "dkw": addr(10), "ws": addr(11)}
    a["bytes"] = max(0, lib.rlscan_norm_rotate_heads_workspace(E, T, H, Hk, D))
    a.update(kw)
    p = by_reference
    return lib.rlscan_norm_rotate_heads_backward(
        fmt, layout, p(a["gq"]), p(a["gk"]), p(a["q"]), p(a["k"]), a["qw"], a["kw"], a["pos"], p(a["dq"]), p(a["dk"]),
        a["dqw"], a["dkw"], a["ws"], a["bytes"], E, T, H, Hk, D, rotate, base, inter, eps, None)


@pytest.mark.parametrize("call", [norm_rotate, norm_rotate_backward])
def test_heads_refusals(lib, call):
    for bad in (dict(E=-1), dict(T=-1), dict(T=2 ** 30), dict(H=-1), dict(Hk=-1), dict(D=0), dict(D=257, rotate=0),
                dict(rotate=-2), dict(rotate=66), dict(rotate=33), dict(E=2 ** 40, T=2 ** 20), dict(H=2 ** 50)):
        assert call(lib, **bad) == ERR_SHAPE, bad
    for bad in (dict(fmt=3), dict(layout=2), dict(base=0.0), dict(base=-1.0), dict(base=float("inf")),
                dict(base=float("nan")), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(lib, **bad) == ERR_PARAM, bad
    assert call(lib, pos=None) == ERR_NULL
    for name, i in (("qw", 2), ("kw", 3), ("pos", 4)):
        assert call(lib, **{name: addr(i) + 2}) == ERR_ALIGN, name
    assert call(lib, q=heads(0, 10, 4, 64, offset=1)) == ERR_ALIGN
    assert call(lib, q=heads(0, 10, 4, 64, head=-1)) == ERR_SHAPE
    names = ("q", "k", "qo", "ko") if call is norm_rotate else ("q", "k", "gq", "gk", "dq", "dk", "ws")
    for name in names:
        assert call(lib, **{name: None}) == ERR_NULL, name


def test_heads_overlap(lib):
    assert norm_rotate(lib, qo=heads(0, 10, 4, 64)) == ERR_ALIAS  # not in place
    assert norm_rotate(lib, qo=heads(4, 10, 4, 64)) == ERR_ALIAS
    assert norm_rotate(lib, ko=heads(5, 10, 2, 64)) == ERR_ALIAS
    assert norm_rotate(lib, qo=heads(5, 10, 4, 64, head=63)) == ERR_ALIAS
    assert norm_rotate(lib, qo=heads(5, 10, 4, 64, env=0)) == ERR_ALIAS
    call = norm_rotate_backward
    assert call(lib, dq=heads(5, 10, 4, 64)) == ERR_ALIAS
    assert call(lib, dqw=addr(10)) == ERR_ALIAS
    assert call(lib, dqw=addr(2)) == ERR_ALIAS
    assert call(lib, ws=addr(7)) == ERR_ALIAS
    assert call(lib, bytes=64) == ERR_WORKSPACE
    assert call(lib, ws=addr(11) + 8) == ERR_ALIGN
    assert norm_rotate(lib, E=0) == OK
    assert norm_rotate(lib, H=0, Hk=0, q=None, k=None, qo=None, ko=None) == OK
    assert call(lib, T=0, dqw=None, dkw=None) == OK
    assert lib.rlscan_norm_rotate_heads_workspace(2, 10, 4, 2, 300) == -1
    assert lib.rlscan_norm_rotate_heads_workspace(-1, 10, 4, 2, 64) == -1
    assert 0 < lib.rlscan_norm_rotate_heads_workspace(2 ** 12, 2 ** 12, 16, 16, 128) <= 2 << 20


# ------------------------------------------------------------------ tables
def embed(lib, R=100, N=50, D=64, fmt=BF16, scale=1.0, table_stride=64, out_stride=64, table=addr(0), tokens=addr(1),
          out=addr(2)):
    return lib.rlscan_embed_tokens(fmt, table, table_stride, tokens, out, out_stride, R, N, D, scale, None)


def embed_backward(lib, R=2000, N=50, D=64, fmt=BF16, scale=1.0, table_stride=64, out_stride=64, table=addr(0),
                   tokens=addr(1), out=addr(2), ws=addr(3), need=None):
    if need is None:
        need = max(0, lib.rlscan_embed_tokens_workspace(R, N, D))
    return lib.rlscan_embed_tokens_backward(fmt, out, out_stride, tokens, table, table_stride, ws, need, R, N, D, scale,
                                            None)


@pytest.mark.parametrize("call", [embed, embed_backward])
def test_table_refusals(lib, call):
    for bad in (dict(R=-1), dict(R=2 ** 26 + 1), dict(N=0), dict(N=-1), dict(N=2 ** 20 + 1), dict(D=0),
                dict(D=32769, table_stride=40000, out_stride=40000), dict(R=2 ** 25, D=129, table_stride=129, out_stride=129),
                dict(table_stride=63), dict(out_stride=63), dict(table_stride=-64), dict(out_stride=2 ** 45)):
        assert call(lib, **bad) == ERR_SHAPE, bad
    for bad in (dict(fmt=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(lib, **bad) == ERR_PARAM, bad
    for name in ("table", "tokens", "out"):
        assert call(lib, **{name: None}) == ERR_NULL, name
    assert call(lib, tokens=addr(1) + 4) == ERR_ALIGN
    assert call(lib, table=addr(0) + 1) == ERR_ALIGN
    assert call(lib, fmt=F32, out=addr(2) + 2) == ERR_ALIGN
    assert call(lib, out=addr(0)) == ERR_ALIAS
    if call is embed:
        assert call(lib, out=addr(1)) == ERR_ALIAS
        assert call(lib, R=0) == OK
    else:
        assert call(lib, table=addr(1)) == ERR_ALIAS
        assert call(lib, ws=None) == ERR_NULL
        assert call(lib, ws=addr(3) + 8) == ERR_ALIGN
        assert call(lib, ws=addr(2)) == ERR_ALIAS
        assert call(lib, need=16) == ERR_WORKSPACE


def test_table_workspace(lib):
    size = lib.rlscan_embed_tokens_workspace
    assert size(1024, 1000, 8) == 0  # few tokens: one launch
    assert size(1025, 10, 8) > 0 and size(1025, 1000, 8) > 0
    assert size(-1, 10, 8) == -1 and size(10, 0, 8) == -1 and size(10, 2 ** 21, 8) == -1 and size(10, 10, 0) == -1
    # four copies of the tokens, and two float32 rows for 32 tokens
    assert size(2 ** 20, 2 ** 16, 512) < 16 * 2 ** 20 + 2 ** 20 * 512 * 4 // 16 + (1 << 20)


def test_binding_refuses_other_heads_and_tables():
    q, k, pos = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 2, 8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        rl.norm_rotate_heads(q, k, positions=pos)
    with pytest.raises(ValueError, match="must be"):
        rl.norm_rotate_heads(q[0, 0], k[0, 0])
    with pytest.raises(TypeError):
        rl.norm_rotate_heads(q.long(), k)
    with pytest.raises(ValueError, match="GPU"):
        rl.embed_tokens(torch.zeros(3, 4), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        rl.embed_tokens_backward([1.0], torch.zeros(2, dtype=torch.int64), 3)
    with pytest.raises(ValueError, match="GPU"):
        rl.embed_tokens_backward(torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64), 3)
