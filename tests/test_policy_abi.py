"""The policy operators without a GPU: refusals of the C ABI and of the Python
binding, workspace sizes, and the test oracle's own gradients.

Every call below is refused (or has nothing to do) before any HIP call.
"""
from __future__ import annotations

import ctypes
import math
import os

import pytest
import torch

import linear_recurrence_scan_reverse_amd as rl
from linear_recurrence_scan_reverse_amd.policy import _Heads
from tests import policy_oracle as po

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


def heads(i, E, T, H, D, offset=0, env=None, step=None, head=None):
    return _Heads(addr(i) + offset, T * H * D if env is None else env, H * D if step is None else step,
                  D if head is None else head)


def forward(lib, E=2, T=100, H=4, Hkv=2, K=64, V=32, fmt=BF16, layout=0, per_step=1, scale=0.125, **kw):
    a = {"q": heads(0, E, T, H, K), "k": heads(1, E, T, Hkv, K), "v": heads(2, E, T, Hkv, V), "g": addr(3),
         "done": addr(4), "init": addr(5), "out": heads(6, E, T, H, V), "final": addr(7), "ws": addr(8)}
    a["bytes"] = max(0, lib.rlscan_linear_attention_workspace(fmt, E, T, H, Hkv, K, V, 0))
    a.update(kw)
    p = lambda x: ctypes.byref(x) if isinstance(x, _Heads) else x
    return lib.rlscan_linear_attention(fmt, layout, p(a["q"]), p(a["k"]), p(a["v"]), a["g"], per_step, a["done"],
                                       a["init"], p(a["out"]), a["final"], a["ws"], a["bytes"], E, T, H, Hkv, K, V,
                                       scale, None)


def backward(lib, E=2, T=100, H=4, Hkv=2, K=64, V=32, fmt=BF16, layout=0, per_step=1, scale=0.125, **kw):
    a = {"do": heads(9, E, T, H, V), "q": heads(0, E, T, H, K), "k": heads(1, E, T, Hkv, K),
         "v": heads(2, E, T, Hkv, V), "g": addr(3), "done": addr(4), "init": addr(5), "d_final": addr(6),
         "dq": heads(10, E, T, H, K), "dk": heads(11, E, T, Hkv, K), "dv": heads(12, E, T, Hkv, V), "dg": addr(13),
         "d_init": addr(14), "ws": addr(15)}
    a["bytes"] = max(0, lib.rlscan_linear_attention_workspace(fmt, E, T, H, Hkv, K, V, 1))
    a.update(kw)
    p = lambda x: ctypes.byref(x) if isinstance(x, _Heads) else x
    return lib.rlscan_linear_attention_backward(
        fmt, layout, p(a["do"]), p(a["q"]), p(a["k"]), p(a["v"]), a["g"], per_step, a["done"], a["init"], a["d_final"],
        p(a["dq"]), p(a["dk"]), p(a["dv"]), a["dg"], a["d_init"], a["ws"], a["bytes"], E, T, H, Hkv, K, V, scale, None)


def step(lib, E=3, S=5, H=4, Hkv=2, K=64, V=32, fmt=BF16, per_row=1, scale=0.125, **kw):
    a = {"q": heads(0, E, 1, H, K), "k": heads(1, E, 1, Hkv, K), "v": heads(2, E, 1, Hkv, V), "g": addr(3),
         "reset": addr(4), "slots": addr(5), "state": addr(6), "out": heads(7, E, 1, H, V)}
    a.update(kw)
    p = lambda x: ctypes.byref(x) if isinstance(x, _Heads) else x
    return lib.rlscan_linear_attention_step(fmt, p(a["q"]), p(a["k"]), p(a["v"]), a["g"], per_row, a["reset"],
                                            a["slots"], a["state"], p(a["out"]), E, S, H, Hkv, K, V, scale, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_sizes(lib, call):
    assert call(lib, E=-1) == ERR_SHAPE
    assert call(lib, T=-1) == ERR_SHAPE
    assert call(lib, T=2 ** 30) == ERR_SHAPE
    assert call(lib, K=0) == ERR_SHAPE
    assert call(lib, V=0) == ERR_SHAPE
    assert call(lib, K=129) == ERR_SHAPE
    assert call(lib, V=129) == ERR_SHAPE
    assert call(lib, H=4, Hkv=3) == ERR_SHAPE
    assert call(lib, H=4, Hkv=0) == ERR_SHAPE
    assert call(lib, E=2 ** 40, T=2 ** 20) == ERR_SHAPE
    assert call(lib, E=2 ** 24, T=1) == ERR_SHAPE  # more blocks than a launch takes
    assert call(lib, fmt=3) == ERR_PARAM
    assert call(lib, layout=2) == ERR_PARAM
    assert call(lib, scale=math.nan) == ERR_PARAM
    assert call(lib, scale=math.inf) == ERR_PARAM


def test_attention_pointers(lib):
    for name in ("q", "k", "v", "g", "out"):
        assert forward(lib, **{name: None}) == ERR_NULL, name
    for name in ("do", "q", "k", "v", "g", "dq", "dk", "dv", "dg", "ws"):
        assert backward(lib, **{name: None}) == ERR_NULL, name
    assert forward(lib, q=_Heads(None, 1, 1, 1)) == ERR_NULL
    assert forward(lib, q=heads(0, 2, 100, 4, 64, offset=1)) == ERR_ALIGN
    assert forward(lib, fmt=F32, q=heads(0, 2, 100, 4, 64, offset=2)) == ERR_ALIGN
    assert forward(lib, g=addr(3) + 2) == ERR_ALIGN
    assert forward(lib, init=addr(5) + 2) == ERR_ALIGN
    assert backward(lib, ws=addr(15) + 4) == ERR_ALIGN
    assert backward(lib, dg=addr(13) + 1) == ERR_ALIGN
    assert backward(lib, bytes=16) == ERR_WORKSPACE
    assert lib.rlscan_status_string(ERR_WORKSPACE) != b"unknown status"


def test_attention_strides_and_overlap(lib):
    assert forward(lib, q=heads(0, 2, 100, 4, 64, step=-256)) == ERR_SHAPE
    assert forward(lib, q=heads(0, 2, 100, 4, 64, env=2 ** 60)) == ERR_SHAPE
    # an output that holds an element twice: broadcast, or rows that run into each other
    assert forward(lib, out=heads(6, 2, 100, 4, 32, env=0)) == ERR_ALIAS
    assert forward(lib, out=heads(6, 2, 100, 4, 32, head=31)) == ERR_ALIAS
    assert forward(lib, out=heads(6, 2, 100, 4, 32, step=127)) == ERR_ALIAS
    # outputs on inputs, on each other and on the workspace
    assert forward(lib, out=heads(0, 2, 100, 4, 32)) == ERR_ALIAS
    assert forward(lib, final=addr(5)) == ERR_ALIAS
    assert forward(lib, final=addr(4)) == ERR_ALIAS
    assert backward(lib, dq=heads(0, 2, 100, 4, 64)) == ERR_ALIAS
    assert backward(lib, dk=heads(10, 2, 100, 2, 64)) == ERR_ALIAS
    assert backward(lib, dg=addr(3)) == ERR_ALIAS
    assert backward(lib, ws=addr(13)) == ERR_ALIAS
    assert backward(lib, d_init=addr(5)) == ERR_ALIAS
    # slices of one buffer side by side may interleave, but not by one element too many
    E, T, H, Hkv, K, V = 2, 100, 4, 2, 64, 32
    row = H * K + Hkv * K + Hkv * V
    part = lambda i, o: heads(i, E, T, H, K, offset=2 * o, env=T * row, step=row)
    over = {"dq": part(10, 0), "dk": part(10, H * K - 8)}
    over["dk"].head = K
    assert backward(lib, **over) == ERR_ALIAS
    # nothing to do is no error and touches nothing
    assert forward(lib, E=0, q=None, k=None, v=None, out=None) == OK
    assert forward(lib, T=0, final=None, q=None, k=None, v=None, out=None) == OK
    assert backward(lib, E=0, do=None, q=None, k=None, v=None, dq=None, dk=None, dv=None) == OK
    assert step(lib, E=0, q=None, k=None, v=None, out=None) == OK
    # ... after the checks of sizes and parameters
    assert forward(lib, E=0, K=200) == ERR_SHAPE


def test_workspace_sizes(lib):
    ws = lib.rlscan_linear_attention_workspace
    assert ws(BF16, 64, 128, 16, 16, 64, 64, 0) == 0  # enough heads: no segments
    assert ws(BF16, 1, 32768, 1, 1, 64, 64, 0) > 0
    assert ws(BF16, 0, 128, 4, 4, 64, 64, 1) == 0
    assert ws(BF16, 2, 128, 4, 2, 64, 64, 1) > ws(BF16, 2, 128, 4, 4, 64, 64, 1) > 0
    assert ws(BF16, 2, 128, 4, 4, 129, 64, 1) == -1
    assert ws(BF16, 2, 128, 4, 3, 64, 64, 1) == -1
    assert ws(7, 2, 128, 4, 4, 64, 64, 1) == -1
    lp = lib.rlscan_action_log_probs_workspace
    assert lp(16384, 18) == 0 and lp(1, 131072) > 0
    assert lp(-1, 4) == -1 and lp(4, 0) == -1 and lp(2 ** 25, 4) == -1


def test_step_refusals(lib):
    assert step(lib, K=129) == ERR_SHAPE
    assert step(lib, S=-1) == ERR_SHAPE
    assert step(lib, slots=None, S=2) == ERR_SHAPE
    assert step(lib, E=2 ** 23, S=2 ** 23, H=1, Hkv=1) == ERR_SHAPE
    assert step(lib, scale=math.nan) == ERR_PARAM
    assert step(lib, fmt=5) == ERR_PARAM
    for name in ("q", "k", "v", "g", "state", "out"):
        assert step(lib, **{name: None}) == ERR_NULL, name
    assert step(lib, state=addr(6) + 2) == ERR_ALIGN
    assert step(lib, slots=addr(5) + 2) == ERR_ALIGN
    assert step(lib, state=addr(3)) == ERR_ALIAS
    assert step(lib, out=heads(0, 3, 1, 4, 32)) == ERR_ALIAS
    assert step(lib, out=heads(7, 3, 1, 4, 32, env=0)) == ERR_ALIAS


def sample(lib, R=4, N=100, fmt=F32, stride=None, t=1.0, k=0, p=1.0, m=0.0, **kw):
    a = {"x": addr(0), "mask": addr(1), "u": addr(2), "ts": None, "ks": None, "ps": None, "ms": None, "a": addr(3),
         "lp": addr(4)}
    a.update(kw)
    return lib.rlscan_sample_actions(fmt, a["x"], N if stride is None else stride, a["mask"], a["u"], a["ts"], a["ks"],
                                     a["ps"], a["ms"], t, k, p, m, a["a"], a["lp"], R, N, None)


def test_sample_refusals(lib):
    assert sample(lib, R=-1) == ERR_SHAPE
    assert sample(lib, R=2 ** 22) == ERR_SHAPE
    assert sample(lib, N=0) == ERR_SHAPE
    assert sample(lib, N=2 ** 20 + 1) == ERR_SHAPE
    assert sample(lib, stride=99) == ERR_SHAPE
    assert sample(lib, fmt=4) == ERR_PARAM
    for t in (-1.0, math.nan, math.inf):
        assert sample(lib, t=t) == ERR_PARAM
    for p in (0.0, -0.5, math.nan):
        assert sample(lib, p=p) == ERR_PARAM
    for m in (-0.1, 1.1, math.nan):
        assert sample(lib, m=m) == ERR_PARAM
    assert sample(lib, k=-1) == ERR_PARAM
    for name in ("x", "u", "a"):
        assert sample(lib, **{name: None}) == ERR_NULL, name
    assert sample(lib, x=addr(0) + 2) == ERR_ALIGN
    assert sample(lib, a=addr(3) + 4) == ERR_ALIGN
    assert sample(lib, ks=addr(5) + 1) == ERR_ALIGN
    assert sample(lib, a=addr(0)) == ERR_ALIAS
    assert sample(lib, lp=addr(2)) == ERR_ALIAS
    assert sample(lib, lp=addr(3)) == ERR_ALIAS
    assert sample(lib, R=0, x=None, u=None, a=None) == OK


def log_probs(lib, R=4, N=100, fmt=F32, stride=None, t=1.0, **kw):
    a = {"x": addr(0), "mask": addr(1), "a": addr(2), "lp": addr(3), "ent": addr(4), "lse": addr(5), "ws": addr(6)}
    a["bytes"] = max(0, lib.rlscan_action_log_probs_workspace(R, N))
    a.update(kw)
    return lib.rlscan_action_log_probs(fmt, a["x"], N if stride is None else stride, a["mask"], a["a"], t, a["lp"],
                                       a["ent"], a["lse"], a["ws"], a["bytes"], R, N, None)


def log_probs_backward(lib, R=4, N=100, fmt=F32, stride=None, d_stride=None, t=1.0, **kw):
    a = {"dlp": addr(7), "dent": addr(8), "x": addr(0), "mask": addr(1), "a": addr(2), "lse": addr(5), "ent": addr(4),
         "dx": addr(9)}
    a.update(kw)
    return lib.rlscan_action_log_probs_backward(fmt, a["dlp"], a["dent"], a["x"], N if stride is None else stride,
                                                a["mask"], a["a"], t, a["lse"], a["ent"], a["dx"],
                                                N if d_stride is None else d_stride, R, N, None)


def test_log_prob_refusals(lib):
    for call in (log_probs, log_probs_backward):
        assert call(lib, R=-1) == ERR_SHAPE
        assert call(lib, R=2 ** 24) == ERR_SHAPE
        assert call(lib, N=0) == ERR_SHAPE
        assert call(lib, stride=99) == ERR_SHAPE
        assert call(lib, fmt=4) == ERR_PARAM
        for t in (0.0, -1.0, math.nan, math.inf, 1e-40):
            assert call(lib, t=t) == ERR_PARAM
        assert call(lib, x=None) == ERR_NULL
        assert call(lib, a=None) == ERR_NULL
        assert call(lib, x=addr(0) + 1) == ERR_ALIGN
        assert call(lib, a=addr(2) + 4) == ERR_ALIGN
    assert log_probs(lib, lse=None) == ERR_NULL
    assert log_probs(lib, R=1, N=131072, bytes=0) == ERR_WORKSPACE
    assert log_probs(lib, R=1, N=131072, ws=None) == ERR_NULL
    assert log_probs(lib, lp=addr(4)) == ERR_ALIAS
    assert log_probs(lib, lp=addr(0)) == ERR_ALIAS
    assert log_probs_backward(lib, d_stride=99) == ERR_SHAPE
    assert log_probs_backward(lib, R=2 ** 20, N=2 ** 29) == ERR_SHAPE
    assert log_probs_backward(lib, dx=None) == ERR_NULL
    assert log_probs_backward(lib, dx=addr(0)) == ERR_ALIAS
    assert log_probs_backward(lib, dx=addr(5)) == ERR_ALIAS
    assert log_probs(lib, R=0, x=None, a=None) == OK


def test_python_refuses_cpu_tensors_and_wrong_ones():
    q = torch.zeros(2, 5, 4, 8)
    g = torch.zeros(2, 5, 4)
    with pytest.raises(ValueError, match="GPU"):
        rl.linear_attention(q, q, q, g)
    with pytest.raises(ValueError, match="GPU"):
        rl.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], torch.zeros(2, 4, 8, 8))
    with pytest.raises(ValueError, match="GPU"):
        rl.sample_actions(torch.zeros(3, 7), torch.zeros(3))
    with pytest.raises(ValueError, match="GPU"):
        rl.action_log_probs(torch.zeros(3, 7), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        rl.linear_attention(q.double(), q, q, g)
    with pytest.raises(ValueError):
        rl.linear_attention(q[0], q, q, g)
    with pytest.raises(TypeError):
        rl.sample_actions([1.0], torch.zeros(1))
    with pytest.raises(ValueError):
        rl.sample_actions(torch.zeros(3, 0), torch.zeros(3))


def test_row_strides():
    from linear_recurrence_scan_reverse_amd.policy import _row_stride
    x = torch.zeros(4, 6, 10)
    assert _row_stride(x, "x") == 10
    assert _row_stride(x[:, :, :7], "x") == 10
    assert _row_stride(x[:, 2], "x") == 60
    assert _row_stride(x[:1, 2:3, :3], "x") == 3
    with pytest.raises(ValueError):
        _row_stride(x[:, :5], "x")
    with pytest.raises(ValueError):
        _row_stride(x.transpose(1, 2), "x")


# ------------------------------------------------------------------ the oracle's own gradients
def _random(seed, E=2, T=7, H=4, Hkv=2, K=3, V=5, per_step=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    d = {"q": n(E, T, H, K), "k": n(E, T, Hkv, K), "v": n(E, T, Hkv, V),
         "g": -torch.rand((E, T, H) if per_step else (H,), generator=gen, dtype=torch.float64),
         "init": n(E, H, K, V), "do": n(E, T, H, V), "df": n(E, H, K, V),
         "done": (torch.rand(E, T, generator=gen) < 0.25).to(torch.uint8)}
    return d


@pytest.mark.parametrize("per_step", [True, False])
@pytest.mark.parametrize("last", [0, 1])
def test_oracle_gradient_is_the_difference_quotient(per_step, last):
    d = _random(3, per_step=per_step)
    d["done"][:, -1] = last

    def loss(**kw):
        x = dict(d, **kw)
        out, final = po.linear_attention(x["q"], x["k"], x["v"], x["g"], x["done"], x["init"])
        return float((out * d["do"]).sum() + (final * d["df"]).sum())

    grads = po.linear_attention_backward(d["do"], d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], d["df"])
    for name, grad in zip(("q", "k", "v", "g", "init"), grads):
        x = d[name]
        gen = torch.Generator().manual_seed(1)
        way = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        h = 1e-5  # central differences: error h^2 * third derivative (about 1e-9) + 1e-16 / h * loss (about 1e-9)
        slope = (loss(**{name: x + h * way}) - loss(**{name: x - h * way})) / (2 * h)
        assert abs(slope - float((grad * way).sum())) < 1e-6 * (1 + abs(slope)), name


def test_oracle_episodes_are_separate_rows():
    """A packed row equals its episodes run one by one."""
    d = _random(5, E=1, T=9)
    d["done"].zero_()
    d["done"][0, 3] = d["done"][0, 4] = 1
    out, final = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"])
    for lo, hi, init in ((0, 4, d["init"]), (4, 5, None), (5, 9, None)):
        part, last = po.linear_attention(d["q"][:, lo:hi], d["k"][:, lo:hi], d["v"][:, lo:hi], d["g"][:, lo:hi], None,
                                         init)
        assert torch.allclose(part, out[:, lo:hi], rtol=1e-12, atol=1e-12)
    assert torch.allclose(final, last, rtol=1e-12, atol=1e-12)


def test_oracle_log_prob_gradient_is_the_difference_quotient():
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(5, 9, generator=gen, dtype=torch.float64) * 3
    a = torch.tensor([0, 8, 3, -1, 4])
    mask = torch.ones(5, 9, dtype=torch.uint8)
    mask[0, 3:6] = 0
    dlp, den = torch.randn(5, generator=gen, dtype=torch.float64), torch.randn(5, generator=gen, dtype=torch.float64)
    grad, _ = po.log_probs_backward(dlp, den, x, a, 0.7, mask)

    def loss(x):
        lp, ent, _ = po.log_probs(x, a, 0.7, mask)
        return float((lp * dlp).sum() + (ent * den).sum())

    way = torch.randn(5, 9, generator=gen, dtype=torch.float64)
    h = 1e-5
    slope = (loss(x + h * way) - loss(x - h * way)) / (2 * h)
    assert abs(slope - float((grad * way).sum())) < 1e-6 * (1 + abs(slope))
