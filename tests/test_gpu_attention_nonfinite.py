"""Linear attention with inf and NaN in some steps: they stay within their episode and reach no
earlier output, as in the recurrence taken step by step, where an episode starts from a zero state.

The oracle runs each episode by itself in float64.  Where it is finite the result has to be, with the
tolerances of test_gpu_linear_attention; elsewhere it has to be inf or NaN.  The log-decay's
gradient is a difference of sums over an episode: checked in episodes without such steps.
"""
import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl
from tests import policy_oracle as po
from tests.test_gpu_linear_attention import TERMS, gpu, half_step, make

pytestmark = pytest.mark.gpu

F32 = TERMS[torch.float32]


def _episodes(d, e):
    """[lo, hi) of row e's episodes: a step after a flagged one, or with a decay below the cut, starts one."""
    T = d["q"].shape[1]
    starts = [t for t in range(1, T) if (d["done"] is not None and d["done"][e, t - 1] != 0)
              or bool((d["g"][e, t] < po.CUT_BELOW).all())]
    return list(zip([0] + starts, starts + [T]))


def _forward(d, magnitude=False):
    E, T, H, K = d["q"].shape
    V = d["v"].shape[3]
    out, final = torch.zeros(E, T, H, V, dtype=torch.float64), torch.zeros(E, H, K, V, dtype=torch.float64)
    for e in range(E):
        for lo, hi in _episodes(d, e):
            part = [d[n][e:e + 1, lo:hi] for n in ("q", "k", "v", "g")]
            init = d["init"][e:e + 1] if lo == 0 and d["init"] is not None else None
            out[e:e + 1, lo:hi], last = po.linear_attention(*part, None, init, magnitude=magnitude)
        if d["done"] is None or d["done"][e, -1] == 0:
            final[e] = last
    return out, final


def _backward(d, magnitude=False):
    E, T, H, K = d["q"].shape
    grads = [torch.zeros(d[n].shape, dtype=torch.float64) for n in ("q", "k", "v", "g", "init")]
    for e in range(E):
        for lo, hi in _episodes(d, e):
            part = [d[n][e:e + 1, lo:hi] for n in ("do", "q", "k", "v", "g")]
            init = d["init"][e:e + 1] if lo == 0 else None
            closed = hi < T or d["done"][e, -1] != 0
            got = po.linear_attention_backward(*part, None, init, None if closed else d["df"][e:e + 1],
                                               magnitude=magnitude)
            for to, x in zip(grads, got[:4]):
                to[e:e + 1, lo:hi] = x
            if lo == 0:
                grads[4][e] = got[4][0]
            else:
                grads[3][e, lo] = 0  # across a cut, whatever lies on its two sides
    return grads


def _agree(got, want, size, terms, what, where=None):
    got = got.cpu()
    where = torch.ones_like(want, dtype=torch.bool) if where is None else where
    finite = torch.isfinite(want) & torch.isfinite(size)
    wrong = (torch.isfinite(got) != finite) & where
    assert not wrong.any(), "%s: %d elements, first %s" % (what, wrong.sum(), wrong.nonzero()[0].tolist())
    finite &= where
    err = (got.double() - want).abs()[finite]
    tol = (half_step(got.dtype) * want.abs() + terms * size)[finite] + 1e-30
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert err.numel() == 0 or (err / tol).max() <= 1.0, "%s: %.3g times the tolerance" % (what, (err / tol).max())


def _clean(d, names):
    """[E, T]: steps of episodes in which all of these are finite."""
    E, T = d["q"].shape[:2]
    clean = torch.ones(E, T, dtype=torch.bool)
    for e in range(E):
        for lo, hi in _episodes(d, e):
            clean[e, lo:hi] = all(bool(torch.isfinite(d[n][e, lo:hi]).all()) for n in names)
            if lo == 0 and d["init"] is not None:
                clean[e, :hi] &= bool(torch.isfinite(d["init"][e]).all())
            if hi == T and d["df"] is not None and d["done"][e, -1] == 0:
                clean[e, lo:] &= bool(torch.isfinite(d["df"][e]).all())
    return clean


def _check(d):
    dt = d["q"].dtype
    out, final = rl.linear_attention(*(gpu(d[n]) for n in ("q", "k", "v", "g", "done", "init")), with_state=True)
    want, size = _forward(d), _forward(d, True)
    _agree(out, want[0], size[0], TERMS[dt], "out")
    _agree(final, want[1], size[1], F32, "final state")
    got = rl.linear_attention_backward(*(gpu(d[n]) for n in ("do", "q", "k", "v", "g", "done", "init", "df")))
    want, size = _backward(d), _backward(d, True)
    for i, name in enumerate(("dq", "dk", "dv")):
        _agree(got[i], want[i], size[i], TERMS[dt], name)
    _agree(got[4], want[4], size[4], F32, "d_init")
    clean = _clean(d, ("q", "k", "v", "do")).unsqueeze(2).expand_as(d["g"])
    assert clean.any() and not clean.all()
    top = torch.where(clean & torch.isfinite(size[3]), size[3], 0.0).amax(1, keepdim=True).expand_as(size[3])
    _agree(got[3], torch.where(clean, want[3], 0.0), top, F32, "dg", clean)


def _spoil(d, name, steps, value, one=True):
    """Sets one element (or all) of a head of these steps."""
    for n, t in enumerate(steps):
        h = n % d[name].shape[2]
        if one:
            d[name][n % d[name].shape[0], t, h, (7 * n) % d[name].shape[3]] = value
        else:
            d[name][n % d[name].shape[0], t, h] = value


STEPS = (10, 31, 32, 63, 64, 70, 129, 149)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,V", [(64, 64), (40, 24), (33, 65), (128, 128)])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_they_stay_within_their_episode(dtype, K, V, name):
    for value, one in ((float("inf"), True), (float("nan"), False)):
        d = make(K + V, 2, 150, 4, 2, K, V, dtype, p_done=0.08)
        _spoil(d, name, STEPS, value, one)
        _check(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("name", ["k", "v", "do"])
def test_rows_in_segments(dtype, D, name):
    d = make(5, 1, 1100, 1, 1, D, D, dtype, p_done=0.01, decay=0.01)
    fmt = {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    assert rl.lib().rlscan_linear_attention_workspace(fmt, 1, 1100, 1, 1, D, D, 0) > 0
    d["done"][0, -1] = 0
    _spoil(d, name, (3, 300, 511, 700), -float("inf"))
    _check(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_states(dtype, D):
    """An initial state or the final state's gradient that is not finite, with a cut before the row's end, or a decay that cuts."""
    d = make(6, 3, 100, 2, 1, D, D, dtype, p_done=0.0)
    d["done"] = torch.zeros(3, 100, dtype=torch.uint8)
    d["done"][0, 40] = 1
    d["done"][1, 99] = 1
    d["g"][1, 7] = -float("inf")
    d["done"][2, 64] = 1
    d["init"][0, 0, 3, 5] = float("inf")
    d["init"][1, 1] = float("nan")
    d["df"][1, 0] = float("nan")  # of a closed row: not taken
    d["df"][2, 1, 9, 2] = -float("inf")
    _check(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_state_that_overflows(dtype):
    """Finite inputs whose products pass float32: the episodes around keep their values."""
    d = make(7, 1, 200, 1, 1, 64, 64, dtype, p_done=0.0)
    d["done"] = torch.zeros(1, 200, dtype=torch.uint8)
    d["done"][0, [49, 59, 120]] = 1
    for t in (52, 55):
        d["k"][0, t], d["v"][0, t] = 1e30, -1e30
    out = rl.linear_attention(*(gpu(d[n]) for n in ("q", "k", "v", "g", "done", "init"))).cpu()
    got = rl.linear_attention_backward(*(gpu(d[n]) for n in ("do", "q", "k", "v", "g", "done", "init", "df")))
    want, size = _forward(d), _forward(d, True)
    grads, gsize = _backward(d), _backward(d, True)
    clean = torch.ones(1, 200, 1, dtype=torch.bool)
    clean[0, 50:60] = False
    assert not torch.isfinite(out[0, 52:60]).any()
    pick = lambda x: torch.where(clean.unsqueeze(3), x, torch.zeros_like(x))
    _agree(pick(out), pick(want[0]), pick(size[0]), TERMS[d["q"].dtype], "out")
    for i in range(3):
        _agree(pick(got[i].cpu()), pick(grads[i]), pick(gsize[i]), TERMS[d["q"].dtype], "dq dk dv"[3 * i:3 * i + 2])
    top = torch.where(clean, gsize[3], 0.0).amax(1, keepdim=True).expand_as(gsize[3])
    _agree(torch.where(clean, got[3].cpu(), 0.0), torch.where(clean, grads[3], 0.0), top, F32, "dg")


def test_acting_and_learning_agree():
    """Steps that reset a state which is not finite give what the whole row gives."""
    d = make(8, 2, 40, 2, 1, 32, 32, "f32", p_done=0.0)
    d["done"] = torch.zeros(2, 40, dtype=torch.uint8)
    d["done"][:, 19] = 1
    d["v"][0, 10, 1, 4] = float("inf")
    d["k"][1, 15, 0] = float("nan")
    out = rl.linear_attention(*(gpu(d[n]) for n in ("q", "k", "v", "g", "done", "init")))
    state, reset = gpu(d["init"]).clone(), None
    for t in range(40):
        o = rl.linear_attention_step(*(gpu(d[n][:, t].contiguous()) for n in ("q", "k", "v", "g")), state, reset)
        reset = gpu(d["done"][:, t].contiguous())
        assert torch.equal(torch.isfinite(o), torch.isfinite(out[:, t])), t
        assert torch.allclose(o, out[:, t], rtol=1e-4, atol=1e-4, equal_nan=True) or not torch.isfinite(o).all()
    assert torch.isfinite(out[:, 20:]).all() and not torch.isfinite(out[:, :20]).all()
