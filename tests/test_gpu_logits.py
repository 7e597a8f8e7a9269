"""Action sampling and action log-probabilities on the GPU against the float64 oracle.

Sampled actions have to be equal wherever the choice is not next to a border: the
oracle says how near u and the top_p and min_p borders came (``gap``), and both
sides' sums differ by at most N roundings to 2^-43 (2^20 * 2^-44 < 1e-7 for the
longest rows, about 2^-44 * sqrt(N) as they fall); draws nearer than 1e-9 are not used.
Log-probabilities and entropies are float32: half a step of the value (2^-24), and for
what is summed before it float32's rounding of z = (x - max) / temperature (2^-24 |z|
for the difference's quotient), of exp2 (2^-23 and its argument's 2^-24 |z|) and of a sum of
some dozen partial sums, each 2^-24: 2^-20 (1 + |z|).  A gradient adds its own half step.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import linear_recurrence_scan_reverse_amd as rl
from tests import policy_oracle as po

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def logits(seed, R, N, dtype="f32", spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(R, N, generator=gen) * spread).to(DTYPES[dtype]), torch.rand(R, generator=gen)


def column(x, R):
    return x.tolist() if isinstance(x, torch.Tensor) else [float(np.float32(x))] * R


def check_sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mask=None, sure=False):
    """Compares with the oracle; with `sure` no draw may be too near a border to tell."""
    dev = lambda v: v.cuda() if isinstance(v, torch.Tensor) else v
    a, lp = rl.sample_actions(x.cuda(), u.cuda(), temperature=dev(temperature), top_k=dev(top_k), top_p=dev(top_p),
                              min_p=dev(min_p), mask=dev(mask))
    a, lp = a.cpu(), lp.cpu()
    R = x.shape[0]
    t, k, p, m = column(temperature, R), column(top_k, R), column(top_p, R), column(min_p, R)
    used = 0
    for r in range(R):
        want, wlp, gap = po.sample_row(x[r].double().numpy(), float(u[r]), t[r], int(k[r]), p[r], m[r],
                                       None if mask is None else mask[r].numpy())
        if gap < 1e-9 and not sure:
            continue
        used += 1
        assert a[r] == want, (r, int(a[r]), want, gap)
        assert abs(float(lp[r]) - wlp) <= 2.0 ** -24 * abs(wlp) + 1e-9, (r, float(lp[r]), wlp)
    assert used >= R // 2
    return a, lp


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 9, 18, 63, 64, 65, 255, 257, 1023, 1024, 1025, 4095, 4096, 4097, 10007])
def test_sample_sizes(dtype, N):
    x, u = logits(N, 9, N, dtype)
    check_sample(x, u)
    check_sample(x, u, 0.7, top_k=min(5, N))
    check_sample(x, u, 0.7, top_p=0.8)
    check_sample(x, u, 1.3, min_p=0.05)
    check_sample(x, u, 0.9, top_k=40, top_p=0.9, min_p=0.01)
    check_sample(x, u, 0.9, top_k=N - 1, top_p=0.999)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [32768, 131072, 2 ** 20])
def test_sample_large_rows(dtype, N):
    x, u = logits(N, 4, N, dtype)
    check_sample(x, u, 0.8)
    check_sample(x, u, 0.8, top_p=0.9)
    check_sample(x, u, 0.8, top_k=400, top_p=0.95)
    check_sample(x, u, 0.8, top_k=N // 2, top_p=0.9, min_p=1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [50, 3000, 20000])
def test_sample_settings_of_each_row(dtype, N):
    R = 24
    x, u = logits(N + 1, R, N, dtype)
    gen = torch.Generator().manual_seed(N)
    temperature = 0.3 + 2 * torch.rand(R, generator=gen)
    top_k = torch.randint(-2, N + 10, (R,), generator=gen, dtype=torch.int32)
    top_p = 0.3 + 0.8 * torch.rand(R, generator=gen)
    min_p = 0.1 * torch.rand(R, generator=gen) - 0.02
    temperature[:2] = torch.tensor([0.0, -1.0])  # the largest logit
    check_sample(x, u, temperature, top_k, top_p, min_p)
    check_sample(x, u, 1.0, top_k, 0.9, min_p)


@pytest.mark.parametrize("N", [40, 3000, 30000])
def test_sample_temperatures(N):
    x, u = logits(5, 6, N)
    for t in (0.0, 1e-6, 1e-3, 0.05, 20.0, 1e4):
        check_sample(x, u, t)
        check_sample(x, u, t, top_k=N // 3)  # far below what the coarse bins of a low temperature resolve
        check_sample(x, u, t, top_p=0.7)


@pytest.mark.parametrize("N", [4, 64, 1024, 4096, 16384])
def test_sample_equal_logits(N):
    """All logits equal: every sum is exact on both sides, borders included; equal logits go by index."""
    R = 33
    x = torch.full((R, N), 1.5)
    u = torch.arange(R, dtype=torch.float32) / R
    u[-1] = 1 - 2.0 ** -24
    check_sample(x, u, sure=True)
    check_sample(x, u, top_k=3, sure=True)
    check_sample(x, u, top_p=0.5, sure=True)
    check_sample(x, u, top_k=N // 2, top_p=0.5, sure=True)
    check_sample(x, u, min_p=1.0, sure=True)
    u = torch.arange(R, dtype=torch.float32) / 32
    u[-1] = 0.5
    check_sample(x, u, sure=True)  # u on the borders themselves


@pytest.mark.parametrize("N", [300, 3000, 12000])
def test_sample_few_values(N):
    """Many equal logits around the threshold: which of them stay goes by their index."""
    gen = torch.Generator().manual_seed(N)
    x = torch.randint(-3, 3, (12, N), generator=gen).float() * math.log(2.0)
    u = torch.rand(12, generator=gen)
    for k in (1, 2, N // 7, N // 3, N - 1):
        check_sample(x, u, top_k=k)
        check_sample(x, u, top_k=k, top_p=0.77)
    for p in (0.1, 0.501, 0.9):
        check_sample(x, u, top_p=p)


@pytest.mark.parametrize("N", [18, 2000, 9000])
def test_sample_masks(N):
    """Masked logits may hold anything; the type's lowest value is legal; rows without a legal action get -1."""
    x, u = logits(7, 12, N)
    gen = torch.Generator().manual_seed(2)
    mask = (torch.rand(12, N, generator=gen) < 0.6).to(torch.uint8) * 255
    mask[:, 3] = 1
    mask[0] = 0
    mask[1] = 0
    mask[1, N - 1] = 1
    x[mask == 0] = float("nan")
    x[2][mask[2] == 0] = float("inf")
    x[3, 3] = torch.finfo(torch.float32).min
    x[4] = -float("inf")
    x[5] = -float("inf")
    x[5, 3] = -2.0
    x[6] = torch.finfo(torch.float32).min
    x[7][mask[7] != 0] = torch.finfo(torch.float32).max
    x[8, 3] = float("nan")  # not legal either
    x[9, 3] = float("inf")  # counts as the largest float
    for kw in ({}, {"top_k": 4}, {"top_p": 0.9}, {"top_k": 4, "top_p": 0.9, "min_p": 0.1}):
        a, lp = check_sample(x, u, mask=mask, **kw)
        assert a[0] == -1 and lp[0] == 0 and a[4] == -1 and lp[4] == 0
        assert a[1] == N - 1 and lp[1] == 0 and a[5] == 3
        assert torch.all(mask[torch.arange(12)[a >= 0], a[a >= 0]] != 0)
    check_sample(x, u, mask=mask != 0)


def test_sample_edges_of_u():
    x, _ = logits(8, 4, 5000)
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan")):
        a, lp = rl.sample_actions(x.cuda(), torch.full((4,), u, device="cuda"), top_k=10)
        top = x.topk(10, dim=1).indices
        assert all(int(a[r]) in top[r].tolist() for r in range(4)), u
        if u == 0.0:
            assert torch.equal(a.cpu(), top.min(1).values)
        if u == 1 - 2.0 ** -24:
            assert torch.equal(a.cpu(), top.max(1).values)


def test_sample_strides_shapes_streams_and_graphs():
    x, u = logits(9, 12, 5000, "bf16")
    base = rl.sample_actions(x.cuda(), u.cuda(), top_p=0.9)
    for lead in (0, 1, 3, 8):
        wide = torch.zeros(12, 5000 + lead + 3, dtype=torch.bfloat16, device="cuda")
        wide[:, lead:lead + 5000] = x.cuda()
        got = rl.sample_actions(wide[:, lead:lead + 5000], u.cuda(), top_p=0.9)
        assert all(torch.equal(a, b) for a, b in zip(got, base))
    got = rl.sample_actions(x.cuda().view(3, 4, 5000), u.cuda().view(3, 4), top_p=0.9)
    assert got[0].shape == (3, 4) and torch.equal(got[0].flatten(), base[0])
    one = rl.sample_actions(x[0].cuda(), u[0].cuda(), top_p=0.9)
    assert one[0].shape == () and one[0] == base[0][0]
    none = rl.sample_actions(x[:0].cuda(), u[:0].cuda())
    assert none[0].shape == (0,)
    side = torch.cuda.Stream()
    xs, us = x.cuda(), u.cuda()
    side.wait_stream(torch.cuda.current_stream())
    got = rl.sample_actions(xs, us, top_p=0.9, stream=side)
    side.synchronize()
    assert torch.equal(got[0], base[0])
    big, bu = logits(10, 1, 131072)
    big, bu = big.cuda(), bu.cuda()
    work = lambda: rl.sample_actions(xs, us, top_k=50, top_p=0.9) + rl.sample_actions(big, bu, top_p=0.9)
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        us.copy_(torch.rand(12, generator=gen, device="cuda"))
        bu.copy_(torch.rand(1, generator=gen, device="cuda"))
        big.copy_(torch.randn(1, 131072, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, work()))


def test_sample_frequencies():
    """40000 draws of one row follow its probabilities (5 standard deviations)."""
    x = torch.tensor([1.0, 0.0, 2.0, -1.0, 0.5]).repeat(40000, 1)
    u = torch.rand(40000, generator=torch.Generator().manual_seed(0))
    a, _ = rl.sample_actions(x.cuda(), u.cuda(), temperature=0.8, top_k=4)
    p = torch.softmax(torch.tensor([1.0, 0.0, 2.0, -math.inf, 0.5]) / 0.8, 0)
    share = torch.bincount(a.cpu(), minlength=5) / 40000
    assert torch.all((share - p).abs() <= 5 * (p * (1 - p) / 40000).sqrt() + 1e-12)


def test_sample_refusals():
    x, u = logits(1, 4, 10)
    x, u = x.cuda(), u.cuda()
    with pytest.raises(TypeError):
        rl.sample_actions(x, u.double())
    with pytest.raises(ValueError):
        rl.sample_actions(x, u[:3])
    with pytest.raises(TypeError):
        rl.sample_actions(x, u, top_k=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        rl.sample_actions(x, u, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        rl.sample_actions(x.t(), u)
    with pytest.raises(ValueError):
        rl.sample_actions(x, u, mask=torch.ones(4, 9, device="cuda", dtype=torch.uint8))
    for kw in ({"temperature": -1.0}, {"top_p": 0.0}, {"min_p": 1.5}, {"top_k": -3}):
        with pytest.raises(rl.RlscanError):
            rl.sample_actions(x, u, **kw)


# ------------------------------------------------------------------ log-probabilities
def check_log_probs(x, a, temperature=1.0, mask=None):
    """Forward and backward against the oracle."""
    R, N = x.shape
    gen = torch.Generator().manual_seed(R)
    dlp, den = torch.randn(R, generator=gen), torch.randn(R, generator=gen)
    dev = lambda v: None if v is None else v.cuda()
    T = float(np.float32(temperature))
    lp, ent, lse = rl.action_log_probs(x.cuda(), a.cuda(), temperature=temperature, mask=dev(mask))
    wlp, went, wlse = po.log_probs(x, a, T, mask)
    z = x.double() / T
    if mask is not None:
        z = torch.where(mask != 0, z, torch.full_like(z, -math.inf))
    top = z.max(1).values
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    size = 1 + torch.where(torch.isfinite(wlp), wlp, torch.zeros_like(wlp)).abs() + top.abs()

    def near(got, want, size):
        # a value past float32's range is infinite in it
        want = want if got.dtype == torch.float64 else torch.where(want.abs() > torch.finfo(torch.float32).max,
                                                                   want.sign() * math.inf, want)
        got = got.double().cpu()
        fin = torch.isfinite(want)
        assert torch.equal(got[~fin], want[~fin])
        bad = (got - want).abs()[fin] - (2.0 ** -24 * want.abs() + 2.0 ** -20 * size)[fin]
        assert bad.numel() == 0 or bad.max() <= 0, float(bad.max())

    near(lp, wlp, size)
    # p |log p| summed: exp2's error times |z| up to the entropy's own size, squared at worst
    near(ent, went, (1 + went.abs()) ** 2)
    near(lse, wlse, size + wlse.abs().nan_to_num(0, 0, 0))
    for g1, g2 in ((dlp, den), (dlp, None), (None, den)):
        d = rl.action_log_probs_backward(dev(g1), dev(g2), x.cuda(), a.cuda(), lse, ent, temperature=temperature,
                                         mask=dev(mask))
        want, terms = po.log_probs_backward(g1, g2, x, a, T, mask)
        err = (d.double().cpu() - want).abs()
        tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 2.0 ** -20 * terms * (2 + top.abs() + went.abs()).unsqueeze(1)
        tol = tol + {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}[x.dtype]
        assert torch.all(err <= tol), float((err / tol).max())
    return lp.cpu(), ent.cpu()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [1, 2, 3, 7, 8, 9, 18, 63, 64, 65, 511, 512, 513, 2047, 2048, 2049, 10007])
def test_log_probs_sizes(dtype, N):
    x, _ = logits(N, 11, N, dtype)
    gen = torch.Generator().manual_seed(N)
    a = torch.randint(0, N, (11,), generator=gen)
    check_log_probs(x, a)
    check_log_probs(x, a, 0.3)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,N", [(1, 131072), (3, 50021), (2, 16384), (40, 16385), (1, 2 ** 21 + 3)])
def test_log_probs_long_rows_are_split(dtype, R, N):
    assert rl.lib().rlscan_action_log_probs_workspace(R, N) > 0
    x, _ = logits(N, R, N, dtype)
    a = torch.randint(0, N, (R,), generator=torch.Generator().manual_seed(R))
    check_log_probs(x, a, 0.8)


@pytest.mark.parametrize("N", [18, 3000, 40000])
def test_log_probs_masks(N):
    x, _ = logits(3, 10, N)
    gen = torch.Generator().manual_seed(2)
    mask = (torch.rand(10, N, generator=gen) < 0.6).to(torch.uint8) * 3
    mask[:, 3] = 1
    mask[:, 4] = 0
    mask[0] = 0
    mask[1] = 0
    mask[1, 3] = 1
    a = torch.full((10,), 3)
    a[2] = 4   # not legal: -inf
    a[3] = -1  # padded step
    a[4] = N
    a[5] = -2 ** 40
    x[mask == 0] = float("nan")
    x[6][mask[6] == 0] = -float("inf")
    x[7, 5:9] = -float("inf")
    x[8, 3] = torch.finfo(torch.float32).min
    lp, ent = check_log_probs(x, a, 0.9, mask)
    assert lp[0] == 0 and ent[0] == 0 and lp[1] == 0 and ent[1] == 0
    assert lp[2] == -math.inf and torch.all(lp[3:6] == 0)


def test_log_probs_extreme_values():
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[big, -big, 0.0], [-big, -big, -big], [1e30, 1e30, 1e30], [0.0, -1e4, -1e4],
                      [-math.inf, -math.inf, 2.0], [88.0, -88.0, 100.0]])
    a = torch.tensor([0, 1, 2, 0, 2, 2])
    lp, ent, lse = rl.action_log_probs(x.cuda(), a.cuda())
    assert torch.allclose(lp.cpu(), torch.tensor([0.0, -math.log(3), -math.log(3), 0.0, 0.0, -6.1442e-06]), atol=1e-6)
    assert torch.allclose(ent.cpu()[:5], torch.tensor([0.0, math.log(3), math.log(3), 0.0, 0.0]), atol=1e-6)
    d = rl.action_log_probs_backward(torch.ones(6, device="cuda"), torch.ones(6, device="cuda"), x.cuda(), a.cuda(),
                                     lse, ent)
    assert torch.isfinite(d).all() and torch.all(d[4, :2] == 0)
    # an illegal row's logits are not used, and a NaN in a legal place shows
    x[0, 1] = float("nan")
    lp, ent, lse = rl.action_log_probs(x.cuda(), a.cuda())
    assert math.isnan(lp[0]) and math.isnan(ent[0]) and math.isnan(lse[0]) and torch.isfinite(lp[1:]).all()
    d = rl.action_log_probs_backward(torch.ones(6, device="cuda"), None, x.cuda(), a.cuda(), lse, ent)
    assert torch.isnan(d[0]).all() and torch.isfinite(d[1:]).all()


def test_log_probs_strides_shapes_streams_and_graphs():
    x, _ = logits(4, 12, 5000, "f16")
    a = torch.randint(0, 5000, (12,), generator=torch.Generator().manual_seed(0)).cuda()
    x = x.cuda()
    g1, g2 = torch.randn(12, device="cuda"), torch.randn(12, device="cuda")

    def both(x, a, g1, g2, **kw):
        f = rl.action_log_probs(x, a, **{n: v for n, v in kw.items() if n != "d_logits"})
        return f + (rl.action_log_probs_backward(g1, g2, x, a, f[2], f[1], **kw),)

    base = both(x, a, g1, g2)
    for lead in (0, 1, 3, 8):
        wide = torch.zeros(12, 5000 + lead + 3, dtype=torch.float16, device="cuda")
        wide[:, lead:lead + 5000] = x
        dw = torch.full_like(wide, 7.0)
        got = both(wide[:, lead:lead + 5000], a, g1, g2, d_logits=dw[:, lead:lead + 5000])
        for p, q in zip(got, base):  # the order of the sums goes by alignment: a few roundings
            assert torch.allclose(p.float(), q.float(), rtol=2e-3, atol=1e-5)
        assert torch.all(dw[:, :lead] == 7) and torch.all(dw[:, lead + 5000:] == 7)
        got = both(wide[:, lead:lead + 5000], a, g1, g2)  # another alignment of the gradient
        assert torch.allclose(got[3].float(), base[3].float(), rtol=2e-3, atol=1e-5)
    got = both(x.view(3, 4, 5000), a.view(3, 4), g1.view(3, 4), g2.view(3, 4))
    assert got[3].shape == (3, 4, 5000) and all(torch.equal(p.flatten(), q.flatten()) for p, q in zip(got, base))
    none = both(x[:0], a[:0], g1[:0], g2[:0])
    assert none[3].shape == (0, 5000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(x, a, g1, g2, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, base))
    big = torch.randn(2, 65536, device="cuda")
    work = lambda: both(x, a, g1, g2) + both(big, a[:2], g1[:2], g2[:2])
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x.copy_(torch.randn(12, 5000, generator=gen, device="cuda"))
        big.copy_(torch.randn(2, 65536, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(p, q) for p, q in zip(got, work()))


def test_rows_past_32_bits():
    """Logits whose last row begins past 2^32 bytes."""
    R, N, stride = 3, 1000, 2 ** 30 + 40
    x, u = logits(5, R, N)
    far = torch.zeros((R - 1) * stride + N, device="cuda")
    view = far.as_strided((R, N), (stride, 1))
    view.copy_(x)
    a = torch.tensor([3, 500, 999]).cuda()
    assert torch.equal(rl.sample_actions(view, u.cuda(), top_k=7)[0], rl.sample_actions(x.cuda(), u.cuda(), top_k=7)[0])
    f, base = rl.action_log_probs(view, a), rl.action_log_probs(x.cuda(), a)
    assert all(torch.equal(p, q) for p, q in zip(f, base))
    g = torch.ones(R, device="cuda")
    want = rl.action_log_probs_backward(g, g, x.cuda(), a, base[2], base[1])
    got = rl.action_log_probs_backward(g, g, view, a, f[2], f[1], d_logits=torch.zeros_like(far).as_strided((R, N), (stride, 1)))
    assert torch.equal(got, want)


def test_log_prob_refusals():
    x, _ = logits(1, 4, 10)
    x = x.cuda()
    a = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        rl.action_log_probs(x, a.int())
    with pytest.raises(ValueError):
        rl.action_log_probs(x, a[:3])
    with pytest.raises(rl.RlscanError):
        rl.action_log_probs(x, a, temperature=0.0)
    lp, ent, lse = rl.action_log_probs(x, a)
    with pytest.raises(rl.RlscanError):
        rl.action_log_probs_backward(lp, None, x, a, lse, ent, d_logits=x)
    with pytest.raises(TypeError):
        rl.action_log_probs_backward(lp, None, x, a, None, ent)
