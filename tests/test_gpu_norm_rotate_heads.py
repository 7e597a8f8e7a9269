"""Normalised and rotated heads and their gradients against the float64 oracle."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def draw(E, T, H, Hk, D, dtype, seed=0, far=1000):
    g = torch.Generator().manual_seed(100 * seed + D)
    n = lambda *s: torch.randn(*s, generator=g)
    return {"q": (3 * n(E, T, H, D)).to(dtype), "k": n(E, T, Hk, D).to(dtype), "qw": 1 + 0.2 * n(D), "kw": n(D),
            "pos": torch.randint(-far, far + 1, (E, T), generator=g, dtype=torch.int32),
            "dq": n(E, T, H, D).to(dtype), "dk": n(E, T, Hk, D).to(dtype)}


def on_gpu(d):
    return {k: v.cuda() for k, v in d.items()}


def check(d, got, rotate, grads=None, **how):
    dt = d["q"].dtype
    for i, (x, w, dy) in enumerate((("q", "qw", "dq"), ("k", "kw", "dk"))):
        want = so.Heads(d[x], d[w], d["pos"], rotate, dy=None if grads is None else d[dy], **how)
        so.close(got[i], want.y, so.stored(want.y, want.y_b, dt), x)
        if grads is not None:
            so.close(grads[i], want.dx, so.stored(want.dx, want.dx_b, dt), "d" + x)
            so.close(grads[2 + i], want.dw, want.dw_b + so.U * want.dw.abs(), "d_%s_weight" % x)


def both(c, rotate, **how):
    args = (c["q"], c["k"], c["qw"], c["kw"], c["pos"])
    return (rl.norm_rotate_heads(*args, rotate=rotate, **how),
            rl.norm_rotate_heads_backward(c["dq"], c["dk"], *args, rotate=rotate, **how))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotate", [
    (1, 0), (2, 2), (3, 2), (7, 4), (16, 16), (16, 8), (24, 24), (33, 32), (40, 40), (64, 64), (64, 32), (72, 36),
    (80, 40), (96, 96), (100, 50), (128, 128), (128, 64), (160, 160), (192, 96), (250, 250), (255, 254), (256, 256),
    (256, 0)])
def test_heads(D, rotate, interleaved, dtype):
    d = draw(2, 9, 3, 2, D, dtype)
    got, grads = both(on_gpu(d), rotate, interleaved=interleaved)
    check(d, got, rotate, grads, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,T,H,Hk", [(1, 1, 1, 1), (1, 1, 16, 4), (1, 1, 1, 7), (3, 1, 5, 2), (1, 70, 4, 1),
                                      (40, 37, 4, 4), (9, 1000, 1, 1), (5, 2000, 3, 1)])
def test_numbers_of_tokens_and_heads(E, T, H, Hk, dtype):
    d = draw(E, T, H, Hk, 64, dtype, seed=1)
    got, grads = both(on_gpu(d), 64)
    check(d, got, 64, grads)


@pytest.mark.parametrize("base,eps", [(10000.0, 1e-6), (500000.0, 0.0), (1.0, 0.5), (0.25, 1e-5)])
def test_far_positions(base, eps):
    # an angle is a position times a frequency (at most 4 here), each with a relative error of a few
    # 2^-53: 2^21 * 4 * 2^-50 is far below U
    d = draw(2, 30, 2, 1, 64, torch.float32, seed=2, far=2 ** 21)
    d["pos"][0, :3] = torch.tensor([2 ** 21, -2 ** 21, 0], dtype=torch.int32)
    got, grads = both(on_gpu(d), 64, base=base, eps=eps)
    check(d, got, 64, grads, base=base, eps=eps)
    d = draw(1, 5, 1, 1, 128, torch.float32, seed=3)
    d["pos"][0] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1, 1], dtype=torch.int32)
    got = rl.norm_rotate_heads(*[on_gpu(d)[n] for n in ("q", "k", "qw", "kw", "pos")])
    for i, (x, w) in enumerate((("q", "qw"), ("k", "kw"))):
        want = so.Heads(d[x], d[w], d["pos"], 128)
        # 2^31 times a frequency with a relative error of a few 2^-53 (its power's and the product's):
        # 2^31 * 4 * 2^-53 = 2^-20, 16 of U of the pair's size
        so.close(got[i], want.y, 1.5 * want.y_b, x)


def test_normalising_alone_and_without_weights():
    d = draw(2, 9, 3, 2, 48, torch.bfloat16, seed=4)
    c = on_gpu(d)
    for pos, rotate in ((None, 0), (c["pos"], 48)):
        got = rl.norm_rotate_heads(c["q"], c["k"], None, c["kw"], pos)
        grads = rl.norm_rotate_heads_backward(c["dq"], c["dk"], c["q"], c["k"], None, c["kw"], pos)
        assert grads[2] is None
        for i, (x, w, dy) in enumerate((("q", None, "dq"), ("k", d["kw"], "dk"))):
            want = so.Heads(d[x], w, d["pos"], rotate, dy=d[dy])
            so.close(got[i], want.y, so.stored(want.y, want.y_b, torch.bfloat16), x)
            so.close(grads[i], want.dx, so.stored(want.dx, want.dx_b, torch.bfloat16), dy)
            if w is not None:
                so.close(grads[2 + i], want.dw, want.dw_b + so.U * want.dw.abs(), "dw")
    # a buffer for the gradient of a weight that is not given
    dw = torch.empty(48, device="cuda")
    grads = rl.norm_rotate_heads_backward(c["dq"], c["dk"], c["q"], c["k"], d_q_weight=dw)
    want = so.Heads(d["q"], None, None, 0, dy=d["dq"])
    so.close(dw, want.dw, want.dw_b + so.U * want.dw.abs(), "dw")
    assert grads[2] is dw and grads[3] is None


@pytest.mark.parametrize("dtype", DTYPES)
def test_time_major_steps_and_strides(dtype):
    E, T, H, Hk, D = 3, 10, 4, 2, 32
    d = draw(E, T, H, Hk, D, dtype, seed=5)
    c = on_gpu(d)
    tm = {k: v.transpose(0, 1).contiguous() if v.dim() > 1 else v for k, v in c.items()}
    got, grads = both(tm, 16, time_major=True)
    check(d, [g.transpose(0, 1) for g in got], 16, [g.transpose(0, 1) for g in grads[:2]] + list(grads[2:]))
    # slices of one projection, odd distances: every load by elements
    for pad in (0, 1, 4):
        fused = torch.cat([c["q"], c["k"], torch.zeros(E, T, 1, D, dtype=dtype, device="cuda")], 2)
        fused = torch.nn.functional.pad(fused.flatten(2), (pad, pad))
        heads = lambda h0, n: fused[..., pad + h0 * D:pad + (h0 + n) * D].unflatten(-1, (n, D))
        out = torch.full_like(fused, 5.0)
        to = lambda h0, n: out[..., pad + h0 * D:pad + (h0 + n) * D].unflatten(-1, (n, D))
        got = rl.norm_rotate_heads(heads(0, H), heads(H, Hk), c["qw"], c["kw"], c["pos"], q_out=to(0, H),
                                   k_out=to(H, Hk))
        check(d, got, D)
        assert (out[..., pad + (H + Hk) * D:] == 5).all() and (out[..., :pad] == 5).all()
        grads = rl.norm_rotate_heads_backward(c["dq"], c["dk"], heads(0, H), heads(H, Hk), c["qw"], c["kw"], c["pos"],
                                              dq=to(0, H), dk=to(H, Hk))
        check(d, got=[g.clone() for g in rl.norm_rotate_heads(heads(0, H), heads(H, Hk), c["qw"], c["kw"], c["pos"])],
              rotate=D, grads=grads)
    # one step of every row, and keys that all heads of a row share
    for t in (0, T - 1):
        got = rl.norm_rotate_heads(c["q"][:, t], c["k"][:, t], c["qw"], c["kw"], c["pos"][:, t].contiguous())
        one = {k: v[:, t:t + 1] if v.dim() > 1 else v for k, v in d.items()}
        check(one, [g.unsqueeze(1) for g in got], D)
    wide = c["k"][:, :, :1].expand(E, T, 3, D)
    got = rl.norm_rotate_heads(c["q"], wide, c["qw"], c["kw"], c["pos"])
    check(dict(d, k=d["k"][:, :, :1].expand(E, T, 3, D)), got, D)


def test_empty():
    for E, T, H, Hk in ((0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0)):
        c = on_gpu(draw(E, T, H, Hk, 16, torch.float32))
        got, grads = both(c, 16)
        assert got[0].shape == (E, T, H, 16) and got[1].shape == (E, T, Hk, 16)
        assert not grads[2].any() and not grads[3].any()
    d = draw(2, 3, 0, 2, 16, torch.float32)
    got, grads = both(on_gpu(d), 16)
    want = so.Heads(d["k"], d["kw"], d["pos"], 16, dy=d["dk"])
    so.close(got[1], want.y, so.stored(want.y, want.y_b, torch.float32), "k")
    assert not grads[2].any()
    so.close(grads[3], want.dw, want.dw_b + so.U * want.dw.abs(), "dw")


def test_zeros_and_not_finite():
    d = draw(1, 6, 2, 2, 64, torch.float32, seed=6)
    d["q"][0, 1, 0] = 0.0
    clean = on_gpu(d)
    ref, _ = both(clean, 64)
    check(d, ref, 64)
    d["q"][0, 2, 1, 5] = math.inf
    d["k"][0, 3, 0, 6] = math.nan
    got, _ = both(on_gpu(d), 64)
    same = torch.ones(1, 6, 2, dtype=torch.bool, device="cuda")
    q_same, k_same = same.clone(), same.clone()
    q_same[0, 2, 1] = False
    k_same[0, 3, 0] = False
    assert torch.equal(got[0][q_same], ref[0][q_same]) and torch.equal(got[1][k_same], ref[1][k_same])
    assert torch.isnan(got[0][0, 2, 1]).any() and torch.isnan(got[1][0, 3, 0]).all()


def test_gradients_against_differences():
    d = draw(1, 3, 2, 1, 10, torch.float32, seed=7, far=50)
    _, grads = both(on_gpu(d), 6)
    dd = {k: v.double() if v.dtype == torch.float32 else v for k, v in d.items()}

    def loss():
        return sum((so.Heads(dd[x], dd[w], dd["pos"], 6).y * dd[dy]).sum()
                   for x, w, dy in (("q", "qw", "dq"), ("k", "kw", "dk")))

    eps = 1e-6
    for name, g in zip(("q", "k", "qw", "kw"), grads):
        flat = dd[name].view(-1)
        for i in range(0, flat.numel(), 3):
            old = flat[i].item()
            flat[i] = old + eps
            up = loss()
            flat[i] = old - eps
            down = loss()
            flat[i] = old
            want = ((up - down) / (2 * eps)).item()
            # float64 differences: 2^-53 of losses near 30 over 1e-6; float32: a hundred U of sums near 10
            assert abs(g.reshape(-1)[i].item() - want) < 1e-4 * max(1.0, abs(want)), (name, i)


def test_same_every_time_streams_and_graphs():
    c = on_gpu(draw(4, 300, 6, 2, 128, torch.bfloat16, seed=8))
    first = both(c, 128)
    first = first[0] + first[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(c, 128, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, other[0] + other[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both(c, 128)
    for seed in (9, 10, 11):
        for k, v in on_gpu(draw(4, 300, 6, 2, 128, torch.bfloat16, seed=seed)).items():
            c[k].copy_(v)
        want = both(c, 128)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(captured[0] + captured[1], want[0] + want[1]))


def test_far_offsets():
    far = 2 ** 31 + 64
    d = draw(2, 5, 2, 1, 64, torch.bfloat16, seed=12)
    c = on_gpu(d)
    make = lambda: torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 5, 2, 64), (far, 128, 64, 1))
    q, q_out = make(), make()
    q.copy_(c["q"])
    got = rl.norm_rotate_heads(q, c["k"], c["qw"], c["kw"], c["pos"], q_out=q_out)
    check(d, got, 64)
