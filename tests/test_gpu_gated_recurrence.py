"""The gated recurrence, its gradients and its single step against the float64 oracle."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def draw(E, T, D, dtype, seed=0, p_done=0.1, init=True, low=0.008, high=0.84):
    g = torch.Generator().manual_seed(1000 * seed + 10 * T + D)
    n = lambda *s: torch.randn(*s, generator=g)
    d = {"x": n(E, T, D).to(dtype), "ig": n(E, T, D).to(dtype), "dg": n(E, T, D).to(dtype),
         "rate": torch.exp(math.log(low) + math.log(high / low) * torch.rand(D, generator=g)),
         "done": (torch.rand(E, T, generator=g) < p_done) if p_done else None,
         "init": n(E, D) if init else None, "d_out": n(E, T, D).to(dtype), "d_final": n(E, D) if init else None}
    return d


def on_gpu(d):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}


def check(d, got, grads=None, what=""):
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], d["done"], d["init"],
                         d["d_out"] if grads is not None else None, d["d_final"])
    dt = d["x"].dtype
    out, final, marks = got
    so.close(out, want.out, so.stored(want.out, want.out_b, dt), what + " out")
    so.close(final, want.final, want.final_b, what + " final state")
    so.close(marks, want.states[:, :-1][:, ::16], want.states_b[:, :-1][:, ::16] + so.TINY[torch.float32],
             what + " marks")
    if grads is None:
        return
    for name, g in zip(("dx", "di", "dr"), grads):
        w = getattr(want, name)
        so.close(g, w, so.stored(w, getattr(want, name + "_b"), dt), what + " " + name)
    so.close(grads[3], want.d_rate, want.d_rate_b + so.U * want.d_rate.abs(), what + " d_rate")
    so.close(grads[4], want.d_init, want.d_init_b, what + " d_init")


def both(c, **kw):
    got = rl.gated_recurrence(c["x"], c["ig"], c["dg"], c["rate"], c["done"], c["init"], with_state=True,
                              with_marks=True, **kw)
    return got, rl.gated_recurrence_backward(c["d_out"], c["x"], c["ig"], c["dg"], c["rate"], got[2], c["done"],
                                             c["d_final"], **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,T,D", [
    (1, 1, 1), (2, 2, 3), (3, 15, 64), (1, 16, 65), (2, 17, 7), (2, 31, 128), (3, 64, 33), (1, 65, 64), (2, 127, 20),
    (1, 128, 5), (1, 129, 130), (2, 255, 64), (1, 257, 96), (1, 700, 40), (70, 5, 64), (5, 100, 250), (1, 2500, 66),
    (2, 4097, 10)])
def test_rows(E, T, D, dtype):
    d = draw(E, T, D, dtype)
    check(d, *both(on_gpu(d)))


@pytest.mark.parametrize("E,T,D", [(1100, 70, 64), (1100, 70, 70), (4200, 20, 64), (9000, 3, 66)])
def test_many_rows(E, T, D):
    # every number of waves to a block, and blocks that take several rows for their share of d_rate
    d = draw(E, T, D, torch.bfloat16)
    check(d, *both(on_gpu(d)))


@pytest.mark.parametrize("p_done,init", [(0.0, False), (0.0, True), (1.0, True), (0.5, False)])
@pytest.mark.parametrize("T", [1, 40, 1500])
def test_cuts_and_states(p_done, init, T):
    d = draw(2, T, 70, torch.float32, seed=1, p_done=p_done, init=init)
    got, grads = both(on_gpu(d))
    check(d, got, grads)
    if p_done == 1.0:
        assert not got[1].any() and not grads[2][:, 1:].any()  # no step but the first sees the one before it


@pytest.mark.parametrize("low,high", [(1e-5, 1e-3), (1.0, 200.0)])
def test_long_and_short_memories(low, high):
    d = draw(2, 3000, 64, torch.float32, seed=2, p_done=0.0, low=low, high=high)
    check(d, *both(on_gpu(d)))


def test_long_memory_in_norm():
    # float32 roundings of a memory of about 10^4 steps: 2 for each step, of either sign, so their
    # sum is near sqrt(2 * 10^4) halves of U, 70 U; three times that
    d = draw(1, 30000, 64, torch.float32, seed=3, p_done=0.0, low=1e-4, high=2e-4)
    got, _ = both(on_gpu(d))
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], None, d["init"])
    off = (got[0].cpu().double() - want.out).norm() / want.out.norm()
    assert off.item() < 210 * so.U


@pytest.mark.parametrize("dtype", DTYPES)
def test_time_major_and_strides(dtype):
    E, T, D = 3, 75, 41
    d = draw(E, T, D, dtype, seed=4)
    c = on_gpu(d)
    tm = {k: (v.transpose(0, 1).contiguous() if k in ("x", "ig", "dg", "done", "d_out") else v) for k, v in c.items()}
    got, grads = both(tm, time_major=True)
    check(d, (got[0].transpose(0, 1), got[1], got[2]), [g.transpose(0, 1) for g in grads[:3]] + list(grads[3:]))
    # slices of one projection, into slices of one buffer; an input gate that all rows share
    fused = torch.cat([c["x"], c["ig"], c["dg"]], 2)
    s = dict(c, x=fused[..., :D], ig=fused[..., D:2 * D], dg=fused[..., 2 * D:])
    out = torch.full((E, T, 3 * D + 2), 7.0, dtype=dtype, device="cuda")
    got = rl.gated_recurrence(s["x"], s["ig"], s["dg"], s["rate"], s["done"], s["init"], with_state=True,
                              with_marks=True, out=out[..., 1:D + 1])
    grads = rl.gated_recurrence_backward(s["d_out"], s["x"], s["ig"], s["dg"], s["rate"], got[2], s["done"],
                                         s["d_final"], dx=out[..., D + 1:2 * D + 1], d_input_gate=torch.empty_like(c["x"]),
                                         d_decay_gate=out[..., 2 * D + 1:3 * D + 1])
    check(d, got, grads)
    assert (out[..., 0] == 7).all() and (out[..., -1] == 7).all()
    one = c["ig"][:1].expand(E, T, D)
    d["ig"] = one.cpu()
    check(d, *both(dict(c, ig=one)))


def test_given_buffers():
    d = draw(2, 50, 30, torch.bfloat16, seed=5)
    c = on_gpu(d)
    out, final = torch.empty_like(c["x"]), torch.empty(2, 30, device="cuda")
    marks = torch.empty(2, 4, 30, device="cuda")
    got = rl.gated_recurrence(c["x"], c["ig"], c["dg"], c["rate"], c["done"], c["init"], out=out, final_state=final,
                              marks=marks)
    assert [g.data_ptr() for g in got] == [out.data_ptr(), final.data_ptr(), marks.data_ptr()]
    bufs = [torch.empty_like(c["x"]) for _ in range(3)] + [torch.empty(30, device="cuda"), torch.empty(2, 30, device="cuda")]
    grads = rl.gated_recurrence_backward(c["d_out"], c["x"], c["ig"], c["dg"], c["rate"], marks, c["done"], c["d_final"],
                                         dx=bufs[0], d_input_gate=bufs[1], d_decay_gate=bufs[2], d_rate=bufs[3],
                                         d_init_state=bufs[4])
    assert [g.data_ptr() for g in grads] == [b.data_ptr() for b in bufs]
    check(d, got, grads)
    assert torch.is_tensor(rl.gated_recurrence(c["x"], c["ig"], c["dg"], c["rate"]))


def test_empty():
    for E, T, D in ((0, 5, 8), (3, 0, 8), (2, 5, 0)):
        c = on_gpu(draw(E, T, D, torch.float32))
        got, grads = both(c)
        assert got[0].shape == (E, T, D) and got[2].shape == (E, -(-T // 16), D)
        if T == 0:
            assert torch.equal(got[1], c["init"]) and torch.equal(grads[4], c["d_final"])
        assert not grads[3].any()
    c = on_gpu(draw(3, 0, 8, torch.float32, init=False))
    got, grads = both(c)
    assert not got[1].any() and not grads[4].any()


def test_held_states():
    # a decay gate of -inf holds the state: padding in a row; its step has no gradient
    d = draw(2, 60, 64, torch.float32, seed=6)
    d["dg"][:, 20:41] = -math.inf
    got, grads = both(on_gpu(d))
    check(d, got, grads)
    held = ~d["done"][:, 19:40]  # a step that starts anew holds nothing
    assert not grads[0][:, 20:41][held].any() and not grads[2][:, 20:41].any()
    # and one of +inf lets go at the channel's rate
    d["dg"][:, 20:41] = math.inf
    check(d, *both(on_gpu(d)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_not_finite_stays_in_its_episode(dtype):
    T = 900
    d = draw(2, T, 64, dtype, seed=7, p_done=0.0)
    done = torch.zeros(2, T, dtype=torch.bool)
    done[:, [99, 399, 415, 640]] = True
    d["done"] = done
    clean = {k: v.clone() for k, v in d.items()}
    bad = {k: v.clone() for k, v in d.items()}
    bad["x"][0, 120, 3] = math.inf
    bad["x"][0, 500, 5] = math.nan
    bad["dg"][1, 400, 6] = math.nan  # a step that starts anew does not look at it
    bad["ig"][1, 650, 8] = math.nan
    bad["init"][1, 9] = math.inf
    bad["d_out"][0, 300, 10] = math.inf
    got, grads = both(on_gpu(bad))
    ref, ref_grads = both(on_gpu(clean))
    same = torch.ones(2, T, 64, dtype=torch.bool)
    same[0, 100:400, [3, 10]] = False
    same[0, 416:641, 5] = False
    same[1, 641:, 8] = False
    same[1, :100, 9] = False
    same = same.cuda()
    assert torch.equal(got[0][same], ref[0][same])
    for i in range(3):
        ok = same.clone()
        ok[1, 400, 6] = True
        assert torch.equal(grads[i][ok], ref_grads[i][ok]), i
    assert not torch.isfinite(got[0][0, 120:400, 3]).any() and torch.isfinite(got[0][0, 400:, 3]).all()
    assert not torch.isfinite(got[0][1, :100, 9]).any() and torch.isfinite(got[0][1, 100:, 9]).all()
    assert torch.isfinite(got[0][1, :, 6]).all() and torch.isfinite(grads[2][1, :, 6]).all()
    fine = [c for c in range(64) if c not in (3, 5, 8, 9, 10)]
    assert torch.equal(grads[3][fine], ref_grads[3][fine])


def test_gradients_against_differences():
    # central differences of the float64 oracle's loss, independent of the formulas of its gradients
    d = draw(2, 20, 3, torch.float32, seed=8)
    _, grads = both(on_gpu(d))
    dd = {k: v.double() if torch.is_tensor(v) and v.dtype == torch.float32 else v for k, v in d.items()}

    def loss(c):
        r = so.Recurrence(c["x"], c["ig"], c["dg"], c["rate"], c["done"], c["init"])
        return (r.out * c["d_out"]).sum() + (r.final * c["d_final"]).sum()

    eps = 1e-5
    for name, g in zip(("x", "ig", "dg", "rate", "init"), grads):
        flat = dd[name].view(-1)
        for i in range(0, flat.numel(), 7 if flat.numel() > 20 else 1):
            old = flat[i].item()
            flat[i] = old + eps
            up = loss(dd)
            flat[i] = old - eps
            down = loss(dd)
            flat[i] = old
            want = ((up - down) / (2 * eps)).item()
            # differences: eps^2 of third derivatives up to (1 / rate)^2.5; float32: a few dozen U of sums near 10
            assert abs(g.view(-1)[i].item() - want) < 2e-4 * max(1.0, abs(want)), (name, i)


def test_same_every_time():
    c = on_gpu(draw(5, 1200, 100, torch.bfloat16, seed=9))
    a, ga = both(c)
    for _ in range(3):
        b, gb = both(c)
        assert all(torch.equal(x, y) for x, y in zip(a + ga, b + gb))


def test_streams_and_graphs():
    d = draw(1, 3000, 70, torch.float32, seed=10)
    c = on_gpu(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, grads = both(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(d, got, grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both(c)
    for seed in (11, 12, 13):
        n = draw(1, 3000, 70, torch.float32, seed=seed)
        for k, v in n.items():
            if torch.is_tensor(v):
                c[k].copy_(v)
        want, want_grads = both(c)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured[0] + captured[1], want + want_grads):
            assert torch.equal(x, y)


def test_far_offsets():
    # rows further apart than 2^32 bytes
    far = 2 ** 31 + 64
    big = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda")
    d = draw(2, 33, 64, torch.bfloat16, seed=14)
    c = on_gpu(d)
    x = big.as_strided((2, 33, 64), (far, 64, 1))
    x.copy_(c["x"])
    out = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 33, 64), (far, 64, 1))
    got = rl.gated_recurrence(x, c["ig"], c["dg"], c["rate"], c["done"], c["init"], with_state=True, with_marks=True,
                              out=out)
    check(d, got)


# ------------------------------------------------------------------ single steps
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,D", [(1, 1), (3, 7), (2, 64), (5, 300), (1, 2048)])
def test_steps_are_the_rows(E, D, dtype):
    T = 12
    d = draw(E, T, D, dtype, seed=15, p_done=0.2)
    c = on_gpu(d)
    slots = torch.randperm(E + 3, generator=torch.Generator().manual_seed(1))[:E].to(torch.int32).cuda()
    pool = torch.full((E + 3, D), math.nan, device="cuda")
    pool[slots.long()] = c["init"]
    outs = []
    for t in range(T):
        reset = c["done"][:, t - 1].contiguous() if t else None
        outs.append(rl.gated_recurrence_step(c["x"][:, t], c["ig"][:, t], c["dg"][:, t], c["rate"], pool, reset, slots))
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], d["done"], d["init"])
    so.close(torch.stack(outs, 1), want.out, so.stored(want.out, want.out_b, dtype), "steps")
    so.close(pool[slots.long()], want.states[:, -1], want.states_b[:, -1] + so.TINY[torch.float32], "pool")
    others = torch.ones(E + 3, dtype=torch.bool, device="cuda")
    others[slots.long()] = False
    assert torch.isnan(pool[others]).all()


def test_step_without_a_state():
    c = on_gpu(draw(4, 1, 70, torch.float32, seed=16, p_done=0.0))
    pool = torch.randn(5, 70, device="cuda")
    before = pool.clone()
    slots = torch.tensor([2, -1, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = rl.gated_recurrence_step(c["x"][:, 0], c["ig"][:, 0], c["dg"][:, 0], c["rate"], pool, None, slots)
    assert not out[1:].any() and out[0].any()
    rest = [0, 1, 3, 4]
    assert torch.equal(pool[rest], before[rest]) and not torch.equal(pool[2], before[2])
    # a state that is dropped may hold anything
    pool[2] = math.nan
    out = rl.gated_recurrence_step(c["x"][:, 0], c["ig"][:, 0], c["dg"][:, 0], c["rate"], pool,
                                   torch.ones(4, dtype=torch.uint8, device="cuda"), slots)
    assert torch.isfinite(out).all() and torch.isfinite(pool[2]).all()
