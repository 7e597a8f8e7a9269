"""The gated recurrence where a state or a gradient is infinite: it stays so, with its sign, until its episode
ends, and nothing else changes by a bit."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402
from tests.test_gpu_gated_recurrence import both, draw, on_gpu  # noqa: E402

pytestmark = pytest.mark.gpu


def kinds(x):
    """0 finite, 1 and -1 infinite, 2 NaN."""
    x = x.detach().cpu().double()
    return torch.where(torch.isnan(x), torch.full_like(x, 2), torch.where(torch.isinf(x), x.sign(), torch.zeros_like(x)))


# one row and many, one wave to a block, four and sixteen, and rows cut into segments
@pytest.mark.parametrize("E,T", [(2, 9), (2, 40), (2, 300), (270, 90), (2, 1500)])
@pytest.mark.parametrize("low,high", [(0.008, 0.84), (1.5, 4.0), (30.0, 90.0)])
def test_infinite_values_stay(E, T, low, high):
    d = draw(E, T, 64, torch.float32, seed=50, p_done=0.0, low=low, high=high)
    done = torch.zeros(E, T, dtype=torch.bool)
    done[:, 2 * T // 3] = True  # every row: an episode that ends inside it
    done[1, T // 2] = True
    d["done"] = done
    clean = {k: v.clone() for k, v in d.items()}
    d["x"][0, T // 3, 3] = math.inf
    d["x"][0, 0, 4] = -math.inf
    d["x"][1, T - 2, 5] = math.inf
    d["init"][1, 9] = -math.inf
    d["d_out"][0, T // 3, 10] = math.inf
    d["d_out"][1, T - 1, 11] = -math.inf
    d["d_final"][0, 12] = math.inf
    d["x"][1, 1, 13], d["x"][1, 2, 13] = math.inf, -math.inf  # their sum is NaN
    got, grads = both(on_gpu(d))
    ref, ref_grads = both(on_gpu(clean))
    # Two rows are all that the oracle is asked for.  A sum over infinite parts of either sign has no value.
    two = {k: v[:2] if torch.is_tensor(v) and k != "rate" else v for k, v in d.items()}
    want = so.Recurrence(two["x"], two["ig"], two["dg"], two["rate"], two["done"], two["init"], two["d_out"],
                         two["d_final"])
    assert torch.equal(kinds(got[0][:2]), kinds(want.out)) and torch.equal(kinds(got[1][:2]), kinds(want.final))
    for i, name in enumerate(("dx", "di", "dr")):
        assert torch.equal(kinds(grads[i][:2]), kinds(getattr(want, name))), name
    assert torch.equal(kinds(grads[4][:2]), kinds(want.d_init))
    assert (kinds(want.out) == 1).sum() > T // 3 and (kinds(want.dx) == 1).any()
    for a, b in zip((got[0], got[1]) + grads[:3] + grads[4:], (ref[0], ref[1]) + ref_grads[:3] + ref_grads[4:]):
        fine = torch.isfinite(a)
        touched = torch.zeros_like(a, dtype=torch.bool)
        touched[:2, ..., [3, 4, 5, 9, 10, 11, 12, 13]] = True
        assert fine[~touched].all() and torch.equal(a[~touched], b[~touched])
    fine = [c for c in range(64) if c not in (3, 4, 5, 9, 10, 11, 12, 13)]
    assert torch.equal(grads[3][fine], ref_grads[3][fine])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinite_values_stay_in_16_bits(dtype):
    d = draw(3, 200, 70, dtype, seed=51, p_done=0.02)
    d["x"][0, 60, 3], d["x"][2, 5, 69] = math.inf, -math.inf
    d["d_out"][1, 150, 8] = -math.inf
    got, grads = both(on_gpu(d))
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], d["done"], d["init"], d["d_out"], d["d_final"])
    assert torch.equal(kinds(got[0]), kinds(want.out)) and torch.equal(kinds(grads[4]), kinds(want.d_init))
    for i, name in enumerate(("dx", "di", "dr")):
        assert torch.equal(kinds(grads[i]), kinds(getattr(want, name))), name


@pytest.mark.parametrize("rate", [0.0, 0.01, 0.5, 3.0, 100.0])
def test_infinite_states_of_single_steps(rate):
    g = torch.Generator().manual_seed(52)
    x, gate = torch.randn(4, 40, generator=g).cuda(), torch.randn(4, 40, generator=g).cuda()
    state = torch.randn(4, 40, generator=g).cuda()
    state[0, 3], state[1, 4], state[2, 5] = math.inf, -math.inf, math.inf
    reset = torch.tensor([0, 0, 1, 0], dtype=torch.uint8).cuda()
    out = rl.gated_recurrence_step(x, gate, gate, torch.full((40,), rate).cuda(), state, reset)
    want = torch.zeros(4, 40)
    want[0, 3], want[1, 4] = 1, -1
    assert torch.equal(kinds(out), want.double()) and torch.equal(out, state)


@pytest.mark.parametrize("T,D", [(1, 5), (2, 64), (7, 33), (64, 7), (300, 40)])
@pytest.mark.parametrize("p_done", [0.2, 0.5, 0.9])
def test_infinite_values_between_many_ends(T, D, p_done):
    # episodes of one step and more: an infinite value may enter any step, and be dropped behind it
    E = 60
    d = draw(E, T, D, torch.float32, seed=53, p_done=p_done)
    g = torch.Generator().manual_seed(100 * T + D)
    for name, rate in (("x", 0.02), ("init", 0.1), ("d_out", 0.02), ("d_final", 0.1)):
        at = torch.rand(d[name].shape, generator=g) < rate
        sign = torch.where(torch.rand(d[name].shape, generator=g) < 0.5, -math.inf, math.inf)
        d[name] = torch.where(at, sign, d[name])
    got, grads = both(on_gpu(d))
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], d["done"], d["init"], d["d_out"], d["d_final"])
    for name, a, b in (("out", got[0], want.out), ("final state", got[1], want.final), ("dx", grads[0], want.dx),
                       ("d_input_gate", grads[1], want.di), ("d_decay_gate", grads[2], want.dr),
                       ("d_init_state", grads[4], want.d_init)):
        assert torch.equal(kinds(a), kinds(b)), name
