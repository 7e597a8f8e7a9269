"""Sampling from rows with several +inf logits, as float16 logits that overflowed: they tie at
the top of the row, and which of them stay goes by their index.  The float64 oracle takes +inf
for the largest float32; weights of ties are equal whole numbers, so every sum is exact
on both sides and no draw is too near a border to tell.
"""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_logits import check_sample, logits

pytestmark = pytest.mark.gpu

# one wave, four waves, a block, and blocks that share a row
SIZES = [40, 600, 1024, 3000, 4096, 10007, 40003]


def _rows(dtype, N, infinite):
    """Six rows with +inf at `infinite` places each; the other logits are ordinary."""
    x, _ = logits(N, 6, N, dtype)
    gen = torch.Generator().manual_seed(N + infinite)
    for r in range(6):
        x[r, torch.randperm(N, generator=gen)[:infinite]] = float("inf")
    return x, torch.arange(6, dtype=torch.float32) / 6 + 0.01


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,infinite", [(N, n) for N in SIZES for n in (1, 2, 5, 600) if n < N])
def test_infinite_logits_tie(dtype, N, infinite):
    x, u = _rows(dtype, N, infinite)
    first = torch.isinf(x).int().argmax(1)
    a, lp = check_sample(x, u, 0.0, sure=True)
    assert torch.equal(a, first) and torch.all(lp == 0)
    a, lp = check_sample(x, u, top_k=1, sure=True)
    assert torch.equal(a, first) and torch.all(lp == 0)
    for kw in ({"top_k": 3}, {"top_k": max(1, infinite - 1)}, {"top_k": infinite + 7}, {"top_p": 0.5},
               {"top_p": 0.999, "min_p": 1.0}, {"top_k": max(1, infinite - 1), "top_p": 0.4}, {}):
        a, _ = check_sample(x, u, sure=True, **kw)
        assert torch.isinf(x[torch.arange(6), a]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_masked_infinite_logits_are_not_taken(dtype):
    x, u = _rows(dtype, 3000, 4)
    mask = torch.ones(6, 3000, dtype=torch.uint8)
    first = torch.isinf(x).int().argmax(1)
    mask[torch.arange(6), first] = 0
    for kw in ({"temperature": 0.0}, {"top_k": 2}, {"top_p": 0.6}):
        a, _ = check_sample(x, u, mask=mask, sure=True, **kw)
        assert torch.all(a > first) and torch.isinf(x[torch.arange(6), a]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,infinite", [(700, 1), (700, 3), (3000, 600), (40003, 600)])
def test_infinite_logits_stand_above_the_largest_finite_one(dtype, N, infinite):
    x, u = _rows(dtype, N, infinite)
    x[:, 1::2] = torch.where(torch.isinf(x[:, 1::2]), x[:, 1::2], torch.finfo(x.dtype).max)
    for kw in ({}, {"temperature": 0.0}, {"top_k": infinite}, {"top_k": infinite + 2}, {"top_p": 0.7}):
        a, _ = check_sample(x, u, sure=True, **kw)
        assert torch.isinf(x[torch.arange(6), a]).all()
    # with nothing above it the largest finite value is an ordinary tie
    x = torch.where(torch.isinf(x), 0.0, x)
    for kw in ({"temperature": 0.0}, {"top_k": 2}, {"top_p": 0.3}):
        check_sample(x, u, sure=True, **kw)
