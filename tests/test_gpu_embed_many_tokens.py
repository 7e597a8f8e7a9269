"""The table's gradient of more tokens than the sort's waves take at once: past 65536 a wave places its tokens in
several rounds of 64, and the second digit's counts are of blocks of more than 1024."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402
from tests.test_gpu_embed_tokens import draw  # noqa: E402

pytestmark = pytest.mark.gpu


def total(d_out, tokens, N):
    """Sums, sums of absolute values and numbers of terms of every row, in float64."""
    ok = (tokens >= 0) & (tokens < N)
    t, d = tokens[ok], d_out[ok].double()
    zero = torch.zeros(N, d_out.shape[1], dtype=torch.float64)
    return zero.index_add(0, t, d), zero.index_add(0, t, d.abs()), torch.bincount(t, minlength=N).double()


# one digit and two; the least number past one round, and many rounds
@pytest.mark.parametrize("how", ["zipf", "even", "one", "rising", "falling", "padding"])
@pytest.mark.parametrize("R,N,D", [(65537, 64, 4), (70001, 1024, 2), (70001, 3000, 4), (200000, 64007, 2),
                                   (1100003, 5000, 1), (1 << 20, 1 << 20, 2)])
def test_many_tokens(R, N, D, how):
    # whole numbers below 2^24 in all: their sums are exact, and a token out of place is one row more or less
    d = draw(R, N, D, torch.float32, seed=60, how=how)
    values = torch.randint(-8, 9, (R, D), generator=torch.Generator().manual_seed(R)).float()
    got = rl.embed_tokens_backward(values.cuda(), d["tokens"].cuda(), N)
    want, _, _ = total(values, d["tokens"], N)
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_many_tokens_of_any_value(dtype):
    R, N, D, scale = 150001, 2000, 6, 0.7
    d = draw(R, N, D, dtype, seed=61, how="zipf")
    on = d["d"].cuda(), d["tokens"].cuda()
    got = rl.embed_tokens_backward(*on, N, scale=scale)
    want, size, count = total(d["d"], d["tokens"], N)
    bound = (count[:, None] + 2) * so.U * size * scale
    so.close(got, want * scale, so.stored(want * scale, bound, dtype), "table's gradient")
    assert torch.equal(got, rl.embed_tokens_backward(*on, N, scale=scale))
