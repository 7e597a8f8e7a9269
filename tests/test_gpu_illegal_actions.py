"""A taken action that is not legal: a mask byte of 0 and a logit of -inf say the same, in the
log-probability (-inf), the entropy and the gradient (0 where not legal, -p_j of the others)."""
import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [2, 18, 3000, 40003])
def test_masked_and_infinite_logits_agree(dtype, N):
    gen = torch.Generator().manual_seed(N)
    x = torch.randn(7, N, generator=gen).to(dtype).cuda()
    a = torch.randint(0, N, (7,), generator=gen).cuda()
    dlp, den = torch.randn(7, generator=gen).cuda(), torch.randn(7, generator=gen).cuda()
    rows = torch.arange(7, device="cuda")
    mask = torch.ones(7, N, dtype=torch.uint8, device="cuda")
    mask[rows, a] = 0
    below = x.clone()
    below[rows, a] = -math.inf
    for g1, g2 in ((dlp, den), (dlp, None)):
        want = rl.action_log_probs(x, a, temperature=0.7, mask=mask)
        got = rl.action_log_probs(below, a, temperature=0.7)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        assert torch.all(got[0] == -math.inf)
        want = rl.action_log_probs_backward(g1, g2, x, a, want[2], want[1], temperature=0.7, mask=mask)
        got = rl.action_log_probs_backward(g1, g2, below, a, got[2], got[1], temperature=0.7)
        assert torch.equal(got, want) and torch.all(got[rows, a] == 0)


def test_gradient_is_that_of_the_legal_ones():
    """d log p_a / d x_j = -p_j for j other than a, whatever x_a; float32: half a step of p and of its exponential's
    argument, |x| 2^-24 < 2^-21, and 2^-23 of the exponential."""
    x = torch.tensor([[0.5, -math.inf, 2.0, -1.0]])
    a = torch.tensor([1])
    lp, ent, lse = rl.action_log_probs(x.cuda(), a.cuda())
    d = rl.action_log_probs_backward(torch.ones(1).cuda(), None, x.cuda(), a.cuda(), lse, ent).cpu()
    want = -torch.softmax(x.double(), 1)
    assert d[0, 1] == 0 and torch.all((d - want).abs() <= want.abs() * 2.0 ** -19)
