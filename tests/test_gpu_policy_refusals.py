"""Arguments past the range of what the C entries take are refused, not wrapped into it."""
import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl


@pytest.mark.gpu
@pytest.mark.parametrize("k", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 5, -2 ** 64])
def test_negative_top_k(k):
    x, u = torch.randn(3, 40, device="cuda"), torch.rand(3, device="cuda")
    with pytest.raises(rl.RlscanError):
        rl.sample_actions(x, u, top_k=k)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [40, 2 ** 31, 2 ** 32 + 5, 2 ** 70])
def test_top_k_past_the_row_is_off(k):
    x, u = torch.randn(3, 40, device="cuda"), torch.rand(3, device="cuda")
    assert torch.equal(rl.sample_actions(x, u, top_k=k)[0], rl.sample_actions(x, u)[0])


@pytest.mark.gpu
def test_heads_of_no_size():
    q, v = torch.zeros(2, 5, 4, 0, device="cuda"), torch.zeros(2, 5, 4, 8, device="cuda")
    g = torch.zeros(4, device="cuda")
    with pytest.raises(rl.RlscanError):
        rl.linear_attention(q, q, v, g)
    with pytest.raises(rl.RlscanError):
        rl.linear_attention_backward(v, q, q, v, g)
    with pytest.raises(rl.RlscanError):
        rl.linear_attention_step(q[:, 0], q[:, 0], v[:, 0], g, torch.zeros(2, 4, 0, 8, device="cuda"))
