"""Call forms of the sequence operators that only a C program can ask for, on the GPU."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,T", [(2, 3), (1, 1), (0, 5), (70000, 900)])
def test_weight_gradients_of_no_heads(E, T):
    # zeros, and no position is looked at: there are no tokens without heads
    lib, D = rl.lib(), 48
    need = lib.rlscan_norm_rotate_heads_workspace(E, T, 0, 0, D)
    workspace = torch.full((need // 4,), 3.0, device="cuda")
    d_weights = torch.full((2, D), 7.0, device="cuda")
    st = lib.rlscan_norm_rotate_heads_backward(
        0, 0, None, None, None, None, None, None, None, None, None, d_weights[0].data_ptr(), d_weights[1].data_ptr(),
        workspace.data_ptr(), need, E, T, 0, 0, D, D, 10000.0, 0, 1e-6, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert not d_weights.any()
