"""Linear attention's paths of long rows that shorter ones do not reach: segments of heads wider than
64, marked boundaries past 512 steps of such heads, and the decay's gradient past one tile of
4096 steps.  Oracle and tolerances are those of test_gpu_linear_attention."""
import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl
from tests.test_gpu_linear_attention import check_backward, check_forward, make

pytestmark = pytest.mark.gpu

FMT = {"f32": 0, "bf16": 1, "f16": 2}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,V", [(128, 128), (100, 128), (128, 40), (127, 65)])
@pytest.mark.parametrize("T,H,G", [(600, 1, 1), (1100, 2, 2), (2113, 1, 1)])
def test_segments_of_wide_heads(dtype, K, V, T, H, G):
    for backward in (0, 1):
        assert rl.lib().rlscan_linear_attention_workspace(FMT[dtype], 1, T, H, H // G, K, V, backward) > 0
    # segments: as much workspace as their states and decays take
    assert rl.lib().rlscan_linear_attention_workspace(FMT[dtype], 1, T, H, H // G, K, V, 0) >= 2 * H * 128 * 128 * 4
    d = make(T + K, 1, T, H, G, K, V, dtype, p_done=0.003, decay=0.01)
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_between_cuts(dtype):
    """A cut at, before and after each segment's first step; a row that no cut divides."""
    T = 2048
    for at in (None, -1, 0, 1):
        d = make(5, 1, T, 1, 1, 128, 128, dtype, p_done=0.0, decay=0.005)
        if at is not None:
            d["done"] = torch.zeros(1, T, dtype=torch.uint8)
            d["done"][0, [t + at for t in range(256, T, 256)]] = 1
        check_forward(d)
        check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("per_step", [True, False])
@pytest.mark.parametrize("T", [4096, 4097, 8200])
def test_decay_gradient_past_one_tile(dtype, per_step, T):
    d = make(T, 1, T, 1, 1, 16, 24, dtype, per_step=per_step, p_done=0.0, decay=0.01)
    check_backward(d)
    for cut in (4094, 4095, 4096):  # the step after starts afresh; 4096 begins a tile and a marked boundary
        if cut >= T:
            continue
        d["done"] = torch.zeros(1, T, dtype=torch.uint8)
        d["done"][0, cut] = 1
        got = check_backward(d)
        if per_step and cut + 1 < T:
            assert got[3][0, cut + 1, 0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_heads_of_several_rows(dtype):
    """Several rows and heads at once, with a short last chunk: every index of the workspace counts."""
    d = make(9, 3, 1000, 4, 2, 128, 96, dtype, p_done=0.01, decay=0.01)
    check_forward(d)
    check_backward(d)
