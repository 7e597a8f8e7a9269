"""Rows of logits that blocks share: the same actions and log-probabilities as one block a row
gives, where the shared passes suffice and where they do not (a
cut bin that overflows the list, more candidates than are ranked, fewer legal logits than top_k)."""
import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl

pytestmark = pytest.mark.gpu

SETTINGS = {
    "top_p": dict(top_p=0.9),
    "all": dict(),
    "min_p": dict(min_p=0.01, temperature=1.5),
    "top_k": dict(top_k=50),
    "top_k and top_p": dict(top_k=300, top_p=0.8, min_p=0.02),
    "more candidates than are ranked": dict(top_k=2000, top_p=0.95),
    "greedy": dict(temperature=0.0),
    "hot": dict(temperature=50.0, top_p=0.7),
    "cold": dict(temperature=0.05, top_p=0.99),
}


def _one_block_a_row(x, u, mask, kw):
    R, N = x.shape
    a = torch.full((R,), -7, dtype=torch.int64, device="cuda")
    lp = torch.full((R,), 9.0, device="cuda")
    fmt = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[x.dtype]
    st = rl.lib().rlscan_sample_actions(fmt, x.data_ptr(), N, None if mask is None else mask.data_ptr(), u.data_ptr(),
                                        None, None, None, None, kw.get("temperature", 1.0), kw.get("top_k", 0),
                                        kw.get("top_p", 1.0), kw.get("min_p", 0.0), a.data_ptr(), lp.data_ptr(), R, N,
                                        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return a, lp


def _rows(kind, R, N, dtype):
    g = torch.Generator().manual_seed(11)
    x = torch.randn(R, N, generator=g) * 2
    mask = None
    if kind == "equal":
        x = torch.zeros(R, N)
    elif kind == "two values":
        x = (torch.rand(R, N, generator=g) < 0.5).float()
    elif kind == "masked":
        mask = (torch.rand(R, N, generator=g) < 0.3).to(torch.uint8)
        mask[0] = 0
        mask[1] = 0
        mask[1, N - 3] = 1
    elif kind == "odd values":
        x[0, ::7] = float("-inf")
        x[0, 5] = float("nan")
        x[1, 100] = float("inf")
        x[2] = -3e38
        x[3] = float("-inf")
    return x.to(dtype), mask, torch.rand(R, generator=g)


@pytest.mark.parametrize("setting", SETTINGS)
@pytest.mark.parametrize("kind,R,N,dtype", [
    ("normal", 1, 131072, torch.float32), ("normal", 4, 32768, torch.float32), ("normal", 5, 50007, torch.bfloat16),
    ("normal", 4, 40483, torch.float16), ("equal", 4, 33333, torch.float32), ("two values", 4, 36865, torch.bfloat16),
    ("masked", 4, 40003, torch.float32), ("odd values", 4, 34567, torch.float32), ("normal", 64, 32771, torch.bfloat16),
])
def test_same_as_one_block_a_row(kind, R, N, dtype, setting):
    kw = SETTINGS[setting]
    x, mask, u = _rows(kind, R, N, dtype)
    xd, ud, md = x.cuda(), u.cuda(), None if mask is None else mask.cuda()
    assert rl.lib().rlscan_sample_actions_workspace(R, N) > 0
    got = rl.sample_actions(xd, ud, mask=md, **kw)
    want = _one_block_a_row(xd, ud, md, kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_at_any_offset():
    x = torch.randn(4, 32768 + 16)
    u = torch.rand(4).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        wide = x.to(dtype).cuda()
        for lead in range(8):
            part = wide[:, lead:lead + 32775]
            for kw in (dict(top_p=0.9), dict(top_k=40), dict()):
                got, want = rl.sample_actions(part, u, **kw), _one_block_a_row(part.contiguous(), u, None, kw)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_workspace_is_checked():
    x, u = torch.randn(2, 40000, device="cuda"), torch.rand(2, device="cuda")
    a, lp = torch.empty(2, dtype=torch.int64, device="cuda"), torch.empty(2, device="cuda")
    need = rl.lib().rlscan_sample_actions_workspace(2, 40000)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(p, n):
        return rl.lib().rlscan_sample_actions_shared(0, x.data_ptr(), 40000, None, u.data_ptr(), None, None, None, None,
                                                     1.0, 0, 0.9, 0.0, a.data_ptr(), lp.data_ptr(), p, n, 2, 40000,
                                                     torch.cuda.current_stream().cuda_stream)

    assert call(ws.data_ptr(), need - 1) == 7
    assert call(ws.data_ptr() + 4, need) == 5
    assert call(x.data_ptr(), need) == 6
    assert call(ws.data_ptr(), need) == 0


def test_settings_of_its_own_for_each_row():
    R, N = 12, 40000
    x, _, u = _rows("normal", R, N, torch.float32)
    ks = torch.tensor([0, 5, 0, 400, 3000, 0] * 2, dtype=torch.int32)
    ps = torch.tensor([1.0, 0.9, 0.5, 0.95, 0.9, 0.99] * 2)
    got = rl.sample_actions(x.cuda(), u.cuda(), top_k=ks.cuda(), top_p=ps.cuda())
    for r in range(R):
        want = _one_block_a_row(x[r:r + 1].cuda(), u[r:r + 1].cuda(), None,
                                dict(top_k=int(ks[r]), top_p=float(ps[r])))
        assert got[0][r] == want[0][0] and got[1][r] == want[1][0]
