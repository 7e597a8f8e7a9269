"""The example that runs the policy operators together: what acting computes one step at a
time is what learning computes over the window, its gradients are those of plain torch in
float64, and it learns the task."""
import importlib.util
import pathlib

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = pathlib.Path(__file__).resolve().parents[1] / "examples" / "recurrent_policy.py"
SPEC = importlib.util.spec_from_file_location("recurrent_policy", PATH)
example = importlib.util.module_from_spec(SPEC)
SPEC.loader.exec_module(example)


def _window(dtype, environments=24, steps=37, symbols=5):
    torch.manual_seed(3)
    policy = example.Policy(symbols, heads=2, dim=16).cuda()
    task = example.Task(environments, symbols, torch.Generator("cuda").manual_seed(4))
    state = torch.zeros(environments, 2, 16, 16, device="cuda")
    reset = torch.ones(environments, dtype=torch.bool, device="cuda")
    example.act(policy, task, state, reset, 9, dtype)  # so that the window starts inside episodes
    start = state.masked_fill(reset[:, None, None, None], 0.0)
    return policy, start, example.act(policy, task, state, reset, steps, dtype)


def test_acting_and_learning_agree():
    # float32: sums of 37 steps x 16 features in two orders, log-probabilities of order 1
    policy, start, window = _window(torch.float32)
    _, log_probs = example.loss_of(policy, window, start, torch.zeros(24, device="cuda"), torch.float32)
    assert (log_probs.detach() - window[2]).abs().max().item() < 2e-5
    assert window[4].any() and start.abs().sum() > 0


def test_gradients_are_those_of_plain_torch():
    policy, start, window = _window(torch.float32)
    bootstrap = torch.full((24,), 0.3, device="cuda")
    loss, _ = example.loss_of(policy, window, start, bootstrap, torch.float32)
    got = torch.autograd.grad(loss, list(policy.parameters()))

    plain = example.Policy(5, heads=2, dim=16).double()
    plain.load_state_dict({n: p.detach().cpu().double() for n, p in policy.state_dict().items()})
    shown, actions, behaviour, reward, done = [x.cpu() for x in window]
    q, k, v = plain.project(shown, torch.float64)
    s, outs = start.cpu().double(), []
    for t in range(shown.shape[1]):
        if t:
            s = s * (~done[:, t - 1]).double()[:, None, None, None]
        s = plain.log_decay().exp()[None, :, None, None] * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(16 ** -0.5 * (q[:, t, :, :, None] * s).sum(-2))
    o = torch.stack(outs, 1).flatten(-2)
    logits, values = plain.action(o), plain.value(o).squeeze(-1)
    log_p = logits.log_softmax(-1)
    log_probs = log_p.gather(-1, actions[..., None]).squeeze(-1)
    entropies = -(log_p.exp() * log_p).sum(-1)
    rho = (log_probs.detach() - behaviour.double()).exp().clamp(max=1.0)
    target = values.detach()
    vs, advantages, after = torch.empty_like(target), torch.empty_like(target), torch.zeros(24, dtype=torch.float64)
    next_v = next_vs = bootstrap.cpu().double()
    for t in reversed(range(shown.shape[1])):
        live = 0.5 * (~done[:, t]).double()
        delta = rho[:, t] * (reward[:, t].double() + live * next_v - target[:, t])
        after = delta + live * rho[:, t] * after
        vs[:, t] = target[:, t] + after
        advantages[:, t] = rho[:, t] * (reward[:, t].double() + live * next_vs - target[:, t])
        next_v, next_vs = target[:, t], vs[:, t]
    want_loss = (-(advantages * log_probs) + 0.5 * (values - vs) ** 2 - 0.01 * entropies).mean()
    want = torch.autograd.grad(want_loss, list(plain.parameters()))
    # the head's own float32 products and sums over 888 steps: 888^0.5 roundings of 2^-24 and a
    # few products' worth, on gradients that partly cancel
    for g, w in zip(got, want):
        scale = w.abs().max().item()
        assert (g.cpu().double() - w).abs().max().item() < 1e-4 * scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_it_learns(dtype):
    rewards = example.train(updates=60, environments=128, steps=32, symbols=4, dtype=dtype)
    assert sum(rewards[-5:]) / 5 > 0.6 > 0.4 > rewards[0]  # chance: 0.25
