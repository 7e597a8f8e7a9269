"""The example that runs the sequence operators together: what acting computes one step at a time
is what learning computes over the window, and its gradients are those of plain torch in float64."""
import importlib.util
import pathlib

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = pathlib.Path(__file__).resolve().parents[1] / "examples" / "token_policy.py"
SPEC = importlib.util.spec_from_file_location("token_policy", PATH)
example = importlib.util.module_from_spec(SPEC)
SPEC.loader.exec_module(example)
E, T, SYMBOLS = 24, 45, 5


def _window(dtype):
    torch.manual_seed(5)
    policy = example.Policy(SYMBOLS, heads=2, dim=16).cuda()
    with torch.no_grad():
        for w in (policy.q_weight, policy.k_weight):
            w.copy_(1 + 0.2 * torch.randn_like(w))
    task = example.Task(E, SYMBOLS, 2, torch.Generator("cuda").manual_seed(6))
    memories = example.Memories(policy, E)
    example.act(policy, task, memories, 9, dtype)  # so that the window starts inside episodes
    start = memories.start()
    return policy, start, example.act(policy, task, memories, T, dtype)


def _plain(policy, window, start):
    """The same loss by plain torch in float64 on the CPU: (loss, log-probabilities, parameters)."""
    plain = example.Policy(SYMBOLS, heads=2, dim=16).double()
    plain.load_state_dict({n: p.detach().cpu().double() for n, p in policy.state_dict().items()})
    shown, positions, actions, _, reward, done = [x.cpu() for x in window]
    x = plain.table[shown]
    heads = torch.nn.functional.linear(x, plain.qkv.weight, plain.qkv.bias).unflatten(-1, (6, 16))
    freq = 10000.0 ** (-torch.arange(8, dtype=torch.float64) / 8)
    angle = (positions.double()[..., None] * freq)[:, :, None]

    def turned(z, weight):
        z = weight * z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6)
        a, b = z[..., :8], z[..., 8:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    q, k, v = turned(heads[:, :, :2], plain.q_weight), turned(heads[:, :, 2:4], plain.k_weight), heads[:, :, 4:]
    s, h = start[0].cpu().double(), start[1].cpu().double()
    rate, outs = plain.rate.exp(), []
    for t in range(T):
        fresh = done[:, t - 1, None] if t else start[2].cpu()[:, None]
        s, h = s * (~fresh).double()[..., None, None], h * (~fresh).double()
        s = (-plain.head_rate.exp()).exp()[None, :, None, None] * s + k[:, t, :, :, None] * v[:, t, :, None, :]
        o = (16 ** -0.5 * (q[:, t, :, :, None] * s).sum(-2)).flatten(-2)
        u, i, r = torch.nn.functional.linear(x[:, t] + o, plain.gates.weight, plain.gates.bias).chunk(3, -1)
        log_a = -rate * torch.sigmoid(r)
        m = torch.where(fresh, torch.ones_like(log_a), torch.sqrt(-torch.expm1(2 * log_a)))
        h = log_a.exp() * h + m * torch.sigmoid(i) * u
        outs.append(h)
    log_p = torch.nn.functional.linear(torch.stack(outs, 1), plain.action.weight, plain.action.bias).log_softmax(-1)
    log_probs = log_p.gather(-1, actions[..., None]).squeeze(-1)
    entropies = -(log_p.exp() * log_p).sum(-1)
    reward = reward.double()
    loss = (-(reward - reward.mean()) * log_probs - 0.01 * entropies).mean()
    return loss, log_probs, list(plain.parameters())


def test_acting_and_learning_agree():
    # Roundings of float32 (2^-24 each) along a step's chain: products of 32 and sums over 45 steps x 16
    # features in two orders, 150 of them worst case in the relative sense, on logits of order 1 made
    # from states of order 4: 4 * 150 * 2^-24 = 4e-5
    policy, start, window = _window(torch.float32)
    _, log_probs = example.loss_of(policy, window, start, torch.float32)
    assert (log_probs.detach() - window[3]).abs().max().item() < 4e-5
    assert window[5].any() and start[0].any() and start[2].any() and not start[2].all() and (window[1] > 9).any()


def test_gradients_are_those_of_plain_torch():
    policy, start, window = _window(torch.float32)
    loss, log_probs = example.loss_of(policy, window, start, torch.float32)
    got = torch.autograd.grad(loss, list(policy.parameters()))
    want_loss, want_probs, parameters = _plain(policy, window, start)
    want = torch.autograd.grad(want_loss, parameters)
    assert (log_probs.detach().cpu().double() - want_probs.detach()).abs().max().item() < 4e-5
    # a chain of products and sums over 1080 steps, whose float32 roundings are of either sign: about
    # 1080^0.5 + 150 of 2^-24, on gradients that cancel to a tenth of their terms
    for (name, _), g, w in zip(policy.named_parameters(), got, want):
        scale = w.abs().max().item()
        assert (g.cpu().double() - w).abs().max().item() < 1.2e-4 * scale, name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_it_runs_in_16_bits(dtype):
    policy, start, window = _window(dtype)
    assert window[2].min().item() >= 0 and window[2].max().item() < SYMBOLS
    loss, log_probs = example.loss_of(policy, window, start, dtype)
    grads = torch.autograd.grad(loss, list(policy.parameters()))
    assert torch.isfinite(loss) and torch.isfinite(log_probs).all()
    assert all(torch.isfinite(g).all() and g.any() for g in grads)


def test_training_runs():
    rewards = example.train(updates=3, environments=40, steps=21)
    assert len(rewards) == 3 and all(0.0 <= r <= 1.0 for r in rewards)


def test_a_captured_step_of_acting_is_replayed():
    """Look-up, heads, attention, recurrence and sampling of one step in a graph, replayed between eager steps
    on pools of their own: every replay gives what the eager step gives."""
    rl = example.rl
    torch.manual_seed(7)
    policy = example.Policy(SYMBOLS, heads=2, dim=16).cuda()
    head_decay, rate = -policy.head_rate.detach().exp(), policy.rate.detach().exp()
    table, qw, kw = policy.table.detach(), policy.q_weight.detach(), policy.k_weight.detach()
    g = torch.Generator("cuda").manual_seed(8)
    draws = []
    for t in range(5):
        draws.append((torch.randint(-1, SYMBOLS, (E,), generator=g, device="cuda"),
                      torch.full((E,), t, dtype=torch.int32, device="cuda"),
                      torch.randn(2, E, 3 * 32, generator=g, device="cuda"), torch.rand(E, generator=g, device="cuda"),
                      torch.rand(E, generator=g, device="cuda") < 0.2))

    def step(shown, position, noise, uniforms, reset, pools):
        x = rl.embed_tokens(table, shown)
        q, k, v = (noise[0] + torch.cat([x, x, x], 1)).unflatten(-1, (6, 16)).split(2, dim=-2)
        q, k = rl.norm_rotate_heads(q, k, qw, kw, position)
        o = rl.linear_attention_step(q, k, v, head_decay, pools[0], reset)
        u, i, r = (noise[1] + torch.cat([o.flatten(-2)] * 3, 1)).chunk(3, dim=-1)
        h = rl.gated_recurrence_step(u, i, r, rate, pools[1], reset)
        return rl.sample_actions(h[:, :SYMBOLS].contiguous(), uniforms) + (h,)

    def pools():
        return torch.zeros(E, 2, 16, 16, device="cuda"), torch.zeros(E, 32, device="cuda")

    held = [x.clone() for x in draws[0]]
    kept, eager = pools(), pools()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held, pools())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*held, kept)
    for p in kept:
        p.zero_()
    for draw in draws:
        for x, y in zip(held, draw):
            x.copy_(y)
        graph.replay()
        want = step(*draw, eager)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(captured, want))
        assert all(torch.equal(x, y) for x, y in zip(kept, eager))
