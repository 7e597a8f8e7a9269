"""A policy over tokens, built from librlscan's sequence operators: a table looked up by token,
normalised and rotated queries and keys, linear attention, a gated recurrence, sampled
actions, and the gradients of all of it.

The task: every step shows a symbol, and pays 1 for the action that names the symbol shown `lag`
steps before it in the episode (the first steps of an episode pay nothing).

    python examples/token_policy.py [--updates 200] [--environments 256] [--dtype bf16]

Acting takes one step at a time: the attention's and the recurrence's states stay in pools, and
each environment counts the steps of its episode, which are the positions that heads are rotated
by.  Learning takes whole windows from the states that the window began with.
"""
import argparse
import math
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent))
sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from recurrent_policy import ActionLogProbs, Memory  # noqa: E402


class Embedding(torch.autograd.Function):
    """``rl.embed_tokens`` for autograd; the table's gradient is made in the activations' type."""

    @staticmethod
    def forward(ctx, table, tokens, dtype):
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.dtype = table.shape[0], table.dtype
        return rl.embed_tokens(table.to(dtype), tokens)

    @staticmethod
    def backward(ctx, d_out):
        (tokens,) = ctx.saved_tensors
        return rl.embed_tokens_backward(d_out.contiguous(), tokens, ctx.rows).to(ctx.dtype), None, None


class Heads(torch.autograd.Function):
    """``rl.norm_rotate_heads`` for autograd: (q, k)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        return rl.norm_rotate_heads(q, k, q_weight, k_weight, positions)

    @staticmethod
    def backward(ctx, d_q, d_k):
        return rl.norm_rotate_heads_backward(d_q.contiguous(), d_k.contiguous(), *ctx.saved_tensors) + (None,)


class Recurrence(torch.autograd.Function):
    """``rl.gated_recurrence`` for autograd; flags and the state it starts from get no gradient."""

    @staticmethod
    def forward(ctx, x, input_gate, decay_gate, rate, done, state, reset):
        out, marks = rl.gated_recurrence(x, input_gate, decay_gate, rate, done, state, reset=reset, with_marks=True)
        ctx.save_for_backward(x, input_gate, decay_gate, rate, marks, done, reset)
        return out

    @staticmethod
    def backward(ctx, d_out):
        *inputs, reset = ctx.saved_tensors
        return rl.gated_recurrence_backward(d_out.contiguous(), *inputs, reset=reset)[:4] + (None, None, None)


class Policy(torch.nn.Module):
    def __init__(self, symbols, heads=4, dim=32):
        super().__init__()
        self.heads, self.dim, width = heads, dim, heads * dim
        self.table = torch.nn.Parameter(torch.randn(symbols, width))
        self.qkv = torch.nn.Linear(width, 3 * width)
        self.q_weight = torch.nn.Parameter(torch.ones(dim))
        self.k_weight = torch.nn.Parameter(torch.ones(dim))
        self.gates = torch.nn.Linear(width, 3 * width)
        self.action = torch.nn.Linear(width, symbols)
        # heads forget over about 2 to 100 steps at first, channels over 2 to 1000
        self.head_rate = torch.nn.Parameter(torch.linspace(math.log(0.01), math.log(0.5), heads))
        self.rate = torch.nn.Parameter(torch.linspace(math.log(0.002), math.log(1.0), width))

    def project(self, x):
        """Queries, keys and values of what a step shows."""
        return self.qkv(x.float()).to(x.dtype).unflatten(-1, (3 * self.heads, self.dim)).split(self.heads, dim=-2)

    def mix(self, x, o):
        """The recurrence's input and its two gates, from what is shown and what attention found."""
        return self.gates(x.float() + o.flatten(-2).float()).to(x.dtype).chunk(3, dim=-1)

    def logits(self, h):
        return self.action(h.float()).to(h.dtype)


class Memories:
    """What acting keeps of each environment: both states and the step of its episode."""

    def __init__(self, policy, environments, device="cuda"):
        heads, dim = policy.heads, policy.dim
        self.attention = torch.zeros(environments, heads, dim, dim, device=device)
        self.recurrence = torch.zeros(environments, heads * dim, device=device)
        self.position = torch.zeros(environments, dtype=torch.int32, device=device)
        self.reset = torch.ones(environments, dtype=torch.bool, device=device)

    def start(self):
        """Both states and the resets as the window that follows takes them: an episode may have just ended."""
        return self.attention.masked_fill(self.reset[:, None, None, None], 0.0), self.recurrence.clone(), self.reset.clone()


class Task:
    def __init__(self, environments, symbols, lag, generator):
        self.symbols, self.lag, self.generator = symbols, lag, generator
        self.past = torch.full((environments, lag), -1, dtype=torch.int64, device=generator.device)
        self.shown = self._fresh()

    def _fresh(self):
        return torch.randint(self.symbols, self.past.shape[:1], generator=self.generator, device=self.past.device)

    def step(self, actions):
        """(reward, done); the next symbol is in self.shown."""
        reward = (actions == self.past[:, 0]).float()
        done = torch.rand(actions.shape, generator=self.generator, device=actions.device) < 1 / 32
        self.past = torch.cat([self.past[:, 1:], self.shown[:, None]], 1).masked_fill(done[:, None], -1)
        self.shown = self._fresh()
        return reward, done


@torch.no_grad()
def act(policy, task, memories, steps, dtype):
    """Plays a window; the memories are moved on in place.  Returns its arrays, [E, T]."""
    window, m = [], memories
    head_decay, rate, table = -policy.head_rate.exp(), policy.rate.exp(), policy.table.to(dtype)
    for _ in range(steps):
        shown, position = task.shown, m.position.masked_fill_(m.reset, 0).clone()
        x = rl.embed_tokens(table, shown)
        q, k, v = policy.project(x)
        q, k = rl.norm_rotate_heads(q, k, policy.q_weight, policy.k_weight, position)
        o = rl.linear_attention_step(q, k, v, head_decay, m.attention, m.reset)
        h = rl.gated_recurrence_step(*policy.mix(x, o), rate, m.recurrence, m.reset)
        uniforms = torch.rand(shown.shape, generator=task.generator, device=shown.device)
        actions, log_probs = rl.sample_actions(policy.logits(h), uniforms)
        reward, done = task.step(actions)
        m.position += 1
        m.reset.copy_(done)
        window.append((shown, position, actions, log_probs, reward, done))
    return [torch.stack(x, dim=1) for x in zip(*window)]


def loss_of(policy, window, start, dtype, entropy_weight=0.01):
    """(loss, log-probabilities under the policy as it is now) of a window played from `start`.
    An action is paid at once or not at all, so its reward alone is what it is weighed by."""
    shown, positions, actions, _, reward, done = window
    x = Embedding.apply(policy.table, shown, dtype)
    q, k, v = policy.project(x)
    q, k = Heads.apply(q, k, policy.q_weight, policy.k_weight, positions)
    o = Memory.apply(q, k, v, -policy.head_rate.exp(), done, start[0])
    h = Recurrence.apply(*policy.mix(x, o), policy.rate.exp(), done, *start[1:])
    log_probs, entropies = ActionLogProbs.apply(policy.logits(h), actions)
    loss = (-(reward - reward.mean()) * log_probs - entropy_weight * entropies).mean()
    return loss, log_probs


def train(updates=200, environments=256, steps=64, symbols=4, lag=2, dtype=torch.bfloat16, seed=0, report=None):
    """Mean reward of each update's window; chance is 1 / symbols where there is one to be had."""
    torch.manual_seed(seed)
    device = torch.device("cuda")
    policy = Policy(symbols).to(device)
    optimizer = torch.optim.Adam(policy.parameters(), lr=3e-3)
    task = Task(environments, symbols, lag, torch.Generator(device).manual_seed(seed))
    memories = Memories(policy, environments)
    rewards = []
    for update in range(updates):
        start = memories.start()
        window = act(policy, task, memories, steps, dtype)
        loss, _ = loss_of(policy, window, start, dtype)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        rewards.append(window[4].mean())
        if report and (update + 1) % report == 0:
            print("update %4d  reward %.3f" % (update + 1, rewards[-1].item()), flush=True)
    return [r.item() for r in rewards]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--updates", type=int, default=200)
    parser.add_argument("--environments", type=int, default=256)
    parser.add_argument("--steps", type=int, default=64)
    parser.add_argument("--dtype", choices=("bf16", "f16", "f32"), default="bf16")
    args = parser.parse_args()
    train(args.updates, args.environments, args.steps,
          dtype={"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[args.dtype], report=10)
