"""A policy that remembers, trained with librlscan: linear attention over the episode as
its memory, sampled actions, V-trace targets and the gradients of all of it.

The task: the first step of an episode shows one of `symbols`, later steps show nothing,
and every step pays 1 for the action that names the symbol.  Episodes end at random.

    python examples/recurrent_policy.py [--updates 150] [--environments 256] [--dtype bf16]

Acting takes one step at a time: ``linear_attention_step`` moves each environment's state
and ``sample_actions`` picks the action.  Learning takes whole windows: ``linear_attention``
reads the same memory for all steps at once, ``action_log_probs`` gives V-trace its
importance ratios and the loss its entropy, and the two backward functions return the
gradients to torch.
"""
import argparse
import math
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
import linear_recurrence_scan_reverse_amd as rl  # noqa: E402


class Memory(torch.autograd.Function):
    """``rl.linear_attention`` for autograd; done and the state it starts from get no gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, done, state):
        ctx.save_for_backward(q, k, v, log_decay, done, state)
        return rl.linear_attention(q, k, v, log_decay, done, state)

    @staticmethod
    def backward(ctx, d_out):
        q, k, v, log_decay, done, state = ctx.saved_tensors
        dq, dk, dv, dg, _ = rl.linear_attention_backward(d_out.contiguous(), q, k, v, log_decay, done, state)
        return dq, dk, dv, dg, None, None


class ActionLogProbs(torch.autograd.Function):
    """``rl.action_log_probs`` for autograd: (log_probs, entropies)."""

    @staticmethod
    def forward(ctx, logits, actions):
        log_probs, entropies, lse = rl.action_log_probs(logits, actions)
        ctx.save_for_backward(logits, actions, lse, entropies)
        return log_probs, entropies

    @staticmethod
    def backward(ctx, d_log_probs, d_entropies):
        logits, actions, lse, entropies = ctx.saved_tensors
        return rl.action_log_probs_backward(d_log_probs.contiguous(), d_entropies.contiguous(), logits, actions, lse,
                                            entropies), None


class Policy(torch.nn.Module):
    def __init__(self, symbols, heads=4, dim=32):
        super().__init__()
        self.heads, self.dim = heads, dim
        self.qkv = torch.nn.Embedding(symbols + 1, 3 * heads * dim)  # of what a step shows; `symbols` is nothing
        self.action = torch.nn.Linear(heads * dim, symbols)
        self.value = torch.nn.Linear(heads * dim, 1)
        # heads forget at their own rates, over about 2 to 100 steps at first
        self.rate = torch.nn.Parameter(torch.linspace(math.log(0.01), math.log(0.5), heads))

    def log_decay(self):
        return -self.rate.exp()

    def project(self, shown, dtype):
        x = self.qkv(shown).to(dtype)
        return x.unflatten(-1, (3 * self.heads, self.dim)).split(self.heads, dim=-2)

    def heads_of(self, o, dtype):
        o = o.flatten(-2).float()
        return self.action(o).to(dtype), self.value(o).squeeze(-1)


class Task:
    def __init__(self, environments, symbols, generator):
        self.symbols, self.generator = symbols, generator
        self.target = torch.randint(symbols, (environments,), generator=generator, device=generator.device)
        self.shown = self.target.clone()

    def step(self, actions):
        """(reward, done); the next thing shown is in self.shown."""
        n, dev = self.target.shape, self.target.device
        reward = (actions == self.target).float()
        done = torch.rand(n, generator=self.generator, device=dev) < 1 / 16
        fresh = torch.randint(self.symbols, n, generator=self.generator, device=dev)
        self.target = torch.where(done, fresh, self.target)
        self.shown = torch.where(done, fresh, torch.full_like(fresh, self.symbols))
        return reward, done


@torch.no_grad()
def act(policy, task, state, reset, steps, dtype):
    """Plays a window; `state` and `reset` are moved on in place.  Returns its arrays, [E, T]."""
    window = []
    log_decay = policy.log_decay()
    for _ in range(steps):
        shown = task.shown
        q, k, v = policy.project(shown, dtype)
        logits, _ = policy.heads_of(rl.linear_attention_step(q, k, v, log_decay, state, reset), dtype)
        uniforms = torch.rand(shown.shape, generator=task.generator, device=shown.device)
        actions, log_probs = rl.sample_actions(logits, uniforms)
        reward, done = task.step(actions)
        reset.copy_(done)
        window.append((shown, actions, log_probs, reward, done))
    return [torch.stack(x, dim=1) for x in zip(*window)]


def loss_of(policy, window, state, bootstrap, dtype, gamma=0.5, entropy_weight=0.01):
    """(loss, log-probabilities under the policy as it is now) of a window played from `state`."""
    shown, actions, behaviour, reward, done = window
    q, k, v = policy.project(shown, dtype)
    o = Memory.apply(q, k, v, policy.log_decay(), done, state)
    logits, values = policy.heads_of(o, dtype)
    log_probs, entropies = ActionLogProbs.apply(logits, actions)
    with torch.no_grad():
        targets, advantages = rl.vtrace(reward, values.detach().contiguous(), log_probs.detach() - behaviour, done,
                                        bootstrap_value=bootstrap, gamma=gamma)
    loss = (-(advantages * log_probs) + 0.5 * (values - targets) ** 2 - entropy_weight * entropies).mean()
    return loss, log_probs


def train(updates=150, environments=256, steps=64, symbols=8, dtype=torch.bfloat16, seed=0, report=None):
    """Mean reward of each update's window; chance is 1 / symbols."""
    torch.manual_seed(seed)
    device = torch.device("cuda")
    policy = Policy(symbols).to(device)
    optimizer = torch.optim.Adam(policy.parameters(), lr=1e-2)
    task = Task(environments, symbols, torch.Generator(device).manual_seed(seed))
    state = torch.zeros(environments, policy.heads, policy.dim, policy.dim, device=device)
    reset = torch.ones(environments, dtype=torch.bool, device=device)
    rewards = []
    for update in range(updates):
        start = state.masked_fill(reset[:, None, None, None], 0.0)  # an episode may have ended with the last window
        window = act(policy, task, state, reset, steps, dtype)
        with torch.no_grad():  # the value after the window, from a state that is then forgotten
            q, k, v = policy.project(task.shown, dtype)
            o = rl.linear_attention_step(q, k, v, policy.log_decay(), state.clone(), reset)
            bootstrap = policy.heads_of(o, dtype)[1]
        loss, _ = loss_of(policy, window, start, bootstrap, dtype)
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        rewards.append(window[3].mean())
        if report and (update + 1) % report == 0:
            print("update %4d  reward %.3f" % (update + 1, rewards[-1].item()), flush=True)
    return [r.item() for r in rewards]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--updates", type=int, default=150)
    parser.add_argument("--environments", type=int, default=256)
    parser.add_argument("--steps", type=int, default=64)
    parser.add_argument("--dtype", choices=("bf16", "f16", "f32"), default="bf16")
    args = parser.parse_args()
    train(args.updates, args.environments, args.steps,
          dtype={"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[args.dtype], report=10)
