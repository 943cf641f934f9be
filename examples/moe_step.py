"""Data-parallel training of a small mixture-of-experts block over virtual
workers: route, experts, residual with dropout, backward, one DynamiQ round per
step.

Every worker holds the same weights and its own tokens.  A step
  * routes all workers' tokens and takes ONE balance loss over them
    (``train.route`` with a list: the statistics are folded over the workers);
  * runs the chosen experts, weighted by the gates, and adds the result to the
    residual stream under dropout, whose mask depends on (seed, step, worker,
    layer) and is drawn again in the backward pass;
  * differentiates each worker's loss by its own copy of the weights, and sums
    the workers' flattened gradients in a compressed round (``dq.Plan.allreduce``,
    the step as its round index);
  * applies the mean gradient.

    python examples/moe_step.py [--steps 60] [--workers 4] [--exact] [--grouped] [--keep]

``--exact`` sums the gradients in fp32 instead, for comparison.  ``--grouped`` runs all
experts at once (``train.experts``) instead of one after the other, ``--keep`` does so from
activations kept in 8 bits.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from compressed_hop_gradient_amd import dq, train  # noqa: E402

HIDDEN, FFN, EXPERTS, TOP_K, CLASSES, LAYERS = 64, 128, 16, 2, 16, 2
DROPOUT, BALANCE = 0.1, 0.02


def init(seed=0, device="cuda"):
    """Weights, fp32; names are the keys of the gradient's layout."""
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, scale):
        return (torch.randn(*shape, generator=g) * scale).to(device)

    w = {"out": randn(HIDDEN, CLASSES, scale=HIDDEN ** -0.5)}
    for i in range(LAYERS):
        w[f"router{i}"] = randn(HIDDEN, EXPERTS, scale=HIDDEN ** -0.5)
        w[f"up{i}"] = randn(EXPERTS, HIDDEN, FFN, scale=HIDDEN ** -0.5)
        w[f"down{i}"] = randn(EXPERTS, FFN, HIDDEN, scale=0.5 * FFN ** -0.5)
    return w


def batch(worker, step, tokens, device="cuda"):
    """A worker's tokens and labels: clusters whose label is a fixed function."""
    g = torch.Generator().manual_seed(1000003 * step + worker)
    centers = torch.randn(64, HIDDEN, generator=torch.Generator().manual_seed(7))
    which = torch.randint(0, 64, (tokens,), generator=g)
    x = centers[which] + 0.3 * torch.randn(tokens, HIDDEN, generator=g)
    return x.to(device), (which * 5 % CLASSES).to(device)


def experts(x, ids, gates, up, down):
    """sum_s gate_s expert_{id_s}(x), one expert's tokens at a time."""
    y = torch.zeros_like(x)
    for e in range(EXPERTS):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            h = F.relu(x[token] @ up[e]) @ down[e]
            y = y.index_add(0, token, h * gates[token, slot, None])
    return y


def losses(weights, data, step, training=True, grouped=False, keep=False):
    """Each worker's task loss, and the balance loss of all workers' tokens."""
    def run(x, ids, g, up, down, n, i):
        if not grouped:
            return experts(x, ids, g, up, down)
        return train.experts(x, ids, g, up, down, act="relu", keep=keep, rnd=step, worker=n, site=LAYERS + 2 * i)

    xs = [x for x, _ in data]
    balance, counts = 0.0, []
    for i in range(LAYERS):
        r = train.route([x @ w[f"router{i}"] for x, w in zip(xs, weights)], TOP_K)
        balance = balance + r.loss / LAYERS
        counts.append(r.counts)
        xs = [train.dropout(run(x, ids, g, w[f"up{i}"], w[f"down{i}"], n, i), DROPOUT, residual=x, training=training,
                            rnd=step, worker=n, site=i)
              for n, (x, ids, g, w) in enumerate(zip(xs, r.ids, r.gates, weights))]
    task = [F.cross_entropy(x @ w["out"], y) for x, w, (_, y) in zip(xs, weights, data)]
    return task, balance, counts


class Trainer:
    """The workers' weights (one storage, a leaf per worker), the plan of the
    gradient round and the optimizer step."""

    def __init__(self, workers=4, tokens=256, avg_bits=5.0, exact=False, lr=0.5, seed=0, grouped=False, keep=False):
        self.weights, self.workers, self.tokens, self.exact, self.lr = init(seed), workers, tokens, exact, lr
        self.grouped, self.keep = grouped or keep, keep
        self.sizes = [w.numel() for w in self.weights.values()]
        self.n = (sum(self.sizes) + 255) // 256 * 256            # whole super-groups
        self.plan = dq.Plan(self.n, workers, dq.RING, avg_bits)
        self.grads = [torch.zeros(self.n, device="cuda") for _ in range(workers)]

    def step(self, step):
        leaves = [{k: w.detach().requires_grad_() for k, w in self.weights.items()} for _ in range(self.workers)]
        data = [batch(n, step, self.tokens) for n in range(self.workers)]
        task, balance, counts = losses(leaves, data, step, grouped=self.grouped, keep=self.keep)
        # the balance loss is one for all workers: its gradient by each worker's
        # weights is that worker's share, times the workers because the sum below
        # is averaged
        total = sum(task) + BALANCE * self.workers * balance.sum()
        flat = torch.autograd.grad(total, [w for l in leaves for w in l.values()])
        k = len(self.weights)
        for n in range(self.workers):
            torch.cat([g.reshape(-1) for g in flat[n * k:n * k + k]], out=self.grads[n][:sum(self.sizes)])
        if self.exact:
            mean = sum(self.grads[1:], self.grads[0].clone()) / self.workers
        else:
            self.plan.set(dq.OPT_ROUND, step)
            mean = self.plan.allreduce(self.grads) / self.workers
        for w, g in zip(self.weights.values(), mean[:sum(self.sizes)].split(self.sizes)):
            w -= self.lr * g.view_as(w)
        return (sum(task) / self.workers).item(), balance.item(), counts


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--workers", type=int, default=4)
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--exact", action="store_true")
    p.add_argument("--grouped", action="store_true")
    p.add_argument("--keep", action="store_true")
    a = p.parse_args()
    t = Trainer(a.workers, a.tokens, exact=a.exact, grouped=a.grouped, keep=a.keep)
    for step in range(a.steps):
        task, balance, counts = t.step(step)
        if step % 10 == 0 or step == a.steps - 1:
            share = counts[0].double() / counts[0].sum()
            print(f"step {step:4d}  loss {task:.4f}  balance {balance:.4f}  busiest expert {share.max():.3f}", flush=True)


if __name__ == "__main__":
    main()
