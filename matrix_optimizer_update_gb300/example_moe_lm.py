"""A small mixture-of-experts language model trained with every operator of the library.

    python -m matrix_optimizer_update_gb300.example_moe_lm [--steps N] [--distill]

One step: tokens -> embedding -> router -> ``Router`` sends rows to the experts
-> experts' products -> ``Router`` combines them -> head -> ``Head`` gives the
loss (cross entropy, or distillation from the stored top logits of a teacher)
and its gradients, without the logits. The experts' and the router's matrices
are updated by ``Muon``, embedding and head by AdamW (``dmuon_adamw_flat``).

The data is synthetic: the next token is a fixed random function of the last,
which the model has to learn by heart.
"""

from __future__ import annotations

import argparse
import functools

import torch

from . import dmuon as dm


def first_derivative(backward):
    """A backward pass that is an error with create_graph=True: the library's calls leave no graph, so a second
    derivative through them would silently be missing. (once_differentiable refuses only where the gradient that
    comes in has a graph, not where saved tensors have one.)"""

    @functools.wraps(backward)
    def checked(ctx, grad):
        if torch.is_grad_enabled():
            raise RuntimeError("the library's operators have no second derivatives")
        return backward(ctx, grad)

    return checked


class Dispatch(torch.autograd.Function):
    """xs = x's rows in expert order."""

    @staticmethod
    def forward(ctx, x, router, route):
        ctx.router, ctx.route = router, route
        return router.dispatch(x, route)

    @staticmethod
    @first_derivative
    def backward(ctx, dxs):
        return ctx.router.dispatch_backward(dxs.contiguous(), ctx.route), None, None


class Combine(torch.autograd.Function):
    """y = each token's expert rows, weighted."""

    @staticmethod
    def forward(ctx, ys, weights, router, route):
        ctx.router, ctx.route = router, route
        ctx.save_for_backward(ys, weights)
        return router.combine(ys, weights, route)

    @staticmethod
    @first_derivative
    def backward(ctx, dy):
        dys, dw = ctx.router.combine_backward(dy.contiguous(), *ctx.saved_tensors, ctx.route)
        return dys, dw, None, None


class Xent(torch.autograd.Function):
    """Each token's cross entropy, without the logits."""

    @staticmethod
    def forward(ctx, hidden, weight, head, targets):
        loss, lse = head.xent(hidden, weight, targets)
        ctx.head = head
        ctx.save_for_backward(hidden, weight, targets, lse, loss)
        return loss

    @staticmethod
    @first_derivative
    def backward(ctx, grad):
        hidden, weight, targets, lse, loss = ctx.saved_tensors
        return (*ctx.head.xent_backward(hidden, weight, targets, lse, grad.contiguous(), loss=loss), None, None)


class Distill(torch.autograd.Function):
    """Each token's divergence from a teacher's top logits."""

    @staticmethod
    def forward(ctx, hidden, weight, head, top_ids, top_logits, temperature):
        loss, lse = head.distill(hidden, weight, top_ids, top_logits, temperature)
        ctx.head, ctx.temperature = head, temperature
        ctx.save_for_backward(hidden, weight, top_ids, top_logits, lse)
        return loss

    @staticmethod
    @first_derivative
    def backward(ctx, grad):
        hidden, weight, ids, logits, lse = ctx.saved_tensors
        return (*ctx.head.distill_backward(hidden, weight, ids, logits, ctx.temperature, lse, grad.contiguous()), None,
                None, None, None)


class Model:
    """Embedding, one mixture-of-experts layer with a residual, a norm, and a head."""

    def __init__(self, vocab=1000, dim=128, inner=256, experts=8, top=2, max_tokens=512, max_top=16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(rows, cols, std):
            return (torch.randn(rows, cols, generator=g, device="cuda") * std).to(torch.bfloat16).requires_grad_()

        self.experts, self.top = experts, top
        self.embedding = matrix(vocab, dim, 1.0)
        self.head_weight = matrix(vocab, dim, 0.02)
        self.router_weight = matrix(experts, dim, dim ** -0.5)
        self.up = [matrix(inner, dim, dim ** -0.5) for _ in range(experts)]
        self.down = [matrix(dim, inner, inner ** -0.5) for _ in range(experts)]
        self.router = dm.Router.create(max_tokens, top, experts)
        self.head = dm.Head.create(max_tokens, vocab, dim, max_top=max_top)
        # Muon for the matrices inside, AdamW for embedding and head
        self.matrices = [self.router_weight, *self.up, *self.down]
        self.muon = dm.Muon.create([tuple(p.shape) for p in self.matrices])
        self.momenta = [torch.zeros(p.shape, device="cuda") for p in self.matrices]
        self.others = [self.embedding, self.head_weight]
        self.moments = [(torch.zeros(p.shape, device="cuda"), torch.zeros(p.shape, device="cuda")) for p in self.others]
        self.steps = 0

    def hidden(self, tokens):
        x = self.embedding[tokens]
        probs = torch.softmax((x @ self.router_weight.T).float(), dim=1)
        weights, ids = probs.topk(self.top, dim=1)
        route = self.router.sort(ids)
        xs = Dispatch.apply(x, self.router, route)
        rows = [b - a for a, b in zip(route.offsets.tolist(), route.offsets[1:].tolist())]
        parts = torch.split(xs, rows)  # every assignment has an expert, so the rows add up
        ys = torch.cat([torch.nn.functional.silu(p @ u.T) @ d.T for p, u, d in zip(parts, self.up, self.down)])
        y = x + Combine.apply(ys, weights.contiguous(), self.router, route)
        y = y.float()
        return (y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def losses(self, tokens, targets, teacher=None, temperature=2.0):
        """Per-token losses; ``teacher`` = (top ids, top logits) for distillation."""
        h = self.hidden(tokens)
        if teacher is None:
            return Xent.apply(h, self.head_weight, self.head, targets)
        return Distill.apply(h, self.head_weight, self.head, *teacher, temperature)

    def step(self, lr=0.02, adamw_lr=3e-3):
        """Update every parameter from its gradient, and clear the gradients."""
        self.steps += 1
        stream = torch.cuda.current_stream().cuda_stream
        with torch.no_grad():
            self.muon.step(self.matrices, [p.grad if p.grad is not None else torch.zeros_like(p)
                                           for p in self.matrices], self.momenta, lr=lr)
            for p, (m, v) in zip(self.others, self.moments):
                dm.dmuon_adamw_flat(p.data_ptr(), p.grad.data_ptr(), m.data_ptr(), v.data_ptr(), p.numel(),
                                    lr=adamw_lr, weight_decay=0.0, step=self.steps, stream=stream)
        for p in (*self.matrices, *self.others):
            p.grad = None


def batches(vocab, tokens, seed=1):
    """Endless (token, next token) pairs of a fixed random map; every 16th target does not count."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    follow = torch.randint(0, vocab, (vocab,), generator=g, device="cuda")
    while True:
        x = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        y = follow[x].clone()
        y[::16] = -100
        yield x, y


def teacher_lists(y, vocab, top, seed=2):
    """A teacher that is fairly sure of y, and has other ideas of its own."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.randint(0, vocab, (y.numel(), top), generator=g, device="cuda")
    logits = torch.randn(y.numel(), top, generator=g, device="cuda")
    ids[:, 0], logits[:, 0] = y, 8.0   # y = -100: the entry is not in the list
    return ids, logits


def train(steps=60, distill=False, tokens=512, vocab=1000, log=print):
    model = Model(vocab=vocab, max_tokens=tokens)
    history = []
    for i, (x, y) in zip(range(steps), batches(vocab, tokens)):
        loss = model.losses(x, y, teacher_lists(y, vocab, 16) if distill else None)
        mean = loss.sum() / (y >= 0).sum()
        mean.backward()
        model.step()
        history.append(float(mean.detach()))
        if log and (i % 10 == 0 or i == steps - 1):
            log(f"step {i}: {'distillation' if distill else 'cross entropy'} {history[-1]:.4f}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--distill", action="store_true", help="learn from a teacher's top logits")
    a = ap.parse_args()
    train(a.steps, a.distill)
