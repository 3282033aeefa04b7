"""A small mixture-of-experts language model trained with every operator of the library.

    python -m matrix_optimizer_update_gb300.example_moe_lm [--steps N] [--distill | --policy] [--max-norm X]

One step: tokens -> embedding -> router -> ``Router`` sends rows to the experts
-> experts' products -> ``Router`` combines them -> head -> ``Head`` gives the
loss (cross entropy, or distillation from the stored top logits of a teacher)
and its gradients, without the logits. The experts' and the router's matrices
are updated by ``Muon``, embedding and head by AdamW (``dmuon_adamw_flat``),
after ``GradClip`` has clipped all gradients where a largest norm is given.

With ``--policy`` the model learns from what it generates: ``Experts`` and
``Head.logprobs`` give its likeliest next tokens, one of them is chosen by its
probability, and the gradient of the choice's log probability, weighted by whether
it was right, and of the entropy trains the model.

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
    def checked(ctx, *grads):
        if torch.is_grad_enabled():
            raise RuntimeError("the library's operators have no second derivatives")
        return backward(ctx, *grads)

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


class Logprob(torch.autograd.Function):
    """Each token's log probability of its target, and the entropy, without the logits."""

    @staticmethod
    def forward(ctx, hidden, weight, head, targets):
        scores = head.logprobs(hidden, weight, targets)
        ctx.head = head
        ctx.save_for_backward(hidden, weight, targets, scores.logp, scores.entropy, scores.lse)
        return scores.logp, scores.entropy

    @staticmethod
    @first_derivative
    def backward(ctx, grad_logp, grad_entropy):
        hidden, weight, targets, *scores = ctx.saved_tensors
        scores = dm.Logprobs(*scores, None, None)
        return (*ctx.head.logprobs_backward(hidden, weight, targets, scores, grad_logp.contiguous(),
                                            grad_entropy.contiguous()), None, None)


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
        # the experts' matrices side by side, as Experts reads them; each is a parameter of its own for training
        self.ups = torch.stack([matrix(inner, dim, dim ** -0.5).detach() for _ in range(experts)])
        self.downs = torch.stack([matrix(dim, inner, inner ** -0.5).detach() for _ in range(experts)])
        self.up = [m.detach().requires_grad_() for m in self.ups]
        self.down = [m.detach().requires_grad_() for m in self.downs]
        # made for few tokens: at most 2048 assignments a call
        self.layer = dm.Experts.create(min(max_tokens, 2048 // top), top, experts, dim, inner)
        self.clip = dm.GradClip.create()
        self.router = dm.Router.create(max_tokens, top, experts)
        self.head = dm.Head.create(max_tokens, vocab, dim, max_top=max_top)
        # Muon for the matrices inside, AdamW for embedding and head
        self.matrices = [self.router_weight, *self.up, *self.down]
        self.muon = dm.Muon.create([tuple(p.shape) for p in self.matrices])
        self.momenta = [torch.zeros(p.shape, device="cuda") for p in self.matrices]
        self.others = [self.embedding, self.head_weight]
        self.moments = [(torch.zeros(p.shape, device="cuda"), torch.zeros(p.shape, device="cuda")) for p in self.others]
        self.steps = 0

    def routing(self, x):
        probs = torch.softmax((x @ self.router_weight.T).float(), dim=1)
        return probs.topk(self.top, dim=1)

    @staticmethod
    def norm(y):
        y = y.float()
        return (y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def hidden(self, tokens):
        x = self.embedding[tokens]
        weights, ids = self.routing(x)
        route = self.router.sort(ids)
        xs = Dispatch.apply(x, self.router, route)
        rows = [b - a for a, b in zip(route.offsets.tolist(), route.offsets[1:].tolist())]
        parts = torch.split(xs, rows)  # every assignment has an expert, so the rows add up
        ys = torch.cat([torch.nn.functional.silu(p @ u.T) @ d.T for p, u, d in zip(parts, self.up, self.down)])
        return self.norm(x + Combine.apply(ys, weights.contiguous(), self.router, route))

    @torch.no_grad()
    def serve(self, tokens):
        """The hidden states of tokens that are generated: nothing is read back to the host, and it can be captured."""
        x = self.embedding[tokens]
        weights, ids = self.routing(x)
        parts = zip(*(t.split(self.layer.max_tokens) for t in (x, ids, weights.contiguous())))
        return self.norm(x + torch.cat([self.layer.forward(*part, self.ups, self.downs) for part in parts]))

    @torch.no_grad()
    def choose(self, tokens, top=16, generator=None):
        """A next token for each token, one of the ``top`` likeliest by its probability among them; anything, or -1,
        where the logits are not finite."""
        scores = self.head.logprobs(self.serve(tokens), self.head_weight, top=top)
        # (torch ends the process on probabilities that are no numbers or all zeros)
        pick = torch.multinomial(scores.top_logp.exp().nan_to_num(0.0, 0.0, 0.0) + 1e-30, 1, generator=generator)
        return scores.top_ids.gather(1, pick)[:, 0]

    def losses(self, tokens, targets, teacher=None, temperature=2.0):
        """Per-token losses; ``teacher`` = (top ids, top logits) for distillation."""
        h = self.hidden(tokens)
        if teacher is None:
            return Xent.apply(h, self.head_weight, self.head, targets)
        return Distill.apply(h, self.head_weight, self.head, *teacher, temperature)

    def policy(self, tokens, chosen):
        """Per-token log probabilities of chosen next tokens, and entropies."""
        return Logprob.apply(self.hidden(tokens), self.head_weight, self.head, chosen)

    def step(self, lr=0.02, adamw_lr=3e-3, max_norm=None):
        """Update every parameter from its gradient, and clear the gradients. With ``max_norm`` they are clipped to it
        first; returns their norm before that then."""
        self.steps += 1
        stream = torch.cuda.current_stream().cuda_stream
        norm = None
        with torch.no_grad():
            if max_norm is not None:
                norm = self.clip.clip([p.grad for p in (*self.matrices, *self.others) if p.grad is not None], max_norm)
            self.muon.step(self.matrices, [p.grad if p.grad is not None else torch.zeros_like(p)
                                           for p in self.matrices], self.momenta, lr=lr)
            for p, (m, v) in zip(self.others, self.moments):
                dm.dmuon_adamw_flat(p.data_ptr(), p.grad.data_ptr(), m.data_ptr(), v.data_ptr(), p.numel(),
                                    lr=adamw_lr, weight_decay=0.0, step=self.steps, stream=stream)
        for p in (*self.matrices, *self.others):
            p.grad = None
        return norm


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


def policy_loss(logp, entropy, right, counts, bonus):
    """The loss whose gradient makes choices that were right more likely, by how much better they did than the tokens
    that count did on average, with a bonus for entropy; and that average."""
    n = counts.sum().clamp(min=1)
    right = (right & counts).float()
    average = right.sum() / n
    advantage = torch.where(counts, right - average, 0.0)
    return -(advantage * logp + bonus * torch.where(counts, entropy, 0.0)).sum() / n, average


def reinforce(steps=60, tokens=512, vocab=1000, warm=15, bonus=0.01, max_norm=1.0, log=print):
    """Learn from the model's own choices, after ``warm`` steps of cross entropy that make some of them right; returns
    what part of those that count were, step by step."""
    model = Model(vocab=vocab, max_tokens=tokens)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    history = []
    data = batches(vocab, tokens)
    for _, (x, y) in zip(range(warm), data):
        (model.losses(x, y).sum() / (y >= 0).sum()).backward()
        model.step(max_norm=max_norm)
    for i, (x, y) in zip(range(steps), data):
        counts = y >= 0
        chosen = model.choose(x, generator=g)
        chosen = torch.where(counts, chosen, y)  # tokens that do not count have no choice
        logp, entropy = model.policy(x, chosen)
        loss, average = policy_loss(logp, entropy, chosen == y, counts, bonus)
        loss.backward()
        norm = model.step(max_norm=max_norm)
        history.append(float(average))
        if log and (i % 10 == 0 or i == steps - 1):
            log(f"step {i}: {100 * history[-1]:.1f} % right, entropy {float(entropy.detach()[counts].mean()):.2f}, "
                f"gradient norm {float(norm):.3f}")
    return history


def train(steps=60, distill=False, tokens=512, vocab=1000, max_norm=None, log=print):
    model = Model(vocab=vocab, max_tokens=tokens)
    history = []
    for i, (x, y) in zip(range(steps), batches(vocab, tokens)):
        loss = model.losses(x, y, teacher_lists(y, vocab, 16) if distill else None)
        mean = loss.sum() / (y >= 0).sum()
        mean.backward()
        model.step(max_norm=max_norm)
        history.append(float(mean.detach()))
        if log and (i % 10 == 0 or i == steps - 1):
            log(f"step {i}: {'distillation' if distill else 'cross entropy'} {history[-1]:.4f}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    how = ap.add_mutually_exclusive_group()
    how.add_argument("--distill", action="store_true", help="learn from a teacher's top logits")
    how.add_argument("--policy", action="store_true", help="learn from the model's own choices")
    ap.add_argument("--max-norm", type=float, default=None, help="clip the gradients to this norm")
    a = ap.parse_args()
    if a.policy:
        reinforce(a.steps, max_norm=1.0 if a.max_norm is None else a.max_norm)
    else:
        train(a.steps, a.distill, max_norm=a.max_norm)
