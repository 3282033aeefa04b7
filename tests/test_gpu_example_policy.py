"""The example's generating and learning from it: the serving form agrees with the training form, the gradients are
those of the same formulas in plain torch, and the steps run."""

import pytest
import torch

from matrix_optimizer_update_gb300 import example_moe_lm as ex

pytestmark = pytest.mark.gpu


def small(tokens=200):
    return ex.Model(vocab=300, dim=64, inner=96, experts=4, top=2, max_tokens=tokens)


def test_serving_is_the_training_forward_pass():
    model = small()
    x, _ = next(ex.batches(300, 200))
    with torch.no_grad():
        want = model.hidden(x).float()
        got = model.serve(x).float()
    # both round x + y and the norm to bf16, the training form also u, h and each expert's rows: six roundings of 2^-8
    assert torch.linalg.norm(got - want) <= 6 * 2.0 ** -8 * torch.linalg.norm(want)


def test_choices_are_among_the_likeliest():
    model = small()
    x, _ = next(ex.batches(300, 200))
    with torch.no_grad():
        z = model.serve(x).double() @ model.head_weight.double().T
    best = z.sort(dim=1, descending=True, stable=True).indices[:, :5]
    assert torch.equal(model.choose(x, top=1), best[:, 0])
    for _ in range(3):
        assert bool((model.choose(x, top=5)[:, None] == best).any(1).all())


def test_generating_captured():
    model = small(5)
    x = torch.randint(0, 300, (5,), device="cuda")
    model.head.logprobs(model.serve(x), model.head_weight, top=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scores = model.head.logprobs(model.serve(x), model.head_weight, top=4)
    for _ in range(3):
        x.copy_(torch.randint(0, 300, (5,), device="cuda"))
        graph.replay()
        want = model.head.logprobs(model.serve(x), model.head_weight, top=4)
        assert torch.equal(scores.top_ids, want.top_ids) and torch.equal(scores.top_logp, want.top_logp)


def test_policy_gradients_are_those_of_plain_torch():
    model = small()
    x, y = next(ex.batches(300, 200))
    logp, entropy = model.policy(x, y)
    weight = torch.linspace(-1, 1, 200, device="cuda")
    (weight * logp + 0.3 * entropy).sum().backward()
    w = {n: getattr(model, n).detach().float().requires_grad_() for n in ("embedding", "head_weight", "router_weight")}
    up = [p.detach().float().requires_grad_() for p in model.up]
    down = [p.detach().float().requires_grad_() for p in model.down]
    h = w["embedding"][x]
    with torch.no_grad():
        ids = torch.softmax((model.embedding[x] @ model.router_weight.T).float(), 1).topk(2, dim=1).indices
    probs = torch.softmax(h @ w["router_weight"].T, 1)
    every = torch.stack([torch.nn.functional.silu(h @ u.T) @ d.T for u, d in zip(up, down)], 1)
    mix = torch.zeros(200, 4, device="cuda").scatter(1, ids, probs.gather(1, ids))
    out = h + (every * mix[:, :, None]).sum(1)
    out = out * torch.rsqrt(out.square().mean(1, keepdim=True) + 1e-6)
    every = torch.log_softmax(out @ w["head_weight"].T, 1)
    chosen = torch.where(y >= 0, every.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0)
    (weight * chosen - 0.3 * (every.exp() * every).sum(1)).sum().backward()
    pairs = [(getattr(model, n), w[n]) for n in w] + list(zip(model.up, up)) + list(zip(model.down, down))
    for got, want in pairs:
        # about ten roundings to bf16 (2^-8 each) between loss and weight, independent of each other
        off = torch.linalg.norm(got.grad.float() - want.grad) / torch.linalg.norm(want.grad)
        assert off < 10 * 2.0 ** -8


def test_steps_run_and_clip():
    assert all(0.0 <= r <= 1.0 for r in ex.reinforce(steps=4, tokens=64, vocab=100, log=None))
    assert all(h == h for h in ex.train(steps=3, tokens=64, vocab=100, max_norm=0.1, log=None))
    model = small()
    x, y = next(ex.batches(300, 200))
    model.losses(x, y).sum().backward()
    params = [*model.matrices, *model.others]
    want = sum(float(p.grad.double().square().sum()) for p in params) ** 0.5
    grads = [p.grad for p in params]
    norm = model.step(max_norm=want / 8)
    assert abs(float(norm) - want) < 1e-5 * want
    after = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    assert abs(after - want / 8) < 2.0 ** -8 * want / 8
    assert all(p.grad is None for p in params)
