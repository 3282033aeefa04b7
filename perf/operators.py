"""Measured cases of the operators a training step runs around the optimizer.

Three operators: the softmax cross entropy of a language model's head, in
pieces of the vocabulary and with its gradient; the distillation loss of the
same head from a teacher's top logits, with its gradient; and the routing of
tokens to experts and back, with the router's weights and its gradient.

``run`` computes them either with elementary torch operations in 32 bits
(``own`` false) or through the framework's calls (``own`` true).
"""

import math

import torch

own = False

IGNORE = -100


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the head's cross entropy. One token scored against a 32000-entry vocabulary: latency, and the
        # time to read the head's weight once.
        dict(name="xent score 1 token", op="xent", backward=False, tokens=1, vocab=32000, dim=2048, masked=0.0),
        # a short fine-tuning batch, most of it prompt (ignored), with an odd vocabulary and odd length
        dict(name="xent train 77 tokens", op="xent", backward=True, tokens=77, vocab=50257, dim=1024, masked=0.6),
        # a micro-batch on the hidden size of the MoE matrix set
        dict(name="xent train 2048 tokens", op="xent", backward=True, tokens=2048, vocab=32000, dim=2048, masked=0.1),
        # perplexity over two packed sequences of 4096, a few tokens short
        dict(name="xent score 8189 tokens", op="xent", backward=False, tokens=8189, vocab=128000, dim=4096,
             masked=0.0),
        # one sequence of 4096 tokens on the largest matrix set's hidden size: the largest case
        dict(name="xent train 4096 tokens", op="xent", backward=True, tokens=4096, vocab=128000, dim=4096,
             masked=0.1),
        # distillation. A handful of tokens and eight teacher logits each
        dict(name="distill 16 tokens", op="distill", tokens=16, vocab=32000, dim=1536, top=8, temperature=1.0,
             masked=0.2),
        # a micro-batch with 64 teacher logits stored per token, an odd vocabulary and an odd length
        dict(name="distill 1999 tokens", op="distill", tokens=1999, vocab=50257, dim=2048, top=64, temperature=2.0,
             masked=0.1),
        # a sequence of 4096 tokens with 128 teacher logits each
        dict(name="distill 4096 tokens", op="distill", tokens=4096, vocab=128000, dim=2048, top=128,
             temperature=1.5, masked=0.05),
        # routing to experts. One token to 8 of the MoE set's 64 experts: latency
        dict(name="route 1 token", op="route", backward=False, tokens=1, top=8, experts=64, dim=2048, dtype="bf16",
             dropped=0.0),
        # a chunk of a prompt, odd length, some assignments dropped at the experts' capacity
        dict(name="route 1021 tokens", op="route", backward=False, tokens=1021, top=6, experts=64, dim=2048,
             dtype="bf16", dropped=0.05),
        # a training micro-batch in 32 bits
        dict(name="route train 4096 f32", op="route", backward=True, tokens=4096, top=8, experts=64, dim=2048,
             dtype="f32", dropped=0.0),
        # a training batch of four sequences of 4096 tokens
        dict(name="route train 16384", op="route", backward=True, tokens=16384, top=8, experts=128, dim=4096,
             dtype="bf16", dropped=0.02),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent", "distill", "route", "route"])
    if op == "route":
        case = dict(op="route", backward=rng.random() < 0.6, tokens=_between(rng, 1, 16384), top=rng.randint(1, 8),
                    experts=_between(rng, 8, 256), dim=8 * _between(rng, 32, 512), dtype=rng.choice(["bf16", "f32"]),
                    dropped=rng.choice([0.0, 0.02, 0.1]))
        if case["dtype"] == "f32" and case["backward"]:
            case["tokens"] = min(case["tokens"], 8192 - rng.randint(0, 300))
        return case
    while True:
        tokens, vocab, dim = _between(rng, 1, 8192), _between(rng, 8000, 128000), 8 * _between(rng, 32, 512)
        backward = op == "distill" or rng.random() < 0.6
        if (6 if backward else 2) * tokens * vocab * dim <= 6 * 4096 * 128000 * 4096:
            break
    masked = rng.choice([0.0, 0.1, 0.5])
    if op == "xent":
        return dict(op="xent", backward=backward, tokens=tokens, vocab=vocab, dim=dim, masked=masked)
    return dict(op="distill", tokens=tokens, vocab=vocab, dim=dim, top=_between(rng, 1, 128),
                temperature=rng.choice([1.0, 1.5, 2.0, 4.0]), masked=masked)


def work(case):
    t, d = case["tokens"], case["dim"]
    if case["op"] == "route":
        e = 2 if case["dtype"] == "bf16" else 4
        n = t * case["top"]
        rows = (t * d + n * d) * e          # a row per token on one side, a row per assignment on the other
        bytes_ = n * 8 + 2 * n * 4 + (case["experts"] + 1) * 4 + 2 * rows + n * 4
        flops = 2 * n * d
        if case["backward"]:
            bytes_ += rows + n * d * e + n * 4 + rows  # dy, ys -> dys, dweights; dxs -> dx
            flops += 3 * n * d + n * d
        return {"bytes": bytes_, "flops": flops}
    v = case["vocab"]
    backward = case.get("backward", True)
    ids = t * 8 if case["op"] == "xent" else t * case["top"] * 12
    bytes_ = 2 * (t * d + v * d) + ids + t * 8
    flops = 2 * t * v * d
    if backward:
        bytes_ += 2 * (t * d + v * d) + t * 4
        flops *= 3
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _frequent(shape, vocab, g):
    """Token ids with the frequencies of text: the n-th most frequent about 1/n of the time."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)


def _head_inputs(case, g):
    """Hidden states after a final norm, a head weight, and tokens that the model predicts with
    anything from no to full confidence."""
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    weight = (torch.randn(v, d, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    targets = _frequent((t,), v, g)
    hidden = torch.randn(t, d, generator=g, device="cuda")
    row = weight[targets].float()
    sure = 16.0 * torch.rand(t, 1, generator=g, device="cuda")
    hidden += row * (sure / row.square().sum(1, keepdim=True))
    return hidden.to(torch.bfloat16), weight, targets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "route":
        t, k, e, d = case["tokens"], case["top"], case["experts"], case["dim"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a router whose experts are not equally liked
        score = torch.randn(t, e, generator=g, device="cuda") + torch.randn(1, e, generator=g, device="cuda")
        top = score.topk(k, dim=1)
        ids = top.indices
        weights = torch.softmax(top.values, dim=1)
        if case["dropped"]:
            ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < case["dropped"], -1, ids)
        n = t * k
        s.update(ids=ids, weights=weights,
                 x=torch.randn(t, d, generator=g, device="cuda").to(dtype),
                 ys=torch.randn(n, d, generator=g, device="cuda").to(dtype))
        if case["backward"]:
            s.update(dy=(torch.randn(t, d, generator=g, device="cuda") * 1e-2).to(dtype),
                     dxs=(torch.randn(n, d, generator=g, device="cuda") * 1e-2).to(dtype))
    else:
        hidden, weight, targets = _head_inputs(case, g)
        t, v = case["tokens"], case["vocab"]
        masked = torch.rand(t, generator=g, device="cuda") < case["masked"]
        s.update(hidden=hidden, weight=weight)
        if case["op"] == "xent":
            s["targets"] = torch.where(masked, IGNORE, targets)
        else:
            # a teacher that likes the same token best, then a falling list of distinct others; some
            # tokens have fewer entries than the list holds (-inf, id -1), masked ones have none
            k = case["top"]
            place = torch.arange(k, device="cuda")
            ids = torch.sort(_frequent((t, k), v, g), dim=1).values - place
            ids = (torch.cummax(ids, dim=1).values + place).minimum(v - k + place)
            order = torch.argsort(torch.rand(t, k, generator=g, device="cuda"), dim=1, stable=True)
            ids = torch.gather(ids, 1, order)
            seen = (ids == targets[:, None]).any(1)
            ids[:, 0] = torch.where(seen, ids[:, 0], targets)
            fall = torch.rand(t, k, generator=g, device="cuda") * (8.0 / k)
            logits = 14.0 - torch.cumsum(fall, dim=1) - 2.0 * torch.log1p(place.float())
            kept = 1 + (torch.rand(t, 1, generator=g, device="cuda") * 1.5 * k).long()
            gone = (place[None, :] >= kept) | masked[:, None]
            s.update(top_ids=torch.where(gone, -1, ids), top_logits=torch.where(gone, -math.inf, logits))
        if case.get("backward", True):
            # the gradient of the mean over the tokens that count
            s["grad"] = torch.where(masked, 0.0, 1.0) / (~masked).sum().clamp(min=1)
    if own:
        from matrix_optimizer_update_gb300 import dmuon as dm
        if case["op"] == "route":
            s["router"] = dm.Router.create(case["tokens"], case["top"], case["experts"])
        else:
            s["head"] = dm.Head.create(case["tokens"], case["vocab"], case["dim"], max_top=case.get("top", 0))
    return s


# --------------------------------------------------------------------------
# the plain forms and the framework's calls
# --------------------------------------------------------------------------

def run(s):
    return {"xent": _xent, "distill": _distill, "route": _route}[s["op"]](s)


def _xent(s):
    h, w, y = s["hidden"], s["weight"], s["targets"]
    if own:
        head = s["head"]
        loss, lse = head.xent(h, w, y)
        if not s["backward"]:
            return {"loss": loss, "lse": lse}
        dh, dw = head.xent_backward(h, w, y, lse, s["grad"])
        return {"loss": loss, "lse": lse, "dhidden": dh, "dweight": dw}
    hf, wf = h.float(), w.float()
    z = hf @ wf.T
    counts = (y >= 0) & (y < w.shape[0])
    at = torch.where(counts, y, 0)[:, None]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    # the target's share apart from the others': the loss of a sure token is small beside its logits
    hit = e.gather(1, at)
    others = e.scatter(1, at, torch.where(counts[:, None], 0.0, hit)).sum(1, keepdim=True)
    total = others + torch.where(counts[:, None], hit, 0.0)
    lse = (top + torch.log(total))[:, 0]
    far = lse - z.gather(1, at)[:, 0]
    loss = torch.where(counts, torch.where(hit > others, torch.log1p(others / hit), far[:, None])[:, 0], 0.0)
    if not s["backward"]:
        return {"loss": loss, "lse": lse}
    g = torch.where(counts, s["grad"], 0.0)[:, None]
    dz = e * (g / total)
    dz.scatter_add_(1, at, -g)
    return {"loss": loss, "lse": lse, "dhidden": (dz @ wf).to(h.dtype), "dweight": (dz.T @ hf).to(w.dtype)}


def _distill(s):
    h, w, ids, tau = s["hidden"], s["weight"], s["top_ids"], s["temperature"]
    if own:
        head = s["head"]
        loss, lse = head.distill(h, w, ids, s["top_logits"], tau)
        dh, dw = head.distill_backward(h, w, ids, s["top_logits"], tau, lse, s["grad"])
        return {"loss": loss, "lse": lse, "dhidden": dh, "dweight": dw}
    hf, wf = h.float(), w.float()
    given = (ids >= 0) & (ids < w.shape[0])
    at = torch.where(given, ids, 0)
    t = torch.where(given, s["top_logits"].float(), -math.inf)
    best = t.amax(1, keepdim=True)
    q = torch.exp((t - torch.where(best == -math.inf, 0.0, best)) / tau)
    mass = q.sum(1, keepdim=True)
    some = mass > 0
    q = torch.where(some, q / mass, 0.0)
    z = (hf @ wf.T) / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    # the listed entries' share apart from the others', as the loss may be small beside the logits
    on = q > 0
    zt = z.gather(1, at)
    peak = torch.where(on, zt, -math.inf).amax(1, keepdim=True)
    peak = torch.where(some, peak, top)
    hit = torch.where(on, torch.exp(zt - peak), 0.0).sum(1, keepdim=True)
    listed_too = torch.zeros_like(e).scatter_add_(1, at, on.float()) > 0
    others = torch.where(listed_too, 0.0, e).sum(1, keepdim=True)
    total = others + hit * torch.exp(peak - top)
    lse = top + torch.log(total)
    lse_hit = torch.where(some, peak + torch.log(hit), lse)
    ratio = others / hit * torch.exp(top - peak)
    rest = torch.where(ratio < 1, torch.log1p(ratio), lse - lse_hit)
    kl = (q * (torch.log(torch.where(on, q, 1.0)) - zt + lse_hit)).sum(1) + torch.where(some, rest, 0.0)[:, 0]
    g = torch.where(some[:, 0], s["grad"] * tau, 0.0)[:, None]
    dz = e * (g / total)
    dz.scatter_add_(1, at, -g * q)
    return {"loss": kl * (tau * tau), "lse": lse[:, 0], "dhidden": (dz @ wf).to(h.dtype),
            "dweight": (dz.T @ hf).to(w.dtype)}


def _route(s):
    x, ids, weights, ys = s["x"], s["ids"], s["weights"], s["ys"]
    t, k = ids.shape
    if own:
        router = s["router"]
        route = router.sort(ids)
        xs = router.dispatch(x, route)
        y = router.combine(ys, weights, route)
        out = {"dest": route.dest, "source": route.source, "offsets": route.offsets, "xs": xs, "y": y}
        if s["backward"]:
            out["dys"], out["dweights"] = router.combine_backward(s["dy"], ys, weights, route)
            out["dx"] = router.dispatch_backward(s["dxs"], route)
        return out
    n, experts = t * k, s["experts"]
    flat = ids.reshape(n)
    kept = (flat >= 0) & (flat < experts)
    key = torch.where(kept, flat, experts)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(0)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = torch.cumsum(counts, 0)
    dest = torch.empty_like(order)
    dest[order] = torch.arange(n, device=key.device)
    dest = torch.where(kept, dest, -1)
    live = (torch.arange(n, device=key.device) < offsets[experts])[:, None]
    xs = torch.where(live, x[order // k], 0.0)
    at = dest.clamp(min=0)
    on = kept.reshape(t, k, 1)
    rows = torch.where(on, ys[at].float().reshape(t, k, -1), 0.0)
    y = (rows * weights[:, :, None]).sum(1)
    out = {"dest": dest.reshape(t, k).int(), "source": torch.where(live[:, 0], order, -1).int(),
           "offsets": offsets.int(), "xs": xs, "y": y.to(x.dtype)}
    if s["backward"]:
        dyf = s["dy"].float()
        w = weights.reshape(n)[order][:, None]
        out["dys"] = torch.where(live, dyf[order // k] * w, 0.0).to(x.dtype)
        out["dweights"] = (rows * dyf[:, None, :]).sum(2)
        back = torch.where(on, s["dxs"][at].float().reshape(t, k, -1), 0.0)
        out["dx"] = back.sum(1).to(x.dtype)
    return out


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    t, v = case["tokens"], case["vocab"]
    backward = case.get("backward", True)
    if (6 if backward else 2) * t * v * case["dim"] > 1.6e13:
        return None
    h, w = s["hidden"].double(), s["weight"].double()
    tau = float(case.get("temperature", 1.0))
    loss, lse = torch.zeros(t, dtype=torch.float64, device="cuda"), torch.zeros(t, dtype=torch.float64, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros_like(w) if backward else None
    for a in range(0, t, 1024):
        b = min(a + 1024, t)
        logp = torch.log_softmax(h[a:b] @ w.T / tau, dim=1)
        lse[a:b] = (h[a:b] * w[0]).sum(1) / tau - logp[:, 0]
        # the wanted distribution, spread over the vocabulary
        want = torch.zeros_like(logp)
        if case["op"] == "xent":
            y = s["targets"][a:b]
            rows = torch.nonzero(y != IGNORE)[:, 0]
            want[rows, y[rows]] = 1.0
        else:
            rows, slot = torch.nonzero(torch.isfinite(s["top_logits"][a:b]), as_tuple=True)
            q = torch.softmax(s["top_logits"][a:b].double() / tau, dim=1)
            want[rows, s["top_ids"][a:b][rows, slot]] = q[rows, slot]
        entropy = torch.special.entr(want).sum(1)
        loss[a:b] = tau * tau * (-(want * logp).sum(1) - entropy)
        if backward:
            on = want.sum(1, keepdim=True)
            dz = (logp.exp() * on - want) * (s["grad"][a:b, None].double() * tau)
            dh[a:b] = dz @ w
            dw += dz.T @ h[a:b]
    out = {"loss": loss, "lse": lse}
    if backward:
        out.update(dhidden=dh, dweight=dw)
    return out


def _exact_route(s):
    t, k = s["ids"].shape
    d = s["x"].shape[1]
    out = {"dest": None, "source": None, "offsets": None}
    # where each assignment's row lies: those of smaller experts, then earlier ones of its own
    ids = s["ids"].reshape(-1).tolist()
    start, where = [0] * (s["experts"] + 1), []
    for e in ids:
        if e >= 0:
            start[e + 1] += 1
    for e in range(s["experts"]):
        start[e + 1] += start[e]
    for e in ids:
        where.append(start[e] if e >= 0 else -1)
        if e >= 0:
            start[e] += 1
    where = torch.tensor(where, device="cuda").reshape(t, k)
    y = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    xs = torch.zeros(t * k, d, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(y), torch.zeros(t, k, dtype=torch.float64, device="cuda")
    dys = torch.zeros(t * k, d, dtype=torch.float64, device="cuda") if s["backward"] else None
    for j in range(k):
        on = torch.nonzero(where[:, j] >= 0)[:, 0]
        at = where[on, j]
        w = s["weights"][on, j, None].double()
        xs[at] = s["x"][on].double()
        y[on] += w * s["ys"][at].double()
        if s["backward"]:
            dy = s["dy"][on].double()
            dys[at] = w * dy
            dw[on, j] = (dy * s["ys"][at].double()).sum(1)
            dx[on] += s["dxs"][at].double()
    out.update(xs=xs, y=y)
    if s["backward"]:
        out.update(dys=dys, dweights=dw, dx=dx)
    return out
