"""Measured cases of the operators a language model generates with, and learns from what it generated.

Three operators: a mixture's experts for a few tokens, from the router's ids and
weights to the layer's output; the log probabilities of given tokens at the head,
with the entropy, the top alternatives and the gradients; and the global norm of
many gradient tensors, with their clipping.

``run`` computes them either with elementary torch operations in 32 bits
(``own`` false) or through the framework's calls (``own`` true).
"""

import math

import torch

own = False

IGNORE = -100

# The 2-D matrices and the norm's vectors of one layer, as clipping gets them: of the Qwen2.5-1.5B-shaped
# set, and of the mixture-of-experts set (attention; one expert).
DENSE_LAYER = "1536x1536 256x1536 256x1536 1536x1536 8960x1536 8960x1536 1536x8960 1536 1536"
MOE_ATTENTION = "2048x2048 512x2048 512x2048 2048x2048 2048 2048 64x2048"
MOE_EXPERT = "1408x2048 1408x2048 2048x1408"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # a mixture's experts. One token of a generation to 8 of the MoE set's 64 experts: latency, and the time
        # to read eight experts' matrices
        dict(name="experts 1 token", op="experts", tokens=1, top=8, experts=64, dim=2048, inner=1408, gated=True,
             dropped=0.0),
        # seven generations at once, of a layer with large experts without a gate
        dict(name="experts 7 ungated", op="experts", tokens=7, top=2, experts=8, dim=1536, inner=8960, gated=False,
             dropped=0.0),
        # an odd number of generations, some assignments dropped, sizes that are no multiples of a tile
        dict(name="experts 33 odd", op="experts", tokens=33, top=6, experts=60, dim=2056, inner=1000, gated=True,
             dropped=0.05),
        # 64 generations at once: nearly every expert's matrices are read
        dict(name="experts 64 tokens", op="experts", tokens=64, top=8, experts=64, dim=2048, inner=1408, gated=True,
             dropped=0.0),
        # log probabilities. One generated token with five alternatives: latency, and the time to read the head
        dict(name="logprobs 1 token", op="logprobs", backward=False, tokens=1, vocab=32000, dim=2048, top=5,
             temperature=1.0, masked=0.0),
        # a short answer scored, with twenty alternatives, an odd vocabulary and an odd length
        dict(name="logprobs 61 tokens", op="logprobs", backward=False, tokens=61, vocab=50257, dim=1024, top=20,
             temperature=0.8, masked=0.2),
        # a sequence of 4096 tokens, three short, scored with twenty alternatives: the largest case
        dict(name="logprobs 4093 tokens", op="logprobs", backward=False, tokens=4093, vocab=128000, dim=4096, top=20,
             temperature=1.0, masked=0.1),
        # a policy's gradient from a short answer behind a prompt, with a bonus for entropy
        dict(name="policy 77 tokens", op="logprobs", backward=True, tokens=77, vocab=50257, dim=1024, top=0,
             temperature=1.0, masked=0.6, bonus=0.01),
        # ... from a micro-batch on the hidden size of the MoE matrix set
        dict(name="policy 2048 tokens", op="logprobs", backward=True, tokens=2048, vocab=32000, dim=2048, top=0,
             temperature=1.0, masked=0.1, bonus=0.01),
        # clipping. The four small fp32 matrices of the toy set: latency
        dict(name="clip 4 small f32", op="clip", sizes="4*128x256", dtype="f32", clip=True, over=3.0),
        # the norm alone, of a layer of the MoE set with its vectors: 199 tensors, matrices in bf16 and vectors in fp32
        dict(name="norm 199 mixed", op="clip", sizes=f"1*{MOE_ATTENTION} 64*{MOE_EXPERT}", dtype="mixed", clip=False,
             over=1.0),
        # every gradient of a 1.5B-parameter model's layers, clipped
        dict(name="clip 252 bf16", op="clip", sizes=f"28*{DENSE_LAYER}", dtype="bf16", clip=True, over=2.7),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "logprobs", "logprobs", "logprobs", "clip"])
    if op == "experts":
        experts = _between(rng, 4, 128)
        top = rng.randint(1, min(8, experts))
        tokens = _between(rng, 1, 64)
        dim, inner = 8 * _between(rng, 32, 512), 8 * _between(rng, 32, 1120)
        while max(experts, tokens * top) * dim * inner > 1.4e9:
            dim, inner = 8 * _between(rng, 32, 512), 8 * _between(rng, 32, 1120)
        return dict(op="experts", tokens=tokens, top=top, experts=experts, dim=dim, inner=inner,
                    gated=rng.random() < 0.7, dropped=rng.choice([0.0, 0.0, 0.1]))
    if op == "logprobs":
        backward = rng.random() < 0.4
        while True:
            tokens, vocab, dim = _between(rng, 1, 4096), _between(rng, 8000, 128000), 8 * _between(rng, 32, 512)
            if (4 if backward else 1) * tokens * vocab * dim <= 4093 * 128000 * 4096:
                break
        case = dict(op="logprobs", backward=backward, tokens=tokens, vocab=vocab, dim=dim,
                    top=0 if backward else rng.choice([0, 1, 5, 20, 32]),
                    temperature=rng.choice([1.0, 0.7, 1.3]), masked=rng.choice([0.0, 0.1, 0.5]))
        if backward:
            case["bonus"] = rng.choice([0.0, 0.01, 0.3])
        return case
    sizes = []
    for _ in range(rng.randint(1, 4)):
        rows, cols = _between(rng, 1, 6000), _between(rng, 8, 6000)
        sizes.append(f"{_between(rng, 1, 40)}*{rows}x{cols} {_between(rng, 1, 5000)}")
    return dict(op="clip", sizes=" ".join(sizes), dtype=rng.choice(["bf16", "f32", "mixed"]), clip=rng.random() < 0.6,
                over=rng.choice([0.7, 2.7, 30.0]))


def _shapes(sizes):
    """'2*3x4 5 1*7' -> [(3, 4), (5,), (3, 4), (5,), (7,)]: a count starts a group that is repeated."""
    out, group, times = [], [], 1
    for word in sizes.split():
        if "*" in word:
            out += group * times
            count, word = word.split("*")
            group, times = [], int(count)
        group.append(tuple(int(n) for n in word.split("x")))
    return out + group * times


def _kinds(case):
    """Each tensor's shape and whether it is bf16: of mixed sets the matrices are, the vectors fp32."""
    return [(s, case["dtype"] == "bf16" or (case["dtype"] == "mixed" and len(s) > 1)) for s in _shapes(case["sizes"])]


def work(case):
    if case["op"] == "clip":
        kinds = _kinds(case)
        elements = sum(math.prod(s) for s, _ in kinds)
        bytes_ = sum(math.prod(s) * (2 if b else 4) for s, b in kinds)
        if not case["clip"]:
            return {"bytes": bytes_ + 4, "flops": 2 * elements}
        return {"bytes": 2 * bytes_ + 4, "flops": 3 * elements}
    t, d = case["tokens"], case["dim"]
    if case["op"] == "experts":
        # the experts that so many assignments are expected to reach, each token's being different
        e, k = case["experts"], case["top"]
        reached = e * (1.0 - (1.0 - k / e) ** t)
        each = (3 if case["gated"] else 2) * d * case["inner"]
        return {"bytes": int(2 * reached * each) + 4 * t * d + 12 * t * k, "flops": 2 * t * k * each}
    v = case["vocab"]
    bytes_ = 2 * (t * d + v * d) + 8 * t + 12 * t + 12 * t * case["top"]
    flops = 2 * t * v * d
    if case["backward"]:
        bytes_ += 2 * (t * d + v * d) + 8 * t
        flops *= 3
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(shape, std, g, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _head_inputs(case, g):
    """Hidden states after a final norm, a head weight, and tokens that the model predicts with anything from
    no to full confidence; the n-th most frequent token is met about 1/n of the time."""
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    weight = _normal((v, d), 0.02, g)
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    targets = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    hidden = torch.randn(t, d, generator=g, device="cuda")
    row = weight[targets].float()
    sure = 16.0 * torch.rand(t, 1, generator=g, device="cuda")
    hidden += row * (sure / row.square().sum(1, keepdim=True))
    return hidden.to(torch.bfloat16), weight, targets


def _gradients(case, g):
    """Gradients as a training program holds them: views of one flat buffer of each type, each tensor with a
    scale of its own."""
    kinds = _kinds(case)
    flat, views = {}, [None] * len(kinds)
    for dtype, here in ((torch.bfloat16, True), (torch.float32, False)):
        mine = [(i, s) for i, (s, b) in enumerate(kinds) if b == here]
        if not mine:
            continue
        buffer = torch.empty(sum(math.prod(s) for _, s in mine), dtype=dtype, device="cuda")
        scales = (10.0 ** (torch.rand(len(mine), generator=g, device="cuda") * 2.0 - 4.0)).tolist()
        at = 0
        for (i, s), scale in zip(mine, scales):
            n = math.prod(s)
            views[i] = buffer[at:at + n].view(s)
            views[i].normal_(0.0, scale, generator=g)
            at += n
        flat[dtype] = buffer
    return flat, views


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "clip":
        flat, s["grads"] = _gradients(case, g)
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(x.float())) ** 2 for x in s["grads"]))
        # what the norm may be: a part of what it is (clipped), or more (left as they are)
        s["max_norm"] = norm / case["over"]
        if case["clip"]:
            s["flat"] = {d: torch.empty_like(f) for d, f in flat.items()}
            at = dict.fromkeys(flat, 0)
            s["out"] = []
            for x in s["grads"]:
                n = x.numel()
                s["out"].append(s["flat"][x.dtype][at[x.dtype]:at[x.dtype] + n].view(x.shape))
                at[x.dtype] += n
    elif case["op"] == "experts":
        t, k, e, d, f = case["tokens"], case["top"], case["experts"], case["dim"], case["inner"]
        # a router whose experts are not equally liked
        score = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(1, e, generator=g, device="cuda")
        top = score.topk(k, dim=1)
        ids = top.indices
        if case["dropped"]:
            ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < case["dropped"], -1, ids)
        s.update(ids=ids, weights=torch.softmax(top.values, dim=1), x=_normal((t, d), 1.0, g),
                 up=_normal((e, f, d), d ** -0.5, g), down=_normal((e, d, f), f ** -0.5, g),
                 gate=_normal((e, f, d), d ** -0.5, g) if case["gated"] else None)
    else:
        s["hidden"], s["weight"], targets = _head_inputs(case, g)
        t = case["tokens"]
        masked = torch.rand(t, generator=g, device="cuda") < case["masked"]
        s["targets"] = torch.where(masked, IGNORE, targets)
        if case["backward"]:
            # advantages and a bonus for entropy, over the tokens that count
            n = (~masked).sum().clamp(min=1)
            advantage = torch.randn(t, generator=g, device="cuda")
            s["grad_logp"] = torch.where(masked, 0.0, -advantage) / n
            s["grad_entropy"] = torch.where(masked, 0.0, -case["bonus"]) / n
    if own:
        from matrix_optimizer_update_gb300 import dmuon as dm
        if case["op"] == "clip":
            s["clipper"] = dm.GradClip.create()
        elif case["op"] == "experts":
            s["layer"] = dm.Experts.create(case["tokens"], case["top"], case["experts"], case["dim"], case["inner"])
        else:
            s["head"] = dm.Head.create(case["tokens"], case["vocab"], case["dim"])
    return s


# --------------------------------------------------------------------------
# the plain forms and the framework's calls
# --------------------------------------------------------------------------

def run(s):
    return {"experts": _experts, "logprobs": _logprobs, "clip": _clip}[s["op"]](s)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _experts(s):
    x, ids, weights, up, down, gate = s["x"], s["ids"], s["weights"], s["up"], s["down"], s["gate"]
    if own:
        return s["layer"].forward(x, ids, weights, up, down, gate=gate)
    t, k = ids.shape
    e, f, d = up.shape
    xf = x.float()
    kept = (ids >= 0) & (ids < e)
    at = torch.where(kept, ids, 0)
    w = torch.where(kept, weights, 0.0)
    if t * k <= e:  # each assignment with its expert's matrices
        rows = xf.repeat_interleave(k, 0)[:, :, None]
        at = at.reshape(-1)
        u = (up[at].float() @ rows)[:, :, 0]
        h = _silu(u) if gate is None else _silu((gate[at].float() @ rows)[:, :, 0]) * u
        y = (down[at].float() @ (h * w.reshape(-1, 1))[:, :, None])[:, :, 0]
        return y.reshape(t, k, d).sum(1).to(x.dtype)
    # every token with every expert, weighted by what the router gave it
    share = torch.zeros(t, e, device=x.device).scatter_add_(1, at, w)
    u = xf @ up.reshape(e * f, d).float().T
    h = _silu(u) if gate is None else _silu(xf @ gate.reshape(e * f, d).float().T) * u
    h = h.reshape(t, e, f) * share[:, :, None]
    return (h.transpose(0, 1) @ down.float().transpose(1, 2)).sum(0).to(x.dtype)


def _logprobs(s):
    h, w, y, top, tau = s["hidden"], s["weight"], s["targets"], s["top"], s["temperature"]
    if own:
        head = s["head"]
        got = head.logprobs(h, w, y, top=top, temperature=tau)
        out = {"logp": got.logp, "entropy": got.entropy, "lse": got.lse}
        if top:
            out.update(top_ids=got.top_ids, top_logp=got.top_logp)
        if s["backward"]:
            out["dhidden"], out["dweight"] = head.logprobs_backward(h, w, y, got, s["grad_logp"], s["grad_entropy"],
                                                                    temperature=tau)
        return out
    hf, wf = h.float(), w.float()
    z = hf @ wf.T
    if tau != 1.0:
        z = z / tau
    counts = (y >= 0) & (y < w.shape[0])
    at = torch.where(counts, y, 0)[:, None]
    peak = z.amax(1, keepdim=True)
    far = z - peak
    e = torch.exp(far)
    # the target's share apart from the others': the log probability of a sure token is small beside its logits
    hit = e.gather(1, at)
    others = e.scatter(1, at, torch.where(counts[:, None], 0.0, hit)).sum(1, keepdim=True)
    total = others + torch.where(counts[:, None], hit, 0.0)
    lse = peak + torch.log(total)
    logp = torch.where(hit > others, -torch.log1p(others / hit), z.gather(1, at) - lse)
    logp = torch.where(counts[:, None], logp, 0.0)
    # the peak's own 1 apart from the sum, too: so is the entropy of a sure distribution
    rest = e.scatter(1, z.argmax(1, keepdim=True), 0.0).sum(1, keepdim=True)
    entropy = torch.log1p(rest) - (e * far).sum(1, keepdim=True) / total
    out = {"logp": logp[:, 0], "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if top:
        # order and border in 64 bits: logits next to each other are nearer than 32 bits tell apart
        ids = z.topk(min(top + 8, w.shape[0]), dim=1).indices.sort(1).values
        near = (w[ids].double() * h.double()[:, None, :]).sum(2)
        order = near.sort(dim=1, descending=True, stable=True)
        out["top_ids"] = ids.gather(1, order.indices)[:, :top]
        out["top_logp"] = (order.values[:, :top] / tau - lse).float()
    if s["backward"]:
        gl, ge = torch.where(counts, s["grad_logp"], 0.0)[:, None], s["grad_entropy"][:, None]
        dz = (far - torch.log(total) + entropy).mul_(ge).add_(gl).mul_(e / total).neg_()
        dz.scatter_add_(1, at, gl)
        if tau != 1.0:
            dz = dz / tau
        out.update(dhidden=(dz @ wf).to(h.dtype), dweight=(dz.T @ hf).to(w.dtype))
    return out


def _clip(s):
    grads = s["grads"]
    if own:
        if not s["clip"]:
            return s["clipper"].norm(grads)
        norm = s["clipper"].clip(grads, s["max_norm"], out=s["out"])
        return {"norm": norm, **{str(d): f for d, f in s["flat"].items()}}
    norm = torch.sqrt(torch.stack([g.float().square().sum().double() for g in grads]).sum())
    if not s["clip"]:
        return norm.float()
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    [o.copy_(g.float() * scale) for o, g in zip(s["out"], grads)]
    return {"norm": norm.float(), **{str(d): f for d, f in s["flat"].items()}}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"experts": _exact_experts, "logprobs": _exact_logprobs, "clip": _exact_clip}[case["op"]](case, s)


def _exact_experts(case, s):
    y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        for j in range(case["top"]):
            on = torch.nonzero(s["ids"][:, j] == e)[:, 0]
            if not len(on):
                continue
            x = s["x"][on].double()
            h = x @ s["up"][e].double().T
            if case["gated"]:
                h = h * torch.nn.functional.silu(x @ s["gate"][e].double().T)
            else:
                h = torch.nn.functional.silu(h)
            y[on] += s["weights"][on, j, None].double() * (h @ s["down"][e].double().T)
    return y


def _exact_logprobs(case, s):
    t, tau = case["tokens"], float(case["temperature"])
    if (6 if case["backward"] else 2) * t * case["vocab"] * case["dim"] > 1.6e13:
        return None
    h, w = s["hidden"].double(), s["weight"].double()
    names = ["logp", "entropy", "lse"]
    out = {n: torch.zeros(t, dtype=torch.float64, device="cuda") for n in names}
    if case["top"]:
        out["top_ids"] = None
        out["top_logp"] = torch.zeros(t, case["top"], dtype=torch.float64, device="cuda")
    if case["backward"]:
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for a in range(0, t, 512):
        b = min(a + 512, t)
        z = h[a:b] @ w.T / tau
        logp = torch.log_softmax(z, dim=1)
        p = logp.exp()
        out["lse"][a:b] = z[:, 0] - logp[:, 0]
        out["entropy"][a:b] = torch.special.entr(p).sum(1)
        rows = torch.nonzero(s["targets"][a:b] != IGNORE)[:, 0]
        ids = s["targets"][a:b][rows]
        out["logp"][a + rows] = logp[rows, ids]
        if case["top"]:
            out["top_logp"][a:b] = torch.sort(logp, dim=1, descending=True).values[:, :case["top"]]
        if case["backward"]:
            # each entry's probability times what it adds beyond the expected, for the log probability and the entropy
            gl, ge = s["grad_logp"][a:b, None].double(), s["grad_entropy"][a:b, None].double()
            one = torch.zeros_like(p)
            one[rows, ids] = 1.0
            dz = gl * (one - p * one.sum(1, keepdim=True)) - ge * p * (logp + out["entropy"][a:b, None])
            dh[a:b] = dz @ w / tau
            dw += dz.T @ h[a:b] / tau
    if case["backward"]:
        out.update(dhidden=dh, dweight=dw)
    return out


def _exact_clip(case, s):
    norm = torch.sqrt(sum((g.double() ** 2).sum() for g in s["grads"]))
    if not case["clip"]:
        return norm
    scale = min(1.0, s["max_norm"] / float(norm))
    parts = {d: [] for d in s["flat"]}
    for g in s["grads"]:
        parts[g.dtype].append(g.reshape(-1).double() * scale)
    return {"norm": norm, **{str(d): torch.cat(p) for d, p in parts.items()}}
