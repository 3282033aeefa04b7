"""Experts, log probabilities and clipping at work at the same time: several objects on streams of their own, from one
thread and from several. Each call's results are those that it has alone."""

import threading

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def jobs():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf16 = lambda t: t.to(torch.bfloat16)  # noqa: E731
    made = []
    for tokens, top, experts, dim, inner in ((1, 4, 16, 1024, 512), (40, 3, 8, 520, 264)):
        layer = dm.Experts.create(tokens, top, experts, dim, inner)
        x, up = bf16(r(tokens, dim)), bf16(r(experts, inner, dim) * dim ** -0.5)
        gate, down = bf16(r(experts, inner, dim) * dim ** -0.5), bf16(r(experts, dim, inner) * inner ** -0.5)
        ids = torch.randint(0, experts, (tokens, top), generator=g, device="cuda")
        weights = torch.softmax(r(tokens, top), 1)
        made.append(lambda layer=layer, a=(x, ids, weights, up, down), gate=gate: [layer.forward(*a, gate=gate)])
    for tokens, vocab, dim in ((5, 20000, 256), (300, 9000, 256)):
        head = dm.Head.create(tokens, vocab, dim)
        h, w, y = bf16(r(tokens, dim)), bf16(r(vocab, dim) * dim ** -0.5), torch.randint(
            0, vocab, (tokens,), generator=g, device="cuda")
        gl, ge = r(tokens), r(tokens)

        def score(head=head, h=h, w=w, y=y, gl=gl, ge=ge):
            s = head.logprobs(h, w, y, top=6)
            return [s.logp, s.entropy, s.top_ids, s.top_logp, *head.logprobs_backward(h, w, y, s, gl, ge)]
        made.append(score)
    for sizes in ([(64, 33)] * 3, [(1000, 1111)] * 9):
        clip, grads = dm.GradClip.create(), [r(*s) for s in sizes]
        made.append(lambda clip=clip, grads=grads: [clip.norm(grads)])
    return made


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_on_streams_at_the_same_time():
    made = jobs()
    want = [job() for job in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for _ in range(15):
        for job, stream in zip(made, streams):
            with torch.cuda.stream(stream):
                got.append(job())
    torch.cuda.synchronize()
    assert all(same(want[k % len(made)], g) for k, g in enumerate(got))


def test_from_threads_at_the_same_time():
    made = jobs()
    want = [job() for job in made]
    torch.cuda.synchronize()
    right = [False] * len(made)

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [made[k]() for _ in range(15)]
            stream.synchronize()
            right[k] = all(same(want[k], g) for g in got)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(right)


def test_two_graphs_that_share_workspaces():
    made = jobs()
    want = [job() for job in made]
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append([job() for job in made])
    for _ in range(5):
        for graph, results in zip(graphs, got):
            for r in results:
                for t in r:
                    t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(same(w, r) for w, r in zip(want, results))
    for _ in range(20):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(same(w, r) for results in got for w, r in zip(want, results))
