"""The head's forward pass where a tile is a single K stage and each pair of SMs has more tiles than the list
between its warps holds: every tile is summed once, by every warp."""

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,vocab,dim", [(128, 200000, 16), (64, 200000, 16), (128, 200000, 64), (100, 400000, 40),
                                              (20, 300000, 8), (200, 300000, 16)])
def test_many_short_tiles(tokens, vocab, dim):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    h = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    z = h.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    # test_gpu_head.py's bound of lse, with A <= dim * max |h| * max |w| and |z| <= A
    a = dim * float(h.abs().max()) * float(w.abs().max())
    ez = (dim + 9) * 2.0 ** -23 * a
    off = 2 * ez + 400 * 2.0 ** -24 + 4 * 2.0 ** -24 * (1 + a) + 2.0 ** -23 * float(want.abs().max())
    head = dm.Head.create(tokens, vocab, dim)
    past = -head.workspace.data_ptr() % 1024 + 1024  # the status word and the counters
    for _ in range(30):
        head.workspace[past:].fill_(255)
        loss, lse = head.xent(h, w, y)
        assert head.read_device_status(torch.cuda.current_stream().cuda_stream) == 0
        assert (lse - want).abs().max() <= off
        assert (loss - (want - z.gather(1, y[:, None])[:, 0])).abs().max() <= 2 * off
