"""Several host threads sort at the same time, each with a scratch and a stream of its own."""

import ctypes
import threading

import pytest
import torch

from matrix_optimizer_update_gb300 import dmuon as dm

pytestmark = pytest.mark.gpu


def test_threads_that_sort_for_different_numbers_of_experts():
    # more than 40 KB of shared memory each, of different sizes: 33 counts for 1024, 700 and 400 experts
    L, n, rounds = dm.lib(), 8192, 8000
    refused, outputs = [], {}

    def work(experts, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ids = torch.randint(0, experts, (n, 1), generator=g, device="cuda")
            dest, source = (torch.empty(n, device="cuda", dtype=torch.int32) for _ in range(2))
            offsets = torch.empty(experts + 1, device="cuda", dtype=torch.int32)
            router = dm.Router.create(n, 1, experts)
        args = (ids.data_ptr(), n, 1, experts, dest.data_ptr(), source.data_ptr(), offsets.data_ptr(),
                router.workspace.data_ptr(), ctypes.c_size_t(router.workspace.numel()), s.cuda_stream)
        for _ in range(rounds):
            if L.dmuon_route_sort(*args) != dm.OK:
                refused.append((experts, L.dmuon_last_error()))
        s.synchronize()
        outputs[seed] = (ids, source)

    threads = [threading.Thread(target=work, args=a) for a in ((1024, 0), (400, 1), (700, 2), (1024, 3))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not refused, (len(refused), refused[:3])
    for ids, source in outputs.values():
        assert torch.equal(source.long(), torch.argsort(ids[:, 0], stable=True))
    assert len(outputs) == len(threads)
