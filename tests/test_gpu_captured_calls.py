"""Attention and losses captured in CUDA graphs without a workspace of the caller's.

A graph's result is compared bit by bit with that of the same call outside it, whichever graph is replayed first, and again
after a larger call and after memory that the allocator had free is written over.
"""
import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_threads import attention, policy, preference  # noqa: E402


# name -> two calls with inputs of their own, and a larger one
CALLS = {
    "preference, long rows": lambda: (preference(40, 32001, torch.bfloat16, 2, 0), preference(24, 40000, torch.float32, 3, 1),
                                      preference(4000, 33000, torch.bfloat16, 40, 2)),
    "preference, short rows": lambda: (preference(40, 1000, torch.bfloat16, 2, 3), preference(24, 900, torch.float32, 3, 4),
                                       preference(200000, 64, torch.bfloat16, 70, 5)),
    "policy": lambda: (policy(40, 32001, torch.bfloat16, 6), policy(24, 50001, torch.float32, 7),
                       policy(250000, 64, torch.bfloat16, 8)),
    "attention": lambda: (attention([(0, 1, 0, 5000), (1, 20, 5000, 3000)], 8, 2, 64, 9),
                          attention([(0, 2000, 0, 2000)], 8, 1, 64, 10), attention([(0, 30000, 0, 30000)], 16, 4, 64, 11)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_two_graphs_without_a_workspace(name):
    first, second, larger = CALLS[name]()
    want = [[x.clone() for x in f()] for f in (first, second)]
    graphs, outs = [], []
    for f in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)

    def replay(order, wipe):
        for i in order:
            for x in outs[i]:
                x.fill_(7)
        if wipe:
            junk = [torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        if wipe:
            assert all(bool((x == 255).all()) for x in junk)
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i])), (name, i)

    replay((1, 0), False)           # the second one first
    replay((0, 1, 1, 0), False)
    larger()                        # a larger workspace outside the graphs
    replay((1, 0), True)
    assert all(torch.equal(a, b) for a, b in zip(want[0], first()))     # and calls outside go on
    del graphs[0], outs[0], want[0]
    larger()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[0], outs[0]))
