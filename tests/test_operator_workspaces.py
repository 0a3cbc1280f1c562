"""Which workspace a call of attention or a loss gets when none is given, without a GPU: memory and streams are stand-ins,
and nothing is launched.

A workspace is what several launches of one call hand each other, so no two calls that may overlap share one: not those of
two host threads on one stream (their launches may interleave), and not a captured call and a later one (the graph runs
again whenever it is replayed).
"""
import threading

import pytest

torch = pytest.importorskip("torch")

from lora_fine_tuning_gb300 import api  # noqa: E402


@pytest.fixture
def on(monkeypatch):
    """Stands for a call on stream 7 of device 0; `on.captures` says whether that stream is being captured."""
    class On(api._On):
        captures = False
        made = []

        def __init__(self, handle=7):
            self.index, self.stream, self.handle = 0, None, handle

        def empty(self, shape, dtype):
            t = torch.full((shape,) if isinstance(shape, int) else shape, 7, dtype=dtype)   # memory is not zero by itself
            On.made.append(t)
            return t

        def capturing(self):
            return On.captures

    On.made = []
    return On


def test_a_threads_calls_on_one_stream_share_one(on):
    a = on().workspace("attn", 1000)
    assert a.numel() >= 1000 and not a.count_nonzero()
    assert on().workspace("attn", 900) is a and on(7).workspace("attn", 1000) is a
    assert on(8).workspace("attn", 1000) is not a and on().workspace("loss", 1000) is not a
    larger = on().workspace("attn", 5 << 20)
    assert larger.numel() >= 5 << 20 and on().workspace("attn", 1000) is larger


def test_threads_do_not_share(on):
    mine, theirs, wait = on().workspace("attn", 1000), [], threading.Barrier(4)

    def work():
        wait.wait(10)   # all alive at once
        theirs.append(on().workspace("attn", 1000))
        wait.wait(10)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len({t.data_ptr() for t in theirs + [mine]}) == 5
    assert on().workspace("attn", 1000) is mine


def test_a_captured_call_has_its_own(on):
    """Zeroed by the graph itself, whatever ran before; neither kept for later calls nor taken from earlier ones."""
    eager = on().workspace("loss", 1000)
    on.captures = True
    first, second = on().workspace("loss", 1000), on().workspace("loss", 1000)
    for ws in (first, second):
        assert ws is not eager and ws.numel() >= 1000 and not ws[:256].count_nonzero()
    assert first.data_ptr() != second.data_ptr()
    on.captures = False
    assert on().workspace("loss", 1000) is eager
    other = on(9)
    on.captures = True
    other.workspace("loss", 1000)
    on.captures = False
    made = len(on.made)
    assert on(9).workspace("loss", 1000) is not None and len(on.made) == made + 1   # the first outside capture


def test_public_workspaces(on, monkeypatch):
    """What a call without a workspace uses can be asked for its status; not during a capture, where each call has its own."""
    class Sizes:
        attn_workspace_size = staticmethod(lambda rows, heads: 4 * rows * heads)
        loss_workspace_size = staticmethod(lambda rows: 4 * rows)

    class On(on):
        def __init__(self, t, stream):
            super().__init__()

    monkeypatch.setattr(api.native, "lib", lambda: Sizes)
    monkeypatch.setattr(api, "_On", On)
    assert api.attn_workspace(100, 8) is on().workspace("attn", 3200)
    assert api.loss_workspace(100) is on().workspace("loss", 400)
    on.captures = True
    for f in (lambda: api.attn_workspace(100, 8), lambda: api.loss_workspace(100)):
        with pytest.raises(RuntimeError, match="ws="):
            f()
