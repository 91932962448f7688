"""How the holders' workspaces grow, with stand-ins for device memory (no GPU needed)."""
import types

import pytest

torch = pytest.importorskip("torch")

from lossless_bit_weight_encode_gb300 import kv  # noqa: E402


class Memory:
    def __init__(self, size):
        self.size = size

    def numel(self):
        return self.size


@pytest.fixture(autouse=True)
def memory(monkeypatch):
    monkeypatch.setattr(torch, "zeros", lambda size, **kw: Memory(size))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(kv, "_workspaces", {})
    monkeypatch.setattr(kv, "_outgrown", [])


def test_shared_prefix_workspaces_kept_are_smaller_than_the_present_one():
    """Their size goes with the tokens, and a batch grows by degrees: what captured graphs may
    still use does not add up."""
    for tokens in range(1, 400):
        size = 50_000 * tokens
        now = kv._workspaces.get((0, 7, "shared"))
        if now is None or now.numel() < size:
            now = kv._grow_shared(0, 7, size)
        assert kv._workspaces[0, 7, "shared"] is now and now.numel() >= size
        assert sum(w.numel() for w in kv._outgrown) <= now.numel()
    assert len(kv._outgrown) < 8


def test_workspaces_of_other_streams_and_calls_are_their_own():
    a, b, c = kv._grow_shared(0, 7, 1 << 20), kv._grow_shared(0, 8, 1 << 20), kv._grow(0, 7, 5 << 20)
    assert len({id(x) for x in (a, b, c)}) == 3 and not kv._outgrown
    assert (a.numel(), b.numel(), c.numel()) == (1 << 20, 1 << 20, 5 << 20)
    assert kv._grow(0, 7, 6 << 20).numel() == 6 << 20  # one size on a device but for its counters
    assert kv._outgrown == [c]


def test_forked_pages_keep_the_workspace_that_a_graph_may_use():
    """Tables that were replaced by larger ones need a larger workspace."""
    pages = types.SimpleNamespace(_ws=None, _outgrown=[], tables=types.SimpleNamespace(device="cuda:0"))
    first = kv.KVPages._grow(pages, 0, 7, 1000)
    second = kv.KVPages._grow(pages, 0, 7, 2000)
    assert pages._ws is second and pages._outgrown == [first] and second.numel() == 2000
