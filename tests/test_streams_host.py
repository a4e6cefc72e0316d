"""CPU: every convenience function that takes a stream allocates through it."""
import inspect

import torch

from combine_topk_idx_multihot_amd import binding as B


def test_every_function_that_allocates_is_wrapped():
    free = {n: f for n, f in vars(B).items() if inspect.isfunction(f) and f.__module__ == B.__name__
            and not n.startswith(("_", "moe_")) and "stream" in inspect.signature(f).parameters}
    assert len(free) >= 16 and "layer_tokens" in free and "route" in free
    for name, f in free.items():
        assert hasattr(f, "__wrapped__"), name
        assert list(inspect.signature(f).parameters)[-1] == "stream", name


def test_stream_by_name_and_by_position(monkeypatch):
    """Both ways of giving one reach the allocation and the call, and what comes back is recorded."""
    seen = []

    class Memory:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            seen.append(("in", self.stream))

        def __exit__(self, *_):
            seen.append(("out", self.stream))

    class Here:
        cuda_stream = 5

    def f(a, b=2, stream=None):
        seen.append(("call", a, b, stream))
        return a, None

    monkeypatch.setattr(B, "_memory_of", Memory)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Here)
    g = B._allocates(f)
    assert g(1) == (1, None) and seen == [("call", 1, 2, None)]
    for call in (lambda: g(1, 3, 7), lambda: g(1, b=3, stream=7)):
        seen.clear()
        call()
        assert seen == [("in", 7), ("call", 1, 3, 7), ("out", 7)]
