"""Memory that a call takes for itself belongs to the stream it runs on: torch's allocator orders a
block's uses by the stream that was current when it was allocated, and would give a block of another
stream away while the call still works in it."""
import ast
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__
    __graft_entry__.build()
    import gated_delta_rule_prologue_b200 as m
    return m


def test_only_one_function_allocates(kda):
    with open(kda.__file__) as f:
        tree = ast.parse(f.read())
    makers = {"empty", "empty_like", "zeros", "zeros_like", "new_empty", "new_zeros", "full"}
    where = [fn.name for fn in ast.walk(tree) if isinstance(fn, ast.FunctionDef)
             for x in ast.walk(fn)
             if isinstance(x, ast.Call) and isinstance(x.func, ast.Attribute) and x.func.attr in makers]
    assert set(where) == {"_new"}, where


def test_every_allocation_names_the_calls_stream(kda):
    with open(kda.__file__) as f:
        tree = ast.parse(f.read())
    calls = [x for x in ast.walk(tree) if isinstance(x, ast.Call) and isinstance(x.func, ast.Name)
             and x.func.id == "_new"]
    assert len(calls) >= 10
    for x in calls:
        assert len(x.args) == 4 and isinstance(x.args[3], ast.Name) and x.args[3].id == "stream", x.lineno


def test_allocates_on_the_given_stream(kda, monkeypatch):
    current = []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    seen = []
    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(list(current)), empty(*a, **k))[1])
    side = torch.cuda.Stream.__new__(torch.cuda.Stream) if torch.cuda.is_available() else _Stream()
    monkeypatch.setattr(kda, "_STREAM", type(side))
    kda._new(16, torch.uint8, "cpu", side)
    kda._new((2, 3), torch.float32, "cpu", None)
    assert seen == [[side], []]


class _Stream:
    cuda_stream = 0
