"""What a call allocates belongs to the stream that its kernels run on: memory from another
stream's pool could be handed out again while they still use it."""
import ast
import contextlib
import inspect

import pytest

import token_indexed_ffn_amd as st

MAKES = {"empty", "zeros", "empty_like", "zeros_like", "new_empty", "new_zeros", "_like", "_rows_out", "_grads_out"}


def functions():   # of the binding, that take a stream
    for f in ast.parse(inspect.getsource(st)).body:
        if isinstance(f, ast.FunctionDef) and "stream" in {a.arg for a in f.args.args + f.args.kwonlyargs} and \
                f.name not in ("_own", "_ws"):
            yield f


def called(node):
    return getattr(node.func, "attr", getattr(node.func, "id", None)) if isinstance(node, ast.Call) else None


@pytest.mark.parametrize("f", functions(), ids=lambda f: f.name)
def test_allocations_are_made_on_the_calls_stream(f):
    within = set()
    for node in ast.walk(f):
        if called(node) == "_own":
            assert isinstance(node.args[0], ast.Name) and node.args[0].id == "stream"
            within |= {id(x) for x in ast.walk(node.args[1])}
    for node in ast.walk(f):
        if called(node) in MAKES:
            assert id(node) in within, f"{f.name}: line {node.lineno}"
        if called(node) == "_ws":
            assert isinstance(node.args[-1], ast.Name) and node.args[-1].id == "stream", f.name


class Tensor:
    def __init__(self, pool):
        self.pool, self.recorded = pool, []

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.fixture
def pools(monkeypatch):
    now = ["current"]

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    monkeypatch.setattr(st.torch.cuda, "stream", on)
    monkeypatch.setattr(st.torch.cuda, "current_stream", lambda *a: now[0])
    monkeypatch.setattr(st.torch, "empty", lambda *a, **k: Tensor(now[0]))
    return now


def test_outputs_come_from_the_stream_and_are_recorded_where_they_are_read(pools):
    made = st._own("side", lambda: {"a": st.torch.empty(3), "b": None})
    assert made["a"].pool == "side" and made["a"].recorded == ["current"] and made["b"] is None
    made = st._own("side", lambda: (st.torch.empty(3), st.torch.empty(3)))
    assert all(t.pool == "side" and t.recorded == ["current"] for t in made)
    assert st._own("side", st.torch.empty, 3).pool == "side"
    made = st._own(None, lambda: st.torch.empty(3))
    assert made.pool == "current" and made.recorded == [] and pools == ["current"]


def test_workspaces_come_from_the_stream(pools):
    assert st._ws(100, None, "cuda", "side").pool == "side"
    assert st._ws(100, None, "cuda", None).pool == "current"
    assert st._ws(0, None, "cuda", "side") is None and pools == ["current"]


def test_the_current_stream_where_torch_offers_no_raw_handle(monkeypatch):
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(st.torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(st, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(st, "_current_device", lambda: 3)
    assert st._stream(None) == 1003 and st._stream(Stream) == 77
    monkeypatch.setattr(st, "_raw_stream", None)
    assert st._stream(None) == 77
