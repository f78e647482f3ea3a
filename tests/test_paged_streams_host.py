"""Streams and workspaces of the paged cache calls, on the CPU: the C library
and torch's streams are replaced by recorders, so that the order of fills, waits
and calls shows."""
import contextlib

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa


class Log(list):
    """What happened, in order; the C library's calls among it."""

    def __init__(self):
        super().__init__()
        self.on_attend = None

    def __getattr__(self, name):
        if not name.startswith("sfa_"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("_bytes"):
                return 1024 * args[1]
            self.append((name, args))
            if name == "sfa_kv_attend" and self.on_attend:
                self.on_attend()
            return 0
        return call


class FakeStream:
    log = None

    def __init__(self, ptr, device=None):
        self.cuda_stream = ptr

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


CURRENT = 0x100


@pytest.fixture
def log(monkeypatch):
    log = Log()
    FakeStream.log = log
    on = [CURRENT]

    @contextlib.contextmanager
    def stream(s):
        on.append(on[-1] if s is None else s.cuda_stream)
        yield
        on.pop()

    empty, zeros = torch.empty, torch.zeros

    def logged(name, fn):
        def call(*args, **kw):
            t = fn(*args, **kw)
            log.append((name, t.data_ptr(), on[-1]))
            return t
        return call

    monkeypatch.setattr(sfa, "_lib", log)
    monkeypatch.setattr(sfa, "_fast", None)
    monkeypatch.setattr(sfa, "_is_cuda_tensor", lambda t: isinstance(t, torch.Tensor))
    monkeypatch.setattr(sfa, "_stream_ptr", lambda s: on[-1] if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(on[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch, "empty", logged("empty", empty))
    monkeypatch.setattr(torch, "zeros", logged("zeros", zeros))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("used on", t.data_ptr(), s.cuda_stream)))
    yield log


@pytest.fixture
def cache(log):
    h = sfa.Handle(0xABC, sfa.SfaConfig(n_layers=1, n_q_heads=4, n_kv_heads=2, head_dim=64))
    pages = lambda: torch.zeros(1, 6, 2, 16, 64, dtype=torch.bfloat16)  # noqa: E731
    c = sfa.SfaPagedCache(h, pages(), pages(), torch.zeros(3, 2, dtype=torch.int32))
    log.clear()
    yield c
    h.ptr = None


def _q(n):
    return torch.zeros(1, 3, n, 4, 64, dtype=torch.bfloat16)


def _attend(cache, n=1, **kw):
    return cache.attend(0, _q(n), torch.zeros(3, dtype=torch.int32), out=torch.zeros(1, 3, n, 256, dtype=torch.bfloat16), **kw)


def _workspaces(log):
    return [args[11] for name, *rest in log if name == "sfa_kv_attend" for args in rest]


def test_a_workspace_belongs_to_one_call(cache, log):
    """attend is two launches: a call of another thread between them, on the
    same stream, must not write the pieces that the second is to join."""
    inner = []

    def second_thread():
        log.on_attend = None
        inner.append(_attend(cache))

    log.on_attend = second_thread
    _attend(cache)
    a, b = _workspaces(log)
    assert inner and a != b


def test_a_workspace_is_not_kept(cache, log):
    """Each call takes its own, while it runs: in a capture that is the graph's
    memory, and no later call can take it from under the graph."""
    for n in (1, 16, 1):
        log.clear()
        _attend(cache, n)
        assert _workspaces(log)[0] in [e[1] for e in log if e[0] == "empty"]


@pytest.mark.parametrize("kind", ["stream", "pointer", "default"])
def test_a_workspace_comes_from_the_pool_of_the_calls_stream(cache, log, kind):
    """So that it is ordered behind what used that memory before, and free
    again only for work behind the call."""
    s = {"stream": FakeStream(0x200), "pointer": 0x200, "default": 0}[kind]
    _attend(cache, stream=s)
    (ptr,) = _workspaces(log)
    assert ("empty", ptr, 0 if kind == "default" else 0x200) in log


@pytest.mark.parametrize("kind", ["stream", "pointer", "default"])
@pytest.mark.parametrize("call", ["plan", "append", "attend"])
def test_new_outputs_are_filled_before_the_call(cache, log, kind, call):
    s = {"stream": FakeStream(0x200), "pointer": 0x200, "default": 0}[kind]
    on = 0 if kind == "default" else 0x200
    ctx = torch.zeros(3, dtype=torch.int32)
    if call == "plan":
        outs = sfa.sfa_tree_plan(cache.handle, torch.zeros(3, 4, dtype=torch.int32), ctx, stream=s)
    elif call == "append":
        k = torch.zeros(1, 3, 4, 2, 64, dtype=torch.bfloat16)
        outs = cache.append(0, _q(4), k, k.clone(), ctx, stream=s)[:1]
    else:
        outs = [cache.attend(0, _q(4), ctx, workspace=torch.zeros(1 << 16, dtype=torch.uint8), stream=s)]
    names = [e[0] for e in log]
    at_call = max(i for i, n in enumerate(names) if n.startswith("sfa_"))
    assert log[at_call][1][-1] == on
    for t in outs:
        fill = next(i for i, e in enumerate(log) if e[0] == "zeros" and e[1] == t.data_ptr())
        if log[fill][2] != on:
            assert ("wait", on, CURRENT) in log[fill:at_call], "the call's stream does not wait for the fill"
            assert ("used on", t.data_ptr(), on) in log
