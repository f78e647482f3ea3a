"""Workspaces and streams of the paged cache calls: captured graphs, several
streams and several host threads."""
import threading

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from test_gpu_paged import Case, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["extension", "ctypes"])
def path(request, monkeypatch):
    """Both ways from Python into the library."""
    if request.param == "ctypes":
        monkeypatch.setattr(sfa, "_fast", None)
    elif sfa._fast is None:
        pytest.skip("the extension is not built")
    return request.param


def _case(seed=51, n=2, ctx=(20001, 3000)):
    """Sequences that are split over CTAs: their pieces go through the workspace."""
    return Case("qwen7b", "bf16", list(ctx), [n] * len(ctx), n, 64, seed=seed)


def test_a_captured_call_keeps_its_workspace(path):
    """A larger call on the same stream, then the graph again, with the rest of
    the freed memory in other hands."""
    c = _case(n=1)
    big = _case(n=60, ctx=(4000, 77), seed=52)
    want = c.cache.attend(0, c.q, c.ctx_d)
    s = torch.cuda.Stream()
    out = torch.zeros_like(want)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        c.cache.attend(0, c.q, c.ctx_d, out=out)              # warm-up
        g = torch.cuda.CUDAGraph()
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        c.cache.attend(0, c.q, c.ctx_d, out=out)
    with torch.cuda.stream(s):
        big_cache = sfa.SfaPagedCache(c.h, big.k_pages, big.v_pages, big.table)
        more = big_cache.attend(0, big.q, big.ctx_d)
        c.cache.attend(0, torch.cat([c.q] * 40, 2).contiguous(), ints([100, 100]))
        size = sfa.sfa_kv_attend_workspace_bytes(c.h, 1)
        held = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(24)]
        for _ in range(3):
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert torch.equal(out, want) and bool(torch.isfinite(more).all())
    assert all(bool((t == 0x5A).all()) for t in held)


def test_two_graphs_of_one_cache_side_by_side(path):
    c = _case()
    qs = [c.q, torch.randn_like(c.q)]
    want = [c.cache.attend(0, q, c.ctx_d) for q in qs]
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):                              # both on torch's own capture stream
            c.cache.attend(0, q, c.ctx_d, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("kind", ["stream", "pointer"])
def test_another_stream_without_a_wait(path, kind):
    """The current stream is still busy with a block of the workspace's size that
    it has given back: a call on another stream must not be handed it."""
    c = _case()
    want = c.cache.attend(0, c.q, c.ctx_d)
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    size = sfa.sfa_kv_attend_workspace_bytes(c.h, c.n)
    torch.cuda.synchronize()
    for _ in range(4):
        blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(6)]
        torch.cuda._sleep(2_000_000)
        for _ in range(20):
            for b in blocks:
                b.fill_(0xFF)
        del blocks, b
        c.cache.attend(0, c.q, c.ctx_d, out=out, stream=s if kind == "stream" else s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
        torch.cuda.synchronize()
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK


def test_host_threads_on_one_stream(path):
    """attend is two launches, which the threads' calls may mix."""
    c = _case()
    N = 4
    qs = [torch.randn_like(c.q) for _ in range(N)]
    want = [c.cache.attend(0, q, c.ctx_d) for q in qs]
    outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(N), []

    def serve(i):
        try:
            start.wait()
            for o in outs[i]:
                c.cache.attend(0, qs[i], c.ctx_d, out=o)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=serve, args=(i,)) for i in range(N)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert all(torch.equal(o, w) for w, row in zip(want, outs) for o in row)


def test_a_given_workspace_is_used(path):
    c = _case()
    want = c.cache.attend(0, c.q, c.ctx_d)
    ws = torch.full((sfa.sfa_kv_attend_workspace_bytes(c.h, c.n),), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    c.cache.attend(0, c.q, c.ctx_d, out=out, workspace=ws)
    assert torch.equal(out, want) and not bool((ws == 0x5A).all())
    with pytest.raises(sfa.SfaError):
        c.cache.attend(0, c.q, c.ctx_d, out=out, workspace=ws[:-1])


@pytest.mark.parametrize("kind", ["stream", "pointer", "default pointer"])
def test_new_outputs_on_another_stream(path, kind):
    """The current stream is busy when it is to fill the new outputs: the fill must
    not come after the call's results."""
    c = _case(ctx=(300, 20))
    parents = ints([[-1, 0], [-1, -1]])
    rope = sfa.SfaRope()
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()

    def step(stream=None):
        pos, mask = sfa.sfa_tree_plan(c.h, parents, c.ctx_d, stream=stream)
        qr, _ = c.cache.append(0, c.q, c.k, c.v, c.ctx_d, positions=pos, rope=rope, stream=stream)
        return pos, mask, qr, c.cache.attend(0, qr, c.ctx_d, mask=mask, stream=stream)

    want = step()
    torch.cuda.synchronize()
    s, busy = torch.cuda.Stream(), torch.cuda.Stream()
    on = {"stream": s, "pointer": s.cuda_stream, "default pointer": 0}[kind]
    for _ in range(3):
        c.k_pages.copy_(k0)
        c.v_pages.copy_(v0)
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(3_000_000)
            got = step(on)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK


@pytest.mark.skipif(sfa._fast is None, reason="the extension is not built")
def test_calls_without_outputs_go_through_the_extension(monkeypatch):
    c = _case(ctx=(300, 20))

    def never(*args):
        raise AssertionError("the ctypes path was taken")

    for name in ("_append_fn", "_attend_fn", "_accept_fn"):
        monkeypatch.setattr(c.cache, name, never)
    monkeypatch.setattr(sfa, "_call_on", never)
    pos, mask = sfa.sfa_tree_plan(c.h, ints([[-1, 0], [-1, -1]]), c.ctx_d)
    qr, kr = c.cache.append(0, c.q, c.k, c.v, c.ctx_d, positions=pos, rope=sfa.SfaRope(), k_out=torch.empty_like(c.k))
    out = c.cache.attend(0, qr, c.ctx_d, mask=mask)
    c.cache.accept(0, 1, ints([[1, 0], [0, 1]]), ints([1, 2]), c.ctx_d)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert out.shape == (1, 2, 2, c.h.cfg.hidden) and bool(torch.isfinite(out).all())
