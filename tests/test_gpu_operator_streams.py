"""Workspaces and new outputs of SfaOperator with captured graphs and other
streams."""
import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from sfa_harness import sfa_config
from workloads import WORKLOADS, TokenSource, make_slots

pytestmark = pytest.mark.gpu


def _setup():
    w = WORKLOADS["qwen05b"].replace(name="streams", n_layers=2, batch=2)
    return w, make_slots(w, "cuda"), TokenSource(w, "cuda")


def test_a_captured_prefill_keeps_its_workspace():
    """A longer prefill replaces the operator's workspace; the graph goes on
    with the one that it captured."""
    w, slots, src = _setup()
    op = sfa.SfaOperator(sfa_config(w), slots, w.batch, device="cuda")
    small, large = src.get(0, 70), src.get(0, 700)
    want = op.prefill(*small)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        op.reset()
        op.prefill(*small, out=out)
    used = op.workspace.data_ptr()
    op.reset()
    op.prefill(*large)
    assert op.workspace.data_ptr() != used
    size = sfa.sfa_prefill_workspace_bytes(op.handle, w.batch, 70)
    held = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(16)]
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((t == 0x5A).all()) for t in held)
    assert op.check() == sfa.SFA_OK


@pytest.mark.parametrize("kind", ["stream", "pointer", "default pointer"])
def test_new_outputs_and_workspace_on_another_stream(kind):
    w, slots, src = _setup()
    q, k, v = src.get(0, 70)
    lens = torch.tensor([70, 33], dtype=torch.int32, device="cuda")
    qd, kd, vd = (x[:, :, 0].contiguous() for x in src.get(70, 71))

    def step(op, stream=None):
        op.reset(stream)
        return op.prefill_ragged(q, k, v, lens, stream=stream), op.decode(qd, kd, vd, stream=stream)

    want = step(sfa.SfaOperator(sfa_config(w), slots, w.batch, device="cuda"))
    s, busy = torch.cuda.Stream(), torch.cuda.Stream()
    on = {"stream": s, "pointer": s.cuda_stream, "default pointer": 0}[kind]
    for _ in range(3):
        op = sfa.SfaOperator(sfa_config(w), slots, w.batch, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(3_000_000)
            got = step(op, on)
        torch.cuda.synchronize()
        assert op.check() == sfa.SFA_OK
        live = ~torch.isnan(want[0])
        assert torch.equal(torch.isnan(got[0]), ~live) and torch.equal(got[0][live], want[0][live])
        assert torch.equal(got[1], want[1])


def test_calls_on_several_streams_in_order():
    """One operator on three streams that wait for one another, its workspace
    growing between them."""
    w, slots, src = _setup()
    parts = [src.get(0, 70), src.get(70, 400), src.get(400, 420), src.get(420, 1200)]
    ref = sfa.SfaOperator(sfa_config(w), slots, w.batch, max_prefill=800, device="cuda")
    want = [ref.prefill(*x) for x in parts]
    op = sfa.SfaOperator(sfa_config(w), slots, w.batch, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got, before = [], None
    for x, s in zip(parts, streams):
        if before is not None:
            s.wait_stream(before)
        got.append(op.prefill(*x, stream=None if s is torch.cuda.current_stream() else s))
        before = s
    torch.cuda.synchronize()
    assert op.check() == sfa.SFA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
