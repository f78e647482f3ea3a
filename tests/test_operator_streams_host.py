"""Streams and workspaces of SfaOperator, on the CPU: the C library and torch's
streams are replaced by recorders."""
import weakref

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from test_paged_streams_host import CURRENT, FakeStream, log  # noqa: F401


@pytest.fixture
def op(log, monkeypatch):  # noqa: F811
    handles = []

    def fake_init(cfg, slots):
        handles.append(sfa.Handle(0xABC, cfg))
        return handles[-1]

    monkeypatch.setattr(sfa, "sfa_init", fake_init)
    monkeypatch.setattr(sfa, "sfa_state_bytes", lambda h, batch: 4096)
    monkeypatch.setattr(sfa, "sfa_prefill_workspace_bytes", lambda h, batch, n: 256 * n)
    monkeypatch.setattr(sfa, "sfa_prefill_layers_workspace_bytes", lambda h, lc, batch, n: 256 * n)
    cfg = sfa.SfaConfig(n_layers=2, n_q_heads=4, n_kv_heads=2, head_dim=64)
    o = sfa.SfaOperator(cfg, torch.zeros(2, 64, cfg.hidden), 3, device="cpu")
    log.clear()
    yield o
    for h in handles:
        h.ptr = None


def _inputs(n):
    mk = lambda heads: torch.zeros(2, 3, n, heads, 64, dtype=torch.bfloat16)  # noqa: E731
    return mk(4), mk(2), mk(2)


def test_a_workspace_that_a_graph_captured_is_kept(op, monkeypatch):
    capturing = [False]
    monkeypatch.setattr(sfa, "_capturing", lambda stream, device: capturing[0])
    op.prefill(*_inputs(4))
    eager = weakref.ref(op.workspace)
    op.prefill(*_inputs(8))
    assert eager() is None                      # no graph: given back
    capturing[0] = True
    op.prefill(*_inputs(8))
    captured = weakref.ref(op.workspace)
    capturing[0] = False
    op.prefill(*_inputs(8))
    op.prefill(*_inputs(64))
    assert captured() is not None and captured() is not op.workspace
    replaced = weakref.ref(op.workspace)        # this one no graph knows
    op.prefill_layers(0, *_inputs(128))
    assert replaced() is None and captured() is not None


@pytest.mark.parametrize("kind", ["stream", "pointer", "default"])
def test_a_new_workspace_is_ordered_behind_its_memorys_use(op, log, kind):  # noqa: F811
    on = 0 if kind == "default" else 0x200
    op.prefill(*_inputs(4), stream={"stream": FakeStream(on), "pointer": on, "default": on}[kind])
    ptr = op.workspace.data_ptr()
    assert ("empty", ptr, on) in log


@pytest.mark.parametrize("kind", ["stream", "pointer", "default"])
@pytest.mark.parametrize("call", ["prefill", "prefill_ragged", "prefill_layers", "decode", "decode_ex"])
def test_new_outputs_are_ordered_before_the_call(op, log, kind, call):  # noqa: F811
    on = 0 if kind == "default" else 0x200
    s = FakeStream(on) if kind == "stream" else on
    if call.startswith("decode"):
        qkv = [x[:, :, 0].contiguous() for x in _inputs(1)]
        out = op.decode(*qkv, stream=s) if call == "decode" else op.decode_ex(0, *qkv, stream=s)
    elif call == "prefill_layers":
        out = op.prefill_layers(0, *_inputs(4), stream=s)
    elif call == "prefill_ragged":
        out = op.prefill_ragged(*_inputs(4), torch.zeros(3, dtype=torch.int32), stream=s)
    else:
        out = op.prefill(*_inputs(4), stream=s)
    at_call = max(i for i, e in enumerate(log) if e[0].startswith("sfa_"))
    assert log[at_call][1][-1] == on
    born = next(i for i, e in enumerate(log) if e[0] == "empty" and e[1] == out.data_ptr())
    if log[born][2] != on:
        assert ("wait", on, CURRENT) in log[born:at_call]
        assert ("used on", out.data_ptr(), on) in log


def test_a_ragged_outputs_fill_comes_before_the_wait(op, log, monkeypatch):  # noqa: F811
    fill = torch.Tensor.fill_
    monkeypatch.setattr(torch.Tensor, "fill_", lambda t, x: (log.append(("fill", t.data_ptr())), fill(t, x))[1])
    out = op.prefill_ragged(*_inputs(4), torch.zeros(3, dtype=torch.int32), stream=0x200)
    names = [e[:2] for e in log]
    assert names.index(("fill", out.data_ptr())) < names.index(("wait", 0x200))


def test_a_workspace_is_marked_as_used_on_every_other_stream(op, log):  # noqa: F811
    """Whatever stream its calls ran on, it goes back behind all of them."""
    op.prefill(*_inputs(8), stream=0x200)
    ptr = op.workspace.data_ptr()
    log.clear()
    op.prefill(*_inputs(8), stream=0x200)
    assert ("used on", ptr, 0x200) not in log    # the pool that it came from
    op.prefill(*_inputs(4), stream=FakeStream(0x300))
    op.prefill(*_inputs(4))
    op.prefill_layers(0, *_inputs(64), stream=0x200)
    assert op.workspace.data_ptr() != ptr
    assert ("used on", ptr, 0x300) in log and ("used on", ptr, CURRENT) in log
