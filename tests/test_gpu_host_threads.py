"""The first CUDA call of a host thread may be one of the library's."""
import threading

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from sfa_harness import sfa_config
from test_gpu_paged import Case
from workloads import WORKLOADS, TokenSource, make_slots

pytestmark = pytest.mark.gpu


def in_new_thread(fn):
    errors = []

    def run():
        try:
            fn()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("fast", [True, False], ids=["extension", "ctypes"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_calls(monkeypatch, dtype, fast):
    if not fast:
        monkeypatch.setattr(sfa, "_fast", None)
    c = Case("qwen05b", dtype, [300, 20], [2, 1], 2, 16, seed=61)
    want = c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d)
    ws = torch.empty(sfa.sfa_kv_attend_workspace_bytes(c.h, 2), dtype=torch.uint8, device="cuda")
    out, qo = torch.zeros_like(want), torch.zeros_like(c.q)
    torch.cuda.synchronize()
    in_new_thread(lambda: c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out, workspace=ws))
    assert torch.equal(out, want)
    in_new_thread(lambda: c.cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=c.lens_d, q_out=qo))
    assert torch.equal(qo[:, 0], c.q[:, 0])
    in_new_thread(lambda: c.cache.accept(0, 1, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), c.lens_d - c.lens_d, c.ctx_d))
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK


@pytest.mark.parametrize("prefill_near", [1, 2])
def test_prefill_and_decode(prefill_near):
    w = WORKLOADS["qwen05b"].replace(name="threads", n_layers=2, batch=2)
    slots, src = make_slots(w, "cuda"), TokenSource(w, "cuda")
    q, k, v = src.get(0, 80)
    qd, kd, vd = (x[:, :, 0].contiguous() for x in src.get(80, 81))
    got = []
    for thread in (lambda fn: fn(), in_new_thread):
        op = sfa.SfaOperator(sfa_config(w), slots, w.batch, max_prefill=80, device="cuda")
        sfa.sfa_debug_set_paths(op.handle, 1, prefill_near)
        out = [torch.zeros(w.n_layers, w.batch, 80, op.cfg.hidden, device="cuda"),
               torch.zeros(w.n_layers, w.batch, op.cfg.hidden, device="cuda")]
        torch.cuda.synchronize()
        thread(lambda: op.prefill(q, k, v, out=out[0]))
        thread(lambda: op.decode(qd, kd, vd, out=out[1]))
        assert op.check() == sfa.SFA_OK
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
