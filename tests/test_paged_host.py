"""Refusals of the paged cache calls and the binding's checks, without a GPU:
nothing here reaches a kernel."""
import ctypes

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from kv_cache_compression_sfa_b200 import build as sfa_build


@pytest.fixture(scope="module")
def lib():
    sfa_build.build()
    return sfa.load_library()


def test_calls_without_a_handle_are_refused(lib):
    c = sfa.sfa_kv_cache(256, 256, 4, 16, 4, 256)
    r = ctypes.byref(c)
    bad = ctypes.c_void_p(None)
    assert lib.sfa_tree_plan(bad, 256, 1, None, 256, 1, 256, 256, None) == sfa.SFA_ERR_INVALID_ARG
    assert lib.sfa_kv_append(bad, r, 0, 1, 256, 256, 256, 1, None, 256, None, None, 1, 256, None, None) == sfa.SFA_ERR_INVALID_ARG
    assert lib.sfa_kv_attend(bad, r, 0, 1, 256, 1, None, 256, None, 1, 256, 256, 1, None) == sfa.SFA_ERR_INVALID_ARG
    assert lib.sfa_kv_accept(bad, r, 0, 1, 256, 1, 256, 256, 1, None) == sfa.SFA_ERR_INVALID_ARG
    assert lib.sfa_kv_attend_workspace_bytes(bad, 4) == 0


def test_rope_checks_its_frequencies():
    with pytest.raises(ValueError):
        sfa.SfaRope(dims=64, inv_freq=[1.0] * 31)
    with pytest.raises(ValueError):
        sfa.SfaRope(inv_freq=[1.0] * 31).check(64)
    sfa.SfaRope(inv_freq=[1.0] * 32).check(64)


class _Recorder:
    """Records the C calls of the binding."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def cache(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(sfa, "_lib", rec)
    monkeypatch.setattr(sfa, "_is_cuda_tensor", lambda t: isinstance(t, torch.Tensor))
    monkeypatch.setattr(sfa, "_stream_ptr", lambda stream: 0x5151)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    h = sfa.Handle(0xABC, sfa.SfaConfig(n_layers=2, n_q_heads=4, n_kv_heads=2, head_dim=64))
    pages = lambda: torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)  # noqa: E731
    c = sfa.SfaPagedCache(h, pages(), pages(), torch.zeros(3, 2, dtype=torch.int32))
    yield c, rec, h
    h.ptr = None


def _new(n=4, layers=1, dtype=torch.bfloat16):
    return (torch.zeros(layers, 3, n, 4, 64, dtype=dtype), torch.zeros(layers, 3, n, 2, 64, dtype=dtype),
            torch.zeros(layers, 3, n, 2, 64, dtype=dtype))


CTX = torch.zeros(3, dtype=torch.int32)


def test_binding_passes_the_c_arguments_in_order(cache):
    c, rec, h = cache
    q, k, v = _new()
    lens, pos, qo, ko = CTX + 1, torch.zeros(3, 4, dtype=torch.int32), torch.zeros_like(q), torch.zeros_like(k)
    rope = sfa.SfaRope()
    c.append(1, q, k, v, CTX, lens=lens, positions=pos, rope=rope, q_out=qo, k_out=ko)
    name, a = rec.calls[-1]
    assert name == "sfa_kv_append" and a[0] == 0xABC and a[2:11] == (
        1, 1, q.data_ptr(), k.data_ptr(), v.data_ptr(), 4, lens.data_ptr(), CTX.data_ptr(), pos.data_ptr())
    assert a[12:] == (3, qo.data_ptr(), ko.data_ptr(), 0x5151)
    mask, out = torch.zeros(3, 4, 1, dtype=torch.int32), torch.zeros(1, 3, 4, 256, dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    assert c.attend(0, q, CTX, lens=lens, mask=mask, out=out, workspace=ws) is out
    name, a = rec.calls[-1]
    assert name == "sfa_kv_attend" and a[2:] == (0, 1, q.data_ptr(), 4, lens.data_ptr(), CTX.data_ptr(), mask.data_ptr(), 3,
                                                 out.data_ptr(), ws.data_ptr(), 4096, 0x5151)
    c.accept(0, 2, pos, lens, CTX)
    name, a = rec.calls[-1]
    assert name == "sfa_kv_accept" and a[2:] == (0, 2, pos.data_ptr(), 4, lens.data_ptr(), CTX.data_ptr(), 3, 0x5151)
    sfa.sfa_tree_plan(h, pos, CTX, positions=pos, mask=mask)
    name, a = rec.calls[-1]
    assert name == "sfa_tree_plan" and a == (0xABC, pos.data_ptr(), 4, None, CTX.data_ptr(), 3, pos.data_ptr(),
                                             mask.data_ptr(), 0x5151)


@pytest.mark.parametrize("what", ["q_dtype", "q_heads", "k_rows", "v_strided", "ctx_dtype", "ctx_len", "lens_len",
                                  "pos_shape", "q_out_alone", "k_out_shape"])
def test_append_rejects_bad_tensors(cache, what):
    c, rec, _ = cache
    q, k, v = _new()
    kw, ctx = {}, CTX
    if what == "q_dtype":
        q = q.float()
    elif what == "q_heads":
        q = q[:, :, :, :2].contiguous()
    elif what == "k_rows":
        k = k[:, :2].contiguous()
    elif what == "v_strided":
        v = v.transpose(2, 3)
    elif what == "ctx_dtype":
        ctx = CTX.long()
    elif what == "ctx_len":
        ctx = CTX[:2]
    elif what == "lens_len":
        kw["lens"] = torch.zeros(4, dtype=torch.int32)
    elif what == "pos_shape":
        kw["positions"] = torch.zeros(3, 5, dtype=torch.int32)
    elif what == "q_out_alone":
        q, kw["q_out"] = None, _new()[0]
    elif what == "k_out_shape":
        kw["k_out"] = torch.zeros(1, 3, 5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        c.append(0, q, k, v, ctx, **kw)
    assert rec.calls == []


@pytest.mark.parametrize("what", ["out_dtype", "out_shape", "mask_words", "mask_dtype", "q_dims", "workspace_dtype"])
def test_attend_rejects_bad_tensors(cache, what):
    c, rec, _ = cache
    q, _, _ = _new()
    kw = {"out": torch.zeros(1, 3, 4, 256, dtype=torch.bfloat16), "mask": torch.zeros(3, 4, 1, dtype=torch.int32)}
    if what == "out_dtype":
        kw["out"] = kw["out"].float()
    elif what == "out_shape":
        kw["out"] = kw["out"][:, :, :3].contiguous()
    elif what == "mask_words":
        kw["mask"] = torch.zeros(3, 4, 2, dtype=torch.int32)
    elif what == "mask_dtype":
        kw["mask"] = kw["mask"].long()
    elif what == "q_dims":
        q = q[0]
    elif what == "workspace_dtype":
        kw["workspace"] = torch.zeros(4096, dtype=torch.float32)
    with pytest.raises(ValueError):
        c.attend(0, q, CTX, **kw)
    assert [n for n, _ in rec.calls if n == "sfa_kv_attend"] == []


@pytest.mark.parametrize("what", ["pages_dtype", "pages_dims", "heads", "v_shape", "table_dtype", "table_dims"])
def test_cache_rejects_bad_tensors(cache, what):
    _, _, h = cache
    k, v = (torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2))
    t = torch.zeros(3, 2, dtype=torch.int32)
    if what == "pages_dtype":
        k = k.float()
    elif what == "pages_dims":
        k = k[0]
    elif what == "heads":
        k = torch.zeros(2, 6, 3, 16, 64, dtype=torch.bfloat16)
    elif what == "v_shape":
        v = torch.zeros(2, 5, 2, 16, 64, dtype=torch.bfloat16)
    elif what == "table_dtype":
        t = t.long()
    elif what == "table_dims":
        t = t[0]
    with pytest.raises(ValueError):
        sfa.SfaPagedCache(h, k, v, t)
