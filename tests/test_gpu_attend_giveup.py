"""A bounded wait of the paged attention that runs out: the call reports it, ends,
and leaves the device and the handle fit for the next one."""
import time

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu

KERNELS = {
    "few": ("qwen05b", [1024], [1], 1, 16),
    "few, long": ("qwen7b", [9000, 400], [2, 1], 2, 64),
    "one": ("qwen7b", [3000, 100], [16, 12], 16, 16),
    "pair": ("qwen7b", [3000, 37], [60, 33], 60, 64),
}


@pytest.mark.parametrize("role", [9, 8, 10, 0, 4], ids=["products", "keys", "values", "softmax 0", "softmax 1"])
@pytest.mark.parametrize("name", KERNELS)
def test_a_wait_that_runs_out(name, role):
    shape, ctx, lens, n, page = KERNELS[name]
    c = Case(shape, "bf16", ctx, lens, n, page, seed=71)
    out = torch.zeros(1, len(ctx), n, c.h.cfg.hidden, device="cuda", dtype=torch.bfloat16)
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out)
    want = out.clone()
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    sfa.sfa_debug_set_wait_limit(c.h, spin_limit=2000, withhold_tile=role)
    t = time.time()
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_ERR_DEVICE_TIMEOUT
    assert time.time() - t < 5.0
    sfa.sfa_debug_set_wait_limit(c.h, 0, -1)
    for _ in range(3):
        out.zero_()
        c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out)
        assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
        assert torch.equal(out, want)
