"""The paged attention in bf16 is off by its result's rounding alone, in every
kernel and whatever else is in the call."""
import random

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
import paged_bound
import paged_reference as ref
from test_gpu_paged import Case, masks

pytestmark = pytest.mark.gpu


def _check(c, mask_rows=None):
    B, n = len(c.ctx), c.n
    mask = None
    if mask_rows is not None:
        mask = torch.stack([ref.pack_mask(mask_rows[b], (n + 31) // 32) for b in range(B)]).cuda()
    out = torch.full((c.q.shape[0], B, n, c.h.cfg.hidden), float("nan"), device="cuda", dtype=c.q.dtype)
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, mask=mask, out=out)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    want, bound = paged_bound.attend(c.q.cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu(), c.ctx, c.lens, mask_rows)
    ref.assert_within(out, want, bound, "attend")
    return out


@pytest.mark.parametrize("B", [1, 18, 19, 60])   # 896 values each: 16,384 lie between 18 and 19
def test_tokens_of_any_batch(B):
    rng = random.Random(B)
    _check(Case("qwen05b", "bf16", [rng.randint(300, 900) for _ in range(B)], [1] * B, 1, 16, seed=41))


@pytest.mark.parametrize("shape,ctx,lens,n,page", [
    ("wide", [500], [1], 1, 16),                                # 64 rows, 4,096 values
    ("wide", [500, 3], [2, 1], 2, 16),                          # one row tile of 128 rows
    ("qwen7b", [700, 90, 400], [9, 9, 2], 9, 64),               # 63 rows
    ("qwen7b", [700, 90, 400], [16, 16, 3], 16, 64),            # one row tile of 112 rows
    ("mha", [1000, 77], [128, 100], 128, 32),                   # one row tile, causal
    ("qwen7b", [700, 90], [40, 33], 40, 16),                    # pairs of row tiles
    ("mqa", [300, 12, 900], [200, 1, 150], 200, 128),
])
@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_kernels(shape, ctx, lens, n, page, kind):
    c = Case(shape, "bf16", ctx, lens, n, page, seed=42)
    _check(c, masks(random.Random(n), lens, n) if kind == "tree" else None)


def test_layers_in_one_call_and_one_by_one():
    """Three layers of ten new tokens: 53,760 values together, 17,920 a layer
    and 1,792 a token."""
    c = Case("qwen05b", "bf16", [70, 300], [10, 7], 10, 16, layers=3, seed=43)
    full = _check(c)
    for l in range(3):
        one = c.cache.attend(l, c.q[l:l + 1].contiguous(), c.ctx_d, lens=c.lens_d)
        want, bound = paged_bound.attend(c.q[l:l + 1].cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu(), c.ctx, c.lens,
                                         layer_begin=l)
        ref.assert_within(one, want, bound, "one layer")
    assert not torch.isnan(full[:, 0]).any()


def test_long_contexts():
    """Split over CTAs and joined."""
    _check(Case("qwen7b", "bf16", [20001, 5000], [2, 1], 2, 64, seed=44))
    _check(Case("mha", "bf16", [9000], [140], 140, 128, seed=45))
