"""Paged cache calls at the ends of their ranges: empty calls, large ragged
batches of chunks and single tokens, far contexts."""
import random

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
import paged_bound
import paged_reference as ref
from test_gpu_paged import Case, handle, ints

pytestmark = pytest.mark.gpu


def test_plan_refuses_positions_past_32_bits():
    h = handle("tiny", "f32")
    far = 2 ** 31 - 1
    pos, mask = sfa.sfa_tree_plan(h, ints([[-1, 0, 1]] * 3), ints([far - 3, far - 2, far]))
    assert sfa.sfa_check_device_status(h) == sfa.SFA_ERR_INVALID_ARG
    assert pos.tolist() == [[far - 3, far - 2, far - 1], [0] * 3, [0] * 3]
    assert mask[0, :, 0].tolist() == [1, 3, 7] and int(mask[1:].abs().sum()) == 0


@pytest.mark.parametrize("n", [1, 16, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_call_without_new_tokens(dtype, n):
    """Every sequence is empty: nothing is written, and the next call is whole."""
    c = Case("qwen7b", dtype, [300, 0, 40], [1, 0, 1], n, 16, seed=81)
    out = torch.full((1, 3, n, c.h.cfg.hidden), 9.0, device="cuda", dtype=c.q.dtype)
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    none = ints([0, 0, 0])
    c.cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=none, q_out=torch.zeros_like(c.q))
    c.cache.attend(0, c.q, c.ctx_d, lens=none, out=out)
    c.cache.accept(0, 1, torch.zeros(3, n, dtype=torch.int32, device="cuda"), none, c.ctx_d)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert bool((out == 9.0).all()) and torch.equal(c.k_pages, k0) and torch.equal(c.v_pages, v0)
    c.check()


@pytest.mark.parametrize("shape,dtype,B,chunk", [("qwen05b", "bf16", 256, 300), ("mqa", "bf16", 70, 700), ("tiny", "f32", 300, 500),
                                                 ("qwen05b", "bf16", 1200, 200)])
def test_chunks_and_single_tokens_in_one_call(shape, dtype, B, chunk):
    """A batch as a server makes it: some chunks of a prompt, single tokens, and
    sequences without new tokens."""
    rng = random.Random(B)
    lens = [rng.choice([1, 1, 1, 0]) for _ in range(B)]
    ctx = [rng.choice([0, 1, 63, 200]) for _ in range(B)]
    for b in (0, B // 2, B - 1):
        lens[b] = chunk - b % 3
    nq, nkv, d = {"qwen05b": (14, 2, 64), "mqa": (5, 1, 128), "tiny": (2, 2, 64)}[shape]
    c = Case(shape, dtype, ctx, lens, chunk, 32, seed=82)
    out = torch.full((1, B, chunk, nq * d), 9.0, device="cuda", dtype=c.q.dtype)
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    got, q, kp, vp, table = out.cpu(), c.q.cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu()
    for b in range(B):
        assert bool((got[0, b, lens[b]:] == 9.0).all())
        if lens[b]:
            w, bound = paged_bound.attend(q[:, b:b + 1, :lens[b]], kp, vp, table[b:b + 1], [ctx[b]], [lens[b]])
            ref.assert_within(got[:, b:b + 1, :lens[b]], w, bound, f"sequence {b}")
