"""NaN and infinities in the cache, in every kernel of the paged attention:
without influence on rows that do not see them, and what the formula says for
those that do (an infinite value times a positive weight)."""
import math
import random

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
import paged_reference as ref
from test_gpu_paged import Case, masks

pytestmark = pytest.mark.gpu

# rows of a call (new tokens x heads of a group): up to 64, one tile of 128, pairs of them, fp32
KERNELS = {
    "few": ("qwen05b", "bf16", [100, 30, 700], [6, 4, 1], 6, 16),
    "few, many results": ("qwen7b", "bf16", [130, 40, 500, 1, 0, 77, 260, 3], [9, 9, 2, 9, 8, 1, 9, 5], 9, 64),
    "one": ("qwen7b", "bf16", [100, 0, 255], [16, 12, 1], 16, 16),
    "one, long": ("mha", "bf16", [5000], [100], 100, 128),
    "pair": ("qwen7b", "bf16", [100, 37, 0], [40, 1, 33], 40, 16),
    "pair, many tiles": ("mqa", "bf16", [300, 20], [200, 150], 200, 64),
    "pair, long": ("qwen7b", "bf16", [6000], [40], 40, 64),
    "fp32": ("qwen05b", "f32", [100, 30], [6, 4], 6, 16),
    "fp32, rows": ("tiny", "f32", [70, 3], [90, 40], 90, 32),
}


class Cache(Case):
    def __init__(self, name, tree):
        shape, dtype, ctx, lens, n, page = KERNELS[name]
        super().__init__(shape, dtype, ctx, lens, n, page, seed=len(name) + tree)
        self.rows = masks(random.Random(n), lens, n) if tree else None
        self.mask = None
        if tree:
            self.mask = torch.stack([ref.pack_mask(r, (n + 31) // 32) for r in self.rows]).cuda()

    def sees(self, b, i, j):
        """Whether node i of sequence b sees new token j."""
        return j in self.rows[b][i] if self.rows else j <= i

    def run(self):
        nq, d = self.q.shape[3:]
        out = torch.full((1, len(self.ctx), self.n, nq * d), 7.0, device="cuda", dtype=self.q.dtype)
        self.cache.attend(0, self.q, self.ctx_d, lens=self.lens_d, mask=self.mask, out=out)
        assert sfa.sfa_check_device_status(self.h) == sfa.SFA_OK
        return out[0].view(len(self.ctx), self.n, nq, d)

    def at(self, pages, b, slot):
        """[n_kv, d] of a slot."""
        return pages[0, int(self.table[b, slot // self.page]), :, slot % self.page]


def same(got, want):
    return bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


@pytest.fixture(params=[False, True], ids=["causal", "tree"])
def tree(request):
    return request.param


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", KERNELS)
def test_what_no_row_sees(name, tree, bad):
    """Keys and values behind the last token, and in pages of others."""
    c = Cache(name, tree)
    clean = c.run()
    for b, (cx, ln) in enumerate(zip(c.ctx, c.lens)):
        for s in range(cx + ln, -(-(cx + ln) // c.page) * c.page):
            for pages in (c.k_pages, c.v_pages):
                c.at(pages, b, s).fill_(bad)
    for pg in c.spare:
        c.k_pages[:, pg] = bad
        c.v_pages[:, pg] = bad
    assert same(c.run(), clean)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", KERNELS)
def test_a_value_of_a_new_token(name, tree, bad):
    """One element of one KV head: the rows that see the token have it in that
    column, the others and all other columns are as before."""
    c = Cache(name, tree)
    want = c.run().clone()
    G = c.q.shape[3] // c.k_pages.shape[2]
    rng = random.Random(5)
    for b, ln in enumerate(c.lens):
        if ln == 0:
            continue
        j, kh, e = rng.randrange(ln), rng.randrange(c.k_pages.shape[2]), rng.randrange(c.q.shape[4])
        c.at(c.v_pages, b, c.ctx[b] + j)[kh, e] = bad
        for i in range(ln):
            if c.sees(b, i, j):
                want[b, i, kh * G:(kh + 1) * G, e] = bad
    assert same(c.run(), want)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", KERNELS)
def test_a_value_of_the_context(name, tree, bad):
    """Every row sees it; with its opposite in a new token the rows that see both
    have no number."""
    c = Cache(name, tree)
    want = c.run().clone()
    G = c.q.shape[3] // c.k_pages.shape[2]
    rng = random.Random(6)
    for b, ln in enumerate(c.lens):
        if ln == 0 or c.ctx[b] == 0:
            continue
        s, j, kh, e = rng.randrange(c.ctx[b]), rng.randrange(ln), rng.randrange(c.k_pages.shape[2]), rng.randrange(c.q.shape[4])
        c.at(c.v_pages, b, s)[kh, e] = bad
        c.at(c.v_pages, b, c.ctx[b] + j)[kh, e] = -bad
        for i in range(ln):
            want[b, i, kh * G:(kh + 1) * G, e] = math.nan if c.sees(b, i, j) else bad
    assert same(c.run(), want)


@pytest.mark.parametrize("name", KERNELS)
def test_keys_of_a_new_token(name, tree):
    """A key without a number: no row that sees it has one, the others are as
    before."""
    c = Cache(name, tree)
    want = c.run().clone()
    G = c.q.shape[3] // c.k_pages.shape[2]
    rng = random.Random(7)
    for b, ln in enumerate(c.lens):
        if ln == 0:
            continue
        j, kh = rng.randrange(ln), rng.randrange(c.k_pages.shape[2])
        c.at(c.k_pages, b, c.ctx[b] + j)[kh] = math.nan
        for i in range(ln):
            if c.sees(b, i, j):
                want[b, i, kh * G:(kh + 1) * G] = math.nan
    assert same(c.run(), want)
