"""Paged cache operators on the GPU against plain 64-bit forms: trees, append
with rotation, attention over the cache, accepted paths, and a run of them."""
import random

import pytest
import torch

import kv_cache_compression_sfa_b200 as sfa
import paged_reference as ref

pytestmark = pytest.mark.gpu

SHAPES = {"tiny": (2, 2, 64), "qwen05b": (14, 2, 64), "qwen7b": (28, 4, 128), "mqa": (5, 1, 128),
          "wide": (64, 1, 64), "mha": (4, 4, 128)}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def handle(shape, dtype, layers=1):
    nq, nkv, d = SHAPES[shape]
    cfg = sfa.SfaConfig(n_layers=layers, n_q_heads=nq, n_kv_heads=nkv, head_dim=d,
                        in_dtype=sfa.SFA_F32 if dtype == "f32" else sfa.SFA_BF16)
    return sfa.sfa_init(cfg, torch.zeros(layers, cfg.n_slots, cfg.hidden, device="cuda"))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A cache with random contents, scattered pages (-1 behind the last), and
    new tokens."""

    def __init__(self, shape, dtype, ctx, lens, n, page, layers=1, seed=0, scale=1.0):
        self.h = handle(shape, dtype, layers)
        nq, nkv, d = SHAPES[shape]
        self.ctx, self.lens, self.n, self.page = ctx, lens, n, page
        B = len(ctx)
        g = torch.Generator(device="cuda").manual_seed(seed)
        counts = [(c + l + page - 1) // page for c, l in zip(ctx, lens)]
        total = sum(counts) + 2
        ids = list(range(total))
        random.Random(seed).shuffle(ids)
        rows, at = [], 0
        for c in counts:
            rows.append(ids[at:at + c] + [-1] * (max(max(counts), 1) - c))
            at += c
        self.spare = ids[at:]
        self.table = ints(rows)
        mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") * scale).to(DT[dtype])  # noqa: E731
        self.k_pages, self.v_pages = mk(layers, total, nkv, page, d), mk(layers, total, nkv, page, d)
        self.q, self.k, self.v = mk(layers, B, n, nq, d), mk(layers, B, n, nkv, d), mk(layers, B, n, nkv, d)
        self.cache = sfa.SfaPagedCache(self.h, self.k_pages, self.v_pages, self.table)
        self.ctx_d, self.lens_d = ints(ctx), ints(lens)

    def attend(self, mask_rows=None, **kw):
        """(got, ref, bound) of attend on every layer."""
        B, n = len(self.ctx), self.n
        words = (n + 31) // 32
        mask = None
        if mask_rows is not None:
            mask = torch.stack([ref.pack_mask(mask_rows[b], words) for b in range(B)]).cuda()
        L, nq, d = self.q.shape[0], self.q.shape[3], self.q.shape[4]
        out = torch.full((L, B, n, nq * d), float("nan"), device="cuda", dtype=self.q.dtype)
        self.cache.attend(0, self.q, self.ctx_d, lens=self.lens_d, mask=mask, out=out, **kw)
        assert sfa.sfa_check_device_status(self.h) == sfa.SFA_OK
        see = (lambda b, i: None) if mask_rows is None else (lambda b, i: mask_rows[b][i])
        r, bound = ref.attend(self.q.cpu(), self.k_pages.cpu(), self.v_pages.cpu(), self.table.cpu(), self.ctx,
                              self.lens, see)
        return out, r, bound

    def check(self, mask_rows=None, what="attend", **kw):
        out, r, bound = self.attend(mask_rows, **kw)
        ref.assert_within(out, r, bound, what)
        rows = torch.isnan(r).all(-1)
        assert torch.isnan(out.cpu()[rows]).all(), "rows past the sequence were written"
        return out


def tree(rng, n, reach=4):
    return [-1] + [rng.randint(max(-1, i - reach), i - 1) for i in range(1, n)]


def masks(rng, lens, n):
    """Ancestor sets of random trees, padded to n rows."""
    out = []
    for l in lens:
        a = ref.ancestors(tree(rng, max(l, 1)))
        out.append(a + [set()] * (n - len(a)))
    return out


# ------------------------------------------------------------------- plan


@pytest.mark.parametrize("n,lens", [(1, [1, 0]), (7, [7, 3, 0]), (32, [32, 31]), (33, [33, 1]), (64, [64, 40]),
                                    (1024, [1024, 700])])
@pytest.mark.parametrize("kind", ["random", "chain", "flat", "forest"])
def test_tree_plan(n, lens, kind):
    h = handle("tiny", "f32")
    rng = random.Random(n)
    rows = []
    for l in lens:
        if kind == "chain":
            p = list(range(-1, n - 1))
        elif kind == "flat":
            p = [-1] + [0] * (n - 1)
        elif kind == "forest":
            p = [-1 if rng.random() < 0.3 else rng.randint(-1, i - 1) for i in range(n)]
        else:
            p = tree(rng, n)
        rows.append(p[:l] + [12345] * (n - l))      # rows past the length are not looked at
    ctx = [5 * b + 3 for b in range(len(lens))]
    words = (n + 31) // 32
    pos = torch.full((len(lens), n), -7, dtype=torch.int32, device="cuda")
    mask = torch.full((len(lens), n, words), -7, dtype=torch.int32, device="cuda")
    sfa.sfa_tree_plan(h, ints(rows), ints(ctx), lens=ints(lens), positions=pos, mask=mask)
    assert sfa.sfa_check_device_status(h) == sfa.SFA_OK
    for b, l in enumerate(lens):
        a = ref.ancestors(rows[b][:l])
        want = torch.full((n,), -7, dtype=torch.int32)
        wm = torch.full((n, words), -7, dtype=torch.int32)
        if l:
            want[:l] = torch.tensor([ctx[b] + len(s) - 1 for s in a], dtype=torch.int32)
            wm[:l] = ref.pack_mask(a, words)
        assert torch.equal(pos[b].cpu(), want)
        assert torch.equal(mask[b].cpu(), wm)


def test_tree_plan_without_lens_and_new_outputs():
    h = handle("tiny", "f32")
    pos, mask = sfa.sfa_tree_plan(h, ints([[-1, 0, 0, 2]]), ints([10]))
    assert pos.tolist() == [[10, 11, 11, 12]] and mask[0, :, 0].tolist() == [1, 3, 5, 13]


def test_tree_plan_latches_bad_sequences_and_serves_the_others():
    h = handle("tiny", "f32")
    parents = ints([[-1, 1, 0], [-1, 0, 1], [-2, 0, 1], [-1, 0, 1], [-1, 0, 1]])
    pos, mask = sfa.sfa_tree_plan(h, parents, ints([0, 0, 0, -1, 0]), lens=ints([3, 3, 3, 3, 4]))
    assert sfa.sfa_check_device_status(h) == sfa.SFA_ERR_INVALID_ARG
    assert sfa.sfa_check_device_status(h) == sfa.SFA_OK
    assert pos.tolist() == [[0] * 3, [0, 1, 2], [0] * 3, [0] * 3, [0] * 3]
    assert mask[1, :, 0].tolist() == [1, 3, 7] and int(mask[[0, 2, 3, 4]].abs().sum()) == 0


# ----------------------------------------------------------------- append


@pytest.mark.parametrize("shape,dtype", [("tiny", "f32"), ("qwen05b", "bf16"), ("qwen7b", "bf16"), ("qwen7b", "f32"),
                                         ("mqa", "bf16")])
@pytest.mark.parametrize("style,dims,page,layers", [(0, 0, 16, 2), (1, 0, 8, 1), (0, 16, 64, 1), (1, 48, 256, 3),
                                                    (None, 0, 32, 1)])
def test_append(shape, dtype, style, dims, page, layers):
    ctx, lens, n = [0, 5, 100, 7, 31], [9, 1, 0, 4, 9], 9
    c = Case(shape, dtype, ctx, lens, n, page, layers=layers, seed=3)
    nq, nkv, d = SHAPES[shape]
    rng = random.Random(4)
    pos = [[rng.choice([0, 1, 77, 131072, 1_000_003]) + i for i in range(n)] for _ in ctx] if style == 1 else None
    dm = dims or d
    freqs = [1e6 ** (-2.0 * j / dm) for j in range(dm // 2)] if style != 1 else [0.9 ** j for j in range(dm // 2)]
    rope = None if style is None else (sfa.SfaRope(base=1e6, style=style, dims=dims) if style == 0
                                       else sfa.SfaRope(style=style, dims=dims, inv_freq=freqs))
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    qo, ko = torch.full_like(c.q, 9.0), torch.full_like(c.k, 9.0)
    got = c.cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=c.lens_d, positions=None if pos is None else ints(pos),
                         rope=rope, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    half = ref.HALF[DT[dtype]]
    p = torch.tensor(pos) if pos else torch.tensor(ctx)[:, None] + torch.arange(n)
    outs = []
    for x, y in ((c.q, qo), (c.k, ko)):
        r, e = x.cpu().double(), torch.zeros(x.shape, dtype=torch.float64)
        if rope is not None:
            r, e = ref.rotate(r, p[None].expand(layers, -1, -1), freqs, dm, style)
        live = (torch.arange(n) < torch.tensor(lens)[:, None])[None, :, :, None, None]
        bound = e + half * (r.abs() + e) if rope is not None else e
        ref.assert_within(y, torch.where(live, r, 9.0), torch.where(live, bound, 0.0), "rotated")
        outs.append(y)
    want_k, want_v = k0.clone(), v0.clone()
    for b, (cx, ln) in enumerate(zip(ctx, lens)):
        for i in range(ln):
            s = cx + i
            pg = int(c.table[b, s // page])
            want_k[:, pg, :, s % page] = outs[1][:, b, i]   # the cache holds the same rounded keys
            want_v[:, pg, :, s % page] = c.v[:, b, i]
    assert torch.equal(c.k_pages, want_k) and torch.equal(c.v_pages, want_v)


def test_append_in_place_and_without_queries():
    c = Case("qwen05b", "bf16", [3, 20], [4, 4], 4, 16, seed=5)
    rope = sfa.SfaRope(base=1e4)
    q1, k1 = torch.empty_like(c.q), torch.empty_like(c.k)
    c.cache.append(0, c.q, c.k, c.v, c.ctx_d, rope=rope, q_out=q1, k_out=k1)
    kp, vp = c.k_pages.clone(), c.v_pages.clone()
    q2, k2 = c.q.clone(), c.k.clone()
    c.cache.append(0, q2, k2, c.v, c.ctx_d, rope=rope, q_out=q2, k_out=k2)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)
    assert torch.equal(kp, c.k_pages) and torch.equal(vp, c.v_pages)
    c.k_pages.zero_()
    assert c.cache.append(0, None, c.k, c.v, c.ctx_d, rope=rope) == (None, None)
    for b in range(2):
        for i in range(4):
            s = c.ctx[b] + i
            assert torch.equal(c.k_pages[:, int(c.table[b, s // 16]), :, s % 16], k1[:, b, i])


def test_append_serves_a_layer_range():
    c = Case("tiny", "f32", [3], [5], 5, 8, layers=3, seed=6)
    k0 = c.k_pages.clone()
    c.cache.append(1, c.q[:1].contiguous(), c.k[:1].contiguous(), c.v[:1].contiguous(), c.ctx_d)
    assert torch.equal(c.k_pages[0], k0[0]) and torch.equal(c.k_pages[2], k0[2]) and not torch.equal(c.k_pages[1], k0[1])


def test_append_skips_bad_sequences_and_pages():
    c = Case("tiny", "f32", [3, 3, 3, 3], [2, 2, 2, 2], 2, 8, seed=7)
    c.table[1, 0] = 10 ** 6          # page out of range: not written
    kp, vp = c.k_pages.clone(), c.v_pages.clone()
    qo = torch.full_like(c.q, 9.0)
    c.cache.append(0, c.q, c.k, c.v, ints([3, 3, -1, 7]), lens=ints([2, 2, 2, 2]), q_out=qo)   # 7 + 2 > one page of 8
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_ERR_INVALID_ARG
    pg = int(c.table[0, 0])
    kp[:, pg, :, 3:5] = c.k[:, 0].transpose(1, 2)
    vp[:, pg, :, 3:5] = c.v[:, 0].transpose(1, 2)
    assert torch.equal(c.k_pages, kp) and torch.equal(c.v_pages, vp)
    assert torch.equal(qo[:, :2], c.q[:, :2]) and bool((qo[:, 2:] == 9.0).all())


# ----------------------------------------------------------------- attend


@pytest.mark.parametrize("shape,dtype", [("tiny", "f32"), ("qwen05b", "bf16"), ("qwen7b", "bf16"), ("qwen7b", "f32"),
                                         ("mqa", "bf16"), ("wide", "bf16"), ("mha", "bf16"), ("wide", "f32")])
@pytest.mark.parametrize("ctx,lens,n,page", [
    ([0], [1], 1, 8),                                   # the first token
    ([1, 63, 64, 127, 128, 129], [1] * 6, 1, 16),       # around the tiles
    ([0, 5, 300, 17], [5, 0, 3, 5], 5, 32),             # ragged, one without new tokens
    ([255, 256, 0], [17, 1, 2], 17, 256),
])
def test_attend_causal(shape, dtype, ctx, lens, n, page):
    Case(shape, dtype, ctx, lens, n, page, seed=11).check()


@pytest.mark.parametrize("shape,dtype", [("tiny", "f32"), ("qwen05b", "bf16"), ("qwen7b", "bf16"), ("mqa", "f32"),
                                         ("wide", "bf16")])
@pytest.mark.parametrize("ctx,lens,n,page", [
    ([0, 40, 126], [7, 3, 7], 7, 8),
    ([100, 0, 3, 1000], [33, 32, 1, 20], 33, 64),
    ([120, 5], [64, 70], 70, 128),
])
def test_attend_tree(shape, dtype, ctx, lens, n, page):
    c = Case(shape, dtype, ctx, lens, n, page, seed=12)
    c.check(masks(random.Random(n), lens, n))


@pytest.mark.parametrize("shape,dtype,ctx,lens,n,page", [
    ("qwen7b", "bf16", [300, 0, 17], [200, 130, 1], 200, 64),      # several row tiles, causal
    ("qwen05b", "bf16", [1000], [150], 150, 16),
    ("tiny", "f32", [100, 3], [130, 129], 130, 32),
    ("mqa", "bf16", [30, 0, 300, 9, 700], [500, 470, 1, 0, 333], 500, 64),   # many row tiles
    ("tiny", "f32", [100, 0, 5], [600, 577, 3], 600, 32),
])
def test_attend_chunk(shape, dtype, ctx, lens, n, page):
    Case(shape, dtype, ctx, lens, n, page, seed=13).check()


@pytest.mark.parametrize("shape,dtype,ctx", [("qwen7b", "bf16", [20001]), ("qwen05b", "bf16", [9000, 3, 12345]),
                                             ("tiny", "f32", [20000])])
def test_attend_long_context_is_split_and_joined(shape, dtype, ctx):
    c = Case(shape, dtype, ctx, [2] * len(ctx), 2, 64, seed=14)
    a = c.check()
    b = c.check()
    assert torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)]), "two runs differ"


def test_attend_many_sequences():
    rng = random.Random(15)
    B = 300
    ctx = [rng.choice([0, 1, 2, 50, 200]) for _ in range(B)]
    lens = [rng.randint(0, 2) for _ in range(B)]
    Case("tiny", "f32", ctx, lens, 2, 16, seed=15).check()
    Case("qwen05b", "bf16", ctx, lens, 2, 16, seed=15).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_layers(dtype):
    c = Case("qwen05b", dtype, [70, 5], [3, 2], 3, 16, layers=3, seed=16)
    full = c.check()
    one = c.cache.attend(1, c.q[1:2].contiguous(), c.ctx_d, lens=c.lens_d)
    ok = ~torch.isnan(full[1:2])
    assert torch.equal(one[ok], full[1:2][ok])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_rows_that_see_nothing_are_zero(dtype):
    c = Case("qwen05b", dtype, [0, 0, 200], [4, 3, 4], 4, 16, seed=17)
    rows = [[set(), {0}, set(), {0, 1, 2, 3}], [set()] * 4, [set(), {3}, {0}, set()]]
    out = c.check(rows)
    assert int((out[0, 0, 0] != 0).sum()) == 0 and int((out[0, 1, :3] != 0).sum()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attend_unseen_keys_and_values_have_no_influence(dtype, bad):
    """NaN and infinities behind the sequence's last token, and in new tokens
    that a node does not see."""
    c = Case("qwen05b", dtype, [100, 30], [6, 4], 6, 16, seed=18)
    rows = [[{i} for i in range(6)], [{0}, {0, 1}, {0, 2}, {0, 1, 3}] + [set()] * 2]
    clean = c.check(rows)
    for b, (cx, ln) in enumerate(zip(c.ctx, c.lens)):
        for s in range(cx + ln, ((cx + ln + 15) // 16) * 16):    # the rest of the last page
            pg = int(c.table[b, s // 16])
            c.k_pages[:, pg, :, s % 16] = bad
            c.v_pages[:, pg, :, s % 16] = bad
    for pg in c.spare:
        c.k_pages[:, pg] = bad
        c.v_pages[:, pg] = bad
    for b, j in ((0, 2), (1, 3)):                                 # a new token: only its own row sees it
        s = c.ctx[b] + j
        pg = int(c.table[b, s // 16])
        c.k_pages[:, pg, :, s % 16] = bad
        c.v_pages[:, pg, :, s % 16, 0] = bad
    words = 1
    mask = torch.stack([ref.pack_mask(rows[b], words) for b in range(2)]).cuda()
    out = torch.full_like(clean, float("nan"))
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, mask=mask, out=out)
    same = torch.ones(2, 6, dtype=torch.bool)
    same[0, 2] = same[1, 3] = same[1, 4] = same[1, 5] = False
    assert torch.equal(out[0][same], clean[0][same])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_large_scores(dtype):
    """Scores of several hundred: one key takes all the weight."""
    Case("qwen7b", dtype, [500, 40], [3, 3], 3, 16, seed=19, scale=6.0).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_rising_scores(dtype):
    """Keys that grow along the sequence move the running maximum in every tile."""
    c = Case("qwen05b", dtype, [2000], [2], 2, 16, seed=20)
    slots = torch.arange(2002)
    pg = c.table[0, (slots // 16)].long()
    c.q.abs_()
    for s, p in zip(slots.tolist(), pg.tolist()):
        c.k_pages[:, p, :, s % 16] = c.k_pages[:, p, :, s % 16].abs() * (s / 500.0)
    c.check()


def test_attend_skips_bad_sequences_and_reads_bad_pages_as_zero():
    c = Case("qwen05b", "bf16", [20, 20, 20, 20], [2, 2, 2, 2], 2, 16, seed=21)
    out = torch.full((1, 4, 2, c.h.cfg.hidden), 9.0, device="cuda", dtype=torch.bfloat16)
    good = c.cache.attend(0, c.q, c.ctx_d)
    c.table[1, 1] = -5
    c.cache.attend(0, c.q, ints([20, 20, -1, 31]), lens=ints([2, 2, 2, 2]), out=out)   # 31 + 2 > two pages
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_ERR_INVALID_ARG
    assert torch.equal(out[:, 0], good[:, 0]) and bool((out[:, 2:] == 9.0).all())
    assert bool(torch.isfinite(out).all())


def test_attend_on_a_stream_and_in_a_graph():
    c = Case("qwen7b", "bf16", [700, 1], [3, 2], 3, 16, seed=22)
    want = c.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d, out=out, stream=s)
    s.synchronize()
    ok = ~torch.isnan(want)
    assert torch.equal(out[ok], want[ok])
    ws = torch.empty(sfa.sfa_kv_attend_workspace_bytes(c.h, c.n), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    rope = sfa.SfaRope()
    qr = torch.zeros_like(c.q)
    with torch.cuda.graph(g):
        c.cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=c.lens_d, rope=rope, q_out=qr)
        c.cache.attend(0, qr, c.ctx_d, lens=c.lens_d, out=out, workspace=ws)
    for ctx in ([650, 4], [10, 17]):          # other lengths, the same graph
        c.ctx_d.copy_(ints(ctx))
        c.table[1, :2] = torch.tensor([c.spare[0], c.spare[1]], dtype=torch.int32)
        g.replay()
        qe = torch.zeros_like(c.q)
        c.cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=c.lens_d, rope=rope, q_out=qe)
        eager = c.cache.attend(0, qe, c.ctx_d, lens=c.lens_d)
        assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
        assert torch.equal(out[:, 0, :3], eager[:, 0, :3]) and torch.equal(out[:, 1, :2], eager[:, 1, :2])


def test_attend_on_two_streams_at_once():
    a = Case("qwen7b", "bf16", [3000, 20], [2, 1], 2, 16, seed=25)
    b_q = torch.randn_like(a.q)
    want = [a.cache.attend(0, q, a.ctx_d, lens=a.lens_d) for q in (a.q, b_q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, o in zip(streams, (a.q, b_q), outs):
            a.cache.attend(0, q, a.ctx_d, lens=a.lens_d, out=o, stream=s)
    torch.cuda.synchronize()
    assert sfa.sfa_check_device_status(a.h) == sfa.SFA_OK
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_attend_shared_prefix_pages():
    """Two sequences whose first pages are the same."""
    c = Case("qwen05b", "bf16", [64, 64], [3, 3], 3, 16, seed=26)
    c.table[1, :4] = c.table[0, :4]
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_queries_reach_their_own_row_alone(dtype):
    c = Case("qwen05b", dtype, [200, 9], [3, 3], 3, 16, seed=27)
    clean = c.check()
    c.q[0, 0, 1, 4] = float("nan")
    out = c.cache.attend(0, c.q, c.ctx_d, lens=c.lens_d)
    d = 64
    assert torch.isnan(out[0, 0, 1, 4 * d:5 * d]).all()
    out[0, 0, 1, 4 * d:5 * d] = clean[0, 0, 1, 4 * d:5 * d]
    assert torch.equal(out, clean)


# ---------------------------------------------------------------- refusals


def test_calls_refuse_before_any_launch():
    import ctypes
    c = Case("qwen05b", "bf16", [5, 6], [2, 2], 2, 16, layers=2, seed=28)
    lib, h = sfa.load_library(), c.h.ptr
    P = lambda t: t.data_ptr()  # noqa: E731
    ws = torch.empty(sfa.sfa_kv_attend_workspace_bytes(c.h, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, 2, 2, c.h.cfg.hidden, dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in (c.k_pages, c.v_pages, out)]

    def cache(**kw):
        x = dict(k_pages=P(c.k_pages), v_pages=P(c.v_pages), n_pages=c.k_pages.shape[1], page_size=16,
                 max_pages=c.table.shape[1], page_table=P(c.table))
        x.update(kw)
        return ctypes.byref(sfa.sfa_kv_cache(*[x[f] for f, _ in sfa.sfa_kv_cache._fields_]))

    def attend(cc=None, l0=0, lc=2, q=P(c.q), n=2, ctx=P(c.ctx_d), mask=None, B=2, o=P(out), w=P(ws), wb=ws.numel(), hh=h):
        return lib.sfa_kv_attend(hh, cc or cache(), l0, lc, q, n, None, ctx, mask, B, o, w, wb, None)

    def append(cc=None, l0=0, lc=2, q=P(c.q), k=P(c.k), v=P(c.v), n=2, rope=None, B=2, qo=P(c.q), ko=None):
        return lib.sfa_kv_append(h, cc or cache(), l0, lc, q, k, v, n, None, P(c.ctx_d), None,
                                 None if rope is None else ctypes.byref(rope.c), B, qo, ko, None)

    def accept(cc=None, l0=0, lc=2, path=P(c.table), n=1, na=P(c.lens_d), B=2):
        return lib.sfa_kv_accept(h, cc or cache(), l0, lc, path, n, na, P(c.ctx_d), B, None)

    inv, ali, uns, wsp = sfa.SFA_ERR_INVALID_ARG, sfa.SFA_ERR_ALIGNMENT, sfa.SFA_ERR_UNSUPPORTED, sfa.SFA_ERR_WORKSPACE
    for call in (attend, append, accept):
        for kw in (dict(l0=-1), dict(l0=1), dict(lc=0), dict(lc=3), dict(l0=2 ** 31 - 1, lc=2), dict(n=-1), dict(B=0)):
            assert call(**kw) == inv, (call, kw)
        for kw in (dict(k_pages=None), dict(v_pages=None), dict(page_table=None), dict(page_size=0), dict(n_pages=0),
                   dict(max_pages=0)):
            assert call(cc=cache(**kw)) == inv, (call, kw)
        assert call(cc=cache(k_pages=P(c.k_pages) + 8)) == ali
        for kw in (dict(page_size=4), dict(page_size=24), dict(page_size=512), dict(n_pages=2 ** 31), dict(n_pages=2 ** 29),
                   dict(max_pages=2 ** 26 + 1)):
            assert call(cc=cache(**kw)) == uns, (call, kw)
        assert call(n=0) == sfa.SFA_OK
    assert attend(q=None) == inv and attend(o=None) == inv and attend(ctx=None) == inv and attend(hh=None) == inv
    assert attend(q=P(c.q) + 2) == ali and attend(w=P(ws) + 4) == ali
    assert attend(w=None) == wsp and attend(wb=ws.numel() - 1) == wsp
    assert attend(n=1025, mask=P(c.table)) == uns and attend(B=4097) == uns and attend(n=2 ** 30) == uns
    assert append(k=None) == inv and append(v=None) == inv and append(q=None) == inv and append(qo=None) == inv
    assert append(ko=P(c.k) + 2) == ali and append(n=2 ** 30) == uns
    for rope, code in ((sfa.SfaRope(style=2), inv), (sfa.SfaRope(dims=8), inv), (sfa.SfaRope(dims=80), inv),
                       (sfa.SfaRope(base=0.0), inv), (sfa.SfaRope(base=float("inf")), inv),
                       (sfa.SfaRope(inv_freq=[float("nan")] * 32), inv)):
        assert append(rope=rope) == code
    assert accept(path=None) == inv and accept(na=None) == inv and accept(n=1025) == uns
    one = torch.zeros(2, 1025, dtype=torch.int32, device="cuda")
    assert lib.sfa_tree_plan(h, P(one), 1025, None, P(c.ctx_d), 2, P(one), None, None) == uns
    assert lib.sfa_tree_plan(h, P(one), 2, None, P(c.ctx_d), 2, None, None, None) == inv
    assert lib.sfa_tree_plan(h, None, 2, None, P(c.ctx_d), 2, P(one), None, None) == inv
    assert lib.sfa_tree_plan(h, P(one), 2, None, None, 2, P(one), None, None) == inv
    assert sfa.sfa_kv_attend_workspace_bytes(c.h, 0) == 0
    torch.cuda.synchronize()
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k_pages, c.v_pages, out)))


def test_binding_refuses_and_takes_empty_calls():
    c = Case("qwen05b", "bf16", [5, 6], [2, 2], 2, 16, seed=29)
    with pytest.raises(ValueError):
        c.cache.attend(0, c.q.float(), c.ctx_d)
    with pytest.raises(ValueError):
        c.cache.attend(0, c.q.cpu(), c.ctx_d)
    with pytest.raises(ValueError):
        c.cache.attend(0, c.q, c.ctx_d.cpu(), out=torch.zeros(1, 2, 2, 896, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        c.cache.append(0, c.q, c.k, c.v.transpose(3, 4), c.ctx_d, q_out=c.q)
    with pytest.raises(ValueError):
        c.cache.accept(0, 1, c.ctx_d[:, None].long(), c.lens_d, c.ctx_d)
    with pytest.raises(sfa.SfaError):
        c.cache.attend(1, c.q, c.ctx_d)
    assert c.cache.attend(0, c.q[:, :, :0].contiguous(), c.ctx_d).shape == (1, 2, 0, 896)
    c.cache.append(0, c.q[:, :, :0].contiguous(), c.k[:, :, :0].contiguous(), c.v[:, :, :0].contiguous(), c.ctx_d)
    c.cache.accept(0, 1, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), ints([0, 0]), c.ctx_d)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK


@pytest.mark.skipif(sfa._fast is None, reason="the extension is not built")
def test_extension_and_ctypes_paths_agree(monkeypatch):
    c = Case("qwen05b", "bf16", [50, 6], [3, 2], 3, 16, seed=30)
    rope = sfa.SfaRope()
    runs = []
    for fast in (True, False):
        if not fast:
            monkeypatch.setattr(sfa, "_fast", None)
        cache = sfa.SfaPagedCache(c.h, c.k_pages.clone(), c.v_pages.clone(), c.table)
        assert (cache._spec is not None) == fast
        qo, out = torch.zeros_like(c.q), torch.zeros(1, 2, 3, 896, dtype=torch.bfloat16, device="cuda")
        pos, mask = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, 1, dtype=torch.int32, device="cuda")
        sfa.sfa_tree_plan(c.h, ints([[-1, 0, 0], [-1, 0, 1]]), c.ctx_d, lens=c.lens_d, positions=pos, mask=mask)
        cache.append(0, c.q, c.k, c.v, c.ctx_d, lens=c.lens_d, positions=pos, rope=rope, q_out=qo)
        cache.attend(0, qo, c.ctx_d, lens=c.lens_d, mask=mask, out=out)
        cache.accept(0, 1, ints([[0, 2, 0], [1, 0, 0]]), ints([2, 1]), c.ctx_d)
        runs.append([pos, mask, qo, out, cache.k_pages, cache.v_pages])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ----------------------------------------------------------------- accept


@pytest.mark.parametrize("shape,dtype", [("tiny", "f32"), ("qwen05b", "bf16"), ("qwen7b", "bf16")])
@pytest.mark.parametrize("page", [8, 64])
def test_accept(shape, dtype, page):
    n = 40
    ctx = [0, 5, 61, 100, 7]
    paths = [[0, 1, 2], [3, 7, 8, 39], [], list(range(1, 40, 2)), list(range(20, 40))]   # sources that are destinations too
    c = Case(shape, dtype, ctx, [n] * 5, n, page, layers=2, seed=23)
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    c.cache.accept(0, 2, ints([p + [0] * (n - len(p)) for p in paths]), ints([len(p) for p in paths]), c.ctx_d)
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_OK
    wk, wv = k0.clone(), v0.clone()
    at = lambda b, s: (int(c.table[b, s // page]), s % page)  # noqa: E731
    for b, p in enumerate(paths):
        for i, s in enumerate(p):
            (sp, sr), (dp, dr) = at(b, ctx[b] + s), at(b, ctx[b] + i)
            wk[:, dp, :, dr] = k0[:, sp, :, sr]
            wv[:, dp, :, dr] = v0[:, sp, :, sr]
    assert torch.equal(c.k_pages, wk) and torch.equal(c.v_pages, wv)


def test_accept_skips_bad_paths():
    c = Case("tiny", "f32", [3] * 6, [6] * 6, 6, 8, seed=24)
    k0 = c.k_pages.clone()
    paths = [[2, 2, 3], [3, 1, 4], [-1, 2, 3], [1, 2, 6], [1, 2, 3], [1, 2, 3]]
    c.cache.accept(0, 1, ints([p + [0] * 3 for p in paths]), ints([3, 3, 3, 3, 7, 3]), ints([3, 3, 3, 3, 3, -2]))
    assert sfa.sfa_check_device_status(c.h) == sfa.SFA_ERR_INVALID_ARG
    assert torch.equal(c.k_pages, k0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_whose_offsets_pass_32_bits(dtype):
    """Page ids whose element offsets are above 2^31 (bytes above 2^32), in
    every call."""
    nq, nkv, d = SHAPES["qwen7b"]
    h = handle("qwen7b", dtype)
    page, n_pages = 256, 2 ** 31 // (nkv * 256 * d) + 40
    k_pages, v_pages = (torch.empty(1, n_pages, nkv, page, d, device="cuda", dtype=DT[dtype]) for _ in range(2))
    ids = [n_pages - 1, 3, n_pages - 30, n_pages - 7]
    g = torch.Generator(device="cuda").manual_seed(33)
    for p in ids:
        k_pages[:, p].normal_(generator=g)
        v_pages[:, p].normal_(generator=g)
    low = [torch.stack([x[:, p] for p in ids], 1) for x in (k_pages, v_pages)]     # the same pages in a small cache
    big = sfa.SfaPagedCache(h, k_pages, v_pages, ints([ids[:2], ids[2:]]))
    small = sfa.SfaPagedCache(h, *low, ints([[0, 1], [2, 3]]))
    q = torch.randn(1, 2, 5, nq, d, generator=g, device="cuda").to(DT[dtype])
    k, v = (torch.randn(1, 2, 5, nkv, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    ctx = ints([300, 254])
    outs = []
    for c in (big, small):
        qr, _ = c.append(0, q, k, v, ctx, rope=sfa.SfaRope())
        out = c.attend(0, qr, ctx)
        c.accept(0, 1, ints([[1, 3, 4, 0, 0], [0, 2, 4, 0, 0]]), ints([3, 3]), ctx)
        outs.append((qr, out))
    assert sfa.sfa_check_device_status(h) == sfa.SFA_OK
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for x, y in ((k_pages, low[0]), (v_pages, low[1])):
        assert all(torch.equal(x[:, p], y[:, i]) for i, p in enumerate(ids))


# --------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_drafted_step_as_it_is_used(dtype):
    """Prompt in by append and attend, a tree planned, appended and attended,
    one path accepted, and the SFA enhancement of the accepted tokens added to
    their exact attention: every tree node's output is the output of a plain
    step over its own path, and the cache after accept is the cache of that
    path."""
    nq, nkv, d = SHAPES["qwen05b"]
    layers, B, page, n = 2, 2, 16, 12
    h = handle("qwen05b", dtype, layers)
    T = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(31)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(T)  # noqa: E731
    pool = lambda: torch.zeros(layers, 12, nkv, page, d, device="cuda", dtype=T)  # noqa: E731
    tree_cache = sfa.SfaPagedCache(h, pool(), pool(), ints([[0, 2, 4, 6], [11, 9, 7, 5]]))
    path_cache = sfa.SfaPagedCache(h, pool(), pool(), ints([[1, 3, 5, 7], [0, 2, 4, 6]]))
    rope = sfa.SfaRope(base=1e6)
    prompt, lens = [21, 9], ints([21, 9])
    ctx = ints([0, 0])
    q, k, v = mk(layers, B, 21, nq, d), mk(layers, B, 21, nkv, d), mk(layers, B, 21, nkv, d)
    for c in (tree_cache, path_cache):
        qr, _ = c.append(0, q, k, v, ctx, lens=lens, rope=rope)
        c.attend(0, qr, ctx, lens=lens)
    ctx = lens.clone()
    parents = [[-1, 0, 0, 1, 1, 2, 3, 3, 5, 6, 6, 8], [-1, 0, 1, 1, 0, 4, 4, 5, 2, 2, 9, 10]]
    path = [[0, 1, 3, 6, 10], [0, 4, 5]]
    pos, mask = sfa.sfa_tree_plan(h, ints(parents), ctx)
    q, k, v = mk(layers, B, n, nq, d), mk(layers, B, n, nkv, d), mk(layers, B, n, nkv, d)
    k_out = torch.empty_like(k)
    qr, _ = tree_cache.append(0, q, k, v, ctx, positions=pos, rope=rope, k_out=k_out)
    out = tree_cache.attend(0, qr, ctx, mask=mask)
    idx = torch.zeros(B, 5, dtype=torch.long, device="cuda")
    for b in range(B):
        idx[b, :len(path[b])] = torch.tensor(path[b])
    take = lambda x: torch.stack([x[:, b, idx[b]] for b in range(B)], 1).contiguous()  # noqa: E731
    n_acc = ints([5, 3])
    qp, _ = path_cache.append(0, take(q), take(k), take(v), ctx, lens=n_acc, rope=rope)
    plain = path_cache.attend(0, qp, ctx, lens=n_acc)
    for b in range(B):
        m = len(path[b])
        assert torch.equal(qp[:, b, :m], take(qr)[:, b, :m])
        # the same keys in another order of slots: the bound of both results
        r, bound = ref.attend(take(qr)[:, b:b + 1, :m].cpu(), path_cache.k_pages.cpu(), path_cache.v_pages.cpu(),
                              path_cache.page_table[b:b + 1].cpu(), [prompt[b]], [m], lambda b_, i: None)
        ref.assert_within(take(out)[:, b:b + 1, :m], r, bound, "tree")
        ref.assert_within(plain[:, b:b + 1, :m], r, bound, "path")
    tree_cache.accept(0, layers, torch.nn.functional.pad(idx, (0, n - 5)).to(torch.int32), n_acc, ctx)
    for b in range(B):
        m = prompt[b] + len(path[b])
        for x, y in ((tree_cache.k_pages, path_cache.k_pages), (tree_cache.v_pages, path_cache.v_pages)):
            for layer in range(layers):
                assert torch.equal(ref.gather(x, layer, tree_cache.page_table[b], m),
                                   ref.gather(y, layer, path_cache.page_table[b], m))
    # the accepted tokens enter the SFA state, whose enhancement is added to their attention
    slots = torch.randn(layers, 64, nq * d, generator=g, device="cuda")
    cfg = h.cfg
    op = sfa.SfaOperator(cfg, slots, B, max_prefill=5)
    x = op.prefill_ragged(take(qr), take(k_out), take(v), n_acc)      # x + enhancement
    op.reset()
    op.set_output_mode(sfa.SFA_OUT_ADD_BF16 if dtype == "bf16" else sfa.SFA_OUT_ADD_F32)
    total = take(out)
    op.prefill_ragged(take(qr), take(k_out), take(v), n_acc, out=total)
    zero = sfa.SfaOperator(sfa.SfaConfig(**{**cfg.__dict__, "alpha_base": 0.0}), slots, B, max_prefill=5)
    x0 = zero.prefill_ragged(take(qr), take(k_out), take(v), n_acc)   # x alone
    assert op.check() == zero.check() == sfa.sfa_check_device_status(h) == sfa.SFA_OK
    for b in range(B):
        m = len(path[b])
        want = take(out)[:, b, :m].double() + (x - x0)[:, b, :m].double()
        # the enhancement from two runs (the operator's tolerance each) and one rounding
        tol = (2e-3 if dtype == "bf16" else 1e-4) * (1 + x[:, b, :m].abs().double()) * 2 + ref.HALF[T] * want.abs()
        assert bool(((total[:, b, :m].double() - want).abs() <= tol).all())


def test_few_and_many_results_agree():
    """The same sequence in a call of few values (P in two parts) and in one of
    many: both within their bounds, and the former nearer."""
    c = Case("qwen05b", "bf16", [700] * 40, [1] * 40, 1, 16, seed=34)
    many = c.check()
    k = {}
    for b in (0, 17):
        one = sfa.SfaPagedCache(c.h, c.k_pages, c.v_pages, c.table[b:b + 1].contiguous())
        k[b] = one.attend(0, c.q[:, b:b + 1].contiguous(), c.ctx_d[b:b + 1].contiguous())
    r, bound = ref.attend(c.q.cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu(), c.ctx, c.lens, lambda b, i: None)
    for b, out in k.items():
        ref.assert_within(out, r[:, b:b + 1], bound[:, b:b + 1] / 2, "few")   # without the rounding of P
        assert float((out.double().cpu() - r[:, b:b + 1]).norm()) <= float((many[:, b:b + 1].double().cpu() - r[:, b:b + 1]).norm())
