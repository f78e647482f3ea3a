"""Measured cases of the paged key/value cache operators.

Four operators serve a drafted batch over an exact paged cache, layer by layer, next to the SFA calls:
  plan    ancestor masks and rotation positions of a tree of drafted tokens, from the parent of every node;
  append  keys (rotated to their positions) and values of the new tokens into their pages, and rotated queries and keys out;
  attend  softmax attention of the new tokens over the cache, every node seeing the context and its own ancestors;
  accept  the accepted path's keys and values moved up behind the context.

A cache is k_pages and v_pages [layers][pages][kv heads][page size][head_dim] with page_table [batch][max pages]; sequence b has
ctx_lens[b] tokens before the call and lens[b] new ones at the slots behind them.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _shape(nq, nkv, d, dtype="bf16"):
    return {"nq": nq, "nkv": nkv, "d": d, "dtype": dtype}


QWEN05B = _shape(14, 2, 64)
QWEN7B = _shape(28, 4, 128)
TINY = _shape(2, 2, 64, "f32")


def listed():
    return [
        # one sequence, one new token: the latency of a chat turn's step, one layer
        {"name": "attend token, 1 sequence", "op": "attend", **QWEN05B, "batch": 1, "n": 1, "tree": False, "ctx_lo": 1024, "ctx_hi": 1024,
         "page": 16, "ragged": False, "shape": 1},
        # the step of a full serving batch, one layer: 256 sequences of many lengths
        {"name": "attend token, 256 sequences", "op": "attend", **QWEN7B, "batch": 256, "n": 1, "tree": False, "ctx_lo": 1024, "ctx_hi": 4096,
         "page": 64, "ragged": False, "shape": 2},
        # verification of drafted trees for a medium batch, lengths from a few tokens to 8,192, ragged trees
        {"name": "attend tree, 32 sequences", "op": "attend", **QWEN7B, "batch": 32, "n": 16, "tree": True, "ctx_lo": 17, "ctx_hi": 8192,
         "page": 16, "ragged": True, "shape": 3},
        # a large tree over one long document
        {"name": "attend tree, long context", "op": "attend", **QWEN7B, "batch": 1, "n": 64, "tree": True, "ctx_lo": 65500, "ctx_hi": 65500,
         "page": 128, "ragged": False, "shape": 4},
        # a chunk of a long prompt, causal, on top of what is cached already
        {"name": "attend chunk of a prompt", "op": "attend", **QWEN7B, "batch": 2, "n": 2048, "tree": False, "ctx_lo": 1000, "ctx_hi": 8192,
         "page": 64, "ragged": True, "shape": 5},
        # the fp32 form: small heads, odd lengths
        {"name": "attend tree, fp32", "op": "attend", **TINY, "batch": 8, "n": 7, "tree": True, "ctx_lo": 1, "ctx_hi": 515, "page": 16,
         "ragged": True, "shape": 6},
        # one token of one sequence: append's latency
        {"name": "append token, 1 sequence", "op": "append", **QWEN05B, "batch": 1, "n": 1, "tree": False, "ctx_lo": 1024, "ctx_hi": 1024,
         "page": 16, "ragged": False, "layers": 1, "rope": 1e6, "shape": 7},
        # prompts entering the cache
        {"name": "append prompts", "op": "append", **QWEN7B, "batch": 4, "n": 16384, "tree": False, "ctx_lo": 1, "ctx_hi": 100, "page": 64,
         "ragged": True, "layers": 1, "rope": 1e6, "shape": 8},
        # a path of one sequence accepted, every layer
        {"name": "accept, 1 sequence", "op": "accept", **QWEN05B, "batch": 1, "n": 16, "layers": 24, "ctx_lo": 500, "ctx_hi": 500, "page": 16,
         "shape": 9},
        # paths of a batch accepted, every layer
        {"name": "accept, 32 sequences", "op": "accept", **QWEN7B, "batch": 32, "n": 64, "layers": 28, "ctx_lo": 20, "ctx_hi": 90, "page": 16,
         "shape": 10},
        # a drafted tree of one sequence, and trees of a batch
        {"name": "plan, 1 sequence", "op": "plan", **QWEN05B, "batch": 1, "n": 16, "ragged": False, "ctx_lo": 1024, "ctx_hi": 1024, "shape": 11},
        {"name": "plan, 256 sequences", "op": "plan", **QWEN7B, "batch": 256, "n": 64, "ragged": True, "ctx_lo": 1, "ctx_hi": 8192, "shape": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "accept", "plan"])
    dtype = "f32" if op != "accept" and rng.random() < 0.2 else "bf16"
    d = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
    case = {"op": op, **_shape(nq, nkv, d, dtype), "page": rng.choice([8, 16, 32, 64, 128, 256]), "shape": rng.randrange(1 << 30)}
    ragged = rng.random() < 0.5
    if op == "attend":
        small = dtype == "f32"
        kind = rng.choice(["token", "tree", "chunk"])
        hi = _log(rng, 1, 2048 if small else 32768)
        room = 2_000_000 // max(1, hi * nkv * d // 128)  # cached tokens x heads of the call
        n = 1 if kind == "token" else _log(rng, 2, 64) if kind == "tree" else _log(rng, 17, 256 if small else 1024)
        most = (4e9 if small else 1.2e11) / (4.0 * d * nq)  # query tokens x cached tokens
        n = max(1, min(n, int(most / (hi + n))))
        work = max(1, int(most / (n * (hi + n))))
        batch = _log(rng, 1, max(1, min(256, room, work)))
        return {**case, "batch": batch, "n": n, "tree": kind == "tree", "ctx_lo": max(1, hi // rng.choice([1, 2, 30])), "ctx_hi": hi, "ragged": ragged}
    if op == "append":
        n = _log(rng, 1, 8192)
        batch = _log(rng, 1, max(1, min(256, 32768 // n)))
        return {**case, "batch": batch, "n": n, "tree": n <= 64 and rng.random() < 0.5, "ctx_lo": 1, "ctx_hi": _log(rng, 1, 2000), "ragged": ragged,
                "layers": 1 if n * batch > 2048 else rng.choice([1, 2, 5]), "rope": rng.choice([1e4, 5e5, 1e6])}
    if op == "accept":
        return {**case, "batch": _log(rng, 1, 24), "n": _log(rng, 1, 64), "layers": rng.choice([1, 3, 12, 24]), "ctx_lo": 1, "ctx_hi": _log(rng, 1, 90)}
    return {**case, "batch": _log(rng, 1, 256), "n": _log(rng, 1, 64), "ragged": ragged, "ctx_lo": 1, "ctx_hi": _log(rng, 1, 8192)}


# ------------------------------------------------------------------ shapes


def _geometry(case):
    """Lengths, trees and paths of a case: plain numbers that the case alone settles."""
    rng = random.Random(case["shape"])
    B, n = case["batch"], case["n"]
    ctx = [_log(rng, case["ctx_lo"], case["ctx_hi"]) if case["ctx_hi"] > case["ctx_lo"] else case["ctx_lo"] for _ in range(B)]
    lens = [rng.randint(1, n) if case.get("ragged") else n for _ in range(B)]
    parents, depth = [], []
    if case.get("tree") or case["op"] in ("plan", "accept"):
        for _ in range(B):
            p = [-1] + [rng.randint(max(0, i - 8), i - 1) for i in range(1, n)]
            dep = [0] * n
            for i in range(1, n):
                dep[i] = dep[p[i]] + 1
            parents.append(p)
            depth.append(dep)
    paths = []
    if case["op"] == "accept":
        # the accepted nodes lie behind the slots that they move to, but for the root
        for _ in range(B):
            m = rng.randint(1, min(6, n))
            later = sorted(rng.sample(range(m, n), min(m - 1, n - m)))
            paths.append([0] + later)
    return ctx, lens, parents, depth, paths


def _pages(case, ctx, n):
    return [(c + n + case["page"] - 1) // case["page"] for c in ctx]


def work(case):
    ctx, lens, _, depth, paths = _geometry(case)
    nq, nkv, d, esz = case["nq"], case["nkv"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "plan":
        words = (case["n"] + 31) // 32
        return {"bytes": sum(4 * l + 4 * l + 4 * l * words + 8 for l in lens), "flops": 0}
    if case["op"] == "accept":
        moved = sum(sum(1 for i, s in enumerate(p) if s != i) for p in paths)
        return {"bytes": case["layers"] * moved * 2 * 2 * nkv * d * esz + sum(4 * len(p) for p in paths), "flops": 0}
    if case["op"] == "append":
        T = sum(lens) * case["layers"]
        # q, k and v read; rotated q and k, and the cached k and v written
        return {"bytes": T * d * esz * ((nq + 2 * nkv) + (nq + nkv) + 2 * nkv), "flops": T * d * 3 * (nq + nkv)}
    kv = sum(c + l for c, l in zip(ctx, lens))
    seen = sum(l * c + (sum(depth[b][:l]) + l if case["tree"] else l * (l + 1) // 2) for b, (c, l) in enumerate(zip(ctx, lens)))
    return {"bytes": kv * nkv * d * 2 * esz + 2 * sum(lens) * nq * d * esz, "flops": 4 * d * nq * seen}


# ------------------------------------------------------------------ inputs


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1_000_003 + 17)
    hg = random.Random(seed * 7919 + 5)
    ctx, lens, parents, depth, paths = _geometry(case)
    B, n, nq, nkv, d, ps = case["batch"], case["n"], case["nq"], case["nkv"], case["d"], case.get("page", 16)
    L, dt = case.get("layers", 1), DTYPES[case["dtype"]]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    st = {"case": case, "ctx": ints(ctx), "lens": ints(lens)}
    if case["op"] == "plan":
        # other trees for another seed: the nodes that hang directly on the root change
        par = [[p if i == 0 or hg.random() < 0.9 else 0 for i, p in enumerate(row)] for row in parents]
        words = (n + 31) // 32
        st["parents"] = ints(par)
        st["positions"] = torch.zeros(B, n, dtype=torch.int32, device=dev)
        st["mask"] = torch.zeros(B, n, words, dtype=torch.int32, device=dev)
        return st
    counts = _pages(case, ctx, n)
    total = sum(counts) + 3
    ids = list(range(total))
    hg.shuffle(ids)
    table, at = [], 0
    for c in counts:
        table.append(ids[at:at + c] + [-1] * (max(counts) - c))  # entries behind the last page are never read
        at += c
    st["table"] = ints(table)
    st["k_pages"] = torch.randn(L, total, nkv, ps, d, generator=g, device=dev, dtype=dt)
    st["v_pages"] = torch.randn(L, total, nkv, ps, d, generator=g, device=dev, dtype=dt)
    if case["op"] == "accept":
        st["path"] = ints([p + [0] * (n - len(p)) for p in paths])
        st["n_accept"] = ints([len(p) for p in paths])
        st["rows"] = ([b for b, p in enumerate(paths) for _ in p], [i for p in paths for i in range(len(p))])
    else:
        st["q"] = torch.randn(L, B, n, nq, d, generator=g, device=dev, dtype=dt)
        st["rows"] = ([b for b in range(B) for _ in range(lens[b])], [i for b in range(B) for i in range(lens[b])])
    st["rows"] = tuple(torch.tensor(x, dtype=torch.int64, device=dev) for x in st["rows"])
    if case["op"] == "append":
        st["k"] = torch.randn(L, B, n, nkv, d, generator=g, device=dev, dtype=dt)
        st["v"] = torch.randn(L, B, n, nkv, d, generator=g, device=dev, dtype=dt)
        st["q_out"] = torch.zeros_like(st["q"])
        st["k_out"] = torch.zeros_like(st["k"])
        st["positions"] = ints([[ctx[b] + x for x in depth[b]] for b in range(B)]) if case["tree"] else None
    if case["op"] == "attend":
        st["out"] = torch.zeros(L, B, n, nq * d, device=dev, dtype=dt)
        st["mask"] = _pack(_reach(ints(parents))) if case["tree"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import kv_cache_compression_sfa_b200 as sfa
        cfg = sfa.SfaConfig(n_layers=case.get("layers", 1), n_q_heads=case["nq"], n_kv_heads=case["nkv"], head_dim=case["d"],
                            in_dtype=sfa.SFA_BF16 if case["dtype"] == "bf16" else sfa.SFA_F32)
        slots = torch.zeros(cfg.n_layers, cfg.n_slots, cfg.hidden, device="cuda")
        st["sfa"] = sfa
        st["handle"] = sfa.sfa_init(cfg, slots)
        if "k_pages" in st:
            st["cache"] = sfa.SfaPagedCache(st["handle"], st["k_pages"], st["v_pages"], st["table"])
        if case["op"] == "append":
            st["rope"] = sfa.SfaRope(base=case["rope"])
    return st


# --------------------------------------------------------------- plain forms


def _reach(parents):
    """[B, n] parents -> [B, n, n]: node j is node i or an ancestor of it."""
    B, n = parents.shape
    idx = torch.arange(n, device=parents.device)
    r = ((parents[:, :, None] == idx) | (idx[:, None] == idx)).float()
    for _ in range(max(1, (n - 1).bit_length())):
        r = (r @ r > 0).float()
    return r > 0


def _pack(bits):
    """[B, n, n] truth values -> [B, n, words] int32, bit j % 32 of word j // 32."""
    B, n, _ = bits.shape
    words = (n + 31) // 32
    full = torch.zeros(B, n, words * 32, dtype=torch.int64, device=bits.device)
    full[:, :, :n] = bits
    w = (full.view(B, n, words, 32) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _plan(st):
    n = st["parents"].shape[1]
    live = torch.arange(n, device=st["lens"].device) < st["lens"][:, None]
    r = _reach(st["parents"])
    pos = st["ctx"][:, None] + r.sum(-1).to(torch.int32) - 1
    st["positions"].copy_(torch.where(live, pos, st["positions"]))
    st["mask"].copy_(torch.where(live[:, :, None], _pack(r), st["mask"]))
    return {"positions": st["positions"], "mask": st["mask"]}


def _slots(st, b, i):
    """Page and row of slot ctx + i of sequence b."""
    ps = st["k_pages"].shape[3]
    slot = st["ctx"].long()[b] + i
    return st["table"].long()[b, slot // ps], slot % ps


def _rotate(x, pos, base):
    """Halves x1, x2 of the head dim turned by the angle of pos: (x1 c - x2 s, x2 c + x1 s). Angles in 64 bits."""
    h = x.shape[-1] // 2
    inv = base ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    a = pos.double()[..., None] * inv
    c, s = a.cos().float(), a.sin().float()
    c, s = c[..., None, :], s[..., None, :]
    x1, x2 = x[..., :h].float(), x[..., h:].float()
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1).to(x.dtype)


def _append(st):
    b, i = st["rows"]
    n, base = st["q"].shape[2], st["case"]["rope"]
    pos = st["positions"] if st["positions"] is not None else st["ctx"][:, None] + torch.arange(n, device=b.device, dtype=torch.int32)
    q, k = _rotate(st["q"], pos, base), _rotate(st["k"], pos, base)
    page, row = _slots(st, b, i)
    st["q_out"][:, b, i] = q[:, b, i]
    st["k_out"][:, b, i] = k[:, b, i]
    st["k_pages"][:, page, :, row] = k[:, b, i].transpose(0, 1)
    st["v_pages"][:, page, :, row] = st["v"][:, b, i].transpose(0, 1)
    return {"q": st["q_out"], "k": st["k_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _attend(st):
    L, B, n, nq, d = st["q"].shape
    nkv, ps = st["k_pages"].shape[2:4]
    S = st["table"].shape[1] * ps
    table = st["table"].long().clamp(min=0)
    gather = lambda x: x[0][table].permute(0, 2, 1, 3, 4).reshape(B, nkv, S, d).float()  # noqa: E731
    q = st["q"][0].float().view(B, n, nkv, nq // nkv, d).permute(0, 2, 1, 3, 4).reshape(B, nkv, -1, d)
    s = (q @ gather(st["k_pages"]).transpose(2, 3) * (1.0 / math.sqrt(d))).view(B, nkv, n, nq // nkv, S)
    col = torch.arange(S, device=q.device)
    rel = col - st["ctx"][:, None]                                       # [B, S]: slot behind the context
    new = (rel >= 0) & (rel < st["lens"][:, None])
    if st["mask"] is None:
        sees = rel[:, None, :] <= torch.arange(n, device=q.device)[:, None]
    else:
        at = rel.clamp(0, n - 1)
        word = st["mask"].gather(2, (at // 32)[:, None, :].expand(B, n, S))
        sees = ((word >> (at % 32)[:, None, :]) & 1) > 0
    sees = (rel < 0)[:, None, :] | (new[:, None, :] & sees)
    s = torch.where(sees[:, None, :, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, nkv, -1, S) @ gather(st["v_pages"])).view(B, nkv, n, nq // nkv, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, nq * d)
    live = (torch.arange(n, device=q.device) < st["lens"][:, None])[:, :, None]
    st["out"][0].copy_(torch.where(live, o.to(st["out"].dtype), st["out"][0]))
    return {"out": st["out"]}


def _accept(st):
    b, i = st["rows"]
    sp, sr = _slots(st, b, st["path"].long()[b, i])
    dp, dr = _slots(st, b, i)
    for x in (st["k_pages"], st["v_pages"]):
        x[:, dp, :, dr] = x[:, sp, :, sr]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def run(st):
    op = st["case"]["op"]
    if own:
        sfa, h, cache = st["sfa"], st["handle"], st.get("cache")
        if op == "plan":
            sfa.sfa_tree_plan(h, st["parents"], st["ctx"], lens=st["lens"], positions=st["positions"], mask=st["mask"])
            return {"positions": st["positions"], "mask": st["mask"]}
        if op == "append":
            cache.append(0, st["q"], st["k"], st["v"], st["ctx"], lens=st["lens"], positions=st["positions"], rope=st["rope"],
                         q_out=st["q_out"], k_out=st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
        if op == "attend":
            cache.attend(0, st["q"], st["ctx"], lens=st["lens"], mask=st["mask"], out=st["out"])
            return {"out": st["out"]}
        cache.accept(0, st["case"]["layers"], st["path"], st["n_accept"], st["ctx"])
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    return {"plan": _plan, "append": _append, "attend": _attend, "accept": _accept}[op](st)


# --------------------------------------------------------------------- 64 bits


def _exact_append(case, st):
    ctx, lens, _, depth, _ = _geometry(case)
    d, ps = case["d"], case["page"]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    qo, ko = torch.zeros_like(st["q"], dtype=torch.float64), torch.zeros_like(st["k"], dtype=torch.float64)
    freq = torch.tensor([case["rope"] ** (-2.0 * j / d) for j in range(d // 2)], dtype=torch.float64, device="cuda")
    table = st["table"].tolist()
    for b, (c, n) in enumerate(zip(ctx, lens)):
        pos = torch.tensor([c + (depth[b][i] if case["tree"] else i) for i in range(n)], dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones(n, d // 2, dtype=torch.float64, device="cuda"), pos[:, None] * freq)[None, :, None, :]
        for src, dst in ((st["q"], qo), (st["k"], ko)):
            x = src[:, b, :n].double()
            z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
            dst[:, b, :n] = torch.cat([z.real, z.imag], -1)
        first, last = c // ps, (c + n - 1) // ps
        for pg in range(first, last + 1):  # the run of rows that falls into one page
            lo, hi = max(c, pg * ps), min(c + n, (pg + 1) * ps)
            kp[:, table[b][pg], :, lo - pg * ps:hi - pg * ps] = ko[:, b, lo - c:hi - c].transpose(1, 2)
            vp[:, table[b][pg], :, lo - pg * ps:hi - pg * ps] = st["v"][:, b, lo - c:hi - c].double().transpose(1, 2)
    return {"q": qo, "k": ko, "k_pages": kp, "v_pages": vp}


def _exact_attend(case, st):
    ctx, lens, parents, _, _ = _geometry(case)
    nq, nkv, d, ps = case["nq"], case["nkv"], case["d"], case["page"]
    out = torch.zeros_like(st["out"], dtype=torch.float64)
    table = st["table"].tolist()
    for b, (c, n) in enumerate(zip(ctx, lens)):
        S = c + n
        pages = table[b][:(S + ps - 1) // ps]
        see = torch.ones(n, n, dtype=torch.bool).tril()
        if case["tree"]:
            see.zero_()
            for i in range(n):
                j = i
                while j >= 0:
                    see[i, j] = True
                    j = parents[b][j]
        hidden = ~see.cuda()
        for kh in range(nkv):
            k = st["k_pages"][0, pages, kh].reshape(-1, d)[:S].double()
            v = st["v_pages"][0, pages, kh].reshape(-1, d)[:S].double()
            for h in range(kh * (nq // nkv), (kh + 1) * (nq // nkv)):
                s = st["q"][0, b, :n, h].double() @ k.T / math.sqrt(d)
                s[:, c:].masked_fill_(hidden, -math.inf)
                out[0, b, :n, h * d:(h + 1) * d] = torch.softmax(s, -1) @ v
    return {"out": out}


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, _inputs(case, seed))
    if case["op"] == "attend":
        return _exact_attend(case, _inputs(case, seed))
    return None  # whole numbers and copies
