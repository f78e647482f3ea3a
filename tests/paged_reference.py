"""Plain 64-bit forms of the paged cache operators, token by token, and the
error bounds that their tests allow.

Bounds are worst cases, not fits.  u = 2^-24 is half a step of fp32 and h half
a step of the result's type (2^-8 for bf16, 2^-24 for fp32).

attend, with S = sum_j p_j |v_j|, A = max_j sum_i |q_i k_ji| / sqrt(d), N
visible keys of which the row's largest probability is p <= 1:
  * a score is d products summed in 32 bits and scaled: off by (d + 4) 2u A
    (2u: the tensor cores may truncate where they add);
  * the exponential and the running rescale add 2^-21 relative, and sums of N
    terms N 2u; all of these enter numerator and denominator, hence twice;
  * with bf16 inputs each p may be rounded to bf16 before it meets v (2^-8), and
    again enters numerator and denominator (the kernel's p is two bf16 numbers:
    paged_bound has that narrower bound);
  * the result is rounded once: h |o|.
append: the angle's fraction of a turn is held to 2^-25, which is 2^-22 of
arc; sine, cosine and two products add as much: 2^-20 (|x1| + |x2|), and the
rounding h |x|.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def ancestors(parents):
    """[n] parents -> list of ancestor-or-self sets."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if p >= 0 else set()))
    return out


def pack_mask(rows, words):
    """list of sets -> int32 [n, words]."""
    m = torch.zeros(len(rows), words, dtype=torch.int64)
    for i, r in enumerate(rows):
        for j in r:
            m[i, j // 32] |= 1 << (j % 32)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32)


def gather(pages, layer, table, count):
    """[count, n_kv, d] fp64: the first `count` slots of one sequence."""
    ps = pages.shape[3]
    need = (count + ps - 1) // ps
    x = pages[layer, table[:need].long()].double()          # [need, n_kv, ps, d]
    return x.permute(0, 2, 1, 3).reshape(need * ps, *x.shape[1::2])[:count]


def attend(q, k_pages, v_pages, table, ctx, lens, visible, layer_begin=0):
    """q [Lc, B, n, nq, d] on the CPU; visible(b, i) -> set of new tokens that
    node i sees, or None for those up to itself.  Returns (out, bound) fp64
    [Lc, B, n, H], NaN in rows that are not written."""
    Lc, B, n, nq, d = q.shape
    nkv = k_pages.shape[2]
    G = nq // nkv
    out = torch.full((Lc, B, n, nq * d), math.nan, dtype=torch.float64)
    bound = torch.zeros_like(out)
    p_round = 2 * 2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0
    for l in range(Lc):
        for b in range(B):
            if lens[b] == 0:
                continue
            k = gather(k_pages, layer_begin + l, table[b], ctx[b] + lens[b])
            v = gather(v_pages, layer_begin + l, table[b], ctx[b] + lens[b])
            for i in range(lens[b]):
                see = visible(b, i)
                new = list(range(i + 1)) if see is None else sorted(j for j in see if j < lens[b])
                idx = torch.tensor(list(range(ctx[b])) + [ctx[b] + j for j in new], dtype=torch.long)
                if len(idx) == 0:
                    out[l, b, i] = 0.0
                    continue
                kk, vv = k[idx], v[idx]                                    # [N, nkv, d]
                qq = q[l, b, i].double().view(nkv, G, d)
                s = torch.einsum("gcd,jgd->gcj", qq, kk) / math.sqrt(d)
                p = torch.softmax(s, -1)
                o = torch.einsum("gcj,jgd->gcd", p, vv)
                A = (torch.einsum("gcd,jgd->gcj", qq.abs(), kk.abs()) / math.sqrt(d)).amax(-1)   # [g, c]
                S = torch.einsum("gcj,jgd->gcd", p, vv.abs())
                rel = p_round + 2 * (2 * U * (d + 4) * A + 2.0 ** -21 + 2 * U * len(idx))
                out[l, b, i] = o.reshape(-1)
                bound[l, b, i] = (rel[..., None] * S + HALF[q.dtype] * (o.abs() + rel[..., None] * S)).reshape(-1)
    return out, bound


def rotate(x, pos, freqs, dims, style):
    """x [..., heads, d] fp64, pos [...]: the rotated x and its bound without
    the result's rounding."""
    y = x.clone()
    a = pos.double()[..., None, None] * torch.tensor(freqs, dtype=torch.float64)
    c, s = a.cos(), a.sin()
    if style == 0:
        i1, i2 = slice(0, dims // 2), slice(dims // 2, dims)
    else:
        i1, i2 = slice(0, dims, 2), slice(1, dims, 2)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    e = torch.zeros_like(x)
    e[..., i1] = e[..., i2] = 2.0 ** -20 * (x[..., i1].abs() + x[..., i2].abs())
    return y, e


def assert_within(got, ref, bound, what):
    """Every element that ref defines (not NaN) within bound; NaN elsewhere is
    not looked at."""
    got = got.double().cpu()
    live = ~torch.isnan(ref)
    off = torch.where(live, (got - ref).abs() - bound, torch.zeros_like(ref))
    bad = ~(off <= 0)
    if bad.any():
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(live.sum())} outside; first at {at}: got {got[at]!r}, "
                             f"ref {ref[at]!r}, bound {bound[at]:.3g}")
