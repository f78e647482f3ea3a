"""The 64-bit form of the paged attention over whole sequences, with the error
bound of a kernel that loses nothing but the result's rounding.

As in paged_reference (S = sum_j p_j |v_j|, A the largest sum_i |q_i k_ji| /
sqrt(d), N visible keys, u = 2^-24, h half a step of the result's type), but for
P: its upper half word leaves a rest below 2^-7 of a weight, whose bf16 is off by
2^-8 of itself at most, and the rest carries 2^-22 of the weight more.  That enters
numerator and denominator, so 2 * (2^-15 + 2^-22) takes the place of 2 * 2^-8.
"""
import math

import torch

import paged_reference as ref


def attend(q, k_pages, v_pages, table, ctx, lens, mask_rows=None, layer_begin=0):
    """(out, bound) fp64 [Lc, B, n, H] on the CPU, NaN in rows that are not
    written.  mask_rows[b][i]: set of new tokens that node i sees; None: those
    up to itself."""
    Lc, B, n, nq, d = q.shape
    nkv = k_pages.shape[2]
    G = nq // nkv
    out = torch.full((Lc, B, n, nq * d), math.nan, dtype=torch.float64)
    bound = torch.zeros_like(out)
    p_round = 2 * (2.0 ** -15 + 2.0 ** -22) if q.dtype == torch.bfloat16 else 0.0
    for l in range(Lc):
        for b in range(B):
            if lens[b] == 0:
                continue
            m, S_ = lens[b], ctx[b] + lens[b]
            k = ref.gather(k_pages, layer_begin + l, table[b], S_).permute(1, 0, 2)[:, None]      # [nkv, 1, S, d]
            v = ref.gather(v_pages, layer_begin + l, table[b], S_).permute(1, 0, 2)[:, None]
            see = torch.ones(m, S_, dtype=torch.bool)
            for i in range(m):
                see[i, ctx[b]:] = False
                new = range(i + 1) if mask_rows is None else [j for j in mask_rows[b][i] if j < m]
                see[i, [ctx[b] + j for j in new]] = True
            qq = q[l, b, :m].double().view(m, nkv, G, d).permute(1, 2, 0, 3)                      # [nkv, G, m, d]
            hide = lambda x, w: x.masked_fill(~see, w)  # noqa: E731
            p = torch.softmax(hide(qq @ k.transpose(2, 3) / math.sqrt(d), -math.inf), -1)
            p = torch.nan_to_num(p, nan=0.0)                                                      # a row that sees nothing
            o, S = p @ v, p @ v.abs()
            A = hide(qq.abs() @ k.abs().transpose(2, 3) / math.sqrt(d), 0.0).amax(-1, keepdim=True)
            rel = p_round + 2 * (2 * ref.U * (d + 4) * A + 2.0 ** -21 + 2 * ref.U * see.sum(-1)[:, None])
            e = rel * S
            flat = lambda x: x.permute(2, 0, 1, 3).reshape(m, nq * d)  # noqa: E731
            out[l, b, :m] = flat(o)
            bound[l, b, :m] = flat(e + ref.HALF[q.dtype] * (o.abs() + e))
    return out, bound
