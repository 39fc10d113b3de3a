"""Bounds of attention over chunks of new tokens for each output by the values that it weighs.

With B = max_u (Dk + 1) 2^-24 |scale| sum_d |q_d k_ud| over the tokens seen (float32 accumulation of a
dot product): a score error of B moves a weight by at most 2 B of itself, normaliser included; four
times that stands for both and their product. Weights are rounded to bf16 for their product with V,
each by at most half a step, 2^-8 of itself, and the normaliser is not rounded. Sums over n terms in
float32, cut off or rounded, are off by at most n 2^-23 of what they sum the sizes of, in steps of 16
tokens: 1e-4 up to 12000 tokens. All of these are parts of sum_u p_u |V_u|. The output's own rounding
is 2^-8 |o|. The log-sum-exp: 4 B + 1e-5 (1 + |lse|).
"""
import math

import torch


def exact(b, r):
    """(o, sum_u p_u |V_u|, lse, B) of request r of a Chunks batch in float64."""
    x, bound, v = b.exact(r)
    n, hq, c = x.shape
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = torch.where(total > 0, p / total, 0.0).view(n, b.H, hq // b.H, c)
    o = torch.einsum("nhgc,hcd->nhgd", p, v).flatten(1, 2)
    size = torch.einsum("nhgc,hcd->nhgd", p, v.abs()).flatten(1, 2)
    return o, size, lse, bound


def check_rows(b, only=None):
    """Every output of the call, or those of the rows in the mask `only`."""
    assert int(b.st.item()) == 0
    for r in range(len(b.new)):
        rows = slice(int(b.start[r]), int(b.start[r + 1]))
        if b.new[r] == 0 or (only is not None and not bool(only[rows].any())):
            continue
        o, size, lse, bound = exact(b, r)
        got, z = b.out[rows].double(), b.lse[rows].double()
        over = (got - o).abs() - (8 * bound + 1e-4 + 2.0 ** -8)[..., None] * size - 2.0 ** -8 * o.abs()
        fin = torch.isfinite(lse)
        same = torch.where(fin, (z - lse).abs() <= 4 * bound + 1e-5 * (1 + lse.abs()), z == lse)
        good = over <= 1e-30
        if only is not None:
            good, same = good[only[rows]], same[only[rows]]
        assert bool(good.all()), (r, float(over.max()), int((~good).sum()))
        assert bool(same.all()), r
