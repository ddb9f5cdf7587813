"""What the tests of packed attention's two-term weights share: the bound, and the rounding itself.

Where no sequence has more than one row tile (max_q * Hq / Hkv <= 128) the
tensor-core form takes a weight as two bf16 terms, the second the rounded rest
of the first: off by 2^-8 * 2^-8 of the weight.  The scores here are small
(queries of unit variance, scale 1 / D), so that what else can be off -- fp32
sums of (D + 4) and of m terms, the exponential's 2^-21 -- is below a single
term's 2^-8 by far, and a lost or misplaced second term shows in every element
whose own rounding is small.
"""
import math

import torch


def two_term_bound(want, mag, rel, dtype):
    """Largest error of an output: ref_attend's `rel` and 2^-16 of sum p |v|, and half a step."""
    half = torch.finfo(dtype).eps / 2
    return (rel + 2.0 ** -16) * mag * (1 + half) + half * want.abs() + 1e-37


def rounded(q, k, v, scale, causal, terms, shift=0):
    """One sequence as the tensor cores compute it but for fp64 sums: weights against the row's maximum
    in `terms` bf16 terms, the second term's keys moved on by `shift`; outputs in bf16."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double()
        s = q[:, h].double() @ kh.T * scale
        if causal:
            s = s.masked_fill(torch.arange(m)[None] > torch.arange(n)[:, None] + (m - n), -math.inf)
        p = (s - s.amax(-1, keepdim=True)).exp().float()
        hi = p.bfloat16().float()
        lo = (p - hi).bfloat16().float().roll(shift, -1)
        w = hi.double() + (lo.double() if terms == 2 else 0)
        out[:, h] = w @ vh / p.double().sum(-1, keepdim=True)
    return out.bfloat16()
