"""Attention over 8-bit rows against the formula in 64 bits, with a bound that does not grow with the number of keys
and knows of nothing but what a row sees.

A weight (its value's scale in it) enters the second product in a few terms of 8 bits.  Each may be off by 2^-9 of
itself and by 2^-11, a rounding to f16, and all the small ones together, below the terms' smallest step, by 2^-8 of
the sum of the row's weights.  With codes of 448 at most an output is then off by

    (2^-9 + 2^-11) sum p |v|  +  2^-8 sum p 448 s  +  what the scores are off by  +  half a step of the output

(p the softmax weights, s the values' scales).  The scores: fp32 sums of D + 4 terms, queries in two e4m3 terms (off
by 2^-17 of the row's largest: the largest lies in [2^7, 2^8), the second term's half step is 2^-10); sums over m
keys: m 2^-24."""
import math

import torch

from _quant import quantise


def pages_of(k, v, page, g):
    """fp32 [m, Hkv, D] rows of one sequence -> (pages and scales as the calls take them, table, exact k, v, v's scales)"""
    m, Hkv, D = k.shape
    n = -(-m // page)
    ids = torch.randperm(n + 1, generator=g)[:n]
    out, exact = [], []
    for x in (k, v):
        c, s = quantise(x)
        codes = torch.full((n * page, Hkv, D), 0x7f, dtype=torch.uint8)          # NaN past the end
        codes[:m] = c.view(torch.uint8)
        scale = torch.full((n * page, Hkv), float("nan"))
        scale[:m] = s
        pages = torch.full((n + 1, page, Hkv, D), 0x7f, dtype=torch.uint8)
        pages[ids] = codes.view(n, page, Hkv, D)
        scales = torch.full((n + 1, Hkv, page), float("nan"))
        scales[ids] = scale.view(n, page, Hkv).transpose(1, 2)
        out.append((pages.view(torch.float8_e4m3fn).cuda(), scales.cuda()))
        exact.append((c.double() * s.double()[..., None], s.double()))
    (kp, ks), (vp, vs) = out
    return (kp, vp, ks, vs), ids.to(torch.int32)[None].cuda(), exact[0][0], exact[1][0], exact[1][1]


def formula(q, k, v, v_scale, scale, seen):
    """(output, sum p |v|, sum p 448 s, relative error of the weights by their scores) in 64 bits; seen [n, m]."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    out, mag, big = (torch.zeros(n, Hq, D, dtype=torch.float64) for _ in range(3))
    rel = 0.0
    q = q.double()
    for h in range(Hq):
        kh, vh, vs = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], v_scale[:, h * Hkv // Hq]
        s = (q[:, h] @ kh.T * scale).masked_fill(~seen, -math.inf)
        p = torch.softmax(s, -1)
        out[:, h], mag[:, h], big[:, h] = p @ vh, p @ vh.abs(), (p @ vs * 448)[:, None]
        # (the largest of |q| |k| and of the queries' missing bits; a key's are those of all keys at most)
        off = q[:, h].abs() @ kh.abs().T * (D + 4) * 2.0 ** -24 + 2.0 ** -17 * q[:, h].abs().amax(-1, keepdim=True) * kh.abs().sum(-1)
        rel = max(rel, float(off.max()) * scale)
    return out, mag, big, 2 * rel + 2.0 ** -21 + m * 2.0 ** -24


def bound(out, mag, big, rel, dtype):
    half = torch.finfo(dtype).eps / 2
    return ((2.0 ** -9 + 2.0 ** -11 + rel) * mag + 2.0 ** -8 * big) * (1 + half) + half * out.abs()


def check(got, want, dtype=torch.bfloat16):
    err, tol = (got.cpu().double() - want[0]).abs(), bound(*want, dtype)
    assert torch.isfinite(got).all()
    worst = float((err / tol).max())
    assert worst <= 1, (worst, float(err.norm() / want[0].norm()))
    return worst


# forms of the tensor-core kernel by a kv head's rows: at most 32, one tile of 128, two; trees of each
FORMS = {"few": (1, 7, False), "tile": (16, 7, False), "pairs": (64, 7, False), "tree few": (4, 7, True), "tree": (16, 7, True),
         "tree pairs": (60, 7, True)}


class Sequence:
    """One sequence of m keys whose last n are the new tokens', 2 kv heads of G query heads."""

    def __init__(self, S, k, v, page=64, seed=1):
        self.S, self.m = S, len(k)
        self.cache, self.table, self.k, self.v, self.vs = pages_of(k, v, page, torch.Generator().manual_seed(seed))

    def run(self, q, tree, causal=True, masks=None, max_kv=None):
        S, m, most = self.S, self.m, max_kv or self.m
        n, Hq, D = q.shape
        Hkv = self.k.shape[1]
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        out = torch.empty(n, Hq, D, dtype=q.dtype, device="cuda")
        ws = S.workspace(S.sd_paged_attention_workspace_size(n, 1, n, Hq, Hkv, D, most))
        kp, vp, ks, vs = self.cache
        if tree:
            S.sd_paged_tree_attention(q.cuda(), kp, vp, self.table, torch.tensor(masks).cuda(), i32(0, n), i32(m), n, most, out, D ** -0.5,
                                      ws, ks, vs)
        else:
            S.sd_paged_attention_e4m3(q.cuda(), kp, vp, ks, vs, self.table, i32(0, n), i32(m), n, most, out, D ** -0.5, ws, causal=causal)
        torch.cuda.synchronize()
        assert S.sd_last_attention_path()[0] == 2 and S.sd_fault_word() == 0
        return out

    def want(self, q, tree, causal=True, masks=None):
        n, m = len(q), self.m
        t = torch.arange(m)[None]
        if tree:
            seen = (t < m - n) | (torch.tensor(masks)[:, None] >> (t - (m - n)).clamp(0, 62) & 1).bool()
        else:
            seen = t <= torch.arange(n)[:, None] + m - n if causal else torch.ones(n, m, dtype=torch.bool)
        return formula(q, self.k, self.v, self.vs, q.shape[-1] ** -0.5, seen)
