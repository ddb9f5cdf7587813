"""The 8-bit attention's weights restated, one row: the bound that the GPU tests put on its outputs holds for them, and
tells them from terms that end too early."""
import math

import pytest
import torch

from _quant import quantise
from _quant_sums import bound

M, D = 32768, 64


def upper(x):
    return (x.view(torch.int16) & -256).view(torch.float16)


def three_e5m2(w):
    w = w.half()
    a = upper(w)
    b = upper(w - a)
    c = w - a - b
    return a.double() + b.double() + upper((c.view(torch.int16) + 128).view(torch.float16)).double()


def two_e4m3(w):
    w = w.half().float()
    a = w.clamp(max=448.0).to(torch.float8_e4m3fn).float()
    return a.double() + (w - a).to(torch.float8_e4m3fn).double()


def row(x, v, codes, terms, log_w, top):
    """x: scores in log2 units; a part of 64 keys at a time; m moves up where a weight would pass 2^top."""
    m, out, l = -math.inf, torch.zeros(D, dtype=torch.float64), 0.0
    for a in range(0, M, 64):
        xs, vs = x[a:a + 64], v[a:a + 64]
        t = float((xs + vs.clamp_min(2.0 ** -80).log2()).max())
        if t > m + top - log_w:
            f = 2.0 ** (m - t)
            m, out, l = t, out * f, l * f
        p = torch.exp2(xs - m + log_w)
        out += terms((p * vs).float()) @ codes[a:a + 64]
        l += float(p.sum())
    return out / l


def cases():
    g = torch.Generator().manual_seed(1)
    nat = 1 / math.log(2)
    for nats in (10, 11, 12, 14, 17):
        for flat in (True, False):
            for size in (0.1, 1.0):
                x = (torch.zeros(M) if flat else torch.randn(M, generator=g)).double() * nat
                x[0] = nats * nat
                v = 1 + 0.25 * torch.randn(M, D, generator=g)
                v[0] *= size
                yield x, v
    yield torch.randn(M, generator=g).double() * 3 * nat, torch.randn(M, D, generator=g) * torch.exp(torch.randn(M, 1, generator=g) * 2)
    yield -torch.arange(M).double() * 0.02, 1 + 0.25 * torch.randn(M, D, generator=g)
    v = 1 + 0.25 * torch.randn(M, D, generator=g)
    v[:5000] = 0
    yield torch.randn(M, generator=g).double(), v


def worst(terms, log_w, top):
    found = 0.0
    for x, v in cases():
        c, s = quantise(v)
        c, s = c.double(), s.double()
        p = torch.softmax(x * math.log(2), 0)
        val = c * s[:, None]
        want = p @ val
        tol = bound(want, p @ val.abs(), (p @ s * 448).expand(D), M * 2.0 ** -24, torch.bfloat16)
        found = max(found, float(((row(x, s, c, terms, log_w, top).bfloat16().double() - want).abs() / tol).max()))
    return found


def test_three_terms_keep_a_long_rest():
    assert worst(three_e5m2, 9, 15.7) <= 1


def test_terms_that_end_early_do_not():
    assert worst(two_e4m3, 5, 8.8) > 5
