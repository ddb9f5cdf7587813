"""What the tests of norms, axes, the 8-bit cache and trees over pages share: plain 64-bit forms and their bounds.

Norm and positions.  Against the exact row, u = w x / sqrt(mean x^2 + eps) is off by (D + 8) 2^-24 of itself at
most: the sum of D squares by D 2^-24, halved by the root, and a root, two divisions and two products; the turn
by 6 * 2^-24 (|u_a| + |u_b|) m more (test_gpu_paged).  A stored row is off by half a step besides.
"""
import math

import torch

TOP, TINY = 448.0, 2.0 ** -100


def pair_axes(parts, order):
    if order == "blocks":
        return [a for a, p in enumerate(parts) for _ in range(p)]
    n = len(parts)
    return [i % n if i < n * parts[i % n] else 0 for i in range(sum(parts))]


def norm_turn(x, w, eps, pos, freqs, axis, layout, m=1.0):
    """(exact rows, bound on how far fp32 values are off): x [N, H, D], pos [axes, N], freqs and axis per pair."""
    u = x.double()
    D = u.shape[-1]
    slip = 0.0
    if w is not None:
        u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        slip = (D + 8) * 2.0 ** -24
    R = 2 * len(freqs)
    ang = pos.double()[torch.tensor(axis)].T * freqs.double()          # [N, R / 2]
    c, s = (ang.cos() * m)[:, None], (ang.sin() * m)[:, None]
    i = torch.arange(R // 2)
    a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y, off = u.clone(), u.abs() * slip
    mag = (u[..., a].abs() + u[..., b].abs()) * abs(m)
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    off[..., a] = off[..., b] = mag * (slip + 6 * 2.0 ** -24)
    return y, off


def check_rows(got, want, off, dtype):
    half = torch.finfo(dtype).eps / 2
    err = (got.cpu().double() - want).abs()
    assert (err <= off * (1 + half) + half * want.abs() + 1e-37).all(), float(err.max())


def quantise(x):
    """Codes and scales of fp32 rows, by the definition."""
    top = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    codes = (x.double() * TOP / top.double()).float()          # (exact ties among bf16 rows' quotients stay ties)
    return codes.clamp(-TOP, TOP).to(torch.float8_e4m3fn), (top / TOP)[..., 0]


def check_codes(codes, scale, want, off):
    """A quantised row against the exact values before it: the scale by the largest one, every element by half a
    step (2^-4 of itself, or 2^-10 scale), by what the value was off before, and a product's rounding."""
    top = want.abs().amax(-1)
    slack = off.amax(-1)
    scale = scale.cpu().double()
    assert ((scale * TOP - top.clamp_min(TINY)).abs() <= slack + 2.0 ** -22 * top + 2.0 ** -120).all()
    got = codes.cpu().float().double() * scale[..., None]
    tol = (2.0 ** -4 + 2.0 ** -20) * want.abs() + 2.0 ** -10 * scale[..., None] * (1 + 2.0 ** -20) + 1.07 * off \
        + 1.07 * slack[..., None] * 2.0 ** -4
    assert ((got - want).abs() <= tol).all()


def attend(q, k, v, scale, seen, v_parts=None):
    """One sequence in fp64, seen [n, m]: (out, sum p|v|, sqrt(sum p^2 v^2), relative weight error of fp32 scores,
    largest weight times sqrt(sum v_ref^2), the same times sum |v_ref|).  v_parts: (|codes|, largest scale) of 8-bit
    values; an 8-bit weight is off by a step of the largest one times the largest scale."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    mag, quad, flat2, flat1 = (torch.zeros_like(out) for _ in range(4))
    rel = 0.0
    if m == 0:
        return out, mag, quad, 0.0, flat2, flat1
    q, k, v = q.double(), k.double(), v.double()
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kh.T * scale).masked_fill(~seen, -math.inf)
        ab = q[:, h].abs() @ kh.abs().T * scale
        # fp32 sums, and queries in two e4m3 terms (2^-18 of the row's largest element)
        rel = max(rel, float(ab.max()) * (D + 4) * 2.0 ** -24)
        if v_parts is not None:
            rel = max(rel, float((ab * (D + 4) * 2.0 ** -24 +
                                  2.0 ** -18 * q[:, h].abs().amax(-1)[:, None] * kh.abs().sum(-1) * scale).max()))
        top = s.amax(-1, keepdim=True)
        p = torch.where(s == -math.inf, 0.0, (s - torch.where(top == -math.inf, 0.0, top)).exp())
        z = p.sum(-1, keepdim=True)
        p = torch.where(z > 0, p / z.clamp_min(1e-300), 0.0)
        out[:, h] = p @ vh
        mag[:, h] = p @ vh.abs()
        quad[:, h] = ((p * p) @ (vh * vh)).sqrt()
        if v_parts is not None:
            codes, big = v_parts[0][:, h // G].double(), v_parts[1][h // G]
            peak = p.amax(-1)[:, None] * big
            flat2[:, h] = peak * codes.square().sum(0).sqrt()
            flat1[:, h] = peak * codes.abs().sum(0)
    return out, mag, quad, 2 * rel + 2.0 ** -21 + m * 2.0 ** -24, flat2, flat1


def check_attention(got, want, dtype, terms):
    """terms: 0 fp32 weights, "bf16" one term of 2^-8, "e4m3" two of 2^-8 and 2^-15 of the largest in all."""
    out, mag, quad, rel, flat2, flat1 = want
    got = got.cpu().double()
    half = torch.finfo(dtype).eps / 2
    pr = 2.0 ** -8 if terms else 0.0
    fl = 2.0 ** -15 if terms == "e4m3" else 0.0
    assert torch.isfinite(got).all()
    err = (got - out).abs()
    tol = ((rel + pr) * mag + fl * flat1) * (1 + half) + half * out.abs() + 1e-37
    assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
    if got.numel() > 4096:
        rms = lambda x: float(x.pow(2).mean().sqrt())
        assert rms(err) <= rms(rel * mag) + math.sqrt((half * rms(out)) ** 2 + (pr * rms(quad)) ** 2 + (fl * rms(flat2)) ** 2)


def tree_masks(g, n, depth_bias=0.7):
    """Masks (ancestors and the node) and parents of a random tree."""
    import random
    r = random.Random(int(torch.randint(1 << 30, (1,), generator=g)))
    masks, parents = [], []
    for j in range(n):
        p = -1 if j == 0 else r.randrange(max(0, int(j * depth_bias) - 2), j)
        parents.append(p)
        masks.append((masks[p] if j else 0) | 1 << j)
    return masks, parents


def signed(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)
