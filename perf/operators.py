"""Performance cases of the paged-cache operators: rotary positions, the append of new tokens to a
paged K/V cache, attention of new tokens over that cache, and attention over whole prompts.

Each case is one call.  `run` computes it either in plain torch operations (own = False) or
through the library's entry points (own = True); `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _rope(layout="half", rot=128, theta=1e6, scaling="none", factor=1.0, original=0, low=1.0, high=32.0):
    return dict(layout=layout, rot=rot, theta=theta, scaling=scaling, factor=factor, original=original,
                low=low, high=high)


def listed():
    return [
        # the queries of a 25,119-token video prompt, before its prefill
        dict(name="rotary-prompt", op="rotary", dtype="bf16", N=25119, H=28, D=128, pos0=0, **_rope()),
        # one block of 16 tokens of four long conversations: half of each head turned, stretched context
        dict(name="rotary-blocks-yarn", op="rotary", dtype="bf16", N=64, H=64, D=128, pos0=131072,
             **_rope("interleaved", 64, 1e6, "yarn", 4.0, 32768)),
        # 16 verified slots of eight ragged sequences enter the cache
        dict(name="append-verify-b8", op="append", dtype="bf16", B=8, q_lo=16, q_hi=16, kv_lo=4096, kv_hi=32768,
             page=64, Hq=28, Hkv=4, D=128, **_rope()),
        # a whole prompt enters the cache
        dict(name="append-prompt", op="append", dtype="bf16", B=1, q_lo=25119, q_hi=25119, kv_lo=25119, kv_hi=25119,
             page=16, Hq=28, Hkv=4, D=128, **_rope()),
        # plain decoding of one sequence: a single token over the video's context
        dict(name="paged-decode-b1", op="paged", dtype="bf16", B=1, q_lo=1, q_hi=1, kv_lo=25119, kv_hi=25119,
             page=64, Hq=28, Hkv=4, D=128, causal=True),
        # block verification of a ragged batch
        dict(name="paged-verify-b8", op="paged", dtype="bf16", B=8, q_lo=16, q_hi=16, kv_lo=4096, kv_hi=32768,
             page=16, Hq=28, Hkv=4, D=128, causal=True),
        # decoding, verification and prefill chunks in one ragged batch, some sequences idle
        dict(name="paged-mixed-b12", op="paged", dtype="bf16", B=12, q_lo=0, q_hi=700, kv_lo=1000, kv_hi=9000,
             page=48, Hq=28, Hkv=4, D=128, causal=True),
        # a chunk of a long prompt over what is already cached, the larger model's heads
        dict(name="paged-chunk", op="paged", dtype="bf16", B=1, q_lo=2048, q_hi=2048, kv_lo=32768, kv_hi=32768,
             page=128, Hq=64, Hkv=8, D=128, causal=True),
        # the tiny model of the checks, in fp32
        dict(name="paged-tiny-fp32", op="paged", dtype="fp32", B=1, q_lo=16, q_hi=16, kv_lo=527, kv_hi=527,
             page=16, Hq=4, Hkv=1, D=64, causal=True),
        # a whole video prompt
        dict(name="prompt-video", op="prompt", dtype="bf16", B=1, lo=25119, hi=25119, Hq=28, Hkv=4, D=128, causal=True),
        # a batch of text prompts of very different lengths
        dict(name="prompt-packed-b16", op="prompt", dtype="bf16", B=16, lo=1, hi=2048, Hq=28, Hkv=4, D=128, causal=True),
        # image patches attending to their whole frame
        dict(name="prompt-frames", op="prompt", dtype="bf16", B=32, lo=576, hi=576, Hq=16, Hkv=16, D=64, causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _draw_rope(rng, D):
    kind = rng.choice(["none", "linear", "ntk", "parts", "yarn"])
    rot = rng.choice([D, D, D // 2, D // 4, 20])
    low, high = (1.0, 4.0) if kind == "parts" else (1.0, 32.0)
    return _rope(rng.choice(["half", "interleaved"]), rot, rng.choice([1e4, 5e5, 1e6]), kind,
                 1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0]), 8192, low, high)


def _draw_heads(rng):
    Hq, Hkv = rng.choice([(4, 1), (8, 8), (16, 16), (28, 4), (64, 8), (32, 2), (12, 4)])
    return dict(Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128]))


def draw(rng):
    op = rng.choice(["rotary", "append", "paged", "paged", "prompt", "prompt"])
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    if op == "rotary":
        D, H = rng.choice([64, 128]), rng.choice([1, 4, 8, 28, 64])
        N = _log_int(rng, 1, min(32768, 25119 * 28 * 128 // (H * D * (2 if dtype == "fp32" else 1))))
        return dict(op=op, dtype=dtype, N=N, H=H, D=D, pos0=rng.choice([0, 0, 1000, 1000000]), **_draw_rope(rng, D))
    heads = _draw_heads(rng)
    if op == "append":
        B = _log_int(rng, 1, 64)
        q_hi = _log_int(rng, 1, max(1, 8192 // B))
        room = max(1, 32768 // B - q_hi)
        kv_lo = q_hi + rng.randrange(0, room) // 2
        return dict(op=op, dtype=dtype, B=B, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, kv_lo=kv_lo,
                    kv_hi=kv_lo + rng.randrange(0, room) // 2, page=rng.choice([1, 16, 24, 64, 128, 256]),
                    **heads, **_draw_rope(rng, heads["D"]))
    causal = rng.random() < 0.8
    if op == "paged":
        while True:
            B = _log_int(rng, 1, 64)
            q_hi = _log_int(rng, 1, 2048)
            kv_hi = max(q_hi, _log_int(rng, 64, 40000))
            fl = 4.0 * B * q_hi * kv_hi * heads["Hq"] * heads["D"]
            by = 4.0 * B * kv_hi * heads["Hkv"] * heads["D"] * (2 if dtype == "fp32" else 1)
            if fl < (4e10 if dtype == "fp32" else 1.5e12) and by < 2e9:
                break
        return dict(op=op, dtype=dtype, B=B, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi,
                    kv_lo=max(q_hi, rng.choice([1, kv_hi // 8, kv_hi])), kv_hi=kv_hi,
                    page=rng.choice([8, 16, 16, 24, 64, 80, 128, 256, 5]), causal=causal, **heads)
    while True:
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, 16384)
        fl = 4.0 * B * hi * hi * heads["Hq"] * heads["D"]
        if fl < (4e10 if dtype == "fp32" else 2e12):
            break
    return dict(op=op, dtype=dtype, B=B, lo=rng.choice([0, 1, max(1, hi // 4), hi]), hi=hi, causal=causal, **heads)


# --------------------------------------------------------------------------
# lengths: fixed by the case, so that every seed does the same amount of work
# --------------------------------------------------------------------------

def _spread(n, lo, hi, salt):
    """n whole numbers from lo to hi, both among them where n > 1, spread over the logarithm."""
    if n == 1 or lo == hi:
        return [hi] * n
    vals = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    order = sorted(range(n), key=lambda i: (i * 2654435761 + salt * 40503) % 4294967291)
    return [vals[i] for i in order]


def _lengths(case):
    """(new tokens, cached positions with them) of each sequence."""
    if case["op"] == "prompt":
        q = _spread(case["B"], case["lo"], case["hi"], 1)
        return q, q
    q = _spread(case["B"], case["q_lo"], case["q_hi"], 1)
    kv = _spread(case["B"], case["kv_lo"], case["kv_hi"], 2)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _pairs(q, kv, causal):
    """Visible (row, key) pairs."""
    return sum(a * b - (a * (a - 1) // 2 if causal else 0) for a, b in zip(q, kv))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        n = case["N"] * case["H"]
        return {"bytes": 2 * n * case["D"] * e + 4 * case["N"], "flops": 3 * n * case["rot"]}
    q, kv = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        n = sum(q)
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * D * e + 4 * n, "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    return {"bytes": 2 * sum(q) * Hq * D * e + 2 * sum(b for a, b in zip(q, kv) if a) * Hkv * D * e,
            "flops": 4 * Hq * D * _pairs(q, kv, case["causal"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _cumulative(lens):
    return [0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, sd=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sd).to(dt)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case}
    if case["op"] == "rotary":
        s["x"] = normal(case["N"], case["H"], case["D"])
        s["positions"] = torch.arange(case["pos0"], case["pos0"] + case["N"], dtype=torch.int32, device=dev)
        s["y"] = torch.empty_like(s["x"])
    else:
        q, kv = _lengths(case)
        n, Hq, Hkv, D = sum(q), case["Hq"], case["Hkv"], case["D"]
        s["q_lens"], s["kv_lens"] = q, kv
        s["cu"], s["kv_len"] = i32(_cumulative(q)), i32(kv)
        s["q"] = normal(n, Hq, D, sd=2.0)          # scores of about +-2 once scaled
        s["scale"] = 1.0 / math.sqrt(D)
        s["max_q"], s["max_kv"] = max(q), max(kv)
        s["out"] = torch.empty(n, Hq, D, dtype=dt, device=dev)
    if case["op"] in ("append", "prompt"):
        # the projections of the new tokens, side by side as a fused projection leaves them
        kv_new = normal(n, 2 * Hkv, D)
        s["k"], s["v"] = kv_new[:, :Hkv], kv_new[:, Hkv:]
    if case["op"] in ("append", "paged"):
        # a pool with a few spare pages, handed out in random order
        page = case["page"]
        counts = [-(-b // page) for b in kv]
        n_pages = sum(counts) + 3
        ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        s["table"] = torch.zeros(len(kv), max(counts + [1]), dtype=torch.int32, device=dev)
        at = 0
        for b, c in enumerate(counts):
            s["table"][b, :c] = ids[at:at + c]
            at += c
        s["k_pages"] = normal(n_pages, page, Hkv, D)
        s["v_pages"] = normal(n_pages, page, Hkv, D)
    if case["op"] == "append":
        s["positions"] = i32([p for a, b in zip(q, kv) for p in range(b - a, b)])
    if "rot" in case:
        s["freqs"] = _frequencies(case).to(dev)
        s["magnitude"] = _magnitude(case)
    if own:
        from serving_sd_verify_gb300 import sd_verify as S
        if "rot" in case:
            turns, s["magnitude"] = S.sd_rotary_table(case["rot"], case["theta"], scaling=case["scaling"],
                                                      factor=case["factor"], original_max=case["original"],
                                                      low=case["low"], high=case["high"])
            s["turns"] = turns.to(dev)
        if case["op"] in ("paged", "prompt"):
            s["ws"] = S.workspace(S.sd_paged_attention_workspace_size(
                n, case["B"], s["max_q"], Hq, Hkv, D, s["max_kv"], S.SD_BF16 if dt == torch.bfloat16 else S.SD_FP32))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from serving_sd_verify_gb300 import sd_verify as S
    c = s["case"]
    if c["op"] == "rotary":
        S.sd_rotary(s["x"], s["y"], s["positions"], s["turns"], magnitude=s["magnitude"], layout=c["layout"])
        return s["y"]
    if c["op"] == "append":
        S.sd_rotary_append_paged(s["q"], s["k"], s["v"], s["out"], s["positions"], s["turns"], s["cu"], s["kv_len"],
                                 s["table"], s["k_pages"], s["v_pages"], magnitude=s["magnitude"], layout=c["layout"])
        return s["out"], s["k_pages"], s["v_pages"]
    if c["op"] == "paged":
        S.sd_paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["kv_len"], s["max_q"],
                             s["max_kv"], s["out"], s["scale"], s["ws"], causal=c["causal"])
        return s["out"]
    S.sd_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["max_q"], s["out"], s["scale"], s["ws"],
                          causal=c["causal"])
    return s["out"]


def _frequencies(case):
    """Radians per position of each turned pair, in 64 bits."""
    rot, theta, f = case["rot"], case["theta"], case["factor"]
    if case["scaling"] == "ntk":
        theta = theta * f ** (rot / (rot - 2))
    w = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] in ("parts", "yarn"):
        turns = case["original"] * w / (2 * math.pi)      # over the original context
        keep = ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0, 1)
        w = w / f * (1 - keep) + w * keep
    return w


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _turn(x, positions, s):
    c = s["case"]
    angle = positions.double()[:, None] * s["freqs"][None, :]
    cos = (angle.cos() * s["magnitude"]).float()[:, None, :]
    sin = (angle.sin() * s["magnitude"]).float()[:, None, :]
    y = x.float()
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _attend(q, k, v, scale, causal, out):
    """One sequence: q [n, Hq, D], k and v [m, Hkv, D]; row i sees m - n + i + 1 keys, or all."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    qs = q.float().reshape(n, Hkv, G, D).permute(1, 2, 0, 3)       # Hkv, G, n, D
    ks, vs = k.float().permute(1, 2, 0), v.float().permute(1, 0, 2)
    rows = max(1, min(n, (1 << 29) // (Hq * m)))
    col = torch.arange(m, device=q.device)
    for r in range(0, n, rows):
        e = min(n, r + rows)
        sc = torch.matmul(qs[:, :, r:e].reshape(Hkv, G * (e - r), D), ks) * scale
        if causal:
            limit = torch.arange(m - n + r, m - n + e, device=q.device).repeat(G)
            sc = sc.masked_fill(col[None, None, :] > limit[None, :, None], -math.inf)
        p = (sc - sc.amax(-1, keepdim=True)).exp()
        o = torch.matmul(p, vs) / p.sum(-1, keepdim=True)
        out[r:e] = o.reshape(Hkv, G, e - r, D).permute(2, 0, 1, 3).reshape(e - r, Hq, D).to(out.dtype)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        s["y"].copy_(_turn(s["x"], s["positions"], s))
        return s["y"]
    if c["op"] == "append":
        s["out"].copy_(_turn(s["q"], s["positions"], s))
        k = _turn(s["k"], s["positions"], s)
        at = 0
        for b, (a, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
            p = torch.arange(m - a, m, device=k.device)
            pg, sl = s["table"][b, p // c["page"]].long(), p % c["page"]
            s["k_pages"][pg, sl] = k[at:at + a]
            s["v_pages"][pg, sl] = s["v"][at:at + a]
            at += a
        return s["out"], s["k_pages"], s["v_pages"]
    at = 0
    for b, (a, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if a:
            if c["op"] == "paged":
                p = torch.arange(m, device=s["q"].device)
                pg, sl = s["table"][b, p // c["page"]].long(), p % c["page"]
                k, v = s["k_pages"][pg, sl], s["v_pages"][pg, sl]
            else:
                k, v = s["k"][at:at + a], s["v"][at:at + a]
            _attend(s["q"][at:at + a], k, v, s["scale"], c["causal"], s["out"][at:at + a])
        at += a
    return s["out"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 2.4e12:
        return None
    s = prepare(case, seed)
    dev = torch.device("cuda")
    if "rot" in case:
        # pair i turns by pos * w_i, as a product of complex numbers
        w = torch.tensor([_radians(case, i) for i in range(case["rot"] // 2)], dtype=torch.float64, device=dev)
        unit = torch.polar(torch.full_like(w, _magnitude(case)).expand(len(s["positions"]), -1).contiguous(),
                           s["positions"].double()[:, None] * w)
        half = case["rot"] // 2

        def turn(x):
            y = x.double().clone()
            first = torch.arange(half, device=dev) * (1 if case["layout"] == "half" else 2)
            second = first + (half if case["layout"] == "half" else 1)
            z = torch.complex(y[..., first], y[..., second]) * unit[:, None, :]
            y[..., first], y[..., second] = z.real, z.imag
            return y
        if case["op"] == "rotary":
            return turn(s["x"])
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        seq = torch.repeat_interleave(torch.arange(case["B"], device=dev),
                                      torch.tensor(s["q_lens"], device=dev))
        pos = s["positions"].long()
        flat = s["table"][seq, pos // case["page"]].long() * case["page"] + pos % case["page"]
        kp.view(-1, *kp.shape[2:])[flat] = turn(s["k"])
        vp.view(-1, *vp.shape[2:])[flat] = s["v"].double()
        return turn(s["q"]), kp, vp
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    at = 0
    for b, (a, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if a == 0:
            continue
        if case["op"] == "paged":
            n_pg = -(-m // case["page"])
            ids = s["table"][b, :n_pg].long()
            K = s["k_pages"][ids].reshape(-1, Hkv, D)[:m].double()
            V = s["v_pages"][ids].reshape(-1, Hkv, D)[:m].double()
        else:
            K, V = s["k"][at:at + a].double(), s["v"][at:at + a].double()
        for h in range(Hq):
            kh, vh = K[:, h * Hkv // Hq], V[:, h * Hkv // Hq]
            for r in range(0, a, 4096):
                rows = s["q"][at + r:at + min(a, r + 4096), h].double()
                seen = m if not case["causal"] else m - a + r + len(rows)
                z = rows @ kh[:seen].T * s["scale"]
                if case["causal"]:
                    z += torch.full_like(z, -math.inf).triu(m - a + r + 1)
                out[at + r:at + r + len(rows), h] = torch.softmax(z, -1) @ vh[:seen]
        at += a
    return out


def _radians(case, i):
    """Radians per position of pair i."""
    R, f = case["rot"], case["factor"]
    w = math.pow(case["theta"], -2.0 * i / R)
    if case["scaling"] == "none":
        return w
    if case["scaling"] == "linear":
        return w / f
    if case["scaling"] == "ntk":
        return w * math.pow(f, -2.0 * i / (R - 2))
    # by parts: pairs that turn more than `high` times over the original context stay, those
    # under `low` are stretched by the factor, those between are blended
    r = case["original"] * w / (2.0 * math.pi)
    if r >= case["high"]:
        return w
    if r <= case["low"]:
        return w / f
    g = (r - case["low"]) / (case["high"] - case["low"])
    return (1.0 - g) * w / f + g * w
