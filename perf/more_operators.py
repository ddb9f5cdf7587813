"""Performance cases of the operators around a quantised paged cache: norms of queries and keys with
rotary positions of several axes, the same with the write into a paged cache (as it is, or in 8 bits with
a scale per row), attention over the 8-bit cache, attention of drafted trees over either cache, and the
move of an accepted tree path in it.

Each case is one call.  `run` computes it either in plain torch operations (own = False) or
through the library's entry points (own = True); `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_TOP = 448.0            # the largest e4m3 value
_TINY = 2.0 ** -100     # a row's largest value is taken as this at least


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _axes(layout="half", rot=128, theta=1e6, a0=16, a1=24, a2=24, order="blocks", restart=False, norm=True):
    """a0, a1, a2: pairs that turn by each axis' position; restart: each axis has its own frequencies from the first on."""
    return dict(layout=layout, rot=rot, theta=theta, a0=a0, a1=a1, a2=a2, order=order, restart=restart, norm=norm)


def listed():
    return [
        # queries and keys of a 25,119-token video prompt: time, height and width
        dict(name="norm-rotary-video", op="norm", dtype="bf16", N=25119, Hq=28, Hkv=4, D=128, **_axes()),
        # the patches of one frame in an image tower: rows and columns, fp32
        dict(name="norm-rotary-patches", op="norm", dtype="fp32", N=576, Hq=16, Hkv=16, D=64,
             **_axes("interleaved", 64, 1e4, 16, 16, 0, "blocks", True)),
        # a whole video prompt enters the 8-bit cache
        dict(name="append-e4m3-video", op="append", cache="e4m3", dtype="bf16", B=1, q_lo=25119, q_hi=25119, kv_lo=25119,
             kv_hi=25119, page=64, Hq=28, Hkv=4, D=128, **_axes()),
        # 16 drafted slots of eight ragged sequences enter it
        dict(name="append-e4m3-verify-b8", op="append", cache="e4m3", dtype="bf16", B=8, q_lo=16, q_hi=16, kv_lo=4096,
             kv_hi=32768, page=16, Hq=28, Hkv=4, D=128, **_axes(order="stripes")),
        # a chunk of a prompt enters the cache of the larger model, unquantised
        dict(name="append-chunk", op="append", cache="same", dtype="bf16", B=1, q_lo=2048, q_hi=2048, kv_lo=32768,
             kv_hi=32768, page=128, Hq=64, Hkv=8, D=128, **_axes()),
        # plain decoding of one sequence over the video's context
        dict(name="e4m3-decode-b1", op="attend", cache="e4m3", dtype="bf16", B=1, q_lo=1, q_hi=1, kv_lo=25119, kv_hi=25119,
             page=64, Hq=28, Hkv=4, D=128, causal=True),
        # plain decoding of a batch of conversations
        dict(name="e4m3-decode-b64", op="attend", cache="e4m3", dtype="bf16", B=64, q_lo=1, q_hi=1, kv_lo=1000, kv_hi=9000,
             page=16, Hq=28, Hkv=4, D=128, causal=True),
        # a chunk of a long prompt over what is already cached, the larger model's heads
        dict(name="e4m3-chunk", op="attend", cache="e4m3", dtype="bf16", B=1, q_lo=2048, q_hi=2048, kv_lo=32768, kv_hi=32768,
             page=128, Hq=64, Hkv=8, D=128, causal=True),
        # one drafted tree of 60 nodes over the video's context
        dict(name="tree-b1", op="tree", cache="same", dtype="bf16", B=1, q_lo=60, q_hi=60, kv_lo=25119, kv_hi=25119, page=64,
             Hq=28, Hkv=4, D=128),
        # a ragged batch of trees over the 8-bit cache
        dict(name="tree-e4m3-b8", op="tree", cache="e4m3", dtype="bf16", B=8, q_lo=24, q_hi=60, kv_lo=4096, kv_hi=32768,
             page=16, Hq=28, Hkv=4, D=128),
        # the accepted path of one tree
        dict(name="compact-b1", op="compact", cache="same", dtype="bf16", B=1, T=60, kept=7, kv_lo=25119, kv_hi=25119, page=64,
             Hkv=4, D=128),
        # and of a batch of them in the 8-bit cache
        dict(name="compact-e4m3-b64", op="compact", cache="e4m3", dtype="bf16", B=64, T=60, kept=9, kv_lo=1000, kv_hi=9000,
             page=16, Hkv=8, D=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _draw_axes(rng, D):
    rot = rng.choice([D, D, D // 2])
    half = rot // 2
    n = rng.choice([1, 2, 3, 3])
    parts = [half, 0, 0]
    if n > 1:
        parts = [half - (n - 1) * (half // n)] + [half // n] * (n - 1) + [0] * (3 - n)
    order = rng.choice(["blocks", "stripes"])
    return _axes(rng.choice(["half", "interleaved"]), rot, rng.choice([1e4, 5e5, 1e6]), *parts, order,
                 order == "blocks" and rng.random() < 0.3, rng.random() < 0.8)


def _draw_heads(rng):
    Hq, Hkv = rng.choice([(4, 1), (8, 8), (16, 16), (28, 4), (64, 8), (32, 2), (12, 4)])
    return dict(Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128]))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend", "tree", "tree", "compact"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    cache = "e4m3" if rng.random() < 0.7 else "same"
    h = _draw_heads(rng)
    if op == "norm":
        room = 25119 * 32 * 128 // ((h["Hq"] + h["Hkv"]) * h["D"] * (2 if dtype == "fp32" else 1))
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, min(32768, room)), **h, **_draw_axes(rng, h["D"]))
    if op == "append":
        B = _log_int(rng, 1, 64)
        q_hi = _log_int(rng, 1, max(1, 8192 // B))
        room = max(1, 32768 // B - q_hi)
        kv_lo = q_hi + rng.randrange(0, room) // 2
        return dict(op=op, cache=cache, dtype=dtype, B=B, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, kv_lo=kv_lo,
                    kv_hi=kv_lo + rng.randrange(0, room) // 2, page=rng.choice([1, 16, 24, 64, 128, 256]), **h,
                    **_draw_axes(rng, h["D"]))
    if op == "compact":
        T = rng.randrange(20, 65)
        B = _log_int(rng, 1, 64)
        kv_lo = _log_int(rng, T, 4000)
        return dict(op=op, cache=cache, dtype=dtype, B=B, T=T, kept=rng.randrange(0, 10), kv_lo=kv_lo,
                    kv_hi=kv_lo + rng.randrange(0, 40000 // B), page=rng.choice([1, 16, 24, 64, 128]), Hkv=h["Hkv"], D=h["D"])
    while True:
        B = _log_int(rng, 1, 64)
        q_hi = rng.randrange(1, 65) if op == "tree" else _log_int(rng, 1, 2048)
        kv_hi = max(q_hi, _log_int(rng, 64, 40000))
        fl = 4.0 * B * q_hi * kv_hi * h["Hq"] * h["D"]
        if fl < (4e10 if dtype == "fp32" else 1.0e12) and 2.0 * B * kv_hi * h["Hkv"] * h["D"] < 1e9:
            break
    c = dict(op=op, cache=cache if op == "tree" else "e4m3", dtype=dtype, B=B, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi,
             kv_lo=max(q_hi, rng.choice([1, kv_hi // 8, kv_hi])), kv_hi=kv_hi, page=rng.choice([8, 16, 16, 24, 64, 80, 128, 256, 5]),
             **h)
    return c if op == "tree" else dict(c, causal=rng.random() < 0.8)


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
    if case["op"] == "norm":
        return [case["N"]], [case["N"]]
    q = [case["T"]] * case["B"] if case["op"] == "compact" else _spread(case["B"], case["q_lo"], case["q_hi"], 1)
    kv = _spread(case["B"], case["kv_lo"], case["kv_hi"], 2)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _row(case):
    """Bytes of one cached row of K or V."""
    return case["D"] + 4 if case["cache"] == "e4m3" else case["D"] * (2 if case["dtype"] == "bf16" else 4)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    q, kv = _lengths(case)
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "compact":
        return {"bytes": case["B"] * (4 * case["kept"] * Hkv * _row(case) + 4 * case["kept"] + 8), "flops": 0}
    Hq, n = case["Hq"], sum(q)
    if case["op"] == "norm":
        rows = n * (Hq + Hkv)
        return {"bytes": 2 * rows * D * e + 12 * n, "flops": rows * (4 * D + 3 * case["rot"])}
    if case["op"] == "append":
        return {"bytes": n * ((2 * Hq + 2 * Hkv) * D * e + 2 * Hkv * _row(case) + 12),
                "flops": n * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    pairs = sum(a * b - (a * (a - 1) // 2 if case.get("causal", True) else 0) for a, b in zip(q, kv))
    return {"bytes": 2 * n * Hq * D * e + 2 * sum(b for a, b in zip(q, kv) if a) * Hkv * _row(case),
            "flops": 4 * Hq * D * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _cumulative(lens):
    return [0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist()


def _quantise(x):
    """(codes, scale) of rows of 32-bit values."""
    top = x.abs().amax(-1, keepdim=True).clamp_min(_TINY)
    return (x * (_TOP / top)).clamp(-_TOP, _TOP).to(torch.float8_e4m3fn), (top / _TOP)[..., 0]


def _video_positions(n):
    """Time, height and width of n tokens: 64 of text, then frames of 14 x 14."""
    i = torch.arange(n)
    f = (i - 64).clamp_min(0)
    return torch.stack([torch.where(i < 64, i, 64 + f // 196), torch.where(i < 64, i, 64 + f % 196 // 14),
                        torch.where(i < 64, i, 64 + f % 14)]).to(torch.int32)


def _tree(rng, n):
    """Ancestor masks (with the node itself) of a random tree of n nodes in topological order."""
    masks = [1]
    for j in range(1, n):
        parent = 0 if j <= 10 else int(rng[j] * j * 0.7)
        masks.append(masks[parent] | 1 << j)
    return [m - (1 << 64) if m >> 63 else m for m in masks[:n]]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    q, kv = _lengths(case)
    n, Hkv, D = sum(q), case["Hkv"], case["D"]

    def normal(*shape, sd=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sd).to(dt)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case, "q_lens": q, "kv_lens": kv}
    if "Hq" in case:
        Hq = case["Hq"]
        s["q"] = normal(n, Hq, D, sd=2.0)          # scores of about +-2 once scaled
        s["out"] = torch.empty(n, Hq, D, dtype=dt, device=dev)
    if case["op"] in ("norm", "append"):
        # the projections of the new tokens, side by side as a fused projection leaves them
        new = normal(n, 2 * Hkv, D)
        s["k"], s["v"] = new[:, :Hkv], new[:, Hkv:]
        s["q_weight"], s["k_weight"] = (torch.ones(D, device=dev).to(dt) + normal(D, sd=0.2) for _ in range(2))
        s["eps"] = 1e-6
        p = [_video_positions(b)[:, b - a:] for a, b in zip(q, kv)]
        s["positions"] = torch.cat(p, 1).to(dev)[:_n_axes(case)].contiguous()
        s["axis"] = torch.tensor(_pair_axes(case), device=dev)
        s["freqs"] = _frequencies(case).to(dev)
    if case["op"] == "norm":
        s["k_out"] = torch.empty(n, Hkv, D, dtype=dt, device=dev)
    else:
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
        s["k_scale"] = s["v_scale"] = None
        for x in ("k", "v"):
            rows = normal(n_pages, page, Hkv, D)
            if case["cache"] == "e4m3":
                rows, scale = _quantise(rows.float())
                s[x + "_scale"] = scale.transpose(1, 2).contiguous()      # pages, heads, slots
            s[x + "_pages"] = rows
        s["cu"], s["kv_len"] = i32(_cumulative(q)), i32(kv)
    if case["op"] in ("attend", "tree"):
        s["scale"] = 1.0 / math.sqrt(D)
        s["max_q"], s["max_kv"] = max(q), max(kv)
    if case["op"] == "tree":
        draws = torch.rand(len(q), 64, generator=g, device=dev).tolist()
        s["mask"] = torch.tensor([m for r, a in zip(draws, q) for m in _tree(r, a)], dtype=torch.int64, device=dev)
    if case["op"] == "compact":
        # the kept nodes of each path: beyond the slots that they move to, as they are where the drafts branch early
        T, kept = case["T"], case["kept"]
        s["ctx_len"] = s["kv_len"] - (T - 1)
        order = torch.rand(len(q), T - 1 - kept, generator=g, device=dev).argsort(1)[:, :kept].sort(1).values + 1 + kept
        s["path"] = torch.full((len(q), T), -1, dtype=torch.int32, device=dev)
        s["path"][:, :kept] = order.to(torch.int32)
        s["n_accepted"] = torch.full((len(q),), kept, dtype=torch.int32, device=dev)
    if own:
        from serving_sd_verify_gb300 import sd_verify as S
        if "axis" in s:
            if case["restart"]:
                turns = torch.cat([S.sd_rotary_table(2 * p, case["theta"])[0] for p in _parts(case)])
            else:
                turns = S.sd_rotary_table(case["rot"], case["theta"])[0]
            s["turns"] = turns.to(dev)
        if case["op"] in ("attend", "tree"):
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
    if c["op"] in ("norm", "append"):
        w = dict(q_weight=s["q_weight"], k_weight=s["k_weight"]) if c["norm"] else {}
        w.update(eps=s["eps"], axes=_parts(c), axes_order=c["order"], layout=c["layout"])
    if c["op"] == "norm":
        S.sd_norm_rotary(s["q"], s["out"], s["k"], s["k_out"], s["positions"], s["turns"], **w)
        return s["out"], s["k_out"]
    if c["op"] == "append":
        S.sd_norm_rotary_append_paged(s["q"], s["k"], s["v"], s["out"], s["positions"], s["turns"], s["cu"], s["kv_len"],
                                      s["table"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], **w)
        return s["out"], _cache_of(s)
    if c["op"] == "attend":
        S.sd_paged_attention_e4m3(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                                  s["kv_len"], s["max_q"], s["max_kv"], s["out"], s["scale"], s["ws"], causal=c["causal"])
        return s["out"]
    if c["op"] == "tree":
        S.sd_paged_tree_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["mask"], s["cu"], s["kv_len"],
                                  s["max_q"], s["max_kv"], s["out"], s["scale"], s["ws"], s["k_scale"], s["v_scale"])
        return s["out"]
    S.sd_compact_tree_paged(s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s["path"], s["n_accepted"],
                            s["k_scale"], s["v_scale"])
    return _cache_of(s)


def _cache_of(s):
    return [s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale") if s[x] is not None]


def _parts(case):
    return [p for p in (case["a0"], case["a1"], case["a2"]) if p]


def _n_axes(case):
    return len(_parts(case))


def _pair_axes(case):
    """The axis of each turned pair: in blocks, or by turns while an axis has pairs left (the first takes what is over)."""
    parts = _parts(case)
    if case["order"] == "blocks":
        return [a for a, p in enumerate(parts) for _ in range(p)]
    n = len(parts)
    return [i % n if i % n and i < n * parts[i % n] else 0 for i in range(sum(parts))]


def _frequencies(case):
    """Radians per position of each turned pair, in 64 bits."""
    if not case["restart"]:
        return case["theta"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    return torch.cat([case["theta"] ** (-torch.arange(p, dtype=torch.float64) / p) for p in _parts(case)])


def _norm(x, weight, s):
    x = x.float()
    if not s["case"]["norm"]:
        return x
    return x * (1.0 / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt()) * weight.float()


def _turn(y, s):
    """32-bit rows with the positions applied."""
    c = s["case"]
    angle = s["positions"].double()[s["axis"]].T * s["freqs"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1)


def _new_slots(s):
    """(page, slot) of every new token."""
    q_len = s["cu"].diff().long()
    n = s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(s["q_lens"]), device=q_len.device), q_len, output_size=n)
    pos = torch.arange(n, device=q_len.device) - s["cu"][seq] + (s["kv_len"] - q_len)[seq]
    page = s["case"]["page"]
    return s["table"][seq, pos // page].long(), pos % page


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _all_rows(s, x):
    """K or V of every sequence as 32-bit values, [B, table columns * page, Hkv, D]."""
    c = s["case"]
    ids = s["table"].long()
    rows = _bytes(s[x + "_pages"])[ids]
    if c["cache"] == "e4m3":
        rows = rows.view(torch.float8_e4m3fn).float() * s[x + "_scale"][ids].transpose(2, 3)[..., None]
    return rows.float().flatten(1, 2)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        s["out"].copy_(_turn(_norm(s["q"], s["q_weight"], s), s))
        s["k_out"].copy_(_turn(_norm(s["k"], s["k_weight"], s), s))
        return s["out"], s["k_out"]
    if c["op"] == "append":
        s["out"].copy_(_turn(_norm(s["q"], s["q_weight"], s), s))
        pg, sl = _new_slots(s)
        k, v = _turn(_norm(s["k"], s["k_weight"], s), s), s["v"].float()
        if c["cache"] == "e4m3":
            k, ks = _quantise(k)
            v, vs = _quantise(v)
            s["k_scale"][pg, :, sl], s["v_scale"][pg, :, sl] = ks, vs
        _bytes(s["k_pages"])[pg, sl] = _bytes(k.to(s["k_pages"].dtype))
        _bytes(s["v_pages"])[pg, sl] = _bytes(v.to(s["v_pages"].dtype))
        return s["out"], _cache_of(s)
    if c["op"] == "compact":
        T, kept, page = c["T"], c["kept"], c["page"]
        seq = torch.arange(c["B"], device=s["table"].device)[:, None]
        old = s["ctx_len"].long()[:, None] - 1 + s["path"][:, :kept].long()
        new = s["ctx_len"].long()[:, None] + torch.arange(kept, device=seq.device)
        a, b = s["table"][seq, old // page].long(), s["table"][seq, new // page].long()
        for x in ("k", "v"):
            rows = _bytes(s[x + "_pages"])
            rows[b, new % page] = rows[a, old % page]
            if c["cache"] == "e4m3":
                s[x + "_scale"][b, :, new % page] = s[x + "_scale"][a, :, old % page]
        return _cache_of(s)
    # attention: the batch padded to its longest sequences
    B, Hq, Hkv, D, Q = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_q"]
    G = Hq // Hkv
    cu, kv = s["cu"].long(), s["kv_len"].long()
    q_len = cu.diff()
    i = torch.arange(Q, device=cu.device)
    rows = (cu[:-1, None] + i).clamp_max(len(s["q"]) - 1)
    qs = s["q"][rows].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    k, v = _all_rows(s, "k")[:, :s["max_kv"]], _all_rows(s, "v")[:, :s["max_kv"]]
    sc = torch.matmul(qs, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, Hkv, G, Q, -1)
    j = torch.arange(sc.shape[-1], device=cu.device)
    first = (kv - q_len)[:, None, None]                    # the first new token's position
    if c["op"] == "tree":
        bits = s["mask"][rows][:, :, None] >> (j[None, None, :] - first).clamp(0, 63) & 1
        seen = (j < first) | ((bits == 1) & (j < kv[:, None, None]))
    elif c["causal"]:
        seen = j <= first + i[None, :, None]
    else:
        seen = (j < kv[:, None, None]).expand(B, Q, -1)
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    z = p.sum(-1, keepdim=True)
    # slots past a sequence's end hold no values of it
    v = v * (j < kv[:, None])[:, :, None, None]
    o = torch.matmul(p.view(B, Hkv, G * Q, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, G, Q, D) / z
    real = i < q_len[:, None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)[real])
    return s["out"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _on_grid(y):
    """Nearest e4m3 value, ties to the even one: steps of an eighth of the power of two below, 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-_TOP, _TOP)


def exact(case, seed):
    if work(case)["flops"] > 2.4e12:
        return None
    s = prepare(case, seed)
    dev = torch.device("cuda")
    e4m3 = case.get("cache") == "e4m3"
    if case["op"] == "norm":
        return _exact_rows(s, "q"), _exact_rows(s, "k")
    page = case["page"]
    cache = [s[x].double() for x in ("k_pages", "v_pages", "k_scale", "v_scale") if s[x] is not None]
    if case["op"] == "append":
        new = [_exact_rows(s, "k"), s["v"].double()]
        at = 0
        for b, (a, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
            pos = torch.arange(m - a, m, device=dev)
            pg, sl = s["table"][b].long()[torch.div(pos, page, rounding_mode="floor")], torch.remainder(pos, page)
            for x in range(2):
                rows = new[x][at:at + a]
                if e4m3:
                    scale = rows.abs().amax(-1).clamp_min(_TINY) / _TOP
                    cache[2 + x][pg, :, sl] = scale
                    rows = _on_grid(rows / scale[..., None])
                cache[x][pg, sl] = rows
            at += a
        return _exact_rows(s, "q"), cache
    if case["op"] == "compact":
        for b in range(case["B"]):
            first = int(s["ctx_len"][b]) - 1
            for d in range(case["kept"]):
                src, dst = first + int(s["path"][b, d]), first + 1 + d
                a, z = int(s["table"][b, src // page]), int(s["table"][b, dst // page])
                for x in range(2):
                    cache[x][z, dst % page] = cache[x][a, src % page]
                    if e4m3:
                        cache[2 + x][z, :, dst % page] = cache[2 + x][a, :, src % page]
        return cache
    Hq, Hkv = case["Hq"], case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    at = 0
    for b, (a, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if a == 0:
            continue
        ids = s["table"][b, :-(-m // page)].long()
        K, V = (_bytes(s[x])[ids].view(s[x].dtype).double() for x in ("k_pages", "v_pages"))
        if e4m3:
            K = K * s["k_scale"][ids].double().permute(0, 2, 1).unsqueeze(-1)
            V = V * s["v_scale"][ids].double().permute(0, 2, 1).unsqueeze(-1)
        K, V = (x.reshape(-1, Hkv, case["D"])[:m] for x in (K, V))
        hide = torch.zeros(a, m, dtype=torch.bool, device=dev)
        if case["op"] == "tree":
            word = s["mask"][at:at + a]
            hide[:, m - a:] = torch.stack([(word & (1 << t if t < 63 else -(1 << 63))) == 0 for t in range(a)], 1)
        elif case["causal"]:
            hide = torch.ones(a, m, dtype=torch.bool, device=dev).triu(m - a + 1)
        for h in range(Hq):
            z = s["q"][at:at + a, h].double() @ K[:, h * Hkv // Hq].T * s["scale"]
            out[at:at + a, h] = torch.softmax(z.masked_fill(hide, -math.inf), -1) @ V[:, h * Hkv // Hq]
        at += a
    return out


def _exact_rows(s, x):
    """Queries or keys normed and turned, as products of complex numbers."""
    case = s["case"]
    y = s[x].double().clone()
    if case["norm"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["D"] + s["eps"]) * s[x + "_weight"].double()
    half = case["rot"] // 2
    dev = y.device
    angle = torch.stack([s["positions"][a].double() * _radians(case, i) for i, a in enumerate(_pair_axes(case))], 1)
    unit = torch.polar(torch.ones_like(angle), angle)
    first = torch.arange(half, device=dev) * (1 if case["layout"] == "half" else 2)
    second = first + (half if case["layout"] == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * unit[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _radians(case, i):
    """Radians per position of pair i."""
    if not case["restart"]:
        return math.pow(case["theta"], -2.0 * i / case["rot"])
    for p in _parts(case):
        if i < p:
            return math.pow(case["theta"], -float(i) / p)
        i -= p
