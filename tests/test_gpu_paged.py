"""Rotary positions, the paged K/V cache and packed attention against plain
64-bit implementations.

Bounds.  Rotary: the angle is right to 2^-32 turns plus the rounding of an
eighth of a turn to fp32, sincospif and the products round a few times more:
6 * 2^-24 (|a| + |b|) m in all, and the output's half step.
Attention: with s = scale q.k, the scores' error is at most
ds = (D + 4) 2^-24 scale sum |q_d k_d| (fp32 accumulation), so a weight is off
by 2 ds relative at most (its own and the maximum's), by 2^-21 from the
exponential and by n 2^-24 from sums of n terms: together `rel`.  The output is
off by at most rel * sum p |v|, by 2^-8 sum p |v| more where the weights are
rounded to bf16 (tensor cores), and by its own half step.  The roundings are
independent, so over many elements their root mean square is held to the
half steps taken in quadrature.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_LENGTH, BAD_PAGE, WAIT_GAVE_UP = 1 << 7, 1 << 8, 1 << 3


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    yield sd_verify
    sd_verify.sd_set_attention_path(0)
    sd_verify.sd_set_wait_test(0, 0)


@pytest.fixture(autouse=True)
def _clean(S):
    yield
    S.sd_set_attention_path(0)
    S.sd_set_wait_test(0, 0)


def cumulative(lens):
    return torch.tensor([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int32)


def randn(gen, *shape, dtype=torch.float32, sd=1.0):
    return (torch.randn(*shape, generator=gen) * sd).to(dtype)


def dt_code(S, dtype):
    return S.SD_BF16 if dtype == torch.bfloat16 else S.SD_FP32


# --------------------------------------------------------------------------
# plain implementations
# --------------------------------------------------------------------------

def ref_attend(q, k, v, scale, causal):
    """One sequence in fp64: (out, sum p|v|, sqrt(sum p^2 v^2), largest relative weight error)."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    mag, quad = out.clone(), out.clone()
    rel = 0.0
    if m == 0:
        return out, mag, quad, rel
    q, k, v = q.double(), k.double(), v.double()
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = q[:, h] @ kh.T * scale
        ab = q[:, h].abs() @ kh.abs().T * scale
        rel = max(rel, float(ab.max()) * (D + 4) * 2.0 ** -24)
        if causal:
            i = torch.arange(n)[:, None] + (m - n)
            s = s.masked_fill(torch.arange(m)[None] > i, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.where(s == -math.inf, torch.zeros(()).double(), (s - torch.where(top == -math.inf, 0.0, top)).exp())
        z = p.sum(-1, keepdim=True)
        p = torch.where(z > 0, p / z.clamp_min(1e-300), torch.zeros(()).double())
        out[:, h] = p @ vh
        mag[:, h] = p @ vh.abs()
        quad[:, h] = ((p * p) @ (vh * vh)).sqrt()
    return out, mag, quad, 2 * rel + 2.0 ** -21 + m * 2.0 ** -24


def check(got, want, mag, quad, rel, dtype, p_bf16):
    got = got.cpu().double()
    half = torch.finfo(dtype).eps / 2
    pr = 2.0 ** -8 if p_bf16 else 0.0
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    tol = (rel + pr) * mag * (1 + half) + half * want.abs() + 1e-37
    assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
    if got.numel() > 4096:
        rms = lambda x: float(x.pow(2).mean().sqrt())
        assert rms(err) <= rms(rel * mag) + math.sqrt((half * rms(want)) ** 2 + (pr * rms(quad)) ** 2)


def rope_ref(x, pos, R, theta, layout, m=1.0):
    y = x.double().clone()
    w = theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    ang = pos.double()[:, None, None] * w
    c, s = ang.cos() * m, ang.sin() * m
    i = torch.arange(R // 2)
    a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * c - v * s
    y[..., b] = v * c + u * s
    mag = torch.zeros_like(y)
    mag[..., a] = mag[..., b] = (u.abs() + v.abs()) * m
    return y, mag


def check_rope(got, want, mag, dtype):
    half = torch.finfo(dtype).eps / 2
    err = (got.cpu().double() - want).abs()
    slip = 6 * 2.0 ** -24 * mag
    assert (err <= slip * (1 + half) + half * want.abs()).all(), float(err.max())


# --------------------------------------------------------------------------
# rotary
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,H,D,R", [(1, 1, 64, 64), (5, 28, 128, 128), (33, 3, 128, 32), (7, 5, 64, 20), (3, 2, 30, 6),
                                     (130, 4, 96, 96)])
def test_rotary(S, dtype, layout, N, H, D, R):
    g = torch.Generator().manual_seed(N + R)
    x = randn(g, N, H, D, dtype=dtype)
    pos = torch.randint(-(1 << 20), 1 << 20, (N,), generator=g, dtype=torch.int32)
    pos[0] = 0
    turns, m = S.sd_rotary_table(R, 1e6)
    want, mag = rope_ref(x, pos, R, 1e6, layout)
    y = torch.full_like(x, 7.0).cuda()
    S.sd_rotary(x.cuda(), y, pos.cuda(), turns.cuda(), layout=layout)
    check_rope(y, want, mag, dtype)
    # in place, and a view whose rows start off 16 bytes (the scalar path): the same bits
    z = x.cuda()
    S.sd_rotary(z, z, pos.cuda(), turns.cuda(), layout=layout)
    assert torch.equal(z, y)
    wide = torch.zeros(N, H, D + 1, dtype=dtype, device="cuda")
    v = wide[:, :, 1:]
    v.copy_(x.cuda())
    S.sd_rotary(v, v, pos.cuda(), turns.cuda(), layout=layout)
    assert torch.equal(v, y) and float(wide[:, :, 0].abs().max()) == 0.0
    # head-major memory
    t = x.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    o = torch.empty(H, N, D, dtype=dtype, device="cuda").transpose(0, 1)
    S.sd_rotary(t, o, pos.cuda(), turns.cuda(), layout=layout)
    assert torch.equal(o, y)
    assert S.sd_fault_word() == 0


def test_rotary_far_positions_and_magnitude(S):
    """The fp64 frequency behind a word is off by a few of its 2^-53 (one power, one division): at
    position 2^31 - 1 that is 2^31 * 2^-50 radians for the first pairs, plus the bound above."""
    g = torch.Generator().manual_seed(3)
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 1, 123456789, 1], dtype=torch.int32)
    x = randn(g, 5, 2, 64)
    turns, m = S.sd_rotary_table(64, 1e4, scaling="yarn", factor=1.0, original_max=8192)
    assert m == 1.0
    y = torch.empty(5, 2, 64, device="cuda")
    S.sd_rotary(x.cuda(), y, pos.cuda(), turns.cuda(), magnitude=1.25)
    want, mag = rope_ref(x, pos, 64, 1e4, "half", 1.25)
    # the reference's own angle, rounded to fp64, is off by 2^31 * 2^-53 as well
    slip = (6 * 2.0 ** -24 + 2.0 ** 31 * 2.0 ** -49) * mag
    assert ((y.cpu().double() - want).abs() <= slip + 2.0 ** -24 * want.abs()).all()


def test_rotary_gradient_is_the_turn_back(S):
    """The map is linear and its transpose the turn by the negated position: <dy, R x> = <R' dy, x>,
    the formula's gradient, and differences give the same."""
    g = torch.Generator().manual_seed(4)
    N, H, D = 6, 3, 64
    x, dy = randn(g, N, H, D), randn(g, N, H, D)
    pos = torch.arange(100, 100 + N, dtype=torch.int32)
    turns, _ = S.sd_rotary_table(D, 1e4)
    gx = torch.empty(N, H, D, device="cuda")
    S.sd_rotary(dy.cuda(), gx, (-pos).cuda(), turns.cuda())
    xr = x.double().requires_grad_()
    w = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    c, s = (pos.double()[:, None, None] * w).cos(), (pos.double()[:, None, None] * w).sin()
    a, b = xr[..., :D // 2], xr[..., D // 2:]
    (torch.cat([a * c - b * s, b * c + a * s], -1) * dy.double()).sum().backward()
    mag = torch.cat([dy[..., :D // 2].abs() + dy[..., D // 2:].abs()] * 2, -1).double()
    assert ((gx.cpu().double() - xr.grad).abs() <= 7 * 2.0 ** -24 * mag).all()
    # differences: the map is linear, so one step of size 1 in one element is exact up to rounding
    e = torch.zeros(N, H, D)
    e[2, 1, 5] = 1.0
    ye = torch.empty(N, H, D, device="cuda")
    S.sd_rotary(e.cuda(), ye, pos.cuda(), turns.cuda())
    diff = float((ye.cpu().double() * dy.double()).sum())
    assert abs(diff - float(gx[2, 1, 5])) <= 14 * 2.0 ** -24 * float(mag[2, 1, 5])


# --------------------------------------------------------------------------
# a paged cache
# --------------------------------------------------------------------------

class Pool:
    """Pages handed out in random order; spare pages and unused table entries hold nonsense."""

    def __init__(self, g, kv_lens, page, Hkv, D, dtype, head_major=False, fill=float("nan")):
        need = [-(-n // page) for n in kv_lens]
        self.page, self.kv_lens, n = page, kv_lens, sum(need) + 2
        ids = torch.randperm(n, generator=g, dtype=torch.int64).to(torch.int32)
        self.table = torch.full((len(kv_lens), max(need + [1]) + 1), -5, dtype=torch.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = ids[at:at + c]
            at += c
        shape = (n, Hkv, page, D) if head_major else (n, page, Hkv, D)
        self.k, self.v = (torch.full(shape, fill, dtype=dtype) for _ in range(2))
        if head_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.head_major = head_major

    def slots(self, b, n=None):
        p = torch.arange(self.kv_lens[b] if n is None else n)
        return self.table[b, p // self.page].long(), p % self.page

    def write(self, b, k, v):
        i = self.slots(b)
        self.k[i], self.v[i] = k, v

    def cuda(self):
        dense = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.head_major else t.cuda()
        return dense(self.k), dense(self.v), self.table.cuda()


def paged_case(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, causal, path=0, head_major=False, seed=0, extra=3,
               sd=2.0, strided_q=False, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(q_lens)
    N = n + extra
    q = randn(g, N, Hq, D, dtype=dtype, sd=sd)
    pool = Pool(g, kv_lens, page, Hkv, D, dtype, head_major)
    ks, vs = [], []
    for b, m in enumerate(kv_lens):
        ks.append(randn(g, m, Hkv, D, dtype=dtype))
        vs.append((randn(g, m, Hkv, D) + offset).to(dtype))
        pool.write(b, ks[b], vs[b])
    scale = 1 / math.sqrt(D)
    kp, vp, table = pool.cuda()
    out = torch.full((N, Hq, D), 123.0, dtype=dtype, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(N, len(q_lens), max(q_lens), Hq, Hkv, D, max(kv_lens),
                                                         dt_code(S, dtype)))
    qd = q.cuda()
    if strided_q:
        wide = torch.full((N, Hq + 2, D + 8), float("nan"), dtype=dtype, device="cuda")
        wide[:, 1:Hq + 1, :D] = qd
        qd = wide[:, 1:Hq + 1, :D]
    S.sd_set_attention_path(path)
    args = (qd, kp, vp, table, cumulative(q_lens).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(),
            max(q_lens), max(kv_lens), out, scale, ws)
    S.sd_paged_attention(*args, causal=causal)
    torch.cuda.synchronize()
    used = S.sd_last_attention_path()[0]
    assert S.sd_fault_word() == 0
    assert int(ws[256:256 + 608].sum()) == 0, "counters not returned to zero"
    at = 0
    for b, c in enumerate(q_lens):
        if c:
            want = ref_attend(q[at:at + c], ks[b], vs[b], scale, causal)
            check(out[at:at + c], *want, dtype, used == 2)
        at += c
    assert bool((out[at:] == 123.0).all()), "rows behind the last sequence were written"
    return args, out


HEADS = [(28, 4, 128), (4, 1, 64), (8, 8, 64), (16, 2, 128), (64, 1, 128), (3, 1, 128), (64, 64, 64)]


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("q_lens,kv_lens,page", [
    ([1], [1], 16), ([1], [129], 8), ([0, 1, 2, 0], [5, 1, 200, 0], 16), ([16, 16, 16], [16, 700, 1500], 64),
    ([130, 1, 300, 37], [130, 129, 513, 1000], 24)])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention(S, dtype, path, Hq, Hkv, D, q_lens, kv_lens, page, causal):
    paged_case(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, causal, path)


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
@pytest.mark.parametrize("page", [8, 16, 40, 48, 64, 128, 256, 384])
def test_page_sizes_and_orders(S, dtype, path, page):
    paged_case(S, [3, 40], [257, 511], 28, 4, 128, dtype, page, True, path, seed=page)
    paged_case(S, [2, 9], [300, 77], 8, 2, 64, dtype, page, True, path, head_major=True, strided_q=True, seed=page + 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [1, 5, 12, 100])
def test_odd_pages_run_on_cuda_cores(S, dtype, page):
    paged_case(S, [3, 40], [257, 511], 28, 4, 128, dtype, page, True, seed=page)
    assert S.sd_last_attention_path()[0] == 1
    if dtype == torch.bfloat16:
        with pytest.raises(S.SdError) as e:
            paged_case(S, [3, 40], [257, 511], 28, 4, 128, dtype, page, True, path=2)
        assert e.value.status == S.SD_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
def test_rows_that_see_nothing_give_zeros(S, dtype, path):
    # more new tokens than cached positions: the first rows see nothing
    args, out = paged_case(S, [5, 40, 300], [3, 0, 20], 28, 4, 128, dtype, 16, True, path)
    assert float(out[:2].abs().max()) == 0.0 and float(out[5:45].abs().max()) == 0.0
    assert float(out[45:45 + 280].abs().max()) == 0.0


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [20000]), ([16], [5000]), ([1] * 40, list(range(1, 4001, 100))),
                                            ([600], [3500]), ([33, 64, 2], [4000, 100, 2500])])
def test_long_caches_are_shared_among_ctas(S, dtype, path, q_lens, kv_lens):
    paged_case(S, q_lens, kv_lens, 28, 4, 128, dtype, 64, True, path, seed=5)


@pytest.mark.parametrize("path", [1, 2])
def test_sharp_and_offset_distributions(S, path):
    # scores of +-60 (one key takes all), and values with a mean far above their spread
    paged_case(S, [40, 1], [700, 3000], 28, 4, 128, torch.bfloat16, 64, True, path, sd=20.0)
    paged_case(S, [40, 1], [700, 3000], 28, 4, 128, torch.bfloat16, 64, True, path, offset=50.0)


# --------------------------------------------------------------------------
# prompts
# --------------------------------------------------------------------------

def prompt_case(S, lens, Hq, Hkv, D, dtype, causal, path=0, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    N = n + extra
    qkv = randn(g, N, Hq + 2 * Hkv, D, dtype=dtype)
    qkv[n:] = float("nan")
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]      # views of one fused projection
    out = torch.full((N, Hq, D), 123.0, dtype=dtype, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(N, len(lens), max(lens), Hq, Hkv, D, max(lens),
                                                         dt_code(S, dtype)))
    scale = 1.5 / math.sqrt(D)
    S.sd_set_attention_path(path)
    S.sd_prompt_attention(q, k, v, cumulative(lens).cuda(), max(lens), out, scale, ws, causal=causal)
    torch.cuda.synchronize()
    used = S.sd_last_attention_path()[0]
    assert S.sd_fault_word() == 0
    at = 0
    for c in lens:
        if c:
            x = qkv[at:at + c]
            check(out[at:at + c], *ref_attend(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], scale, causal), dtype,
                  used == 2)
        at += c
    assert bool((out[at:] == 123.0).all())
    return out


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("lens", [[1], [17], [1, 0, 130, 1, 2], [300, 257]])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_attention(S, dtype, path, Hq, Hkv, D, lens, causal):
    prompt_case(S, lens, Hq, Hkv, D, dtype, causal, path, extra=2)


@pytest.mark.parametrize("lens,causal", [([2049], True), ([1500, 3, 700], False), ([127, 128, 129, 1, 640], True)])
def test_longer_prompts(S, lens, causal):
    prompt_case(S, lens, 28, 4, 128, torch.bfloat16, causal, 2, seed=2)
    prompt_case(S, lens, 8, 8, 64, torch.bfloat16, causal, 2, seed=3)


# --------------------------------------------------------------------------
# append, and a run of them together
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D,R,page", [(28, 4, 128, 128, 16), (4, 1, 64, 20, 5), (6, 6, 64, 32, 1), (5, 1, 128, 128, 64)])
def test_append(S, dtype, layout, Hq, Hkv, D, R, page):
    g = torch.Generator().manual_seed(page)
    q_lens, kv_lens = [3, 0, 1, 40], [3, 9, 100, 47]
    n = sum(q_lens)
    N = n + 2
    pool = Pool(g, kv_lens, page, Hkv, D, dtype, head_major=page == 64, fill=0.5)
    x = randn(g, N, Hq + 2 * Hkv, D, dtype=dtype)
    dev = x.cuda()
    turns, _ = S.sd_rotary_table(R, 1e4)
    kp, vp, table = pool.cuda()
    cache_pos = torch.cat([torch.arange(b - a, b) for a, b in zip(q_lens, kv_lens)] + [torch.zeros(2)]).to(torch.int32)
    cu, kv = cumulative(q_lens).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
    for pos in (None, cache_pos * 3 + 7):
        qo = torch.full((N, Hq, D), 9.0, dtype=dtype, device="cuda")
        S.sd_rotary_append_paged(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], qo,
                                 None if pos is None else pos.cuda(), turns.cuda(), cu, kv, table, kp, vp,
                                 layout=layout)
        at = cache_pos if pos is None else pos
        qw, qm = rope_ref(x[:n, :Hq], at[:n], R, 1e4, layout)
        kw, km = rope_ref(x[:n, Hq:Hq + Hkv], at[:n], R, 1e4, layout)
        check_rope(qo[:n], qw, qm, dtype)
        assert bool((qo[n:] == 9.0).all())
        t, written = 0, torch.zeros(kp.shape[:2], dtype=torch.bool)
        for b, c in enumerate(q_lens):
            pg, sl = pool.slots(b)
            pg, sl = pg[kv_lens[b] - c:], sl[kv_lens[b] - c:]
            written[pg, sl] = True
            check_rope(kp.cpu()[pg, sl], kw[t:t + c], km[t:t + c], dtype)
            assert torch.equal(vp.cpu()[pg, sl], x[t:t + c, Hq + Hkv:])
            t += c
        assert bool((kp.cpu()[~written] == 0.5).all()) and bool((vp.cpu()[~written] == 0.5).all())
    # without queries: the same pages
    k2, v2, _ = pool.cuda()
    S.sd_rotary_append_paged(None, dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], None, pos.cuda(), turns.cuda(), cu, kv,
                             table, k2, v2, layout=layout)
    assert torch.equal(k2, kp) and torch.equal(v2, vp)
    assert S.sd_fault_word() == 0


def test_a_prompt_then_blocks_over_the_paged_cache(S):
    """A conversation as it is served: two prompts enter the cache with their attention computed in
    one go, then in chunks, then blocks of 16 follow.  The chunked pass gives what the whole prompt
    gave, a chain of blocks what sd_verify_attention gives on a contiguous cache."""
    g = torch.Generator().manual_seed(8)
    Hq, Hkv, D, page, dtype = 28, 4, 128, 16, torch.bfloat16
    lens, T = [300, 77], 16
    pool = Pool(g, [n + T for n in lens], page, Hkv, D, dtype)
    kp, vp, table = pool.cuda()
    x = randn(g, sum(lens), Hq + 2 * Hkv, D, dtype=dtype).cuda()
    turns = S.sd_rotary_table(D, 1e6)[0].cuda()
    cu, kv = cumulative(lens).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.empty(sum(lens), Hq, D, dtype=dtype, device="cuda")
    S.sd_rotary_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q, None, turns, cu, kv, table, kp, vp)
    k = torch.empty(sum(lens), Hkv, D, dtype=dtype, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    S.sd_rotary(x[:, Hq:Hq + Hkv], k, pos, turns)
    scale = 1 / math.sqrt(D)
    ws = S.workspace(S.sd_paged_attention_workspace_size(sum(lens), 2, 300, Hq, Hkv, D, 316))
    whole, chunked = torch.zeros_like(q), torch.zeros_like(q)
    v = x[:, Hq + Hkv:].contiguous()
    S.sd_prompt_attention(q, k, v, cu, 300, whole, scale, ws)
    starts, done = cumulative(lens).tolist(), [0, 0]
    for step in ([100, 77], [1, 0], [199, 0]):
        rows = torch.cat([torch.arange(starts[b] + done[b], starts[b] + done[b] + c) for b, c in enumerate(step)]).cuda()
        done = [d + c for d, c in zip(done, step)]
        o = torch.empty(sum(step), Hq, D, dtype=dtype, device="cuda")
        S.sd_paged_attention(q[rows], kp, vp, table, cumulative(step).cuda(), torch.tensor(done, dtype=torch.int32).cuda(),
                             max(step), max(done), o, scale, ws)
        chunked[rows] = o
    qc, kc, vc = q.cpu(), k.cpu(), v.cpu()
    for got in (whole, chunked):
        for b in range(2):
            s = slice(starts[b], starts[b + 1])
            check(got[s], *ref_attend(qc[s], kc[s], vc[s], scale, True), dtype, True)
    # a block of 16 for each
    y = randn(g, 2 * T, Hq + 2 * Hkv, D, dtype=dtype).cuda()
    cub, kvb = cumulative([T, T]).cuda(), torch.tensor([n + T for n in lens], dtype=torch.int32).cuda()
    qb = torch.empty(2 * T, Hq, D, dtype=dtype, device="cuda")
    S.sd_rotary_append_paged(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], qb, None, turns, cub, kvb, table, kp, vp)
    ob = torch.empty_like(qb)
    S.sd_paged_attention(qb, kp, vp, table, cub, kvb, T, 316, ob, scale, ws)
    cache_k = torch.zeros(2, 316, Hkv, D, dtype=dtype, device="cuda")
    cache_v = torch.zeros_like(cache_k)
    for b in range(2):
        pg, sl = pool.slots(b)
        cache_k[b, :len(pg)], cache_v[b, :len(pg)] = kp[pg.cuda(), sl.cuda()], vp[pg.cuda(), sl.cuda()]
    want = torch.empty(2, T, Hq, D, device="cuda")
    wv = S.workspace(S.sd_verify_attention_workspace_size(2, T, Hq, Hkv, D, 301))
    S.sd_verify_attention(qb.view(2, T, Hq, D), cache_k, cache_v, torch.tensor([n + 1 for n in lens], dtype=torch.int32).cuda(),
                          301, want, scale, wv)
    for b in range(2):
        n = lens[b] + T
        r = ref_attend(qb.view(2, T, Hq, D)[b].cpu(), cache_k[b, :n].cpu(), cache_v[b, :n].cpu(), scale, True)
        check(ob.view(2, T, Hq, D)[b], *r, dtype, True)
        assert float((ob.view(2, T, Hq, D)[b].float() - want[b]).abs().max()) <= \
            float(((2.0 ** -7 + r[3]) * r[1] + 2.0 ** -8 * r[0].abs()).max()) + 2e-3
    assert S.sd_fault_word() == 0


# --------------------------------------------------------------------------
# guards, order, capture
# --------------------------------------------------------------------------

def small(S, dtype=torch.bfloat16, path=0, seed=1):
    return paged_case(S, [5, 16], [40, 900], 28, 4, 128, dtype, 16, True, path, seed=seed)


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
def test_bad_lengths_and_pages_set_the_fault_word(S, dtype, path):
    args, out = small(S, dtype, path)
    good = out.clone()
    call = lambda **kw: (S.sd_set_attention_path(path), S.sd_paged_attention(*[kw.get(str(i), a) for i, a in enumerate(args)]),
                         torch.cuda.synchronize(), S.sd_fault_word())[3]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    assert call() == 0
    assert call(**{"4": i32(0, 5, 1000)}) & BAD_LENGTH          # past N
    assert call(**{"4": i32(-3, 5, 21)}) & BAD_LENGTH
    assert call(**{"4": i32(0, 30, 21)}) & BAD_LENGTH           # decreasing (and past N)
    assert call(**{"5": i32(40, 2 ** 30)}) & BAD_LENGTH         # past max_kv and the table
    assert call(**{"5": i32(-1, 900)}) & BAD_LENGTH
    assert call(**{"6": 3}) & BAD_LENGTH                        # more new tokens than max_q
    table = args[3].clone()
    table[1, 2], table[1, 5] = -1, 1 << 20
    assert call(**{"3": table}) & BAD_PAGE
    # a call after all that is exact again
    out.fill_(0)
    assert call() == 0
    assert torch.equal(out[:21], good[:21])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_guards(S, dtype):
    g = torch.Generator().manual_seed(2)
    pool = Pool(g, [20, 20], 16, 2, 64, dtype, fill=0.25)
    kp, vp, table = pool.cuda()
    kv = randn(g, 8, 2, 64, dtype=dtype).cuda()
    turns = S.sd_rotary_table(64, 1e4)[0].cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    bad = table.clone()
    bad[1, 1] = 99
    run = lambda cu, n, t: (S.sd_rotary_append_paged(None, kv, kv, None, None, turns, cu, n, t, kp, vp),
                            torch.cuda.synchronize(), S.sd_fault_word())[2]
    assert run(i32(0, 4, 8), i32(2, 1000), table) == BAD_LENGTH      # negative positions, positions past the table
    assert run(i32(0, 0, 8), i32(0, 24), bad) == BAD_PAGE
    keep = torch.ones(kp.shape[:2], dtype=torch.bool)
    for b, p in ((0, 0), (0, 1)):       # the two tokens of the first call whose positions are >= 0
        keep[int(table[b, p // 16]), p % 16] = False
    assert bool((kp.cpu()[keep] == 0.25).all()) and bool((vp.cpu()[keep] == 0.25).all())


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
def test_wait_gives_up_then_recovers(S, dtype, path):
    args, out = paged_case(S, [16], [6000], 28, 4, 128, dtype, 64, True, path)
    good, ws = out.clone(), args[10]
    S.sd_set_attention_path(path)
    S.sd_set_wait_test(1, 1_000_000)
    S.sd_paged_attention(*args)
    torch.cuda.synchronize()
    S.sd_set_wait_test(0, 0)
    assert S.sd_fault_word() & WAIT_GAVE_UP
    assert int(ws[256:256 + 608].sum()) == 0
    out.fill_(0)
    S.sd_paged_attention(*args)
    torch.cuda.synchronize()
    assert S.sd_fault_word() == 0 and torch.equal(out[:16], good[:16])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_repeats_are_bit_identical_and_calls_can_be_captured(S, dtype):
    args, out = paged_case(S, [33, 1, 200], [4000, 3000, 900], 28, 4, 128, dtype, 64, True)
    first = out.clone()
    for _ in range(3):
        out.fill_(0)
        S.sd_paged_attention(*args)
        torch.cuda.synchronize()
        assert torch.equal(out[:234], first[:234])
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            S.sd_paged_attention(*args)
            S.sd_rotary(out, out, torch.zeros(out.shape[0], dtype=torch.int32, device="cuda"),
                        torch.zeros(64, dtype=torch.int64, device="cuda"))       # turned by nothing
    out.fill_(0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:234], first[:234])
    # a captured call reads the lengths of the moment it is replayed
    args[5].copy_(torch.tensor([400, 300, 900], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    S.sd_paged_attention(*args)
    torch.cuda.synchronize()
    assert torch.equal(out[:234], replayed[:234]) and not torch.equal(out[:33], first[:33])
    assert S.sd_fault_word() == 0


def test_two_streams_with_their_own_workspaces(S):
    a = paged_case(S, [16] * 4, [3000] * 4, 28, 4, 128, torch.bfloat16, 64, True, seed=1)
    b = paged_case(S, [300], [2500], 28, 4, 128, torch.bfloat16, 64, True, seed=2)
    want = [a[1].clone(), b[1].clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (args, _), st in zip((a, b), streams):
            S.sd_paged_attention(*args, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a[1], want[0]) and torch.equal(b[1], want[1])
    assert S.sd_fault_word() == 0


def test_workspace_too_small_and_reuse_across_shapes(S):
    args, out = small(S)
    with pytest.raises(S.SdError) as e:
        S.sd_paged_attention(*args[:10], S.workspace(256))
    assert e.value.status == S.SD_ERR_WORKSPACE
    big = S.workspace(S.sd_paged_attention_workspace_size(4096, 64, 4096, 28, 4, 128, 65536))
    good = out.clone()
    for _ in range(2):
        out.fill_(0)
        S.sd_paged_attention(*args[:10], big)
        torch.cuda.synchronize()
        assert torch.equal(out[:21], good[:21])


# --------------------------------------------------------------------------
# large pools, many sequences, shared pages
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 2)])
def test_pools_beyond_32_bit_offsets(S, dtype, path):
    """Pages whose first element lies past 2^31: a pool of 2^31 + 2^21 elements of which a few pages
    at both ends are used, through the append, the attention and a table that is a view."""
    Hq, Hkv, D, page = 8, 4, 128, 64
    per = page * Hkv * D
    n_pages = (1 << 31) // per + 64
    kp = torch.empty(n_pages, page, Hkv, D, dtype=dtype, device="cuda")
    vp = torch.empty_like(kp)
    g = torch.Generator().manual_seed(6)
    ids = torch.tensor([n_pages - 1, 0, n_pages - 2, 3], dtype=torch.int32)
    wide = torch.full((2, 9), -7, dtype=torch.int32)
    wide[0, 2:4], wide[1, 2:4] = ids[:2], ids[2:]
    table = wide.cuda()[:, 2:7]
    lens = [100, 70]
    x = randn(g, sum(lens), Hq + 2 * Hkv, D, dtype=dtype)
    dev, cu = x.cuda(), cumulative(lens).cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    turns = torch.zeros(D // 2, dtype=torch.int64, device="cuda")        # turned by nothing: the cache holds x
    q = torch.empty(sum(lens), Hq, D, dtype=dtype, device="cuda")
    S.sd_rotary_append_paged(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], q, None, turns, cu, kv, table, kp, vp)
    out = torch.empty_like(q)
    ws = S.workspace(S.sd_paged_attention_workspace_size(sum(lens), 2, 100, Hq, Hkv, D, 100, dt_code(S, dtype)))
    S.sd_set_attention_path(path)
    scale = 1 / math.sqrt(D)
    S.sd_paged_attention(q, kp, vp, table, cu, kv, 100, 100, out, scale, ws)
    torch.cuda.synchronize()
    used = S.sd_last_attention_path()[0]
    assert S.sd_fault_word() == 0
    at = 0
    for c in lens:
        r = x[at:at + c]
        check(out[at:at + c], *ref_attend(r[:, :Hq], r[:, Hq:Hq + Hkv], r[:, Hq + Hkv:], scale, True), dtype, used == 2)
        at += c
    del kp, vp
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,path", [(torch.float32, 0), (torch.bfloat16, 2)])
@pytest.mark.parametrize("B", [33, 300, 1500])
def test_many_sequences(S, dtype, path, B):
    q_lens = [(i * 7) % 4 for i in range(B)]
    kv_lens = [max(a, (i * 37) % 150) for i, a in enumerate(q_lens)]
    paged_case(S, q_lens, kv_lens, 4, 2, 64, dtype, 16, True, path, seed=B)


@pytest.mark.parametrize("path", [1, 2])
def test_sequences_that_share_pages(S, path):
    """Two sequences with one prefix (the same pages), and one that appears twice."""
    g = torch.Generator().manual_seed(9)
    Hq, Hkv, D, page, dtype = 28, 4, 128, 16, torch.bfloat16
    kp, vp = (randn(g, 12, page, Hkv, D, dtype=dtype) for _ in range(2))
    table = torch.tensor([[1, 5, 7, 2], [1, 5, 3, 0], [1, 5, 7, 2]], dtype=torch.int32)
    kv_lens, q_lens = [60, 40, 60], [2, 5, 2]
    q = randn(g, 9, Hq, D, dtype=dtype)
    q[7:] = q[:2]
    out = torch.empty(9, Hq, D, dtype=dtype, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(9, 3, 5, Hq, Hkv, D, 60))
    S.sd_set_attention_path(path)
    S.sd_paged_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cumulative(q_lens).cuda(),
                         torch.tensor(kv_lens, dtype=torch.int32).cuda(), 5, 60, out, 0.1, ws)
    at = 0
    for b, c in enumerate(q_lens):
        i = torch.arange(kv_lens[b])
        k, v = (t[table[b, i // page].long(), i % page] for t in (kp, vp))
        check(out[at:at + c], *ref_attend(q[at:at + c], k, v, 0.1, True), dtype, path == 2)
        at += c
    assert torch.equal(out[7:], out[:2])


def test_values_behind_what_a_unit_sees_may_be_anything(S):
    """Non-finite keys and values in the slots past kv_len, inside the last page and in the pages behind it."""
    g = torch.Generator().manual_seed(10)
    Hq, Hkv, D, page, dtype = 8, 2, 64, 32, torch.bfloat16
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        pool = Pool(g, [70, 33], page, Hkv, D, dtype, fill=bad)
        ks, vs = [], []
        for b, m in enumerate((70, 33)):
            ks.append(randn(g, m, Hkv, D, dtype=dtype))
            vs.append(randn(g, m, Hkv, D, dtype=dtype))
            pool.write(b, ks[b], vs[b])
        kp, vp, table = pool.cuda()
        q = randn(g, 40, Hq, D, dtype=dtype)
        ws = S.workspace(S.sd_paged_attention_workspace_size(40, 2, 39, Hq, Hkv, D, 70))
        for path in (1, 2):
            for causal in (True, False):
                out = torch.empty(40, Hq, D, dtype=dtype, device="cuda")
                S.sd_set_attention_path(path)
                S.sd_paged_attention(q.cuda(), kp, vp, table, cumulative([39, 1]).cuda(),
                                     torch.tensor([70, 33], dtype=torch.int32).cuda(), 39, 70, out, 0.125, ws, causal=causal)
                check(out[:39], *ref_attend(q[:39], ks[0], vs[0], 0.125, causal), dtype, path == 2)
                check(out[39:], *ref_attend(q[39:], ks[1], vs[1], 0.125, causal), dtype, path == 2)


def test_output_rows_on_16_byte_boundaries(S):
    g = torch.Generator().manual_seed(12)
    x = randn(g, 150, 12, 64, dtype=torch.bfloat16)
    dev = x.cuda()
    buf = torch.full((150 * 8 * 64 + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(150, 1, 150, 8, 2, 64, 150))
    for off in (0, 8, 16, 24):
        out = buf[off:off + 150 * 8 * 64].view(150, 8, 64)
        S.sd_prompt_attention(dev[:, :8], dev[:, 8:10], dev[:, 10:], cumulative([150]).cuda(), 150, out, 0.125, ws)
        check(out, *ref_attend(x[:, :8], x[:, 8:10], x[:, 10:], 0.125, True), torch.bfloat16, True)
    with pytest.raises(S.SdError) as e:
        S.sd_prompt_attention(dev[:, :8], dev[:, 8:10], dev[:, 10:], cumulative([150]).cuda(), 150,
                              buf[4:4 + 150 * 8 * 64].view(150, 8, 64), 0.125, ws)
    assert e.value.status == S.SD_ERR_INVALID_ARG


def test_nothing_is_written_outside_the_buffers(S):
    """Canary bytes around the output, the pools and the workspace of each call."""
    PAD = 4096

    def padded(shape, dtype, fill=0):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((PAD + n + (-n) % 256 + PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        t = buf[PAD:PAD + n].view(dtype).view(shape)
        t.fill_(fill)
        return t, (buf, n)

    g = torch.Generator().manual_seed(14)
    for dtype in (torch.bfloat16, torch.float32):
        Hq, Hkv, D, page = 12, 4, 128, 24
        q_lens, kv_lens = [3, 40, 0, 150], [3, 77, 5, 400]
        n = sum(q_lens)
        marks = []
        pages = [padded((24, page, Hkv, D), dtype, 0.5) for _ in range(2)]
        q_out, out = padded((n, Hq, D), dtype), padded((n, Hq, D), dtype)
        size = S.sd_paged_attention_workspace_size(n, 4, 150, Hq, Hkv, D, 400, dt_code(S, dtype))
        ws = padded((size,), torch.uint8)
        marks += [m for _, m in (*pages, q_out, out, ws)]
        table = torch.randperm(24, generator=g).to(torch.int32)
        rows, at = torch.zeros(4, 17, dtype=torch.int32), 0
        for b, m in enumerate(kv_lens):
            c = -(-m // page)
            rows[b, :c] = table[at:at + c]
            at += c
        x = randn(g, n, Hq + 2 * Hkv, D, dtype=dtype).cuda()
        turns = S.sd_rotary_table(64, 1e4)[0].cuda()
        cu, kv = cumulative(q_lens).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
        S.sd_rotary_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q_out[0], None, turns, cu, kv,
                                 rows.cuda(), pages[0][0], pages[1][0])
        pool = pages[0][0].clone(), pages[1][0].clone()
        for path in (1, 2) if dtype == torch.bfloat16 else (1,):
            S.sd_set_attention_path(path)
            S.sd_paged_attention(q_out[0], pages[0][0], pages[1][0], rows.cuda(), cu, kv, 150, 400, out[0], 0.1, ws[0])
            S.sd_prompt_attention(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu, 150, out[0], 0.1, ws[0])
        S.sd_rotary(out[0], out[0], torch.arange(n, dtype=torch.int32, device="cuda"), turns, layout="interleaved")
        torch.cuda.synchronize()
        assert torch.equal(pool[0], pages[0][0]) and torch.equal(pool[1], pages[1][0])
        for buf, nb in marks:
            assert bool((buf[:PAD] == 0xA5).all()) and bool((buf[PAD + nb:] == 0xA5).all())
    assert S.sd_fault_word() == 0
