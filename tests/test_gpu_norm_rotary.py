"""Norms of queries and keys with positions of several axes, and their write into paged caches as they are or in 8
bits, against plain 64-bit forms (bounds in _quant)."""
import pytest
import torch

from _quant import check_codes, check_rows, norm_turn, pair_axes, quantise

pytestmark = pytest.mark.gpu

BAD_LENGTH, BAD_PAGE = 1 << 7, 1 << 8


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    return sd_verify


def freqs(R, theta=1e4):
    return theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)


def rand(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


CASES = [  # N, Hq, Hk, D, R, axes, order
    (1, 1, 1, 64, 64, None, "blocks"), (5, 28, 4, 128, 128, (16, 24, 24), "blocks"), (33, 3, 1, 128, 32, (6, 5, 5), "stripes"),
    (7, 5, 2, 64, 20, (4, 6), "blocks"), (3, 2, 1, 30, 6, (1, 1, 1), "stripes"), (40, 16, 16, 64, 64, (8, 8, 8, 8), "stripes"),
    (9, 6, 2, 256, 256, (64, 64), "blocks"), (4, 2, 1, 1024, 1024, (500, 12), "stripes"), (11, 3, 3, 512, 128, (64,), "blocks"),
    (130, 4, 4, 96, 96, (16, 16, 16), "blocks"), (2, 9, 0, 128, 64, (32,), "blocks"), (3, 2, 2, 2, 2, None, "blocks")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hk,D,R,axes,order", CASES)
def test_norm_rotary(S, dtype, layout, N, Hq, Hk, D, R, axes, order):
    g = torch.Generator().manual_seed(N + R)
    A = len(axes) if axes else 1
    x = rand(g, N, Hq + Hk, D, dtype=dtype) * torch.logspace(-3, 3, Hq + Hk).to(dtype)[:, None]
    pos = torch.randint(-(1 << 20), 1 << 20, (A, N), generator=g, dtype=torch.int32)
    pos[:, 0] = 0
    wq, wk = rand(g, D, dtype=dtype) + 1, rand(g, D, dtype=dtype) * 3
    turns, _ = S.sd_rotary_table(R, 1e4)
    axis = pair_axes(axes, order) if axes else [0] * (R // 2)
    dev = x.cuda()
    kw = dict(axes=axes, axes_order=order, layout=layout, eps=1e-5)
    for weights in ((wq, wk), (None, wk), (None, None)):
        cw = dict(q_weight=None if weights[0] is None else weights[0].cuda(),
                  k_weight=None if weights[1] is None else weights[1].cuda(), magnitude=1.25, **kw)
        qo = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
        ko = torch.full((N, Hk, D), 7.0, dtype=dtype, device="cuda") if Hk else None
        S.sd_norm_rotary(dev[:, :Hq], qo, dev[:, Hq:] if Hk else None, ko, pos.cuda(), turns.cuda(), **cw)
        check_rows(qo, *norm_turn(x[:, :Hq], weights[0], 1e-5, pos, freqs(R), axis, layout, 1.25), dtype)
        if Hk:
            check_rows(ko, *norm_turn(x[:, Hq:], weights[1], 1e-5, pos, freqs(R), axis, layout, 1.25), dtype)
        # in place over the fused rows: the same bits
        z = x.cuda()
        S.sd_norm_rotary(z[:, :Hq], z[:, :Hq], z[:, Hq:] if Hk else None, z[:, Hq:] if Hk else None, pos.cuda(),
                         turns.cuda(), **cw)
        assert torch.equal(z[:, :Hq], qo) and (not Hk or torch.equal(z[:, Hq:], ko))
        # rows off 16 bytes, head-major outputs: within the same bounds
        wide = torch.zeros(N, Hq, D + 1, dtype=dtype, device="cuda")
        wide[:, :, 1:] = dev[:, :Hq]
        o = torch.empty(Hq, N, D, dtype=dtype, device="cuda").transpose(0, 1)
        S.sd_norm_rotary(wide[:, :, 1:], o, None, None, pos.cuda(), turns.cuda(), **cw)
        check_rows(o, *norm_turn(x[:, :Hq], weights[0], 1e-5, pos, freqs(R), axis, layout, 1.25), dtype)
    assert S.sd_fault_word() == 0


def test_one_axis_without_norm_is_sd_rotary(S):
    g = torch.Generator().manual_seed(1)
    for D, R, dtype in ((128, 128, torch.bfloat16), (64, 32, torch.float32)):
        x = rand(g, 50, 5, D, dtype=dtype).cuda()
        pos = torch.randint(0, 1 << 20, (50,), generator=g, dtype=torch.int32).cuda()
        turns = S.sd_rotary_table(R, 1e6)[0].cuda()
        a, b = torch.empty_like(x), torch.empty_like(x)
        S.sd_rotary(x, a, pos, turns)
        S.sd_norm_rotary(x, b, None, None, pos, turns)
        assert torch.equal(a, b)
        # equal positions on every axis: as one axis
        S.sd_norm_rotary(x, b, None, None, pos[None].expand(2, -1).contiguous(), turns, axes=(R // 4, R // 4))
        assert torch.equal(a, b)


def test_own_frequencies_of_each_axis(S):
    g = torch.Generator().manual_seed(2)
    x = rand(g, 20, 4, 64)
    pos = torch.randint(0, 100, (2, 20), generator=g, dtype=torch.int32)
    t = S.sd_rotary_table(32, 1e4)[0]
    y = torch.empty(20, 4, 64, device="cuda")
    S.sd_norm_rotary(x.cuda(), y, None, None, pos.cuda(), torch.cat([t, t]).cuda(), axes=(16, 16))
    check_rows(y, *norm_turn(x, None, 0, pos, torch.cat([freqs(32)] * 2), pair_axes((16, 16), "blocks"), "half"), torch.float32)


def test_rows_of_zeros_and_of_extremes(S):
    """eps keeps a row of zeros at zero; rows up to fp32's square root of its range norm; NaN stays in its row."""
    D = 128
    w = torch.ones(D)
    x = torch.zeros(6, 1, D)
    x[1] = 1e18
    x[2] = 1e-18
    x[3, 0, 5] = float("nan")
    x[4] = torch.linspace(-1, 1, D)
    pos = torch.zeros(6, dtype=torch.int32)
    y = torch.empty(6, 1, D, device="cuda")
    turns = S.sd_rotary_table(D, 1e4)[0].cuda()
    S.sd_norm_rotary(x.cuda(), y, None, None, pos.cuda(), turns, q_weight=w.cuda(), eps=1e-6)
    y = y.cpu()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4, 5]]).all()
    assert float(y[0].abs().max()) == 0.0
    assert (y[1] - 1).abs().max() <= (D + 8) * 2.0 ** -24
    want, off = norm_turn(x[4:5], w, 1e-6, pos[None, 4:5], freqs(D), [0] * 64, "half")
    check_rows(y[4:5], want, off, torch.float32)


# --------------------------------------------------------------------------
# into a cache
# --------------------------------------------------------------------------

def place(g, kv_lens, page):
    need = [-(-n // page) for n in kv_lens]
    n = sum(need) + 2
    ids = torch.randperm(n, generator=g).to(torch.int32)
    table = torch.full((len(kv_lens), max(need + [1]) + 1), -5, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        at += c
    return n, table


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,R,page,axes,order", [
    (28, 4, 128, 128, 16, (16, 24, 24), "blocks"), (4, 1, 64, 20, 5, (4, 6), "stripes"), (6, 6, 64, 32, 1, None, "blocks"),
    (5, 1, 128, 128, 64, (22, 21, 21), "stripes"), (3, 2, 30, 6, 24, (1, 2), "blocks"), (2, 3, 256, 256, 8, None, "blocks")])
def test_append(S, dtype, layout, quantised, Hq, Hkv, D, R, page, axes, order):
    g = torch.Generator().manual_seed(page + R)
    q_lens, kv_lens = [3, 0, 1, 40], [3, 9, 100, 47]
    n = sum(q_lens)
    N = n + 2
    pages, table = place(g, kv_lens, page)
    x = rand(g, N, Hq + 2 * Hkv, D, dtype=dtype)
    dev = x.cuda()
    wq, wk = rand(g, D, dtype=dtype) + 1, rand(g, D, dtype=dtype) + 1
    A = len(axes) if axes else 1
    axis = pair_axes(axes, order) if axes else [0] * (R // 2)
    turns = S.sd_rotary_table(R, 1e4)[0].cuda()
    cu = torch.tensor([0] + torch.tensor(q_lens).cumsum(0).tolist(), dtype=torch.int32).cuda()
    kv = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    cached = torch.cat([torch.arange(b - a, b) for a, b in zip(q_lens, kv_lens)] + [torch.zeros(2)]).to(torch.int32)
    given = torch.randint(0, 1 << 16, (A, N), generator=g, dtype=torch.int32)
    for pos in (None, given):
        ct = torch.float8_e4m3fn if quantised else dtype
        kp, vp = (torch.full((pages, Hkv, page, D), 0.5).to(ct).cuda().transpose(1, 2) for _ in range(2))   # head-major
        sc = [torch.full((pages, Hkv, page), -3.0, device="cuda") for _ in range(2)] if quantised else [None, None]
        qo = torch.full((N, Hq, D), 9.0, dtype=dtype, device="cuda")
        args = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-6, axes=axes, axes_order=order, layout=layout)
        S.sd_norm_rotary_append_paged(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], qo,
                                      None if pos is None else pos.cuda(), turns, cu, kv, table.cuda(), kp, vp, *sc, **args)
        at = cached[None].expand(A, -1) if pos is None else pos
        check_rows(qo[:n], *norm_turn(x[:n, :Hq], wq, 1e-6, at[:, :n], freqs(R), axis, layout), dtype)
        assert bool((qo[n:] == 9.0).all())
        kw, ko = norm_turn(x[:n, Hq:Hq + Hkv], wk, 1e-6, at[:, :n], freqs(R), axis, layout)
        t, written = 0, torch.zeros(pages, page, dtype=torch.bool)
        for b, c in enumerate(q_lens):
            i = torch.arange(kv_lens[b] - c, kv_lens[b])
            pg, sl = table[b, i // page].long(), i % page
            written[pg, sl] = True
            rows = slice(t, t + c)
            if quantised and c:
                codes = lambda z: z.cpu().view(torch.uint8)[pg, sl].view(torch.float8_e4m3fn)
                check_codes(codes(kp), sc[0].cpu()[pg, :, sl], kw[rows], ko[rows])
                vc, vs = quantise(x[rows, Hq + Hkv:].float())
                assert torch.equal(codes(vp).view(torch.uint8), vc.view(torch.uint8))
                assert torch.equal(sc[1].cpu()[pg, :, sl], vs)
            elif c:
                check_rows(kp.cpu()[pg, sl], kw[rows], ko[rows], dtype)
                assert torch.equal(vp.cpu()[pg, sl], x[rows, Hq + Hkv:])
            t += c
        for z in (kp, vp):
            assert bool((z.cpu().float()[~written] == 0.5).all())
        if quantised:
            assert all(bool((s.cpu().transpose(1, 2)[~written] == -3.0).all()) for s in sc)
        # without queries: the same cache
        k2, v2 = (torch.full((pages, Hkv, page, D), 0.5).to(ct).cuda().transpose(1, 2) for _ in range(2))
        s2 = [torch.full((pages, Hkv, page), -3.0, device="cuda") for _ in range(2)] if quantised else [None, None]
        S.sd_norm_rotary_append_paged(None, dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], None,
                                      None if pos is None else pos.cuda(), turns, cu, kv, table.cuda(), k2, v2, *s2, **args)
        assert torch.equal(k2.float(), kp.float()) and torch.equal(v2.float(), vp.float())
        assert not quantised or (torch.equal(s2[0], sc[0]) and torch.equal(s2[1], sc[1]))
    assert S.sd_fault_word() == 0


def test_values_are_copied_bit_for_bit(S):
    """Into a cache of their own type every bit pattern goes as it is, NaNs and their payloads among them."""
    for dtype, it, D in ((torch.bfloat16, torch.int16, 128), (torch.bfloat16, torch.int16, 30), (torch.float32, torch.int32, 64)):
        g = torch.Generator().manual_seed(D)
        info = torch.iinfo(it)
        bits = torch.randint(info.min, info.max, (64, 2, D), generator=g, dtype=it)
        v = bits.view(dtype).cuda()
        k = torch.zeros_like(v)
        kp, vp = (torch.zeros(5, 16, 2, D, dtype=dtype, device="cuda") for _ in range(2))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        S.sd_norm_rotary_append_paged(None, k, v, None, None, S.sd_rotary_table(2, 1e4)[0].cuda(), i32([0, 64]), i32([64]),
                                      i32([[3, 1, 0, 4]]), kp, vp)
        assert torch.equal(vp[[3, 1, 0, 4]].view(it).view(64, 2, D).cpu(), bits)
    assert S.sd_fault_word() == 0


def test_append_of_rows_of_zeros_and_tiny_ones(S):
    """A row of zeros gets codes of zero and the smallest scale; one of 2^-90 keeps its relative precision."""
    D = 64
    x = torch.zeros(3, 1, D)
    x[1, 0] = torch.linspace(-1, 1, D) * 2.0 ** -90
    x[2, 0, 3] = 5.0
    kp, vp = (torch.ones(1, 4, 1, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    sc = [torch.zeros(1, 1, 4, device="cuda") for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    S.sd_norm_rotary_append_paged(None, x.cuda(), x.cuda(), None, i32(0, 0, 0), S.sd_rotary_table(D, 1e4)[0].cuda(), i32(0, 3),
                                  i32(3), i32(0)[None], kp, vp, *sc)
    want, ws = quantise(x)
    for codes, s in ((kp, sc[0]), (vp, sc[1])):
        assert torch.equal(codes[0, :3].float().cpu(), want.float())
        assert torch.equal(s[0, 0, :3].cpu(), ws[:, 0]) and float(s[0, 0, 3]) == 0.0
        assert bool((codes[0, 3].float() == 1).all())
    assert S.sd_fault_word() == 0


@pytest.mark.parametrize("D,page", [(128, 16), (30, 5)])
def test_bad_lengths_and_pages_write_nothing_else(S, D, page):
    g = torch.Generator().manual_seed(3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    x = rand(g, 4, 3, D).cuda()
    turns = S.sd_rotary_table(2, 1e4)[0].cuda()
    for kv, table, bit in (([2, 1], [[0], [7]], BAD_PAGE), ([2, 1], [[-1], [1]], BAD_PAGE), ([page + 1, 2], [[0], [1]], BAD_LENGTH),
                           ([1, 2], [[0], [1]], BAD_LENGTH), ([2, -4], [[0], [1]], BAD_LENGTH)):
        pool = torch.full((4, page, 1, D), 0.5, device="cuda").to(torch.float8_e4m3fn)
        kp, vp = pool[1:3], pool.clone()[1:3]
        sc = [torch.full((4, 1, page), 2.0, device="cuda") for _ in range(2)]
        S.sd_norm_rotary_append_paged(x[:, :1], x[:, 1:2], x[:, 2:], torch.empty(4, 1, D, device="cuda"), None, turns,
                                      i32([0, 2, 4]), i32(kv), i32(table), kp, vp, sc[0][:2], sc[1][:2])
        torch.cuda.synchronize()
        assert S.sd_fault_word() & bit
        assert bool((pool[0].float() == 0.5).all()) and bool((pool[3].float() == 0.5).all())
        assert all(bool((s[2:] == 2.0).all()) for s in sc)
