"""Norms, positions and cache writes of calls long enough that a CTA takes several tokens (from about 1,800 on; eight
from about 7,300): against the 64-bit forms and, bit for bit, against the same rows in short calls."""
import pytest
import torch

from _quant import check_codes, check_rows, norm_turn, pair_axes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    return sd_verify


def freqs(R, theta=1e4):
    return theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)


# N, Hq, Hk, D, R, axes: heads fewer and more than the rows a CTA holds at a time, one head, none of the keys
ROWS = [(1831, 3, 1, 128, 128, (16, 24, 24)), (2743, 1, 1, 64, 32, (6, 5, 5)), (4001, 28, 4, 128, 128, None),
        (7303, 5, 0, 64, 64, (16, 16)), (9001, 40, 2, 64, 64, None), (8000, 1, 2, 512, 512, (128, 128)), (7297, 2, 1, 32, 32, None)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hk,D,R,axes", ROWS)
def test_norm_rotary(S, dtype, layout, N, Hq, Hk, D, R, axes):
    g = torch.Generator().manual_seed(N)
    A = len(axes) if axes else 1
    x = torch.randn(N, Hq + Hk, D, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 16, (A, N), generator=g, dtype=torch.int32)
    wq, wk = (torch.randn(D, generator=g) + 1).to(dtype), (torch.randn(D, generator=g) + 1).to(dtype)
    turns = S.sd_rotary_table(R, 1e4)[0].cuda()
    axis = pair_axes(axes, "blocks") if axes else [0] * (R // 2)
    kw = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), axes=axes, layout=layout, eps=1e-6)
    dev, p = x.cuda(), pos.cuda()

    def call(src, dst, a, b):
        keys = (src[a:b, Hq:], dst[a:b, Hq:]) if Hk else (None, None)
        S.sd_norm_rotary(src[a:b, :Hq], dst[a:b, :Hq], *keys, p[:, a:b].contiguous(), turns, **kw)
    y, short, place = torch.empty_like(dev), torch.empty_like(dev), dev.clone()
    call(dev, y, 0, N)
    call(place, place, 0, N)
    for a in range(0, N, 1000):
        call(dev, short, a, min(N, a + 1000))
    assert torch.equal(y, place) and torch.equal(y, short)
    at = torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 40, N)])
    check_rows(y[at.cuda(), :Hq], *norm_turn(x[at, :Hq], wq, 1e-6, pos[:, at], freqs(R), axis, layout), dtype)
    if Hk:
        check_rows(y[at.cuda(), Hq:], *norm_turn(x[at, Hq:], wk, 1e-6, pos[:, at], freqs(R), axis, layout), dtype)
    assert S.sd_fault_word() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,page,q_lens", [
    (28, 4, 128, 16, [5000, 1, 0, 3, 2, 0, 1, 2500]), (2, 1, 64, 5, [3] * 900 + [0] * 20 + [1] * 40), (0, 2, 128, 64, [4000, 4001]),
    (1, 1, 64, 16, [1] * 8000), (6, 3, 256, 8, [1900])])
def test_append(S, dtype, quantised, given, Hq, Hkv, D, page, q_lens):
    """Sequences that begin and end within a CTA's tokens, tokens behind the last one, queries in place or none."""
    g = torch.Generator().manual_seed(page)
    n, pad = sum(q_lens), 5
    N, B = n + pad, len(q_lens)
    kv_lens = [c + int(e) for c, e in zip(q_lens, torch.randint(0, 2 * page, (B,), generator=g))]
    cols = max(-(-m // page) for m in kv_lens)
    need = [-(-m // page) for m in kv_lens]
    pages = sum(need)
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, cols), -7, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        at += c
    x = torch.randn(N, Hq + 2 * Hkv, D, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 16, (3, N), generator=g, dtype=torch.int32)
    axes = (D // 2 - 2 * (D // 6), D // 6, D // 6)
    axis = pair_axes(axes, "blocks")
    wq, wk = (torch.randn(D, generator=g) + 1).to(dtype), (torch.randn(D, generator=g) + 1).to(dtype)
    turns = S.sd_rotary_table(D, 1e4)[0].cuda()
    dev, tab = x.cuda(), table.cuda()
    ct = torch.float8_e4m3fn if quantised else dtype

    def cache():
        return [torch.full((pages, page, Hkv, D), 0.5, device="cuda").to(ct) for _ in range(2)], \
            [torch.full((pages, Hkv, page), -3.0, device="cuda") for _ in range(2)] if quantised else [None, None]

    def call(c, q, q_out, a, b, lens, kv, rows):
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32).cuda()
        S.sd_norm_rotary_append_paged(q, dev[a:b, Hq:Hq + Hkv], dev[a:b, Hq + Hkv:], q_out, pos[:, a:b].contiguous().cuda() if given else None,
                                      turns, cu, torch.tensor(kv, dtype=torch.int32).cuda(), tab[rows], *c[0], *c[1], q_weight=wq.cuda(),
                                      k_weight=wk.cuda(), axes=axes)
    long, short = cache(), cache()
    qo = torch.full((N, Hq, D), 9.0, dtype=dtype, device="cuda") if Hq else None
    call(long, dev[:, :Hq] if Hq else None, qo, 0, N, q_lens, kv_lens, slice(None))
    if Hq:                                        # in place
        z = dev[:, :Hq].contiguous()
        again = cache()
        call(again, z, z, 0, N, q_lens, kv_lens, slice(None))
        assert torch.equal(z[:n], qo[:n]) and torch.equal(z[n:], dev[n:, :Hq]) and bool((qo[n:] == 9.0).all())
    # in calls of at most 1,000 tokens
    qs = torch.empty(n, Hq, D, dtype=dtype, device="cuda") if Hq else None
    b = done = at = 0
    while b < B:
        a, lens, kv, first = at, [], [], b
        while b < B and at - a < 1000:
            take = min(q_lens[b] - done, 1000 - (at - a))
            lens.append(take)
            kv.append(kv_lens[b] - q_lens[b] + done + take)
            at, done = at + take, done + take
            if done < q_lens[b]:
                break
            b, done = b + 1, 0
        call(short, dev[a:at, :Hq] if Hq else None, qs[a:at] if Hq else None, a, at, lens, kv, slice(first, first + len(lens)))
    bits = lambda t: t.view(torch.uint8)
    for s, t in zip(long[0] + long[1], short[0] + short[1]):
        assert s is None or torch.equal(bits(s), bits(t))
    assert not Hq or torch.equal(qo[:n], qs)
    # and the formula, of some sequences' rows
    start = torch.tensor([0] + q_lens).cumsum(0)
    for b in sorted({0, B // 2, B - 1}):
        c = min(q_lens[b], 50)
        if not c:
            continue
        rows = torch.arange(int(start[b + 1]) - c, int(start[b + 1]))
        i = torch.arange(kv_lens[b] - c, kv_lens[b])
        pg, sl = table[b, i // page].long(), i % page
        p = pos[:, rows] if given else i[None].expand(3, -1)
        want, off = norm_turn(x[rows, Hq:Hq + Hkv], wk, 1e-6, p, freqs(D), axis, "half")
        if quantised:
            check_codes(bits(long[0][0]).cpu()[pg, sl].view(torch.float8_e4m3fn), long[1][0].cpu()[pg, :, sl], want, off)
        else:
            check_rows(long[0][0].cpu()[pg, sl], want, off, dtype)
            assert torch.equal(long[0][1].cpu()[pg, sl], x[rows, Hq + Hkv:])
        if Hq:
            check_rows(qo[rows.cuda()], *norm_turn(x[rows, :Hq], wq, 1e-6, p, freqs(D), axis, "half"), dtype)
    assert S.sd_fault_word() == 0
