"""Attention over a paged cache in 8 bits, trees over either cache, the move of an accepted path, and a run of them,
against plain 64-bit forms (bounds in _quant)."""
import math

import numpy as np
import pytest
import torch

import oracle
from _quant import attend, check_attention, check_rows, norm_turn, pair_axes, quantise, signed, tree_masks

pytestmark = pytest.mark.gpu

BAD_COMMIT, BAD_LENGTH, BAD_PAGE, WAIT_GAVE_UP = 1 << 6, 1 << 7, 1 << 8, 1 << 3


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


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def cumulative(lens):
    return i32([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist())


class Pool:
    """Pages handed out in random order; spare pages, slots past the end and their scales hold nonsense."""

    def __init__(self, g, kv_lens, page, Hkv, D, dtype, quantised, head_major=False, sd=1.0, spread=0.0):
        need = [-(-n // page) for n in kv_lens]
        n = sum(need) + 2
        self.page, self.kv_lens, self.head_major = page, kv_lens, head_major
        ids = torch.randperm(n, generator=g).to(torch.int32)
        self.table = torch.full((len(kv_lens), max(need + [1]) + 1), -5, dtype=torch.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = ids[at:at + c]
            at += c
        self.t = {}
        self.values = {"k": [], "v": []}
        self.codes = []
        for x in ("k", "v"):
            pages = torch.full((n, page, Hkv, D), float("nan")).to(torch.float8_e4m3fn if quantised else dtype)
            scale = torch.full((n, Hkv, page), float("nan"))
            for b, m in enumerate(kv_lens):
                rows = torch.randn(m, Hkv, D, generator=g) * sd
                if spread:
                    rows *= torch.exp(torch.randn(m, Hkv, 1, generator=g) * spread)
                rows = rows.to(dtype)
                p = torch.arange(m)
                pg, sl = self.table[b, p // page].long(), p % page
                if quantised:
                    c, s = quantise(rows.float())
                    pages.view(torch.uint8)[pg, sl] = c.view(torch.uint8)
                    scale[pg, :, sl] = s
                    rows = c.float().double() * s.double()[..., None]
                    if x == "v":
                        self.codes.append((c.float().abs(), s.amax(0).double() if m else torch.zeros(Hkv)))
                else:
                    pages[pg, sl] = rows
                self.values[x].append(rows)
            if head_major:
                pages = pages.transpose(1, 2).contiguous().transpose(1, 2)
            self.t[x + "_pages"], self.t[x + "_scale"] = pages, scale if quantised else None

    def cuda(self):
        def move(t):
            if t is None:
                return None
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.head_major and t.dim() == 4 else t.cuda()
        return [move(self.t[x]) for x in ("k_pages", "v_pages", "k_scale", "v_scale")], self.table.cuda()


def case(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, *, tree=False, causal=True, quantised=True, path=0, head_major=False,
         seed=0, extra=3, sd=2.0, strided=False, spread=0.5, masks=None):
    g = torch.Generator().manual_seed(seed)
    n = sum(q_lens)
    N = n + extra
    q = (torch.randn(N, Hq, D, generator=g) * sd).to(dtype)
    q[n:] = float("nan")
    pool = Pool(g, kv_lens, page, Hkv, D, dtype, quantised, head_major, spread=spread)
    (kp, vp, ks, vs), table = pool.cuda()
    out = torch.full((N, Hq, D), 123.0, dtype=dtype, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(N, len(q_lens), max(q_lens), Hq, Hkv, D, max(kv_lens),
                                                         S.SD_BF16 if dtype == torch.bfloat16 else S.SD_FP32))
    qd = q.cuda()
    if strided:
        wide = torch.full((N, Hq + 2, D + 8), float("nan"), dtype=dtype, device="cuda")
        wide[:, 1:Hq + 1, :D] = qd
        qd = wide[:, 1:Hq + 1, :D]
    scale = 1 / math.sqrt(D)
    cu, kv = cumulative(q_lens).cuda(), i32(kv_lens).cuda()
    S.sd_set_attention_path(path)
    if tree:
        if masks is None:
            masks = [w for a in q_lens for w in tree_masks(g, a)[0]]
        words = signed(masks + [0x5555] * extra).cuda()

        def call(o=out, w=ws):
            S.sd_paged_tree_attention(qd, kp, vp, table, words, cu, kv, max(q_lens), max(kv_lens), o, scale, w, ks, vs)
    else:
        def call(o=out, w=ws):
            S.sd_paged_attention_e4m3(qd, kp, vp, ks, vs, table, cu, kv, max(q_lens), max(kv_lens), o, scale, w, causal=causal)
    call()
    torch.cuda.synchronize()
    used = S.sd_last_attention_path()[0]
    assert S.sd_fault_word() == 0
    assert int(ws[256:256 + 4096].sum()) == 0, "counters not returned to zero"
    terms = 0 if used == 1 else "e4m3" if quantised else "bf16"
    at = 0
    for b, (a, m) in enumerate(zip(q_lens, kv_lens)):
        if a:
            j = torch.arange(m)[None]
            if tree:
                w = masks[at:at + a]
                seen = torch.tensor([[t < m - a or bool(w[i] >> (t - (m - a)) & 1) for t in range(m)] for i in range(a)]).view(a, m)
            else:
                seen = j <= torch.arange(a)[:, None] + (m - a) if causal else (j >= 0).expand(a, m)
            want = attend(q[at:at + a], pool.values["k"][b], pool.values["v"][b], scale, seen,
                          pool.codes[b] if terms == "e4m3" else None)
            check_attention(out[at:at + a], want, dtype, terms)
        at += a
    assert bool((out[at:] == 123.0).all()), "rows behind the last sequence were written"
    return call, out, ws


PATHS = [(torch.float32, 0), (torch.bfloat16, 1), (torch.bfloat16, 0)]
HEADS = [(28, 4, 128), (4, 1, 64), (8, 8, 64), (16, 2, 128), (64, 1, 128), (3, 1, 128)]


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("q_lens,kv_lens,page", [
    ([1], [1], 16), ([1], [129], 8), ([0, 1, 2, 0], [5, 1, 200, 0], 16), ([16, 16, 16], [16, 700, 1500], 64),
    ([130, 1, 300, 37], [130, 129, 513, 1000], 24)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(S, dtype, path, Hq, Hkv, D, q_lens, kv_lens, page, causal):
    case(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, causal=causal, path=path)


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("page", [1, 5, 8, 12, 16, 40, 48, 64, 128, 256, 384])
def test_pages_and_orders(S, dtype, path, page):
    case(S, [3, 40], [257, 511], 28, 4, 128, dtype, page, path=path, seed=page)
    case(S, [2, 9], [300, 77], 8, 2, 64, dtype, page, path=path, head_major=True, strided=True, seed=page + 1)
    case(S, [3, 40], [257, 511], 28, 4, 128, dtype, page, path=path, seed=page, tree=True)
    case(S, [3, 40], [257, 511], 8, 2, 64, dtype, page, path=path, seed=page, tree=True, quantised=False, strided=True)


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("q_lens,kv_lens,page", [
    ([1], [1], 16), ([64], [64], 8), ([0, 60, 2, 64], [5, 200, 300, 190], 16), ([60], [1500], 64), ([7, 33, 64], [135, 160, 127 + 64], 24)])
def test_trees(S, dtype, path, quantised, Hq, Hkv, D, q_lens, kv_lens, page):
    case(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, tree=True, path=path, quantised=quantised)


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("m", [64, 65, 127, 128, 129, 190, 191, 192, 193, 300])
def test_trees_across_tiles(S, dtype, path, quantised, m):
    """64 nodes with arbitrary masks, descendants among them, and bits past the tree in a smaller one."""
    g = torch.Generator().manual_seed(m)
    words = [int(x) for x in torch.randint(-(1 << 62), 1 << 62, (64 + 20,), generator=g)]
    words[:2] = [-1, 1 << 63]
    words = [w & (1 << 64) - 1 for w in words]
    words[64] |= 1 << 5
    for i in range(65, 84):
        words[i] |= 1 << 63 | 1           # past a tree of 20 nodes
    case(S, [64, 20], [m, 70], 28, 4, 128, dtype, 16 if m % 2 else 64, tree=True, path=path, quantised=quantised, masks=words)


@pytest.mark.parametrize("dtype,path", PATHS)
def test_rows_that_see_nothing_give_zeros(S, dtype, path):
    call, out, _ = case(S, [5, 40, 300], [3, 0, 20], 28, 4, 128, dtype, 16, path=path)
    assert float(out[:2].abs().max()) == 0.0 and float(out[5:45 + 280].abs().max()) == 0.0
    for quantised in (True, False):
        call, out, _ = case(S, [3, 2], [3, 50], 28, 4, 128, dtype, 16, path=path, tree=True, quantised=quantised, masks=[1, 0, 5, 1, 0])
        assert float(out[1].abs().max()) == 0.0


@pytest.mark.parametrize("dtype,path", PATHS)
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [20000]), ([16], [5000]), ([1] * 40, list(range(1, 4001, 100))),
                                            ([600], [3500]), ([33, 64, 2], [4000, 100, 2500])])
def test_long_caches_are_shared_among_ctas(S, dtype, path, q_lens, kv_lens):
    case(S, q_lens, kv_lens, 28, 4, 128, dtype, 64, path=path, seed=5)
    if max(q_lens) <= 64:
        for quantised in (True, False):
            case(S, q_lens, [max(a, b) for a, b in zip(q_lens, kv_lens)], 28, 4, 128, dtype, 16, path=path, seed=6, tree=True,
                 quantised=quantised)


@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (8, 8, 64), (32, 1, 128), (16, 1, 64), (4, 2, 128)])
def test_few_rows(S, Hq, Hkv, D):
    """At most 32 rows of a kv head: decoding, a few drafted tokens, small trees; short and shared among many CTAs."""
    n = max(1, 32 // (Hq // Hkv))
    g = torch.Generator().manual_seed(Hq)
    for q_lens, kv_lens in (([n], [n]), ([1, n, 0, 1], [1, 130, 7, 64]), ([1] * 9, [31, 32, 33, 127, 128, 129, 160, 161, 300]),
                            ([n, 1], [9000, 5000])):
        for page in (8, 64):
            case(S, q_lens, kv_lens, Hq, Hkv, D, torch.bfloat16, page, seed=n)
            assert S.sd_last_attention_path()[0] == 2
        case(S, q_lens, kv_lens, Hq, Hkv, D, torch.bfloat16, 16, seed=n, causal=False)
        case(S, q_lens, kv_lens, Hq, Hkv, D, torch.bfloat16, 16, seed=n, tree=True)


@pytest.mark.parametrize("path", [1, 0])
def test_sharp_weights_and_uneven_rows(S, path):
    """Scores of +-60, and rows whose scales differ by many powers of two."""
    case(S, [40, 1], [700, 3000], 28, 4, 128, torch.bfloat16, 64, path=path, sd=20.0)
    case(S, [40, 1, 16], [700, 3000, 1000], 28, 4, 128, torch.bfloat16, 16, path=path, sd=0.5, spread=3.0)
    case(S, [1], [2000], 8, 1, 64, torch.bfloat16, 64, path=path, spread=4.0, sd=0.3)


@pytest.mark.parametrize("path", [1, 0])
def test_values_of_zero_and_zero_queries(S, path):
    """Rows of zeros have the smallest scale: they take their weight and give nothing."""
    g = torch.Generator().manual_seed(9)
    m, Hq, Hkv, D, page = 500, 28, 4, 128, 16
    k, v = torch.randn(m, Hkv, D, generator=g), torch.randn(m, Hkv, D, generator=g)
    v[torch.rand(m, generator=g) < 0.5] = 0
    v[:150] = 0
    kc, ks = quantise(k)
    vc, vs = quantise(v)
    n_pages = -(-m // page)
    pad = n_pages * page - m
    paged = lambda c: torch.cat([c.view(torch.uint8), torch.zeros(pad, Hkv, D, dtype=torch.uint8)]).view(torch.float8_e4m3fn).view(
        n_pages, page, Hkv, D).cuda()
    sc = lambda s: torch.cat([s, torch.zeros(pad, Hkv)]).view(n_pages, page, Hkv).transpose(1, 2).contiguous().cuda()
    for q in (torch.randn(16, Hq, D, generator=g).bfloat16() * 2, torch.zeros(16, Hq, D, dtype=torch.bfloat16)):
        out = torch.empty(16, Hq, D, dtype=torch.bfloat16, device="cuda")
        ws = S.workspace(S.sd_paged_attention_workspace_size(16, 1, 16, Hq, Hkv, D, m))
        S.sd_set_attention_path(path)
        S.sd_paged_attention_e4m3(q.cuda(), paged(kc), paged(vc), sc(ks), sc(vs), torch.arange(n_pages, dtype=torch.int32)[None].cuda(),
                                  i32([0, 16]).cuda(), i32([m]).cuda(), 16, m, out, D ** -0.5, ws)
        torch.cuda.synchronize()
        seen = torch.arange(m)[None] <= torch.arange(16)[:, None] + m - 16
        eight = S.sd_last_attention_path()[0] == 2
        want = attend(q, kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None], D ** -0.5, seen,
                      (vc.float().abs(), vs.amax(0).double()) if eight else None)
        check_attention(out, want, torch.bfloat16, "e4m3" if eight else 0)
    assert S.sd_fault_word() == 0


def test_queries_of_any_size(S):
    """Queries are split by a power of two of their own row: the same outputs for q 2^e and scale 2^-e."""
    g = torch.Generator().manual_seed(10)
    pool = Pool(g, [300], 16, 4, 128, torch.bfloat16, True)
    (kp, vp, ks, vs), table = pool.cuda()
    q = torch.randn(7, 28, 128, generator=g).bfloat16().cuda()
    ws = S.workspace(S.sd_paged_attention_workspace_size(7, 1, 7, 28, 4, 128, 300))
    outs = []
    for e in (0, 40, -40):
        out = torch.empty_like(q)
        S.sd_paged_attention_e4m3(q * 2.0 ** e, kp, vp, ks, vs, table, i32([0, 7]).cuda(), i32([300]).cuda(), 7, 300, out,
                                  128 ** -0.5 * 2.0 ** -e, ws)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("path", [1, 0])
def test_bad_pages_and_lengths(S, path):
    g = torch.Generator().manual_seed(11)
    for quantised in (True, False):
        pool = Pool(g, [100, 40], 16, 4, 128, torch.bfloat16, quantised)
        (kp, vp, ks, vs), table = pool.cuda()
        q = torch.randn(6, 28, 128, generator=g).bfloat16().cuda()
        ws = S.workspace(S.sd_paged_attention_workspace_size(6, 2, 3, 28, 4, 128, 200))
        words = torch.full((6,), 7, dtype=torch.int64, device="cuda")
        S.sd_set_attention_path(path)
        for col, page, kv, bit in ((2, 99, [100, 40], BAD_PAGE), (0, -1, [100, 40], BAD_PAGE), (0, None, [200, 40], BAD_LENGTH),
                                   (0, None, [-3, 40], BAD_LENGTH)):
            t = table.clone()
            if page is not None:
                t[0, col] = page
            t[:, -1] = 0
            out = torch.full_like(q, 5.0)
            S.sd_paged_tree_attention(q, kp, vp, t, words, i32([0, 3, 6]).cuda(), i32(kv).cuda(), 3, 150, out, 0.1, ws, ks, vs)
            torch.cuda.synchronize()
            assert S.sd_fault_word() & bit, (quantised, col, page, kv)
            assert int(ws[256:256 + 4096].sum()) == 0
            if page is not None:           # a page that is none reads as zeros; the other sequence is as ever
                v = torch.cat([x[None] for x in pool.values["v"][1:]])[0]
                want = attend(q[3:].cpu(), pool.values["k"][1], v, 0.1, torch.cat([torch.ones(3, 37), torch.ones(3, 3)], 1).bool(),
                              pool.codes[1] if quantised and path == 0 else None)
                check_attention(out[3:], want, torch.bfloat16, 0 if path == 1 else "e4m3" if quantised else "bf16")


def test_wait_gives_up_then_recovers(S):
    for tree, quantised in ((False, True), (True, True), (True, False)):
        call, out, ws = case(S, [16], [20000], 28, 4, 128, torch.bfloat16, 64, tree=tree, quantised=quantised)
        good = out.clone()
        S.sd_set_wait_test(1, 1_000_000)
        call()
        torch.cuda.synchronize()
        S.sd_set_wait_test(0, 0)
        assert S.sd_fault_word() & WAIT_GAVE_UP
        assert int(ws[256:256 + 4096].sum()) == 0
        out.fill_(1.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out[:16], good[:16]) and S.sd_fault_word() == 0


def test_graphs_and_streams(S):
    """A captured call replays on other streams and gives the eager call's bits; two graphs may share a workspace in order."""
    for tree, quantised in ((False, True), (True, True), (True, False)):
        call, out, ws = case(S, [16, 1, 40], [3000, 700, 500], 28, 4, 128, torch.bfloat16, 16, tree=tree, quantised=quantised)
        good = out.clone()
        side = torch.cuda.Stream()
        graphs = []
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                call()
            graphs.append(gr)
        out.fill_(3.0)
        with torch.cuda.stream(side):
            graphs[0].replay()
            graphs[1].replay()
        side.synchronize()
        assert torch.equal(out[:57], good[:57])


# --------------------------------------------------------------------------
# an accepted path
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,quantised", [(torch.bfloat16, True), (torch.bfloat16, False), (torch.float32, False)])
@pytest.mark.parametrize("Hkv,D,page,T", [(4, 128, 16, 60), (1, 64, 5, 16), (8, 32, 64, 64), (2, 128, 1, 30)])
def test_compaction(S, dtype, quantised, Hkv, D, page, T):
    g = torch.Generator().manual_seed(T + page)
    ctx = [1, 40, 333, 100]
    kept = [0, 1, T - 1, min(7, T - 1)]
    pool = Pool(g, [c - 1 + T for c in ctx], page, Hkv, D, dtype, quantised, head_major=page == 64)
    path = torch.full((4, T), -1, dtype=torch.int32)
    for b, n in enumerate(kept):
        # any order, also one that a depth's destination is another's source of
        path[b, :n] = (torch.randperm(T - 1, generator=g)[:n] + 1).to(torch.int32)
    parts, table = pool.cuda()
    want = [None if t is None else t.cpu().clone() for t in parts]
    for b, n in enumerate(kept):
        old = [ctx[b] - 1 + int(path[b, d]) for d in range(n)]
        for t in want:
            if t is None:
                continue
            raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
            at = lambda i: (int(pool.table[b, i // page]), i % page) if t.dim() == 4 else (int(pool.table[b, i // page]), slice(None), i % page)
            rows = [raw[at(i)].clone() for i in old]
            for d, r in enumerate(rows):
                raw[at(ctx[b] + d)] = r
    S.sd_compact_tree_paged(parts[0], parts[1], table, i32(ctx).cuda(), path.cuda(), i32(kept).cuda(), parts[2], parts[3])
    torch.cuda.synchronize()
    assert S.sd_fault_word() == 0
    bits = lambda t: t.contiguous().view(torch.uint8)
    for got, w in zip(parts, want):
        assert w is None or torch.equal(bits(got.cpu()), bits(w))


def test_compaction_skips_what_is_out_of_range(S):
    g = torch.Generator().manual_seed(12)
    pool = Pool(g, [60], 16, 2, 64, torch.bfloat16, True)
    for ctx, path, n, table, bit in (
            (45, [3, 20], 2, None, BAD_COMMIT), (45, [0, 2], 2, None, BAD_COMMIT), (45, [3, 5], 17, None, BAD_COMMIT),
            (45, [3, 5], -1, None, BAD_COMMIT), (0, [3, 5], 2, None, BAD_COMMIT), (2 ** 31 - 1, [3, 5], 2, None, BAD_COMMIT),
            (45, [3, 5], 2, 99, BAD_PAGE), (45, [3, 5], 2, -1, BAD_PAGE)):
        parts, t = pool.cuda()
        before = [x.clone() for x in parts]
        if table is not None:
            t[0, 2] = table
        p = torch.full((1, 16), -1, dtype=torch.int32)
        p[0, :2] = i32(path)
        S.sd_compact_tree_paged(parts[0], parts[1], t, i32([ctx]).cuda(), p.cuda(), i32([n]).cuda(), parts[2], parts[3])
        torch.cuda.synchronize()
        assert S.sd_fault_word() & bit, (ctx, path, n, table)
        for a, b in zip(parts, before):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# --------------------------------------------------------------------------
# a run of them
# --------------------------------------------------------------------------

@pytest.mark.parametrize("quantised", [True, False])
def test_a_tree_is_drafted_verified_and_committed(S, quantised):
    """A prompt enters the cache, a tree over it is verified, its accepted path moved, and the next token decoded:
    as if the path's tokens alone had been appended."""
    g = torch.Generator().manual_seed(20)
    Hq, Hkv, D, page, n, T = 28, 4, 128, 16, 250, 30
    parts, order = (16, 24, 24), "blocks"
    turns = S.sd_rotary_table(D, 1e6)[0].cuda()
    wq, wk = (torch.randn(D, generator=g) * 0.2 + 1).bfloat16().cuda(), (torch.randn(D, generator=g) * 0.2 + 1).bfloat16().cuda()
    rows = torch.randn(n + T + 1, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    masks, parents = tree_masks(g, T, 0.4)
    depth = [0] * T
    for j in range(1, T):
        depth[j] = depth[parents[j]] + 1
    leaf = max(range(T), key=lambda j: depth[j])
    path = []
    while leaf > 0:
        path.insert(0, leaf)
        leaf = parents[leaf]
    positions = torch.cat([torch.arange(n), torch.tensor([n + d for d in depth]), torch.tensor([n + len(path) + 1])]).to(torch.int32)
    positions = torch.stack([positions, positions // 3, positions % 50]).cuda()
    table = torch.randperm(30, generator=g).to(torch.int32)[None].cuda()
    dt = torch.float8_e4m3fn if quantised else torch.bfloat16

    def fresh():
        pages = [torch.zeros(30, page, Hkv, D, device="cuda").to(dt) for _ in range(2)]
        return pages, [torch.zeros(30, Hkv, page, device="cuda") for _ in range(2)] if quantised else [None, None]

    def append(cache, which, kv_len):
        m = len(which)
        x = rows[which]
        q = torch.empty(m, Hq, D, dtype=torch.bfloat16, device="cuda")
        S.sd_norm_rotary_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q, positions[:, which].contiguous(), turns,
                                      i32([0, m]).cuda(), i32([kv_len]).cuda(), table, *cache[0], *cache[1], q_weight=wq,
                                      k_weight=wk, axes=parts, axes_order=order)
        return q

    def attention(cache, q, kv_len, words=None):
        m = len(q)
        out = torch.empty_like(q)
        ws = S.workspace(S.sd_paged_attention_workspace_size(m, 1, m, Hq, Hkv, D, kv_len))
        at = (i32([0, m]).cuda(), i32([kv_len]).cuda(), m, kv_len, out, D ** -0.5, ws)
        if words is not None:
            S.sd_paged_tree_attention(q, *cache[0], table, signed(words).cuda(), *at, *cache[1])
        elif quantised:
            S.sd_paged_attention_e4m3(q, *cache[0], *cache[1], table, *at)
        else:
            S.sd_paged_attention(q, *cache[0], table, *at)
        return out

    cache = fresh()
    append(cache, list(range(n)), n)
    q = append(cache, list(range(n, n + T)), n + T)
    tree = attention(cache, q, n + T, masks)
    S.sd_compact_tree_paged(*cache[0], table, i32([n + 1]).cuda(), torch.tensor([path + [-1] * (T - len(path))], dtype=torch.int32).cuda(),
                            i32([len(path)]).cuda(), *cache[1])
    kept = n + 1 + len(path)
    q1 = append(cache, [n + T], kept + 1)
    last = attention(cache, q1, kept + 1)
    # the path alone
    plain = fresh()
    append(plain, list(range(n)) + [n] + [n + j for j in path], kept)
    q2 = append(plain, [n + T], kept + 1)
    want = attention(plain, q2, kept + 1)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(last, want)
    pos = torch.arange(kept + 1)
    pg, sl = table[0, pos // page].long(), pos % page
    for a, b in zip(cache[0], plain[0]):
        assert torch.equal(a.view(torch.uint8)[pg, sl] if quantised else a[pg, sl], b.view(torch.uint8)[pg, sl] if quantised else b[pg, sl])
    # the tree's nodes along the path see what a causal chain of them sees
    chain = attention(plain, torch.cat([q[:1], q[path]]), kept)
    got, ref = tree[[0] + path].float(), chain.float()
    # both are off by a weight's 2^-8 and a half step at most, of averages of values up to |v|'s largest
    top = float(rows[:, Hq + Hkv:].abs().max())
    assert float((got - ref).abs().max()) <= 4 * 2.0 ** -8 * top
    assert S.sd_fault_word() == 0


@pytest.mark.parametrize("quantised", [True, False])
def test_pools_past_32_bit_offsets(S, quantised):
    """Pages whose offsets, in elements and in scales' bytes, pass 2^32: the same bits as in a pool of three."""
    g = torch.Generator().manual_seed(30)
    Hq, Hkv, D, page, n = 32, 8, 128, 128, 300
    far = 36000 if quantised else 33100
    dt = torch.uint8 if quantised else torch.bfloat16
    x = torch.randn(n, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    turns = S.sd_rotary_table(D, 1e6)[0].cuda()
    path = torch.full((1, 40), -1, dtype=torch.int32)
    path[0, :3] = i32([4, 9, 30])
    results = []
    for pages, ids in ((3, [2, 0, 1]), (far, [far - 1, 1, far - 2])):
        kp, vp = (torch.empty(pages, page, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
        sc = [torch.empty(pages, Hkv, page, device="cuda") for _ in range(2)] if quantised else [None, None]
        if quantised:
            kp, vp = kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
        table = i32([ids]).cuda()
        q = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
        S.sd_norm_rotary_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q, None, turns, i32([0, n]).cuda(), i32([n]).cuda(),
                                      table, kp, vp, *sc)
        S.sd_compact_tree_paged(kp, vp, table, i32([n - 39]).cuda(), path.cuda(), i32([3]).cuda(), *sc)
        outs = []
        for forced in (0, 1):
            S.sd_set_attention_path(forced)
            out = torch.empty(40, Hq, D, dtype=torch.bfloat16, device="cuda")
            ws = S.workspace(S.sd_paged_attention_workspace_size(40, 1, 40, Hq, Hkv, D, n))
            words = signed([(1 << 40) - 1] * 40).cuda()
            S.sd_paged_tree_attention(q[-40:], kp, vp, table, words, i32([0, 40]).cuda(), i32([n]).cuda(), 40, n, out, D ** -0.5, ws, *sc)
            outs.append(out)
        rows = [(t.view(torch.uint8) if quantised else t)[ids] for t in (kp, vp)]
        results.append(outs + [r.flatten(0, 1)[:n] for r in rows] + ([s[ids].transpose(1, 2).flatten(0, 1)[:n] for s in sc] if quantised else []))
        del kp, vp, sc
    assert all(torch.equal(a, b) for a, b in zip(*results)) and S.sd_fault_word() == 0
