"""CPU checks of the calls with norms and axes, the 8-bit cache and trees over pages: refusals on the host (status
codes, no launch) and in the binding."""
import pytest
import torch

FAKE = 0x10000      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    return sd_verify


def cache(S, **kw):
    d = dict(k=FAKE, v=FAKE, strides=S.Strides(16 * 4 * 128, 4 * 128, 128), table=FAKE, table_stride=8, table_cols=8,
             n_pages=10, page_size=16)
    d.update(kw)
    return S.PagedCache(**d)


def axes(S, *pairs, order=0, n=None):
    return S.RopeAxes(len(pairs) if n is None else n, tuple(pairs[:4]), order)


def norm(S, **kw):
    d = dict(q=FAKE, q_tok=512, q_head=128, qo=FAKE + 4096, qo_tok=512, qo_head=128, k=FAKE, k_tok=512, k_head=128,
             ko=FAKE + 4096, ko_tok=512, ko_head=128, wq=FAKE, wk=FAKE, eps=1e-6, pos=FAKE, stride=8, axes=axes(S, 16, 24, 24),
             turns=FAKE, m=1.0, N=8, Hq=4, Hk=2, D=128, R=128, lay=0, dt=0)
    d.update(kw)
    return S.load().sd_norm_rotary(*(d[x] for x in ("q", "q_tok", "q_head", "qo", "qo_tok", "qo_head", "k", "k_tok", "k_head",
                                                    "ko", "ko_tok", "ko_head", "wq", "wk", "eps", "pos", "stride", "axes",
                                                    "turns", "m", "N", "Hq", "Hk", "D", "R", "lay", "dt")), None)


def test_norm_rotary_refusals(S):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None), dict(turns=None), dict(turns=FAKE + 4),
               dict(pos=FAKE + 2), dict(wq=FAKE + 1), dict(wk=FAKE + 1), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
               dict(R=0), dict(R=63), dict(R=130), dict(D=2048), dict(Hq=0), dict(Hk=-1), dict(N=-1), dict(lay=2), dict(dt=2),
               dict(m=nan), dict(q_tok=100), dict(qo_head=64), dict(k_head=64), dict(ko_tok=100), dict(stride=0),
               dict(qo=FAKE, qo_tok=1024), dict(ko=FAKE, ko_head=256), dict(axes=axes(S, 16, 24, 23)),
               dict(axes=axes(S, 64, 0)), dict(axes=axes(S, 70, -6)), dict(axes=axes(S, 64, order=2)),
               dict(axes=axes(S, n=0)), dict(axes=axes(S, 16, 16, 16, 16, n=5)), dict(R=64)):
        assert norm(S, **kw) == S.SD_ERR_INVALID_ARG, kw
    assert norm(S, Hq=5000) == S.SD_ERR_UNSUPPORTED
    assert norm(S, N=0) == S.SD_OK and norm(S, N=0, axes=None) == S.SD_OK


def append(S, c=None, sc="own", **kw):
    d = dict(q=FAKE, qo=FAKE + 4096, k=FAKE, v=FAKE, kv_tok=512, wq=None, wk=FAKE, eps=1e-6, pos=FAKE, stride=8, axes=None,
             turns=FAKE, cu=FAKE, kv=FAKE, N=8, B=2, Hkv=4)
    d.update(kw)
    sc = S.PageScales(FAKE, FAKE) if sc == "own" else sc
    return S.load().sd_norm_rotary_append_paged(
        d["q"], 512, 128, d["k"], d["v"], d["kv_tok"], 128, d["qo"], d["wq"], d["wk"], d["eps"], d["pos"], d["stride"],
        d["axes"], d["turns"], 1.0, 128, 0, d["cu"], d["kv"], c if c is not None else cache(S), sc, d["N"], d["B"], 4, d["Hkv"],
        128, 0, None)


def test_append_refusals(S):
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(cu=None), dict(kv=None), dict(turns=None),
               dict(B=0), dict(Hkv=0), dict(kv_tok=100), dict(c=cache(S, k=None)), dict(c=cache(S, n_pages=0)),
               dict(c=cache(S, strides=S.Strides(1, 512, 128))), dict(sc=S.PageScales(None, FAKE)),
               dict(sc=S.PageScales(FAKE, None)), dict(sc=S.PageScales(FAKE + 8, FAKE)), dict(eps=-1.0),
               dict(axes=axes(S, 1, 2)), dict(k=FAKE + 1)):
        assert append(S, **kw) == S.SD_ERR_INVALID_ARG, kw
    assert append(S, sc=None, c=cache(S, k=FAKE + 1)) == S.SD_ERR_INVALID_ARG
    assert append(S, N=0) == S.SD_OK and append(S, N=0, sc=None) == S.SD_OK


def attend(S, tree, c=None, sc="own", **kw):
    d = dict(q=FAKE, q_tok=28 * 128, q_head=128, cu=FAKE, kv=FAKE, max_q=16, max_kv=128, out=FAKE, N=32, B=2, Hq=28, Hkv=4,
             D=128, dt=0, scale=1.0, ws=FAKE, mask=FAKE)
    d.update(kw)
    sc = S.PageScales(FAKE, FAKE) if sc == "own" else sc
    c = c if c is not None else cache(S)
    tail = (d["cu"], d["kv"], d["max_q"], d["max_kv"], d["out"], d["N"], d["B"], d["Hq"], d["Hkv"], d["D"], d["dt"], d["scale"])
    end = (d["ws"], 1 << 40, None)
    if tree:
        return S.load().sd_paged_tree_attention(d["q"], d["q_tok"], d["q_head"], c, sc, d["mask"], *tail, *end)
    return S.load().sd_paged_attention_e4m3(d["q"], d["q_tok"], d["q_head"], c, sc, *tail, 1, *end)


@pytest.mark.parametrize("tree", [False, True])
def test_attention_refusals(S, tree):
    bad, uns = S.SD_ERR_INVALID_ARG, S.SD_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(out=None), dict(cu=None), dict(kv=None), dict(q=FAKE + 8), dict(out=FAKE + 8),
               dict(q_tok=28 * 128 + 4), dict(q_head=64), dict(B=0), dict(B=70000), dict(N=-1), dict(max_kv=-1),
               dict(max_q=-1), dict(Hq=27), dict(dt=2), dict(scale=0.0), dict(scale=float("nan")),
               dict(c=cache(S, k=FAKE + 8)), dict(c=cache(S, table=None)), dict(c=cache(S, n_pages=0)),
               dict(c=cache(S, strides=S.Strides(16 * 4 * 128, 4 * 128 + 8, 128))), dict(sc=S.PageScales(None, FAKE)),
               dict(sc=S.PageScales(FAKE, FAKE + 4))):
        assert attend(S, tree, **kw) == bad, kw
    assert attend(S, tree, D=96) == uns and attend(S, tree, Hq=65 * 4) == uns
    assert attend(S, tree, N=0) == S.SD_OK
    if tree:
        assert attend(S, tree, max_q=65) == bad and attend(S, tree, mask=None) == bad and attend(S, tree, mask=FAKE + 4) == bad
        # bf16 pages: strides of 16 bytes
        assert attend(S, tree, sc=None, c=cache(S, strides=S.Strides(16 * 4 * 128, 4 * 128 + 4, 128))) == bad
    else:
        assert attend(S, tree, sc=None) == bad


def test_compact_refusals(S):
    def call(c=None, sc=None, **kw):
        d = dict(ctx=FAKE, path=FAKE, n=FAKE, B=2, T=16, Hkv=4, D=128, dt=0)
        d.update(kw)
        return S.load().sd_compact_tree_paged(c if c is not None else cache(S), sc, d["ctx"], d["path"], d["n"], d["B"], d["T"],
                                              d["Hkv"], d["D"], d["dt"], None)
    for kw in (dict(ctx=None), dict(path=None), dict(n=None), dict(path=FAKE + 2), dict(B=0), dict(T=0), dict(T=65), dict(Hkv=0),
               dict(Hkv=5000), dict(D=0), dict(dt=2), dict(c=cache(S, k=FAKE + 8)), dict(c=cache(S, table=None)),
               dict(sc=S.PageScales(FAKE, None)), dict(c=cache(S, strides=S.Strides(16 * 4 * 128, 4 * 128 + 4, 128)))):
        assert call(**kw) == S.SD_ERR_INVALID_ARG, kw
    assert call(D=100) == S.SD_ERR_UNSUPPORTED and call(D=512) == S.SD_ERR_UNSUPPORTED
    assert call(sc=S.PageScales(FAKE, FAKE), D=24) == S.SD_ERR_UNSUPPORTED


def test_binding_refusals(S):
    q = torch.zeros(4, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(32, dtype=torch.int64)
    pages = torch.zeros(2, 16, 1, 64)
    sc = torch.zeros(2, 1, 16)
    for call in (lambda: S.sd_norm_rotary(q, q, None, None, i, t),
                 lambda: S.sd_norm_rotary_append_paged(None, q, q, None, None, t, i, i[:1], i[None], pages, pages),
                 lambda: S.sd_paged_attention_e4m3(q, pages, pages, sc, sc, i[None], i, i[:1], 4, 4, q, 1.0, sc),
                 lambda: S.sd_paged_tree_attention(q, pages, pages, i[None], t[:4], i, i[:1], 4, 4, q, 1.0, sc),
                 lambda: S.sd_compact_tree_paged(pages, pages, i[None], i[:1], i[None], i[:1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        S._axes_arg((16, 15), "blocks", 32)
    with pytest.raises(ValueError):
        S._axes_arg((8,) * 5, "blocks", 40)
    with pytest.raises(ValueError):
        S._axes_arg((16, 16), "rows", 32)
    for bad in (torch.zeros(3, 8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(2, 8),
                torch.zeros(2, 7, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.int32).T):
        with pytest.raises(ValueError):
            S._axes_positions(bad, 2, 8)
    for a, b, p in ((None, sc, pages), (sc, sc, pages), (sc[:1], sc, pages.to(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            S._page_scales(a, b, p, torch.float32)
    with pytest.raises(ValueError):
        S._page_scales(None, None, pages, torch.bfloat16)
