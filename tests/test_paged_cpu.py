"""CPU checks of the rotary, paged-cache and packed-attention entry points:
the rotary table against its formula, workspace sizes, and refusals on the
host (status codes, no launch)."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    return sd_verify


def frequency(i, R, theta, scaling, factor, L, low, high):
    w = theta ** (-2.0 * i / R)
    if scaling == "linear":
        return w / factor
    if scaling == "ntk":
        return (theta * factor ** (R / (R - 2))) ** (-2.0 * i / R)
    if scaling in ("parts", "yarn"):
        g = min(1.0, max(0.0, (L * w / (2 * math.pi) - low) / (high - low)))
        return (1 - g) * w / factor + g * w
    return w


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts", "yarn"])
@pytest.mark.parametrize("R,theta,factor", [(128, 1e6, 4.0), (64, 1e4, 8.0), (20, 5e5, 1.0), (4, 1e4, 2.5)])
def test_rotary_table_follows_the_formula(S, scaling, R, theta, factor):
    turns, m = S.sd_rotary_table(R, theta, scaling=scaling, factor=factor, original_max=8192, low=1.0, high=4.0)
    assert turns.shape == (R // 2,) and turns.dtype == torch.int64
    for i, word in enumerate(turns.tolist()):
        t = frequency(i, R, theta, scaling, factor, 8192, 1.0, 4.0) / (2 * math.pi)
        # both sides round a handful of fp64 operations, the power among them: 16 ulps of the value
        assert abs((word % 2 ** 64) / 2.0 ** 64 - t % 1.0) <= 16 * 2.0 ** -53 * t + 2.0 ** -64
    want = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    assert abs(m - want) <= 2.0 ** -23 * want


def test_rotary_table_of_two_and_whole_turns(S):
    # theta < 1 gives frequencies above one turn per position: only the fraction counts
    turns, _ = S.sd_rotary_table(4, 1e-3)
    t = (1e-3 ** -0.5) / (2 * math.pi)
    assert abs((turns[1].item() % 2 ** 64) / 2.0 ** 64 - t % 1.0) <= 16 * 2.0 ** -53 * t
    assert S.sd_rotary_table(2, 1e4)[0].shape == (1,)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1026), dict(theta=0.0), dict(theta=-1.0),
    dict(theta=float("inf")), dict(theta=float("nan")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("nan")), dict(scaling="ntk", rot_dim=2, factor=2.0),
    dict(scaling="yarn", factor=2.0, original_max=0), dict(scaling="parts", factor=2.0, original_max=10, low=4.0, high=4.0),
    dict(scaling="parts", factor=2.0, original_max=10, low=-1.0, high=4.0)])
def test_rotary_table_refusals(S, kw):
    args = dict(rot_dim=64, theta=1e4)
    args.update(kw)
    with pytest.raises(S.SdError) as e:
        S.sd_rotary_table(**args)
    assert e.value.status == S.SD_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        S.sd_rotary_table(64, 1e4, scaling="other")


def test_workspace_sizes(S):
    f = S.sd_paged_attention_workspace_size
    base = f(128, 8, 16, 28, 4, 128, 32768)
    assert base > 256
    for more in ((256, 8, 16, 28, 4, 128, 32768), (128, 16, 16, 28, 4, 128, 32768), (128, 8, 32, 28, 4, 128, 32768),
                 (128, 8, 16, 28, 4, 128, 65536)):
        assert f(*more) >= base
    assert f(128, 8, 16, 28, 4, 96, 32768) == 0 and f(128, 0, 16, 28, 4, 128, 32768) == 0
    assert f(128, 8, 16, 65, 1, 128, 32768) == 0 and f(128, 8, 16, 30, 4, 128, 32768) == 0
    assert f(0, 1, 0, 4, 1, 64, 0) > 0


FAKE = 0x10000      # 16-byte aligned, never dereferenced


def cache(S, **kw):
    d = dict(k=FAKE, v=FAKE, strides=S.Strides(16 * 4 * 128, 4 * 128, 128), table=FAKE, table_stride=8, table_cols=8,
             n_pages=10, page_size=16)
    d.update(kw)
    return S.PagedCache(**d)


def paged(S, c=None, **kw):
    d = dict(q=FAKE, q_tok=28 * 128, q_head=128, cu=FAKE, kv=FAKE, max_q=16, max_kv=128, out=FAKE, N=32, B=2, Hq=28,
             Hkv=4, D=128, dt=0, scale=1.0, causal=1, ws=FAKE, ws_bytes=1 << 40)
    d.update(kw)
    return S.load().sd_paged_attention(d["q"], d["q_tok"], d["q_head"], c if c is not None else cache(S), d["cu"],
                                       d["kv"], d["max_q"], d["max_kv"], d["out"], d["N"], d["B"], d["Hq"], d["Hkv"],
                                       d["D"], d["dt"], d["scale"], d["causal"], d["ws"], d["ws_bytes"], None)


def test_paged_attention_refusals(S):
    bad, uns = S.SD_ERR_INVALID_ARG, S.SD_ERR_UNSUPPORTED
    assert paged(S, q=None) == bad and paged(S, out=None) == bad and paged(S, cu=None) == bad
    assert paged(S, kv=None) == bad and paged(S, q=FAKE + 8) == bad and paged(S, out=FAKE + 8) == bad
    assert paged(S, q_tok=28 * 128 + 4) == bad and paged(S, q_head=64) == bad
    assert paged(S, B=0) == bad and paged(S, B=70000) == bad and paged(S, N=-1) == bad
    assert paged(S, max_kv=-1) == bad and paged(S, max_kv=2 ** 26 + 1) == bad and paged(S, max_q=-1) == bad
    assert paged(S, Hq=27) == bad and paged(S, D=96) == uns and paged(S, Hq=65 * 4) == uns and paged(S, dt=7) == bad
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert paged(S, scale=s) == bad
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(n_pages=0), dict(page_size=0), dict(table_cols=0),
               dict(table_stride=0), dict(k=FAKE + 8), dict(strides=S.Strides(16 * 4 * 128, 4 * 128, 64)),
               dict(strides=S.Strides(16 * 4 * 128, 4 * 128 + 4, 128)), dict(table=FAKE + 2)):
        assert paged(S, cache(S, **kw)) == bad, kw
    assert S.load().sd_paged_attention(FAKE, 3584, 128, None, FAKE, FAKE, 16, 128, FAKE, 32, 2, 28, 4, 128, 0, 1.0, 1,
                                       FAKE, 1 << 30, None) == bad
    # nothing to do, and said so without a GPU
    assert paged(S, N=0) == S.SD_OK


def test_prompt_attention_refusals(S):
    def call(**kw):
        d = dict(q=FAKE, q_tok=28 * 128, k=FAKE, v=FAKE, kv_tok=512, kv_head=128, cu=FAKE, max_len=64, N=64, B=2, D=128,
                 scale=1.0)
        d.update(kw)
        return S.load().sd_prompt_attention(d["q"], d["q_tok"], 128, d["k"], d["v"], d["kv_tok"], d["kv_head"], d["cu"],
                                            d["max_len"], FAKE, d["N"], d["B"], 28, 4, d["D"], 0, d["scale"], 1, FAKE,
                                            1 << 40, None)
    bad = S.SD_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(kv_tok=516), dict(kv_head=64),
               dict(k=FAKE + 8), dict(max_len=-1), dict(B=0), dict(scale=0.0)):
        assert call(**kw) == bad, kw
    assert call(D=80) == S.SD_ERR_UNSUPPORTED
    assert call(N=0) == S.SD_OK


def test_rotary_refusals(S):
    def call(**kw):
        d = dict(x=FAKE, x_tok=512, x_head=128, y=FAKE + 4096, y_tok=512, y_head=128, pos=FAKE, turns=FAKE, m=1.0, N=8,
                 H=4, D=128, rot=128, lay=0, dt=0)
        d.update(kw)
        return S.load().sd_rotary(d["x"], d["x_tok"], d["x_head"], d["y"], d["y_tok"], d["y_head"], d["pos"],
                                  d["turns"], d["m"], d["N"], d["H"], d["D"], d["rot"], d["lay"], d["dt"], None)
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(turns=None), dict(turns=FAKE + 4), dict(rot=0),
               dict(rot=130), dict(rot=63), dict(D=2048), dict(H=0), dict(N=-1), dict(lay=2), dict(dt=3),
               dict(y_head=64), dict(x_tok=100), dict(y=FAKE, y_tok=1024), dict(m=float("nan")), dict(x=FAKE + 1)):
        assert call(**kw) == S.SD_ERR_INVALID_ARG, kw
    assert call(N=0) == S.SD_OK

    def append(c=None, **kw):
        d = dict(q=FAKE, qo=FAKE + 4096, k=FAKE, v=FAKE, cu=FAKE, kv=FAKE, turns=FAKE, B=2, N=8, Hkv=4, kv_tok=512)
        d.update(kw)
        return S.load().sd_rotary_append_paged(d["q"], 512, 128, d["k"], d["v"], d["kv_tok"], 128, d["qo"], FAKE,
                                               d["turns"], 1.0, 128, 0, d["cu"], d["kv"],
                                               c if c is not None else cache(S), d["N"], d["B"], 4, d["Hkv"], 128, 0,
                                               None)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(cu=None), dict(kv=None), dict(turns=None),
               dict(B=0), dict(Hkv=0), dict(kv_tok=100), dict(c=cache(S, k=None)), dict(c=cache(S, n_pages=0)),
               dict(c=cache(S, strides=S.Strides(1, 512, 128)))):
        assert append(**kw) == S.SD_ERR_INVALID_ARG, kw
    assert append(N=0) == S.SD_OK


def test_binding_refusals(S):
    q = torch.zeros(4, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(2, 16, 1, 64)
    with pytest.raises(ValueError):
        S.sd_prompt_attention(q, q, q, i, 4, q, 1.0, torch.zeros(8))
    with pytest.raises(ValueError):
        S.sd_paged_attention(q, pages, pages, i[None], i, i[:1], 4, 4, q, 1.0, torch.zeros(8))
    with pytest.raises(ValueError):
        S.sd_rotary(q, q, i, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        S.sd_rotary_append_paged(None, q, q, None, None, torch.zeros(32, dtype=torch.int64), i, i[:1], i[None], pages, pages)
