"""The binding's short way (fast_calls.cpp) against its long one: the same bits from the same arguments, the same
refusals, and the short way taken by the calls that every check lets through."""
import pytest
import torch

from _quant import quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    return sd_verify


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def calls(S):
    """name -> (the binding's function, its short way's, arguments by name, outputs)"""
    g = torch.Generator().manual_seed(1)
    N, Hq, Hkv, D, page, pages = 20, 8, 2, 128, 16, 4
    x = torch.randn(N, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    w = torch.rand(D, generator=g).bfloat16().cuda()
    qo, ko = torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(N, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.randint(0, 99, (3, N), generator=g, dtype=torch.int32).cuda()
    turns = S.sd_rotary_table(D, 1e4)[0].cuda()
    rows = [quantise(torch.randn(pages, page, Hkv, D, generator=g)) for _ in range(2)]
    kp, vp = (r[0].cuda() for r in rows)
    ks, vs = (r[1].transpose(1, 2).contiguous().cuda() for r in rows)
    cu, kv, table = i32([0, 4, 20]), i32([30, 32]), i32([[0, 1], [3, 2]])
    out = torch.empty_like(qo)
    ws = S.workspace(S.sd_paged_attention_workspace_size(N, 2, 16, Hq, Hkv, D, 32))
    rope = dict(positions=pos, turns=turns, q_weight=w, k_weight=w, axes=(16, 24, 24), axes_order="stripes", layout="interleaved",
                eps=1e-5, magnitude=1.5)
    cache = dict(k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, page_table=table)
    at = dict(cu_q=cu, kv_len=kv, max_q=16, max_kv=32, out=out, scale=0.1, ws=ws)
    return {
        "norm": (S.sd_norm_rotary, "norm_rotary", dict(q=q, q_out=qo, k=k, k_out=ko, **rope), (qo, ko)),
        "append": (S.sd_norm_rotary_append_paged, "append", dict(q=q, k=k, v=v, q_out=qo, cu_q=cu, kv_len=kv, **rope, **cache),
                   (qo, kp, vp, ks, vs)),
        "attend": (S.sd_paged_attention_e4m3, "attend", dict(q=qo, causal=False, **cache, **at), (out,)),
        "tree": (S.sd_paged_tree_attention, "attend", dict(q=qo, tree_mask=torch.full((N,), 0xffff, device="cuda"), **cache, **at), (out,)),
        "compact": (S.sd_compact_tree_paged, "compact",
                    dict(**cache, ctx_len=i32([10, 12]), path=i32([[2, 5, -1], [1, -1, -1]]).repeat(1, 3)[:, :8].contiguous(),
                         n_accepted=i32([2, 1])), (kp, vp, ks, vs)),
    }


def bits(t):
    return t.contiguous().view(torch.uint8)


class Counting:
    def __init__(self, fast):
        self.fast, self.taken = fast, []

    def __getattr__(self, name):
        def call(*a):
            r = getattr(self.fast, name)(*a)
            self.taken.append((name, r))
            return r
        return call


@pytest.mark.parametrize("name", ["norm", "append", "attend", "tree", "compact"])
def test_same_bits_either_way(S, calls, monkeypatch, name):
    fn, short, kw, outs = calls[name]
    before = [o.clone() for o in outs]
    results = []
    for way in ("short", "long", "stream"):
        for o, b in zip(outs, before):
            bits(o).copy_(bits(b)) if o.is_contiguous() else o.copy_(b)
        counting = Counting(S._fast)
        monkeypatch.setattr(S, "_fast", counting if way != "long" else None)
        fn(**kw, **(dict(stream=torch.cuda.current_stream()) if way == "stream" else {}))
        monkeypatch.undo()
        assert counting.taken == ([(short, S.SD_OK)] if way == "short" else [])
        torch.cuda.synchronize()
        results.append([bits(o).clone() for o in outs])
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))
    assert S.sd_fault_word() == 0


BAD = {
    "norm": [dict(q_out=None), dict(k=None), dict(positions=None), dict(axes=(16, 24)), dict(axes=(8,) * 8), dict(axes_order="rows"),
             dict(layout="other"), dict(turns="float"), dict(q_weight="short"), dict(positions="int64"), dict(q="cpu"), dict(eps=-1.0),
             dict(q_out="float"), dict(positions="strided")],
    "append": [dict(q=None), dict(k_scale=None), dict(v="short"), dict(cu_q="short"), dict(kv_len="int64"), dict(page_table="int64"),
               dict(k_pages="uint8"), dict(k_scale="short"), dict(axes=(64, 0)), dict(k_weight="cpu"), dict(positions="short")],
    "attend": [dict(k_scale=None), dict(v_scale="float64"), dict(out="strided"), dict(max_q=-1), dict(scale=0.0), dict(ws="tiny"),
               dict(q="cpu"), dict(k_pages="uint8"), dict(kv_len="short")],
    "tree": [dict(tree_mask="short"), dict(tree_mask="int32"), dict(max_q=65), dict(k_scale=None), dict(ws="tiny"), dict(out="float")],
    "compact": [dict(path="int64"), dict(n_accepted="short"), dict(ctx_len="short"), dict(k_scale=None), dict(k_pages="cpu")],
}


def spoiled(t, how):
    if how == "short":
        return t[:-1].contiguous()
    if how == "strided":
        return torch.stack([t, t], -1)[..., 0]
    if how == "cpu":
        return t.cpu()
    if how == "tiny":
        return t[:256]
    if how == "uint8":
        return t.view(torch.uint8)
    return t.to(dict(float=torch.float32, float64=torch.float64, int64=torch.int64, int32=torch.int32)[how])


@pytest.mark.parametrize("name", sorted(BAD))
def test_same_refusals_either_way(S, calls, monkeypatch, name):
    fn, _, kw, outs = calls[name]
    before = [bits(o).clone() for o in outs]
    for bad in BAD[name]:
        (key, how), = bad.items()
        args = dict(kw, **{key: spoiled(kw[key], how) if isinstance(how, str) and isinstance(kw[key], torch.Tensor) else how})
        said = []
        for way in (S._fast, None):
            monkeypatch.setattr(S, "_fast", way)
            with pytest.raises((ValueError, TypeError, AttributeError, S.SdError)) as e:
                fn(**args)
            monkeypatch.undo()
            said.append((type(e.value), str(e.value)))
        assert said[0] == said[1], (bad, said)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(o), b) for o, b in zip(outs, before)) and S.sd_fault_word() == 0
