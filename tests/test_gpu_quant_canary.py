"""Canary padding around every buffer of the calls with norms and axes, the 8-bit cache and trees over pages
(test_gpu_canary says how): nothing is written outside the buffers given, or into an input."""
import pytest
import torch

from _quant import quantise, signed, tree_masks
from test_gpu_canary import Arena

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    yield sd_verify
    sd_verify.sd_set_attention_path(0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


@pytest.mark.parametrize("D,R", [(128, 128), (64, 20), (30, 6)])
@pytest.mark.parametrize("quantised", [True, False])
def test_norm_and_append(S, D, R, quantised):
    g = torch.Generator().manual_seed(D)
    a = Arena()
    N, Hq, Hkv, page = 19, 5, 2, 8
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16()
    q, k, v, w = a.inp(rand(N, Hq, D)), a.inp(rand(N, Hkv, D)), a.inp(rand(N, Hkv, D)), a.inp(rand(D))
    pos, turns = a.inp(torch.randint(0, 99, (2, N), generator=g, dtype=torch.int32)), a.inp(S.sd_rotary_table(R, 1e4)[0])
    qo, ko = a.out((N, Hq, D), torch.bfloat16, 0), a.out((N, Hkv, D), torch.bfloat16, 0)
    axes = (R // 2 - 1, 1)
    S.sd_norm_rotary(q, qo, k, ko, pos, turns, q_weight=w, k_weight=w, axes=axes)
    cu, kv, table = a.inp(i32([0, 3, 3, 19])), a.inp(i32([3, 5, 20])), a.inp(i32([[2, 9, 9], [9, 9, 9], [0, 3, 1]]))
    dt = torch.uint8 if quantised else torch.bfloat16
    kp, vp = (a.out((4, page, Hkv, D), dt, 0) for _ in range(2))
    sc = [a.out((4, Hkv, page), torch.float32, 0) for _ in range(2)] if quantised else [None, None]
    if quantised:
        kp, vp = kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    S.sd_norm_rotary_append_paged(q, k, v, qo, pos, turns, cu, kv, table, kp, vp, *sc, q_weight=w, k_weight=w, axes=axes)
    a.check()
    assert S.sd_fault_word() == 0
    S.sd_compact_tree_paged(kp, vp, a.inp(i32([[0, 3, 1]])), a.inp(i32([5])), a.inp(i32([[2, 7] + [-1] * 14])), a.inp(i32([2])), *sc) \
        if D % 16 == 0 else None
    a.check()
    assert S.sd_fault_word() == 0


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 2], [300, 77], 7), ([16, 5], [1000, 64], 7), ([60, 33], [700, 129], 4)])
def test_attention(S, D, quantised, path, q_lens, kv_lens, G):
    g = torch.Generator().manual_seed(sum(q_lens))
    a = Arena()
    Hkv, page = 2, 16
    Hq, n = G * Hkv, sum(q_lens)
    q = a.inp(torch.randn(n, Hq, D, generator=g).bfloat16())
    pages = -(-max(kv_lens) // page) * 2
    cache = []
    scales = [None, None]
    for i in range(2):
        rows = torch.randn(pages, page, Hkv, D, generator=g)
        if quantised:
            c, s = quantise(rows)
            cache.append(a.inp(raw(c)).view(torch.float8_e4m3fn))
            scales[i] = a.inp(s.transpose(1, 2).contiguous())
        else:
            cache.append(a.inp(rows.bfloat16()))
    table = a.inp(torch.arange(pages, dtype=torch.int32).view(2, -1))
    cu, kv = a.inp(i32([0, q_lens[0], n])), a.inp(i32(kv_lens))
    mask = a.inp(signed([w for m in q_lens for w in tree_masks(g, m)[0]]))
    out = a.out((n, Hq, D), torch.bfloat16, float("nan"))
    ws = a.workspace(S.sd_paged_attention_workspace_size(n, 2, max(q_lens), Hq, Hkv, D, max(kv_lens)))
    S.sd_set_attention_path(path)
    if quantised:
        S.sd_paged_attention_e4m3(q, *cache, *scales, table, cu, kv, max(q_lens), max(kv_lens), out, 0.1, ws)
        assert S.sd_last_attention_path()[0] == path
        a.check()
        assert bool(torch.isfinite(out).all())
        out.fill_(float("nan"))
    S.sd_paged_tree_attention(q, *cache, table, mask, cu, kv, max(q_lens), max(kv_lens), out, 0.1, ws, *scales)
    assert S.sd_last_attention_path()[0] == path
    a.check()
    assert bool(torch.isfinite(out).all()) and S.sd_fault_word() == 0
