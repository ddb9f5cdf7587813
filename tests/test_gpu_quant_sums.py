"""Attention over 8-bit rows where many small weights add up: a key far above a long flat rest, and scores that fall."""
import pytest
import torch

from _quant_sums import FORMS, Sequence, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    sd_verify.sd_fault_word()
    return sd_verify


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m,sink,size", [(32768, 0, 0.1), (32768, 0, 1.0), (20001, 0, 0.0), (24000, 11111, 0.1), (20500, 20400, 1.0)])
@pytest.mark.parametrize("flat", [True, False])
def test_one_key_far_above_the_rest(S, form, D, m, sink, size, flat):
    """One key 9 to 14 nats (by query head and token) above the others, whose scores are equal or spread by a nat and
    whose values have a common mean; its own values smaller, as large, or zero."""
    n, G, tree = FORMS[form]
    g = torch.Generator().manual_seed(m + D)
    k = torch.zeros(m, 2, D) if flat else torch.randn(m, 2, D, generator=g)
    if not flat:
        k -= k.mean(-1, keepdim=True)          # (orthogonal to the queries' common part)
        k[:, :, 0] += torch.randn(m, 2, generator=g) * D ** 0.5
    v = 1 + 0.25 * torch.randn(m, 2, D, generator=g)
    k[sink] = 1.0
    v[sink] *= size
    nats = torch.linspace(9, 14, n * 2 * G).view(n, 2 * G, 1)
    q = (nats * D ** -0.5).expand(n, 2 * G, D).clone()
    if not flat:
        q[:, :, 0] += 1.0
    q = q.bfloat16()
    masks = [(1 << (i + 1)) - 1 for i in range(n)]
    seq = Sequence(S, k, v)
    check(seq.run(q, tree, masks=masks), seq.want(q, tree, masks=masks))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("step", [1e-3, 0.02, 0.4, -1e-3])
def test_scores_that_fall_or_rise(S, form, step):
    """Every key's score a little below the one before it: a row's unit follows them down and up again."""
    n, G, tree = FORMS[form]
    D, m = 128, 20000
    g = torch.Generator().manual_seed(n)
    x = -step * torch.arange(m, dtype=torch.float64) % 40       # (and starts again)
    k = (x / D ** 0.5).float()[:, None, None].expand(m, 2, D).clone()
    v = 1 + 0.25 * torch.randn(m, 2, D, generator=g)
    q = torch.ones(n, 2 * G, D).bfloat16()
    masks = [(1 << (i + 1)) - 1 for i in range(n)]
    seq = Sequence(S, k, v)
    check(seq.run(q, tree, masks=masks), seq.want(q, tree, masks=masks))


@pytest.mark.parametrize("form", FORMS)
def test_rows_of_zeros_before_the_others(S, form):
    """Values of zero take their weight whatever comes behind them, thousands of them or one far above the rest."""
    n, G, tree = FORMS[form]
    D, m = 128, 9000
    g = torch.Generator().manual_seed(n)
    k = torch.randn(m, 2, D, generator=g)
    v = 1 + 0.25 * torch.randn(m, 2, D, generator=g)
    q = torch.randn(n, 2 * G, D, generator=g).bfloat16()
    masks = [(1 << (i + 1)) - 1 for i in range(n)]
    for zeros in (slice(0, 5000), slice(7, 8), slice(64, 128), slice(1, m, 2)):
        w = v.clone()
        w[zeros] = 0
        seq = Sequence(S, k, w)
        check(seq.run(q, tree, masks=masks), seq.want(q, tree, masks=masks))


@pytest.mark.parametrize("n", [1, 4, 16])
@pytest.mark.parametrize("size", [0.1, 1.0])
def test_one_key_far_above_the_rest_in_a_batch(S, n, size):
    """300 sequences over the same pages, so that a CTA goes through all of a unit's keys by itself; tokens see all."""
    G, D, m, B = 7, 128, 32768, 300
    g = torch.Generator().manual_seed(n)
    k = torch.zeros(m, 1, D)
    v = 1 + 0.25 * torch.randn(m, 1, D, generator=g)
    k[0] = 1.0
    v[0] *= size
    q = (torch.linspace(9, 14, n * G).view(n, G, 1) * D ** -0.5).expand(n, G, D).bfloat16().contiguous()
    seq = Sequence(S, k, v, page=128)
    kp, vp, ks, vs = seq.cache
    out = torch.empty(B * n, G, D, dtype=torch.bfloat16, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(B * n, B, n, G, 1, D, m))
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    S.sd_paged_attention_e4m3(q.cuda().repeat(B, 1, 1), kp, vp, ks, vs, seq.table.repeat(B, 1), cu,
                              torch.full((B,), m, dtype=torch.int32, device="cuda"), n, m, out, D ** -0.5, ws, causal=False)
    torch.cuda.synchronize()
    assert S.sd_last_attention_path()[0] == 2 and S.sd_fault_word() == 0
    want = [x.repeat(20, 1, 1) if torch.is_tensor(x) else x for x in seq.want(q, False, causal=False)]
    for a in range(0, B * n, 20 * n):
        check(out[a:a + 20 * n], want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("max_kv", [1 << 16, (1 << 16) + 1, 1 << 20, 1 << 25])
def test_loose_bounds(S, form, max_kv):
    """The weights' unit grows with what the sequences may hold, from 2^16 keys on: the same bound."""
    n, G, tree = FORMS[form]
    D, m = 128, 3000
    g = torch.Generator().manual_seed(n)
    k = torch.randn(m, 2, D, generator=g)
    v = (1 + 0.25 * torch.randn(m, 2, D, generator=g)) * torch.exp(torch.randn(m, 2, 1, generator=g))
    q = 3 * torch.randn(n, 2 * G, D, generator=g).bfloat16()
    masks = [(1 << (i + 1)) - 1 for i in range(n)]
    seq = Sequence(S, k, v)
    check(seq.run(q, tree, masks=masks, max_kv=max_kv), seq.want(q, tree, masks=masks))
