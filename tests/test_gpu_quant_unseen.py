"""Attention over 8-bit rows: what a row does not see takes nothing from it, whatever its size."""
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
@pytest.mark.parametrize("m", [70, 200, 3000])
def test_rows_keep_their_bits_when_an_unseen_value_grows(S, form, D, m):
    """One new token's values 1 to 10^6 times the others': every token that does not see it has the same bits."""
    n, G, tree = FORMS[form]
    n = max(n, 4 if form == "few" else n)
    g = torch.Generator().manual_seed(m + D)
    k, v = torch.randn(m, 2, D, generator=g), torch.randn(m, 2, D, generator=g)
    q = torch.randn(n, 2 * G, D, generator=g).bfloat16()
    loud = n // 2                       # this new token's values
    masks = [1 << i | (1 if i != loud else 0) for i in range(n)]
    rows = [i for i in range(n) if i != loud] if tree else list(range(loud))
    outs = []
    for size in (1.0, 30.0, 1e3, 1e6):
        w = v.clone()
        w[m - n + loud] *= size
        seq = Sequence(S, k, w)
        outs.append(seq.run(q, tree, masks=masks))
        out, mag, big, rel = seq.want(q, tree, masks=masks)
        check(outs[-1][rows], (out[rows], mag[rows], big[rows], rel))
    for o in outs[1:]:
        assert torch.equal(o[rows], outs[0][rows])


@pytest.mark.parametrize("form", FORMS)
def test_a_loud_key_that_hardly_counts(S, form):
    """A seen key of large values and next to no weight: its values' size does not take the others' precision."""
    n, G, tree = FORMS[form]
    D, m = 128, 1500
    g = torch.Generator().manual_seed(n)
    k, v = torch.randn(m, 2, D, generator=g) * 0.3, torch.randn(m, 2, D, generator=g)
    q = torch.full((n, 2 * G, D), 1.0).bfloat16()
    k[5] = -4.0                         # 45 nats below the rest
    v[5] = 1e4 * torch.randn(2, D, generator=g)
    masks = [(1 << (i + 1)) - 1 for i in range(n)]
    seq = Sequence(S, k, v)
    check(seq.run(q, tree, masks=masks), seq.want(q, tree, masks=masks))
