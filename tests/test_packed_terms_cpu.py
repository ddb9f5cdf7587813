"""The bound that the GPU tests put on two-term weights tells them from what it is there to catch."""
import pytest
import torch

from _packed import rounded, two_term_bound
from test_gpu_paged import randn, ref_attend


@pytest.mark.parametrize("n,m,Hq,Hkv,D", [(1, 40, 8, 2, 64), (16, 130, 7, 1, 128), (2, 700, 4, 4, 64), (16, 900, 28, 4, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_the_bound_holds_for_two_terms_and_for_nothing_less(n, m, Hq, Hkv, D, causal):
    g = torch.Generator().manual_seed(m)
    q, k, v = (randn(g, r, h, D, dtype=torch.bfloat16) for r, h in ((n, Hq), (m, Hkv), (m, Hkv)))
    want, mag, _, rel = ref_attend(q, k, v, 1 / D, causal)
    tol = two_term_bound(want, mag, rel, torch.bfloat16)
    over = lambda *a: float(((rounded(q, k, v, 1 / D, causal, *a).double() - want).abs() > tol).double().mean())
    assert over(2) == 0.0
    # no second term, and one that belongs to the next key or to one 8 keys on
    for planted in ((1,), (2, 1), (2, 8)):
        assert over(*planted) > 0.01, planted
