"""Forms of packed attention that its other tests do not tell apart or do not
reach: the one-tile form's two-term weights, units finished by exactly two
CTAs whose wait gives up, and work lines counted in more than one key."""
import math

import pytest
import torch

from _packed import two_term_bound
from test_gpu_paged import (HEADS, WAIT_GAVE_UP, Pool, S, _clean, check, cumulative, dt_code, randn,  # noqa: F401
                            ref_attend)
from test_packed_plan_cpu import batch, offsets, replay  # noqa: F401

pytestmark = pytest.mark.gpu


def paged(S, q_lens, kv_lens, Hq, Hkv, D, dtype, page, scale, seed, max_q=None, max_kv=None):
    """(arguments of a call, rows' queries, keys and values per sequence)"""
    g = torch.Generator().manual_seed(seed)
    n = sum(q_lens)
    q = randn(g, n, Hq, D, dtype=dtype)
    pool = Pool(g, kv_lens, page, Hkv, D, dtype)
    seqs, at = [], 0
    for b, (a, m) in enumerate(zip(q_lens, kv_lens)):
        k, v = randn(g, m, Hkv, D, dtype=dtype), randn(g, m, Hkv, D, dtype=dtype)
        pool.write(b, k, v)
        seqs.append((slice(at, at + a), q[at:at + a], k, v))
        at += a
    max_q, max_kv = max_q or max(q_lens), max_kv or max(kv_lens)
    ws = S.workspace(S.sd_paged_attention_workspace_size(n, len(q_lens), max_q, Hq, Hkv, D, max_kv, dt_code(S, dtype)))
    out = torch.full((n, Hq, D), 123.0, dtype=dtype, device="cuda")
    kp, vp, table = pool.cuda()
    return (q.cuda(), kp, vp, table, cumulative(q_lens).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(), max_q,
            max_kv, out, scale, ws), seqs


def two_terms(out, want, mag, _, rel):
    assert bool(((out.cpu().double() - want).abs() <= two_term_bound(want, mag, rel, torch.bfloat16)).all())


# --------------------------------------------------------------------------
# two-term weights
# --------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_one_tile_units_over_pages_have_two_term_weights(S, Hq, Hkv, D, page, causal):
    T = min(16, 128 // (Hq // Hkv))
    q_lens, kv_lens = [T, 1, 0, T, 1], [T, 40, 9, 131, 700]
    args, seqs = paged(S, q_lens, kv_lens, Hq, Hkv, D, torch.bfloat16, page, 1 / D, seed=page)
    S.sd_set_attention_path(2)
    S.sd_paged_attention(*args, causal=causal)
    torch.cuda.synchronize()
    assert S.sd_last_attention_path()[0] == 2 and S.sd_fault_word() == 0
    for rows, q, k, v in seqs:
        if len(q):
            two_terms(args[8][rows], *ref_attend(q, k, v, 1 / D, causal))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_one_tile_prompts_have_two_term_weights(S, Hq, Hkv, D, causal):
    top = 128 // (Hq // Hkv)
    lens = [min(top, n) for n in (40, 1, 128, 17)]
    g = torch.Generator().manual_seed(D)
    x = randn(g, sum(lens), Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    dev, out = x.cuda(), torch.empty(sum(lens), Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(sum(lens), 4, top, Hq, Hkv, D, top))
    S.sd_set_attention_path(2)
    S.sd_prompt_attention(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], cumulative(lens).cuda(), top, out, 1 / D,
                          ws, causal=causal)
    torch.cuda.synchronize()
    at = 0
    for n in lens:
        r = x[at:at + n]
        two_terms(out[at:at + n], *ref_attend(r[:, :Hq], r[:, Hq:Hq + Hkv], r[:, Hq + Hkv:], 1 / D, causal))
        at += n
    assert S.sd_fault_word() == 0


@pytest.mark.parametrize("page", [8, 16, 64])
def test_shared_units_have_two_term_weights(S, page):
    args, seqs = paged(S, [1, 16, 1], [9000, 6000, 300], 28, 4, 128, torch.bfloat16, page, 1 / 128, seed=page)
    S.sd_set_attention_path(2)
    S.sd_paged_attention(*args)
    torch.cuda.synchronize()
    for rows, q, k, v in seqs:
        two_terms(args[8][rows], *ref_attend(q, k, v, 1 / 128, True))
    assert S.sd_fault_word() == 0


# --------------------------------------------------------------------------
# units of two CTAs
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, 2), (torch.bfloat16, 1), (torch.float32, 1)])
@pytest.mark.parametrize("q_lens,kv_lens", [([16], [700]), ([18, 18], [700, 700]), ([300, 150], [700, 400])])
def test_a_unit_of_two_ctas_gives_up_then_recovers(S, replay, dtype, path, q_lens, kv_lens):
    """The CTA that opens such a unit waits for the other's part and joins it itself, on the tensor cores,
    with a counter protocol of its own; the batches are those whose shared units all have two."""
    Hq, Hkv, D = 28, 4, 128
    args, seqs = paged(S, q_lens, kv_lens, Hq, Hkv, D, dtype, 64, 1 / math.sqrt(D), seed=4)
    out, ws = args[8], args[10]
    S.sd_set_attention_path(path)
    S.sd_paged_attention(*args)
    torch.cuda.synchronize()
    grid = S.sd_last_attention_path()[1]
    if path == 2:
        plan, = replay([batch(offsets(q_lens), kv_lens, Hkv=Hkv, G=Hq // Hkv, tensor=1, causal=1, grid=grid)])
        assert plan["what"] == "ok" and plan["most"] == 2, plan
    good = out.clone()
    for rows, q, k, v in seqs:
        check(good[rows], *ref_attend(q, k, v, 1 / math.sqrt(D), True), dtype, path == 2)
    for _ in range(2):
        S.sd_set_wait_test(1, 1_000_000)
        S.sd_paged_attention(*args)
        torch.cuda.synchronize()
        S.sd_set_wait_test(0, 0)
        assert S.sd_fault_word() & WAIT_GAVE_UP
        assert not ws[256:256 + 4 * grid].any()
        out.fill_(0)
        S.sd_paged_attention(*args)
        torch.cuda.synchronize()
        assert S.sd_fault_word() == 0 and torch.equal(out, good)


# --------------------------------------------------------------------------
# work lines counted in more than one key
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, 2), (torch.bfloat16, 1), (torch.float32, 1)])
@pytest.mark.parametrize("q_lens,kv_lens,max_q,causal", [
    ([1, 16, 2, 0], [3000, 700, 1, 5], 16, True),
    ([40, 300, 1, 0, 7], [40, 2000, 3000, 0, 9], 348, True),
    ([1] * 40, [100 * i for i in range(40)], 1, True),
    ([130, 64], [900, 64], 194, False)])
def test_loose_bounds_shift_the_work_line(S, replay, dtype, path, q_lens, kv_lens, max_q, causal):
    """max_kv as loose as it may be: lines of 2e9 to 2e10 keys in the host's eyes.  The plan of each is
    first replayed on the host."""
    Hq, Hkv, D = 32, 8, 128
    plan, = replay([batch(offsets(q_lens), kv_lens, Hkv=Hkv, G=Hq // Hkv, tensor=int(path == 2), causal=int(causal),
                          max_q=max_q, max_kv=1 << 26)])
    assert plan["what"] == "ok" and plan["fault"] == 0 and plan["shift"] >= 1, plan
    args, seqs = paged(S, q_lens, kv_lens, Hq, Hkv, D, dtype, 16, 1 / math.sqrt(D), seed=5, max_q=max_q, max_kv=1 << 26)
    S.sd_set_attention_path(path)
    S.sd_paged_attention(*args, causal=causal)
    torch.cuda.synchronize()
    used, grid = S.sd_last_attention_path()
    assert S.sd_fault_word() == 0 and used == path and not args[10][256:256 + 4 * grid].any()
    for rows, q, k, v in seqs:
        if len(q):
            check(args[8][rows], *ref_attend(q, k, v, 1 / math.sqrt(D), causal), dtype, path == 2)
