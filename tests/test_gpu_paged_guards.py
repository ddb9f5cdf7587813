"""Guards of the paged-cache calls that well-formed input never meets: packed
offsets that are none, against the reading the header gives them."""
import pytest
import torch

from test_gpu_paged import BAD_LENGTH, Pool, S, _clean, check_rope, randn, rope_ref  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# --------------------------------------------------------------------------
# the append
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("N,cu,kv,tokens", [
    # `tokens`: first row, rows and first cache position of each sequence, offsets clamped to [0, N]
    (8, [0, 50], [60], [(0, 8, 52)]),                              # past N
    (8, [0, 4, 100], [20, 200], [(0, 4, 16), (4, 4, 196)]),
    (8, [-3, 5], [20], [(0, 5, 15)]), (5, [-3, 5], [20], [(0, 5, 15)]),      # negative
    (25, [0, 30, 21], [40, 50], [(0, 25, 15)]),                    # past N, then decreasing
    (8, [0, 8, 4], [30, 30], [(0, 8, 22)]),                        # decreasing where no token looks
])
def test_append_clamps_offsets_and_reports_them(S, dtype, positions, N, cu, kv, tokens):
    g = torch.Generator().manual_seed(N + len(cu))
    Hq, Hkv, D, page, R = 3, 2, 64, 16, 64
    pool = Pool(g, [208] * len(kv), page, Hkv, D, dtype, fill=0.25)
    kp, vp, table = pool.cuda()
    x = randn(g, N, Hq + 2 * Hkv, D, dtype=dtype)
    dev = x.cuda()
    turns = S.sd_rotary_table(R, 1e4)[0].cuda()
    pos = torch.arange(N, dtype=torch.int32) * 5 + 3
    qo = torch.full((N, Hq, D), 9.0, dtype=dtype, device="cuda")
    S.sd_rotary_append_paged(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], qo, pos.cuda() if positions else None,
                             turns, i32(*cu), i32(*kv), table, kp, vp)
    torch.cuda.synchronize()
    assert S.sd_fault_word() == BAD_LENGTH
    kc, vc, qc = kp.cpu(), vp.cpu(), qo.cpu()
    kept = torch.ones(kc.shape[:2], dtype=torch.bool)
    mine = torch.zeros(N, dtype=torch.bool)
    for b, (row, n, first) in enumerate(tokens):
        rows, at = slice(row, row + n), torch.arange(first, first + n)
        pg, sl = pool.table[b, at // page].long(), at % page
        kept[pg, sl] = False
        mine[rows] = True
        turn = pos[rows] if positions else at
        check_rope(kc[pg, sl], *rope_ref(x[rows, Hq:Hq + Hkv], turn, R, 1e4, "half"), dtype)
        assert torch.equal(vc[pg, sl], x[rows, Hq + Hkv:])
        if cu[-1] >= N or row + n <= cu[-1]:       # queries behind cu_q[B] stay
            check_rope(qc[rows], *rope_ref(x[rows, :Hq], turn, R, 1e4, "half"), dtype)
    assert bool((kc[kept] == 0.25).all()) and bool((vc[kept] == 0.25).all())
    assert bool((qc[~mine] == 9.0).all())


def test_append_reports_lengths_of_idle_sequences(S):
    """Each sequence's length is looked over, by itself and among hundreds, its tokens present or not."""
    g = torch.Generator().manual_seed(1)
    for B in (1, 3, 129, 700):
        pool = Pool(g, [16] * B, 16, 1, 64, torch.bfloat16, fill=0.25)
        kp, vp, table = pool.cuda()
        table.clamp_(min=0)
        x = randn(g, 1, 1, 64, dtype=torch.bfloat16).cuda()
        turns = S.sd_rotary_table(64, 1e4)[0].cuda()
        cu = torch.zeros(B + 1, dtype=torch.int32)
        cu[-1] = 1                                 # the last sequence's one token
        for bad in (None, -1, 33):                 # two pages of 16 in the table
            for at in {0, B // 2, B - 1}:
                kv = torch.full((B,), 16, dtype=torch.int32)
                if bad is not None:
                    kv[at] = bad
                S.sd_rotary_append_paged(None, x, x, None, None, turns, cu.cuda(), kv.cuda(), table, kp, vp)
                torch.cuda.synchronize()
                assert S.sd_fault_word() == (0 if bad is None else BAD_LENGTH)


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, 2), (torch.bfloat16, 1), (torch.float32, 1)])
def test_overlapping_sequences_past_the_work_line_are_refused(S, dtype, path):
    """64 sequences, every other one all of 32,768 rows over 40,000 keys: far more work than a call's
    line holds, and what 32 bits leave of its sum is not.  Nothing is computed; the next call on the
    same workspace is exact."""
    N, B, Hq, Hkv, D, page = 32768, 64, 64, 8, 64, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(N, Hq, D, generator=g, device="cuda").to(dtype)
    kp, vp = (torch.randn(8, page, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    table = torch.arange(B * 625, device="cuda").remainder(8).to(torch.int32).view(B, 625)
    out = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
    ws = S.workspace(S.sd_paged_attention_workspace_size(N, B, N, Hq, Hkv, D, 40000, S._dt(q)))
    S.sd_set_attention_path(path)
    args = (N, 40000, out, D ** -0.5, ws)
    small = i32(*([0, 3] + [3] * (B - 2) + [10])), torch.full((B,), 300, dtype=torch.int32, device="cuda")
    S.sd_paged_attention(q, kp, vp, table, *small, *args)
    torch.cuda.synchronize()
    good = out[:10].clone()
    assert S.sd_fault_word() == 0 and not bool((good == 7.0).all())
    out.fill_(7.0)
    for causal in (False, True):
        S.sd_paged_attention(q, kp, vp, table, i32(*([0, N] * (B // 2) + [0])),
                             torch.full((B,), 40000, dtype=torch.int32, device="cuda"), *args, causal=causal)
        torch.cuda.synchronize()
        assert S.sd_fault_word() == BAD_LENGTH
        assert bool((out == 7.0).all())
    S.sd_paged_attention(q, kp, vp, table, *small, *args)
    torch.cuda.synchronize()
    assert S.sd_fault_word() == 0 and torch.equal(out[:10], good)


def counters(S, ws):
    """The counters of a call's whole grid, which it leaves at zero."""
    n = S.sd_last_attention_path()[1]
    assert 1 <= n <= 1024
    return ws[256:256 + 4 * n].view(torch.int32)


@pytest.mark.parametrize("D", [64, 128])
def test_calls_of_different_grids_share_a_workspace(S, D):
    """One CTA, a few, and as many as there are, on both paths and in both types, one after the other on
    one workspace: each as on a workspace of its own, with every counter of its grid back at zero."""
    g = torch.Generator(device="cuda").manual_seed(D)
    Hq, Hkv, page = 8, 2, 16
    shapes = [([1], [1]), ([40, 3], [300, 20]), ([1, 16, 700, 2], [9000, 3000, 2000, 40]), ([2], [60]), ([1] * 90, [500] * 90)]
    size = max(S.sd_paged_attention_workspace_size(sum(a), len(a), max(a), Hq, Hkv, D, max(b), t)
               for a, b in shapes for t in (S.SD_BF16, S.SD_FP32))
    shared = S.workspace(size)
    calls = []
    for dtype, path in ((torch.bfloat16, 2), (torch.bfloat16, 1), (torch.float32, 1)):
        for q_lens, kv_lens in shapes:
            n, B, cols = sum(q_lens), len(q_lens), -(-max(kv_lens) // page)
            kp, vp = (torch.randn(cols + 5, page, Hkv, D, generator=g, device="cuda").to(dtype) for _ in range(2))
            table = (torch.arange(B * cols, device="cuda") * 7).remainder(cols + 5).to(torch.int32).view(B, cols)
            q = torch.randn(n, Hq, D, generator=g, device="cuda").to(dtype)
            out = torch.empty_like(q)
            cu = torch.tensor([0] + q_lens).cumsum(0).to(torch.int32).cuda()
            args = (q, kp, vp, table, cu, i32(*kv_lens), max(q_lens), max(kv_lens), out, D ** -0.5)
            own = S.workspace(size)
            S.sd_set_attention_path(path)
            S.sd_paged_attention(*args, own)
            torch.cuda.synchronize()
            assert not counters(S, own).any()
            calls.append((path, args, out.clone()))
    grids = set()
    for path, args, want in calls + calls[::-1]:
        S.sd_set_attention_path(path)
        args[8].fill_(0)
        S.sd_paged_attention(*args, shared)
        torch.cuda.synchronize()
        grids.add(S.sd_last_attention_path()[1])
        assert torch.equal(args[8], want)
        assert not shared[256:256 + 4 * 1024].any()
    assert S.sd_fault_word() == 0 and min(grids) < 10 and max(grids) > 152
