"""How packed attention divides its work, run on the host: packed_plan.cpp takes
the plan from the kernels' own header, a warp's lanes as coroutines, and checks
that every tile of every unit is dealt out exactly once and that the CTAs of a
shared unit agree about it."""
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "serving_sd_verify_gb300", "csrc")
BAD_LENGTH = 1 << 7


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "packed_plan")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    # (longjmp between the lanes' stacks is what the fortified one refuses)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-U_FORTIFY_SOURCE", "-I", CSRC, "-I", os.path.join(cuda, "include"),
                        os.path.join(HERE, "packed_plan.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(batches):
        r = subprocess.run([exe], input="\n".join(batches), capture_output=True, text=True, timeout=300)
        lines = r.stdout.splitlines()
        assert r.returncode == 0 and len(lines) == len(batches), (r.returncode, r.stderr, lines)
        keys = ("fault", "total", "shift", "active", "parts", "most")
        return [dict(zip(keys, map(int, x.split()[:6])), what=x.split(None, 6)[6]) for x in lines]
    return run


def batch(cu, kv, Hkv=8, G=8, tensor=1, causal=0, max_q=None, max_kv=None, slots=1 << 26, N=None, grid=0, rows=0,
          shift=-1):
    """One batch as packed_plan.cpp reads it; kv None: prompts."""
    N = cu[-1] if N is None else N
    max_q = max(b - a for a, b in zip(cu, cu[1:])) if max_q is None else max_q
    max_kv = max(kv or [max_q]) if max_kv is None else max_kv
    head = [len(cu) - 1, Hkv, G, tensor, causal, int(kv is None), N, max_q, max_kv, slots, grid, rows, shift]
    return " ".join(map(str, [*head, *cu, *(kv or [])]))


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("tensor", [0, 1])
@pytest.mark.parametrize("B", [20, 32, 33, 64, 1024, 2500])
def test_sequences_that_overlap_past_the_line_are_refused(replay, B, tensor):
    """Every other sequence is the whole of 32,768 rows: the line is far past 32 bits, and what is
    left of its sum is not.  All of it is refused, and said so, whatever the batch's size."""
    N = 32768
    cu = [0 if b % 2 == 0 else N for b in range(B + 1)]
    for causal in (0, 1):
        r, = replay([batch(cu, [40000] * B, tensor=tensor, causal=causal, max_q=N)])
        assert r["fault"] == BAD_LENGTH and r["total"] == 0 and r["active"] == 0, r


def test_the_longest_lines_are_dealt_out(replay):
    cases = []
    for grid in (0, 1, 2, 5, 18, 43):
        cases.append(batch([0, 32768], [260000], causal=1, max_kv=1 << 25, grid=grid))               # a loose bound
        cases.append(batch([0, 15], [1 << 26], Hkv=4, G=1, grid=grid))
        cases.append(batch(offsets([15] * 7), [1 << 26] * 7, Hkv=4, G=1, grid=grid))                 # 1.88e9 keys
        cases.append(batch(offsets([1] * 70), [3900000 + b for b in range(70)], Hkv=7, G=4, grid=grid))
    for r in replay(cases):
        assert r["what"] == "ok" and r["fault"] == 0, r
    assert replay(cases[:1])[0]["shift"] == 8 and replay(cases[2:3])[0]["total"] > 1.8e9


@pytest.mark.parametrize("seed", range(4))
def test_random_batches_are_dealt_out_exactly(replay, seed):
    rng = random.Random(seed)
    cases = []
    for i in range(40):
        tensor = rng.randrange(2)
        B = rng.choice([1, 1, 2, 12, 32, 33, 40, 200, 1500])
        top = rng.choice([1, 3, 16, 600] if B > 40 else [1, 3, 16, 600, 5000])
        q = [0 if rng.random() < 0.1 else rng.randint(1, top) for _ in range(B)]
        kv = None if rng.random() < 0.3 else \
            [rng.randint(0, 500) if rng.random() < 0.05 else a + rng.choice([0, rng.randint(0, 300), rng.randint(0, 40000)])
             for a in q]
        if not sum(q):
            q[-1] = 1
        cases.append(batch(offsets(q), kv, Hkv=rng.randint(1, 8), G=rng.choice([1, 2, 3, 4, 7, 8, 16]), tensor=tensor,
                           causal=int(rng.random() < 0.75), N=sum(q) + rng.randint(0, 3),
                           grid=rng.choice([0, 0, 0, rng.randint(1, 20)]),
                           max_kv=None if kv is None else rng.choice([max(kv), 1 << 26]),
                           shift=rng.choice([-1, -1, rng.randint(1, 8 if tensor else 6)])))
    for c, r in zip(cases, replay(cases)):
        assert r["what"] in ("ok", "refused") and r["fault"] == 0, (r, c[:120])


@pytest.mark.parametrize("D", [64, 128])
def test_the_counters_room_is_the_same_for_every_grid(D):
    """A workspace holds 1,024 counters in front of the partials, whatever the call's grid: the rest of a
    large call's is whole pairs of slots, 256 rows of D + 2 floats each (or four of 64)."""
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    size = sd_verify.sd_paged_attention_workspace_size(4096, 64, 4096, 28, 4, D, 65536)
    assert (size - 256 - 4 * 1024) % (2 * 256 * (D + 2) * 4) == 0
