"""What the integer 4-bit projections' plan chooses, over random sizes: only
kernels that exist, all of them, within their limits."""
import math
import random
import shutil

import pytest

from tests.w4g_plan import compile_planner, plans

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return compile_planner(tmp_path_factory.mktemp("plan"))


def log_int(rng, lo, hi):
    return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def random_cases(count):
    rng = random.Random(7)
    for _ in range(count):
        group = rng.choice([32, 64, 128])
        experts = rng.choice([1, 1, rng.randint(2, 1024)])
        rows = log_int(rng, 1, 40 * experts if rng.random() < 0.7 else 100000)
        grouped = experts > 1 or rng.random() < 0.2
        yield (rows, log_int(rng, 1, 40000), group * log_int(rng, 1, 40000 // group), group, experts, grouped,
               grouped and rng.random() < 0.5)


def test_every_kernel_is_reached_and_no_other(exe):
    cases = list(random_cases(40000))
    decode, tiles = set(), set()
    for (rows, n, k, group, experts, grouped, indexed), p in zip(cases, plans(exe, cases)):
        if p.few:
            assert rows <= 16 * experts and rows <= max(4096, 4 * experts)
            assert p.ks in (1, 2, 4, 8) and p.ks * 2 <= max(2, -(-k // 256))
            assert 3 <= p.slots <= 6 and 1 <= p.gemv_grid <= 148
            decode.add((group, p.rt, p.nt))
        else:
            assert rows > 4 * experts and 1 <= p.gemm_grid <= 148 and p.split == 1
            tiles.add((group, p.bm))
    want = {(g, rt, nt) for g in (64, 128) for rt, nt in ((1, 1), (2, 1), (4, 1), (1, 2), (2, 2))}
    want |= {(32, rt, nt) for rt in (1, 2) for nt in (1, 2)}
    assert decode == want
    assert tiles == {(g, bm) for g in (32, 64, 128) for bm in (32, 64, 128, 192)}


def test_the_decode_kernel_sums_in_an_order_of_k_alone(exe):
    """The warps along K depend on neither the rows, the weight rows nor the
    experts."""
    rng = random.Random(3)
    for k in (32, 512, 1024, 2048, 4096, 14336):
        cases = [(rng.randint(1, 4), log_int(rng, 1, 20000), k, 32, 1, False, False) for _ in range(50)]
        cases += [(rng.randint(1, 64), log_int(rng, 1, 4000), k, 32, rng.randint(16, 512), True, True)
                  for _ in range(50)]
        assert len({p.ks for p in plans(exe, cases)}) == 1
