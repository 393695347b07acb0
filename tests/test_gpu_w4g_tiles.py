"""Every kernel of the integer 4-bit projections over several tiles or items
per CTA, against a float64 evaluation on the device of all outputs; the
planner (tests/w4g_plan.py) says that the cases here and in test_gpu_w4g.py
run them all.  Tolerances as there."""
import shutil

import numpy as np
import pytest
import torch

import block_scaled_precision_requant_b200 as bsr
from tests.test_gpu_w4g import DENSE, DEV, GROUPED, SHARED_K, dev, make_acts, make_weight, offsets_of
from tests.w4g_plan import compile_planner, plans

pytestmark = pytest.mark.gpu

# rows, n, k, group: more tiles than SMs, the last ones ragged in rows, weight rows and (G < 128) K
DENSE_TILES = [
    # 192 rows per tile, up to four tiles per CTA
    (2523, 3001, 384, 128), (2516, 3001, 192, 64), (2519, 3001, 224, 32), (3900, 3001, 2080, 32),
    # 128
    (1355, 5003, 384, 128), (1351, 5003, 192, 64), (1358, 5003, 224, 32),
    # two CTAs along K of tiles of 128 and of 192 rows
    (385, 1501, 1152, 128), (387, 1501, 1088, 64), (261, 2003, 1056, 32),
    (585, 2003, 1152, 128), (582, 2003, 1088, 64), (588, 2003, 1056, 32),
]
# rows, experts, n, k, group
GROUPED_TILES = [
    # 192 rows per tile
    (3977, 8, 2003, 384, 128), (3914, 8, 2003, 192, 64), (3926, 8, 2003, 224, 32),
    # 128 and 64
    (1745, 8, 3001, 384, 128), (1788, 8, 3001, 192, 64), (1741, 8, 3001, 224, 32), (534, 8, 5003, 1056, 32),
    (395, 8, 3001, 384, 128), (397, 8, 3001, 192, 64),
    # so many experts that the stages are as few as they get
    (90869, 1024, 129, 384, 128), (83169, 1024, 129, 192, 64), (90877, 1024, 129, 224, 32),
    (41397, 1024, 129, 384, 128), (33661, 300, 129, 224, 32),
]
GROUPED_ITEMS = [
    # four, two and one tiles of 16 weight rows per item, several items per warp
    (201, 128, 3001, 384, 128), (210, 128, 3001, 192, 64), (384, 128, 1501, 2048, 64), (199, 128, 1501, 224, 32),
    (125, 128, 997, 1152, 128), (687, 128, 2003, 448, 64), (615, 128, 517, 1056, 32),
    # two activation tiles per item
    (1222, 128, 1501, 448, 64), (1076, 128, 200, 256, 128), (1044, 128, 1000, 256, 128), (1071, 128, 1000, 256, 32),
    (1144, 128, 200, 128, 64), (65, 8, 100, 1024, 32),
    # so many experts that the rings are as short as they get
    (1895, 1024, 333, 384, 128), (1955, 1024, 333, 192, 64), (2745, 1024, 129, 224, 32), (673, 1024, 129, 1152, 128),
]


def values(w):
    """float64 weight on the device."""
    q, s, z = w
    v = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).double()
    size = v.shape[-1] // s.shape[-1]
    z = 8.0 if z is None else z.double().repeat_interleave(size, dim=-1)
    return (v - z) * s.double().repeat_interleave(size, dim=-1)


def check(out, a, w, k, group, what):
    a, v = a.double(), values(w)
    ref, mag = a @ v.T, a.abs() @ v.abs().T
    tol = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * (group + k // group + 18) * 2.0 ** -23 * mag
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("zero,half", [(False, True), (True, False)])
@pytest.mark.parametrize("m,n,k,group", DENSE_TILES)
def test_dense_tiles(m, n, k, group, zero, half):
    w = dev(make_weight(m + n + k, (), n, k, group, zero, half))
    a = make_acts(n, m, k).to(DEV)
    guard = torch.full((m + 2, n), 7.0, device=DEV, dtype=torch.bfloat16)
    bsr.w4g_proj(a, *w, out=guard[1:-1])
    check(guard[1:-1], a, w, k, group, "")
    assert bool((guard[0] == 7.0).all()) and bool((guard[-1] == 7.0).all())
    assert torch.equal(bsr.w4g_proj(a, *w), guard[1:-1])
    assert bsr.device_status() == 0


def skewed_counts(seed, rows, experts):
    """Empty groups, single rows, popular experts; a tail behind the last group."""
    rng = np.random.default_rng(seed)
    share = np.exp(2.0 * rng.standard_normal(experts)) * (rng.random(experts) < 0.8)
    counts = rng.multinomial(rows - rows // 20, share / share.sum())
    return [int(c) for c in counts]


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = compile_planner(tmp_path_factory.mktemp("plan"))
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    return lambda cases: plans(exe, cases, sms)


@pytest.mark.parametrize("even", [False, True])
@pytest.mark.parametrize("r,experts,n,k,group", GROUPED_TILES + GROUPED_ITEMS)
def test_grouped_tiles(r, experts, n, k, group, even, planner):
    w = dev(make_weight(n + k, (experts,), n, k, group, not even, even))
    counts = [r // experts] * (experts - 1) + [r - r // experts * (experts - 1)] if even else \
        skewed_counts(r, r, experts)
    off = offsets_of(counts).to(DEV)
    a = make_acts(k, 301, k).to(DEV)
    rows = torch.randint(0, 301, (r,), generator=torch.Generator().manual_seed(r), dtype=torch.int32).to(DEV)
    out = torch.full((r, n), 7.0, device=DEV, dtype=torch.bfloat16)
    bsr.w4g_proj_grouped(a, off, *w, rows=rows, out=out)
    x = a[rows.long()]
    ordered = torch.full((r, n), 7.0, device=DEV, dtype=torch.bfloat16)
    bsr.w4g_proj_grouped(x, off, *w, out=ordered)
    for got, what in ((out, "with a row index"), (ordered, "in order")):
        at = 0
        for e, c in enumerate(counts):
            if c:
                check(got[at:at + c], x[at:at + c], tuple(None if t is None else t[e] for t in w), k, group, (what, e))
                at += c
        assert bool((got[at:] == 7.0).all())
    # a row index costs the tensor-core kernel a copy of the rows, so that the
    # call without one may take it where the other does not
    one, two = planner([(r, n, k, group, experts, True, indexed) for indexed in (True, False)])
    assert one.few >= two.few
    if one == two:
        assert torch.equal(out, ordered)
    assert bsr.device_status() == 0


def test_the_cases_run_every_kernel(planner):
    """The decode kernel by group, tiles per item and activation tiles, the
    tensor-core kernel by group and rows per tile with more tiles than CTAs,
    and by CTAs along K."""
    cases = [(m, n, k, g, 1, False, False) for m, n, k, g in DENSE + SHARED_K + DENSE_TILES]
    grouped = [(sum(c), len(c), n, k, g) for c, n, k, g in GROUPED] + GROUPED_TILES + GROUPED_ITEMS
    cases += [(r, n, k, g, e, True, True) for r, e, n, k, g in grouped]
    decode, several_items, tiles, several_tiles, shared = set(), set(), set(), set(), set()
    for (r, n, k, g, e, is_grouped, _), p in zip(cases, planner(cases)):
        if p.few:
            kernel = (g, p.rt, p.nt)
            decode.add(kernel)
            used = e * (1 - (1 - 1 / e) ** r)
            if used * -(-n // (16 * p.rt)) > p.gemv_grid * (16 // p.ks):
                several_items.add(kernel)
        elif p.split > 1:
            shared.add((p.bm, p.split))
        else:
            tiles.add((g, p.bm))
            if r / p.bm * -(-n // 128) > 1.5 * p.gemm_grid:
                several_tiles.add((g, p.bm))
    every = {(g, rt, nt) for g in (64, 128) for rt, nt in ((1, 1), (2, 1), (4, 1), (1, 2), (2, 2))}
    every |= {(32, rt, nt) for rt in (1, 2) for nt in (1, 2)}
    assert decode == every, every - decode
    assert several_items >= {(64, 4, 1), (128, 4, 1), (32, 2, 1), (64, 2, 1), (128, 2, 1)}, several_items
    assert tiles == {(g, bm) for g in (32, 64, 128) for bm in (32, 64, 128, 192)}, tiles
    assert several_tiles >= {(g, bm) for g in (32, 64, 128) for bm in (128, 192)}, several_tiles
    assert shared >= {(32, 2), (32, 4), (64, 2), (128, 2), (192, 2)}, shared
