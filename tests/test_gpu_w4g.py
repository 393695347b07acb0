"""Integer 4-bit projections (dense and grouped by expert) against the
float64 oracle.

Tolerance, per output: the result is rounded once to BF16 (at most 2^-8 of the
value) from float32 sums of exact products.  A group's sum has G terms and an
output adds K/G scaled groups plus at most 16 partial sums of warps or CTAs; each
addition is off by at most 2^-23 (a tensor-core addition may truncate) and
each scaling by 2^-24 of the sum of magnitudes S, hence
|err| <= 2^-8 |ref| + (1 + 2^-8) (G + K/G + 18) 2^-23 S."""
import numpy as np
import pytest
import torch

import block_scaled_precision_requant_b200 as bsr
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make_weight(seed, lead, n, k, group, zero=False, half=False):
    g = torch.Generator().manual_seed(seed)
    shape = tuple(lead) + (n, k // group)
    q = torch.randint(0, 256, tuple(lead) + (n, k // 2), dtype=torch.uint8, generator=g)
    s = ((torch.rand(shape, generator=g) + 0.1) * 0.02 * torch.where(torch.rand(shape, generator=g) < 0.1, -1.0, 1.0))
    z = torch.randint(0, 16, shape, dtype=torch.uint8, generator=g) if zero else None
    return q, s.to(torch.float16 if half else torch.bfloat16), z


def make_acts(seed, m, k):
    return torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).bfloat16()


def dev(w):
    return tuple(None if t is None else t.to(DEV) for t in w)


def reference(a, w):
    q, s, z = w
    return oracle.w4g_proj(a.double().numpy(), q.numpy(), s.double().numpy(), None if z is None else z.numpy())


def check(out, ref, mag, k, group, what=""):
    got = out.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (group + k // group + 18) * 2.0 ** -23 * mag
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:5].tolist())


DENSE = [
    # one token: odd rows, one group per row, several groups, long K
    (1, 1, 32, 32), (1, 5, 64, 64), (1, 130, 128, 128), (1, 4096, 4096, 128), (1, 77, 14336, 64), (1, 33, 96, 32),
    # a few tokens around the token tiles
    (2, 257, 1024, 128), (7, 100, 640, 128), (8, 513, 2048, 64), (9, 48, 4160, 32), (15, 31, 512, 64),
    (16, 1000, 1152, 128), (17, 129, 384, 128), (31, 200, 2080, 32), (33, 300, 576, 64),
    # prompts: ragged tiles in every direction
    (64, 128, 256, 64), (127, 127, 128, 128), (129, 385, 1056, 32), (200, 1, 192, 64), (300, 1000, 4096, 128),
    (513, 260, 320, 64), (1000, 17, 32, 32),
]


@pytest.mark.parametrize("zero,half", [(False, False), (True, True)])
@pytest.mark.parametrize("m,n,k,group", DENSE)
def test_dense(m, n, k, group, zero, half):
    w = make_weight(m + n + k, (), n, k, group, zero, half)
    a = make_acts(n, m, k)
    out = bsr.w4g_proj(a.to(DEV), *dev(w))
    ref, mag = reference(a, w)
    check(out, ref, mag, k, group)
    assert bsr.device_status() == 0


def offsets_of(counts):
    return torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32)


GROUPED = [
    ([1], 40, 64, 32), ([0, 1, 0], 33, 128, 128), ([1] * 8, 130, 512, 64), ([3, 0, 0, 9, 1, 8, 17, 0], 257, 640, 128),
    ([0] * 63 + [2], 100, 256, 64), ([20, 1, 33, 0, 64, 65], 129, 192, 64), ([300, 0, 129, 7, 128], 200, 1152, 128),
    ([1000, 1], 65, 96, 32), ([5] * 200, 24, 160, 32), ([40] * 16, 384, 1024, 128), ([200, 190, 1, 0], 500, 2080, 32),
]


def grouped_reference(a, counts, w, rows):
    q, s, z = w
    refs, mags, at = [], [], 0
    src = a.double().numpy()
    for e, c in enumerate(counts):
        x = np.zeros((c, a.shape[1]))
        for i in range(c):
            r = int(rows[at + i])
            if 0 <= r < a.shape[0]:
                x[i] = src[r]
        ref, mag = oracle.w4g_proj(x, q[e].numpy(), s[e].double().numpy(), None if z is None else z[e].numpy())
        refs.append(ref)
        mags.append(mag)
        at += c
    return np.concatenate(refs), np.concatenate(mags)


@pytest.mark.parametrize("zero,half", [(True, False), (False, True)])
@pytest.mark.parametrize("counts,n,k,group", GROUPED)
def test_grouped(counts, n, k, group, zero, half):
    r = sum(counts)
    w = make_weight(n + k, (len(counts),), n, k, group, zero, half)
    a = make_acts(k, max(3, r // 2), k)
    rows = torch.randint(0, a.shape[0], (r,), generator=torch.Generator().manual_seed(r), dtype=torch.int32)
    ref, mag = grouped_reference(a, counts, w, rows.numpy())
    out = bsr.w4g_proj_grouped(a.to(DEV), offsets_of(counts).to(DEV), *dev(w), rows=rows.to(DEV))
    check(out, ref, mag, k, group, "indexed rows")
    # without an index: the rows already in order, the same bits
    ordered = a[rows.long()].to(DEV)
    again = bsr.w4g_proj_grouped(ordered, offsets_of(counts).to(DEV), *dev(w))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert bsr.device_status() == 0


@pytest.mark.parametrize("scale", [1, 40])
def test_rows_past_the_groups_are_left(scale):
    """Rows of `out` past the last group keep what they held; a row index
    outside `a` stands for zeros; late offsets are clamped to R."""
    counts = [3 * scale, 0, 5 * scale]
    used, n, k = sum(counts), 70, 128
    r = used + 9 * scale
    w = make_weight(5, (3,), n, k, 64, True)
    a = make_acts(6, 11, k)
    rows = torch.randint(0, 11, (r,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    rows[1], rows[used - 1] = -1, 11
    ref, mag = grouped_reference(a, counts, w, rows.numpy())
    out = torch.full((r, n), 7.0, dtype=torch.bfloat16, device=DEV)
    bsr.w4g_proj_grouped(a.to(DEV), offsets_of(counts).to(DEV), *dev(w), rows=rows.to(DEV), out=out)
    check(out[:used], ref, mag, k, 64)
    assert bool((out[used:] == 7.0).all())
    assert bool((out[1] == 0).all()) and bool((out[used - 1] == 0).all())
    wild = torch.tensor([0, counts[0], counts[0] - 2, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    bsr.w4g_proj_grouped(a.to(DEV), wild, *dev(w), rows=rows.to(DEV), out=out)
    ref, mag = grouped_reference(a, [counts[0], 0, r - counts[0]], w, rows.numpy())
    check(out, ref, mag, k, 64, "clamped offsets")
    assert bsr.device_status() == 0


@pytest.mark.parametrize("raw", [[0, 120, 200, 150], [7, 90, 40, -3], [0, 200, 2 ** 31 - 1, 0], [-5, -1, 30, 30],
                                 [0, 0, 0, -1]])
@pytest.mark.parametrize("rows_max", [12, 200])
def test_offsets_that_fall_are_clamped_with_a_row_index(raw, rows_max):
    """An offset below the one before it stands for the one before, the last
    one too, on the decode kernel and past it: the rows that the clamped groups
    have are computed, the ones behind them are left."""
    n, k, group = 70, 256, 64
    w = make_weight(32, (3,), n, k, group, True)
    a = make_acts(33, 50, k)
    raw = [o * rows_max // 200 if 0 < o <= 200 else o for o in raw]
    ends = np.minimum(np.maximum.accumulate([0] + raw[1:]), rows_max)
    counts, used = np.diff(ends).tolist(), int(ends[-1])
    rows = torch.randint(0, 50, (rows_max,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    off = torch.tensor(raw, dtype=torch.int32, device=DEV)
    need = bsr.w4g_proj_grouped_scratch_bytes(rows_max, 3, k)
    # scratch that holds another call's rows: NaN
    scratch = torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None
    out = torch.full((rows_max, n), 7.0, dtype=torch.bfloat16, device=DEV)
    bsr.w4g_proj_grouped(a.to(DEV), off, *dev(w), rows=rows.to(DEV), out=out, scratch=scratch)
    ref, mag = grouped_reference(a, counts, w, rows.numpy())
    check(out[:used], ref, mag, k, group)
    assert bool((out[used:] == 7.0).all())
    plain = torch.full((rows_max, n), 7.0, dtype=torch.bfloat16, device=DEV)
    bsr.w4g_proj_grouped(a[rows.long()].to(DEV), off, *dev(w), out=plain)
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
    assert bsr.device_status() == 0


@pytest.mark.parametrize("m", [4, 100])
def test_infinities_and_nan_stay_in_their_row(m):
    n, k = 100, 256
    w = make_weight(8, (), n, k, 128, True)
    a = make_acts(9, m, k)
    clean = bsr.w4g_proj(a.to(DEV), *dev(w))
    a[1, 5], a[2, 7] = float("inf"), float("nan")
    out = bsr.w4g_proj(a.to(DEV), *dev(w))
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[2]).all())
    # inf times a zero weight is NaN, times any other an infinity
    assert not bool(torch.isfinite(out[1]).any())


@pytest.mark.parametrize("m,n,k", [(3, 200, 512), (70, 200, 512)])
def test_row_bits_do_not_depend_on_the_others(m, n, k):
    w = dev(make_weight(10, (), n, k, 64))
    a = make_acts(11, m, k).to(DEV)
    out = bsr.w4g_proj(a, *w)
    other = a.clone()
    other[1:] = 3.0
    assert torch.equal(bsr.w4g_proj(other, *w)[0], out[0])
    assert torch.equal(bsr.w4g_proj(a.flip(0).contiguous(), *w), out.flip(0))


def test_zero_inputs_and_codes():
    n, k = 40, 256
    q, s, _ = make_weight(12, (), n, k, 32)
    a = make_acts(13, 5, k).to(DEV)
    zeros = bsr.w4g_proj(torch.zeros_like(a), q.to(DEV), s.to(DEV))
    assert bool((zeros == 0).all())
    # every code at its zero point: exactly zero, whatever the activations
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8)
    flat = (z | (z << 4)).repeat_interleave(16, dim=1)
    for m in (5, 90):
        x = make_acts(14, m, k).to(DEV)
        assert bool((bsr.w4g_proj(x, flat.to(DEV), s.to(DEV), z.to(DEV)) == 0).all())


def test_weights_past_31_bits():
    """The last expert of a stack whose codes pass 2^31 bytes."""
    experts, n, k, group = 34, 14336, 9216, 128
    q = torch.zeros((experts, n, k // 2), dtype=torch.uint8, device=DEV)
    assert q.numel() > 2 ** 31
    s = torch.zeros((experts, n, k // group), dtype=torch.bfloat16, device=DEV)
    w = make_weight(15, (), n, k, group)
    q[-1], s[-1] = w[0].to(DEV), w[1].to(DEV)
    rows = slice(n - 40, n)
    for m in (2, 60):
        a = make_acts(16, m, k)
        off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
        off[-1] = m
        out = bsr.w4g_proj_grouped(a.to(DEV), off, q, s)
        ref, mag = reference(a, (w[0][rows], w[1][rows], None))
        check(out[:, rows], ref, mag, k, group)


def test_streams_and_graphs():
    """On a side stream, and two captured graphs replayed in turn with new
    inputs, against eager calls."""
    n, k = 300, 512
    w = dev(make_weight(17, (4,), n, k, 64))
    a = make_acts(18, 40, k).to(DEV)
    off = offsets_of([3, 0, 30, 7]).to(DEV)
    eager = bsr.w4g_proj_grouped(a, off, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = bsr.w4g_proj_grouped(a, off, *w)
    explicit = bsr.w4g_proj_grouped(a, off, *w, stream=side)
    side.synchronize()
    assert torch.equal(on_side, eager) and torch.equal(explicit, eager)
    graphs, outs, ins = [], [], [a.clone(), a[:3].clone()]
    dense = tuple(None if t is None else t[1] for t in w)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsr.w4g_proj_grouped(ins[0], off, *w) if i == 0 else bsr.w4g_proj(ins[1], *dense))
        graphs.append(g)
    for seed in (19, 20):
        ins[0].copy_(make_acts(seed, 40, k))
        ins[1].copy_(make_acts(seed + 5, 3, k))
        for g in graphs:
            g.replay()
        graphs[0].replay()
        assert torch.equal(outs[0], bsr.w4g_proj_grouped(ins[0], off, *w))
        assert torch.equal(outs[1], bsr.w4g_proj(ins[1], *dense))


def test_empty_and_refusals():
    w = dev(make_weight(21, (), 8, 64, 32))
    a = make_acts(22, 4, 64).to(DEV)
    assert bsr.w4g_proj(a[:0], *w).shape == (0, 8)
    with pytest.raises(ValueError, match="contiguous"):
        bsr.w4g_proj(make_acts(22, 64, 4).to(DEV).t(), *w)
    with pytest.raises(ValueError, match="CUDA"):
        bsr.w4g_proj(a, w[0].cpu(), w[1])
    with pytest.raises(TypeError):
        bsr.w4g_proj(a.half(), *w)
    with pytest.raises(bsr.BsrError, match="BSR_EALIGN"):
        bsr.w4g_proj(torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64), *w)


def test_all_rows_of_one_of_many_experts():
    """Groups unlike what the host expects: every row in the last expert, on
    the decode kernel (4 rows per expert on average) and past it."""
    n, k, group = 150, 320, 64
    w = make_weight(23, (64,), n, k, group, True)
    for r in (256, 1500):
        a = make_acts(24, r, k)
        off = offsets_of([0] * 63 + [r]).to(DEV)
        out = bsr.w4g_proj_grouped(a.to(DEV), off, *dev(w))
        ref, mag = reference(a, tuple(t[63] for t in w))
        check(out, ref, mag, k, group)
        # the first expert alone, the rest of the rows behind the last group
        off = torch.full((65,), 5, dtype=torch.int32, device=DEV)
        off[0] = 0
        out = bsr.w4g_proj_grouped(a.to(DEV), off, *dev(w), out=torch.full((r, n), 2.0, dtype=torch.bfloat16,
                                                                            device=DEV))
        ref, mag = reference(a[:5], tuple(t[0] for t in w))
        check(out[:5], ref, mag, k, group)
        assert bool((out[5:] == 2.0).all())
    assert bsr.device_status() == 0


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_and_zero_points_at_any_alignment(m, group):
    """Scales aligned to 2 bytes and zero points to 1, views into larger
    buffers."""
    n, k = 70, 1024
    q, s, z = make_weight(25, (), n, k, group, True, True)
    sb = torch.zeros(s.numel() + 3, dtype=s.dtype, device=DEV)[3:].view(s.shape).copy_(s)
    zb = torch.zeros(z.numel() + 5, dtype=z.dtype, device=DEV)[5:].view(z.shape).copy_(z)
    a = make_acts(26, m, k)
    out = bsr.w4g_proj(a.to(DEV), q.to(DEV), sb, zb)
    assert torch.equal(out, bsr.w4g_proj(a.to(DEV), q.to(DEV), s.to(DEV), z.to(DEV)))
    ref, mag = reference(a, (q, s, z))
    check(out, ref, mag, k, group)


def test_magnitudes_of_activations():
    """Activations from 2^-100 to 2^100 in one row, and outliers beside codes
    at their zero point: the products are exact, so the bound holds as it is."""
    n, k, group = 64, 512, 128
    q, s, z = make_weight(27, (), n, k, group, True)
    for m in (2, 40):
        a = make_acts(28, m, k).double() * 2.0 ** torch.randint(-100, 101, (m, k), generator=torch.Generator().manual_seed(1))
        a = a.bfloat16()
        ref, mag = reference(a, (q, s, z))
        check(bsr.w4g_proj(a.to(DEV), q.to(DEV), s.to(DEV), z.to(DEV)), ref, mag, k, group, "wide")
        a = make_acts(29, m, k)
        a[:, 7] = 2.0 ** 40
        q2 = q.clone()
        q2[:, 3] = (q2[:, 3] & 15) | (z[:, 0] << 4)  # element 7 at its zero point
        ref, mag = reference(a, (q2, s, z))
        check(bsr.w4g_proj(a.to(DEV), q2.to(DEV), s.to(DEV), z.to(DEV)), ref, mag, k, group, "outlier")


def test_first_call_inside_a_capture():
    """A process whose first calls are captured, with nothing warmed up."""
    import os
    import subprocess
    import sys

    code = """
import torch
import block_scaled_precision_requant_b200 as bsr
torch.manual_seed(0)
q = torch.randint(0, 256, (4, 256, 64), dtype=torch.uint8, device="cuda")
s = torch.rand(4, 256, 1, device="cuda").bfloat16()
d = torch.randint(0, 256, (4, 128, 128), dtype=torch.uint8, device="cuda")
t = torch.rand(4, 128, 2, device="cuda").bfloat16()
outs, ins = [], []
g = torch.cuda.CUDAGraph()
for m in (2, 90):
    ins.append((torch.randn(m, 128, device="cuda").bfloat16(), torch.randn(m, 4, device="cuda")))
torch.cuda.synchronize()
with torch.cuda.graph(g):
    for x, lg in ins:
        outs.append(bsr.w4g_moe_mlp(x, lg, (q, s, None), (q, s, None), (d, t, None), 2))
        outs.append(bsr.w4g_proj(x, q[0], s[0]))
g.replay()
torch.cuda.synchronize()
for i, (x, lg) in enumerate(ins):
    assert torch.equal(outs[2 * i], bsr.w4g_moe_mlp(x, lg, (q, s, None), (q, s, None), (d, t, None), 2))
    assert torch.equal(outs[2 * i + 1], bsr.w4g_proj(x, q[0], s[0]))
assert bsr.device_status() == 0
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("ok"), p.stderr[-2000:]


def test_a_tensor_of_another_device_is_made_current(monkeypatch):
    """Where the current device is another one, the call runs with the
    tensor's device current and puts the old one back."""
    w = dev(make_weight(30, (), 8, 64, 32))
    a = make_acts(31, 4, 64).to(DEV)
    want = bsr.w4g_proj(a, *w)
    entered = []

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            entered.append("out")

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 5)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    assert torch.equal(bsr.w4g_proj(a, *w), want)
    assert entered == [0, "out"]


def test_given_stream_owns_what_the_call_allocates(monkeypatch):
    """With ``stream=`` the scratch and outputs come from that stream's memory:
    the current stream, which does not wait for it, is never handed them while
    the call runs."""
    g = torch.Generator(device=DEV).manual_seed(8)
    experts, n, k, r = 4, 256, 512, 200
    a = torch.randn(64, k, generator=g, device=DEV).to(torch.bfloat16)
    off = torch.tensor([0, 60, 60, 150, 200], dtype=torch.int32, device=DEV)
    rows = torch.randint(0, 64, (r,), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randint(0, 256, (experts, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(experts, n, k // 64, generator=g, device=DEV).to(torch.bfloat16)
    want = bsr.w4g_proj_grouped(a, off, q, s, rows=rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen = []
    plain = bsr._scratch

    def record(*args):
        got = plain(*args)
        seen.append(got)
        return got

    monkeypatch.setattr(bsr, "_scratch", record)
    torch.cuda.empty_cache()
    out = bsr.w4g_proj_grouped(a, off, q, s, rows=rows, stream=side)
    (address, size), = seen
    assert size > 0
    held = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(3)]
    assert address not in [t.data_ptr() for t in held]
    side.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError, match="contiguous"):
        bsr.w4g_proj_grouped(a, off, q, s, rows=rows, scratch=torch.empty(2 * size, dtype=torch.uint8, device=DEV)[::2])


SHARED_K = [
    # few tiles and a K of at least eight stages of 128: two, four or eight CTAs per tile
    (17, 1, 1024, 128), (33, 300, 2080, 32), (17, 1000, 4160, 64), (50, 1920, 4096, 128), (100, 77, 4256, 32),
    (130, 513, 1152, 128), (192, 129, 8192, 64), (300, 1024, 1088, 64), (200, 2300, 2048, 128), (17, 4700, 2048, 32),
]


@pytest.mark.parametrize("zero,half", [(False, True), (True, False)])
@pytest.mark.parametrize("m,n,k,group", SHARED_K)
def test_dense_with_k_shared_by_a_cluster(m, n, k, group, zero, half):
    w = make_weight(m + n + k, (), n, k, group, zero, half)
    a = make_acts(n, m, k)
    x, wd = a.to(DEV), dev(w)
    out = bsr.w4g_proj(x, *wd)
    ref, mag = reference(a, w)
    check(out, ref, mag, k, group)
    guard = torch.full((m + 2, n), 7.0, device=DEV, dtype=torch.bfloat16)
    for _ in range(3):
        bsr.w4g_proj(x, *wd, out=guard[1:-1])
        assert torch.equal(guard[1:-1], out)
    assert bool((guard[0] == 7.0).all()) and bool((guard[-1] == 7.0).all())
    assert bsr.device_status() == 0


def test_shared_k_back_to_back_on_two_streams():
    """Launches whose clusters follow or meet one another: the same bits."""
    w = make_weight(5, (), 2048, 4096, 64, True, False)
    wd = dev(w)
    xs = [make_acts(i, m, 4096).to(DEV) for i, m in enumerate((17, 100, 64, 33))]
    want = [bsr.w4g_proj(x, *wd) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for r in range(10):
        for i, x in enumerate(xs):
            got.append((i, bsr.w4g_proj(x, *wd, stream=streams[(r + i) % 2])))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)
    assert bsr.device_status() == 0


def test_first_shared_k_call_inside_a_capture():
    import os
    import subprocess
    import sys

    code = """
import torch
import block_scaled_precision_requant_b200 as bsr
torch.manual_seed(0)
q = torch.randint(0, 256, (512, 1024), dtype=torch.uint8, device="cuda")
s = torch.rand(512, 32, device="cuda").bfloat16()
x = torch.randn(40, 2048, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = bsr.w4g_proj(x, q, s)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, bsr.w4g_proj(x, q, s)) and bsr.device_status() == 0
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("ok"), p.stderr[-2000:]
