"""Expert router, combine and the expert MLP against the oracle.

Integer results are equal.  Weights: exp to 2 float32 steps, sums of at most
E terms and one division, so 2^-24 (E + 8) relative.  Combine: one BF16
rounding (2^-8 of the value) of a float32 sum of at most top_k + 1 terms,
2^-24 (2 top_k + 2) of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import block_scaled_precision_requant_b200 as bsr
import oracle
from tests.test_gpu_w4g import dev, make_acts, make_weight

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make_logits(seed, t, e, bf16=False, mask=0.1, ties=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, e, generator=g)
    if ties:
        x = (x * 2).round() / 2
    drop = torch.rand(t, e, generator=g)
    x = torch.where(drop < mask / 2, torch.tensor(float("nan")), torch.where(drop < mask, -torch.inf, x))
    x[t // 2] = -torch.inf
    return x.bfloat16() if bf16 else x


def check_route(route, x, top_k, renorm):
    ids, w, off, rows, pos = oracle.moe_route(x.double().numpy(), top_k, renorm)
    for name, ref in (("ids", ids), ("offsets", off), ("rows", rows), ("pos", pos)):
        assert np.array_equal(getattr(route, name).cpu().numpy(), ref), name
    got = route.weights.double().cpu().numpy()
    assert np.all(np.abs(got - w) <= 2.0 ** -24 * (x.shape[1] + 8) * np.abs(w))


ROUTES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 64, 8), (33, 65, 6), (128, 8, 2), (129, 31, 4), (300, 96, 8),
          (1000, 128, 8), (70, 384, 8), (513, 512, 10), (40, 1000, 32), (260, 1024, 1)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("t,e,k", ROUTES)
def test_route(t, e, k, bf16):
    for renorm, ties in ((True, False), (False, True)):
        x = make_logits(t + e + k, t, e, bf16, mask=0.1 if e > 4 else 0.0, ties=ties)
        check_route(bsr.moe_route(x.to(DEV), k, renormalize=renorm), x, k, renorm)


def test_route_extremes():
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[big, -big, 0.0, -0.0], [-big, -big, -torch.inf, -big], [torch.inf, 1.0, torch.inf, big],
                      [0.0, -0.0, 1e-45, -1e-45], [torch.nan] * 4, [-torch.inf, -torch.inf, 5.0, -torch.inf]])
    for renorm in (True, False):
        check_route(bsr.moe_route(x.to(DEV), 3, renormalize=renorm), x, 3, renorm)


def test_route_no_tokens():
    r = bsr.moe_route(torch.empty(0, 6, device=DEV), 2)
    assert r.ids.shape == (0, 2) and r.rows.shape == (0,) and r.offsets.tolist() == [0] * 7


def test_route_large_is_deterministic():
    """More tokens than two waves of blocks: sorted groups, every pair once."""
    t, e, k = 40000, 100, 6
    x = torch.randn(t, e, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    x[-100:] = -torch.inf
    a, b = bsr.moe_route(x, k), bsr.moe_route(x, k)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    used = int(a.offsets[-1])
    assert used == (t - 100) * k and bool((a.rows[used:] == -1).all())
    order = torch.sort(torch.where(a.ids < 0, e, a.ids).flatten(), stable=True).indices[:used]
    assert torch.equal(a.rows[:used].long(), order // k)
    assert torch.equal(a.pos.flatten()[order].long(), torch.arange(used, device=DEV))
    assert torch.equal(torch.bincount(a.ids.flatten().clamp(min=0)[a.ids.flatten() >= 0], minlength=e),
                       (a.offsets[1:] - a.offsets[:-1]).long())


@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (3, 2, 5), (7, 8, 130), (33, 3, 2048), (64, 6, 1412), (5, 32, 24)])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(t, k, n, residual):
    g = torch.Generator().manual_seed(t * n)
    r = t * k
    y = torch.randn(r, n, generator=g).bfloat16()
    pos = torch.randint(-1, r + 1, (t, k), generator=g, dtype=torch.int32)  # skipped and repeated rows among them
    w = torch.rand(t, k, generator=g) - 0.3
    res = torch.randn(t, n, generator=g).bfloat16() if residual else None
    out = bsr.moe_combine(y.to(DEV), pos.to(DEV), w.to(DEV), residual=None if res is None else res.to(DEV))
    ref, mag = oracle.moe_combine(y.double().numpy(), pos.numpy(), w.numpy(),
                                  None if res is None else res.double().numpy())
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * (2 * k + 3) * mag)
    if residual:  # in place
        own = res.to(DEV)
        assert torch.equal(bsr.moe_combine(y.to(DEV), pos.to(DEV), w.to(DEV), residual=own, out=own), out)


def test_combine_skips_what_a_dropped_slot_names():
    """A skipped position contributes nothing even with a NaN weight, and a
    token with none gives zeros."""
    y = torch.full((2, 16), torch.nan, dtype=torch.bfloat16, device=DEV)
    pos = torch.tensor([[-1, -1], [2, -7]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[torch.nan, 1.0], [torch.inf, 1.0]], device=DEV)
    assert bool((bsr.moe_combine(y, pos, w) == 0).all())


def mlp_steps(x, logits, gate, up, down, k, renorm, residual):
    r = bsr.moe_route(logits, k, renormalize=renorm)
    g = bsr.w4g_proj_grouped(x, r.offsets, *gate, rows=r.rows)
    u = bsr.w4g_proj_grouped(x, r.offsets, *up, rows=r.rows)
    y = bsr.w4g_proj_grouped(bsr.silu_mul(g, u), r.offsets, *down)
    return bsr.moe_combine(y, r.pos, r.weights, residual=residual)


MLPS = [(1, 4, 2, 64, 128, 32), (5, 8, 3, 192, 256, 64), (40, 16, 4, 96, 160, 32), (300, 6, 2, 384, 512, 128),
        (700, 3, 3, 128, 64, 64)]


@pytest.mark.parametrize("t,e,k,inner,hidden,group", MLPS)
def test_mlp(t, e, k, inner, hidden, group):
    """The operators in a row: the same bits as the calls one by one, and the
    float64 evaluation within the BF16 roundings of the tensors between."""
    gate, up = (make_weight(s, (e,), inner, hidden, group, s == 1) for s in (1, 2))
    down = make_weight(3, (e,), hidden, inner, 32, True, True)
    x = make_acts(4, t, hidden)
    logits = make_logits(5, t, e, mask=0.0)
    res = make_acts(6, t, hidden)
    args = [x.to(DEV), logits.to(DEV), dev(gate), dev(up), dev(down), k]
    out = bsr.w4g_moe_mlp(*args, residual=res.to(DEV))
    assert torch.equal(out.view(torch.int16), mlp_steps(*args, True, res.to(DEV)).view(torch.int16))
    plain = bsr.w4g_moe_mlp(*args, renormalize=False)
    assert torch.equal(plain.view(torch.int16), mlp_steps(*args, False, None).view(torch.int16))
    assert bool((plain[t // 2] == 0).all())  # a token that no expert takes
    ids, w, *_ = oracle.moe_route(logits.double().numpy(), k, False)
    want = np.zeros((t, hidden))
    slack = np.zeros((t, hidden))
    eps = 2.0 ** -8
    for i in range(t):
        for s in range(k):
            j = ids[i, s]
            if j < 0:
                continue
            a = x[i:i + 1].double().numpy()
            part = [[None if p is None else p[j] for p in wt] for wt in (gate, up, down)]
            part = [(q.numpy(), sc.double().numpy(), None if z is None else z.numpy()) for q, sc, z in part]
            g, g_mag = oracle.w4g_proj(a, *part[0])
            u, u_mag = oracle.w4g_proj(a, *part[1])
            h = g / (1 + np.exp(-g)) * u
            # gate and up are rounded to BF16 (and float32-summed: 2^-15 of the
            # magnitudes is more than (G + K/G + 18) 2^-23 here); |silu'| <= 1.1, |silu(g)| <= |g|
            dg, du = eps * np.abs(g) + 2.0 ** -15 * g_mag, eps * np.abs(u) + 2.0 ** -15 * u_mag
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du
            dh = dh + (eps + 2.0 ** -20) * (np.abs(h) + dh)
            y, y_mag = oracle.w4g_proj(h, *part[2])
            _, spread = oracle.w4g_proj(dh, *part[2])
            dy = spread + eps * (np.abs(y) + spread) + 2.0 ** -15 * (y_mag + spread)
            want[i] += w[i, s] * y[0]
            slack[i] += w[i, s] * dy[0] + 2.0 ** -18 * w[i, s] * np.abs(y[0])
    tol = slack + eps * (np.abs(want) + slack)
    assert np.all(np.abs(plain.double().cpu().numpy() - want) <= tol)
    assert bsr.device_status() == 0


def test_mlp_in_a_graph_with_padding():
    """A captured MLP of a padded batch, replayed with other inputs and other
    padding, beside a second graph with its own scratch."""
    e, k, inner, hidden = 8, 2, 128, 256
    ws = [dev(make_weight(i, (e,), n, kk, 64)) for i, (n, kk) in enumerate([(inner, hidden), (inner, hidden),
                                                                           (hidden, inner)])]
    graphs, ins, outs = [], [], []
    for t in (24, 200):
        x, lg = make_acts(t, t, hidden).to(DEV), make_logits(t, t, e, mask=0.0).to(DEV)
        bsr.w4g_moe_mlp(x, lg, *ws, k)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsr.w4g_moe_mlp(x, lg, *ws, k))
        graphs.append(g)
        ins.append((x, lg))
    for seed in (1, 2):
        for x, lg in ins:
            x.copy_(make_acts(seed, x.shape[0], hidden))
            lg.copy_(make_logits(seed, x.shape[0], e, mask=0.0))
            lg[x.shape[0] - 5 * seed:] = -torch.inf
        for g in graphs:
            g.replay()
        for (x, lg), out in zip(ins, outs):
            assert torch.equal(out, bsr.w4g_moe_mlp(x, lg, *ws, k))
            assert bool((out[x.shape[0] - 5 * seed:] == 0).all())


def test_two_threads_on_two_streams():
    import threading

    e, k, inner, hidden, t = 4, 2, 128, 128, 50
    ws = [dev(make_weight(i, (e,), 128, 128, 32)) for i in range(3)]
    data = [(make_acts(i, t, hidden).to(DEV), make_logits(i, t, e, mask=0.0).to(DEV)) for i in range(2)]
    want = [bsr.w4g_moe_mlp(x, lg, *ws, k) for x, lg in data]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got[i].append(bsr.w4g_moe_mlp(*data[i], *ws, k))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i]) and len(got[0]) == len(got[1]) == 10


def test_refusals():
    x = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="top_k"):
        bsr.moe_route(x, 9)
    with pytest.raises(ValueError, match="top_k"):
        bsr.moe_route(x, 0)
    with pytest.raises(TypeError):
        bsr.moe_route(x.half(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        bsr.moe_route(torch.zeros(8, 4, device=DEV).t(), 2)
    with pytest.raises(bsr.BsrError, match="BSR_EINVAL"):
        bsr.moe_route(torch.zeros(2, 1025, device=DEV), 2)
    y = torch.zeros(8, 16, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        bsr.moe_combine(y, torch.zeros(4, 2, device=DEV), torch.zeros(4, 2, device=DEV))


@pytest.mark.parametrize("t,e,k,inner,hidden,group", [(1700, 4, 2, 1504, 544, 32), (1500, 6, 3, 1088, 640, 64),
                                                      (700, 1024, 8, 64, 96, 32), (20, 1024, 8, 128, 128, 128)])
def test_mlp_of_large_tiles_and_many_experts(t, e, k, inner, hidden, group):
    """The bits of the calls one by one, with a residual, zero points, FP16
    scales, masked experts and weights over all of them."""
    gate, up = (dev(make_weight(s, (e,), inner, hidden, group, True, s == 2)) for s in (1, 2))
    down = dev(make_weight(3, (e,), hidden, inner, 32, False, True))
    x, res = make_acts(4, t, hidden).to(DEV), make_acts(5, t, hidden).to(DEV)
    logits = make_logits(6, t, e, bf16=True).to(DEV)
    for renorm, r in ((True, res), (False, None)):
        out = bsr.w4g_moe_mlp(x, logits, gate, up, down, k, renormalize=renorm, residual=r)
        want = mlp_steps(x, logits, gate, up, down, k, renorm, r)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        left = out[t // 2]  # a token that no expert takes
        assert torch.equal(left, torch.zeros_like(left) if r is None else r[t // 2])
    assert bsr.device_status() == 0
