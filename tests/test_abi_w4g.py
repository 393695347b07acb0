"""Argument checks of the integer 4-bit and expert entry points (no GPU
needed: each returns before it touches a device or a pointer)."""
import ctypes

import pytest
import torch

import block_scaled_precision_requant_b200 as bsr
from block_scaled_precision_requant_b200 import build

P = ctypes.c_void_p
OK, EINVAL, EALIGN, ESHAPE, ESCRATCH = 0, 1, 2, 3, 4
A = P(256)


@pytest.fixture(scope="module")
def L():
    build.build()
    return bsr.lib()


def weight(q=256, scale=256, zero=None, kind=0, group=64):
    return ctypes.byref(bsr._W4gWeight(q, scale, zero, kind, group))


def test_constants_match_the_header():
    import os
    import re

    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bsr.h")).read()
    d = dict(re.findall(r"^#define (BSR_(?:W4G|MOE)_\w+) (\d+)u?$", src, flags=re.M))
    assert d == {"BSR_W4G_SCALE_BF16": "0", "BSR_W4G_SCALE_FP16": "1", "BSR_MOE_MAX_EXPERTS": "1024",
                 "BSR_MOE_MAX_TOP_K": "32", "BSR_MOE_LOGITS_F32": "0", "BSR_MOE_LOGITS_BF16": "1",
                 "BSR_MOE_RENORMALIZE": "1"}
    fields = re.search(r"typedef struct bsr_w4g_weight \{(.*?)\}", src, flags=re.S).group(1)
    assert re.findall(r"(\w+);", fields) == [n for n, _ in bsr._W4gWeight._fields_]


def test_proj(L):
    assert L.bsr_w4g_proj(A, None, A, 1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(kind=2), A, 1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(group=16), A, 1, 8, 64, None) == ESHAPE
    assert L.bsr_w4g_proj(A, weight(), A, 1, 8, 96, None) == ESHAPE and "group 64" in bsr.last_error()
    assert L.bsr_w4g_proj(A, weight(), A, 1, 8, 0, None) == ESHAPE
    assert L.bsr_w4g_proj(A, weight(), A, -1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(), A, 1, 2 ** 31, 64, None) == EINVAL
    assert L.bsr_w4g_proj(None, weight(), A, 1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(q=None), A, 1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(q=264), A, 1, 8, 64, None) == EALIGN
    assert L.bsr_w4g_proj(A, weight(scale=257), A, 1, 8, 64, None) == EALIGN
    assert L.bsr_w4g_proj(P(264), weight(), A, 1, 8, 64, None) == EALIGN
    assert L.bsr_w4g_proj(A, weight(), P(257), 1, 8, 64, None) == EALIGN
    assert L.bsr_w4g_proj(None, weight(None, None), None, 0, 8, 64, None) == OK
    assert L.bsr_w4g_proj(None, weight(None, None), None, 8, 0, 64, None) == OK


def test_proj_grouped(L):
    def call(a=A, a_rows=4, off=A, rows=A, w=None, out=A, r=4, e=2, n=8, k=64, scratch=None, nbytes=0):
        return L.bsr_w4g_proj_grouped(a, a_rows, off, rows, w or weight(), out, r, e, n, k, scratch, nbytes, None)

    assert call(e=0) == EINVAL and call(e=1025) == EINVAL and call(n=2 ** 30, e=2) == EINVAL
    assert call(r=-1) == EINVAL and call(a_rows=-1) == EINVAL
    assert call(off=None) == EINVAL and call(a=None) == EINVAL and call(out=None) == EINVAL
    assert call(rows=None, a_rows=3) == EINVAL and "row index" in bsr.last_error()
    assert call(off=P(258)) == EALIGN and call(rows=P(258)) == EALIGN and call(a=P(264)) == EALIGN
    assert call(w=weight(q=8)) == EALIGN and call(k=32) == ESHAPE
    assert call(a=None, off=None, rows=None, out=None, r=0) == OK
    # many rows per expert and a row index: the rows in group order
    assert L.bsr_w4g_proj_grouped_scratch_bytes(8, 2, 64) == 0
    need = L.bsr_w4g_proj_grouped_scratch_bytes(33, 2, 64)
    assert need == (33 * 64 * 2 + 255) // 256 * 256 and L.bsr_w4g_proj_grouped_scratch_bytes(-1, 2, 64) == 0
    assert call(r=33) == ESCRATCH and call(r=33, scratch=A, nbytes=need - 1) == ESCRATCH
    assert call(r=33, scratch=P(128), nbytes=need) == EALIGN


def test_route(L):
    def call(logits=A, kind=0, t=4, e=8, k=2, flags=0, out=(A, A, A, A, A), scratch=None, nbytes=0):
        return L.bsr_moe_route(logits, kind, t, e, k, flags, *out, scratch, nbytes, None)

    assert call(e=0) == EINVAL and call(e=1025) == EINVAL and call(k=0) == EINVAL and call(k=9) == EINVAL
    assert call(e=64, k=33) == EINVAL and call(t=-1) == EINVAL and call(t=2 ** 30, k=2) == EINVAL
    assert call(kind=2) == EINVAL and call(flags=2) == EINVAL and call(logits=None) == EINVAL
    assert call(logits=P(258)) == EALIGN and call(logits=P(257), kind=1) == EALIGN
    for i in range(5):
        assert call(out=tuple(None if j == i else A for j in range(5))) == EINVAL
        assert call(out=tuple(P(258) if j == i else A for j in range(5))) == EALIGN
    assert L.bsr_moe_route_scratch_bytes(64, 8) == 0
    need = L.bsr_moe_route_scratch_bytes(129, 8)
    assert need == 5 * 8 * 4 and L.bsr_moe_route_scratch_bytes(10 ** 6, 64) <= 128 * 64 * 4
    assert call(t=129) == ESCRATCH and call(t=129, scratch=A, nbytes=need - 1) == ESCRATCH
    assert call(t=129, scratch=P(258), nbytes=need) == EALIGN


def test_combine(L):
    def call(y=A, rows=8, pos=A, w=A, res=None, out=A, t=4, k=2, n=8):
        return L.bsr_moe_combine(y, rows, pos, w, res, out, t, k, n, None)

    assert call(t=-1) == EINVAL and call(k=0) == EINVAL and call(k=33) == EINVAL and call(n=-1) == EINVAL
    assert call(y=None) == EINVAL and call(pos=None) == EINVAL and call(w=None) == EINVAL and call(out=None) == EINVAL
    assert call(y=P(257)) == EALIGN and call(pos=P(258)) == EALIGN and call(res=P(257)) == EALIGN
    assert call(None, 0, None, None, None, None, 0) == OK and call(None, 0, None, None, None, None, n=0) == OK


def test_mlp(L):
    need = L.bsr_w4g_moe_mlp_scratch_bytes(4, 8, 2, 64, 128)
    assert need > 0 and need % 256 == 0
    for bad in ((0, 8, 2, 64, 128), (4, 0, 2, 64, 128), (4, 8, 9, 64, 128), (4, 8, 2, 0, 128), (4, 8, 2, 64, 0)):
        assert L.bsr_w4g_moe_mlp_scratch_bytes(*bad) == 0

    def call(x=A, logits=A, kind=0, gate=None, up=None, down=None, res=None, out=A, t=4, e=8, k=2, flags=1, inner=64,
             hidden=128, scratch=A, nbytes=need):
        return L.bsr_w4g_moe_mlp(x, logits, kind, gate or weight(), up or weight(), down or weight(), res, out, t, e,
                                 k, flags, inner, hidden, scratch, nbytes, None)

    assert call(k=9) == EINVAL and call(flags=4) == EINVAL and call(kind=3) == EINVAL and call(x=None) == EINVAL
    assert call(inner=96) == ESHAPE and call(hidden=96) == ESHAPE and call(down=weight(group=48)) == ESHAPE
    assert call(up=weight(q=None)) == EINVAL and call(down=weight(q=8)) == EALIGN and call(x=P(258)) == EALIGN
    assert call(scratch=None) == ESCRATCH and call(nbytes=need - 1) == ESCRATCH and call(scratch=P(128)) == EALIGN
    assert call(x=None, logits=None, out=None, t=0) == OK


def test_binding_refuses_before_the_library():
    a = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsr.w4g_proj(a, q, s)
    with pytest.raises(ValueError, match="dimensions"):
        bsr._dims(a[0], 2, "a")
    with pytest.raises(ValueError, match="CUDA"):
        bsr.w4g_proj_grouped(a, torch.zeros(2, dtype=torch.int32), q, s)
    with pytest.raises(TypeError):
        bsr.w4g_proj([1.0], q, s)
    for bad, error in ((a.half(), TypeError), (a.t(), ValueError), (a[:1], ValueError), (a, ValueError),
                       (None, TypeError)):
        with pytest.raises(error):
            bsr._ptr(bad, torch.bfloat16, (2, 64), "a", 0)
    with pytest.raises(ValueError, match="top_k"):
        bsr.moe_route(torch.zeros(2, 4), 5)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        bsr.moe_route(torch.zeros(2, 4, dtype=torch.float64), 2)
    for groups, kind, error in ((3, torch.bfloat16, ValueError), (1, torch.float32, TypeError),
                                (4, torch.bfloat16, ValueError), (0, torch.bfloat16, ValueError)):
        with pytest.raises(error):
            bsr._w4g_weight(q, torch.zeros(8, groups, dtype=kind), None, (), 8, 64, -1, "w")


def test_sizes_near_31_bits_are_refused(L):
    """The kernels count rows and elements of K in 32 bits, up to a tile past
    the end: 2^31 - 256 is the largest size."""
    top = 2 ** 31 - 256
    big = top + 32  # a multiple of 32
    assert L.bsr_w4g_proj(A, weight(), A, 1, top + 1, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(), A, top + 1, 8, 64, None) == EINVAL
    assert L.bsr_w4g_proj(A, weight(group=32), A, 1, 8, big, None) == EINVAL

    def grouped(a_rows=4, r=4, e=2, n=8):
        return L.bsr_w4g_proj_grouped(A, a_rows, A, A, weight(), A, r, e, n, 64, None, 0, None)

    assert grouped(r=top + 1) == EINVAL and grouped(a_rows=top + 1) == EINVAL and grouped(n=2 ** 30 - 127) == EINVAL
    assert "2^31 - 256" in bsr.last_error()
    assert L.bsr_moe_route(A, 0, 2 ** 30 - 127, 8, 2, 0, A, A, A, A, A, None, 0, None) == EINVAL
    assert L.bsr_moe_combine(A, 4, A, A, None, A, 2 ** 30 - 127, 2, 8, None) == EINVAL
    assert L.bsr_moe_combine(A, top + 1, A, A, None, A, 4, 2, 8, None) == EINVAL
    w = weight(group=32)
    assert L.bsr_w4g_moe_mlp(A, A, 0, w, w, w, None, A, 4, 8, 2, 0, top // 8 + 32, 64, A, 0, None) == EINVAL
    assert L.bsr_w4g_moe_mlp_scratch_bytes(4, 8, 2, big, 64) == 0


def test_mlp_scratch_past_64_bits_is_refused(L):
    """Sizes that each hold but whose scratch bytes pass 64 bits: no wrapped
    size, and the call refuses them before it looks at the scratch."""
    top, group = 2 ** 31 - 256, weight(group=32)

    def call(t, e, k, inner, hidden):
        return L.bsr_w4g_moe_mlp(A, A, 0, group, group, group, None, A, t, e, k, 0, inner, hidden, A, 2 ** 64 - 1, None)

    for t, e, k, inner, hidden in ((top, 1, 1, top, 32), (top, 1, 1, top, top), (2 ** 30, 1, 1, top, top),
                                   (top // 2, 2, 2, top // 2 - 64, 64), (top, 1, 1, 2 ** 30, 2 ** 30)):
        assert L.bsr_w4g_moe_mlp_scratch_bytes(t, e, k, inner, hidden) == 0
        assert call(t, e, k, inner, hidden) == EINVAL and "scratch" in bsr.last_error()
    for t, e, k, inner, hidden in ((2 ** 26 - 8, 32, 32, 2 ** 26 - 32, 2 ** 26 - 32), (2 ** 20, 1, 1, top, top)):
        pairs = t * k
        least = pairs * 2 * (3 * inner + 2 * hidden)
        assert least <= L.bsr_w4g_moe_mlp_scratch_bytes(t, e, k, inner, hidden) <= least + 2 ** 37


@pytest.mark.parametrize("bad", [[[1.0, 2.0]], None, 3])
def test_what_is_not_a_tensor_is_a_type_error(bad, monkeypatch):
    """Every tensor argument, whichever is looked at first; CPU tensors stand
    in for the device's."""
    monkeypatch.setattr(bsr, "_like", lambda t, name, stream: (-1, bsr._HERE))
    a = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    e3, off = (q[None], s[None], None), torch.zeros(2, dtype=torch.int32)
    lg, pos, wt = torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    calls = [lambda: bsr.w4g_proj(a, bad, s), lambda: bsr.moe_route(bad, 1), lambda: bsr.moe_combine(bad, pos, wt),
             lambda: bsr.moe_combine(a, bad, wt), lambda: bsr.moe_combine(a, pos, bad),
             lambda: bsr.w4g_proj_grouped(a, off, bad, s), lambda: bsr.w4g_moe_mlp(bad, lg, e3, e3, e3, 1),
             lambda: bsr.w4g_moe_mlp(a, bad, e3, e3, e3, 1), lambda: bsr.w4g_moe_mlp(a, lg, bad, e3, e3, 1),
             lambda: bsr.w4g_moe_mlp(a, lg, e3, bad, e3, 1), lambda: bsr.w4g_moe_mlp(a, lg, e3, e3, bad, 1),
             lambda: bsr.w4g_moe_mlp(a, lg, (bad, s, None), e3, e3, 1),
             lambda: bsr.w4g_moe_mlp(a, lg, (q[None], bad, None), e3, e3, 1)]
    if bad is not None:  # stands for every row in order, zero points of 8, memory of the call's own
        calls += [lambda: bsr.w4g_proj_grouped(a, off, q[None], s[None], rows=bad), lambda: bsr.w4g_proj(a, q, s, bad),
                  lambda: bsr._scratch(bad, 8, a)]
    for call in calls:
        with pytest.raises(TypeError, match="must be"):
            call()
    for short in ((q[None], s[None]), (q[None], s[None], None, None)):
        with pytest.raises(TypeError, match="gate must be"):
            bsr.w4g_moe_mlp(a, lg, short, e3, e3, 1)
