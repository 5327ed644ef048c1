"""Refusals of the 4-bit matrix and expert routing calls: bad arguments are
turned away before anything is launched (no GPU needed; the addresses are never
dereferenced)."""
import numpy as np
import pytest
import torch

from oracle import moe, mx4
from trellis_coded_bit_b200 import exl3

A, B, C, D, E, F, G = (i << 28 for i in range(1, 8))  # aligned, 256 MiB apart
MIS = A + 8
INV, WS, OK = exl3.EXL3_ERR_INVALID_ARG, exl3.EXL3_ERR_WORKSPACE, exl3.EXL3_OK
BIG = 1 << 27


def test_scale_stride():
    for k in (32, 512, 544, 4096, 1 << 22):
        assert exl3.exl3_mx4_scale_stride(k) == mx4.stride(k)
    for k in (0, -32, 16, 48, (1 << 22) + 32):
        assert exl3.exl3_mx4_scale_stride(k) == 0


def quantize(x=A, dtype=0, signs=None, rotate=0, pos=None, topk=1, out_rows=4, codes=B, scales=C, rows=4, k=256):
    return exl3.load().exl3_mx4_quantize(x, dtype, signs, rotate, pos, topk, out_rows, codes, scales, rows, k, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=MIS), dict(codes=None), dict(codes=B + 4), dict(scales=None),
                                 dict(scales=C + 8), dict(signs=D + 2), dict(dtype=3), dict(dtype=-1), dict(rows=-1),
                                 dict(rows=(1 << 30) + 1), dict(k=0), dict(k=40), dict(k=160, rotate=1),
                                 dict(codes=A), dict(scales=A), dict(codes=C), dict(signs=B),
                                 dict(pos=D, topk=0), dict(pos=D, topk=1025), dict(pos=D + 4), dict(pos=B, topk=2),
                                 dict(pos=D, out_rows=-1)])
def test_quantize_refusals(bad):
    assert quantize(**bad) == INV


def test_no_rows_is_no_work():
    lib = exl3.load()
    assert quantize(rows=0, x=None, codes=None, scales=None) == OK
    assert quantize(pos=D, out_rows=0, codes=None, scales=None) == OK
    assert lib.exl3_mx4_dequantize(None, None, None, 0, 0, 64, None) == OK
    assert lib.exl3_mx4_matmul(None, None, B, C, None, 0, 0, 64, 8, None, 0, None) == OK
    assert lib.exl3_mx4_linear(None, 0, None, 0, B, C, None, 0, 64, 8, None, 0, None) == OK
    assert lib.exl3_mx4_matmul_experts(None, None, None, B, C, None, 0, 0, 64, 8, 2, None, 0, None) == OK
    assert lib.exl3_moe_gather(None, 0, None, 0, 2, 8, 4, None, None) == OK
    assert lib.exl3_moe_gather(A, 0, B, 2, 2, 8, 0, None, None) == OK
    assert lib.exl3_moe_combine(A, 0, None, None, 0, 2, 8, 4, None, 0, None) == OK
    assert lib.exl3_moe_combine_grad(None, A, 0, None, None, 0, 2, 8, 4, B, C, None) == OK


@pytest.mark.parametrize("bad", [dict(codes=None), dict(scales=None), dict(w=None), dict(w=C + 8), dict(dtype=7),
                                 dict(k=8), dict(rows=-2), dict(w=A), dict(w=B)])
def test_dequantize_refusals(bad):
    a = dict(codes=A, scales=B, w=C, dtype=0, rows=4, k=256)
    a.update(bad)
    assert exl3.load().exl3_mx4_dequantize(a["codes"], a["scales"], a["w"], a["dtype"], a["rows"], a["k"], None) == INV


def matmul(xc=A, xs=B, wc=C, ws=D, y=E, dtype=0, m=4, k=256, n=64, space=F, nb=BIG):
    return exl3.load().exl3_mx4_matmul(xc, xs, wc, ws, y, dtype, m, k, n, space, nb, None)


SIZES = [dict(m=-1), dict(m=(1 << 30) + 1), dict(k=0), dict(k=100), dict(n=0), dict(n=(1 << 24) + 1), dict(dtype=3),
         dict(dtype=9)]


@pytest.mark.parametrize("bad", SIZES + [dict(xc=None), dict(xs=MIS), dict(wc=None), dict(ws=D + 4), dict(y=None),
                                         dict(y=E + 2), dict(y=A), dict(y=C)])
def test_matmul_refusals(bad):
    assert matmul(**bad) == INV


def test_matmul_workspace():
    need = exl3.exl3_mx4_matmul_workspace_size(4, 256, 64)
    assert need > 65536
    for bad in (dict(space=None), dict(space=F + 8), dict(nb=need - 1)):
        assert matmul(**bad) == WS
    assert exl3.exl3_mx4_matmul_workspace_size(4, 100, 64) == 0
    assert exl3.exl3_mx4_linear_workspace_size(4, 256, 64) >= need + 4 * 128 + 4 * 16
    assert exl3.exl3_mx4_linear_workspace_size(4, 256, 0) == 0
    assert exl3.exl3_mx4_matmul_experts_workspace_size(4, 256, 64, 513) == 0


@pytest.mark.parametrize("bad", SIZES + [dict(dtype=2), dict(x=None), dict(x=MIS), dict(signs=G + 8), dict(wc=None), dict(ws=None),
                                         dict(y=None), dict(y=A), dict(y=C), dict(rotate=1, k=96)])
def test_linear_refusals(bad):
    a = dict(x=A, dtype=0, signs=None, rotate=0, wc=C, ws=D, y=E, m=4, k=256, n=64, space=F, nb=BIG)
    a.update(bad)
    assert exl3.load().exl3_mx4_linear(*a.values(), None) == INV


@pytest.mark.parametrize("bad", SIZES[:3] + SIZES[4:] + [dict(off=None), dict(off=G + 4), dict(off=E), dict(experts=0),
                                                         dict(experts=513), dict(wc=None), dict(y=B)])
def test_experts_refusals(bad):
    a = dict(xc=A, xs=B, off=G, wc=C, ws=D, y=E, dtype=0, m=4, k=256, n=64, experts=3, space=F, nb=BIG)
    a.update(bad)
    assert exl3.load().exl3_mx4_matmul_experts(*a.values(), None) == INV
    a.update(xc=A, xs=B, off=G, wc=C, ws=D, y=E, dtype=0, m=4, k=256, n=64, experts=3, nb=100)
    assert exl3.load().exl3_mx4_matmul_experts(*a.values(), None) == WS


@pytest.mark.parametrize("bad", [dict(ids=None), dict(ids=MIS), dict(off=None), dict(pos=None), dict(pos=C + 4),
                                 dict(tokens=-1), dict(topk=0), dict(topk=1025), dict(experts=0), dict(experts=1025),
                                 dict(tokens=1 << 24, topk=128), dict(pos=A), dict(off=A), dict(off=C)])
def test_sort_refusals(bad):
    a = dict(ids=A, tokens=16, topk=2, experts=8, off=B, pos=C, space=D, nb=BIG)
    a.update(bad)
    assert exl3.load().exl3_moe_sort(*a.values(), None) == INV


def test_sort_workspace():
    need = exl3.exl3_moe_sort_workspace_size(16, 2, 8)
    lib = exl3.load()
    assert lib.exl3_moe_sort(A, 16, 2, 8, B, C, None, BIG, None) == WS
    assert lib.exl3_moe_sort(A, 16, 2, 8, B, C, D, need - 1, None) == WS
    assert exl3.exl3_moe_sort_workspace_size(16, 0, 8) == 0


ROUTE = [dict(dtype=3), dict(tokens=-1), dict(topk=0), dict(h=0), dict(rows=-1), dict(pos=None), dict(pos=B + 4)]


@pytest.mark.parametrize("bad", ROUTE + [dict(x=None), dict(x=MIS), dict(xs=None), dict(xs=C + 2), dict(xs=A), dict(xs=B)])
def test_gather_refusals(bad):
    a = dict(x=A, dtype=0, pos=B, tokens=4, topk=2, h=16, rows=8, xs=C)
    a.update(bad)
    assert exl3.load().exl3_moe_gather(*a.values(), None) == INV


@pytest.mark.parametrize("bad", ROUTE + [dict(ys=None), dict(w=D + 4), dict(y=None), dict(y=A), dict(y=B), dict(y=D), dict(ydt=1), dict(ydt=2),
                                         dict(dtype=2, ydt=3)])
def test_combine_refusals(bad):
    a = dict(ys=A, dtype=0, pos=B, w=D, tokens=4, topk=2, h=16, rows=8, y=C, ydt=0)
    a.update(bad)
    assert exl3.load().exl3_moe_combine(*a.values(), None) == INV


@pytest.mark.parametrize("bad", ROUTE + [dict(dy=None), dict(ys=None), dict(w=D + 8), dict(dys=E + 4), dict(dw=F + 4),
                                         dict(dys=None, dw=None), dict(dys=A), dict(dys=G), dict(dw=B), dict(dw=E)])
def test_combine_grad_refusals(bad):
    a = dict(dy=A, ys=G, dtype=0, pos=B, w=D, tokens=4, topk=2, h=16, rows=8, dys=E, dw=F)
    a.update(bad)
    assert exl3.load().exl3_moe_combine_grad(*a.values(), None) == INV


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((4, 64))
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    sc = torch.zeros((4, 16), dtype=torch.uint8)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        exl3.exl3_mx4_quantize(x)
    with pytest.raises(ValueError):
        exl3.exl3_mx4_quantize(torch.zeros(64))
    with pytest.raises(ValueError):
        exl3.exl3_mx4_dequantize(u8, sc[:, :8])
    with pytest.raises(ValueError):
        exl3.exl3_mx4_matmul(u8, sc, torch.zeros((4, 48), dtype=torch.uint8), sc)
    with pytest.raises(TypeError):
        exl3.exl3_moe_gather(x, pos)
    with pytest.raises(ValueError):
        exl3.exl3_moe_gather(x, pos[:3])
    with pytest.raises(ValueError):
        exl3.exl3_moe_combine_grad(x, torch.zeros((8, 32)), pos)


def test_oracles_agree_with_the_definitions():
    """The oracle's own checks: every magnitude is its own code, ties go to the
    even code, packing is undone by unpacking, the rotation is orthogonal, and
    the routing of a small case is that written out by hand."""
    v = np.concatenate([mx4.MAGNITUDE, -mx4.MAGNITUDE, mx4.MAGNITUDE, -mx4.MAGNITUDE])[None, :]
    c, s = mx4.quantize(v)
    assert s[0, 0] == 127 and np.array_equal(mx4.values(c, s), v)
    ties = np.zeros((1, 32))
    ties[0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5]
    c, s = mx4.quantize(ties)
    assert np.array_equal(mx4.values(c, s)[0, :8], [0, 1, 1, 2, 2, 4, 4, 6])
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (3, 160)).astype(np.uint8)
    s = rng.integers(0, 256, (3, 5)).astype(np.uint8)
    uc, us = mx4.unpack(*mx4.pack(c, s))
    assert np.array_equal(uc, c) and np.array_equal(us, s)
    x = rng.standard_normal((2, 256))
    assert np.allclose(mx4.rotate(mx4.rotate(x)), x) and np.allclose((mx4.rotate(x) ** 2).sum(), (x ** 2).sum())
    offsets, pos = moe.sort(np.array([[2, 0], [0, -1], [2, 7]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4] and pos.tolist() == [[2, 0], [1, -1], [3, -1]]
