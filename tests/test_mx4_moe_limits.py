"""The sizes that the header states for the 4-bit and routing calls: one past each
is turned away before anything is launched (no GPU; no address is dereferenced)."""
import pytest

from trellis_coded_bit_b200 import exl3

A, B, C, D, E, F, G = (i << 44 for i in range(1, 8))  # aligned, far apart
INV = exl3.EXL3_ERR_INVALID_ARG
ROUTE = [dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(topk=0), dict(topk=1025), dict(h=0), dict(h=(1 << 22) + 1),
         dict(rows=-1), dict(rows=(1 << 31) + 1)]


@pytest.mark.parametrize("bad", ROUTE)
def test_routing(bad):
    a = dict(tokens=4, topk=2, h=16, rows=8)
    a.update(bad)
    t, k, h, r = a.values()
    lib = exl3.load()
    assert lib.exl3_moe_gather(A, 0, B, t, k, h, r, C, None) == INV
    assert lib.exl3_moe_combine(A, 0, B, D, t, k, h, r, C, 0, None) == INV
    assert lib.exl3_moe_combine_grad(A, G, 0, B, D, t, k, h, r, E, F, None) == INV


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=-1), dict(n=(1 << 24) + 1), dict(m=-1), dict(m=(1 << 30) + 1),
                                 dict(k=(1 << 22) + 32), dict(k=33)])
def test_products(bad):
    a = dict(m=4, k=256, n=64)
    a.update(bad)
    m, k, n = a.values()
    lib = exl3.load()
    assert lib.exl3_mx4_matmul(A, B, C, D, E, 0, m, k, n, F, 1 << 40, None) == INV
    assert lib.exl3_mx4_linear(A, 0, None, 0, C, D, E, m, k, n, F, 1 << 40, None) == INV
    assert lib.exl3_mx4_matmul_experts(A, B, G, C, D, E, 0, m, k, n, 2, F, 1 << 40, None) == INV
    assert lib.exl3_mx4_matmul_experts(A, B, G, C, D, E, 0, 4, 256, (1 << 21) + 1, 512, F, 1 << 40, None) == INV


@pytest.mark.parametrize("bad", [dict(topk=0), dict(topk=1025), dict(out_rows=(1 << 30) + 1), dict(rows=(1 << 30) + 1)])
def test_quantize_into_positions(bad):
    a = dict(topk=2, out_rows=8, rows=4)
    a.update(bad)
    assert exl3.load().exl3_mx4_quantize(A, 0, None, 0, B, a["topk"], a["out_rows"], C, D, a["rows"], 256, None) == INV
