"""Codes behind the rotation where even the fp64 sums are rounded: bf16 values of
one group that span more than 53 bits, whose sum lies within a few of fp64's last
bits of a tie between codes.  The quantiser and a layer that quantises its own
tokens have to take the same code (one order of additions in both)."""
import numpy as np
import pytest
import torch

from trellis_coded_bit_b200 import exl3

TIE, SCALE = 5.0, 0.088388347648318440550  # between the codes of 4 and 6; 1/sqrt(128)


def bf16(v):
    return torch.tensor(v, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def tree(v):
    """Neighbours first: the order of a butterfly."""
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v[..., 0]


def in_turn(v):
    """Each 32 columns one after the other, then the four sums as a tree."""
    v = v.reshape(4, 32)
    s = np.zeros(4)
    for c in range(32):
        s = s + v[:, c]
    return tree(s)


def group(rng):
    """128 bf16 values for which the two orders give values on two sides of the
    tie (or on it and beside it) in column 0 of their rotation."""
    while True:
        x = bf16(rng.standard_normal(128) * 2.0 ** -47)
        left = TIE / SCALE
        for c in rng.choice(128, 6, replace=False):
            x[c] = bf16(left)
            left -= x[c]
        x[rng.integers(128)] = bf16(rng.standard_normal() * 2.0 ** -45)
        a, b = tree(x) * SCALE, in_turn(x) * SCALE
        if abs(a - TIE) < 1e-12 and abs(b - TIE) < 1e-12 and (a > TIE) != (b > TIE):
            return x


def test_such_groups_exist():
    x = group(np.random.default_rng(0))
    assert np.array_equal(bf16(x), x) and tree(x) != in_turn(x)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,n", [(1, 512, 64), (2, 2048, 300)])
def test_layer_and_quantiser_agree(m, k, n):
    exl3.load()
    rng = np.random.default_rng(m)
    x = torch.from_numpy(np.stack([np.concatenate([group(rng) for _ in range(k // 128)]) for _ in range(m)]))
    x = x.to(torch.bfloat16).cuda()
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda())
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    y = exl3.exl3_mx4_linear(x, wc, wsc, rotate=True, workspace=ws)
    xc, xs = exl3.exl3_mx4_quantize(x, rotate=True)
    assert torch.equal(y, exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=torch.bfloat16, workspace=ws))
