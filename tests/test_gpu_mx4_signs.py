"""4-bit quantisation with signs that are not +-1 (any fp16 numbers that multiply
x's columns): codes and scales have to be those of the exact products, without the
rotation and behind it, in the quantiser and in a layer that quantises its own
tokens.  A code is a whole number: nothing may differ."""
import numpy as np
import pytest
import torch

from oracle import mx4
from trellis_coded_bit_b200 import exl3

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    exl3.load()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().double().numpy()


def make_signs(rng, k, kind):
    s = rng.choice([-1.0, 1.0], k)
    if kind != "one in 64":
        part = rng.random(k) < 0.7
        s[part] = rng.uniform(-2, 2, part.sum())
        s[rng.random(k) < 0.05] = 0.0
    else:  # most lanes see +-1 alone, some do not
        s[::64] = rng.uniform(0.5, 1.5, len(s[::64]))
    return torch.from_numpy(s).half()


def beside_ties(rng, x, s, dtype):
    """Some columns of x as near as the type comes to a border between codes,
    divided by the column's sign; the block's largest stays in [4, 8)."""
    x = x.double().numpy().copy()
    sv = s.double().numpy()
    for b in range(x.shape[1] // 32):
        cols = 32 * b + rng.choice(32, 12, replace=False)
        for row in range(x.shape[0]):
            for c in cols[:11]:
                if sv[c]:
                    x[row, c] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * rng.choice([-1, 1]) / sv[c]
            top = cols[11] if sv[cols[11]] else cols[0]
            x[row, top] = 6.0 / sv[top] if sv[top] else 0.0
    return torch.from_numpy(x).to(dtype)


def same(codes, scales, v):
    """The codes and scales of the exact products v (numpy, fp64)."""
    rc, rs = mx4.quantize(v)
    gc, gs = mx4.unpack(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(gs, rs)
    assert np.array_equal(mx4.values(gc, gs), mx4.values(rc, rs), equal_nan=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["any", "one in 64"])
@pytest.mark.parametrize("rows,k", [(1, 32), (5, 416), (40, 1024)])
def test_without_rotation(dtype, kind, rows, k):
    rng = np.random.default_rng(rows + k)
    s = make_signs(rng, k, kind)
    x = beside_ties(rng, torch.from_numpy(rng.uniform(-4, 4, (rows, k))), s, dtype)
    codes, scales = exl3.exl3_mx4_quantize(x.cuda(), signs=s.cuda())
    same(codes, scales, x.double().numpy() * s.double().numpy())


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("rotate", [False, True])
def test_products_outside_fp32(dtype, rotate):
    """Finite products above fp32's range and below its smallest numbers."""
    k = 256
    rng = np.random.default_rng(3)
    x = np.zeros((6, k))
    x[0] = torch.finfo(dtype).max
    x[1, :40] = -3.0e38
    x[2] = rng.uniform(1, 2, k) * 2.0 ** -125
    x[3] = rng.uniform(1, 2, k) * 2.0 ** -132
    x[4] = 2.0 ** -130
    x[5, 7] = np.inf
    s = np.full(k, 7.0)
    s[1::2] = -0.3
    s[64:96] = 2.0 ** -20
    x, s = torch.from_numpy(x).to(dtype), torch.from_numpy(s).half()
    codes, scales = exl3.exl3_mx4_quantize(x.cuda(), signs=s.cuda(), rotate=rotate)
    xv, sv = x.double().numpy(), s.double().numpy()
    if rotate:
        xv[5, 7] = 0.0  # (the oracle's rotation is a product with zeros in it: without the infinity)
        want = mx4.rotate(xv, sv)
        want[5, :128] = np.nan
        want[5, 128:] = 0.0
        same(codes, scales, want)
    else:
        same(codes, scales, xv * sv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["any", "one in 64"])
@pytest.mark.parametrize("rows,k", [(1, 128), (5, 640), (33, 1024)])
def test_behind_the_rotation(dtype, kind, rows, k):
    rng = np.random.default_rng(rows + k)
    s = make_signs(rng, k, kind)
    x = torch.from_numpy(rng.standard_normal((rows, k))).to(dtype)
    codes, scales = exl3.exl3_mx4_quantize(x.cuda(), signs=s.cuda(), rotate=True)
    same(codes, scales, mx4.rotate(x.double().numpy(), s.double().numpy()))


def ties_behind_the_rotation(rng, rows, k, s, dtype):
    """x whose products with s, rotated, hold values within 2^-18 of the tie
    between the codes 4 and 6 (5 times sqrt(128) at four columns of a group, whose
    sum is one value; three of the columns have sign 1)."""
    x = torch.from_numpy(rng.standard_normal((rows, k))).to(dtype)
    sv = s.double()
    for row in range(rows):
        for g in range(row % 2, k // 128, 2):
            left = 5.0 * np.sqrt(128.0)
            x[row, 128 * g:128 * (g + 1)] = 0
            for col in (1, 32, 64, 96):
                part = torch.tensor(left / float(sv[128 * g + col]), dtype=torch.float64).to(dtype)
                x[row, 128 * g + col] = part
                left -= float(part) * float(sv[128 * g + col])
    return x


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("m,k,n,rotate", [(1, 512, 300, True), (2, 512, 300, True), (1, 2048, 2048, True), (2, 4096, 520, True),
                                          (5, 512, 136, True), (1, 544, 77, False), (2, 2080, 4097, False), (9, 96, 40, False)])
def test_layer(dtype, m, k, n, rotate):
    """A layer of a token or two quantises them itself: the product with the
    oracle's codes, bit for bit."""
    rng = np.random.default_rng(m + k + n)
    s = make_signs(rng, k, "any")
    if rotate:
        for col in (1, 32, 64, 96):
            s[col::128] = 0.77 if col == 1 else 1.0
        x = ties_behind_the_rotation(rng, m, k, s, dtype)
        v = mx4.rotate(x.double().numpy(), s.double().numpy())
    else:
        x = beside_ties(rng, torch.from_numpy(rng.uniform(-4, 4, (m, k))), s, dtype)
        if dtype == torch.bfloat16:
            x[0, :32] = 3.0e38  # products above fp32's range
        v = x.double().numpy() * s.double().numpy()
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda())
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    y = exl3.exl3_mx4_linear(x.cuda(), wc, wsc, signs=s.cuda(), rotate=rotate, workspace=ws)
    xc, xs = (dev(a) for a in mx4.pack(*mx4.quantize(v)))
    want = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=dtype, workspace=ws)
    assert torch.equal(torch.nan_to_num(y.float(), nan=77.0), torch.nan_to_num(want.float(), nan=77.0))


@pytest.mark.parametrize("dtype", TYPES[1:])
def test_rotated_products_below_normal_numbers(dtype):
    """One or a few columns that make the block's scale and 120 whose products fp32
    can only round to multiples of 2^-149, for scales from the smallest on."""
    rng = np.random.default_rng(8)
    k, rows = 256, 96
    x = rng.uniform(-1, 1, (rows, k)) * 2.0 ** -127
    for r in range(rows):
        x[r, rng.choice(k, 6, replace=False)] = rng.uniform(1, 2, 6) * 2.0 ** (-122 + r // 4)
    s = torch.from_numpy(rng.uniform(0.5, 1, k)).half()
    x = torch.from_numpy(x).to(dtype)
    codes, scales = exl3.exl3_mx4_quantize(x.cuda(), signs=s.cuda(), rotate=True)
    same(codes, scales, mx4.rotate(x.double().numpy(), s.double().numpy()))
