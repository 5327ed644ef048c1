"""4-bit microscaled matrices (exl3_mx4_*) against plain numpy in 64 bits.

Quantisation has to give the definition's codes exactly.  A product of two
4-bit matrices is one rounding to the output type (half a step, eps/2 of the
value) of an fp32 sum of k exact products; k additions, each off by at most
2^-23 of the sum of magnitudes S (a truncating adder), give k 2^-23 S.  With
equal scales every partial sum is a multiple of a quarter below 2^22, so the
fp32 sum is exact and the output must be the rounded exact value.
"""
import numpy as np
import pytest
import torch

from oracle import moe, mx4
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


def unpacked(codes, scales):
    return mx4.unpack(codes.cpu().numpy(), scales.cpu().numpy())


# ------------------------------------------------------------ quantisation ---

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (17, 160), (2, 512), (5, 544), (4, 4096), (300, 96)])
def test_quantize(dtype, rows, k):
    rng = np.random.default_rng(rows * k)
    x = torch.from_numpy(rng.standard_normal((rows, k)) * 10.0 ** rng.integers(-3, 3, (rows, 1))).to(dtype).cuda()
    codes, scales = exl3.exl3_mx4_quantize(x)
    rc, rs = mx4.quantize(host(x))
    gc, gs = unpacked(codes, scales)
    assert np.array_equal(gs, rs) and np.array_equal(gc, rc)
    assert not scales[:, k // 32:].any()
    for out in TYPES:
        assert torch.equal(exl3.exl3_mx4_dequantize(codes, scales, dtype=out).cpu(),
                           torch.from_numpy(mx4.values(rc, rs)).to(out))


def test_quantize_borders():
    """Every border of the rounding, its fp32 neighbours, both signs, at scales
    from the smallest to the largest; ties go to the even code."""
    borders = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.9999995],
                       dtype=np.float32)
    around = np.concatenate([borders, np.nextafter(borders, np.float32(9)), np.nextafter(borders, np.float32(-9))])
    around = np.concatenate([around, -around]).astype(np.float32)
    rows = []
    for e in (-126, -100, -1, 0, 1, 60, 125):
        for i in range(0, len(around), 31):
            part = np.zeros(32, dtype=np.float32)
            part[:len(around[i:i + 31])] = around[i:i + 31]
            part[31] = 4.0  # keeps the block's largest magnitude in [4, 8)
            rows.append(np.ldexp(part, e))
    x = np.stack(rows).astype(np.float32)
    rc, rs = mx4.quantize(x)
    gc, gs = unpacked(*exl3.exl3_mx4_quantize(dev(x)))
    assert np.array_equal(gs, rs) and np.array_equal(gc, rc)


def test_quantize_extremes():
    """Zeros, the smallest and largest values, infinities and NaN."""
    x = np.zeros((12, 64), dtype=np.float32)
    x[1, 3] = -0.0
    x[2, :] = np.float32(1e-45)
    x[3, :] = np.float32(-3e-39)
    x[4, :] = np.finfo(np.float32).max
    x[5, ::2] = np.float32(1.2e-38)
    x[6, 40] = np.inf
    x[7, 2] = np.nan
    x[8, 63] = -np.inf
    x[9, :32] = np.float32(2.0 ** -126)
    x[10, :] = np.float32(2.0 ** 127)
    x[11, :32] = np.finfo(np.float32).tiny * 3
    codes, scales = exl3.exl3_mx4_quantize(dev(x))
    rc, rs = mx4.quantize(x)
    gc, gs = unpacked(codes, scales)
    assert np.array_equal(gs, rs) and np.array_equal(gc, rc)
    back = exl3.exl3_mx4_dequantize(codes, scales, dtype=torch.float32).cpu().numpy()
    assert np.array_equal(back, mx4.values(rc, rs).astype(np.float32), equal_nan=True)
    assert np.isnan(back[6, 32:]).all() and np.isfinite(back[6, :32]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,signed", [(1, 128, True), (5, 384, False), (33, 1024, True), (2, 8192, True)])
def test_quantize_rotated(dtype, rows, k, signed):
    rng = np.random.default_rng(k + rows)
    x = rng.standard_normal((rows, k))
    x[:, rng.choice(k, k // 64, replace=False)] *= 20
    x = torch.from_numpy(x).to(dtype).cuda()
    signs = torch.from_numpy(rng.choice([-1.0, 1.0], k)).half().cuda() if signed else None
    codes, scales = exl3.exl3_mx4_quantize(x, signs=signs, rotate=True)
    rc, rs = mx4.quantize(mx4.rotate(host(x), None if signs is None else host(signs)))
    assert np.array_equal(mx4.values(*unpacked(codes, scales)), mx4.values(rc, rs))


def test_quantize_rotated_extremes():
    x = np.zeros((6, 256), dtype=np.float32)
    x[0, 0] = np.inf
    x[1, 130] = np.nan
    x[2, :] = np.finfo(np.float32).max   # the sum leaves fp32, the scale its range
    x[3, 5] = 1e-45
    x[4, :128] = 1.0                     # one coefficient, 127 exact zeros
    codes, scales = exl3.exl3_mx4_quantize(dev(x), rotate=True)
    gc, gs = unpacked(codes, scales)
    assert (gs[0, :4] == 255).all() and (gs[0, 4:] == 0).all() and (gs[1, 4:] == 255).all()
    rc, rs = mx4.quantize(mx4.rotate(x[2:]))
    assert np.array_equal(gs[2:], rs) and np.array_equal(mx4.values(gc, gs)[2:], mx4.values(rc, rs))


def test_quantize_signs_without_rotation():
    rng = np.random.default_rng(3)
    x, s = rng.standard_normal((4, 96)).astype(np.float16), rng.choice([-1.0, 1.0], 96).astype(np.float16)
    rc, rs = mx4.quantize(x.astype(np.float64) * s)
    gc, gs = unpacked(*exl3.exl3_mx4_quantize(dev(x), signs=dev(s)))
    assert np.array_equal(gc, rc) and np.array_equal(gs, rs)


@pytest.mark.parametrize("rotate", [False, True])
def test_quantize_into_positions(rotate):
    rng = np.random.default_rng(4)
    rows, topk, k, out_rows = 9, 3, 640, 20
    x = rng.standard_normal((rows, k)).astype(np.float32)
    pos = np.full(rows * topk, -1, dtype=np.int32)
    named = rng.choice(rows * topk, 15, replace=False)
    pos[named] = rng.permutation(out_rows)[:15]
    pos[[i for i in range(rows * topk) if i not in named][:2]] = [out_rows, 2 ** 31 - 1]  # outside: skipped
    pos = pos.reshape(rows, topk)
    codes = torch.full((out_rows, k // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((out_rows, mx4.stride(k)), 0xA5, dtype=torch.uint8, device="cuda")
    exl3.exl3_mx4_quantize(dev(x), rotate=rotate, positions=dev(pos), out_rows=out_rows, codes=codes, scales=scales)
    pc, ps = exl3.exl3_mx4_quantize(dev(x), rotate=rotate)
    seen = set()
    for r in range(rows):
        for p in pos[r]:
            if 0 <= p < out_rows:
                assert torch.equal(codes[p], pc[r]) and torch.equal(scales[p], ps[r])
                seen.add(int(p))
    rest = [r for r in range(out_rows) if r not in seen]
    assert (codes[rest] == 0xA5).all() and (scales[rest] == 0xA5).all()


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(32) % 16, (256, 1)).astype(np.uint8)
    scales = np.arange(256, dtype=np.uint8)[:, None]
    pc, ps = (dev(a) for a in mx4.pack(codes, scales))
    ref = torch.from_numpy(mx4.values(codes, scales))
    for dtype in TYPES:
        out = exl3.exl3_mx4_dequantize(pc, ps, dtype=dtype).cpu()
        assert torch.equal(torch.nan_to_num(out.float(), nan=77.0), torch.nan_to_num(ref.to(dtype).float(), nan=77.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_onto_16_byte_alignment(dtype):
    """An output that starts on 16 bytes but not on 32."""
    rng = np.random.default_rng(6)
    c, s = operand(rng, 5, 96, 100, 140)
    pc, ps = (dev(a) for a in mx4.pack(c, s))
    skip = 16 // torch.empty((), dtype=dtype).element_size()
    buf = torch.zeros(5 * 96 + 2 * skip, dtype=dtype, device="cuda")
    out = buf[skip:skip + 5 * 96].view(5, 96)
    assert out.data_ptr() % 32 == 16
    exl3.exl3_mx4_dequantize(pc, ps, out=out)
    assert torch.equal(out.cpu(), torch.from_numpy(mx4.values(c, s)).to(dtype))
    assert not buf[:skip].any() and not buf[-skip:].any()


# ----------------------------------------------------------------- product ---

def operand(rng, rows, k, low=127, high=127):
    """Random codes, scale bytes in [low, high]."""
    return rng.integers(0, 16, (rows, k)).astype(np.uint8), rng.integers(low, high + 1, (rows, k // 32)).astype(np.uint8)


def product(x, w, dtype, ws=None, **kw):
    m, k = x[0].shape
    n = w[0].shape[0]
    if ws is None:
        ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    y = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=dtype, workspace=ws, **kw)
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
    return y


SHAPES = [(1, 32, 1), (1, 256, 128), (1, 64, 5), (2, 96, 129), (16, 128, 128), (17, 288, 130), (15, 512, 64),
          (32, 1024, 200), (33, 256, 384), (64, 544, 257), (65, 2048, 100), (128, 320, 256), (129, 768, 300),
          (200, 4096, 128), (256, 256, 256), (257, 160, 131), (300, 4000, 1000), (1, 4096, 4096), (8, 14336, 512),
          (513, 512, 640), (40, 8192, 77),
          # pairs of CTAs: whole tiles, split tiles, odd rows and channels
          (520, 1536, 13001), (1100, 544, 9100), (2100, 96, 4360), (40000, 64, 272),
          # a long sum
          (3, 262144, 40),
          # tiles of fewer channels than 128, one or two for each SM, odd and cut ones
          (40, 4096, 4100), (100, 1536, 19001), (128, 640, 333), (20, 1056, 30011), (1, 4096, 14344), (64, 8192, 1000),
          # the same with several token tiles
          (129, 8192, 2056), (333, 4000, 5001), (1000, 1056, 700),
          # two or four parts of k side by side: whole, cut and missing ones, odd channels
          (1, 2048, 4096), (2, 2080, 1001), (3, 1056, 5000), (4, 4000, 4737), (5, 1088, 300), (8, 5632, 8192),
          (7, 2592, 2049), (4, 1184, 3), (1, 14336, 4000), (1, 8192, 9480)]


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_product_exact_with_equal_scales(m, k, n):
    """Each partial sum is exact in fp32: the output is the rounded exact value,
    whatever the tile, the split and the order."""
    rng = np.random.default_rng(m + k + n)
    x, w = operand(rng, m, k), operand(rng, n, k)
    ref = mx4.values(*x) @ mx4.values(*w).T
    assert np.abs(ref).max() < 60000
    for dtype in TYPES:
        assert torch.equal(product(x, w, dtype).cpu(), torch.from_numpy(ref).to(dtype))
    if m * n > 1 << 20:  # the same on pairs of CTAs or not: bit for bit on every call
        assert torch.equal(product(x, w, torch.float16), product(x, w, torch.float16))


@pytest.mark.parametrize("m,k,n", SHAPES)
def test_product_with_scales(m, k, n):
    """Every block has its own scale (the scale of another row, block or half
    would be off by powers of two)."""
    rng = np.random.default_rng(7 * m + k + n)
    x, w = operand(rng, m, k, 118, 130), operand(rng, n, k, 112, 124)
    y = host(product(x, w, torch.float16))
    xv, wv = mx4.values(*x), mx4.values(*w)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.abs(ref).max() < 60000
    # 2^-25: half a step of the smallest fp16 values
    assert np.all(np.abs(y - ref) <= 2.0 ** -11 * np.abs(ref) + k * 2.0 ** -23 * mag + 2.0 ** -25)
    assert np.all(np.abs(host(product(x, w, torch.float32)) - ref) <= k * 2.0 ** -23 * mag)


def test_product_scales_of_single_blocks():
    """One nonzero block per row of x, everything else zero: the product picks
    exactly that block's scale and codes."""
    k, n = 1088, 96
    m = k // 32
    rng = np.random.default_rng(11)
    w = operand(rng, n, k, 120, 134)
    xc = np.zeros((m, k), dtype=np.uint8)
    for b in range(m):
        xc[b, 32 * b + b % 32] = 2  # 1.0
    x = (xc, rng.integers(120, 135, (m, k // 32)).astype(np.uint8))
    y = host(product(x, w, torch.float16))
    assert np.array_equal(y, (mx4.values(*x) @ mx4.values(*w).T).astype(np.float16).astype(np.float64))


def test_product_nan_scale_stays_in_its_row():
    rng = np.random.default_rng(12)
    m, k, n = 20, 512, 140
    x, w = operand(rng, m, k), operand(rng, n, k)
    x[1][3, 5] = 255
    w[1][130, 0] = 255
    y = product(x, w, torch.float16).cpu().float().numpy()
    bad = np.zeros((m, n), dtype=bool)
    bad[3] = True
    bad[:, 130] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def test_padding_bytes_of_scales_are_not_read():
    """Bytes behind k/32 may hold anything, 255 included."""
    rng = np.random.default_rng(13)
    for m, k, n in ((3, 96, 40), (40, 288, 130)):
        x, w = operand(rng, m, k), operand(rng, n, k)
        xc, xs = (dev(a) for a in mx4.pack(*x))
        wc, wsc = (dev(a) for a in mx4.pack(*w))
        xs[:, k // 32:] = 255
        wsc[:, k // 32:] = 255
        ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
        y = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, workspace=ws)
        assert torch.equal(y.cpu(), torch.from_numpy(mx4.values(*x) @ mx4.values(*w).T).half())


def test_product_large_and_repeatable():
    """A prompt-sized product on sampled entries, twice the same bits with one
    workspace, which afterwards serves another shape and the trellis GEMM's calls."""
    rng = np.random.default_rng(14)
    m, k, n = 700, 4096, 5000
    x, w = operand(rng, m, k, 120, 127), operand(rng, n, k, 118, 124)
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    y = product(x, w, torch.bfloat16, ws)
    assert torch.equal(y, product(x, w, torch.bfloat16, ws))
    rows, cols = rng.integers(0, m, 4000), rng.integers(0, n, 4000)
    xv, wv = mx4.values(*x)[rows], mx4.values(*w)[cols]
    ref, mag = (xv * wv).sum(1), (np.abs(xv) * np.abs(wv)).sum(1)
    got = host(y)[rows, cols]
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * mag)
    x2, w2 = operand(rng, 3, 512), operand(rng, 300, 512)
    assert torch.equal(product(x2, w2, torch.float16, ws).cpu(),
                       torch.from_numpy(mx4.values(*x2) @ mx4.values(*w2).T).half())


@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("m,k,n,rotate", [(1, 4096, 512, True), (5, 256, 130, True), (70, 1024, 200, False),
                                          (1, 96, 33, False), (300, 512, 256, True), (2, 128, 40, True), (2, 1152, 4200, True),
                                          (2, 32, 300, False), (1, 1056, 129, False), (1, 2080, 4097, False), (2, 4096, 4096, True), (1, 8192, 5000, True), (1, 14336, 640, True), (3, 640, 128, True)])
def test_linear_is_quantize_then_product(dtype, m, k, n, rotate):
    rng = np.random.default_rng(m + n)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(dtype).cuda()
    x[0, 7] = 0.0
    signs = torch.from_numpy(rng.choice([-1.0, 1.0], k)).half().cuda() if rotate else None
    wm = rng.standard_normal((n, k)) * 0.02
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(wm).float().cuda(), signs=signs, rotate=rotate)
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    y = exl3.exl3_mx4_linear(x, wc, wsc, signs=signs, rotate=rotate, workspace=ws)
    xc, xs = exl3.exl3_mx4_quantize(x, signs=signs, rotate=rotate)
    assert torch.equal(y, exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=dtype, workspace=ws))
    # and it is the layer: the rotation cancels, what is left is the rounding
    # of both operands (relative 4-bit errors near 0.1 each, independent)
    if m * n > 500 and rotate:
        ref = host(x) @ wm.T
        assert np.linalg.norm(host(y) - ref) <= 0.25 * np.linalg.norm(ref)


@pytest.mark.parametrize("m", [1, 2, 9])
def test_linear_of_infinities_and_values_beside_borders(m):
    """A row with an infinity becomes NaN and leaves the others alone; a row
    whose rotated values lie on rounding borders takes the exact path."""
    rng = np.random.default_rng(50 + m)
    k, n = 512, 300
    x = np.zeros((m, k), dtype=np.float16)
    x[0, 0::128] = 1.0     # every rotated value 1/sqrt(128): the scale's border
    x[0, 130] = 2.0
    if m > 1:
        x[1, 5] = np.inf
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda())
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    y = exl3.exl3_mx4_linear(dev(x), wc, wsc, rotate=True, workspace=ws)
    xc, xs = exl3.exl3_mx4_quantize(dev(x), rotate=True)
    assert torch.equal(y[0], exl3.exl3_mx4_matmul(xc, xs, wc, wsc, workspace=ws)[0])
    assert torch.isfinite(y[0]).all() and (m == 1 or torch.isnan(y[1]).all()) and torch.isfinite(y[2:]).all()
    xq = mx4.values(*mx4.quantize(mx4.rotate(x[:1])))
    ref = xq @ mx4.values(*unpacked(wc, wsc)).T
    mag = np.abs(xq) @ np.abs(mx4.values(*unpacked(wc, wsc))).T
    assert np.all(np.abs(host(y[:1]) - ref) <= 2.0 ** -11 * np.abs(ref) + k * 2.0 ** -23 * mag + 2.0 ** -25)


# ----------------------------------------------------------------- experts ---

@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("m,k,n", [(1, 512, 300), (2, 512, 300), (1, 2048, 2048), (2, 4096, 520)])
def test_linear_of_codes_beside_ties(dtype, m, k, n):
    """Rotated values within 2^-24 of the tie between the codes 4 and 6, on both
    sides, whole blocks of them, some in every unit: the layer's own
    quantisation takes the codes of the exact sums."""
    rng = np.random.default_rng(k + m)
    x = torch.from_numpy(rng.standard_normal((m, k))).to(dtype)
    for row in range(m):
        for g in range(row, k // 128, 3):
            left = 5.0 * np.sqrt(128.0) + (g % 2 * 2 - 1) * 2.0 ** -21  # the tie, scaled by sqrt(128)
            x[row, 128 * g:128 * (g + 1)] = 0
            for col in (0, 32, 64, 96):   # one Walsh row is their sum; the others differ by signs
                part = torch.tensor(left, dtype=torch.float64).to(dtype)
                x[row, 128 * g + col] = part
                left -= float(part)
            assert abs(left) < 2.0 ** -20
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda())
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    y = exl3.exl3_mx4_linear(x.cuda(), wc, wsc, rotate=True, workspace=ws)
    codes, scales = mx4.quantize(mx4.rotate(host(x), None))
    xc, xs = (dev(v) for v in mx4.pack(codes, scales))
    assert torch.equal(y, exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=dtype, workspace=ws))


def experts_case(rng, counts, k, n, spare=0, low=120, high=127):
    counts = np.asarray(counts)
    rows = int(counts.sum()) + spare
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return offsets, operand(rng, rows, k, low, high), operand(rng, len(counts) * n, k, low, high)


@pytest.mark.parametrize("counts,k,n,spare", [([1], 64, 20, 0), ([0, 3, 0, 0, 1], 256, 130, 2), ([5, 0, 17, 2], 544, 100, 1),
                                              ([40, 1, 0, 90, 16], 512, 256, 0), ([300, 2, 130], 1024, 128, 7),
                                              ([0, 0], 128, 64, 4), ([1] * 40, 256, 48, 0), ([700, 1, 300], 256, 200, 0),
                                              ([900, 0, 257, 1500, 3, 640], 512, 3000, 5), ([200] * 16, 288, 2600, 0),
                                              ([3], 2112, 1000, 1), ([2], 4096, 2049, 2), ([100], 4096, 300, 2)])
def test_experts(counts, k, n, spare):
    rng = np.random.default_rng(sum(counts) + k)
    offsets, x, w = experts_case(rng, counts, k, n, spare)
    e, rows = len(counts), len(x[0])
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_experts_workspace_size(rows, k, n, e))
    y = torch.full((rows, n), 5.0, dtype=torch.float16, device="cuda")
    for _ in range(2):
        exl3.exl3_mx4_matmul_experts(xc, xs, dev(offsets), wc.view(e, n, -1), wsc.view(e, n, -1), y=y, workspace=ws)
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
    xv, wv = mx4.values(*x), mx4.values(*w).reshape(e, n, k)
    got = host(y)
    for i in range(e):
        r = slice(offsets[i], offsets[i + 1])
        ref, mag = xv[r] @ wv[i].T, np.abs(xv[r]) @ np.abs(wv[i]).T
        assert np.all(np.abs(got[r] - ref) <= 2.0 ** -11 * np.abs(ref) + k * 2.0 ** -23 * mag + 2.0 ** -25)
    assert np.all(got[offsets[-1]:] == 5.0)  # rows behind the last expert keep what they held


def test_experts_offsets_outside_the_rows():
    """Offsets above the rows are taken to the end, none is read or written outside."""
    rng = np.random.default_rng(21)
    k, n = 256, 64
    x, w = operand(rng, 10, k), operand(rng, 3 * n, k)
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_experts_workspace_size(10, k, n, 3))
    off = torch.tensor([0, 4, 1000, 2000], dtype=torch.int32, device="cuda")
    y = exl3.exl3_mx4_matmul_experts(xc, xs, off, wc.view(3, n, -1), wsc.view(3, n, -1), workspace=ws)
    xv, wv = mx4.values(*x), mx4.values(*w).reshape(3, n, k)
    ref = np.concatenate([xv[:4] @ wv[0].T, xv[4:] @ wv[1].T])
    assert torch.equal(y.cpu(), torch.from_numpy(ref).half())


def test_more_than_32_bits_of_elements():
    """Matrices whose element offsets pass 2^31: the last rows against the same rows alone."""
    rows, k = 600000, 4096
    x = torch.zeros((rows, k), dtype=torch.float16, device="cuda")
    x[-3:] = torch.randn((3, k), device="cuda").half()
    codes, scales = exl3.exl3_mx4_quantize(x, rotate=True)
    c3, s3 = exl3.exl3_mx4_quantize(x[-3:].clone(), rotate=True)
    assert torch.equal(codes[-3:], c3) and torch.equal(scales[-3:], s3) and not codes[:-3].any()
    assert torch.equal(exl3.exl3_mx4_dequantize(codes, scales, out=x)[-3:], exl3.exl3_mx4_dequantize(c3, s3))
    codes, scales = exl3.exl3_mx4_quantize(x)
    assert torch.equal(codes[-3:], exl3.exl3_mx4_quantize(x[-3:].clone())[0])
    del x, codes, scales
    rng = np.random.default_rng(61)
    m, n, k = 70000, 32768, 64
    x, w = operand(rng, m, k), operand(rng, n, k)
    y = product(x, w, torch.float16)
    for r in (0, 65535, 65537, m - 1):
        ref = mx4.values(x[0][r:r + 1], x[1][r:r + 1]) @ mx4.values(*w).T
        assert torch.equal(y[r].cpu(), torch.from_numpy(ref[0]).half())


def test_captured_expert_layer():
    """The run of calls of an expert layer, captured once and replayed on other
    tokens, choices and weights in the same buffers."""
    rng = np.random.default_rng(23)
    tokens, topk, experts, k, n = 300, 2, 8, 256, 264
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((experts * n, k))).float().cuda(), rotate=True)
    wc, wsc = wc.view(experts, n, -1), wsc.view(experts, n, -1)
    x = torch.empty((tokens, k), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((tokens, topk), dtype=torch.int32, device="cuda")
    gate = torch.empty((tokens, topk), device="cuda")
    ws = exl3.new_workspace(max(exl3.exl3_moe_sort_workspace_size(tokens, topk, experts),
                                exl3.exl3_mx4_matmul_experts_workspace_size(tokens * topk, k, n, experts)))

    def layer():
        offsets, pos = exl3.exl3_moe_sort(ids, experts, workspace=ws)
        xc, xs = exl3.exl3_mx4_quantize(x, rotate=True, positions=pos, out_rows=tokens * topk)
        ys = exl3.exl3_mx4_matmul_experts(xc, xs, offsets, wc, wsc, dtype=torch.float32, workspace=ws)
        return exl3.exl3_moe_combine(ys, pos, weights=gate, dtype=torch.bfloat16)

    def fill(seed, one=None):
        r = np.random.default_rng(seed)
        x.copy_(torch.from_numpy(r.standard_normal((tokens, k))))
        chosen = r.integers(-1, experts, (tokens, topk)) if one is None else np.full((tokens, topk), one)
        ids.copy_(torch.from_numpy(chosen.astype(np.int32)))
        gate.copy_(torch.from_numpy(r.random((tokens, topk))))

    fill(1)
    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for seed, one in ((2, None), (3, 7), (4, -1)):  # mixed, one expert takes all, none chosen
        fill(seed, one)
        graph.replay()
        got = y.clone()
        assert torch.equal(got, layer())
        assert one != -1 or not got.any()
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK


def test_expert_layer():
    """The run of calls a mixture-of-experts layer makes, against the same in 64 bits."""
    rng = np.random.default_rng(22)
    tokens, topk, experts, k, n = 37, 2, 6, 256, 384
    ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    ids[5] = -1
    x = rng.standard_normal((tokens, k)).astype(np.float16)
    signs = rng.choice([-1.0, 1.0], k).astype(np.float16)
    wm = (rng.standard_normal((experts * n, k)) * 0.05).astype(np.float32)
    gate = rng.random((tokens, topk)).astype(np.float32)
    rows = tokens * topk
    ws = exl3.new_workspace(max(exl3.exl3_moe_sort_workspace_size(tokens, topk, experts),
                                exl3.exl3_mx4_matmul_experts_workspace_size(rows, k, n, experts)))
    wc, wsc = exl3.exl3_mx4_quantize(dev(wm), signs=dev(signs), rotate=True)
    offsets, pos = exl3.exl3_moe_sort(dev(ids), experts, workspace=ws)
    xc, xs = exl3.exl3_mx4_quantize(dev(x), signs=dev(signs), rotate=True, positions=pos, out_rows=rows)
    ys = exl3.exl3_mx4_matmul_experts(xc, xs, offsets, wc.view(experts, n, -1), wsc.view(experts, n, -1), workspace=ws)
    y = host(exl3.exl3_moe_combine(ys, pos, weights=dev(gate)))
    ys32 = exl3.exl3_mx4_matmul_experts(xc, xs, offsets, wc.view(experts, n, -1), wsc.view(experts, n, -1),
                                        dtype=torch.float32, workspace=ws)
    once = host(exl3.exl3_moe_combine(ys32, pos, weights=dev(gate), dtype=torch.float16))
    xv = mx4.values(*mx4.quantize(mx4.rotate(x, signs)))
    wv = mx4.values(*mx4.quantize(mx4.rotate(wm, signs))).reshape(experts, n, k)
    ref, mag = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        for j in range(topk):
            if ids[t, j] >= 0:
                ref[t] += gate[t, j] * (wv[ids[t, j]] @ xv[t])
                mag[t] += gate[t, j] * (np.abs(wv[ids[t, j]]) @ np.abs(xv[t]))
    # two roundings to fp16 (an expert's output, the sum), fp32 sums of k and topk terms
    assert np.all(np.abs(y - ref) <= (2 * 2.0 ** -11 + (k + topk) * 2.0 ** -23) * mag + 2.0 ** -24)
    # fp32 between the two calls: one rounding
    assert np.all(np.abs(once - ref) <= 2.0 ** -11 * np.abs(ref) + (k + topk) * 2.0 ** -23 * mag + 2.0 ** -25)
    assert not y[5].any()


# ------------------------------------------------------------ how it is called ---

@pytest.mark.parametrize("m,k,n", [(20, 2048, 2000), (600, 2048, 14000)])  # single CTAs, and pairs
def test_timeout_is_reported_and_cleared(m, k, n):
    rng = np.random.default_rng(30)
    x, w = operand(rng, m, k), operand(rng, n, k)
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    exl3.exl3_debug_set_wait_limit_ns(1)
    try:
        exl3.exl3_mx4_matmul(xc, xs, wc, wsc, workspace=ws)
        assert exl3.exl3_workspace_status(ws, clear=True) == exl3.EXL3_ERR_TIMEOUT
    finally:
        exl3.exl3_debug_set_wait_limit_ns(0)
    y = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, workspace=ws)
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
    cols = rng.integers(0, n, 500)
    assert torch.equal(y[:, dev(cols)].cpu(), torch.from_numpy(mx4.values(*x) @ mx4.values(*w)[cols].T).half())


@pytest.mark.parametrize("flags", [0, exl3.EXL3_LAUNCH_PDL])
def test_side_stream_graph_and_overlapped_launches(flags):
    """A captured layer replayed on new inputs, with and without overlapped
    launches, equals the plain calls; two graphs keep a workspace each."""
    rng = np.random.default_rng(31)
    m, k, n = 3, 1024, 700
    x = torch.from_numpy(rng.standard_normal((m, k))).half().cuda()
    layers = [exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k)) * 0.02).float().cuda()) for _ in range(2)]
    torch.cuda.synchronize()
    nb = exl3.exl3_mx4_linear_workspace_size(m, k, n)
    outs, graphs, spaces = [], [], []
    exl3.exl3_set_launch_flags(flags)
    try:
        for wc, wsc in layers:
            ws = exl3.new_workspace(nb)
            y = torch.empty((m, n), dtype=torch.float16, device="cuda")
            exl3.exl3_mx4_linear(x, wc, wsc, rotate=True, y=y, workspace=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(3):
                    exl3.exl3_mx4_linear(x, wc, wsc, rotate=True, y=y, workspace=ws)
            outs.append(y)
            graphs.append(g)
            spaces.append(ws)
        side = torch.cuda.Stream()
        for _ in range(3):
            x.copy_(torch.from_numpy(rng.standard_normal((m, k))).half())
            torch.cuda.synchronize()
            graphs[0].replay()
            with torch.cuda.stream(side):
                graphs[1].replay()
            torch.cuda.synchronize()
            for (wc, wsc), y in zip(layers, outs):
                plain = exl3.exl3_mx4_linear(x, wc, wsc, rotate=True, workspace=exl3.new_workspace(nb), stream=side)
                side.synchronize()
                assert torch.equal(plain, y)
    finally:
        exl3.exl3_set_launch_flags(0)


GUARD = 4096


class Guarded:
    """A device buffer between two 4 KiB regions of a byte pattern."""

    def __init__(self, shape, dtype, zero=False):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.n = n
        self.buf = torch.full((2 * GUARD + n,), 0xA5, dtype=torch.uint8, device="cuda")
        body = self.buf[GUARD:GUARD + n]
        if zero:
            body.zero_()
        self.view = body.view(dtype).view(shape)

    def intact(self):
        torch.cuda.synchronize()
        return bool((self.buf[:GUARD] == 0xA5).all()) and bool((self.buf[GUARD + self.n:] == 0xA5).all())


@pytest.mark.parametrize("m,k,n", [(1, 32, 8), (3, 160, 40), (17, 256, 136), (130, 512, 264), (260, 96, 8)])
def test_no_write_outside(m, k, n):
    rng = np.random.default_rng(m)
    x = torch.from_numpy(rng.standard_normal((m, k))).half().cuda()
    codes, scales = Guarded((m, k // 2), torch.uint8), Guarded((m, mx4.stride(k)), torch.uint8)
    exl3.exl3_mx4_quantize(x, codes=codes.view, scales=scales.view)
    back = Guarded((m, k), torch.float16)
    exl3.exl3_mx4_dequantize(codes.view, scales.view, out=back.view)
    w = operand(rng, n, k)
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    y = Guarded((m, n), torch.float16)
    ws = Guarded((exl3.exl3_mx4_matmul_workspace_size(m, k, n),), torch.uint8, zero=True)
    for _ in range(2):
        exl3.exl3_mx4_matmul(codes.view, scales.view, wc, wsc, y=y.view, workspace=ws.view)
    ws2 = Guarded((exl3.exl3_mx4_linear_workspace_size(m, k, n),), torch.uint8, zero=True)
    y2 = Guarded((m, n), torch.float16)
    exl3.exl3_mx4_linear(x, wc, wsc, y=y2.view, workspace=ws2.view)
    off = dev(np.array([0, m // 2, m], dtype=np.int32))
    half = n // 2
    y3 = Guarded((m, half), torch.bfloat16)
    y4 = Guarded((m, n), torch.float32)
    exl3.exl3_mx4_matmul(codes.view, scales.view, wc, wsc, y=y4.view, workspace=ws.view)
    ws3 = Guarded((exl3.exl3_mx4_matmul_experts_workspace_size(m, k, half, 2),), torch.uint8, zero=True)
    exl3.exl3_mx4_matmul_experts(codes.view, scales.view, off, wc.view(2, half, -1), wsc.view(2, half, -1), y=y3.view,
                                 workspace=ws3.view)
    assert all(g.intact() for g in (codes, scales, back, y, ws, ws2, y2, y3, ws3, y4))
    assert torch.equal(y.view, y2.view)
