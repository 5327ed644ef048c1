"""Expert routing (exl3_moe_*) against plain numpy in 64 bits.

Tolerances: a 16-bit output is one rounding (half a step, eps/2 of the value)
of an fp32 sum; the fp32 sum of n products, each addition and product rounded
by 2^-24, is off by at most n 2^-23 of the sum of magnitudes (to first order).
"""
import numpy as np
import pytest
import torch

from oracle import moe
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
    return t.cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def workspace(tokens, topk, experts):
    return exl3.new_workspace(exl3.exl3_moe_sort_workspace_size(tokens, topk, experts))


def route(rng, tokens, topk, experts, lost=0.1):
    """ids with some choices outside the experts, and their rows."""
    ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    ids[rng.random((tokens, topk)) < lost] = -1
    return ids


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 128), (7, 3, 5), (33, 2, 1024), (512, 2, 8),
                                                 (1025, 1, 3), (1000, 6, 64), (70000, 4, 1024), (140001, 1, 33)])
def test_sort(tokens, topk, experts):
    rng = np.random.default_rng(tokens + topk)
    ids = route(rng, tokens, topk, experts)
    if tokens > 4:
        ids[3] = experts + 5  # behind the last expert: no row either
    ws = workspace(tokens, topk, experts)
    offsets, positions = exl3.exl3_moe_sort(dev(ids), experts, workspace=ws)
    ro, rp = moe.sort(ids, experts)
    assert np.array_equal(host(offsets), ro) and np.array_equal(host(positions), rp)
    assert not ws[:65536].any()  # the matmul calls' counters


@pytest.mark.parametrize("kind", ["one expert", "none", "descending"])
def test_sort_extremes(kind):
    tokens, topk, experts = 3000, 2, 16
    ids = {"one expert": np.full((tokens, topk), 7), "none": np.full((tokens, topk), -1),
           "descending": 15 - np.arange(tokens * topk).reshape(tokens, topk) * 16 // (tokens * topk)}[kind].astype(np.int32)
    offsets, positions = exl3.exl3_moe_sort(dev(ids), experts, workspace=workspace(tokens, topk, experts))
    ro, rp = moe.sort(ids, experts)
    assert np.array_equal(host(offsets), ro) and np.array_equal(host(positions), rp)


def test_no_tokens():
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    offsets, positions = exl3.exl3_moe_sort(ids, 4, workspace=workspace(0, 2, 4))
    assert not offsets.any() and positions.shape == (0, 2)
    x = torch.empty((0, 16), device="cuda")
    assert exl3.exl3_moe_gather(x, positions).shape == (0, 16)
    assert exl3.exl3_moe_combine(torch.zeros((3, 16), device="cuda"), positions).shape == (0, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,topk,experts,h", [(1, 1, 2, 1), (1, 8, 16, 4096), (5, 2, 3, 7), (65, 3, 8, 264),
                                                   (40, 8, 8, 1111), (300, 4, 32, 2048)])
def test_gather_combine_and_gradients(dtype, tokens, topk, experts, h):
    rng = np.random.default_rng(tokens * h + topk)
    ids = route(rng, tokens, topk, experts)
    _, pos = moe.sort(ids, experts)
    rows = tokens * topk + 3
    p = dev(pos)
    x = torch.from_numpy(rng.standard_normal((tokens, h))).to(dtype).cuda()
    fill = torch.full((rows, h), 9.0, dtype=dtype, device="cuda")
    xs = exl3.exl3_moe_gather(x, p, out=fill.clone())
    assert np.array_equal(host(xs), moe.gather(host(x), pos, host(fill)))  # copies, and the other rows as they were

    ys = torch.from_numpy(rng.standard_normal((rows, h))).to(dtype).cuda()
    ys[:][torch.from_numpy(np.setdiff1d(np.arange(rows), pos.reshape(-1))).cuda()] = float("nan")  # rows of no token
    w = rng.random((tokens, topk)).astype(np.float32)
    w[pos < 0] = np.nan  # a weight without a row is not used
    for weights in (w, None):
        y = host(exl3.exl3_moe_combine(ys, p, weights=None if weights is None else dev(weights)))
        ref = moe.combine(host(ys), pos, weights)
        mag = moe.combine(np.abs(host(ys)), pos, None if weights is None else np.abs(weights))
        assert np.all(np.abs(y - ref) <= half_step(dtype) * np.abs(ref) + topk * 2.0 ** -23 * mag + 2.0 ** -25)

    if dtype == torch.float32:  # fp32 rows, the sum rounded once to 16 bits
        for out in TYPES[:2]:
            y = host(exl3.exl3_moe_combine(ys, p, weights=dev(w), dtype=out))
            ref, mag = moe.combine(host(ys), pos, w), moe.combine(np.abs(host(ys)), pos, np.abs(w))
            assert np.all(np.abs(y - ref) <= half_step(out) * np.abs(ref) + topk * 2.0 ** -23 * mag + 2.0 ** -25)

    dy = torch.from_numpy(rng.standard_normal((tokens, h))).to(dtype).cuda()
    for weights in (w, None):
        dys, dw = exl3.exl3_moe_combine_grad(dy, ys, p, None if weights is None else dev(weights), dys=fill.clone())
        rd, rw = moe.combine_grad(host(dy), host(ys), pos, weights, host(fill))
        assert np.all(np.abs(host(dys) - rd) <= (half_step(dtype) + 2.0 ** -23) * np.abs(rd) + 2.0 ** -25)
        _, mag = moe.combine_grad(np.abs(host(dy)), np.abs(host(ys)), pos, weights, host(fill))
        assert np.all(np.abs(host(dw) - rw) <= h * 2.0 ** -23 * mag)


def test_gradients_against_differences():
    """The bilinear form sum(G . combine(ys, w)): its differences in ys, w and
    (through gather) x against the gradient calls, in fp32."""
    rng = np.random.default_rng(5)
    tokens, topk, experts, h = 6, 2, 3, 12
    ids = route(rng, tokens, topk, experts)
    _, pos = moe.sort(ids, experts)
    p, rows = dev(pos), tokens * topk
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    x, ys, w, g, gx = f(tokens, h), f(rows, h), f(tokens, topk), f(tokens, h), f(rows, h)
    zero = torch.zeros_like(ys)
    dys, dw = exl3.exl3_moe_combine_grad(g, ys, p, w, dys=zero.clone())
    dx = exl3.exl3_moe_combine(gx, p)
    loss = lambda a, b: float((g.double() * exl3.exl3_moe_combine(a, p, weights=b).double()).sum())  # noqa: E731
    back = lambda a: float((gx.double() * exl3.exl3_moe_gather(a, p, out=zero.clone()).double()).sum())  # noqa: E731
    # linear in each argument, so a step of 1 has no truncation error; fp32
    # sums of about 100 terms below 16 leave 100 * 16 * 2^-24 < 1e-4
    for t, grad, fn in ((ys, dys, lambda a: loss(a, w)), (w, dw, lambda a: loss(ys, a)), (x, dx, back)):
        for i in range(0, t.numel(), 5):
            up = t.clone()
            up.view(-1)[i] += 1.0
            assert abs(fn(up) - fn(t) - float(grad.view(-1)[i])) <= 1e-4


def test_positions_outside_the_rows_are_skipped():
    x = torch.randn((3, 8), device="cuda")
    pos = torch.tensor([[0, 99], [-5, 2], [4, 2147483647]], dtype=torch.int32, device="cuda")
    out = exl3.exl3_moe_gather(x, pos, out=torch.zeros((4, 8), device="cuda"))
    assert torch.equal(out, torch.stack((x[0], torch.zeros(8, device="cuda"), x[1], torch.zeros(8, device="cuda"))))
    y = exl3.exl3_moe_combine(out, pos)
    assert torch.equal(y, torch.stack((x[0], x[1], torch.zeros(8, device="cuda"))))


def test_large_rows_past_32_bits():
    """Element offsets above 2^31: the last rows of a buffer of 2^32 bytes and more."""
    h, rows = 4096, (1 << 31) // 4096 + 64
    ys = torch.zeros((rows, h), dtype=torch.float16, device="cuda")
    pos = torch.tensor([[rows - 1], [rows - 40]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, h), device="cuda").half()
    exl3.exl3_moe_gather(x, pos, out=ys)
    assert torch.equal(ys[rows - 1], x[0]) and torch.equal(ys[rows - 40], x[1])
    assert torch.equal(exl3.exl3_moe_combine(ys, pos), x)
    dys, dw = exl3.exl3_moe_combine_grad(x, ys, pos, torch.full((2, 1), 2.0, device="cuda"), dys=ys.clone())
    assert torch.equal(dys[rows - 1], 2 * x[0]) and torch.equal(dys[rows - 40], 2 * x[1])


def test_side_stream_and_graph():
    """On another stream than the current one, and captured and replayed with
    new inputs in the same buffers."""
    rng = np.random.default_rng(9)
    tokens, topk, experts, h = 1500, 2, 8, 128
    ids, x = dev(route(rng, tokens, topk, experts)), torch.randn((tokens, h), device="cuda")
    w, ws = torch.rand((tokens, topk), device="cuda"), workspace(tokens, topk, experts)
    side = torch.cuda.Stream()
    out = torch.zeros((tokens * topk, h), device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty((tokens, topk), dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)

    def step(stream=None):
        exl3.exl3_moe_sort(ids, experts, offsets=offsets, positions=pos, workspace=ws, stream=stream)
        exl3.exl3_moe_gather(x, pos, out=out, stream=stream)
        exl3.exl3_moe_combine(out, pos, weights=w, y=y, stream=stream)

    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        ids.copy_(dev(route(r, tokens, topk, experts)))
        x.copy_(torch.randn((tokens, h), device="cuda"))
        graph.replay()
        got = y.clone()
        step()
        assert torch.equal(got, y)
        ro, rp = moe.sort(host(ids), experts)
        assert np.array_equal(host(offsets), ro) and np.array_equal(host(pos), rp)
    assert first.shape == y.shape
