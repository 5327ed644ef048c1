"""What the header promises of the 4-bit calls beyond a single product: split sums
in a fixed order, one workspace for these calls and the trellis calls in turn, and
the same results with overlapped launches (EXL3_LAUNCH_PDL)."""
import numpy as np
import pytest
import torch

from oracle import mx4
from trellis_coded_bit_b200 import exl3, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    exl3.load()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def operand(rng, rows, k, low, high):
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    return codes, rng.integers(low, high + 1, (rows, k // 32)).astype(np.uint8)


class Disturbance:
    """Work of changing length on another stream, so that the parts of a product
    arrive in another order each time."""

    def __init__(self):
        self.stream = torch.cuda.Stream()
        self.a = torch.randn((1024, 1024), device="cuda")
        self.n = 0

    def __enter__(self):
        self.n += 1
        with torch.cuda.stream(self.stream):
            for _ in range(self.n % 5):
                torch.matmul(self.a[:256 * (1 + self.n % 4)], self.a)

    def __exit__(self, *_):
        torch.cuda.synchronize()


# tiles that several CTAs share along k: one row of tiles, a single narrow tile, the
# tiles left over behind whole ones, and the same on pairs of CTAs
SPLIT = [(8, 14336, 512), (3, 262144, 40), (16, 16384, 2100), (100, 14336, 300), (600, 8192, 14000), (2000, 14336, 5201)]


@pytest.mark.parametrize("m,k,n", SPLIT)
def test_split_sums_in_a_fixed_order(m, k, n):
    """Scales that spread over 2^24, so that sums in another order differ; and the
    sums themselves on some columns (k additions, each off by 2^-23 of the sum of
    magnitudes at most)."""
    rng = np.random.default_rng(m + n)
    x, w = operand(rng, m, k, 115, 127), operand(rng, n, k, 115, 127)
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    first = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=torch.float32, workspace=ws)
    some = Disturbance()
    for _ in range(20):
        with some:
            y = exl3.exl3_mx4_matmul(xc, xs, wc, wsc, dtype=torch.float32, workspace=ws)
        assert torch.equal(y, first)
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
    cols = np.unique(np.concatenate([rng.integers(0, n, 60), [0, n - 1]]))
    xv, wv = mx4.values(*x), mx4.values(w[0][cols], w[1][cols])
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.all(np.abs(first[:, dev(cols)].cpu().double().numpy() - ref) <= k * 2.0 ** -23 * mag)


@pytest.mark.parametrize("m,k,n", [(600, 8192, 14000), (2000, 14336, 5201)])
def test_split_tiles_of_pairs_exact_with_equal_scales(m, k, n):
    """Partial sums are exact in fp32: the output is the rounded exact value."""
    rng = np.random.default_rng(k + n)
    x, w = operand(rng, m, k, 127, 127), operand(rng, n, k, 127, 127)
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    args = [dev(a) for a in mx4.pack(*x) + mx4.pack(*w)]
    ref = torch.from_numpy(mx4.values(*x)).cuda().double() @ torch.from_numpy(mx4.values(*w)).cuda().double().T
    for dtype in (torch.float16, torch.float32):
        assert torch.equal(exl3.exl3_mx4_matmul(*args, dtype=dtype, workspace=ws), ref.to(dtype))


@pytest.mark.parametrize("counts,k,n", [([3, 0, 1, 2], 14336, 300), ([40, 0, 16, 90], 8192, 256), ([900, 0, 257, 1500, 3, 640], 8192, 3000)])
def test_experts_sums_in_a_fixed_order(counts, k, n):
    rng = np.random.default_rng(sum(counts))
    rows, e = sum(counts) + 2, len(counts)
    offsets = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    x, w = operand(rng, rows, k, 115, 127), operand(rng, e * n, k, 115, 127)
    xc, xs = (dev(a) for a in mx4.pack(*x))
    wc, wsc = (dev(a) for a in mx4.pack(*w))
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_experts_workspace_size(rows, k, n, e))
    some, first = Disturbance(), None
    for _ in range(12):
        y = torch.zeros((rows, n), device="cuda")
        with some:
            exl3.exl3_mx4_matmul_experts(xc, xs, offsets, wc.view(e, n, -1), wsc.view(e, n, -1), y=y, workspace=ws)
        first = y if first is None else first
        assert torch.equal(y, first)
    xv, cols = mx4.values(*x), rng.integers(0, n, 40)
    for i in range(e):
        r = slice(sum(counts[:i]), sum(counts[:i + 1]))
        wv = mx4.values(w[0][i * n + cols], w[1][i * n + cols])
        ref, mag = xv[r] @ wv.T, np.abs(xv[r]) @ np.abs(wv).T
        assert np.all(np.abs(first[r][:, dev(cols)].cpu().double().numpy() - ref) <= k * 2.0 ** -23 * mag)
    assert not first[sum(counts):].any()


# ------------------------------------------------------------ one workspace ---

def test_one_workspace_for_trellis_and_4_bit_calls():
    """In turn on one workspace, with and without split sums, twice around: every
    output as with a workspace of its own."""
    rng = np.random.default_rng(5)
    calls, sizes = [], [exl3.exl3_moe_sort_workspace_size(9000, 4, 64)]

    def four(m, k, n):
        args = [dev(a) for a in mx4.pack(*operand(rng, m, k, 118, 127)) + mx4.pack(*operand(rng, n, k, 118, 127))]
        sizes.append(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
        calls.append(lambda ws: exl3.exl3_mx4_matmul(*args, dtype=torch.float32, workspace=ws))

    def trellis(name, m, k, n, K):
        L = inputs.make_layer(m, k, n, K, seed=m)
        args = [dev(a) for a in (L.x, L.trellis, L.suh, L.svh)]
        sizes.append(getattr(exl3, name + "_workspace_size")(m, k, n, K))
        calls.append(lambda ws: getattr(exl3, name)(*args, K, workspace=ws))

    def layer(m, k, n):
        x = torch.from_numpy(rng.standard_normal((m, k))).half().cuda()
        w = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda(), rotate=True)
        sizes.append(exl3.exl3_mx4_linear_workspace_size(m, k, n))
        calls.append(lambda ws: exl3.exl3_mx4_linear(x, *w, rotate=True, workspace=ws))

    ids = torch.from_numpy(rng.integers(-1, 64, (9000, 4)).astype(np.int32)).cuda()
    four(8, 14336, 512)
    trellis("exl3_gemv", 3, 4096, 2048, 4)
    layer(1, 14336, 640)
    trellis("exl3_gemm", 96, 2048, 1024, 3)
    calls.append(lambda ws: exl3.exl3_moe_sort(ids, 64, workspace=ws)[1])
    four(600, 8192, 14000)
    trellis("exl3_gemv", 1, 8192, 1024, 2)
    layer(40, 4096, 300)
    trellis("exl3_gemm", 600, 4096, 2048, 2)
    four(40, 8192, 2001)
    trellis("exl3_gemv", 16, 2048, 1024, 5)
    shared = exl3.new_workspace(max(sizes))
    want = [c(exl3.new_workspace(max(sizes))) for c in calls]
    torch.cuda.synchronize()
    for order in (range(len(calls)), reversed(range(len(calls)))):
        for i in order:
            assert torch.equal(calls[i](shared), want[i]), i
            assert exl3.exl3_workspace_status(shared) == exl3.EXL3_OK


# ------------------------------------------------------- overlapped launches ---

class Flags:
    def __init__(self, flags):
        self.flags = flags

    def __enter__(self):
        exl3.exl3_set_launch_flags(self.flags)

    def __exit__(self, *_):
        exl3.exl3_set_launch_flags(0)


@pytest.mark.parametrize("m,sizes", [(1, [512, 4096, 1024, 14336, 384]), (2, [4096, 4096, 512, 2048]), (3, [1024, 640, 4096]),
                                     (64, [2048, 1024, 4096, 512]), (700, [2048, 14080, 1024])])
def test_layers_back_to_back(m, sizes):
    """A chain of layers, each reading what the one before has just written, on one
    workspace: launched overlapped, then replayed overlapped, the results of plain
    launches on every repeat."""
    rng = np.random.default_rng(m)
    weights = [exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k)) * k ** -0.5).float().cuda(), rotate=True)
               for k, n in zip(sizes, sizes[1:])]
    x = torch.empty((m, sizes[0]), dtype=torch.bfloat16, device="cuda")
    ys = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for n in sizes[1:]]
    ws = exl3.new_workspace(max(exl3.exl3_mx4_linear_workspace_size(m, k, n) for k, n in zip(sizes, sizes[1:])))

    def chain():
        h = x
        for (wc, wsc), y in zip(weights, ys):
            h = exl3.exl3_mx4_linear(h, wc, wsc, rotate=True, y=y, workspace=ws)

    def fill(seed):
        x.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((m, sizes[0]))))

    want = []
    for seed in range(6):
        fill(seed)
        chain()
        want.append([y.clone() for y in ys])
    torch.cuda.synchronize()
    with Flags(exl3.EXL3_LAUNCH_PDL):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(2):
                chain()
        for run in (chain, graph.replay):
            for seed in range(6):
                fill(seed)
                run()
                run()
                assert all(torch.equal(a, b) for a, b in zip(want[seed], ys))
        torch.cuda.synchronize()
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK


@pytest.mark.parametrize("flags", [0, exl3.EXL3_LAUNCH_PDL])
@pytest.mark.parametrize("tokens,topk,experts,k,n", [(40, 2, 8, 512, 264), (9000, 2, 16, 256, 640), (5000, 4, 8, 256, 2600)])
def test_expert_layer_overlapped(flags, tokens, topk, experts, k, n):
    """Sort (two launches from 1025 choices on), quantise into the order, products
    and combine, whose buffers and workspace the next pass overwrites."""
    rng = np.random.default_rng(tokens)
    wc, wsc = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((experts * n, k))).float().cuda(), rotate=True)
    wc, wsc = wc.view(experts, n, -1), wsc.view(experts, n, -1)
    rows = tokens * topk
    ws = exl3.new_workspace(max(exl3.exl3_moe_sort_workspace_size(tokens, topk, experts),
                                exl3.exl3_mx4_matmul_experts_workspace_size(rows, k, n, experts)))
    xs = [torch.from_numpy(rng.standard_normal((tokens, k))).to(torch.bfloat16).cuda() for _ in range(4)]
    ids = [dev(rng.integers(-1, experts, (tokens, topk)).astype(np.int32)) for _ in range(4)]
    gates = [dev(rng.random((tokens, topk)).astype(np.float32)) for _ in range(4)]
    buf = dict(offsets=torch.empty(experts + 1, dtype=torch.int32, device="cuda"),
               pos=torch.empty((tokens, topk), dtype=torch.int32, device="cuda"),
               codes=torch.zeros((rows, k // 2), dtype=torch.uint8, device="cuda"),
               scales=torch.zeros((rows, mx4.stride(k)), dtype=torch.uint8, device="cuda"),
               ys=torch.zeros((rows, n), device="cuda"))

    def layer(i, y):
        exl3.exl3_moe_sort(ids[i], experts, offsets=buf["offsets"], positions=buf["pos"], workspace=ws)
        exl3.exl3_mx4_quantize(xs[i], rotate=True, positions=buf["pos"], out_rows=rows, codes=buf["codes"], scales=buf["scales"])
        exl3.exl3_mx4_matmul_experts(buf["codes"], buf["scales"], buf["offsets"], wc, wsc, y=buf["ys"], workspace=ws)
        exl3.exl3_moe_combine(buf["ys"], buf["pos"], weights=gates[i], y=y)

    plain = [torch.empty((tokens, n), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for i in range(4):
        layer(i, plain[i])
        torch.cuda.synchronize()
    outs = [torch.empty_like(p) for p in plain]
    with Flags(flags):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(4):
                layer(i, outs[i])
        for _ in range(3):
            for o in outs:
                o.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(plain, outs))
            for i in (2, 0, 3, 1):
                layer(i, outs[i])
            assert all(torch.equal(a, b) for a, b in zip(plain, outs))
        torch.cuda.synchronize()
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK


# ------------------------------------------------------- waits that run out ---

@pytest.mark.parametrize("m,k,n", [(1, 4096, 4096), (2, 14336, 640), (1, 96, 300), (3, 8192, 4096), (20, 14336, 512)])
def test_layers_whose_waits_run_out(m, k, n):
    """Reported at whatever point it happens, cleared, and without a trace in the
    next call."""
    rng = np.random.default_rng(m + k)
    rotate = k % 128 == 0
    x = torch.from_numpy(rng.standard_normal((m, k))).half().cuda()
    w = exl3.exl3_mx4_quantize(torch.from_numpy(rng.standard_normal((n, k))).float().cuda(), rotate=rotate)
    ws = exl3.new_workspace(exl3.exl3_mx4_linear_workspace_size(m, k, n))
    want = exl3.exl3_mx4_linear(x, *w, rotate=rotate, workspace=ws)
    for limit in (1, 500, 2000, 5000):
        exl3.exl3_debug_set_wait_limit_ns(limit)
        try:
            exl3.exl3_mx4_linear(x, *w, rotate=rotate, workspace=ws)
            assert exl3.exl3_workspace_status(ws, clear=True) in (exl3.EXL3_OK, exl3.EXL3_ERR_TIMEOUT)
        finally:
            exl3.exl3_debug_set_wait_limit_ns(0)
        assert torch.equal(exl3.exl3_mx4_linear(x, *w, rotate=rotate, workspace=ws), want)
        assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
