"""4-bit products on pairs of CTAs: waits that run out at any point of the pair's
work are reported, leave nothing behind that a later call could meet, and the
products before and after are exact (equal scales: every partial sum is exact in
fp32, so the output is the rounded exact value)."""
import numpy as np
import pytest
import torch

from oracle import mx4
from trellis_coded_bit_b200 import exl3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    exl3.load()
    yield


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def operand(rng, rows, k):
    codes, scales = rng.integers(0, 16, (rows, k)).astype(np.uint8), np.full((rows, k // 32), 127, dtype=np.uint8)
    return mx4.values(codes, scales), tuple(dev(a) for a in mx4.pack(codes, scales))


def test_waits_that_run_out_anywhere():
    """Limits from one that ends the first wait to one that lets whole tiles pass."""
    rng = np.random.default_rng(40)
    m, k, n = 600, 2048, 14000
    xv, x = operand(rng, m, k)
    wv, w = operand(rng, n, k)
    cols = rng.integers(0, n, 300)
    ref = torch.from_numpy(xv @ wv[cols].T).half()
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))

    def check():
        y = exl3.exl3_mx4_matmul(*x, *w, workspace=ws)
        assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
        assert torch.equal(y[:, dev(cols)].cpu(), ref)

    check()
    for limit in (1, 300, 1000, 3000, 10000):
        exl3.exl3_debug_set_wait_limit_ns(limit)
        try:
            exl3.exl3_mx4_matmul(*x, *w, workspace=ws)
            assert exl3.exl3_workspace_status(ws, clear=True) in (exl3.EXL3_OK, exl3.EXL3_ERR_TIMEOUT)
        finally:
            exl3.exl3_debug_set_wait_limit_ns(0)
        check()


@pytest.mark.parametrize("m,k,n", [(520, 64, 19000), (2100, 96, 4360), (700, 1056, 14001), (4096, 512, 2048)])
def test_many_calls_in_a_row(m, k, n):
    """Pairs that leave while the next call's begin: a copy or an arrival that
    came after its CTA had left would meet the next call's shared memory."""
    rng = np.random.default_rng(m + n)
    xv, x = operand(rng, m, k)
    wv, w = operand(rng, n, k)
    cols = rng.integers(0, n, 200)
    ws = exl3.new_workspace(exl3.exl3_mx4_matmul_workspace_size(m, k, n))
    outs = [torch.empty((m, n), dtype=torch.float16, device="cuda") for _ in range(8)]
    for _ in range(10):
        for y in outs:
            exl3.exl3_mx4_matmul(*x, *w, y=y, workspace=ws)
    assert exl3.exl3_workspace_status(ws) == exl3.EXL3_OK
    assert torch.equal(outs[0][:, dev(cols)].cpu(), torch.from_numpy(xv @ wv[cols].T).half())
    assert all(torch.equal(outs[0], y) for y in outs[1:])
