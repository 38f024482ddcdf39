"""The E4M3 products when a wait runs out, made without faulting the GPU: the producer stops after a
number of blocks (moe_debug_fp8_stall_after), every bounded wait behind it gives up after about a second,
copies and tensor-core work in flight land, the status word reads MOE_ERR_TIMEOUT, and the same calls are
right again.  The file sorts late: it arms process-wide fault injection."""
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_operators import bq, check_product, operands


@pytest.fixture
def stall():
    yield bq().moe_debug_fp8_stall_after
    bq().moe_debug_fp8_stall_after(-1)
    bq().moe_fp8_get_device_error()  # the next test finds none


# one row and few rows, split over a cluster or not, one and several tiles a CTA; CTA pairs
@pytest.mark.parametrize("blocks", [0, 1, 2])
@pytest.mark.parametrize("R,N,K", [(1, 1024, 4096), (40, 512, 4096), (40, 76000, 640), (2000, 1000, 640),
                                   (4096, 4096, 512)])
def test_product_whose_wait_runs_out_says_so_and_the_next_one_is_right(stall, R, N, K, blocks):
    m = bq()
    a, sa, b, sb = operands(R, N, K, R)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(R, N, device="cuda")
    stall(blocks)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    m.moe_fp8_matmul(a, sa, b, sb, out, status)
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    stall(-1)
    assert int(status) == m.MOE_ERR_TIMEOUT
    assert 0.2 < waited < 10.0, waited  # 2^31 SM clocks: about a second
    status.zero_()
    m.moe_fp8_matmul(a, sa, b, sb, out, status)
    assert int(status) == 0
    rows = slice(None) if R < 100 else slice(R - 40, R)
    check_product(out[rows], a[rows], sa[:, rows], b, sb, K)


def test_grouped_products_in_a_row_behind_one_whose_wait_ran_out(stall):
    """The next kernels are set up while the stalled one waits; they are right."""
    m = bq()
    calls = []
    for counts, N, K in (([3, 0, 17, 1], 200, 640), ([700, 0, 3, 400], 512, 640)):
        R = sum(counts)
        a, sa, b, sb = operands(R, N, K, R, len(counts))
        offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        calls.append((a, sa, b, sb, offsets, torch.zeros(R, N, device="cuda")))
    run = lambda i, status=None: m.moe_fp8_grouped_matmul(*calls[i], status)
    run(0), run(1)
    want = [c[-1].clone() for c in calls]
    for i in (0, 1):
        status, clean = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        stall(1)
        run(i, status)
        stall(-1)
        for c in calls:
            c[-1].zero_()
        run(i, clean), run(1 - i, clean), run(i, clean)
        torch.cuda.synchronize()
        assert int(status) == m.MOE_ERR_TIMEOUT and int(clean) == 0
        assert all(torch.equal(c[-1], w) for c, w in zip(calls, want))


@pytest.mark.parametrize("R,N,K", [(1, 1024, 4096), (2000, 1000, 640)])
@pytest.mark.parametrize("captured", [False, True])
def test_a_wait_that_ran_out_is_known_without_a_status_word(stall, R, N, K, captured):
    m = bq()
    a, sa, b, sb = operands(R, N, K, R)
    out = torch.zeros(R, N, device="cuda")
    m.moe_fp8_matmul(a, sa, b, sb, out)
    assert m.moe_fp8_get_device_error() == m.MOE_OK
    stall(1)
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_fp8_matmul(a, sa, b, sb, out)
        stall(-1)
        g.replay()
    else:
        m.moe_fp8_matmul(a, sa, b, sb, out)
        stall(-1)
    m.moe_fp8_matmul(a, sa, b, sb, out)  # right, and does not clear the error
    assert m.moe_fp8_get_device_error() == m.MOE_ERR_TIMEOUT
    assert m.moe_fp8_get_device_error(0) == m.MOE_OK
    check_product(out[-40:], a[-40:], sa[:, -40:], b, sb, K)
