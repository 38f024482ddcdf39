"""The operators beside the layer on the GPU where their definitions end: offsets that fall, values at
the ends of a function's range, kernels that follow one another, waits that run out."""
import numpy as np
import pytest

import op_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_operators import (DTYPES, bq, check_balance, check_groups, check_product, host, i32, operands, run_quantize,
                                values)


# 40 rows (the kernel for few rows) and many rows of every group (the kernel of CTA pairs)
@pytest.mark.parametrize("offsets,R,N,K", [
    ([0, 30, 10, 40], 40, 64, 128), ([35, 7, 7, -3, 36], 40, 130, 200), ([2 ** 31 - 1, 0, 5], 20, 64, 128),
    ([-2 ** 31, 12, -2 ** 31, 2 ** 31 - 1], 14, 64, 300),
    ([0, 900, 300, 2000, 1500, 1700, 4000], 4100, 512, 640),
])
def test_grouped_product_of_falling_offsets(offsets, R, N, K):
    """An offset below an earlier one counts as that one: every row has one group, the results are those
    of the running maximum and repeat."""
    G = len(offsets) - 1
    a, sa, b, sb = operands(R, N, K, 17, G)
    want = np.maximum.accumulate(np.clip(offsets, 0, R))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    before = torch.randn(R, N, device="cuda")
    out = before.clone()
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, off, out)
    check_groups(out, before, a, sa, b, sb, want, K)
    for _ in range(5):
        again = before.clone()
        bq().moe_fp8_grouped_matmul(a, sa, b, sb, off, again)
        assert torch.equal(out, again)


def test_grouped_product_of_a_thousand_falling_offsets():
    G, N, K, R = 1000, 64, 128, 3000
    a, sa, b, sb = operands(R, N, K, 18, G)
    offsets = np.random.default_rng(3).integers(-10, R + 10, G + 1)
    offsets[: G // 2] = np.sort(offsets[: G // 2] // 4)
    before = torch.zeros(R, N, device="cuda")
    out = before.clone()
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, torch.from_numpy(offsets.astype(np.int32)).cuda(), out)
    check_groups(out, before, a, sa, b, sb, np.maximum.accumulate(np.clip(offsets, 0, R)), K)


# ---- kernels that follow one another -------------------------------------------------------------

def test_products_and_layer_forwards_in_a_row_share_tensor_memory():
    """Every kernel here allocates tensor memory before it waits for the one before it, up to all of an SM's:
    few-row products with and without a K split, pair products and the layer's one-launch tail in turn,
    eager and captured, nothing waited for in between, give what the calls one by one give."""
    import synth
    from harness import router_to_device, to_device
    m = bq()
    wl = synth.WORKLOADS["tiny_q8"]
    li = synth.layer_inputs(wl, 0)
    pack = m.pack_layer(li, max_tokens=8)
    x = to_device(synth.tokens(wl, li.router, 0, 0, 8))
    wr = router_to_device(li.router)
    y = torch.zeros(8, wl.hidden, device="cuda")
    products = []
    for R, N, K in ((1, 256, 512), (40, 512, 1024), (2000, 1000, 256), (4096, 1536, 384), (5, 20000, 130)):
        a, sa, b, sb = operands(R, N, K, R)
        products.append((a, sa, b, sb, torch.zeros(R, N, device="cuda")))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def sequence(wait):
        for i in (0, 1, 2, 3, 4, 1, 3, 0, 3, 4, 0):
            m.moe_fp8_matmul(*products[i], status)
            wait()
            if i != 4:
                m.moe_layer_forward(x, wr, pack, m.MOE_FMT_FROM_PACK, wl.top_k, y)
                wait()

    outs = [p[-1] for p in products] + [y]
    sequence(torch.cuda.synchronize)
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sequence(lambda: None)
    for run in [lambda: sequence(lambda: None)] * 5 + [g.replay] * 5:
        for t in outs:
            t.zero_()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert int(status) == 0 and m.moe_get_device_error(pack) == m.MOE_OK
    pack.free()


# ---- clusters: barriers behind branches of a lane or of a part of a warp ----------------------------

@pytest.mark.parametrize("R,N,K", [(7, 33, 1100), (16, 1001, 1024), (40, 4001, 640), (50, 129, 4096), (3, 1, 2048),
                                   (64, 2047, 260)])
def test_split_products_whose_last_columns_part_a_warp(R, N, K):
    """K split over 2, 4 and 8 CTAs, n not a multiple of a warp's 32 rows of weights."""
    a, sa, b, sb = operands(R, N, K, R * N)
    first = None
    for _ in range(3):
        out = torch.full((R, N), float("nan"), device="cuda")
        bq().moe_fp8_matmul(a, sa, b, sb, out)
        check_product(out, a, sa, b, sb, K)
        first = out if first is None else first
        assert torch.equal(first, out)


@pytest.mark.parametrize("T,E,k", [(1, 33, 5), (17, 129, 3), (33, 200, 8), (100, 511, 10), (128, 1021, 7), (3000, 1021, 7)])
def test_balance_loss_of_every_cluster_size_repeats(T, E, k):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = logits.topk(k, 1).indices.int()
    first = check_balance(logits, idx, None)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, check_balance(logits, idx, None)))


@pytest.mark.parametrize("T", [50, 700])
@pytest.mark.parametrize("E", [3, 4, 7, 60, 1021, 1024])
def test_plan_and_balance_loss_of_every_table_alignment(T, E):
    """Tables in shared memory that start on 16 bytes (E a multiple of 4 or 8) and that do not."""
    g = torch.Generator(device="cuda").manual_seed(E)
    k = min(3, E)
    for dt in (torch.float32, torch.bfloat16):
        logits = torch.randn(T, E, generator=g, device="cuda").to(dt)
        idx = logits.float().topk(k, 1).indices.int()
        check_balance(logits, idx, None)
    counts, offsets, rows, slots = i32(E), i32(E + 1), i32(T * k), i32(T, k)
    bq().moe_expert_plan(idx, E, counts, offsets, rows, slots)
    for got, want in zip((counts, offsets, rows, slots), ref.plan(host(idx), E)):
        assert np.array_equal(host(got), want)


# ---- SwiGLU where the sigmoid is below the smallest normal number -------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [512, 1024, 100, 513])
@pytest.mark.parametrize("low,high", [(-92, -87), (-88, -86), (-104, -93), (-120, 4)])
def test_quantize_swiglu_of_far_negative_gates(low, high, C, dt):
    """silu(g) = g / (1 + exp(-g)) is an fp32 number down to g = -104, though 1 / (1 + exp(-g)) leaves the
    normal ones at -87.3; a large up half brings it back into range.

    Below -87 the kernel forms (g h) h with h = expf(g / 2) (g / 2 is exact): expf is within 2 ulp, 2^-22
    relative, twice, and two products round (2^-24 each); the product's result may be subnormal, rounded
    to 2^-150.  Above it g r(1 + e(g)) with 2^t within 2^-22 and t = -g log2(e) rounded (|t| 2^-24, times
    ln 2, |t| <= 126: 88 2^-24), an addition (2^-24), the reciprocal within 2^-23, a product.  Times up: one
    rounding more.  Together at most 96 * 2^-24 relative and 2^-150 |up|."""
    R = 9
    g = torch.Generator(device="cuda").manual_seed(C)
    gate = (low + (high - low) * torch.rand(R, C, generator=g, device="cuda")).to(DTYPES[dt])
    up = (torch.randn(R, C, generator=g, device="cuda") * 1e30).to(DTYPES[dt])
    codes, scales = run_quantize(torch.cat([gate, up], 1), R, C, swiglu=True)
    v, u = ref.swiglu(host(torch.cat([gate, up], 1))), np.abs(host(up))
    err = np.abs(v) * 96 * 2.0 ** -24 + u * 2.0 ** -150
    nb = -(-C // 128)
    blocks = lambda x: np.pad(x, ((0, 0), (0, nb * 128 - C))).reshape(R, nb, 128).max(2)
    floor = float(ref.FLOOR)
    s = host(scales).T
    amax, most = np.maximum(blocks(np.abs(v)), floor), np.maximum(blocks(np.abs(v) + err), floor)
    least = np.maximum(blocks(np.maximum(np.abs(v) - err, 0)), floor)
    assert np.all(s <= most / 448 * (1 + 2.0 ** -23)) and np.all(s >= least / 448 * (1 - 2.0 ** -23))
    assert amax.min() > 1e3 * floor  # the values count
    per = np.repeat(s, 128, 1)[:, :C]
    # half an E4M3 step: 2^-4 of the value, or 2^-10 of the scale below the smallest normal code
    tol = np.maximum((np.abs(v) + err) * 2.0 ** -4, per * 2.0 ** -10) * (1 + 1e-5) + 2 * err
    assert np.all(np.abs(values(codes) * per - v) <= tol)


# ---- the last tile of columns of the CTA pairs ---------------------------------------------------------

@pytest.mark.parametrize("left", [1, 15, 16, 17, 31, 32, 33, 48, 144, 240, 241])
def test_pair_products_of_every_last_column_step(left):
    """n just above a multiple of the 256 columns of a tile: the last tile's columns are split over both CTAs."""
    R, N, K = 4000, 512 + left, 640
    a, sa, b, sb = operands(R, N, K, left)
    for dt in DTYPES.values():
        out = torch.full((R, N + 7), -9.0, dtype=dt, device="cuda")
        bq().moe_fp8_matmul(a, sa, b, sb, out[:, :N])
        rows = slice(R - 300, R)
        check_product(out[rows, :N], a[rows], sa[:, rows], b, sb, K)
        assert bool((out[:, N:] == -9.0).all()) and torch.isfinite(out).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N", [*range(505, 521), 255, 257, 383, 1027])
def test_pair_products_end_at_their_last_column(N, dt):
    """Rows on 16-byte boundaries in a wider buffer, n at every distance from one: nothing behind it is
    written, in whole tiles of rows and in the last ones of a group."""
    counts, K = [3000, 0, 700, 437], 640
    R = sum(counts)
    a, sa, b, sb = operands(R, N, K, N, len(counts))
    wide = torch.randn(R, -(-N // 8) * 8 + 8, device="cuda").to(DTYPES[dt])
    before = wide.clone()
    offsets = np.concatenate([[0], np.cumsum(counts)])
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, torch.from_numpy(offsets.astype(np.int32)).cuda(), wide[:, :N])
    assert torch.equal(wide[:, N:], before[:, N:])
    last = slice(offsets[2], offsets[3])
    check_product(wide[last, :N], a[last], sa[:, last], b[2], sb[2], K)


# ---- operators behind copies, fills and joined streams ---------------------------------------------------

def test_operators_behind_joined_streams_copies_and_fills():
    """Each operator waits for all that precedes it: inputs that a copy, a fill or another stream's kernel
    has just written, eager and in a captured fork and join, replayed on changed inputs."""
    m = bq()
    R, N, K, E, k = 700, 512, 640, 32, 2
    a, sa, b, sb = operands(R, N, K, 5, E)
    x = torch.empty(R // k, K, device="cuda")
    host_x = torch.empty(R // k, K).pin_memory()
    idx = torch.empty(R // k, k, dtype=torch.int32, device="cuda")
    counts, offsets, rows, slots = i32(E), i32(E + 1), i32(R), i32(R // k, k)
    xq, xs = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, R, device="cuda")
    out, dense = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        x.copy_(host_x, non_blocking=True)
        side.wait_stream(main)
        with torch.cuda.stream(side):  # the plan and a product beside the copies
            m.moe_expert_plan(idx, E, counts, offsets, rows, slots)
            m.moe_fp8_matmul(a, sa, b[0], sb[0], dense)
        out.zero_()
        main.wait_stream(side)
        m.moe_fp8_quantize(x, xq, xs, rows=rows)
        m.moe_fp8_grouped_matmul(xq, xs, b, sb, offsets, out)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            dense.add_(out)
        main.wait_stream(side)
        m.moe_expert_plan(idx, E, counts, offsets, rows, slots)

    def fill(s):
        g = torch.Generator().manual_seed(s)
        host_x.copy_(torch.randn(R // k, K, generator=g))
        idx.copy_(torch.randint(0, E, (R // k, k), generator=g, dtype=torch.int32))

    def want():
        torch.cuda.synchronize()
        m.moe_expert_plan(idx, E, counts, offsets, rows, slots)
        torch.cuda.synchronize()
        m.moe_fp8_quantize(host_x.cuda(), xq, xs, rows=rows)
        torch.cuda.synchronize()
        m.moe_fp8_grouped_matmul(xq, xs, b, sb, offsets, out)
        m.moe_fp8_matmul(a, sa, b[0], sb[0], dense)
        torch.cuda.synchronize()
        dense.add_(out)
        return out.clone(), dense.clone(), slots.clone()

    fill(0)
    want()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for s in range(1, 9):
        fill(s)
        expected = want()
        for call in (run, g.replay):
            for t in (x, out, dense, xs):
                t.fill_(float("nan"))
            xq.fill_(0x7F), rows.fill_(-1), offsets.fill_(0), slots.fill_(-5)
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((out, dense, slots), expected))
