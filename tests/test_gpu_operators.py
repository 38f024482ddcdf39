"""The operators beside the layer on the GPU against plain 64-bit references
(op_reference.py): the expert plan, the balance loss and its gradient, the E4M3
quantisers and the E4M3 products, each at the sizes and masks where it can go
wrong, a run of them together, and their behaviour in graphs and on streams."""
import numpy as np
import pytest

import op_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def bq():
    import block_quantized_expert_moe_b200 as m
    return m


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def i32(*shape):
    return torch.full(shape, -77, dtype=torch.int32, device="cuda")


def code_rows(lead, cols, fill=0xAA):
    """Code rows on 16-byte boundaries, the bytes behind `cols` marked."""
    width = -(-cols // 16) * 16
    return torch.full((*lead, width), fill, dtype=torch.uint8, device="cuda")


def values(codes):
    return ref.E4M3[codes.view(torch.uint8).cpu().numpy()]


# ---- the expert plan ---------------------------------------------------------------

@pytest.mark.parametrize("T,E,k,skew,pad", [
    (1, 1, 1, 0, 0), (1, 512, 10, 0, 0), (8, 512, 10, 0, 2), (3, 7, 7, 0, 0), (64, 64, 8, 1, 5), (33, 1024, 16, 0, 0),
    (409, 60, 10, 1, 0), (410, 1000, 10, 0, 100), (2048, 512, 10, 1, 77), (8192, 512, 10, 1, 0), (5000, 3, 2, 0, 5000),
    (70001, 128, 1, 1, 0), (65536, 512, 10, 0, 1000),
])
def test_plan(T, E, k, skew, pad):
    rng = np.random.default_rng(T + E)
    score = rng.standard_normal((T, E)) + skew * rng.standard_normal(E) if T * E <= 1 << 24 else None
    if score is None:
        idx = rng.integers(0, E, (T, k))
    else:
        idx = np.argpartition(-score, min(k, E) - 1, axis=1)[:, :k]
    if pad:
        idx[rng.permutation(T)[:pad]] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31])
    idx = idx.astype(np.int32)
    counts, offsets, rows, slots = i32(E), i32(E + 1), i32(T * k), i32(T, k)
    bq().moe_expert_plan(torch.from_numpy(idx).cuda(), E, counts, offsets, rows, slots)
    for got, want in zip((counts, offsets, rows, slots), ref.plan(idx, E)):
        assert np.array_equal(host(got), want)


def test_plan_one_expert_takes_everything_and_a_token_repeats_an_expert():
    idx = torch.full((3000, 4), 2, dtype=torch.int32, device="cuda")
    counts, offsets, rows, slots = i32(5), i32(6), i32(12000), i32(3000, 4)
    bq().moe_expert_plan(idx, 5, counts, offsets, rows, slots)
    assert host(counts).tolist() == [0, 0, 12000, 0, 0] and host(offsets).tolist() == [0, 0, 0, 12000, 12000, 12000]
    assert np.array_equal(host(slots).reshape(-1), np.arange(12000))
    assert np.array_equal(host(rows), np.arange(12000) // 4)


def test_plan_of_no_tokens_writes_zero_counts():
    counts, offsets = i32(5), i32(6)
    bq().moe_expert_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5, counts, offsets, i32(0), i32(0, 2))
    assert not host(counts).any() and not host(offsets).any()


# ---- the balance loss ----------------------------------------------------------------

def run_balance(logits, idx, valid, dloss):
    T, E = logits.shape
    m = bq()
    need = m.moe_balance_loss_workspace_bytes(T, E)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    counts, pm = i32(E + 1), torch.full((E,), float("nan"), device="cuda")
    loss, dl = torch.full((1,), float("nan"), device="cuda"), torch.full_like(logits, float("nan"))
    m.moe_balance_loss(logits, idx, counts, pm, loss, ws, valid=valid)
    m.moe_balance_loss_backward(logits, counts, idx.shape[1], torch.tensor([dloss], device="cuda"), dl, valid=valid)
    return loss, counts, pm, dl


# p in fp32: the argument l - m has |l - m| <= 32 here, off by 32 * 2^-24 at most; expf is within 2 ulp
# (4 * 2^-24); the row's sum adds at most 32 + 5 terms in sequence; one division and one product: together
# below 96 * 2^-24.  P adds positive terms: at most T / 16 + 16 + 16 more roundings (here below 300).
P_REL = 400 * 2.0 ** -24


def check_balance(logits, idx, valid, dloss=0.37):
    got = run_balance(logits, idx, valid, dloss)
    loss, counts, P, dl, p, f = ref.balance(host(logits), host(idx), None if valid is None else host(valid),
                                            np.float32(dloss).astype(np.float64))
    assert np.array_equal(host(got[1]), counts)
    assert np.all(np.abs(host(got[2]) - P) <= P_REL * P + 1e-38)
    assert abs(host(got[0])[0] - loss) <= 2 * P_REL * loss
    n = max(1, counts[-1])
    step = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 2.0 ** -24
    tol = dloss / n * p * (f + (p @ f)[:, None]) * P_REL + np.abs(dl) * 1.01 * step + 1e-38
    assert np.all(np.abs(host(got[3]) - dl) <= tol)
    if valid is not None:
        assert not host(got[3])[host(valid) == 0].any()
    return got


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,pad", [
    (1, 1, 1, 0), (1, 512, 10, 0), (2, 4, 4, 1), (64, 64, 8, 3), (31, 60, 6, 0), (33, 257, 3, 10), (100, 1000, 16, 0),
    (257, 128, 2, 0), (300, 512, 10, 300), (512, 1024, 10, 5), (1000, 33, 4, 100), (4099, 512, 10, 500),
])
def test_balance_loss_and_gradient(T, E, k, pad, dt):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(DTYPES[dt])
    idx = logits.float().topk(k, 1).indices.int()
    valid = None
    if pad:
        valid = torch.ones(T, dtype=torch.bool, device="cuda")
        valid[torch.randperm(T, generator=g, device="cuda")[:pad]] = False
    check_balance(logits, idx, valid)


def test_balance_rows_off_16_byte_boundaries():
    g = torch.Generator(device="cuda").manual_seed(5)
    for dt in DTYPES.values():
        buf = torch.randn(40 * 64 + 1, generator=g, device="cuda").to(dt)
        logits = buf[1:].view(40, 64)
        check_balance(logits, logits.float().topk(4, 1).indices.int(), None)


def test_balance_masked_experts_and_masked_rows():
    """-inf and the type's lowest value have probability 0; a row of only -inf adds nothing; NaN and
    infinities in rows that do not count are not seen; idx may hold no choice at all."""
    g = torch.Generator(device="cuda").manual_seed(6)
    for dt in DTYPES.values():
        logits = torch.randn(70, 96, generator=g, device="cuda").to(dt)
        logits[:, 3] = float("-inf")
        logits[:, 4] = torch.finfo(dt).min
        logits[5] = float("-inf")
        valid = torch.ones(70, dtype=torch.uint8, device="cuda")
        logits[9], logits[10] = float("nan"), float("inf")
        valid[9] = valid[10] = 0
        idx = torch.randint(-1, 97, (70, 6), generator=g, device="cuda", dtype=torch.int32)
        got = check_balance(logits, idx, valid)
        assert host(got[2])[3] == 0 and not host(got[3])[5].any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("E", [63, 64])
def test_balance_of_logits_at_the_ends_of_the_type(E, dt):
    """The softmax depends on differences alone: rows of only the lowest value are even, one largest value
    takes its row, and large offsets change nothing.  Differences are 0 to 32, 64, or beyond 100 (p = 0)."""
    t = DTYPES[dt]
    lo, hi = torch.finfo(t).min, torch.finfo(t).max
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.zeros(12, E, device="cuda")
    logits[0] = lo
    logits[1] = lo
    logits[1, ::2] = float("-inf")
    logits[2] = hi
    logits[3, 7] = hi
    logits[4, :20], logits[4, 20:] = hi, lo
    logits[5, :20], logits[5, 20:] = -1e30, lo
    logits[6], logits[6, 5] = 1e30, -1e30
    steps = torch.randint(0, 128, (5, E), generator=g, device="cuda")
    logits[7] = 2.0 ** 21 + 0.25 * steps[0]
    logits[8] = -(2.0 ** 21) - 0.25 * steps[1]
    logits[9] = 2.0 ** 30 + 64 * (steps[2] % 3)
    logits[10] = -(2.0 ** 30) - 64 * (steps[3] % 3)
    logits[11] = 2.0 ** 19 + 0.25 * steps[4]
    logits = logits.to(t)
    idx = torch.randint(0, E, (12, 4), generator=g, device="cuda", dtype=torch.int32)
    check_balance(logits, idx, None)
    for row in range(12):  # each alone, where no other row hides its sum
        check_balance(logits[row:row + 1].clone(), idx[row:row + 1].clone(), None)


def test_balance_nan_reaches_the_loss_and_only_its_row_of_the_gradient():
    logits = torch.zeros(40, 64, device="cuda")
    logits[7, 3] = float("nan")
    idx = torch.zeros(40, 2, dtype=torch.int32, device="cuda")
    loss, _, _, dl = run_balance(logits, idx, None, 1.0)
    assert torch.isnan(loss).all() and torch.isnan(dl[7]).all() and torch.isfinite(dl[:7]).all()
    assert torch.isfinite(dl[8:]).all()


def test_balance_of_no_tokens_and_even_routing():
    m = bq()
    counts, pm, loss = i32(9), torch.full((8,), 5.0, device="cuda"), torch.full((1,), 5.0, device="cuda")
    empty = torch.empty(0, 8, device="cuda")
    m.moe_balance_loss(empty, torch.empty(0, 2, dtype=torch.int32, device="cuda"), counts, pm, loss)
    assert not host(counts).any() and not host(pm).any() and not host(loss).any()
    m.moe_balance_loss_backward(empty, counts, 2, loss, empty.clone())
    idx = (torch.arange(64, device="cuda", dtype=torch.int32) % 8).view(32, 2)
    loss, _, _, dl = run_balance(torch.zeros(32, 8, device="cuda"), idx, None, 1.0)
    assert float(loss) == 1.0 and not host(dl).any()


def test_balance_gradient_against_differences():
    """Central differences of the 64-bit loss in random directions (choices held): the loss is smooth, so
    with h = 1e-4 the quotient is off by O(h^2) = 1e-8 of its third derivative."""
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = torch.randn(50, 40, generator=g, device="cuda")
    idx = logits.topk(4, 1).indices.int()
    dl = host(run_balance(logits, idx, None, 1.0)[3])
    x, i = host(logits), host(idx)
    rng = np.random.default_rng(1)
    for _ in range(5):
        d = rng.standard_normal(x.shape)
        diff = (ref.balance(x + 1e-4 * d, i, None, 1.0)[0] - ref.balance(x - 1e-4 * d, i, None, 1.0)[0]) / 2e-4
        assert abs(diff - (dl * d).sum()) <= 1e-6 * np.abs(dl * d).sum() + 1e-8


# ---- the quantisers ------------------------------------------------------------------

def run_quantize(x, R, C, rows=None, swiglu=False):
    codes = code_rows((R,), C)
    scales = torch.full((-(-C // 128), R), float("nan"), device="cuda")
    bq().moe_fp8_quantize(x, codes[:, :C], scales, rows=rows, swiglu=swiglu)
    assert bool((codes[:, C:] == 0xAA).all())
    return codes[:, :C], scales


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (3, 127), (9, 129), (10, 2048), (17, 1000), (100, 264), (1200, 513)])
def test_quantize_rows_bit_for_bit(R, C, dt):
    g = torch.Generator(device="cuda").manual_seed(R + C)
    x = (torch.randn(R, C, generator=g, device="cuda") * torch.exp(4 * torch.randn(R, 1, generator=g, device="cuda")))
    x = x.to(DTYPES[dt])
    x[0, : min(C, 128)] = 0  # a block of zeros
    codes, scales = run_quantize(x, R, C)
    want, s = ref.quantize(x.float().cpu().numpy())
    assert same(values(codes), want) and same(host(scales), s.T.astype(np.float64))


def test_quantize_ties_subnormals_extremes_and_non_finite():
    x = torch.zeros(12, 256, device="cuda")
    x[0, :17] = torch.tensor([448, 17, 19, 21, 1.0625, 1.1875, 2 ** -9, 2 ** -10, 3 * 2 ** -10, -17, 432, 440, -448,
                              2 ** -7 + 2 ** -10, 464, 0.5, -2 ** -11], device="cuda")
    x[1] = 1e-45
    x[2, 0] = 3.4e38
    x[3, 3] = float("nan")
    x[4, 4] = float("inf")
    x[5, 200] = float("-inf")
    x[6] = torch.finfo(torch.float32).min
    x[7, 1] = 5.3e-36
    x[8, 0], x[8, 1] = 1e-30, 1e-38
    codes, scales = run_quantize(x, 12, 256)
    want, s = ref.quantize(x.cpu().numpy())
    assert same(values(codes), want) and same(host(scales), s.T.astype(np.float64))
    assert np.isnan(values(codes)[3, :128]).all() and np.isfinite(values(codes)[3, 128:]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_gathers_rows_strides_and_odd_addresses(dt):
    g = torch.Generator(device="cuda").manual_seed(3)
    buf = torch.randn(50, 301, generator=g, device="cuda").to(DTYPES[dt])
    x = buf[:, 1:261]  # rows off 16-byte boundaries, stride above the width
    rows = torch.randint(0, 50, (77,), generator=g, device="cuda", dtype=torch.int32)
    rows[5], rows[6], rows[7] = -1, 50, 2 ** 31 - 1
    codes, scales = run_quantize(x, 77, 260, rows=rows)
    src = x.float().cpu().numpy()
    ok = (host(rows) >= 0) & (host(rows) < 50)
    gathered = np.where(ok[:, None], src[np.where(ok, host(rows), 0)], np.float32(0))
    want, s = ref.quantize(gathered)
    assert same(values(codes), want) and same(host(scales), s.T.astype(np.float64))
    # scales into a wider buffer's columns
    wide = torch.full((3, 100), -5.0, device="cuda")
    bq().moe_fp8_quantize(x, code_rows((77,), 260)[:, :260], wide[:, 10:87], rows=rows)
    assert same(host(wide)[:, 10:87], s.T.astype(np.float64))
    assert bool((wide[:, :10] == -5).all()) and bool((wide[:, 87:] == -5).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 512), (5, 100), (33, 513), (700, 256)])
def test_quantize_swiglu(R, C, dt):
    g = torch.Generator(device="cuda").manual_seed(C)
    x = (3 * torch.randn(R, 2 * C, generator=g, device="cuda")).to(DTYPES[dt])
    x[0, 0], x[0, 1], x[0, 2] = -100.0, 100.0, 0.0
    codes, scales = run_quantize(x, R, C, swiglu=True)
    v = ref.swiglu(host(x))
    nb = -(-C // 128)
    pad = np.pad(v, ((0, 0), (0, nb * 128 - C))).reshape(R, nb, 128)
    amax = np.maximum(np.abs(pad).max(2), float(ref.FLOOR))
    # fp32 silu: exp within 2 ulp of an exact argument, an addition, a division within 2 ulp, a product
    rel = 16 * 2.0 ** -24
    s = host(scales).T
    assert np.all(np.abs(s - amax / 448) <= amax / 448 * (rel + 2.0 ** -23))
    per = np.repeat(s, 128, 1)[:, :C]
    # half an E4M3 step: 2^-4 of the value, or 2^-10 of the scale below the smallest normal code
    tol = np.maximum(np.abs(v) * 2.0 ** -4, per * 2.0 ** -10) * (1 + 1e-5) + np.abs(v) * 2 * rel
    assert np.all(np.abs(values(codes) * per - v) <= tol)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("G,N,K", [(0, 1, 1), (0, 128, 128), (0, 130, 300), (3, 257, 129), (5, 64, 512)])
def test_quantize_weight_bit_for_bit(G, N, K, dt):
    lead = (G,) if G else ()
    g = torch.Generator(device="cuda").manual_seed(N)
    w = (0.02 * torch.randn(*lead, N, K, generator=g, device="cuda")).to(DTYPES[dt])
    codes = code_rows((*lead, N), K)
    scales = torch.full((*lead, -(-N // 128), -(-K // 128)), float("nan"), device="cuda")
    bq().moe_fp8_quantize_weight(w, codes[..., :K], scales)
    assert bool((codes[..., K:] == 0xAA).all())
    w, codes, scales = w.view(-1, N, K), codes.view(max(G, 1), N, -1)[..., :K], scales.view(max(G, 1), -(-N // 128), -1)
    for i in range(max(G, 1)):
        want, s = ref.quantize(w[i].float().cpu().numpy(), 128)
        assert same(values(codes[i]), want) and same(host(scales[i]), s.astype(np.float64))


# ---- the products ----------------------------------------------------------------------

def random_codes(lead, cols, g):
    """Codes whose values look like quantised Gaussians, zeros and both largest values among them."""
    c = code_rows(lead, cols, fill=0x7F)  # NaN behind the row's end must never be read
    c[..., :cols] = (torch.randn(*lead, cols, generator=g, device="cuda") * 120).clamp(-448, 448).to(
        torch.float8_e4m3fn).view(torch.uint8)
    return c[..., :cols]


def operands(R, N, K, seed, groups=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = random_codes((R,), K, g)
    sa = torch.exp(torch.randn(kb, R, generator=g, device="cuda")) * 0.01
    lead = () if groups is None else (groups,)
    b = random_codes((*lead, N), K, g)
    sb = torch.exp(torch.randn(*lead, nb, kb, generator=g, device="cuda")) * 0.001
    return a, sa, b, sb


def check_product(got, a, sa, b, sb, K):
    y, mag = ref.product(values(a), host(sa), values(b), host(sb))
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(host(got) - y)
    assert np.all(err <= ref.product_bound(mag, K, half, y)), float((err / np.maximum(mag, 1e-30)).max())


PRODUCT_SIZES = [
    (1, 1, 1), (1, 128, 128), (1, 1024, 2048), (2, 3, 5), (3, 130, 17), (15, 64, 127), (16, 64, 129), (17, 257, 1000),
    (31, 100, 4096), (64, 1024, 2048), (65, 1000, 1111), (128, 128, 256), (129, 700, 640), (333, 1000, 1111),
    (1000, 2049, 300), (2500, 2049, 640), (4096, 1500, 384), (4097, 1537, 130),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,N,K", PRODUCT_SIZES)
def test_product(R, N, K, dt):
    a, sa, b, sb = operands(R, N, K, R + N + K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((R, N), float("nan"), dtype=DTYPES[dt], device="cuda")
    bq().moe_fp8_matmul(a, sa, b, sb, out, status)
    assert int(status) == 0
    check_product(out, a, sa, b, sb, K)


@pytest.mark.parametrize("R,N,K", [(5, 130, 200), (300, 200, 300), (4500, 1400, 200)])
def test_product_strides_and_untouched_columns(R, N, K):
    a, sa, b, sb = operands(R + 3, N + 4, K, 11)
    wide_a = code_rows((R + 3,), K + 64, fill=0x7F)
    wide_a[:, 16:16 + K] = a
    out = torch.full((R + 3, N + 7), -9.0, device="cuda")
    bq().moe_fp8_matmul(wide_a[2:2 + R, 16:16 + K], sa[:, 2:2 + R], b[4:], sb[:-(-N // 128)], out[1:1 + R, 3:3 + N])
    check_product(out[1:1 + R, 3:3 + N], a[2:2 + R], sa[:, 2:2 + R], b[4:], sb[:-(-N // 128)], K)
    out[1:1 + R, 3:3 + N] = -9.0
    assert bool((out == -9.0).all())


def check_groups(out, before, a, sa, b, sb, offsets, K):
    used = np.zeros(out.shape[0], bool)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        used[lo:hi] = True
        if hi > lo:
            check_product(out[lo:hi], a[lo:hi], sa[:, lo:hi], b[e], sb[e], K)
    assert np.array_equal(host(out)[~used], host(before)[~used])


GROUPS = [
    ([1], 128, 128), ([0, 1, 0], 64, 100), ([3, 0, 0, 17, 1], 200, 300), ([64, 65, 0, 128, 2], 130, 256),
    ([1] * 10, 1024, 2048), ([0] * 9 + [1], 384, 640), ([700, 0, 3, 40], 256, 128), ([160, 130, 257, 1, 300] * 8, 384, 256),
    ([200] * 40, 520, 200), ([0] * 500 + [5, 0, 7] + [0] * 521, 64, 64), ([33] * 64, 1024, 512),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped_product(counts, N, K, dt):
    first, behind = 2, 5  # rows outside every group
    R = first + sum(counts) + behind
    a, sa, b, sb = operands(R, N, K, N + K, len(counts))
    offsets = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    out = torch.randn(R, N, device="cuda").to(DTYPES[dt])
    before = out.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, torch.from_numpy(offsets).cuda(), out, status)
    assert int(status) == 0
    check_groups(out, before, a, sa, b, sb, offsets, K)


@pytest.mark.parametrize("counts", [[40, 3, 50], [400, 300, 500] * 20])
def test_grouped_product_keeps_rows_apart(counts):
    """NaN codes, infinite and NaN scales of one row stay in that row; NaN in rows outside every group
    reaches nothing; a group with NaN weights spoils its own rows only."""
    N, K, R = 256, 200, sum(counts) + 8
    a, sa, b, sb = operands(R, N, K, 4, len(counts))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    a[5, 7], a[offsets[-1] + 1] = 0x7F, 0x7F
    sa[0, 9], sa[1, 11] = float("nan"), float("inf")
    b[1, 3, 100] = 0x7F
    out = torch.zeros(R, N, device="cuda")
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, torch.from_numpy(offsets).cuda(), out)
    bad = ~np.isfinite(host(out))
    want = np.zeros((R, N), bool)
    want[[5, 9, 11]] = True
    want[offsets[1]:offsets[2], 3] = True
    assert np.array_equal(bad, want)


def test_grouped_product_clamps_offsets():
    """Offsets outside [0, rows], or falling, are taken into range: nothing outside is touched."""
    N, K, R = 64, 128, 40
    a, sa, b, sb = operands(R, N, K, 4, 4)
    out = torch.zeros(R, N, device="cuda")
    off = torch.tensor([-5, 10, 10, 30, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, off, out)
    check_groups(out, out, a, sa, b, sb, [0, 10, 10, 30, 40], K)


def test_products_repeat_bit_for_bit():
    for R, N, K in ((1, 1024, 2048), (40, 512, 4096), (4096, 1500, 384)):
        a, sa, b, sb = operands(R, N, K, 1)
        out = torch.empty(R, N, device="cuda")
        bq().moe_fp8_matmul(a, sa, b, sb, out)
        for _ in range(5):
            again = torch.full_like(out, float("nan"))
            bq().moe_fp8_matmul(a, sa, b, sb, again)
            assert torch.equal(out, again)


def test_product_by_transposed_weights_is_the_input_gradient():
    """d(a b^T)/da applied to dy is dy b: the same call on the transposed codes and block scales."""
    N, K, R = 384, 256, 70
    _, _, b, sb = operands(1, N, K, 3)
    dy, sdy, _, _ = operands(R, 1, N, 4)
    bt = code_rows((K,), N)[:, :N]
    bt.copy_(b.t())
    da = torch.empty(R, K, device="cuda")
    bq().moe_fp8_matmul(dy, sdy, bt, sb.t().contiguous(), da)
    w = values(b) * np.repeat(np.repeat(host(sb), 128, 0), 128, 1)
    g = values(dy) * np.repeat(host(sdy).T, 128, 1)
    mag = np.abs(g) @ np.abs(w)
    assert np.all(np.abs(host(da) - g @ w) <= ref.product_bound(mag, N, 2.0 ** -24, g @ w))


# ---- together, in graphs, on streams ------------------------------------------------------

class Layer:
    """A routed SwiGLU layer over E4M3 experts composed from the operators, with its buffers."""

    def __init__(self, T, E, k, H, I, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        m = bq()
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        self.x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        self.router = (0.1 * torch.randn(E, H, generator=g, device="cuda")).bfloat16()
        R = T * k
        self.idx, self.gate = i32(T, k), torch.empty(T, k, device="cuda")
        self.counts, self.offsets, self.rows, self.slots = i32(E), i32(E + 1), i32(R), i32(T, k)
        self.route_ws = torch.empty(m.moe_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(max(16, m.moe_balance_loss_workspace_bytes(T, E)), dtype=torch.uint8, device="cuda")
        self.xq, self.xs = code_rows((R,), H)[:, :H], torch.empty(-(-H // 128), R, device="cuda")
        self.hq, self.hs = code_rows((R,), I)[:, :I], torch.empty(-(-I // 128), R, device="cuda")
        self.gu = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.y = torch.zeros(R, H, device="cuda")
        self.w = []
        for n, c in ((2 * I, H), (H, I)):
            w = (0.05 * torch.randn(E, n, c, generator=g, device="cuda")).bfloat16()
            q, s = code_rows((E, n), c)[..., :c], torch.empty(E, -(-n // 128), -(-c // 128), device="cuda")
            m.moe_fp8_quantize_weight(w, q, s)
            self.w.append((q, s))
        self.bcounts, self.pm = i32(E + 1), torch.empty(E, device="cuda")
        self.loss, self.dloss = torch.empty(1, device="cuda"), torch.full((1,), 0.01, device="cuda")
        self.logits = torch.empty(T, E, device="cuda")
        self.dlogits = torch.empty(T, E, device="cuda")

    def run(self, stream=None):
        m = bq()
        m.moe_route_topk(self.x, self.router, self.k, self.idx, self.gate, self.route_ws, stream)
        m.moe_expert_plan(self.idx, self.E, self.counts, self.offsets, self.rows, self.slots, stream)
        m.moe_fp8_quantize(self.x, self.xq, self.xs, rows=self.rows, stream=stream)
        m.moe_fp8_grouped_matmul(self.xq, self.xs, *self.w[0], self.offsets, self.gu, stream=stream)
        m.moe_fp8_quantize(self.gu, self.hq, self.hs, swiglu=True, stream=stream)
        m.moe_fp8_grouped_matmul(self.hq, self.hs, *self.w[1], self.offsets, self.y, stream=stream)
        m.moe_balance_loss(self.logits, self.idx, self.bcounts, self.pm, self.loss, self.ws, stream=stream)
        m.moe_balance_loss_backward(self.logits, self.bcounts, self.k, self.dloss, self.dlogits, stream=stream)

    def check(self):
        """Every stage against its 64-bit reference on the previous stage's outputs."""
        counts, offsets, rows, slots = ref.plan(host(self.idx), self.E)
        assert np.array_equal(host(self.offsets), offsets) and np.array_equal(host(self.slots), slots)
        xq, xs = ref.quantize(self.x.float().cpu().numpy()[rows])
        assert same(values(self.xq), xq) and same(host(self.xs), xs.T.astype(np.float64))
        check_groups(self.gu, self.gu, self.xq, self.xs, *self.w[0], offsets, self.H)
        h = ref.swiglu(host(self.gu))
        hv = values(self.hq) * np.repeat(host(self.hs).T, 128, 1)[:, :self.I]
        tol = np.maximum(np.abs(h) * 2.0 ** -4, np.repeat(host(self.hs).T, 128, 1)[:, :self.I] * 2.0 ** -10)
        assert np.all(np.abs(hv - h) <= tol * (1 + 1e-4) + 1e-30)
        check_groups(self.y, self.y, self.hq, self.hs, *self.w[1], offsets, self.I)
        loss, bc, P, dl, p, f = ref.balance(host(self.logits), host(self.idx), None, host(self.dloss)[0])
        assert np.array_equal(host(self.bcounts), bc) and np.array_equal(host(self.counts), bc[:-1])
        assert abs(host(self.loss)[0] - loss) <= 2 * P_REL * loss
        out = (self.y[self.slots.long()] * self.gate[..., None]).sum(1)  # the layer's combine
        assert torch.isfinite(out).all() and out.shape == (self.T, self.H)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 64, 8, 1024, 256), (13, 16, 4, 512, 192), (700, 32, 6, 512, 256)])
def test_operators_compose_into_a_layer(T, E, k, H, I):
    layer = Layer(T, E, k, H, I, T)
    layer.logits.copy_((layer.x.float() @ layer.router.float().t()))
    layer.run()
    layer.check()


def test_operators_in_captured_graphs_that_share_buffers():
    """Two graphs over the same buffers and workspace, replayed in turn on changed inputs, give what the
    eager calls give."""
    layer = Layer(600, 32, 6, 512, 256, 3)
    fill = lambda s: (layer.x.copy_(torch.randn(600, 512, generator=torch.Generator("cuda").manual_seed(s),
                                                device="cuda")),
                      layer.logits.copy_(layer.x.float() @ layer.router.float().t()))
    fill(0)
    layer.run()  # first calls set kernel attributes outside the capture
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.run()
        graphs.append(g)
    for s in (1, 2, 3):
        fill(s)
        graphs[s % 2].replay()
        torch.cuda.synchronize()
        layer.check()
        y, dl = layer.y.clone(), layer.dlogits.clone()
        layer.y.zero_(), layer.dlogits.zero_()
        layer.run()
        assert torch.equal(y, layer.y) and torch.equal(dl, layer.dlogits)


def test_operators_on_concurrent_streams():
    """Two layers with buffers of their own on two streams at once give what each gives alone."""
    layers = [Layer(300, 32, 6, 512, 256, s) for s in (1, 2)]
    want = []
    for l in layers:
        l.logits.copy_(l.x.float() @ l.router.float().t())
        l.run()
        torch.cuda.synchronize()
        want.append((l.y.clone(), l.dlogits.clone(), l.loss.clone()))
        l.y.zero_(), l.dlogits.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for l, s in zip(layers, streams):
            l.run(s)
    torch.cuda.synchronize()
    for l, (y, dl, loss) in zip(layers, want):
        assert torch.equal(l.y, y) and torch.equal(l.dlogits, dl) and torch.equal(l.loss, loss)


# ---- sizes and buffers where the kernels' variants can go wrong ----------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,N,K", [(20001, 1, 256), (20000, 40, 512), (19000, 272, 128), (4096, 1504, 1152),
                                   (257, 4096, 2048), (3, 75000, 200), (60, 20000, 130)])
def test_product_of_extreme_shapes(R, N, K, dt):
    a, sa, b, sb = operands(R, N, K, R + N)
    out = torch.full((R, N), float("nan"), dtype=DTYPES[dt], device="cuda")
    bq().moe_fp8_matmul(a, sa, b, sb, out)
    check_product(out, a, sa, b, sb, K)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N", [([4000], 1000), ([300, 0, 700, 1, 130] * 6, 1000), ([9], 1000)])
def test_products_leave_the_rest_of_a_wider_buffer(counts, N, dt):
    """Rows on 16-byte boundaries in a wider buffer (whole tiles leave as boxes): columns behind n and rows
    outside every group keep their values."""
    K, first, behind = 300, 3, 40
    R = first + sum(counts) + behind
    a, sa, b, sb = operands(R, N, K, 21, len(counts))
    wide = torch.randn(R, N + 24, device="cuda").to(DTYPES[dt])
    before = wide.clone()
    offsets = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    bq().moe_fp8_grouped_matmul(a, sa, b, sb, torch.from_numpy(offsets).cuda(), wide[:, :N])
    assert torch.equal(wide[:, N:], before[:, N:])
    check_groups(wide[:, :N], before[:, :N], a, sa, b, sb, offsets, K)


def test_products_beyond_32_bit_offsets():
    """Outputs of more than 2^31 elements, weights and codes of more than 2^32 bytes: the last rows, the last
    group and the last codes are right."""
    R, N, K = 300000, 8192, 128
    a, sa, b, sb = operands(R, N, K, 2)
    out = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    bq().moe_fp8_matmul(a, sa, b, sb, out)
    check_product(out[-300:], a[-300:], sa[:, -300:], b, sb, K)
    del out
    G, N, K = 600, 1024, 8192
    a, sa, b, sb = operands(40, N, K, 3)
    weights = torch.zeros(G, N, K, dtype=torch.uint8, device="cuda")
    weights[-1] = b
    scales = torch.zeros(G, *sb.shape, device="cuda")
    scales[-1] = sb
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 40
    out = torch.zeros(40, N, device="cuda")
    bq().moe_fp8_grouped_matmul(a, sa, weights, scales, offsets, out)
    check_product(out, a, sa, b, sb, K)
    del weights
    R, C = 40000, 131072
    x = torch.randn(3, C, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    rows = torch.zeros(R, dtype=torch.int32, device="cuda")
    rows[-1] = 2
    codes, scales = torch.empty(R, C, dtype=torch.uint8, device="cuda"), torch.empty(C // 128, R, device="cuda")
    bq().moe_fp8_quantize(x, codes, scales, rows=rows)
    want, s = ref.quantize(x[2:].float().cpu().numpy())
    assert same(values(codes[-1:]), want) and same(host(scales[:, -1:]), s.T.astype(np.float64))


def test_quantize_scales_over_every_binade():
    """The scale's division by 448 and its inverse, bit for bit, over mantissas of every exponent."""
    rng = np.random.default_rng(4)
    bits = (np.arange(1, 255, dtype=np.uint32)[:, None] << 23 | rng.integers(0, 1 << 23, (254, 128), dtype=np.uint32))
    amax = bits.view(np.float32).reshape(-1)
    x = np.zeros((amax.size, 128), np.float32)
    x[:, 0], x[:, 1] = amax, -amax * np.float32(0.3)
    codes, scales = run_quantize(torch.from_numpy(x).cuda(), *x.shape)
    a = np.maximum(amax, ref.FLOOR)
    s, inv = a / np.float32(448), np.float32(448) / a
    assert np.array_equal(scales[0].cpu().numpy(), s)
    got = values(codes)
    assert np.array_equal(got[:, :2], ref.to_e4m3((x[:, :2] * inv[:, None]).astype(np.float64)))


def test_balance_with_more_choices_than_a_warp():
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(200, 70, generator=g, device="cuda")
    check_balance(logits, logits.topk(50, 1).indices.int(), None)


FIRST_CALLS = """
import torch
import block_quantized_expert_moe_b200 as bq
x = torch.randn(300, 256, device="cuda")
idx = torch.randint(0, 8, (300, 2), device="cuda", dtype=torch.int32)
i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
f = lambda *s: torch.zeros(*s, device="cuda")
c = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
T = [i(8), i(9), i(600), i(300, 2), c(600, 256), f(2, 600), c(8, 256, 256), f(8, 2, 2), f(600, 256), i(9), f(8), f(1), f(300, 8)]
w, logits, dloss, ws = torch.randn(8, 256, 256, device="cuda"), torch.randn(300, 8, device="cuda"), torch.ones(1, device="cuda"), c(1 << 20)
def run():
    bq.moe_expert_plan(idx, 8, *T[:4])
    bq.moe_fp8_quantize(x, T[4], T[5], rows=T[2])
    bq.moe_fp8_quantize_weight(w, T[6], T[7])
    bq.moe_fp8_grouped_matmul(T[4], T[5], T[6], T[7], T[1], T[8])
    bq.moe_balance_loss(logits, idx, T[9], T[10], T[11], ws)
    bq.moe_balance_loss_backward(logits, T[9], 2, dloss, T[12])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in T]
for t in T:
    t.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, T)) and float(T[8].abs().sum()) > 0
print("same")
"""


def test_first_calls_may_be_captured():
    """A process whose first calls of every operator are inside a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_operators_between_layer_forwards():
    """Operators and whole-layer forwards one after another on one stream, nothing waited for (each is set up
    while the one before it finishes), eager and captured: the results of the calls run one by one."""
    import synth
    from harness import router_to_device, to_device
    m = bq()
    wl = synth.WORKLOADS["tiny_q8"]
    li = synth.layer_inputs(wl, 0)
    packs, xs, outs = [], [], []
    for T in (1, 4):  # the single-token kernel and the one-launch tail
        packs.append(m.pack_layer(li, max_tokens=T))
        xs.append(to_device(synth.tokens(wl, li.router, 0, 0, T)))
        outs.append(torch.zeros(T, wl.hidden, device="cuda"))
    wr = router_to_device(li.router)
    layer = Layer(40, 16, 4, 256, 128, 9)
    layer.logits.copy_(layer.x.float() @ layer.router.float().t())

    def forward(i):
        m.moe_layer_forward(xs[i], wr, packs[i], m.MOE_FMT_FROM_PACK, wl.top_k, outs[i])

    def sequence(wait):
        for i in (0, 1, 0, 1):
            layer.run()
            wait()
            forward(i)
            wait()

    results = lambda: [t.clone() for t in (*outs, layer.y, layer.dlogits, layer.loss, layer.slots)]
    sequence(torch.cuda.synchronize)
    want = results()
    for _ in range(3):
        for t in (*outs, layer.y, layer.dlogits, layer.loss):
            t.zero_()
        sequence(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sequence(lambda: None)
    for _ in range(3):
        for t in (*outs, layer.y, layer.dlogits, layer.loss):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    for p in packs:
        assert m.moe_get_device_error(p) == m.MOE_OK
        p.free()
