"""Plain 64-bit references of the operators beside the layer (expert plan, balance
loss, E4M3 quantisers, E4M3 products), written from their definitions in
include/moe.h; they share no code with the CUDA library."""
import numpy as np

FLOOR = np.float32(448.0) * np.float32(2.0 ** -126)
BLOCK = 128


def e4m3_table():
    """Values of the 256 E4M3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits, 0x7f / 0xff NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7f) == 0x7f else (-mag if c & 0x80 else mag)
    return v


E4M3 = e4m3_table()


def to_e4m3(x):
    """Nearest E4M3 values (ties to even) of x (float64, |x| <= 464); NaN stays NaN."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** -6))
    step = np.exp2(e - 4.0)
    return np.round(x / step) * step


def plan(idx, n_experts):
    T, k = idx.shape
    flat = idx.reshape(-1).astype(np.int64)
    used = (flat >= 0) & (flat < n_experts)
    counts = np.bincount(flat[used], minlength=n_experts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    rows = np.full(T * k, -1)
    slots = np.full(T * k, -1)
    order = sorted((p for p in range(T * k) if used[p]), key=lambda p: (flat[p], p))
    for s, p in enumerate(order):
        rows[s], slots[p] = p // k, s
    return counts, offsets, rows, slots.reshape(T, k)


def softmax(logits):
    with np.errstate(invalid="ignore"):
        m = logits.max(1, keepdims=True)
        e = np.exp(logits - np.where(m == -np.inf, 0.0, m))
        s = e.sum(1, keepdims=True)
        return np.where(s == 0, 0.0, e / np.where(s == 0, 1.0, s))


def balance(logits, idx, valid, dloss):
    """(loss, counts [E + 1], P [E], dlogits, p, f) in float64."""
    T, E = logits.shape
    k = idx.shape[1]
    keep = np.ones(T, bool) if valid is None else valid.astype(bool)
    n = int(keep.sum())
    p = np.zeros((T, E))
    if n:
        p[keep] = softmax(logits[keep].astype(np.float64))
    chosen = idx[keep].reshape(-1)
    counts = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
    f = counts * E / (k * max(n, 1))
    P = p.sum(0) / max(n, 1)
    dl = dloss / max(n, 1) * p * (f - (p @ f)[:, None])
    return float(f @ P), np.concatenate([counts, [n]]), P, dl, p, f


def quantize(x32, block_rows=1):
    """(codes' values, scales, inverse) of float32 x by the definition, every step in float32:
    what the kernel must give bit for bit.  x [R, C]; scales [ceil(R / block_rows), ceil(C / 128)]."""
    R, C = x32.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    scales = np.empty((rb, cb), np.float32)
    codes = np.empty((R, C))
    with np.errstate(invalid="ignore"):
        for i in range(rb):
            for j in range(cb):
                at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
                a = np.abs(x32[at]).max()
                a = a if np.isnan(a) else max(a, FLOOR)
                scales[i, j] = np.float32(a) / np.float32(448)
                inv = np.float32(448) / np.float32(a)
                codes[at] = to_e4m3((x32[at] * inv).astype(np.float64))
    return codes, scales


def swiglu(x):
    x = np.asarray(x, np.float64)
    C = x.shape[1] // 2
    g = x[:, :C]
    return g / (1 + np.exp(-g)) * x[:, C:]


def product(a, a_scale, b, b_scale):
    """(out, magnitude) in float64: a [R, K], b [N, K] code values, a_scale [KB, R],
    b_scale [NB, KB]; magnitude is the sum of the terms' absolute values."""
    R, N = a.shape[0], b.shape[0]
    y, mag = np.zeros((R, N)), np.zeros((R, N))
    for i in range(a_scale.shape[0]):
        at = slice(i * BLOCK, (i + 1) * BLOCK)
        s = a_scale[i].astype(np.float64)[:, None] * np.repeat(b_scale[:, i].astype(np.float64), BLOCK)[None, :N]
        y += (a[:, at] @ b[:, at].T) * s
        mag += (np.abs(a[:, at]) @ np.abs(b[:, at]).T) * np.abs(s)
    return y, mag


def product_bound(mag, k, out_eps_half, y):
    """Largest error of the product's fp32 sums, from the terms' magnitudes: a block's 128 products
    (exact in fp32: 4-bit by 4-bit significands) are added with at most 128 roundings of 2^-23 (the
    tensor core may truncate), each block joins the fp32 sum by one FMA, the two scales are multiplied
    with one rounding, split sums add at most 8 more; then one rounding to the output's type."""
    kb = -(-k // BLOCK)
    return mag * (min(k, BLOCK) * 2.0 ** -23 + (kb + 10) * 2.0 ** -24) + np.abs(y) * out_eps_half
