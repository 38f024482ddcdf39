"""The README's combine of the experts' rows, run as it is written there, on the CPU."""
import os
import re

import numpy as np
import torch

import op_reference as ref

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def combine(y, slots, gate):
    text = open(README).read()
    lines = "\n".join(re.findall(r"^(?:chosen|out) = .*slots.*$", text, re.M))
    names = {"torch": torch, "y": y, "slots": slots, "gate": gate}
    exec(lines, names)
    return names["out"]


def test_combine_leaves_padding_out():
    """Pairs without a choice add nothing, whatever the rows that no expert wrote hold; a token of only such
    pairs is 0."""
    rng = np.random.default_rng(0)
    T, E, k, H = 40, 8, 3, 16
    idx = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[5:12] = -1
    idx[20, 1] = E
    _, offsets, rows, slots = ref.plan(idx, E)
    y = rng.standard_normal((T * k, H)).astype(np.float32)
    y[offsets[-1]:] = np.nan
    gate = rng.random((T, k)).astype(np.float32)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if 0 <= idx[t, j] < E:
                want[t] += y[slots[t, j]].astype(np.float64) * gate[t, j]
    got = combine(torch.from_numpy(y), torch.from_numpy(slots.astype(np.int32)), torch.from_numpy(gate)).numpy()
    # k products and k - 1 sums in fp32, each off by 2^-24 of at most the terms' magnitudes
    assert np.all(np.abs(got - want) <= 2 * k * 2.0 ** -24 * k * np.nanmax(np.abs(y)))
    assert not got[5:12].any()


def test_combine_without_rows():
    """Every token padded: no slot is used."""
    y = torch.full((6, 4), float("nan"))
    out = combine(y, torch.full((3, 2), -1, dtype=torch.int32), torch.ones(3, 2))
    assert out.shape == (3, 4) and not out.any()
