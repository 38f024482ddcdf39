"""Limits of the operators beside the layer that show without a device."""
import pytest
import torch

import block_quantized_expert_moe_b200 as bq

F32, I32, U8 = torch.float32, torch.int32, torch.uint8
BIG = 2 ** 32 + 4  # would arrive as 4


def t(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="meta")  # a shape without memory


CASES = {
    "plan of many tokens": lambda: bq.moe_expert_plan(
        t(BIG, 1, dtype=I32), 4, t(4, dtype=I32), t(5, dtype=I32), t(BIG, dtype=I32), t(BIG, 1, dtype=I32)),
    "plan of many experts": lambda: bq.moe_expert_plan(
        t(3, 2, dtype=I32), BIG, t(BIG, dtype=I32), t(BIG + 1, dtype=I32), t(6, dtype=I32), t(3, 2, dtype=I32)),
    "workspace of many tokens": lambda: bq.moe_balance_loss_workspace_bytes(BIG, 8),
    "workspace of many experts": lambda: bq.moe_balance_loss_workspace_bytes(8, BIG),
    "loss of many tokens": lambda: bq.moe_balance_loss(t(BIG, 4), t(BIG, 2, dtype=I32), t(5, dtype=I32), t(4), t(1)),
    "loss of many experts": lambda: bq.moe_balance_loss(
        t(4, BIG), t(4, 2, dtype=I32), t(BIG + 1, dtype=I32), t(BIG), t(1)),
    "gradient of many tokens": lambda: bq.moe_balance_loss_backward(t(BIG, 4), t(5, dtype=I32), 2, t(1), t(BIG, 4)),
    "gradient of many choices": lambda: bq.moe_balance_loss_backward(t(3, 4), t(5, dtype=I32), BIG, t(1), t(3, 4)),
    "gradient of choices far below": lambda: bq.moe_balance_loss_backward(
        t(3, 4), t(5, dtype=I32), 2 - 2 ** 32, t(1), t(3, 4)),
    "quantiser of many rows": lambda: bq.moe_fp8_quantize(t(BIG, 16), t(BIG, 16, dtype=U8), t(1, BIG)),
    "quantiser of many source rows": lambda: bq.moe_fp8_quantize(
        t(BIG, 16), t(3, 16, dtype=U8), t(1, 3), rows=t(3, dtype=I32)),
    "quantiser of many columns": lambda: bq.moe_fp8_quantize(
        t(1, 2 ** 32 + 16), t(1, 2 ** 32 + 16, dtype=U8), t(2 ** 25 + 1, 1)),
    "SwiGLU of many columns": lambda: bq.moe_fp8_quantize(
        t(1, 2 ** 32 + 32), t(1, 2 ** 31 + 16, dtype=U8), t(2 ** 24 + 1, 1), swiglu=True),
    "weights of many rows": lambda: bq.moe_fp8_quantize_weight(
        t(2 ** 32 + 128, 16), t(2 ** 32 + 128, 16, dtype=U8), t(2 ** 25 + 1, 1)),
    "weights of many groups": lambda: bq.moe_fp8_quantize_weight(
        t(BIG, 3, 16), t(BIG, 3, 16, dtype=U8), t(BIG, 1, 1)),
    "product of many rows": lambda: bq.moe_fp8_matmul(
        t(BIG, 16, dtype=U8), t(1, BIG), t(5, 16, dtype=U8), t(1, 1), t(BIG, 5)),
    "product of many columns": lambda: bq.moe_fp8_matmul(
        t(3, 16, dtype=U8), t(1, 3), t(2 ** 32 + 128, 16, dtype=U8), t(2 ** 25 + 1, 1), t(3, 2 ** 32 + 128)),
    "grouped product of many rows": lambda: bq.moe_fp8_grouped_matmul(
        t(BIG, 16, dtype=U8), t(1, BIG), t(2, 5, 16, dtype=U8), t(2, 1, 1), t(3, dtype=I32), t(BIG, 5)),
    "grouped product of many groups": lambda: bq.moe_fp8_grouped_matmul(
        t(3, 16, dtype=U8), t(1, 3), t(BIG, 5, 16, dtype=U8), t(BIG, 1, 1), t(BIG + 1, dtype=I32), t(3, 5)),
}


@pytest.mark.parametrize("case", CASES)
def test_binding_refuses_sizes_that_a_c_int_would_wrap(case):
    with pytest.raises(ValueError, match=r"2\*\*31"):
        CASES[case]()


def test_stall_injection_refuses_other_negative_numbers():
    with pytest.raises(bq.MoeError):
        bq.moe_debug_fp8_stall_after(-2)
    bq.moe_debug_fp8_stall_after(-1)


def test_balance_loss_refuses_more_choices_than_its_counts_hold():
    """Counts are int32, and one expert may be named by every choice."""
    from test_operators_abi import INVALID, call
    assert call("moe_balance_loss", T=1 << 30, k=2, ws_bytes=1 << 16) == INVALID
    assert call("moe_balance_loss", T=(1 << 28) + 1, k=8, ws_bytes=1 << 16) == INVALID


# ---- every rule is written twice: in one expression, and as checks with their reasons ------------------

def cpu(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def layouts():
    """Calls that are right: contiguous, in wider buffers, of one row, one column, one group, no row."""
    c = cpu
    yield "plan", bq.moe_expert_plan, (c(3, 2, dtype=I32), 4, c(4, dtype=I32), c(5, dtype=I32), c(6, dtype=I32),
                                       c(3, 2, dtype=I32))
    yield "no tokens", bq.moe_expert_plan, (c(0, 2, dtype=I32), 4, c(4, dtype=I32), c(5, dtype=I32), c(0, dtype=I32),
                                            c(0, 2, dtype=I32))
    for dt in (F32, torch.bfloat16):
        for valid in (None, c(3, dtype=torch.bool), c(3, dtype=U8)):
            yield "loss", bq.moe_balance_loss, (c(3, 4, dtype=dt), c(3, 2, dtype=I32), c(5, dtype=I32), c(4), c(1),
                                                c(64, dtype=U8), valid)
            yield "gradient", bq.moe_balance_loss_backward, (c(3, 4, dtype=dt), c(5, dtype=I32), 2, c(1),
                                                             c(3, 4, dtype=dt), valid)
    for R, C in ((5, 32), (5, 130), (1, 33), (0, 32), (5, 1), (1, 1)):
        codes, scales = c(R, -(-C // 16) * 16, dtype=U8)[:, :C], c(-(-C // 128), R + 3)[:, 2:R + 2]
        yield "rows", bq.moe_fp8_quantize, (c(R, C), codes, scales)
        yield "wider", bq.moe_fp8_quantize, (c(R, C + 5)[:, 3:C + 3], codes, scales)
        yield "gather", bq.moe_fp8_quantize, (c(9, C), codes, scales, c(R, dtype=I32))
        yield "swiglu", bq.moe_fp8_quantize, (c(R, 2 * C), codes, scales, None, True)
    for R, N, K in ((5, 7, 32), (5, 200, 130), (1, 7, 32), (5, 1, 32), (5, 7, 1), (1, 1, 1), (0, 7, 32)):
        kb, nb, w = -(-K // 128), -(-N // 128), -(-K // 16) * 16
        a, sa, out = c(R, w + 16, dtype=U8)[:, :K], c(kb, R + 2)[:, :R], c(R, N + 3)[:, 1:N + 1]
        b = c(N, w, dtype=U8)[:, :K].view(torch.float8_e4m3fn)
        yield "product", bq.moe_fp8_matmul, (a, sa, b, c(nb, kb), out)
        yield "status", bq.moe_fp8_matmul, (a, sa, b, c(nb, kb), c(R, N, dtype=torch.bfloat16), c(1, dtype=I32))
        for G in (1, 3):
            b = c(G, N, w, dtype=U8)[..., :K]
            yield "groups", bq.moe_fp8_grouped_matmul, (a, sa, b, c(G, nb, kb), c(G + 1, dtype=I32), out)


CALLS = [(f"{name}-{i}", fn, args) for i, (name, fn, args) in enumerate(layouts())]


@pytest.fixture
def recorded(monkeypatch):
    """The arguments that reach the library, by the expression first or by the checks alone."""
    from block_quantized_expert_moe_b200 import operators

    def run(fn, args, checks):
        calls = []
        with monkeypatch.context() as m:
            m.setattr(operators, "_run", lambda f, names, tensors, values, stream: calls.append((f, values)))
            if checks:  # no size passes the expression
                m.setattr(operators, "_INT_MAX", -1)
                m.setattr(operators, "_sizes", lambda **sizes: None)
            fn(*args)
        return calls
    return run


# A stride that is never used (of one row, or of a single row of scales) may differ.
UNUSED = {"moe_fp8_quantize": {2: lambda v: v[4] <= 1, 9: lambda v: v[5] <= 1, 11: lambda v: v[6] <= 128},
          "moe_fp8_matmul": {1: lambda v: v[4] <= 1, 3: lambda v: v[9] <= 128, 6: lambda v: v[8] <= 1,
                             12: lambda v: v[4] <= 1},
          "moe_fp8_grouped_matmul": {1: lambda v: v[4] <= 1, 3: lambda v: v[12] <= 128, 6: lambda v: v[11] <= 1,
                                     15: lambda v: v[4] <= 1}}


@pytest.mark.parametrize("name,fn,args", CALLS, ids=[c[0] for c in CALLS])
def test_the_expression_and_the_checks_pass_the_same_arguments(recorded, name, fn, args):
    (f, fast), = recorded(fn, args, False)
    (g, slow), = recorded(fn, args, True)
    assert f is g and len(fast) == len(slow)
    unused = UNUSED.get(f.__name__, {})
    for i, (x, y) in enumerate(zip(fast, slow)):
        assert x == y or (i in unused and unused[i](fast)), (i, fast, slow)


def test_the_checks_alone_refuse_what_the_binding_refuses(recorded):
    """The refusals of test_operators_abi, without the expression before them."""
    import test_operators_abi as abi
    params = next(m for m in abi.test_binding_refuses_bad_tensors.pytestmark if m.name == "parametrize").args[1]
    for case, over, error, match in params:
        if match == "CUDA" or "status" in over:
            continue  # refused behind the checks
        fn, args = abi.CASES[case]
        with pytest.raises(error, match=match):
            recorded(lambda: fn(**{**args, **over}), (), True)
