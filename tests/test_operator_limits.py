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
