"""Argument checks of the operators beside the layer, at the C ABI and in the
binding, without a device: every refusal comes before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_expert_moe_b200 as bq

import op_reference as ref

INVALID, OK = bq.MOE_ERR_INVALID_ARG, bq.MOE_OK
BUF = np.zeros(1 << 16, np.uint8)
P = BUF.ctypes.data + (-BUF.ctypes.data % 256)


def call(name, **over):
    """Calls entry point `name` with arguments that would pass, some replaced."""
    args = {
        "moe_expert_plan": dict(idx=P, T=8, k=2, E=4, counts=P, offsets=P, rows=P, slots=P, stream=None),
        "moe_balance_loss": dict(logits=P, dt=1, idx=P, valid=None, T=4, E=8, k=2, loss=P, counts=P, pm=P, ws=P,
                                 ws_bytes=4096, stream=None),
        "moe_balance_loss_backward": dict(logits=P, dt=1, counts=P, valid=None, dloss=P, T=4, E=8, k=2, dlogits=P,
                                          stream=None),
        "moe_fp8_quantize": dict(x=P, dt=1, ld=128, rows=None, S=4, R=4, C=128, swiglu=0, codes=P, ldc=128, scales=P,
                                 lds=4, stream=None),
        "moe_fp8_quantize_weight": dict(w=P, dt=1, ld=128, gs=0, G=1, N=4, C=128, codes=P, ldc=128, gsc=0, scales=P,
                                        stream=None),
        "moe_fp8_matmul": dict(a=P, lda=128, sa=P, ldsa=4, R=4, b=P, ldb=128, sb=P, N=8, K=128, out=P, dt=1, ldo=8,
                               status=None, stream=None),
        "moe_fp8_grouped_matmul": dict(a=P, lda=128, sa=P, ldsa=4, R=4, b=P, ldb=128, gsb=1024, sb=P, offsets=P, G=2,
                                       N=8, K=128, out=P, dt=1, ldo=8, status=None, stream=None),
    }[name]
    assert set(over) <= set(args)
    return getattr(bq.lib, name)(*{**args, **over}.values())


@pytest.mark.parametrize("name,over", [
    ("moe_expert_plan", o) for o in (dict(T=-1), dict(k=0), dict(k=5), dict(E=0), dict(E=1025), dict(counts=None),
                                     dict(offsets=None), dict(idx=None), dict(rows=None), dict(slots=None),
                                     dict(idx=P + 2), dict(T=1 << 30, k=2))
] + [
    ("moe_balance_loss", o) for o in (dict(dt=0), dict(dt=3), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9),
                                      dict(logits=None), dict(idx=None), dict(loss=None), dict(counts=None),
                                      dict(pm=None), dict(logits=P + 2), dict(T=100000, ws=None),
                                      dict(T=100000, ws_bytes=64), dict(T=100000, ws=P + 4, ws_bytes=1 << 30))
] + [
    ("moe_balance_loss_backward", o) for o in (dict(dt=7), dict(T=-1), dict(E=1025), dict(k=0), dict(logits=None),
                                               dict(counts=None), dict(dloss=None), dict(dlogits=None),
                                               dict(dlogits=P + 1, dt=2))
] + [
    ("moe_fp8_quantize", o) for o in (dict(dt=0), dict(ld=127), dict(swiglu=1), dict(swiglu=2), dict(S=5), dict(R=-1),
                                      dict(S=-1, rows=P), dict(C=0), dict(C=(1 << 20) + 1), dict(ldc=120), dict(ldc=136),
                                      dict(lds=3), dict(x=None), dict(codes=None), dict(codes=P + 8), dict(scales=None),
                                      dict(x=P + 2), dict(rows=P + 1))
] + [
    ("moe_fp8_quantize_weight", o) for o in (dict(dt=0), dict(G=-1), dict(G=65536), dict(N=-1), dict(C=0), dict(ld=127),
                                             dict(ldc=112), dict(ldc=130), dict(gsc=8), dict(G=2, gs=4, gsc=512),
                                             dict(G=2, gs=512, gsc=16), dict(w=None), dict(codes=None),
                                             dict(codes=P + 4), dict(scales=None))
] + [
    (n, o) for n in ("moe_fp8_matmul", "moe_fp8_grouped_matmul") for o in (
        dict(dt=0), dict(R=-1), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=129), dict(lda=112), dict(lda=136),
        dict(ldb=112), dict(ldb=136), dict(ldo=7), dict(ldsa=3), dict(a=None), dict(b=None), dict(sa=None),
        dict(sb=None), dict(out=None), dict(a=P + 8), dict(b=P + 8), dict(sa=P + 2), dict(out=P + 2),
        dict(status=P + 2), dict(lda=1 << 41))
] + [
    ("moe_fp8_grouped_matmul", o) for o in (dict(offsets=None), dict(offsets=P + 2), dict(G=0), dict(G=1025),
                                            dict(gsb=1000), dict(gsb=512))
])
def test_entry_points_refuse_bad_arguments(name, over):
    assert call(name, **over) == INVALID


def test_entry_points_refuse_more_rows_than_they_index():
    big = (1 << 30) + 1
    assert call("moe_fp8_quantize", R=big, S=big, lds=big) == INVALID
    assert call("moe_fp8_matmul", R=big, ldsa=big) == INVALID
    assert call("moe_fp8_grouped_matmul", R=big, ldsa=big) == INVALID
    assert call("moe_balance_loss", T=big) == INVALID
    assert call("moe_balance_loss_backward", T=big) == INVALID


def test_empty_batches_enqueue_nothing():
    assert call("moe_balance_loss_backward", T=0, logits=None, dlogits=None, counts=None, dloss=None) == OK
    assert call("moe_fp8_quantize", R=0, S=0, x=None, codes=None, scales=None) == OK
    assert call("moe_fp8_quantize_weight", G=0, w=None, codes=None, scales=None) == OK
    assert call("moe_fp8_matmul", R=0, a=None, out=None) == OK
    assert call("moe_fp8_grouped_matmul", R=0, a=None, out=None) == OK
    assert bq.moe_balance_loss_workspace_bytes(0, 8) == 0


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


U8, I32 = torch.uint8, torch.int32
CASES = {
    "plan": (bq.moe_expert_plan, dict(idx=t(3, 2, dtype=I32), n_experts=4, counts=t(4, dtype=I32),
                                      offsets=t(5, dtype=I32), rows=t(6, dtype=I32), slots=t(3, 2, dtype=I32))),
    "balance": (bq.moe_balance_loss, dict(logits=t(3, 4), idx=t(3, 2, dtype=I32), counts=t(5, dtype=I32),
                                          prob_mean=t(4), loss=t(1))),
    "balance_bwd": (bq.moe_balance_loss_backward, dict(logits=t(3, 4), counts=t(5, dtype=I32), top_k=2, dloss=t(1),
                                                       dlogits=t(3, 4))),
    "quantize": (bq.moe_fp8_quantize, dict(x=t(3, 32), codes=t(3, 32, dtype=U8), scales=t(1, 3))),
    "weight": (bq.moe_fp8_quantize_weight, dict(w=t(2, 3, 32), codes=t(2, 3, 32, dtype=U8), scales=t(2, 1, 1))),
    "matmul": (bq.moe_fp8_matmul, dict(a=t(3, 32, dtype=U8), a_scale=t(1, 3), b=t(5, 32, dtype=U8), b_scale=t(1, 1),
                                       out=t(3, 5))),
    "grouped": (bq.moe_fp8_grouped_matmul, dict(a=t(3, 32, dtype=U8), a_scale=t(1, 3), b=t(2, 5, 32, dtype=U8),
                                                b_scale=t(2, 1, 1), offsets=t(3, dtype=I32), out=t(3, 5))),
}


@pytest.mark.parametrize("case,over,error,match", [
    ("plan", {}, ValueError, "CUDA"), ("plan", dict(idx=t(3, 2)), TypeError, "idx"),
    ("plan", dict(idx=t(3, dtype=I32)), ValueError, "2-D"), ("plan", dict(counts=t(5, dtype=I32)), ValueError, "counts"),
    ("plan", dict(rows=t(5, dtype=I32)), ValueError, "rows"),
    ("plan", dict(idx=t(2, 3, dtype=I32).t()), ValueError, "contiguous"),
    ("balance", {}, ValueError, "CUDA"), ("balance", dict(logits=t(3, 4, dtype=torch.float16)), TypeError, "logits"),
    ("balance", dict(idx=t(2, 2, dtype=I32)), ValueError, "idx"), ("balance", dict(counts=t(4, dtype=I32)), ValueError, "counts"),
    ("balance", dict(valid=t(3)), TypeError, "valid"), ("balance", dict(valid=t(4, dtype=U8)), ValueError, "valid"),
    ("balance", dict(logits=t(4, 3).t()), ValueError, "contiguous"), ("balance", dict(loss=t(2)), ValueError, "loss"),
    ("balance_bwd", {}, ValueError, "CUDA"),
    ("balance_bwd", dict(dlogits=t(3, 4, dtype=torch.bfloat16)), TypeError, "dlogits"),
    ("balance_bwd", dict(dloss=t(1, dtype=torch.float64)), TypeError, "dloss"),
    ("quantize", {}, ValueError, "CUDA"), ("quantize", dict(x=t(4, 32)), ValueError, "rows"),
    ("quantize", dict(x=t(3, 33)), ValueError, "columns"), ("quantize", dict(swiglu=True), ValueError, "columns"),
    ("quantize", dict(x=t(3, 33), codes=t(3, 33, dtype=U8)), ValueError, "16"),
    ("quantize", dict(codes=t(3, 32)), TypeError, "codes"), ("quantize", dict(scales=t(3, 1)), ValueError, "scales"),
    ("quantize", dict(rows=t(4, dtype=I32)), ValueError, "rows"), ("quantize", dict(x=t(32, 3).t()), ValueError, "contiguous"),
    ("quantize", dict(x=t(1, 32).expand(3, 32)), ValueError, "overlap"),
    ("weight", {}, ValueError, "CUDA"), ("weight", dict(scales=t(2, 1)), ValueError, "scales"),
    ("weight", dict(w=t(32)), ValueError, "2-D or 3-D"),
    ("matmul", {}, ValueError, "CUDA"), ("matmul", dict(b=t(5, 48, dtype=U8)), ValueError, "b must have shape"),
    ("matmul", dict(a=t(3, 32)), TypeError, "a must"), ("matmul", dict(a_scale=t(2, 3)), ValueError, "a_scale"),
    ("matmul", dict(b_scale=t(1, 2)), ValueError, "b_scale"), ("matmul", dict(out=t(5, 3)), ValueError, "out"),
    ("matmul", dict(out=t(3, 5, dtype=torch.float16)), TypeError, "out"),
    ("matmul", dict(out=t(5, 3).t()), ValueError, "contiguous"), ("matmul", dict(status=t(1)), TypeError, "status"),
    ("grouped", {}, ValueError, "CUDA"), ("grouped", dict(b=t(5, 32, dtype=U8)), ValueError, "3-D"),
    ("grouped", dict(offsets=t(2, dtype=I32)), ValueError, "offsets"),
    ("grouped", dict(offsets=t(3, dtype=torch.int64)), TypeError, "offsets"),
])
def test_binding_refuses_bad_tensors(case, over, error, match):
    fn, args = CASES[case]
    with pytest.raises(error, match=match):
        fn(**{**args, **over})


def test_reference_e4m3_table_and_rounding():
    """The tests' E4M3 table equals torch's type for every code, and its rounding equals torch's cast."""
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(ref.E4M3, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.ldexp(np.linspace(-3, 3, 4001), -9)]).astype(np.float32)
    assert np.array_equal(ref.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())
