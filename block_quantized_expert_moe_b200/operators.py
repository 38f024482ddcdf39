"""Binding of the operators beside the layer (include/moe.h): the expert plan, the
router's balance loss, the E4M3 quantisers and the E4M3 products.

Argument checks and marshalling only.  Small calls are bound by this code, so
it is written for few interpreter steps: one attribute read per property, no
imports inside functions, plain integers handed to ctypes.  Each call runs on its
tensors' device, on `stream` or that device's current stream.
"""
import torch

from . import MOE_DT_BF16, MOE_DT_F32, MOE_OK, MoeError, lib

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_FLOAT_CODE = {_F32: MOE_DT_F32, _BF16: MOE_DT_BF16}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_MASKS = (torch.bool, torch.uint8)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(t, name, dtypes, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, not {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _tensor(t, name, dtypes, shape):
    """A contiguous tensor of one of `dtypes` and of `shape`."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    _refuse(t, name, dtypes, shape)
    raise ValueError(f"{name} must be contiguous")


def _shape(t, name, dims):
    shape = getattr(t, "shape", ())
    if len(shape) != dims:
        raise ValueError(f"{name} must be {dims}-D, not of shape {tuple(shape)}")
    return shape


def _float_code(t, name):
    code = _FLOAT_CODE.get(getattr(t, "dtype", None))
    if code is None:
        raise TypeError(f"{name} must be a torch.float32 or torch.bfloat16 tensor, not "
                        f"{getattr(t, 'dtype', type(t).__name__)}")
    return code


def _rows(t, name, dtypes, shape):
    """A tensor whose rows are contiguous and do not overlap; returns the row stride."""
    cols = shape[-1]
    try:
        if t.dtype in dtypes and t.shape == shape:
            stride = t.stride()
            if stride[-1] == 1 or cols <= 1:
                if shape[-2] <= 1:
                    return cols  # one row (or none): its stride is never used
                if stride[-2] >= cols:
                    return stride[-2]
                raise ValueError(f"{name}'s rows must not overlap")
            raise ValueError(f"{name}'s last dimension must be contiguous")
    except AttributeError:
        pass
    _refuse(t, name, dtypes, shape)


def _code_rows(t, name, shape):
    """Rows of E4M3 codes: their stride in bytes, a multiple of 16."""
    ld = _rows(t, name, _CODES, shape)
    if ld % 16:
        if shape[-2] <= 1:
            return ld + -ld % 16
        raise ValueError(f"{name}'s rows must start on multiples of 16 bytes (row stride {ld}): "
                         "allocate them a multiple of 16 wide and take the first columns")
    return ld


def _off_device(names, tensors, device):
    for name, t in zip(names, tensors):
        if t is not None:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor: the library reads and writes device memory")
            if t.get_device() != device:
                raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{device}")


def _run(fn, names, tensors, args, stream):
    """Checks that every tensor is on one CUDA device, then calls fn(*args, stream) with that device current."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device or device < 0:
            _off_device(names, tensors, device)
    if not tensors[0].is_cuda:
        _off_device(names, tensors, device)
    if stream is None:
        s = _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if torch.cuda.current_device() == device:
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != MOE_OK:
        raise MoeError(status, fn.__name__)


_PLAN = ("idx", "counts", "offsets", "rows", "slots")


def moe_expert_plan(idx, n_experts, counts, offsets, rows, slots, stream=None):
    """The (token, choice) pairs of idx (CUDA int32 [T, k], as moe_route_topk writes
    it; values outside [0, n_experts) are no choice) sorted by expert: counts
    int32 [E], offsets int32 [E + 1], rows int32 [T * k] (each slot's token, -1
    behind the last one in use), slots int32 [T, k] (each pair's slot or -1)."""
    T, k = shape = _shape(idx, "idx", 2)
    i32 = (_I32,)
    _tensor(idx, "idx", i32, shape)
    _tensor(counts, "counts", i32, (n_experts,))
    _tensor(offsets, "offsets", i32, (n_experts + 1,))
    _tensor(rows, "rows", i32, (T * k,))
    _tensor(slots, "slots", i32, shape)
    _run(lib.moe_expert_plan, _PLAN, (idx, counts, offsets, rows, slots),
         (idx.data_ptr(), T, k, n_experts, counts.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr()),
         stream)


def moe_balance_loss_workspace_bytes(n_tokens, n_experts):
    return lib.moe_balance_loss_workspace_bytes(n_tokens, n_experts)


_LOSS = ("logits", "idx", "counts", "prob_mean", "loss", "workspace", "valid")


def moe_balance_loss(logits, idx, counts, prob_mean, loss, workspace=None, valid=None, stream=None):
    """Balance loss of router logits (CUDA [T, E] float32/bfloat16) and choices idx
    (int32 [T, k]) over the tokens `valid` marks (bool/uint8 [T]; None: all):
    loss float32 [1] = sum_e f_e P_e, counts int32 [E + 1] (choices per expert, then
    the tokens that count), prob_mean float32 [E] (P).  workspace: CUDA tensor of
    moe_balance_loss_workspace_bytes(T, E) bytes (None when that is 0)."""
    T, E = shape = _shape(logits, "logits", 2)
    k = _shape(idx, "idx", 2)[1]
    dt = _float_code(logits, "logits")
    _tensor(logits, "logits", (logits.dtype,), shape)
    _tensor(idx, "idx", (_I32,), (T, k))
    _tensor(counts, "counts", (_I32,), (E + 1,))
    _tensor(prob_mean, "prob_mean", (_F32,), (E,))
    _tensor(loss, "loss", (_F32,), (1,))
    mask = ws = None
    ws_bytes = 0
    if valid is not None:
        _tensor(valid, "valid", _MASKS, (T,))
        mask = valid.data_ptr()
    if workspace is not None:
        _tensor(workspace, "workspace", (workspace.dtype,), workspace.shape)
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    _run(lib.moe_balance_loss, _LOSS, (logits, idx, counts, prob_mean, loss, workspace, valid),
         (logits.data_ptr(), dt, idx.data_ptr(), mask, T, E, k, loss.data_ptr(), counts.data_ptr(),
          prob_mean.data_ptr(), ws, ws_bytes), stream)


_LOSS_BACKWARD = ("logits", "counts", "dloss", "dlogits", "valid")


def moe_balance_loss_backward(logits, counts, top_k, dloss, dlogits, valid=None, stream=None):
    """Gradient of moe_balance_loss: dlogits (type and shape of logits) from the counts
    it wrote and dloss (float32 [1], the gradient of the loss)."""
    T, E = shape = _shape(logits, "logits", 2)
    dt = _float_code(logits, "logits")
    same = (logits.dtype,)
    _tensor(logits, "logits", same, shape)
    _tensor(counts, "counts", (_I32,), (E + 1,))
    _tensor(dloss, "dloss", (_F32,), (1,))
    _tensor(dlogits, "dlogits", same, shape)
    mask = None
    if valid is not None:
        _tensor(valid, "valid", _MASKS, (T,))
        mask = valid.data_ptr()
    _run(lib.moe_balance_loss_backward, _LOSS_BACKWARD, (logits, counts, dloss, dlogits, valid),
         (logits.data_ptr(), dt, counts.data_ptr(), mask, dloss.data_ptr(), T, E, top_k, dlogits.data_ptr()), stream)


_QUANTIZE = ("x", "codes", "scales", "rows")


def moe_fp8_quantize(x, codes, scales, rows=None, swiglu=False, stream=None):
    """E4M3 codes [R, C] (float8_e4m3fn or uint8, rows on multiples of 16 bytes) and
    float32 scales [ceil(C / 128), R] of x (CUDA float32/bfloat16): of its rows [R, C],
    of rows[r] for output row r (rows int32 [R]; an index outside x gives zeros),
    or, with swiglu, of silu(x[:, :C]) * x[:, C:] for x [R, 2 C]."""
    S, W = x_shape = _shape(x, "x", 2)
    R, C = shape = _shape(codes, "codes", 2)
    dt = _float_code(x, "x")
    if W != (2 * C if swiglu else C):
        raise ValueError(f"x must have {2 * C if swiglu else C} columns, not {W}")
    index = None
    if rows is not None:
        _tensor(rows, "rows", (_I32,), (R,))
        index = rows.data_ptr()
    elif S != R:
        raise ValueError(f"x must have {R} rows, not {S}")
    ld_x = _rows(x, "x", (x.dtype,), x_shape)
    ld_c = _code_rows(codes, "codes", shape)
    ld_s = _rows(scales, "scales", (_F32,), (-(-C // 128), R))
    _run(lib.moe_fp8_quantize, _QUANTIZE, (x, codes, scales, rows),
         (x.data_ptr(), dt, ld_x, index, S, R, C, 1 if swiglu else 0, codes.data_ptr(), ld_c, scales.data_ptr(), ld_s),
         stream)


_WEIGHT = ("w", "codes", "scales")


def moe_fp8_quantize_weight(w, codes, scales, stream=None):
    """E4M3 codes of w (CUDA float32/bfloat16 [N, K] or [G, N, K]) with a float32 scale
    per 128 x 128 block: scales [ceil(N / 128), ceil(K / 128)] or [G, ...]."""
    shape = getattr(w, "shape", ())
    if len(shape) not in (2, 3):
        raise ValueError(f"w must be 2-D or 3-D, not of shape {tuple(shape)}")
    dt = _float_code(w, "w")
    N, K = shape[-2:]
    G = shape[0] if len(shape) == 3 else 1
    ld_w = _rows(w, "w", (w.dtype,), shape)
    ld_c = _code_rows(codes, "codes", shape)
    _tensor(scales, "scales", (_F32,), tuple(shape[:-2]) + (-(-N // 128), -(-K // 128)))
    gs_w, gs_c = (w.stride(0), codes.stride(0)) if G > 1 else (0, 0)
    _run(lib.moe_fp8_quantize_weight, _WEIGHT, (w, codes, scales),
         (w.data_ptr(), dt, ld_w, gs_w, G, N, K, codes.data_ptr(), ld_c, gs_c, scales.data_ptr()), stream)


_PRODUCT = ("a", "a_scale", "b", "b_scale", "out", "status")


def moe_fp8_matmul(a, a_scale, b, b_scale, out, status=None, stream=None):
    """out [R, N] (CUDA float32/bfloat16) = (a with a_scale) (b with b_scale)^T: a [R, K]
    and b [N, K] E4M3 codes (float8_e4m3fn or uint8, rows on multiples of 16 bytes),
    a_scale float32 [ceil(K / 128), R], b_scale float32 [ceil(N / 128), ceil(K / 128)].
    status: int32 [1] that takes MOE_ERR_TIMEOUT if a device-side wait runs out."""
    R, K = a_shape = _shape(a, "a", 2)
    N = _shape(b, "b", 2)[0]
    dt = _float_code(out, "out")
    KB = -(-K // 128)
    ld_a, ld_b = _code_rows(a, "a", a_shape), _code_rows(b, "b", (N, K))
    ld_s = _rows(a_scale, "a_scale", (_F32,), (KB, R))
    _tensor(b_scale, "b_scale", (_F32,), (-(-N // 128), KB))
    ld_o = _rows(out, "out", (out.dtype,), (R, N))
    st = None
    if status is not None:
        _tensor(status, "status", (_I32,), (1,))
        st = status.data_ptr()
    _run(lib.moe_fp8_matmul, _PRODUCT, (a, a_scale, b, b_scale, out, status),
         (a.data_ptr(), ld_a, a_scale.data_ptr(), ld_s, R, b.data_ptr(), ld_b, b_scale.data_ptr(), N, K, out.data_ptr(),
          dt, ld_o, st), stream)


_GROUPED = ("a", "a_scale", "b", "b_scale", "offsets", "out", "status")


def moe_fp8_grouped_matmul(a, a_scale, b, b_scale, offsets, out, status=None, stream=None):
    """The product of moe_fp8_matmul per expert: rows [offsets[g], offsets[g + 1]) of a by
    matrix g of b [G, N, K] (b_scale [G, ceil(N / 128), ceil(K / 128)]); offsets int32
    [G + 1] as moe_expert_plan writes them.  Rows outside every group keep their out."""
    R, K = a_shape = _shape(a, "a", 2)
    G, N = _shape(b, "b", 3)[:2]
    dt = _float_code(out, "out")
    KB = -(-K // 128)
    ld_a, ld_b = _code_rows(a, "a", a_shape), _code_rows(b, "b", (G, N, K))
    ld_s = _rows(a_scale, "a_scale", (_F32,), (KB, R))
    _tensor(b_scale, "b_scale", (_F32,), (G, -(-N // 128), KB))
    _tensor(offsets, "offsets", (_I32,), (G + 1,))
    ld_o = _rows(out, "out", (out.dtype,), (R, N))
    st = None
    if status is not None:
        _tensor(status, "status", (_I32,), (1,))
        st = status.data_ptr()
    _run(lib.moe_fp8_grouped_matmul, _GROUPED, (a, a_scale, b, b_scale, offsets, out, status),
         (a.data_ptr(), ld_a, a_scale.data_ptr(), ld_s, R, b.data_ptr(), ld_b, b.stride(0) if G > 1 else 0,
          b_scale.data_ptr(), offsets.data_ptr(), G, N, K, out.data_ptr(), dt, ld_o, st), stream)
