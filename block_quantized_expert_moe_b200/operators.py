"""Binding of the operators beside the layer (include/moe.h): the expert plan, the
router's balance loss, the E4M3 quantisers and the E4M3 products.

Argument checks and marshalling only.  Small calls are bound by this code, so
each entry point first tests everything in one expression over plain attribute
reads; only when that fails do the checks run one by one (`_*_checks`), which
accept what the expression is too narrow for and raise the reason otherwise.
Each call runs on its tensors' device, on `stream` or that device's current
stream.
"""
import torch

from . import MOE_DT_BF16, MOE_DT_F32, MOE_ERR_TIMEOUT, MOE_OK, MoeError, lib

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_FLOAT_CODE = {_F32: MOE_DT_F32, _BF16: MOE_DT_BF16}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_MASKS = (torch.bool, torch.uint8)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_INT_MAX = 2 ** 31 - 1  # sizes cross the ABI as C ints, which ctypes would wrap without a word
_NOT_PLAIN = (AttributeError, KeyError, TypeError, ValueError)  # what the one expression raises on other arguments


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


def _sizes(**sizes):
    for name, n in sizes.items():
        if not -_INT_MAX <= n <= _INT_MAX:
            raise ValueError(f"{name} = {n}: a size must be below 2**31")


def _off_device(names, tensors):
    device = tensors[0].get_device()
    for name, t in zip(names, tensors):
        if t is not None:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor: the library reads and writes device memory")
            if t.get_device() != device:
                raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{device}")


def _run(fn, names, tensors, args, stream):
    """Checks that every tensor is on one CUDA device, then calls fn(*args, stream) with that device current."""
    first = tensors[0]
    device = first.get_device()
    same = device >= 0 and first.is_cuda
    for t in tensors:
        if t is not None and t.get_device() != device:
            same = False
    if not same:
        _off_device(names, tensors)
    if stream is None:
        s = _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if _current_device() == device:
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != MOE_OK:
        raise MoeError(status, fn.__name__)


def _plan_checks(idx, n_experts, counts, offsets, rows, slots):
    T, k = shape = _shape(idx, "idx", 2)
    i32 = (_I32,)
    _sizes(tokens=T, top_k=k, n_experts=n_experts)
    _tensor(idx, "idx", i32, shape)
    _tensor(counts, "counts", i32, (n_experts,))
    _tensor(offsets, "offsets", i32, (n_experts + 1,))
    _tensor(rows, "rows", i32, (T * k,))
    _tensor(slots, "slots", i32, shape)
    return T, k


_PLAN = ("idx", "counts", "offsets", "rows", "slots")


def moe_expert_plan(idx, n_experts, counts, offsets, rows, slots, stream=None):
    """The (token, choice) pairs of idx (CUDA int32 [T, k], as moe_route_topk writes
    it; values outside [0, n_experts) are no choice) sorted by expert: counts
    int32 [E], offsets int32 [E + 1], rows int32 [T * k] (each slot's token, -1
    behind the last one in use), slots int32 [T, k] (each pair's slot or -1)."""
    try:
        T, k = shape = idx.shape
        plain = (T | k | n_experts <= _INT_MAX and idx.dtype is _I32 and counts.dtype is _I32 and offsets.dtype is _I32 and rows.dtype is _I32
                 and slots.dtype is _I32 and slots.shape == shape and counts.shape == (n_experts,)
                 and offsets.shape == (n_experts + 1,) and rows.shape == (T * k,) and idx.is_contiguous()
                 and slots.is_contiguous() and counts.is_contiguous() and offsets.is_contiguous()
                 and rows.is_contiguous())
    except _NOT_PLAIN:
        plain = False
    if not plain:
        T, k = _plan_checks(idx, n_experts, counts, offsets, rows, slots)
    _run(lib.moe_expert_plan, _PLAN, (idx, counts, offsets, rows, slots),
         (idx.data_ptr(), T, k, n_experts, counts.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr()),
         stream)


def moe_balance_loss_workspace_bytes(n_tokens, n_experts):
    _sizes(n_tokens=n_tokens, n_experts=n_experts)
    return lib.moe_balance_loss_workspace_bytes(n_tokens, n_experts)


def _loss_checks(logits, idx, counts, prob_mean, loss, workspace, valid):
    T, E = shape = _shape(logits, "logits", 2)
    k = _shape(idx, "idx", 2)[1]
    _sizes(tokens=T, experts=E, top_k=k)
    dt = _float_code(logits, "logits")
    _tensor(logits, "logits", (logits.dtype,), shape)
    _tensor(idx, "idx", (_I32,), (T, k))
    _tensor(counts, "counts", (_I32,), (E + 1,))
    _tensor(prob_mean, "prob_mean", (_F32,), (E,))
    _tensor(loss, "loss", (_F32,), (1,))
    if valid is not None:
        _tensor(valid, "valid", _MASKS, (T,))
    if workspace is not None:
        _tensor(workspace, "workspace", (workspace.dtype,), workspace.shape)
    return T, E, k, dt


_LOSS = ("logits", "idx", "counts", "prob_mean", "loss", "workspace", "valid")


def moe_balance_loss(logits, idx, counts, prob_mean, loss, workspace=None, valid=None, stream=None):
    """Balance loss of router logits (CUDA [T, E] float32/bfloat16) and choices idx
    (int32 [T, k]) over the tokens `valid` marks (bool/uint8 [T]; None: all):
    loss float32 [1] = sum_e f_e P_e, counts int32 [E + 1] (choices per expert, then
    the tokens that count), prob_mean float32 [E] (P).  workspace: CUDA tensor of
    moe_balance_loss_workspace_bytes(T, E) bytes (None when that is 0)."""
    try:
        T, E = logits.shape
        rows, k = idx.shape
        dt = _FLOAT_CODE[logits.dtype]
        plain = (rows == T and T | E | k <= _INT_MAX and idx.dtype is _I32 and counts.dtype is _I32 and prob_mean.dtype is _F32
                 and loss.dtype is _F32 and counts.shape == (E + 1,) and prob_mean.shape == (E,) and loss.shape == (1,)
                 and logits.is_contiguous() and idx.is_contiguous() and counts.is_contiguous()
                 and prob_mean.is_contiguous()
                 and (valid is None or valid.dtype in _MASKS and valid.shape == (T,) and valid.is_contiguous())
                 and (workspace is None or workspace.is_contiguous()))
    except _NOT_PLAIN:
        plain = False
    if not plain:
        T, E, k, dt = _loss_checks(logits, idx, counts, prob_mean, loss, workspace, valid)
    mask = None if valid is None else valid.data_ptr()
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _run(lib.moe_balance_loss, _LOSS, (logits, idx, counts, prob_mean, loss, workspace, valid),
         (logits.data_ptr(), dt, idx.data_ptr(), mask, T, E, k, loss.data_ptr(), counts.data_ptr(),
          prob_mean.data_ptr(), ws, ws_bytes), stream)


def _loss_backward_checks(logits, counts, top_k, dloss, dlogits, valid):
    T, E = shape = _shape(logits, "logits", 2)
    _sizes(tokens=T, experts=E, top_k=top_k)
    dt = _float_code(logits, "logits")
    same = (logits.dtype,)
    _tensor(logits, "logits", same, shape)
    _tensor(counts, "counts", (_I32,), (E + 1,))
    _tensor(dloss, "dloss", (_F32,), (1,))
    _tensor(dlogits, "dlogits", same, shape)
    if valid is not None:
        _tensor(valid, "valid", _MASKS, (T,))
    return T, E, dt


_LOSS_BACKWARD = ("logits", "counts", "dloss", "dlogits", "valid")


def moe_balance_loss_backward(logits, counts, top_k, dloss, dlogits, valid=None, stream=None):
    """Gradient of moe_balance_loss: dlogits (type and shape of logits) from the counts
    it wrote and dloss (float32 [1], the gradient of the loss)."""
    try:
        T, E = shape = logits.shape
        dt = _FLOAT_CODE[logits.dtype]
        plain = (0 <= T | E | top_k <= _INT_MAX and dlogits.dtype is logits.dtype and counts.dtype is _I32 and dloss.dtype is _F32
                 and dlogits.shape == shape and counts.shape == (E + 1,) and dloss.shape == (1,)
                 and logits.is_contiguous() and dlogits.is_contiguous() and counts.is_contiguous()
                 and (valid is None or valid.dtype in _MASKS and valid.shape == (T,) and valid.is_contiguous()))
    except _NOT_PLAIN:
        plain = False
    if not plain:
        T, E, dt = _loss_backward_checks(logits, counts, top_k, dloss, dlogits, valid)
    mask = None if valid is None else valid.data_ptr()
    _run(lib.moe_balance_loss_backward, _LOSS_BACKWARD, (logits, counts, dloss, dlogits, valid),
         (logits.data_ptr(), dt, counts.data_ptr(), mask, dloss.data_ptr(), T, E, top_k, dlogits.data_ptr()), stream)


def _quantize_checks(x, codes, scales, rows, swiglu):
    S, W = x_shape = _shape(x, "x", 2)
    R, C = shape = _shape(codes, "codes", 2)
    _sizes(source_rows=S, rows=R, columns=W)
    dt = _float_code(x, "x")
    if W != (2 * C if swiglu else C):
        raise ValueError(f"x must have {2 * C if swiglu else C} columns, not {W}")
    if rows is not None:
        _tensor(rows, "rows", (_I32,), (R,))
    elif S != R:
        raise ValueError(f"x must have {R} rows, not {S}")
    return (S, R, C, dt, _rows(x, "x", (x.dtype,), x_shape), _code_rows(codes, "codes", shape),
            _rows(scales, "scales", (_F32,), (-(-C // 128), R)))


_QUANTIZE = ("x", "codes", "scales", "rows")


def moe_fp8_quantize(x, codes, scales, rows=None, swiglu=False, stream=None):
    """E4M3 codes [R, C] (float8_e4m3fn or uint8, rows on multiples of 16 bytes) and
    float32 scales [ceil(C / 128), R] of x (CUDA float32/bfloat16): of its rows [R, C],
    of rows[r] for output row r (rows int32 [R]; an index outside x gives zeros),
    or, with swiglu, of silu(x[:, :C]) * x[:, C:] for x [R, 2 C]."""
    try:
        S, W = x.shape
        R, C = codes.shape
        ld_x, one_x = x.stride()
        ld_c, one_c = codes.stride()
        ld_s, one_s = scales.stride()
        dt = _FLOAT_CODE[x.dtype]
        plain = (W == (C + C if swiglu else C) and S | R | W <= _INT_MAX and codes.dtype in _CODES and scales.dtype is _F32
                 and scales.shape == ((C + 127) >> 7, R) and one_x == 1 and one_c == 1
                 and (one_s == 1 or R == 1) and ld_x >= W
                 and ld_c >= C and not ld_c & 15 and ld_s >= R
                 and (S == R if rows is None else rows.dtype is _I32 and rows.shape == (R,) and rows.is_contiguous()))
    except _NOT_PLAIN:
        plain = False
    if not plain:
        S, R, C, dt, ld_x, ld_c, ld_s = _quantize_checks(x, codes, scales, rows, swiglu)
    _run(lib.moe_fp8_quantize, _QUANTIZE, (x, codes, scales, rows),
         (x.data_ptr(), dt, ld_x, None if rows is None else rows.data_ptr(), S, R, C, 1 if swiglu else 0,
          codes.data_ptr(), ld_c, scales.data_ptr(), ld_s), stream)


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
    _sizes(groups=G, rows=N, columns=K)
    ld_w = _rows(w, "w", (w.dtype,), shape)
    ld_c = _code_rows(codes, "codes", shape)
    _tensor(scales, "scales", (_F32,), tuple(shape[:-2]) + (-(-N // 128), -(-K // 128)))
    gs_w, gs_c = (w.stride(0), codes.stride(0)) if G > 1 else (0, 0)
    _run(lib.moe_fp8_quantize_weight, _WEIGHT, (w, codes, scales),
         (w.data_ptr(), dt, ld_w, gs_w, G, N, K, codes.data_ptr(), ld_c, gs_c, scales.data_ptr()), stream)


def _product_checks(a, a_scale, b, b_scale, out, groups):
    R, K = a_shape = _shape(a, "a", 2)
    b_shape = _shape(b, "b", 2 if groups is None else 3)
    N = b_shape[-2]
    _sizes(rows=R, n=N, k=K, groups=b_shape[0])
    dt = _float_code(out, "out")
    KB = -(-K // 128)
    ld_a, ld_b = _code_rows(a, "a", a_shape), _code_rows(b, "b", (*b_shape[:-1], K))
    ld_s = _rows(a_scale, "a_scale", (_F32,), (KB, R))
    _tensor(b_scale, "b_scale", (_F32,), (*b_shape[:-2], -(-N // 128), KB))
    if groups is not None:
        _tensor(groups, "offsets", (_I32,), (b_shape[0] + 1,))
    return R, K, N, dt, ld_a, ld_b, ld_s, _rows(out, "out", (out.dtype,), (R, N))


def _status(status):
    if status is None:
        return None
    _tensor(status, "status", (_I32,), (1,))
    return status.data_ptr()


_PRODUCT = ("a", "a_scale", "b", "b_scale", "out", "status")


def moe_fp8_matmul(a, a_scale, b, b_scale, out, status=None, stream=None):
    """out [R, N] (CUDA float32/bfloat16) = (a with a_scale) (b with b_scale)^T: a [R, K]
    and b [N, K] E4M3 codes (float8_e4m3fn or uint8, rows on multiples of 16 bytes),
    a_scale float32 [ceil(K / 128), R], b_scale float32 [ceil(N / 128), ceil(K / 128)].
    status: int32 [1] that takes MOE_ERR_TIMEOUT if a device-side wait runs out; without one only
    moe_fp8_get_device_error tells."""
    try:
        R, K = a.shape
        N, cols = b.shape
        ld_a, one_a = a.stride()
        ld_b, one_b = b.stride()
        ld_s, one_s = a_scale.stride()
        ld_o, one_o = out.stride()
        dt = _FLOAT_CODE[out.dtype]
        KB = (K + 127) >> 7
        plain = (cols == K and R | N | K <= _INT_MAX and a.dtype in _CODES and b.dtype in _CODES
                 and a_scale.dtype is _F32 and b_scale.dtype is _F32 and a_scale.shape == (KB, R) and b_scale.shape == ((N + 127) >> 7, KB)
                 and out.shape == (R, N) and one_a == 1 and one_b == 1 and (one_s == 1 or R == 1) and one_o == 1
                 and not (ld_a | ld_b) & 15 and ld_a >= K and ld_b >= K and ld_s >= R and ld_o >= N
                 and b_scale.is_contiguous())
    except _NOT_PLAIN:
        plain = False
    if not plain:
        R, K, N, dt, ld_a, ld_b, ld_s, ld_o = _product_checks(a, a_scale, b, b_scale, out, None)
    _run(lib.moe_fp8_matmul, _PRODUCT, (a, a_scale, b, b_scale, out, status),
         (a.data_ptr(), ld_a, a_scale.data_ptr(), ld_s, R, b.data_ptr(), ld_b, b_scale.data_ptr(), N, K, out.data_ptr(),
          dt, ld_o, _status(status)), stream)


_GROUPED = ("a", "a_scale", "b", "b_scale", "offsets", "out", "status")


def moe_fp8_grouped_matmul(a, a_scale, b, b_scale, offsets, out, status=None, stream=None):
    """The product of moe_fp8_matmul per expert: rows [offsets[g], offsets[g + 1]) of a by
    matrix g of b [G, N, K] (b_scale [G, ceil(N / 128), ceil(K / 128)]); offsets int32
    [G + 1] as moe_expert_plan writes them.  Rows outside every group keep their out.
    status as moe_fp8_matmul's."""
    try:
        R, K = a.shape
        G, N, cols = b.shape
        ld_a, one_a = a.stride()
        gs_b, ld_b, one_b = b.stride()
        ld_s, one_s = a_scale.stride()
        ld_o, one_o = out.stride()
        dt = _FLOAT_CODE[out.dtype]
        KB = (K + 127) >> 7
        plain = (cols == K and R | N | K | G <= _INT_MAX and a.dtype in _CODES and b.dtype in _CODES
                 and a_scale.dtype is _F32 and b_scale.dtype is _F32 and offsets.dtype is _I32 and a_scale.shape == (KB, R)
                 and b_scale.shape == (G, (N + 127) >> 7, KB) and offsets.shape == (G + 1,) and out.shape == (R, N)
                 and one_a == 1 and one_b == 1 and (one_s == 1 or R == 1) and one_o == 1 and not (ld_a | ld_b) & 15
                 and ld_a >= K and ld_b >= K and ld_s >= R and ld_o >= N and b_scale.is_contiguous()
                 and offsets.is_contiguous())
    except _NOT_PLAIN:
        plain = False
    if not plain:
        R, K, N, dt, ld_a, ld_b, ld_s, ld_o = _product_checks(a, a_scale, b, b_scale, out, offsets)
        G, gs_b = b.shape[0], b.stride(0)
    _run(lib.moe_fp8_grouped_matmul, _GROUPED, (a, a_scale, b, b_scale, offsets, out, status),
         (a.data_ptr(), ld_a, a_scale.data_ptr(), ld_s, R, b.data_ptr(), ld_b, gs_b if G > 1 else 0, b_scale.data_ptr(),
          offsets.data_ptr(), G, N, K, out.data_ptr(), dt, ld_o, _status(status)), stream)


def moe_fp8_get_device_error(device=None):
    """MOE_ERR_TIMEOUT if a device-side wait of a product on `device` (None: the current one) has run out
    since the last call, whose outputs are then undefined; else MOE_OK.  Waits for the device, then
    clears the error."""
    with torch.cuda.device(device):
        status = lib.moe_fp8_get_device_error()
    if status not in (MOE_OK, MOE_ERR_TIMEOUT):
        raise MoeError(status, "moe_fp8_get_device_error")
    return status
