"""Python binding of the C ABI with the same names: psk_group_run,
psk_softmax_region, psk_norm_region, psk_adamw_tree, the training step's psk_embed,
psk_dropout, psk_norm_backward and psk_policy_loss (plus the host-only psk_group_check,
psk_adamw_scalars and the workspace sizes).  Each function marshals torch tensors (device memory and
the current stream) or plain host arrays into the C structs and calls the
library; every step of the hot path runs in the library's kernels.
"""

from __future__ import annotations

import ctypes

import numpy as np

from . import _native as N


def _dtype_code(t) -> int:
    """The psk_dtype of a tensor; which entry point takes which type is the
    library's to check (int32 is a group's SELECT condition type only)."""
    import torch

    if t.dtype == torch.float32:
        return N.PSK_F32
    if t.dtype == torch.bfloat16:
        return N.PSK_BF16
    if t.dtype == torch.int32:
        return N.PSK_I32
    raise TypeError(f"storage type {t.dtype} is not f32, bf16 or int32")


def _stream_handle(stream) -> int:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _program(tokens, imm):
    toks = np.ascontiguousarray(np.asarray(tokens, dtype=np.uint32).reshape(-1))
    ims = np.ascontiguousarray(np.asarray(imm if imm is not None else [], dtype=np.float32).reshape(-1))
    p = N.psk_program()
    p.tokens = toks.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32))
    p.n_tokens = int(toks.size)
    p.imm = ims.ctypes.data_as(ctypes.POINTER(ctypes.c_float)) if ims.size else None
    p.n_imm = int(ims.size)
    return p, (toks, ims)


def psk_group_check(tokens, n_inputs: int, imm=None):
    """Validate a program on the host; returns (n_nodes, n_values)."""
    p, keep = _program(tokens, imm)
    nn, ns = ctypes.c_int32(0), ctypes.c_int32(0)
    N.check(N.lib().psk_group_check(ctypes.byref(p), int(n_inputs), ctypes.byref(nn), ctypes.byref(ns)))
    return nn.value, ns.value


def _group_args(inputs, out):
    n = len(inputs)
    arr = (N.psk_input * max(n, 1))()
    for i, (t, strides) in enumerate(inputs):
        arr[i].ptr = t.data_ptr()
        arr[i].dtype = _dtype_code(t)
        st = list(strides) + [0] * (N.PSK_MAX_RANK - len(strides))
        for k in range(N.PSK_MAX_RANK):
            arr[i].stride[k] = int(st[k])
    if not out.is_contiguous():
        raise ValueError("the output must be contiguous (row-major)")
    o = N.psk_output()
    o.ptr = out.data_ptr()
    o.dtype = _dtype_code(out)
    o.rank = out.dim()
    for k, s in enumerate(out.shape):
        o.shape[k] = int(s)
    return arr, n, o


_MATH = {"exact": 0, "fast": 1}


def psk_group_prepare(tokens, imm, inputs, out, math: str = "exact") -> None:
    """Validate and compile (cached) the kernel psk_group_run would launch for
    these arguments; needs no device (tensors are inspected, not read)."""
    p, keep = _program(tokens, imm)
    arr, n, o = _group_args(inputs, out)
    N.check(N.lib().psk_group_prepare_ex(ctypes.byref(p), arr, n, ctypes.byref(o), _MATH[math]))


def psk_group_run(tokens, imm, inputs, out, stream=None, math: str = "exact") -> None:
    """inputs: list of (tensor, strides) with one element stride per output axis
    (0 = broadcast), f32 or bf16 values or int32 SELECT conditions; out: a
    contiguous row-major tensor (f32 or bf16).  math "exact" (every node
    correctly rounded) or "fast" (EXP within one f32 ulp, EXPC and ERF within
    two; GELU, LOG and TANH stay correctly rounded)."""
    p, keep = _program(tokens, imm)
    arr, n, o = _group_args(inputs, out)
    N.check(N.lib().psk_group_run_ex(ctypes.byref(p), arr, n, ctypes.byref(o), _MATH[math], _stream_handle(stream)))


def psk_group_run_interp(tokens, imm, inputs, out, stream=None, math: str = "exact") -> None:
    """psk_group_run through the library's precompiled interpreter kernel (no
    run-time compilation): the same arguments and the same result bits,
    slower."""
    p, keep = _program(tokens, imm)
    arr, n, o = _group_args(inputs, out)
    N.check(N.lib().psk_group_run_interp(ctypes.byref(p), arr, n, ctypes.byref(o), _MATH[math],
                                         _stream_handle(stream)))


_ORDER = {"sequential": N.PSK_ORDER_SEQUENTIAL, "blocked": N.PSK_ORDER_BLOCKED,
          "interleaved": N.PSK_ORDER_INTERLEAVED}


def psk_softmax_region(x, y, order=("sequential",), exp_mode: str = "exact", stream=None) -> None:
    """Row softmax of the 2-D tensor x into y (same shape; row strides may
    exceed the row length).  order: ("sequential",), ("blocked", w) or
    ("interleaved", P); exp_mode: "exact" (correctly rounded) or "fast"."""
    if x.dim() != 2 or y.dim() != 2 or tuple(x.shape) != tuple(y.shape):
        raise ValueError("x and y must be 2-D tensors of one shape")
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("rows must be contiguous")
    o = N.psk_order(_ORDER[order[0]], int(order[1]) if len(order) > 1 else 0)
    em = {"exact": N.PSK_EXP_EXACT, "fast": N.PSK_EXP_FAST}[exp_mode]
    rows, cols = x.shape
    N.check(N.lib().psk_softmax_region(x.data_ptr(), _dtype_code(x), y.data_ptr(), _dtype_code(y), rows, cols,
                                       max(x.stride(0), cols), max(y.stride(0), cols), o, em, _stream_handle(stream)))


def _rows2d(*ts):
    for t in ts:
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("row regions take 2-D tensors with contiguous rows")
    if len({tuple(t.shape) for t in ts}) != 1:
        raise ValueError("the row tensors must share one shape")


def psk_softmax_masked(x, y, mask, order=("sequential",), exp_mode: str = "exact", stream=None) -> None:
    """Masked softmax of the rows of x into y; mask: a uint8/bool device tensor
    of shape [cols] (every row) or [rows, cols] (contiguous rows), nonzero
    allows."""
    import torch

    _rows2d(x, y)
    rows, cols = x.shape
    if mask.dtype not in (torch.uint8, torch.bool):
        raise TypeError("the mask must be uint8 or bool")
    if mask.dim() == 1:
        if mask.numel() != cols or (cols > 1 and mask.stride(0) != 1):
            raise ValueError("a mask row must hold cols contiguous values")
        ldm = 0
    else:
        if tuple(mask.shape) != (rows, cols) or mask.stride(1) != 1:
            raise ValueError("a full mask must be [rows, cols] with contiguous rows")
        ldm = max(mask.stride(0), cols)
    o = N.psk_order(_ORDER[order[0]], int(order[1]) if len(order) > 1 else 0)
    em = {"exact": N.PSK_EXP_EXACT, "fast": N.PSK_EXP_FAST}[exp_mode]
    N.check(N.lib().psk_softmax_masked(x.data_ptr(), _dtype_code(x), y.data_ptr(), _dtype_code(y), rows, cols,
                                       max(x.stride(0), cols), max(y.stride(0), cols), mask.data_ptr(), ldm, o, em,
                                       _stream_handle(stream)))


def psk_softmax_backward(y, ct, dx, order=("sequential",), stream=None) -> None:
    """dx = y (ct - sum(ct y)) per row (the softmax region's backward)."""
    _rows2d(y, ct, dx)
    rows, cols = y.shape
    o = N.psk_order(_ORDER[order[0]], int(order[1]) if len(order) > 1 else 0)
    N.check(N.lib().psk_softmax_backward(y.data_ptr(), _dtype_code(y), ct.data_ptr(), _dtype_code(ct),
                                         dx.data_ptr(), _dtype_code(dx), rows, cols, max(y.stride(0), cols),
                                         max(ct.stride(0), cols), max(dx.stride(0), cols), o,
                                         _stream_handle(stream)))


def psk_norm_region(x, y, kind: str, eps: float, gamma=None, beta=None, order=("sequential",),
                    stream=None) -> None:
    """RMSNorm (kind "rms") or LayerNorm ("layer") of the rows of the 2-D
    tensor x into y; gamma / beta: optional 1-D tensors of x's row length, both
    of one storage type."""
    if x.dim() != 2 or y.dim() != 2 or tuple(x.shape) != tuple(y.shape):
        raise ValueError("x and y must be 2-D tensors of one shape")
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("rows must be contiguous")
    params = [t for t in (gamma, beta) if t is not None]
    for t in params:
        if t.dim() != 1 or t.numel() != x.shape[1] or (t.numel() > 1 and t.stride(0) != 1):
            raise ValueError("gamma and beta must be contiguous vectors of the row length")
    if len(params) == 2 and gamma.dtype != beta.dtype:
        raise TypeError("gamma and beta must share one storage type")
    pdt = _dtype_code(params[0]) if params else N.PSK_F32
    o = N.psk_order(_ORDER[order[0]], int(order[1]) if len(order) > 1 else 0)
    k = {"rms": N.PSK_NORM_RMS, "layer": N.PSK_NORM_LAYER}[kind]
    rows, cols = x.shape
    N.check(N.lib().psk_norm_region(x.data_ptr(), _dtype_code(x), y.data_ptr(), _dtype_code(y), rows, cols,
                                    max(x.stride(0), cols), max(y.stride(0), cols), k, float(eps),
                                    gamma.data_ptr() if gamma is not None else None,
                                    beta.data_ptr() if beta is not None else None, pdt, o, _stream_handle(stream)))


def psk_device_status(reset: bool = False) -> int:
    """The pipelined kernels' status word (0: no bounded wait ever timed out)."""
    v = ctypes.c_uint32(0)
    N.check(N.lib().psk_device_status(ctypes.byref(v), 1 if reset else 0))
    return v.value


def psk_test_drop_row(row: int) -> None:
    """Test hook: the pipelined row-region kernels stop producing at local row
    `row` of every CTA (their bounded waits then run out); -1 turns it off."""
    N.check(N.lib().psk_test_drop_row(int(row)))


def psk_test_fast_exp(x, y, stream=None) -> None:
    """Test hook: y = the softmax region's fast exp of x elementwise (f32
    device tensors of equal size, x <= 0)."""
    import torch

    if x.dtype != torch.float32 or y.dtype != torch.float32 or x.numel() != y.numel():
        raise TypeError("x and y must be f32 tensors of equal size")
    if not (x.is_contiguous() and y.is_contiguous()):
        raise ValueError("x and y must be contiguous")
    N.check(N.lib().psk_test_fast_exp(x.data_ptr(), y.data_ptr(), x.numel(), _stream_handle(stream)))


def _hparams(hp) -> N.psk_adamw_hparams:
    h = N.psk_adamw_hparams()
    h.lr, h.beta1, h.beta2 = float(hp.lr), float(hp.beta1), float(hp.beta2)
    h.eps, h.weight_decay, h.t = float(hp.eps), float(hp.weight_decay), int(hp.t)
    return h


def psk_adamw_scalars(hp):
    """The nine f32 scalars the step reads (b1, b2, 1-b1, 1-b2, 1-b1^t, 1-b2^t, lr, eps, wd)."""
    h = _hparams(hp)
    out = (ctypes.c_float * 9)()
    N.check(N.lib().psk_adamw_scalars(ctypes.byref(h), out))
    return np.array(list(out), dtype=np.float32)


def _leaf_table(leaves):
    n = len(leaves)
    arr = (N.psk_leaf * max(n, 1))()
    for i, (th, m, v, g) in enumerate(leaves):
        arr[i].theta, arr[i].m, arr[i].v, arr[i].grad = th.data_ptr(), m.data_ptr(), v.data_ptr(), g.data_ptr()
        arr[i].grad_dtype = _dtype_code(g)
        arr[i].param_dtype = _dtype_code(th)
        if _dtype_code(m) != arr[i].param_dtype or _dtype_code(v) != arr[i].param_dtype:
            raise TypeError("theta, m and v of a leaf must share one storage type")
        arr[i].numel = int(th.numel())
    return arr, n


_LR = {"constant": N.PSK_LR_CONSTANT, "linear": N.PSK_LR_LINEAR, "cosine": N.PSK_LR_COSINE}


def _schedule(kind="constant", warmup=0, total=1, grad_clip=0.0) -> N.psk_adamw_schedule:
    return N.psk_adamw_schedule(_LR[kind], int(warmup), int(total), float(grad_clip))


def psk_adamw_tree(leaves, hp, stream=None) -> None:
    """leaves: list of (theta, m, v, grad) tensors, updated in place."""
    arr, n = _leaf_table(leaves)
    h = _hparams(hp)
    N.check(N.lib().psk_adamw_tree(arr, n, ctypes.byref(h), _stream_handle(stream)))


def psk_adamw_lr(hp, kind="constant", warmup=0, total=1) -> np.float32:
    """The scheduled f32 lr of step hp.t (host only)."""
    h, sc, out = _hparams(hp), _schedule(kind, warmup, total), ctypes.c_float(0)
    N.check(N.lib().psk_adamw_lr(ctypes.byref(h), ctypes.byref(sc), ctypes.byref(out)))
    return np.float32(out.value)


def psk_adamw_workspace(leaves, kind="constant", warmup=0, total=1, grad_clip=0.0) -> int:
    """Device workspace bytes psk_adamw_tree_ex needs (0 without clipping)."""
    arr, n = _leaf_table(leaves)
    sc, out = _schedule(kind, warmup, total, grad_clip), ctypes.c_uint64(0)
    N.check(N.lib().psk_adamw_workspace(arr, n, ctypes.byref(sc), ctypes.byref(out)))
    return int(out.value)


def psk_adamw_tree_ex(leaves, hp, kind="constant", warmup=0, total=1, grad_clip=0.0, workspace=None,
                      stream=None) -> None:
    """psk_adamw_tree with a schedule and global-norm clipping; workspace: a
    device tensor of at least psk_adamw_workspace bytes (needed when clipping)."""
    arr, n = _leaf_table(leaves)
    h, sc = _hparams(hp), _schedule(kind, warmup, total, grad_clip)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    N.check(N.lib().psk_adamw_tree_ex(arr, n, ctypes.byref(h), ctypes.byref(sc), ws_ptr, ws_bytes,
                                      _stream_handle(stream)))


def psk_adamw_group_sqsums(leaves, group_sums, workspace, stream=None) -> None:
    """The squared-norm tree's group sums of `leaves` (pieces of a tree's
    leaves, each starting on a 65,536-element boundary of its leaf), leaf
    after leaf, into the f32 device tensor group_sums; workspace as for
    psk_adamw_tree_ex with clipping."""
    arr, n = _leaf_table(leaves)
    N.check(N.lib().psk_adamw_group_sqsums(arr, n, group_sums.data_ptr(), workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(), _stream_handle(stream)))


def psk_adamw_clip_scale(group_sums, groups_per_leaf, grad_clip, scale, stream=None) -> None:
    """The clip scale from a whole tree's group sums (f32 device tensor, leaf
    order) and its leaves' group counts (ints), into the one-element f32
    device tensor scale."""
    counts = (ctypes.c_int64 * max(1, len(groups_per_leaf)))(*[int(c) for c in groups_per_leaf])
    N.check(N.lib().psk_adamw_clip_scale(group_sums.data_ptr() if group_sums.numel() else None, counts,
                                         len(groups_per_leaf), float(grad_clip), scale.data_ptr(),
                                         _stream_handle(stream)))


def psk_adamw_tree_scaled(leaves, hp, scale, kind="constant", warmup=0, total=1, stream=None) -> None:
    """psk_adamw_tree_ex with every gradient scaled by the device scalar
    `scale` (a sharded step's clip scale) and the schedule's lr."""
    arr, n = _leaf_table(leaves)
    h, sc = _hparams(hp), _schedule(kind, warmup, total, 0.0)
    N.check(N.lib().psk_adamw_tree_scaled(arr, n, ctypes.byref(h), ctypes.byref(sc), scale.data_ptr(),
                                          _stream_handle(stream)))


def psk_adamw_tree_static(leaves, hp, kind="constant", warmup=0, total=1, grad_clip=0.0, stream=None) -> None:
    """psk_adamw_tree_ex whose clipping scratch is the library's fixed device
    buffer (no workspace argument; overlapping calls on one device race)."""
    arr, n = _leaf_table(leaves)
    h, sc = _hparams(hp), _schedule(kind, warmup, total, grad_clip)
    N.check(N.lib().psk_adamw_tree_static(arr, n, ctypes.byref(h), ctypes.byref(sc), _stream_handle(stream)))


# ------------------------------------------- the training step's two ends

# A call's checks run on the host before every launch: tuples and integers are
# fetched once, torch's lookups are bound on the first call.
_CODES = {}
_IDS = {}
_F32 = None
_current_device = _current_stream = None


def _bind_torch() -> None:
    global _F32, _current_device, _current_stream
    import torch

    _CODES.update({torch.float32: N.PSK_F32, torch.bfloat16: N.PSK_BF16})
    _IDS.update({torch.int32: N.PSK_I32, torch.int64: N.PSK_I64})
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_stream = raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # of tensors on a CUDA device
    _F32 = torch.float32     # last: calls on other threads bind for themselves until it is set


def _code(t, what: str) -> int:
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{what}: storage type {t.dtype} is not f32 or bf16")
    return c


def _id_code(t, what: str) -> int:
    c = _IDS.get(t.dtype)
    if c is None:
        raise TypeError(f"{what}: storage type {t.dtype} is not int32 or int64")
    return c


def _same_device(stream, first, *rest) -> int:
    """The stream's handle, the tensors checked to live on the device it runs on (the current one)."""
    if _F32 is None:
        _bind_torch()
    index = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("the tensors must live on one device")
    if index < 0:
        if any(t is not None and t.device != first.device for t in rest):
            raise ValueError("the tensors must live on one device")
        raise ValueError("the tensors must live on a CUDA device")
    if index != _current_device():
        raise ValueError(f"the tensors live on cuda:{index}, which is not the current device")
    if stream is None:
        return _current_stream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream runs on {stream.device}, the tensors live on cuda:{index}")
    return stream.cuda_stream


def _matrix(t, what: str, shape=None) -> int:
    """The leading dimension of a 2-D tensor of contiguous rows."""
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{what} must be a 2-D tensor with contiguous rows")
    if shape is not None and size != shape:
        raise ValueError(f"{what} has shape {tuple(size)}, not {tuple(shape)}")
    if t.is_contiguous():
        return size[1]
    stride = t.stride()
    if stride[1] != 1 and size[1] > 1:
        raise ValueError(f"{what} must be a 2-D tensor with contiguous rows")
    if stride[0] >= size[1]:
        return stride[0]
    if size[0] > 1:
        raise ValueError(f"{what} has rows that overlap")
    return size[1]


def _vector(t, what: str, n: int, f32: bool = False):
    """The address of a contiguous 1-D tensor of n elements (None: NULL)."""
    if t is None:
        return None
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} elements")
    if f32 and t.dtype is not _F32:
        raise TypeError(f"{what} must be f32")
    return t.data_ptr()


def _scratch(t):
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _bytes(f, *sizes) -> int:
    out = ctypes.c_uint64(0)
    N.check(f(*[int(v) for v in sizes], ctypes.byref(out)))
    return int(out.value)


def psk_embed(ids, table, y, scale: float = 1.0, stream=None) -> None:
    """y[i, :] = table[ids[i], :] * scale; ids: int32 or int64, one outside the
    table's rows marks padding and gives a zero row."""
    s = _same_device(stream, table, ids, y)
    n, (vocab, cols) = ids.numel(), table.shape
    ldt, ldy = _matrix(table, "table"), _matrix(y, "y", (n, cols))
    N.check(N.lib().psk_embed(_vector(ids, "ids", n), _id_code(ids, "ids"), n, table.data_ptr(),
                              _code(table, "table"), vocab, cols, ldt, scale, y.data_ptr(), _code(y, "y"), ldy, s))


def psk_embed_workspace(tokens: int, vocab: int, cols: int) -> int:
    """Device workspace bytes psk_embed_backward needs."""
    return _bytes(N.lib().psk_embed_workspace, tokens, vocab, cols)


def psk_embed_backward(ids, ct, dtable, scale: float = 1.0, accumulate: bool = False, workspace=None,
                       stream=None) -> None:
    """dtable[v, :] = scale * (sum of ct[i, :] over ids[i] == v), every row
    written; with accumulate added to the rows that occur, the others left as
    they are.  workspace: a device tensor of at least psk_embed_workspace
    bytes."""
    s = _same_device(stream, dtable, ids, ct, workspace)
    n, (vocab, cols) = ids.numel(), dtable.shape
    ldd, ldc = _matrix(dtable, "dtable"), _matrix(ct, "ct", (n, cols))
    ws, wb = _scratch(workspace)
    N.check(N.lib().psk_embed_backward(_vector(ids, "ids", n), _id_code(ids, "ids"), n, ct.data_ptr(),
                                       _code(ct, "ct"), ldc, scale, dtable.data_ptr(), _code(dtable, "dtable"), vocab,
                                       cols, ldd, 1 if accumulate else 0, ws, wb, s))


def psk_dropout(x, y, p: float, seed: int, offset: int = 0, residual=None, counter=None, stream=None) -> None:
    """y = [residual +] dropout(x) of 2-D tensors (a 1-D tensor as one row),
    the mask drawn from (row, column, seed, offset) and never stored: the
    backward is psk_dropout(ct, dx, p, seed, offset).  counter: a one-element
    int64 device tensor added to offset when the kernel runs (for captured
    graphs)."""
    s = _same_device(stream, x, y, residual, counter)
    if x.dim() == 1:
        if y.dim() != 1 or (residual is not None and residual.dim() != 1):
            raise ValueError("x, y and the residual must have the same shape")
        x, y = x[None], y[None]
        residual = None if residual is None else residual[None]
    ldx, ldy = _matrix(x, "x"), _matrix(y, "y", x.shape)
    ldr = 0 if residual is None else _matrix(residual, "residual", x.shape)
    if counter is not None and (_IDS.get(counter.dtype) != N.PSK_I64 or counter.numel() != 1):
        raise TypeError("counter must be a one-element int64 tensor")
    for v, what in ((seed, "seed"), (offset, "offset")):
        if not 0 <= v < 1 << 64:
            raise ValueError(f"{what} must be in [0, 2^64)")
    rows, cols = x.shape
    N.check(N.lib().psk_dropout(x.data_ptr(), _code(x, "x"), None if residual is None else residual.data_ptr(),
                                0 if residual is None else _code(residual, "residual"), y.data_ptr(), _code(y, "y"),
                                rows, cols, ldx, ldr, ldy, p, seed, offset,
                                None if counter is None else counter.data_ptr(), s))


_NORM = {"rms": N.PSK_NORM_RMS, "layer": N.PSK_NORM_LAYER}


def psk_norm_backward_workspace(rows: int, cols: int) -> int:
    """Device workspace bytes psk_norm_backward needs."""
    return _bytes(N.lib().psk_norm_backward_workspace, rows, cols)


def psk_norm_backward(x, ct, dx, kind: str, eps: float, gamma=None, dgamma=None, dbeta=None, workspace=None,
                      stream=None) -> None:
    """The backward of psk_norm_region(x, y, kind, eps, gamma, beta): dx from
    the cotangent ct of y, and the gradients of gamma and beta (1-D, one
    storage type; None: not wanted).  workspace: a device tensor of at least
    psk_norm_backward_workspace bytes."""
    s = _same_device(stream, x, ct, dx, gamma, dgamma, dbeta, workspace)
    rows, cols = x.shape
    ldx, ldc, ldd = _matrix(x, "x"), _matrix(ct, "ct", x.shape), _matrix(dx, "dx", x.shape)
    g = dgamma if dgamma is not None else dbeta
    if dgamma is not None and dbeta is not None and dgamma.dtype != dbeta.dtype:
        raise TypeError("dgamma and dbeta must share one storage type")
    ws, wb = _scratch(workspace)
    N.check(N.lib().psk_norm_backward(x.data_ptr(), _code(x, "x"), ct.data_ptr(), _code(ct, "ct"), dx.data_ptr(),
                                      _code(dx, "dx"), rows, cols, ldx, ldc, ldd, _NORM[kind], eps,
                                      _vector(gamma, "gamma", cols), 0 if gamma is None else _code(gamma, "gamma"),
                                      _vector(dgamma, "dgamma", cols), _vector(dbeta, "dbeta", cols),
                                      0 if g is None else _code(g, "dgamma"), ws, wb, s))


def psk_token_logp(logits, targets, logp, scale: float = 1.0, stream=None) -> None:
    """logp[r] = log softmax(scale * logits[r])[targets[r]] (f32); targets:
    int32 or int64, one outside the row marks padding (logp 0)."""
    s = _same_device(stream, logits, targets, logp)
    rows, cols = logits.shape
    ldl = _matrix(logits, "logits")
    N.check(N.lib().psk_token_logp(logits.data_ptr(), _code(logits, "logits"), rows, cols, ldl, scale,
                                   _vector(targets, "targets", rows), _id_code(targets, "targets"),
                                   _vector(logp, "logp", rows, True), s))


def psk_policy_loss_workspace(rows: int, cols: int) -> int:
    """Device workspace bytes psk_policy_loss needs."""
    return _bytes(N.lib().psk_policy_loss_workspace, rows, cols)


def psk_policy_loss(logits, targets, old_logp, advantage, weight, loss, logp=None, dlogits=None, ref_logp=None,
                    clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, scale: float = 1.0,
                    workspace=None, stream=None) -> None:
    """The clipped policy loss with a KL term over rows of vocabulary logits:
    loss (two f32: loss, weighted KL sum), logp (f32 per row; None: not
    wanted) and, unless None, dlogits (may be the logits in place).  weight:
    f32 per row (0 leaves a row out), None: 1 / rows.  workspace: a device
    tensor of at least psk_policy_loss_workspace bytes."""
    s = _same_device(stream, logits, targets, old_logp, advantage, weight, loss, logp, dlogits, ref_logp, workspace)
    rows, cols = logits.shape
    ldl = _matrix(logits, "logits")
    ldg = 0 if dlogits is None else _matrix(dlogits, "dlogits", logits.shape)
    ws, wb = _scratch(workspace)
    N.check(N.lib().psk_policy_loss(logits.data_ptr(), _code(logits, "logits"), rows, cols, ldl, scale,
                                    _vector(targets, "targets", rows), _id_code(targets, "targets"),
                                    _vector(old_logp, "old_logp", rows, True),
                                    _vector(ref_logp, "ref_logp", rows, True),
                                    _vector(advantage, "advantage", rows, True),
                                    _vector(weight, "weight", rows, True), clip_low, clip_high, kl_coef,
                                    _vector(loss, "loss", 2, True), _vector(logp, "logp", rows, True),
                                    None if dlogits is None else dlogits.data_ptr(),
                                    0 if dlogits is None else _code(dlogits, "dlogits"), ldg, ws, wb, s))
