"""Matrix-product operators over bf16 and fp16 CUDA tensors: a linear layer
with bias, activation and residual, the same product grouped by expert, softmax
cross entropy over a vocabulary, and their gradients.

Thin ctypes layer over include/uzip_ops.h: the functions named like the C entry
points only marshal arguments, and the torch functions allocate outputs and
workspace and pass the stream.  All arithmetic runs in the library's kernels.

The torch functions are not known to autograd: a training step calls the
*_backward functions itself.  Tensors that require gradients are refused while
grad mode is on, since the results would silently have none; torch.no_grad() or
detach() says that this is meant.  So are tensors with a tangent of forward-mode
differentiation; their primals are taken.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

from . import UZIP_BF16, UZIP_ERR_INVALID_ARG, UZIP_ERR_UNSUPPORTED_DTYPE, UZIP_FP16, UZIP_OK, UzipError, _check, library

UZIP_ACT_NONE, UZIP_ACT_RELU, UZIP_ACT_GELU, UZIP_ACT_SILU = 0, 1, 2, 3
UZIP_MAX_GROUPS = 1024
ACTIVATIONS = {"none": UZIP_ACT_NONE, "relu": UZIP_ACT_RELU, "gelu": UZIP_ACT_GELU, "silu": UZIP_ACT_SILU}

_i32, _i64, _u64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_byref = ctypes.byref


class LinearArgs(ctypes.Structure):
    """uzip_linear_args"""

    _fields_ = [("dtype", _i32), ("act", _i32), ("m", _i64), ("n", _i64), ("k", _i64), ("groups", _i64),
                ("offsets", _vp), ("x", _vp), ("ldx", _i64), ("w", _vp), ("ldw", _i64), ("w_group", _i64),
                ("bias", _vp), ("residual", _vp), ("ldr", _i64), ("y", _vp), ("ldy", _i64), ("z", _vp), ("ldz", _i64)]


class LinearGradArgs(ctypes.Structure):
    """uzip_linear_grad_args"""

    _fields_ = [("dtype", _i32), ("act", _i32), ("m", _i64), ("n", _i64), ("k", _i64), ("groups", _i64),
                ("offsets", _vp), ("dy", _vp), ("lddy", _i64), ("x", _vp), ("ldx", _i64), ("w", _vp), ("ldw", _i64),
                ("w_group", _i64), ("z", _vp), ("ldz", _i64), ("dx", _vp), ("lddx", _i64), ("dw", _vp),
                ("lddw", _i64), ("dw_group", _i64), ("db", _vp)]


class CrossEntropyArgs(ctypes.Structure):
    """uzip_cross_entropy_args"""

    _fields_ = [("dtype", _i32), ("reserved", _i32), ("t", _i64), ("v", _i64), ("d", _i64), ("h", _vp), ("ldh", _i64),
                ("w", _vp), ("ldw", _i64), ("targets", _vp), ("ignore_index", _i64), ("loss", _vp), ("lse", _vp)]


class CrossEntropyGradArgs(ctypes.Structure):
    """uzip_cross_entropy_grad_args"""

    _fields_ = [("dtype", _i32), ("reserved", _i32), ("t", _i64), ("v", _i64), ("d", _i64), ("piece", _i64),
                ("h", _vp), ("ldh", _i64), ("w", _vp), ("ldw", _i64), ("targets", _vp), ("ignore_index", _i64),
                ("lse", _vp), ("dloss", _vp), ("dh", _vp), ("lddh", _i64), ("dw", _vp), ("lddw", _i64)]


_lib = library()
_calls = {}
for _name, _args in (("uzip_linear", LinearArgs), ("uzip_grouped_linear", LinearArgs),
                     ("uzip_linear_backward", LinearGradArgs), ("uzip_grouped_linear_backward", LinearGradArgs),
                     ("uzip_cross_entropy", CrossEntropyArgs), ("uzip_cross_entropy_backward", CrossEntropyGradArgs)):
    _size, _call = getattr(_lib, _name + "_workspace_size"), getattr(_lib, _name)
    _size.argtypes, _size.restype = [ctypes.POINTER(_args)], _u64
    _call.argtypes, _call.restype = [ctypes.POINTER(_args), _vp, _u64, _vp, _vp], ctypes.c_int
    _calls[_name] = (_size, _call)


# ---- C entry points (same names; `args` is one of the structures above) ----

def uzip_linear_workspace_size(args: LinearArgs) -> int:
    return int(_lib.uzip_linear_workspace_size(ctypes.byref(args)))


def uzip_linear(args: LinearArgs, d_workspace: int | None, workspace_bytes: int, d_status: int | None, stream: int) -> int:
    return int(_lib.uzip_linear(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


def uzip_grouped_linear_workspace_size(args: LinearArgs) -> int:
    return int(_lib.uzip_grouped_linear_workspace_size(ctypes.byref(args)))


def uzip_grouped_linear(args: LinearArgs, d_workspace: int | None, workspace_bytes: int, d_status: int | None,
                        stream: int) -> int:
    return int(_lib.uzip_grouped_linear(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


def uzip_linear_backward_workspace_size(args: LinearGradArgs) -> int:
    return int(_lib.uzip_linear_backward_workspace_size(ctypes.byref(args)))


def uzip_linear_backward(args: LinearGradArgs, d_workspace: int | None, workspace_bytes: int, d_status: int | None,
                         stream: int) -> int:
    return int(_lib.uzip_linear_backward(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


def uzip_grouped_linear_backward_workspace_size(args: LinearGradArgs) -> int:
    return int(_lib.uzip_grouped_linear_backward_workspace_size(ctypes.byref(args)))


def uzip_grouped_linear_backward(args: LinearGradArgs, d_workspace: int | None, workspace_bytes: int,
                                 d_status: int | None, stream: int) -> int:
    return int(_lib.uzip_grouped_linear_backward(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


def uzip_cross_entropy_workspace_size(args: CrossEntropyArgs) -> int:
    return int(_lib.uzip_cross_entropy_workspace_size(ctypes.byref(args)))


def uzip_cross_entropy(args: CrossEntropyArgs, d_workspace: int | None, workspace_bytes: int, d_status: int | None,
                       stream: int) -> int:
    return int(_lib.uzip_cross_entropy(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


def uzip_cross_entropy_backward_workspace_size(args: CrossEntropyGradArgs) -> int:
    return int(_lib.uzip_cross_entropy_backward_workspace_size(ctypes.byref(args)))


def uzip_cross_entropy_backward(args: CrossEntropyGradArgs, d_workspace: int | None, workspace_bytes: int,
                                d_status: int | None, stream: int) -> int:
    return int(_lib.uzip_cross_entropy_backward(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))


# ---- torch convenience layer (allocation and streams only) ----------------

def _refuse(what: str):
    raise UzipError(UZIP_ERR_INVALID_ARG, what)


@functools.cache
def _dtypes():
    import torch

    return {torch.bfloat16: UZIP_BF16, torch.float16: UZIP_FP16}


def _dtype_code(t) -> int:
    code = _dtypes().get(t.dtype)
    if code is not None:
        return code
    raise UzipError(UZIP_ERR_UNSUPPORTED_DTYPE, f"dtype {t.dtype}")


def _outside_autograd(t, name):
    import torch

    if torch.is_grad_enabled():
        _refuse(f"{name} requires gradients, which autograd would not get from here: detach it, or call under torch.no_grad()")


@functools.cache
def _forward_ad():
    import torch.autograd.forward_ad

    return torch.autograd.forward_ad


def _dual_level() -> int:
    """Below 0 outside of forward-mode differentiation, where no tensor has a
    tangent (0 where torch does not say: then each is asked)."""
    return getattr(_forward_ad(), "_current_level", 0)


def _no_tangents(**tensors):
    """Refuses dual tensors, which do not show in requires_grad."""
    for name, t in tensors.items():
        if t is not None and t.is_floating_point() and _forward_ad().unpack_dual(t).tangent is not None:
            _refuse(f"{name} has a tangent, which forward-mode differentiation would not get from here: take its primal")


def _matrix(t, name, shape, like):
    """Data pointer and row stride of a CUDA matrix (or batch of matrices)
    whose rows are contiguous."""
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t is not like and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        _refuse(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
    if t.requires_grad:
        _outside_autograd(t, name)
    *_, ld, step = t.stride()
    rows, cols = shape[-2], shape[-1]
    if step != 1 and cols > 1:
        _refuse(f"{name}: the last dimension must be contiguous")
    if ld < cols and rows > 1:
        _refuse(f"{name}: rows overlap")
    return t.data_ptr() or None, ld


def _vector(t, name, shape, dtype, like):
    if t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device() or not t.is_contiguous():
        _refuse(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {like.device}")
    if t.requires_grad:
        _outside_autograd(t, name)
    return t.data_ptr() or None


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        _refuse(f"activation {name!r} is not one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def _operand(t, name, dims):
    if not t.is_cuda or t.dim() != dims:
        _refuse(f"{name}: expected a CUDA tensor of {dims} dimensions")
    return t


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device, and `stream` as the current one: outputs and
    workspace then belong to it."""
    import torch

    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_AS_IS = contextlib.nullcontext()


def _here(device, stream):
    import torch

    if stream is None and device.index == torch._C._cuda_getDevice():
        return _AS_IS
    return _on(device, stream)


def _extras(workspace, status, index):
    """What a call writes beside its outputs lies where it runs.  (Host memory
    is the C entry point's to judge: what is mapped for the device will do.)"""
    if workspace is not None:
        if not workspace.is_contiguous():
            _refuse("workspace: the values between those of a strided tensor are not its own")
        if index != workspace.get_device() >= 0:
            _refuse(f"workspace is on {workspace.device}, the call runs on cuda:{index}")
    if status is not None:
        import torch

        if status.dtype != torch.int32 or not status.numel():
            _refuse(f"status: expected an int32 tensor, not {status.dtype} of {status.numel()} values")
        if index != status.get_device() >= 0:
            _refuse(f"status is on {status.device}, the call runs on cuda:{index}")


def _run(name, args, device, workspace, status, check):
    """Runs one entry point on the current stream."""
    import torch

    size, call = _calls[name]
    ref = _byref(args)
    need = size(ref)
    if workspace is not None or status is not None:
        _extras(workspace, status, device.index)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if status is None and check:
        status = torch.empty((), dtype=torch.int32, device=device)
    _check(call(ref, workspace.data_ptr() if workspace is not None else None,
                workspace.nbytes if workspace is not None else 0, status.data_ptr() if status is not None else None,
                torch._C._cuda_getCurrentRawStream(device.index)), name)
    if check:
        st = int(status.item())
        if st != UZIP_OK:
            raise UzipError(st, name + " (device)")


def _forward(name, x, w, offsets, bias, activation, residual, save_preact, out, workspace, status, check, stream):
    import torch

    _operand(x, "x", 2)
    _operand(w, "w", 3 if offsets is not None else 2)
    if _dual_level() >= 0:
        _no_tangents(x=x, w=w, bias=bias, residual=residual, out=out)
    m, k = x.shape
    n = w.shape[-2]
    groups = 0 if offsets is None else w.shape[0]
    dev = x.device
    a = LinearArgs(_dtype_code(x), _activation(activation), m, n, k, groups)
    a.x, a.ldx = _matrix(x, "x", (m, k), x)
    a.w, a.ldw = _matrix(w, "w", w.shape[:-1] + (k,), x)
    if offsets is not None:
        a.w_group = w.stride(0)
        a.offsets = _vector(offsets, "offsets", (groups + 1,), torch.int64, x)
    if bias is not None:
        a.bias = _vector(bias, "bias", w.shape[:-1], x.dtype, x)
    if residual is not None:
        a.residual, a.ldr = _matrix(residual, "residual", (m, n), x)
    with _here(dev, stream):
        if out is None:
            y = torch.empty((m, n), dtype=x.dtype, device=dev)
            a.y, a.ldy = y.data_ptr() or None, n
        else:
            y = out
            a.y, a.ldy = _matrix(y, "out", (m, n), x)
        z = None
        if save_preact:  # rows on 16-byte boundaries, whatever n: the gradient reads them again
            wide = -(-n // 8) * 8
            z = torch.empty_strided((m, n), (wide, 1), dtype=x.dtype, device=dev)
            a.z, a.ldz = z.data_ptr() or None, wide
        _run(name, a, dev, workspace, status, check)
    return (y, z) if save_preact else y


def _backward(name, dy, x, w, offsets, preact, activation, need_dx, need_dw, need_db, workspace, status, check, stream):
    import torch

    _operand(x, "x", 2)
    _operand(w, "w", 3 if offsets is not None else 2)
    if _dual_level() >= 0:
        _no_tangents(dy=dy, x=x, w=w, preact=preact)
    m, k = x.shape
    n = w.shape[-2]
    groups = 0 if offsets is None else w.shape[0]
    dev = x.device
    a = LinearGradArgs(_dtype_code(x), _activation(activation), m, n, k, groups)
    a.dy, a.lddy = _matrix(dy, "dy", (m, n), x)
    a.x, a.ldx = _matrix(x, "x", (m, k), x)
    a.w, a.ldw = _matrix(w, "w", w.shape[:-1] + (k,), x)
    if offsets is not None:
        a.w_group = w.stride(0)
        a.offsets = _vector(offsets, "offsets", (groups + 1,), torch.int64, x)
    if a.act != UZIP_ACT_NONE:
        if preact is None:
            _refuse(f"activation {activation!r} needs the values before it (save_preact in the forward call)")
        a.z, a.ldz = _matrix(preact, "preact", (m, n), x)
    with _here(dev, stream):
        dx = torch.empty((m, k), dtype=x.dtype, device=dev) if need_dx else None
        dw = torch.empty(w.shape, dtype=x.dtype, device=dev) if need_dw else None
        db = torch.empty(w.shape[:-1], dtype=x.dtype, device=dev) if need_db else None
        if dx is not None:
            a.dx, a.lddx = dx.data_ptr() or None, k
        if dw is not None:
            a.dw, a.lddw, a.dw_group = dw.data_ptr() or None, k, n * k
        if db is not None:
            a.db = db.data_ptr() or None
        _run(name, a, dev, workspace, status, check)
    return dx, dw, db


def linear(x, w, bias=None, *, activation="none", residual=None, save_preact=False, out=None, workspace=None,
           status=None, check=False, stream=None):
    """y = act(x @ w.T + bias) + residual for x [m, k] and w [n, k].

    activation is "none", "relu", "gelu" (error function) or "silu".  With
    save_preact the result is (y, z), z = x @ w.T + bias, which
    linear_backward needs (with padded rows where n is no multiple of 8).  Matrices may have any row stride; the last
    dimension must be contiguous.  Outputs and workspace are allocated on
    `stream` (default: the current one) where they are not given; `status` is
    a 0-dim int32 CUDA tensor, and check=True reads it back (one sync) and
    raises UzipError.
    """
    return _forward("uzip_linear", x, w, None, bias, activation, residual, save_preact, out, workspace, status, check,
                    stream)


def linear_backward(dy, x, w, preact=None, *, activation="none", need_dx=True, need_dw=True, need_db=True,
                    workspace=None, status=None, check=False, stream=None):
    """(dx, dw, db) of linear() for the gradient dy of its result; None for
    those not needed.  The residual's gradient is dy."""
    return _backward("uzip_linear_backward", dy, x, w, None, preact, activation, need_dx, need_dw, need_db, workspace,
                     status, check, stream)


def grouped_linear(x, w, offsets, bias=None, *, activation="none", save_preact=False, out=None, workspace=None,
                   status=None, check=False, stream=None):
    """linear() with the rows of x cut by expert: rows offsets[e] to
    offsets[e + 1] use w[e] (w is [experts, n, k]) and bias[e].  offsets is an
    int64 CUDA tensor of experts + 1 values from 0 to m that never decrease;
    others fill the result with NaN and are reported in `status`."""
    if offsets is None:
        _refuse("grouped_linear needs offsets")
    return _forward("uzip_grouped_linear", x, w, offsets, bias, activation, None, save_preact, out, workspace, status,
                    check, stream)


def grouped_linear_backward(dy, x, w, offsets, preact=None, *, activation="none", need_dx=True, need_dw=True,
                            need_db=True, workspace=None, status=None, check=False, stream=None):
    """(dx, dw, db) of grouped_linear(); dw and db of an expert without rows
    are zero."""
    if offsets is None:
        _refuse("grouped_linear_backward needs offsets")
    return _backward("uzip_grouped_linear_backward", dy, x, w, offsets, preact, activation, need_dx, need_dw, need_db,
                     workspace, status, check, stream)


def cross_entropy(h, w, targets, *, ignore_index=-100, workspace=None, status=None, check=False, stream=None):
    """(loss, lse) of each token: loss = logsumexp(h @ w.T) - (h @ w.T)[target]
    in fp32 for h [t, d], w [v, d] and int64 targets [t].  The logits are never
    stored.  Tokens whose target is ignore_index give 0 and 0; a target
    outside [0, v) gives NaN and is reported in `status`.  lse is what
    cross_entropy_backward needs."""
    import torch

    _operand(h, "h", 2)
    _operand(w, "w", 2)
    if _dual_level() >= 0:
        _no_tangents(h=h, w=w)
    (t, d), v = h.shape, w.shape[0]
    dev = h.device
    a = CrossEntropyArgs(dtype=_dtype_code(h), t=t, v=v, d=d, ignore_index=ignore_index)
    a.h, a.ldh = _matrix(h, "h", (t, d), h)
    a.w, a.ldw = _matrix(w, "w", (v, d), h)
    a.targets = _vector(targets, "targets", (t,), torch.int64, h)
    with _here(dev, stream):
        loss = torch.empty(t, dtype=torch.float32, device=dev)
        lse = torch.empty(t, dtype=torch.float32, device=dev)
        a.loss, a.lse = loss.data_ptr() or None, lse.data_ptr() or None
        _run("uzip_cross_entropy", a, dev, workspace, status, check)
    return loss, lse


def cross_entropy_backward(dloss, h, w, targets, lse, *, ignore_index=-100, need_dh=True, need_dw=True, piece=0,
                           workspace=None, status=None, check=False, stream=None):
    """(dh, dw) of cross_entropy() for the fp32 gradient dloss [t] of each
    token's loss.  The vocabulary is taken `piece` classes at a time (0: as
    many as fit 512 MiB, at most 32768), whose softmax gradient is the only
    workspace of that size."""
    import torch

    _operand(h, "h", 2)
    _operand(w, "w", 2)
    if _dual_level() >= 0:
        _no_tangents(dloss=dloss, h=h, w=w, lse=lse)
    (t, d), v = h.shape, w.shape[0]
    dev = h.device
    a = CrossEntropyGradArgs(dtype=_dtype_code(h), t=t, v=v, d=d, piece=piece, ignore_index=ignore_index)
    a.h, a.ldh = _matrix(h, "h", (t, d), h)
    a.w, a.ldw = _matrix(w, "w", (v, d), h)
    a.targets = _vector(targets, "targets", (t,), torch.int64, h)
    a.lse = _vector(lse, "lse", (t,), torch.float32, h)
    a.dloss = _vector(dloss, "dloss", (t,), torch.float32, h)
    with _here(dev, stream):
        dh = torch.empty((t, d), dtype=h.dtype, device=dev) if need_dh else None
        dw = torch.empty((v, d), dtype=h.dtype, device=dev) if need_dw else None
        if dh is not None:
            a.dh, a.lddh = dh.data_ptr() or None, d
        if dw is not None:
            a.dw, a.lddw = dw.data_ptr() or None, d
        _run("uzip_cross_entropy_backward", a, dev, workspace, status, check)
    return dh, dw
