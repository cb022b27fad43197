"""The paged key-value cache of a language model: rotary positions, storing
keys and values into pages, attention of one new token over them, and the pages
themselves (reserving, forking, freeing, compacting, copying).

Thin ctypes layer over include/uzip_cache.h: the functions named like the C
entry points only marshal arguments, and the torch functions allocate outputs
and workspace and pass the stream.  All arithmetic runs in the library's kernels.

A cache is plain tensors of the caller's: pools k_pages and v_pages of shape
[pages, kv heads, page size, head size] (bf16 or fp16, any strides that are
multiples of 8 with the last dimension contiguous; [layers, pages, ...] for
cache_copy), and its state: refs int32 [pages], table int32 [sequences, width]
and lengths int32 [sequences].  A new cache has zeros in all three.  Like the
other torch functions here these are not known to autograd: rotary_backward is
the gradient of rotary.  Tensors that require gradients are refused while grad
mode is on, and so are tensors with a tangent of forward-mode differentiation.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import _check, library
from .ops import _calls, _dtype_code, _dual_level, _extras, _no_tangents, _on, _outside_autograd, _refuse

_i32, _i64, _u64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_float

UZIP_MAX_HEAD = 256
UZIP_MAX_SEQS = 65536
UZIP_MAX_PAGES = 1572864


def _fields(*names):
    """"x:row:head" is a pointer x and strides x_row, x_head."""
    out = []
    for name in names:
        base, *steps = name.split(":")
        out += [(base, _vp)] + [(s, _i64) for s in steps]
    return out


class RotaryArgs(ctypes.Structure):
    """uzip_rotary_args"""

    _fields_ = [("dtype", _i32), ("interleaved", _i32), ("backward", _i32), ("scale", _f32), ("t", _i64), ("q_heads", _i64),
                ("kv_heads", _i64), ("d", _i64), ("rot", _i64), ("positions", _vp), ("freqs", _vp)] + _fields(
                    "q:q_row:q_head", "k:k_row:k_head", "v:v_row:v_head", "q_out:q_out_row:q_out_head", "k_out:k_out_row:k_out_head") + [
                    ("pages", _i64), ("page", _i64)] + _fields("k_pages:kp_page:kp_head:kp_token", "v_pages:vp_page:vp_head:vp_token", "slots")


class PagedAttentionArgs(ctypes.Structure):
    """uzip_paged_attention_args"""

    _fields_ = [("dtype", _i32), ("reserved", _i32), ("seqs", _i64), ("q_heads", _i64), ("kv_heads", _i64), ("d", _i64), ("pages", _i64),
                ("page", _i64), ("width", _i64)] + _fields("q:q_row:q_head", "k_pages:kp_page:kp_head:kp_token", "v_pages:vp_page:vp_head:vp_token",
                                                           "table:ldt", "lengths") + [
                    ("scale", _f32), ("softcap", _f32), ("window", _i64)] + _fields("out:out_row:out_head", "lse")


class CacheArgs(ctypes.Structure):
    """uzip_cache_args"""

    _fields_ = [("pages", _i64), ("page", _i64), ("seqs", _i64), ("width", _i64), ("refs", _vp), ("table", _vp), ("ldt", _i64), ("lengths", _vp),
                ("n", _i64), ("from_", _vp), ("list", _vp), ("tokens", _i64), ("slots", _vp), ("positions", _vp), ("pairs", _vp)]


class CacheCopyArgs(ctypes.Structure):
    """uzip_cache_copy_args"""

    _fields_ = [("dtype", _i32), ("reserved", _i32), ("layers", _i64), ("heads", _i64), ("page", _i64), ("d", _i64), ("from_pages", _i64),
                ("to_pages", _i64)] + _fields("k:k_layer:k_page:k_head:k_token", "v:v_layer:v_page:v_head:v_token",
                                              "k_to:kt_layer:kt_page:kt_head:kt_token", "v_to:vt_layer:vt_page:vt_head:vt_token", "pairs") + [("n", _i64)]


_lib = library()
for _name, _args in (("uzip_rotary", RotaryArgs), ("uzip_rotary_append", RotaryArgs), ("uzip_paged_attention", PagedAttentionArgs),
                     ("uzip_cache_reserve", CacheArgs), ("uzip_cache_fork", CacheArgs), ("uzip_cache_free", CacheArgs),
                     ("uzip_cache_compact", CacheArgs), ("uzip_cache_copy", CacheCopyArgs)):
    _size, _call = getattr(_lib, _name + "_workspace_size"), getattr(_lib, _name)
    _size.argtypes, _size.restype = [ctypes.POINTER(_args)], _u64
    _call.argtypes, _call.restype = [ctypes.POINTER(_args), _vp, _u64, _vp, _vp], ctypes.c_int
    _calls[_name] = (_size, _call)


# ---- C entry points (same names; `args` is one of the structures above) ----

def _entry(name, args_type):
    size, call = _calls[name]

    def workspace_size(args) -> int:
        return int(size(ctypes.byref(args)))

    def entry(args, d_workspace: int | None, workspace_bytes: int, d_status: int | None, stream: int) -> int:
        return int(call(ctypes.byref(args), d_workspace, workspace_bytes, d_status, stream))

    entry.__name__, workspace_size.__name__ = name, name + "_workspace_size"
    workspace_size.__doc__ = f"Bytes of workspace for a {args_type.__name__}."
    entry.__doc__ = f"{name} of a {args_type.__name__}; returns a uzip_status."
    return entry, workspace_size


uzip_rotary, uzip_rotary_workspace_size = _entry("uzip_rotary", RotaryArgs)
uzip_rotary_append, uzip_rotary_append_workspace_size = _entry("uzip_rotary_append", RotaryArgs)
uzip_paged_attention, uzip_paged_attention_workspace_size = _entry("uzip_paged_attention", PagedAttentionArgs)
uzip_cache_reserve, uzip_cache_reserve_workspace_size = _entry("uzip_cache_reserve", CacheArgs)
uzip_cache_fork, uzip_cache_fork_workspace_size = _entry("uzip_cache_fork", CacheArgs)
uzip_cache_free, uzip_cache_free_workspace_size = _entry("uzip_cache_free", CacheArgs)
uzip_cache_compact, uzip_cache_compact_workspace_size = _entry("uzip_cache_compact", CacheArgs)
uzip_cache_copy, uzip_cache_copy_workspace_size = _entry("uzip_cache_copy", CacheCopyArgs)


# ---- torch convenience layer (allocation and streams only) ----------------
#
# A step of a server makes these calls for every layer, so their host time
# counts: arguments are packed in one go (struct, in the C structure's native
# layout) instead of set one by one, and each tensor is asked for each thing
# once (attention of one token 20 us of host time, 11 so).

class _Entry:
    """A C entry point that takes its structure as packed bytes."""

    def __init__(self, name, args):
        codes = {_i32: "i", _i64: "q", _vp: "P", _f32: "f"}
        self.name = name
        self.pack = struct.Struct("@" + "".join(codes[t] for _, t in args._fields_)).pack
        self.size, self.call = _lib[name + "_workspace_size"], _lib[name]
        self.size.argtypes, self.size.restype = [ctypes.c_char_p], _u64
        self.call.argtypes, self.call.restype = [ctypes.c_char_p, _vp, _u64, _vp, _vp], ctypes.c_int


_ROTARY, _APPEND = _Entry("uzip_rotary", RotaryArgs), _Entry("uzip_rotary_append", RotaryArgs)
_ATTENTION = _Entry("uzip_paged_attention", PagedAttentionArgs)
_RESERVE, _FORK = _Entry("uzip_cache_reserve", CacheArgs), _Entry("uzip_cache_fork", CacheArgs)
_FREE, _COMPACT = _Entry("uzip_cache_free", CacheArgs), _Entry("uzip_cache_compact", CacheArgs)
_COPY = _Entry("uzip_cache_copy", CacheCopyArgs)

_torch = _empty = None


def _load():
    """torch, once it is needed, and _empty(shape, strides, dtype): a tensor on
    the current device.  torch's allocation without its dispatcher takes 3 us
    less of 5 between other calls; it is torch's own, so where a version has it
    no more, or it does not do this, empty_strided does."""
    global _torch, _empty
    import torch

    direct = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
    _empty = direct if direct is not None and _allocates(direct, torch) else (
        lambda shape, steps, dtype: torch.empty_strided(shape, steps, dtype=dtype, device="cuda"))
    _torch = torch
    return torch


def _allocates(f, torch):
    """Whether f(shape, strides, dtype) gives such a tensor on the current device."""
    try:
        dev = torch.cuda.current_device()  # (CUDA is set up from here on)
        t = f((2, 3), (4, 1), torch.int16)
        return (type(t) is torch.Tensor and t.shape == (2, 3) and t.stride() == (4, 1) and t.dtype is torch.int16 and t.get_device() == dev
                and not t.requires_grad)
    except Exception:  # noqa: BLE001  (whatever it takes now, it is not this)
        return False


def _issue(entry, args, dev, workspace, status, check):
    """Runs an entry point on the current stream of device `dev`, the current one."""
    torch = _torch
    if workspace is not None or status is not None:
        _extras(workspace, status, dev)
    if workspace is None:
        need = entry.size(args)
        at = 0
        if need:
            workspace = _empty((need,), (1,), torch.uint8)
            at = workspace.data_ptr()
    else:
        need, at = workspace.nbytes, workspace.data_ptr()
    if status is None and check:
        status = torch.empty((), dtype=torch.int32, device=dev)
    st = entry.call(args, at, need, status.data_ptr() if status is not None else None, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st, entry.name)
    if check:
        _check(int(status.item()), entry.name + " (device)")


def _elsewhere(dev, stream):
    """Whether `stream` or the tensors' device is another than the current one."""
    return stream is not None or dev != _torch._C._cuda_getDevice()


def _device(t, name, dims):
    """The index of the device of a tensor of `dims` dimensions."""
    dev = t.get_device()
    if dev < 0 or t.dim() != dims:
        _refuse(f"{name}: expected a CUDA tensor of {dims} dimensions")
    return dev


def _strides(t, name, shape, dtype, dev):
    """The strides of a tensor whose last dimension is contiguous."""
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(f"{name} is {t.dtype} on {t.device}, expected {dtype} on cuda:{dev}")
    if t.requires_grad:
        _outside_autograd(t, name)
    steps = t.stride()
    if steps[-1] != 1 and shape[-1] > 1:
        _refuse(f"{name}: the last dimension must be contiguous")
    return steps


def _list(t, name, shape, dtype, dev):
    """The address of a contiguous tensor."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    if t.requires_grad:
        _outside_autograd(t, name)
    return t.data_ptr()


def rotary_frequencies(dim, *, base=10000.0, scaling="none", factor=1.0, trained=0, fast=32.0, slow=1.0, device="cuda"):
    """Rotary frequencies of the first `dim` (even) values of a head, for
    rotary() and rotary_append(): a float64 tensor of dim / 2 radians per
    position (finite), f_j = base^(-2 j / dim), stretched for contexts `factor`
    times as long as trained:

    "none"    as they are
    "linear"  f_j / factor
    "ntk"     those of base factor^(dim / (dim - 2)): the fastest stays, the slowest is divided by factor
    "yarn"    f_j (1 - r_j) + f_j / factor r_j with r_j rising from 0 at j = floor(i(fast)) to 1 at j = ceil(i(slow)), where
              i(n) = dim log(trained / (2 pi n)) / (2 log base) is the index whose wave turns n times over the trained positions
    "bands"   the same with r_j falling from 1 to 0 linearly in the number of turns, from `slow` of them to `fast`

    "yarn" goes with an amplitude for rotary()'s scale, usually 0.1 ln(factor) + 1.
    """
    import torch

    if dim < 0 or dim % 2:
        _refuse(f"dim {dim} is not an even number of values")
    if scaling not in ("none", "linear", "ntk", "yarn", "bands"):
        _refuse(f"scaling {scaling!r} is not one of none, linear, ntk, yarn, bands")
    if not (base > 0 and factor > 0):
        _refuse("base and factor must be positive")
    if scaling == "ntk" and dim > 2:
        base *= factor ** (dim / (dim - 2))
    freqs = [base ** (-2.0 * j / dim) for j in range(dim // 2)]
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling in ("yarn", "bands") and dim:
        if trained < 1 or not fast > slow > 0:
            _refuse(f"scaling {scaling!r} needs the trained length, and fast > slow > 0")
        if scaling == "yarn":
            if base <= 1:
                _refuse("scaling 'yarn' needs a base over 1")
            index = lambda turns: dim * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(0, math.floor(index(fast))), min(dim - 1, math.ceil(index(slow)))
            hi = hi if hi != lo else lo + 0.001
            keep = [1 - min(1.0, max(0.0, (j - lo) / (hi - lo))) for j in range(dim // 2)]
        else:
            turns = [trained * f / (2 * math.pi) for f in freqs]
            keep = [min(1.0, max(0.0, (t - slow) / (fast - slow))) for t in turns]
        freqs = [f * (k + (1 - k) / factor) for f, k in zip(freqs, keep)]
    return torch.tensor(freqs, dtype=torch.float64, device=device)


def _rotary(q, k, positions, freqs, interleaved, backward, scale, out, status, check, stream):
    torch = _torch or _load()
    like = q if q is not None else k
    if like is None:
        _refuse("neither q nor k is given")
    dev = _device(like, "q" if q is not None else "k", 3)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _rotary(q, k, positions, freqs, interleaved, backward, scale, out, status, check, None)
    if _dual_level() >= 0:
        _no_tangents(q=q, k=k, freqs=freqs, **dict(zip(("out", "out's second"), out or ())))
    dt, code = like.dtype, _dtype_code(like)
    t, hq, d = like.shape
    hk = 0
    if q is None:
        hq = 0
    if k is not None:
        _device(k, "k", 3)
        hk = k.shape[1]
    pairs = freqs.numel()
    at = _list(positions, "positions", (t,), torch.int64, dev), _list(freqs, "freqs", (pairs,), torch.float64, dev)
    q_out, k_out = out if out is not None else (None, None)
    part = []
    for x, y, h, name in ((q, q_out, hq, "q"), (k, k_out, hk, "k")):
        if x is None:
            part.append((None, (0, 0, 0, 0, 0, 0)))
            continue
        shape = (t, h, d)
        row, head, _ = _strides(x, name, shape, dt, dev)
        if y is None:
            steps = h * d, d, 1
            y = _empty(shape, steps, dt)
        else:
            steps = _strides(y, "out", shape, dt, dev)
        part.append((y, (x.data_ptr(), row, head, y.data_ptr(), steps[0], steps[1])))
    (q_out, a), (k_out, b) = part
    _issue(_ROTARY, _ROTARY.pack(code, 1 if interleaved else 0, backward, scale, t, hq, hk, d, 2 * pairs, *at, *a[:3], *b[:3], 0, 0, 0, *a[3:], *b[3:],
                                 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), dev, None, status, check)
    return q_out, k_out


def rotary(q, k, positions, freqs, *, interleaved=False, scale=1.0, out=None, status=None, check=False, stream=None):
    """(q', k'): the first 2 len(freqs) values of each head of q [t, q heads, d]
    and k [t, kv heads, d] rotated in pairs by positions[i] * freqs[j] and
    multiplied by `scale`, the others copied.  Pairs are (j, j + n) of n pairs,
    or neighbours where `interleaved`.  positions is int64 [t], freqs float64 of
    radians per position (rotary_frequencies); far positions lose nothing.
    Either of q and k may be None.  out: (q', k') to write to, which may be q
    and k themselves."""
    return _rotary(q, k, positions, freqs, interleaved, 0, scale, out, status, check, stream)


def rotary_backward(dq, dk, positions, freqs, *, interleaved=False, scale=1.0, out=None, status=None, check=False, stream=None):
    """(dq', dk'): the gradients of rotary()'s q and k for those of its results:
    the rotation by the opposite angles."""
    return _rotary(dq, dk, positions, freqs, interleaved, 1, scale, out, status, check, stream)


def rotary_append(q, k, v, positions, freqs, k_pages, v_pages, slots, *, interleaved=False, scale=1.0, out=None, status=None, check=False,
                  stream=None):
    """rotary() of q, returned, and of k, which is stored with v into the pages:
    token i at page slots[i] // page size, place slots[i] % page size.  slots is
    int64 [t] (cache_reserve gives them), no two equal; -1 stores nothing, others
    outside the pool store nothing and are reported in `status`."""
    torch = _torch or _load()
    if q is None or k is None or v is None:
        _refuse("rotary_append needs q, k and v")
    dev = _device(q, "q", 3)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rotary_append(q, k, v, positions, freqs, k_pages, v_pages, slots, interleaved=interleaved, scale=scale, out=out, status=status,
                                 check=check)
    if _dual_level() >= 0:
        _no_tangents(q=q, k=k, v=v, freqs=freqs, k_pages=k_pages, v_pages=v_pages, out=out)
    _device(k, "k", 3)
    dt, code = q.dtype, _dtype_code(q)
    t, hq, d = shape = q.shape
    hk = k.shape[1]
    q_row, q_head, _ = _strides(q, "q", shape, dt, dev)
    k_row, k_head, _ = _strides(k, "k", (t, hk, d), dt, dev)
    v_row, v_head, _ = _strides(v, "v", (t, hk, d), dt, dev)
    _device(k_pages, "k_pages", 4)
    pages, heads, page, wide = pool = k_pages.shape
    if heads != hk or wide != d:
        _refuse(f"k_pages has {heads} heads of {wide} values, k has {hk} of {d}")
    kp, vp = _strides(k_pages, "k_pages", pool, dt, dev), _strides(v_pages, "v_pages", pool, dt, dev)
    pairs = freqs.numel()
    if out is None:
        o_row, o_head = hq * d, d
        out = _empty((t, hq, d), (o_row, o_head, 1), dt)
    else:
        o_row, o_head, _ = _strides(out, "out", shape, dt, dev)
    args = _APPEND.pack(code, 1 if interleaved else 0, 0, scale, t, hq, hk, d, 2 * pairs, _list(positions, "positions", (t,), torch.int64, dev),
                        _list(freqs, "freqs", (pairs,), torch.float64, dev), q.data_ptr(), q_row, q_head, k.data_ptr(), k_row, k_head, v.data_ptr(),
                        v_row, v_head, out.data_ptr(), o_row, o_head, 0, 0, 0, pages, page, k_pages.data_ptr(), kp[0], kp[1], kp[2],
                        v_pages.data_ptr(), vp[0], vp[1], vp[2], _list(slots, "slots", (t,), torch.int64, dev))
    _issue(_APPEND, args, dev, None, status, check)
    return out


def paged_attention(q, k_pages, v_pages, table, lengths, *, scale=None, softcap=0.0, window=0, with_lse=False, out=None, workspace=None,
                    status=None, check=False, stream=None):
    """Attention of one new token of each sequence, q [sequences, q heads, d],
    over its keys and values in the pages: softmax(scale q k) v over the last
    `window` of lengths[i] tokens (0: all; the new one counts).  q heads are a
    multiple of the kv heads, which they share in order.  scale is 1 / sqrt(d)
    where not given; softcap c > 0 makes a score s c tanh(s / c).  A sequence of
    length 0 gives zeros.  With with_lse the result is (out, lse), lse the fp32
    log-sum-exp of each head's scores, by which results over parts of a context
    are joined.  A length or page that cannot be gives NaN for its sequence and
    is reported in `status`."""
    torch = _torch or _load()
    dev = _device(q, "q", 3)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return paged_attention(q, k_pages, v_pages, table, lengths, scale=scale, softcap=softcap, window=window, with_lse=with_lse, out=out,
                                   workspace=workspace, status=status, check=check)
    if _dual_level() >= 0:
        _no_tangents(q=q, k_pages=k_pages, v_pages=v_pages, out=out)
    dt, code = q.dtype, _dtype_code(q)
    s, hq, d = shape = q.shape
    q_row, q_head, _ = _strides(q, "q", shape, dt, dev)
    _device(k_pages, "k_pages", 4)
    pages, hk, page, wide = pool = k_pages.shape
    if wide != d:
        _refuse(f"q has heads of {d} values, k_pages of {wide}")
    kp, vp = _strides(k_pages, "k_pages", pool, dt, dev), _strides(v_pages, "v_pages", pool, dt, dev)
    ldt, width = _table(table, dev)
    if table.shape[0] != s:
        _refuse(f"table has {table.shape[0]} rows for {s} queries")
    if out is None:
        o_row, o_head = hq * d, d
        out = _empty((s, hq, d), (o_row, o_head, 1), dt)
    else:
        o_row, o_head, _ = _strides(out, "out", shape, dt, dev)
    lse = _empty((s, hq), (hq, 1), torch.float32) if with_lse else None
    if scale is None:
        scale = d ** -0.5 if d else 0.0
    args = _ATTENTION.pack(code, 0, s, hq, hk, d, pages, page, width, q.data_ptr(), q_row, q_head, k_pages.data_ptr(), kp[0], kp[1], kp[2],
                           v_pages.data_ptr(), vp[0], vp[1], vp[2], table.data_ptr(), ldt, _list(lengths, "lengths", (s,), torch.int32, dev), scale,
                           softcap, window, out.data_ptr(), o_row, o_head, lse.data_ptr() if with_lse else 0)
    _issue(_ATTENTION, args, dev, workspace, status, check)
    return (out, lse) if with_lse else out


def _table(table, dev):
    """Row stride and columns of a table."""
    ldt, step = table.stride() if table.dim() == 2 else (0, 0)
    width = table.shape[-1] if table.dim() == 2 else 0
    if table.dim() != 2 or table.dtype is not _torch.int32 or table.get_device() != dev or (step != 1 and width > 1):
        _refuse(f"table: expected int32 [sequences, pages of a sequence] on cuda:{dev}, its rows contiguous")
    return ldt, width


def _change(entry, state, page_size, workspace, status, check, n=0, start=0, listed=0, tokens=0, slots=0, positions=0, pairs=0):
    """An operation on a cache's state: refs, table, lengths, what _state() gave of them."""
    refs, table, lengths, (pages, seqs, width, ldt, dev) = state
    args = entry.pack(pages, page_size, seqs, width, refs.data_ptr(), table.data_ptr(), ldt, lengths.data_ptr(), n, start, listed, tokens, slots,
                      positions, pairs)
    _issue(entry, args, dev, workspace, status, check)


def _state(refs, table, lengths):
    torch = _torch or _load()
    dev = _device(table, "table", 2)
    ldt, width = _table(table, dev)
    pages, seqs = refs.numel(), table.shape[0]
    _list(refs, "refs", (pages,), torch.int32, dev)
    _list(lengths, "lengths", (seqs,), torch.int32, dev)
    return refs, table, lengths, (pages, seqs, width, ldt, dev)


def cache_reserve(refs, table, lengths, counts, tokens, page_size, *, out=None, workspace=None, status=None, check=False, stream=None):
    """Pages and slots for counts[i] (int32) new tokens of each sequence, at
    most `tokens` in all: (slots, positions, copies).  slots and positions are
    int64 [tokens], in the order of the sequences, -1 and 0 behind the last
    (for rotary_append).  The lowest free pages are taken.  A sequence whose
    part-full last page is shared gets a page in its place: copies int32
    [sequences, 2] holds {old, new} for cache_copy, {-1, -1} elsewhere.  refs,
    table and lengths are updated.  Where pages or columns of the table run out
    nothing changes, slots are -1, and `status` says so."""
    state = _state(refs, table, lengths)
    seqs, dev, torch = state[3][1], state[3][4], _torch
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_reserve(refs, table, lengths, counts, tokens, page_size, out=out, workspace=workspace, status=status, check=check)
    if tokens < 0:
        _refuse(f"{tokens} tokens")
    listed = _list(counts, "counts", (seqs,), torch.int32, dev)
    if out is None:
        out = _empty((tokens,), (1,), torch.int64), _empty((tokens,), (1,), torch.int64), _empty((seqs, 2), (2, 1), torch.int32)
        slots, positions, pairs = out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr()
    else:
        slots, positions = (_list(x, "out", (tokens,), torch.int64, dev) for x in out[:2])
        pairs = _list(out[2], "out", (seqs, 2), torch.int32, dev)
    _change(_RESERVE, state, page_size, workspace, status, check, listed=listed, tokens=tokens, slots=slots, positions=positions, pairs=pairs)
    return out


def cache_fork(refs, table, lengths, parents, children, page_size, *, workspace=None, status=None, check=False, stream=None):
    """children[j] become sequences that share the pages of parents[j] (int32
    indexes, -1 in both: none).  A child must be empty, listed once and nobody's
    parent; else nothing changes, and `status` says so."""
    state = _state(refs, table, lengths)
    dev, torch = state[3][4], _torch
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_fork(refs, table, lengths, parents, children, page_size, workspace=workspace, status=status, check=check)
    n = children.numel()
    _change(_FORK, state, page_size, workspace, status, check, n, _list(parents, "parents", (n,), torch.int32, dev),
            _list(children, "children", (n,), torch.int32, dev))


def cache_free(refs, table, lengths, sequences, page_size, *, workspace=None, status=None, check=False, stream=None):
    """The sequences listed (int32 indexes, each once, -1: none) become empty;
    pages that nobody shares are free.  Where an index is wrong nothing changes,
    and `status` says so."""
    state = _state(refs, table, lengths)
    dev, torch = state[3][4], _torch
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_free(refs, table, lengths, sequences, page_size, workspace=workspace, status=status, check=check)
    n = sequences.numel()
    _change(_FREE, state, page_size, workspace, status, check, n, 0, _list(sequences, "sequences", (n,), torch.int32, dev))


def cache_compact(refs, table, lengths, page_size, *, out=None, workspace=None, status=None, check=False, stream=None):
    """Moves the used pages to the front of the pool: updates refs and table and
    returns moves, int32 [pages // 2, 2] of {from, to} for cache_copy, -1 behind
    the last."""
    state = _state(refs, table, lengths)
    pages, dev, torch = state[3][0], state[3][4], _torch
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_compact(refs, table, lengths, page_size, out=out, workspace=workspace, status=status, check=check)
    if out is None:
        out = _empty((pages // 2, 2), (2, 1), torch.int32)
    _change(_COMPACT, state, page_size, workspace, status, check, pairs=_list(out, "out", (pages // 2, 2), torch.int32, dev))
    return out


def cache_copy(k_pages, v_pages, pairs, *, to=None, status=None, check=False, stream=None):
    """Copies page pairs[j, 0] to page pairs[j, 1] (int32, -1: none) in keys and
    values, for pools [pages, heads, page size, d] or [layers, pages, ...].  `to`
    is another cache's (k_pages, v_pages), such as a buffer that is compressed
    and sent; the same cache where not given.  Where a page does not exist, is
    written twice or (within a cache) also read, nothing is copied, and `status`
    says so."""
    torch = _torch or _load()
    layered = k_pages.dim() == 5
    dev = _device(k_pages, "k_pages", 5 if layered else 4)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_copy(k_pages, v_pages, pairs, to=to, status=status, check=check)
    if _dual_level() >= 0:
        _no_tangents(k_pages=k_pages, v_pages=v_pages, **dict(zip(("to", "to's second"), to or ())))
    dt, code = k_pages.dtype, _dtype_code(k_pages)
    shape = k_pages.shape
    layers, (pages, heads, page, d) = (shape[0], shape[1:]) if layered else (1, shape)

    def place(t, name, shape):  # address, and strides of layers, pages, heads, tokens
        steps = _strides(t, name, shape, dt, dev)
        return (t.data_ptr(), *steps[:4]) if layered else (t.data_ptr(), 0, *steps[:3])

    k, v = place(k_pages, "k_pages", shape), place(v_pages, "v_pages", shape)
    k_to, v_to, to_pages = k, v, pages
    if to is not None:
        _device(to[0], "to", len(shape))
        to_pages = to[0].shape[-4]
        into = (layers, to_pages, heads, page, d) if layered else (to_pages, heads, page, d)
        k_to, v_to = place(to[0], "to", into), place(to[1], "to", into)
    n = pairs.numel() // 2
    _issue(_COPY, _COPY.pack(code, 0, layers, heads, page, d, pages, to_pages, *k, *v, *k_to, *v_to, _list(pairs, "pairs", (n, 2), torch.int32, dev), n),
           dev, None, status, check)
