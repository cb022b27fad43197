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
the gradient of rotary, and tensors that require gradients are refused while
grad mode is on.
"""
from __future__ import annotations

import ctypes
import math

from . import library
from .ops import _calls, _dtype_code, _here, _operand, _outside_autograd, _refuse, _run, _vector

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

def _strided(t, name, shape, like):
    """Data pointer and the strides of all dimensions but the last, which is
    contiguous."""
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t is not like and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        _refuse(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
    if t.requires_grad:
        _outside_autograd(t, name)
    *steps, last = t.stride()
    if last != 1 and shape[-1] > 1:
        _refuse(f"{name}: the last dimension must be contiguous")
    return (t.data_ptr() or None, *steps)


def _pools(k_pages, v_pages, dims, like):
    _operand(k_pages, "k_pages", dims)
    if like is None:
        like = k_pages
    k = _strided(k_pages, "k_pages", k_pages.shape, like)
    return k, _strided(v_pages, "v_pages", k_pages.shape, like)


def rotary_frequencies(dim, *, base=10000.0, scaling="none", factor=1.0, trained=0, fast=32.0, slow=1.0, device="cuda"):
    """Rotary frequencies of the first `dim` (even) values of a head, for
    rotary() and rotary_append(): a float64 tensor of dim / 2 radians per
    position, f_j = base^(-2 j / dim), stretched for contexts `factor` times as
    long as trained:

    "none"    as they are
    "linear"  f_j / factor
    "ntk"     those of base factor^(dim / (dim - 2)): the fastest stays, the slowest is divided by factor
    "yarn"    f_j / factor where a wave turns at most `slow` times over the `trained` positions, f_j where it turns at
              least `fast` times, and between the two by a ramp linear in the index j, from the largest index whose wave
              turns `fast` times down to the smallest whose wave turns `slow` times (rounded outward)
    "bands"   the same with a ramp linear in the number of turns

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


def _rotary(name, q, k, v, positions, freqs, interleaved, backward, scale, out, pools, slots, workspace, status, check, stream):
    import torch

    like = q if q is not None else k
    if like is None:
        _refuse("neither q nor k is given")
    _operand(like, "q" if q is not None else "k", 3)
    t, _, d = like.shape
    hq = q.shape[1] if q is not None else 0
    if k is not None:
        _operand(k, "k", 3)
    hkv = k.shape[1] if k is not None else 0
    _operand(freqs, "freqs", 1)
    dev = like.device
    a = RotaryArgs(_dtype_code(like), bool(interleaved), backward, scale, t, hq, hkv, d, 2 * freqs.shape[0])
    a.positions = _vector(positions, "positions", (t,), torch.int64, like)
    a.freqs = _vector(freqs, "freqs", freqs.shape, torch.float64, like)
    if q is not None:
        a.q, a.q_row, a.q_head = _strided(q, "q", (t, hq, d), like)
    if k is not None:
        a.k, a.k_row, a.k_head = _strided(k, "k", (t, hkv, d), like)
    if v is not None:
        a.v, a.v_row, a.v_head = _strided(v, "v", (t, hkv, d), like)
        (a.k_pages, a.kp_page, a.kp_head, a.kp_token), (a.v_pages, a.vp_page, a.vp_head, a.vp_token) = _pools(*pools, 4, like)
        a.pages, heads, a.page, width = pools[0].shape
        if heads != hkv or width != d:
            _refuse(f"k_pages has {heads} heads of {width} values, k has {hkv} of {d}")
        a.slots = _vector(slots, "slots", (t,), torch.int64, like)
    q_out = k_out = None
    with _here(dev, stream):
        if out is not None:
            q_out, k_out = out if v is None else (out, None)
        if q is not None:
            if q_out is None:
                q_out = torch.empty((t, hq, d), dtype=like.dtype, device=dev)
            a.q_out, a.q_out_row, a.q_out_head = _strided(q_out, "out", (t, hq, d), like)
        if k is not None and v is None:
            if k_out is None:
                k_out = torch.empty((t, hkv, d), dtype=like.dtype, device=dev)
            a.k_out, a.k_out_row, a.k_out_head = _strided(k_out, "out", (t, hkv, d), like)
        _run(name, a, dev, workspace, status, check)
    return (q_out, k_out) if v is None else q_out


def rotary(q, k, positions, freqs, *, interleaved=False, scale=1.0, out=None, status=None, check=False, stream=None):
    """(q', k'): the first 2 len(freqs) values of each head of q [t, q heads, d]
    and k [t, kv heads, d] rotated in pairs by positions[i] * freqs[j] and
    multiplied by `scale`, the others copied.  Pairs are (j, j + n) of n pairs,
    or neighbours where `interleaved`.  positions is int64 [t], freqs float64 of
    radians per position (rotary_frequencies); far positions lose nothing.
    Either of q and k may be None.  out: (q', k') to write to, which may be q
    and k themselves."""
    return _rotary("uzip_rotary", q, k, None, positions, freqs, interleaved, 0, scale, out, None, None, None, status, check, stream)


def rotary_backward(dq, dk, positions, freqs, *, interleaved=False, scale=1.0, out=None, status=None, check=False, stream=None):
    """(dq', dk'): the gradients of rotary()'s q and k for those of its results:
    the rotation by the opposite angles."""
    return _rotary("uzip_rotary", dq, dk, None, positions, freqs, interleaved, 1, scale, out, None, None, None, status, check, stream)


def rotary_append(q, k, v, positions, freqs, k_pages, v_pages, slots, *, interleaved=False, scale=1.0, out=None, status=None, check=False,
                  stream=None):
    """rotary() of q, returned, and of k, which is stored with v into the pages:
    token i at page slots[i] // page size, place slots[i] % page size.  slots is
    int64 [t] (cache_reserve gives them), no two equal; -1 stores nothing, others
    outside the pool store nothing and are reported in `status`."""
    if q is None or k is None or v is None:
        _refuse("rotary_append needs q, k and v")
    return _rotary("uzip_rotary_append", q, k, v, positions, freqs, interleaved, 0, scale, out, (k_pages, v_pages), slots, None, status, check,
                   stream)


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
    import torch

    _operand(q, "q", 3)
    k, v = _pools(k_pages, v_pages, 4, q)
    s, hq, d = q.shape
    pages, hkv, page, width = k_pages.shape
    if width != d:
        _refuse(f"q has heads of {d} values, k_pages of {width}")
    dev = q.device
    if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != s or table.get_device() != q.get_device() or (
            table.shape[1] > 1 and table.stride(1) != 1):
        _refuse(f"table: expected int32 of shape ({s}, pages of a sequence) on {dev}, its rows contiguous")
    a = PagedAttentionArgs(_dtype_code(q), 0, s, hq, hkv, d, pages, page, table.shape[1])
    a.q, a.q_row, a.q_head = _strided(q, "q", q.shape, q)
    a.k_pages, a.kp_page, a.kp_head, a.kp_token = k
    a.v_pages, a.vp_page, a.vp_head, a.vp_token = v
    a.table, a.ldt = table.data_ptr() or None, table.stride(0)
    a.lengths = _vector(lengths, "lengths", (s,), torch.int32, q)
    a.scale, a.softcap, a.window = 1 / math.sqrt(d) if scale is None and d else scale or 0.0, softcap, window
    with _here(dev, stream):
        if out is None:
            out = torch.empty((s, hq, d), dtype=q.dtype, device=dev)
        a.out, a.out_row, a.out_head = _strided(out, "out", q.shape, q)
        lse = None
        if with_lse:
            lse = torch.empty((s, hq), dtype=torch.float32, device=dev)
            a.lse = lse.data_ptr() or None
        _run("uzip_paged_attention", a, dev, workspace, status, check)
    return (out, lse) if with_lse else out


def _state(refs, table, lengths, page_size):
    import torch

    _operand(table, "table", 2)
    s, width = table.shape
    if table.dtype != torch.int32 or (width > 1 and table.stride(1) != 1):
        _refuse("table: expected int32 [sequences, pages of a sequence], its rows contiguous")
    a = CacheArgs(refs.shape[0] if refs.dim() else 0, page_size, s, width)
    a.refs = _vector(refs, "refs", (a.pages,), torch.int32, table)
    a.table, a.ldt = table.data_ptr() or None, table.stride(0)
    a.lengths = _vector(lengths, "lengths", (s,), torch.int32, table)
    return a


def cache_reserve(refs, table, lengths, counts, tokens, page_size, *, out=None, workspace=None, status=None, check=False, stream=None):
    """Pages and slots for counts[i] (int32) new tokens of each sequence, at
    most `tokens` in all: (slots, positions, copies).  slots and positions are
    int64 [tokens], in the order of the sequences, -1 and 0 behind the last
    (for rotary_append).  The lowest free pages are taken.  A sequence whose
    part-full last page is shared gets a page in its place: copies int32
    [sequences, 2] holds {old, new} for cache_copy, {-1, -1} elsewhere.  refs,
    table and lengths are updated.  Where pages or columns of the table run out
    nothing changes, slots are -1, and `status` says so."""
    import torch

    a = _state(refs, table, lengths, page_size)
    a.list = _vector(counts, "counts", lengths.shape, torch.int32, table)
    a.tokens = tokens
    dev = table.device
    with _here(dev, stream):
        if out is None:
            out = (torch.empty(tokens, dtype=torch.int64, device=dev), torch.empty(tokens, dtype=torch.int64, device=dev),
                   torch.empty((a.seqs, 2), dtype=torch.int32, device=dev))
        a.slots = _vector(out[0], "out", (tokens,), torch.int64, table)
        a.positions = _vector(out[1], "out", (tokens,), torch.int64, table)
        a.pairs = _vector(out[2], "out", (a.seqs, 2), torch.int32, table)
        _run("uzip_cache_reserve", a, dev, workspace, status, check)
    return out


def cache_fork(refs, table, lengths, parents, children, page_size, *, workspace=None, status=None, check=False, stream=None):
    """children[j] become sequences that share the pages of parents[j] (int32
    indexes, -1 in both: none).  A child must be empty, listed once and nobody's
    parent; else nothing changes, and `status` says so."""
    import torch

    a = _state(refs, table, lengths, page_size)
    a.n = children.shape[0] if children.dim() else 0
    a.from_ = _vector(parents, "parents", (a.n,), torch.int32, table)
    a.list = _vector(children, "children", (a.n,), torch.int32, table)
    with _here(table.device, stream):
        _run("uzip_cache_fork", a, table.device, workspace, status, check)


def cache_free(refs, table, lengths, sequences, page_size, *, workspace=None, status=None, check=False, stream=None):
    """The sequences listed (int32 indexes, each once, -1: none) become empty;
    pages that nobody shares are free.  Where an index is wrong nothing changes,
    and `status` says so."""
    import torch

    a = _state(refs, table, lengths, page_size)
    a.n = sequences.shape[0] if sequences.dim() else 0
    a.list = _vector(sequences, "sequences", (a.n,), torch.int32, table)
    with _here(table.device, stream):
        _run("uzip_cache_free", a, table.device, workspace, status, check)


def cache_compact(refs, table, lengths, page_size, *, out=None, workspace=None, status=None, check=False, stream=None):
    """Moves the used pages to the front of the pool: updates refs and table and
    returns moves, int32 [pages // 2, 2] of {from, to} for cache_copy, -1 behind
    the last."""
    import torch

    a = _state(refs, table, lengths, page_size)
    dev = table.device
    with _here(dev, stream):
        if out is None:
            out = torch.empty((a.pages // 2, 2), dtype=torch.int32, device=dev)
        a.pairs = _vector(out, "out", (a.pages // 2, 2), torch.int32, table)
        _run("uzip_cache_compact", a, dev, workspace, status, check)
    return out


def cache_copy(k_pages, v_pages, pairs, *, to=None, status=None, check=False, stream=None):
    """Copies page pairs[j, 0] to page pairs[j, 1] (int32, -1: none) in keys and
    values, for pools [pages, heads, page size, d] or [layers, pages, ...].  `to`
    is another cache's (k_pages, v_pages), such as a buffer that is compressed
    and sent; the same cache where not given.  Where a page does not exist, is
    written twice or (within a cache) also read, nothing is copied, and `status`
    says so."""
    import torch

    if k_pages.dim() == 4:
        k_pages, v_pages = k_pages[None], v_pages[None]
        if to is not None:
            to = to[0][None], to[1][None]
    k, v = _pools(k_pages, v_pages, 5, None)
    layers, pages, heads, page, d = k_pages.shape
    a = CacheCopyArgs(_dtype_code(k_pages), 0, layers, heads, page, d, pages, pages, *k, *v, *k, *v)
    if to is not None:
        kt, vt = to
        shape = (layers, kt.shape[1] if kt.dim() == 5 else -1, heads, page, d)
        a.k_to, a.kt_layer, a.kt_page, a.kt_head, a.kt_token = _strided(kt, "to", shape, k_pages)
        a.v_to, a.vt_layer, a.vt_page, a.vt_head, a.vt_token = _strided(vt, "to", shape, k_pages)
        a.to_pages = shape[1]
    a.n = pairs.shape[0] if pairs.dim() else 0
    a.pairs = _vector(pairs, "pairs", (a.n, 2), torch.int32, k_pages)
    with _here(k_pages.device, stream):
        _run("uzip_cache_copy", a, k_pages.device, None, status, check)
