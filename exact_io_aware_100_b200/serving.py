"""Serving operators of libfa.so: rotary positions, a paged key/value cache, the attention that reads it and
the bookkeeping of its pages.

As in the rest of the binding, Python only checks and marshals arguments.  Low-level names mirror ``include/fa.h``
(``fa_rotary``, ``fa_paged_append``, ``fa_paged_decode``, ``fa_pages_*``); ``rotary``, ``paged_append``, ``paged_decode``
and ``pages_*`` build the layouts and allocate the outputs.

A serving step of a batch of sequences, all of it on the device and capturable into a CUDA graph:

    pages_extend(page_table, seq_lens, refcounts, page_size, seqs, tokens)      # lengths grow, pages are found
    q = paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q=q, freqs=freqs)
    o, lse = paged_decode(q, k_pages, v_pages, page_table, seq_lens)

Tensors may live on any CUDA device; a call runs on their device, on that device's current stream or on
``stream``.  With ``stream`` the outputs are allocated on it and the inputs are recorded as in use there.
"""
from __future__ import annotations

import ctypes
import math

import exact_io_aware_100_b200 as _fa

_I32, _I64, _VP = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


def _axes(*names):
    """Three int64 fields per operand: an fa_strides, flat."""
    return [(f"{n}_{axis}", _I64) for n in names for axis in ("batch", "head", "row")]


class FaRotaryLayout(ctypes.Structure):
    """fa_rotary_layout (include/fa.h), its strides flat."""
    _fields_ = [(n, _I32) for n in ("B", "H", "H_kv", "N", "d", "rotary_dim", "interleaved")] + \
               [("positions_batch", _I64)] + _axes("q", "k", "q_out", "k_out")


class FaPagedLayout(ctypes.Structure):
    """fa_paged_layout (include/fa.h), its strides flat."""
    _fields_ = [(n, _I32) for n in ("B", "H", "H_kv", "d", "N", "num_pages", "page_size", "max_pages")] + \
               [("table_stride", _I64)] + _axes("q", "o", "k", "v", "k_pages", "v_pages") + \
               [("cu_seqlens", _VP), ("total", _I32), ("rotary_dim", _I32), ("interleaved", _I32)]


class FaPagesLayout(ctypes.Structure):
    """fa_pages_layout (include/fa.h)."""
    _fields_ = [(n, _I32) for n in ("num_seqs", "num_pages", "page_size", "max_pages")] + [("table_stride", _I64)]


def declare(L) -> None:
    """The C signatures of the serving calls."""
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    RL, DL, GL = (ctypes.POINTER(t) for t in (FaRotaryLayout, FaPagedLayout, FaPagesLayout))
    L.fa_rotary.argtypes = [P, P, P, P, P, P, RL, F, I, I, P]
    L.fa_paged_append.argtypes = [P, P, P, P, P, P, P, P, P, DL, F, P]
    L.fa_paged_decode.argtypes = [P, P, P, P, P, P, P, DL, F, I, P, Z, P]
    L.fa_paged_decode_workspace_size.argtypes = [DL]
    L.fa_paged_decode_workspace_size.restype = Z
    L.fa_pages_workspace_size.argtypes = [GL, I]
    L.fa_pages_workspace_size.restype = Z
    L.fa_pages_extend.argtypes = [P, P, P, GL, P, P, I, P, P, Z, P]
    L.fa_pages_fork.argtypes = [P, P, P, GL, P, P, I, P, P, P, Z, P]
    L.fa_pages_free.argtypes = [P, P, P, GL, P, I, P]
    L.fa_pages_compact.argtypes = [P, P, P, GL, P, P, Z, P]
    L.fa_pages_copy.argtypes = [P, P, P, I, DL, P]
    for name in ("fa_rotary", "fa_paged_append", "fa_paged_decode", "fa_pages_extend", "fa_pages_fork",
                 "fa_pages_free", "fa_pages_compact", "fa_pages_copy"):
        getattr(L, name).restype = I


# ----------------------------------------------------------------- C ABI mirrors
def fa_rotary(q, k, q_out, k_out, positions, freqs, layout: FaRotaryLayout, magnitude: float, inverse: bool,
              dtype: int, stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_rotary(p(q), p(k), p(q_out), p(k_out), p(positions), p(freqs), layout, magnitude,
                                            int(bool(inverse)), dtype, _fa._stream(stream)), "fa_rotary")


def fa_paged_append(q, k, v, o, k_pages, v_pages, page_table, seq_lens, freqs, layout: FaPagedLayout,
                    magnitude: float = 1.0, stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_paged_append(p(q), p(k), p(v), p(o), p(k_pages), p(v_pages), p(page_table),
                                                  p(seq_lens), p(freqs), layout, magnitude, _fa._stream(stream)),
               "fa_paged_append")


def fa_paged_decode(q, k_pages, v_pages, page_table, seq_lens, o, lse, layout: FaPagedLayout, causal: bool, workspace,
                    scale: float | None = None, stream=None) -> None:
    p = _fa._ptr
    scale = 1.0 / math.sqrt(layout.d) if scale is None else float(scale)
    _fa._check(_fa.load_library().fa_paged_decode(p(q), p(k_pages), p(v_pages), p(page_table), p(seq_lens), p(o), p(lse),
                                                  layout, scale, int(bool(causal)), p(workspace),
                                                  _fa._ws_bytes(workspace), _fa._stream(stream)), "fa_paged_decode")


def fa_paged_decode_workspace_size(layout: FaPagedLayout) -> int:
    return int(_fa.load_library().fa_paged_decode_workspace_size(layout))


def fa_pages_workspace_size(layout: FaPagesLayout, n: int) -> int:
    return int(_fa.load_library().fa_pages_workspace_size(layout, n))


def fa_pages_extend(page_table, seq_lens, refcounts, layout: FaPagesLayout, seqs, tokens, status, workspace,
                    stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_pages_extend(p(page_table), p(seq_lens), p(refcounts), layout, p(seqs), p(tokens),
                                                  seqs.numel(), p(status), p(workspace), _fa._ws_bytes(workspace),
                                                  _fa._stream(stream)), "fa_pages_extend")


def fa_pages_fork(page_table, seq_lens, refcounts, layout: FaPagesLayout, src, dst, copies, status, workspace,
                  stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_pages_fork(p(page_table), p(seq_lens), p(refcounts), layout, p(src), p(dst),
                                                src.numel(), p(copies), p(status), p(workspace),
                                                _fa._ws_bytes(workspace), _fa._stream(stream)), "fa_pages_fork")


def fa_pages_free(page_table, seq_lens, refcounts, layout: FaPagesLayout, seqs, stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_pages_free(p(page_table), p(seq_lens), p(refcounts), layout, p(seqs), seqs.numel(),
                                                _fa._stream(stream)), "fa_pages_free")


def fa_pages_compact(page_table, seq_lens, refcounts, layout: FaPagesLayout, copies, workspace, stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_pages_compact(p(page_table), p(seq_lens), p(refcounts), layout, p(copies),
                                                   p(workspace), _fa._ws_bytes(workspace), _fa._stream(stream)),
               "fa_pages_compact")


def fa_pages_copy(k_pages, v_pages, copies, layout: FaPagedLayout, stream=None) -> None:
    p = _fa._ptr
    _fa._check(_fa.load_library().fa_pages_copy(p(k_pages), p(v_pages), p(copies), copies.shape[0], layout,
                                                _fa._stream(stream)), "fa_pages_copy")


# ----------------------------------------------------------------- where a call runs
class _Here:
    """The tensors' device is the current one and its current stream is meant: nothing to set up."""
    __slots__ = ()

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


class _There:
    """Makes the tensors' device and ``stream`` (if given) current for a call.  Tensors used on a stream of the caller's
    are recorded as in use there."""
    __slots__ = ("guards", "tensors", "stream")

    def __init__(self, stream, device, tensors):
        import torch
        self.guards = (torch.cuda.device(device),)
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.guards += (torch.cuda.stream(stream),)
        self.tensors, self.stream = tensors, stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        if self.stream is not None and exc[0] is None:
            import torch
            if not torch.cuda.is_current_stream_capturing():   # a graph keeps its own memory alive
                for t in self.tensors:
                    if t is not None:
                        t.record_stream(self.stream)
        for g in reversed(self.guards):
            g.__exit__(*exc)


_HERE = _Here()


def _launch(stream, *tensors):
    """Where a call on these tensors runs, as a context; checks that they share one CUDA device."""
    import torch
    device = None
    for t in tensors:
        if t is not None:
            index = t.get_device()
            if index != device:
                if index < 0:
                    raise ValueError("expected a CUDA tensor: the library reads and writes device memory only")
                if device is not None:
                    raise ValueError(f"tensors on different devices: cuda:{device} and cuda:{index}")
                device = index
    if stream is None and device == torch.cuda.current_device():
        return _HERE
    return _There(stream, device, tensors)


def _int32(t, name: str, dims: int):
    import torch
    if t.dtype != torch.int32 or t.dim() != dims or (t.stride(-1) != 1 and t.numel() > 1 and t.shape[-1] > 1):
        raise ValueError(f"{name}: expected a {dims}-D int32 tensor, contiguous in its last axis")


def _rows(t, name: str, dims, dtypes):
    """Checks [B, heads, rows, d] (4-D) or packed [rows, heads, d] (3-D); d contiguous."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() not in dims or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name}: expected [B, heads, rows, d]" + (" or packed [rows, heads, d]" if 3 in dims else "") +
                         " with contiguous d")


def _st(t):
    """(batch, head, row) strides of a 4-D or packed 3-D operand; zeros for None."""
    if t is None:
        return 0, 0, 0
    s = t.stride()
    return (s[0], s[1], s[2]) if len(s) == 4 else (0, s[1], s[0])


def _freqs(freqs):
    import torch
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs: expected a contiguous 1-D float64 tensor (rotary_frequencies gives one)")
    return 2 * freqs.numel()


# ----------------------------------------------------------------- rotary positions
def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, low: float | None = None, high: float | None = None,
                       device="cuda"):
    """(freqs, magnitude) of ``rotary``: float64 [rotary_dim / 2] radians per position, base^(-2 i / rotary_dim), and the
    factor on cos and sin.  ``scaling`` stretches them for contexts ``factor`` times the ``original_length`` trained on:

    - ``"linear"``: every frequency divided by ``factor`` (positions interpolated);
    - ``"ntk"``: the base raised to base * factor^(r / (r - 2)), which leaves the fastest pair and divides the slowest
      by ``factor``;
    - ``"bands"``: by the turns n a pair makes over ``original_length``: divided by ``factor`` below ``low`` (1), kept
      above ``high`` (4), blended linearly in n between;
    - ``"yarn"``: divided where n is below ``low`` (1), kept above ``high`` (32), blended linearly in the pair's index
      between (rounded outwards to whole pairs), and magnitude 0.1 ln(factor) + 1.
    """
    import torch
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not base > 0 or not factor >= 1.0:
        raise ValueError("base must be positive and factor at least 1")
    r, magnitude = rotary_dim, 1.0
    if scaling == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("bands", "yarn"):
        if original_length is None or original_length < 1:
            raise ValueError(f"scaling {scaling!r} needs original_length")
        low = 1.0 if low is None else low
        high = (4.0 if scaling == "bands" else 32.0) if high is None else high
        if not 0 < low < high:
            raise ValueError("0 < low < high is needed")
        if scaling == "bands":
            keep = ((original_length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        else:
            # the (fractional) pair that makes n turns: base^(-2 i / r) original_length = 2 pi n
            at = [r * math.log(original_length / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (high, low)]
            first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
            keep = 1 - ((torch.arange(r // 2, dtype=torch.float64) - first) / max(last - first, 1e-3)).clamp(0, 1)
            magnitude = 0.1 * math.log(factor) + 1.0
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), magnitude


def _rotary(q, k, freqs, positions, interleaved, magnitude, out, inverse, stream):
    import torch
    dtypes = (torch.bfloat16, torch.float32)
    _rows(q, "q", (3, 4), dtypes)
    r = _freqs(freqs)
    packed = q.dim() == 3
    if packed:
        N, H, d = q.shape
        B = 1
    else:
        B, H, N, d = q.shape
    H_kv = 0
    if k is not None:
        _rows(k, "k", (q.dim(),), (q.dtype,))
        H_kv = k.shape[1]
        if k.shape[0] != q.shape[0] or k.shape[-1] != d or (not packed and k.shape[2] != N):
            raise ValueError("q and k: batch, rows and d must agree")
    pos_batch = 0
    if positions is not None:
        _int32(positions, "positions", 2 if not packed and positions.dim() == 2 else 1)
        if positions.shape[-1] != N or (positions.dim() == 2 and positions.shape[0] != B):
            raise ValueError("positions: expected one per row ([rows] or [B, rows])")
        pos_batch = positions.stride(0) if positions.dim() == 2 else 0
    with _launch(stream, q, k, freqs, positions, *(out or ())):
        if out is None:
            q_out, k_out = torch.empty_like(q), None if k is None else torch.empty_like(k)
        else:
            q_out, k_out = out
            for name, x, y in (("q", q, q_out), ("k", k, k_out)):
                if (x is None) != (y is None) or (x is not None and (y.shape != x.shape or y.dtype != x.dtype or
                                                                    (d > 1 and y.stride(-1) != 1))):
                    raise ValueError(f"out: {name} must have its input's shape and dtype, d contiguous")
        layout = FaRotaryLayout(B, H, H_kv, N, d, r, int(bool(interleaved)), pos_batch, *_st(q), *_st(k), *_st(q_out),
                                *_st(k_out))
        fa_rotary(q, k, q_out, k_out, positions, freqs, layout, float(magnitude), inverse,
                  _fa.FA_BF16 if q.dtype == torch.bfloat16 else _fa.FA_F32)
    return q_out, k_out


def rotary(q, k, freqs, positions=None, interleaved: bool = False, magnitude: float = 1.0, out=None, stream=None):
    """(q', k'): q [B, H, N, d] and k [B, H_kv, N, d] (bf16 or float32, any strides; or packed [rows, heads, d]; k may be
    None) with the first 2 * len(freqs) columns of every head turned by the angle position * freqs (fa_rotary).
    positions: int32 [N], [B, N], packed [rows]; None: 0 .. N - 1.  ``out``: a pair to write to, which may be (q, k)."""
    return _rotary(q, k, freqs, positions, interleaved, magnitude, out, False, stream)


def rotary_backward(dq, dk, freqs, positions=None, interleaved: bool = False, magnitude: float = 1.0, out=None,
                    stream=None):
    """Gradients of q and k from those of ``rotary``'s outputs: the map's transpose, a turn by the negative angle."""
    return _rotary(dq, dk, freqs, positions, interleaved, magnitude, out, True, stream)


# ----------------------------------------------------------------- the paged cache
def _cache(k_pages, v_pages):
    import torch
    _rows(k_pages, "k_pages", (4,), (torch.bfloat16,))
    _rows(v_pages, "v_pages", (4,), (torch.bfloat16,))
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages: one shape [pages, H_kv, page_size, d]")
    return k_pages.shape


def _table(page_table, seq_lens, B=None):
    _int32(page_table, "page_table", 2)
    _int32(seq_lens, "seq_lens", 1)
    if page_table.shape[0] != seq_lens.shape[0] or (B is not None and B != seq_lens.shape[0]):
        raise ValueError("page_table, seq_lens and the batch must agree")
    return page_table.shape[1]


def paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q=None, freqs=None, interleaved: bool = False,
                 magnitude: float = 1.0, cu_seqlens=None, out=None, stream=None):
    """Writes new keys and values (bf16) into the cache k_pages, v_pages [pages, H_kv, page_size, d] (any strides; pages of
    [pages, page_size, H_kv, d] memory are passed as their transpose(1, 2)), and returns q turned (None without q).

    k, v: [B, H_kv, N, d], or packed [rows, H_kv, d] with int32 offsets ``cu_seqlens`` [B + 1].  ``seq_lens`` are the
    lengths after the call: token i of the n of sequence b goes to position seq_lens[b] - n + i.  With ``freqs`` the
    keys, and q [B, H, N, d] (or packed), are turned as by ``rotary`` at those positions.  A token whose position would
    be negative is padding: not written, and zero in the returned q; so are packed rows outside every sequence, which keep
    their values when ``out`` is q itself."""
    import torch
    P, H_kv, page, d = _cache(k_pages, v_pages)
    packed = cu_seqlens is not None
    for name, t in (("k", k), ("v", v)):
        _rows(t, name, (3 if packed else 4,), (torch.bfloat16,))
        if t.shape[1] != H_kv or t.shape[-1] != d or t.shape != k.shape:
            raise ValueError("k and v: heads and d as in the cache, one shape")
    B = cu_seqlens.numel() - 1 if packed else k.shape[0]
    M = _table(page_table, seq_lens, B)
    if packed:
        _int32(cu_seqlens, "cu_seqlens", 1)
    if q is not None:
        _rows(q, "q", (k.dim(),), (torch.bfloat16,))
        if q.shape[0] != k.shape[0] or q.shape[-1] != d or (not packed and q.shape[2] != k.shape[2]):
            raise ValueError("q and k: batch, rows and d must agree")
    r = 0 if freqs is None else _freqs(freqs)
    with _launch(stream, q, k, v, k_pages, v_pages, page_table, seq_lens, freqs, cu_seqlens, out):
        if out is None:
            out = None if q is None else torch.empty_like(q)
        elif q is None or out.shape != q.shape or out.dtype != q.dtype or (d > 1 and out.stride(-1) != 1):
            raise ValueError("out: must have q's shape and dtype, d contiguous")
        layout = FaPagedLayout(B, 0 if q is None else q.shape[1], H_kv, d, 0 if packed else k.shape[2], P, page, M,
                               page_table.stride(0), *_st(q), *_st(out), *_st(k), *_st(v), *k_pages.stride()[:3],
                               *v_pages.stride()[:3], _fa._ptr(cu_seqlens), k.shape[0] if packed else 0, r,
                               int(bool(interleaved)))
        fa_paged_append(q, k, v, out, k_pages, v_pages, page_table, seq_lens, freqs, layout, float(magnitude))
    return out


def paged_decode(q, k_pages, v_pages, page_table, seq_lens, causal: bool = True, scale: float | None = None, stream=None,
                 workspace=None):
    """O, lse of the last N positions q [B, H, N, d] of each sequence against its seq_lens[b] cached keys (bf16; H a
    multiple of the cache's H_kv).  Rows that see no key (an empty sequence) give O = 0, lse = -inf."""
    import torch
    P, H_kv, page, d = _cache(k_pages, v_pages)
    _rows(q, "q", (4,), (torch.bfloat16,))
    B, H, N, dq = q.shape
    if dq != d:
        raise ValueError("q and the cache: d must agree")
    M = _table(page_table, seq_lens, B)
    with _launch(stream, q, k_pages, v_pages, page_table, seq_lens, workspace):
        o = torch.empty_like(q)
        lse = q.new_empty((B, H, N), dtype=torch.float32)
        layout = FaPagedLayout(B, H, H_kv, d, N, P, page, M, page_table.stride(0), *_st(q), *_st(o), 0, 0, 0, 0, 0, 0,
                               *k_pages.stride()[:3], *v_pages.stride()[:3], None, 0, 0, 0)
        if workspace is None:
            workspace = _fa._workspace(fa_paged_decode_workspace_size(layout), q.device)
        fa_paged_decode(q, k_pages, v_pages, page_table, seq_lens, o, lse, layout, causal, workspace, scale)
    return o, lse


# ----------------------------------------------------------------- bookkeeping of pages
def _pages_state(page_table, seq_lens, refcounts, page_size, *requests):
    M = _table(page_table, seq_lens)
    _int32(refcounts, "refcounts", 1)
    for name, t in requests:
        _int32(t, name, 1)
        if t.numel() != requests[0][1].numel():
            raise ValueError(f"{requests[0][0]} and {name}: one length")
    return FaPagesLayout(page_table.shape[0], refcounts.numel(), int(page_size), M, page_table.stride(0))


def _pages_workspace(layout, n, workspace, device):
    return _fa._workspace(fa_pages_workspace_size(layout, n), device) if workspace is None else workspace


def pages_extend(page_table, seq_lens, refcounts, page_size: int, seqs, tokens, stream=None, workspace=None):
    """Sequences ``seqs`` (int32 [n]) grow by ``tokens`` (int32 [n]) positions and get the pages they need: the free ones
    of lowest number, in the order of the requests.  page_table [S, max_pages], seq_lens [S] and refcounts [pages] (int32)
    are updated in place.  Returns status int32 [n]: FA_OK, FA_ERR_WORKSPACE (no page left) or FA_ERR_INVALID; a request
    that is not FA_OK changed nothing."""
    import torch
    layout = _pages_state(page_table, seq_lens, refcounts, page_size, ("seqs", seqs), ("tokens", tokens))
    with _launch(stream, page_table, seq_lens, refcounts, seqs, tokens, workspace):
        status = torch.empty_like(seqs)
        fa_pages_extend(page_table, seq_lens, refcounts, layout, seqs, tokens, status,
                        _pages_workspace(layout, seqs.numel(), workspace, seqs.device))
    return status


def pages_fork(page_table, seq_lens, refcounts, page_size: int, src, dst, stream=None, workspace=None):
    """The empty sequences ``dst`` (int32 [n]) become copies of ``src``: whole pages are shared, a last page that is not
    full gets a page of its own.  Returns (copies int32 [n, 3], status int32 [n]); ``pages_copy`` with ``copies`` then
    brings the contents over, in each layer's cache."""
    import torch
    layout = _pages_state(page_table, seq_lens, refcounts, page_size, ("src", src), ("dst", dst))
    with _launch(stream, page_table, seq_lens, refcounts, src, dst, workspace):
        status = torch.empty_like(src)
        copies = torch.empty((src.numel(), 3), dtype=torch.int32, device=src.device)
        fa_pages_fork(page_table, seq_lens, refcounts, layout, src, dst, copies, status,
                      _pages_workspace(layout, src.numel(), workspace, src.device))
    return copies, status


def pages_free(page_table, seq_lens, refcounts, page_size: int, seqs, stream=None) -> None:
    """Sequences ``seqs`` (int32 [n]) become empty; their pages are free once no other sequence holds them."""
    layout = _pages_state(page_table, seq_lens, refcounts, page_size, ("seqs", seqs))
    with _launch(stream, page_table, seq_lens, refcounts, seqs):
        fa_pages_free(page_table, seq_lens, refcounts, layout, seqs)


def pages_compact(page_table, seq_lens, refcounts, page_size: int, stream=None, workspace=None):
    """Moves the pages in use to the lowest numbers.  Returns copies int32 [pages // 2, 3] for ``pages_copy``."""
    import torch
    layout = _pages_state(page_table, seq_lens, refcounts, page_size)
    with _launch(stream, page_table, seq_lens, refcounts, workspace):
        copies = torch.empty((refcounts.numel() // 2, 3), dtype=torch.int32, device=refcounts.device)
        fa_pages_compact(page_table, seq_lens, refcounts, layout, copies,
                         _pages_workspace(layout, 0, workspace, refcounts.device))
    return copies


def pages_copy(k_pages, v_pages, copies, stream=None) -> None:
    """Copies pages within k_pages, v_pages [pages, H_kv, page_size, d] (any strides) as ``copies`` lists them."""
    P, H_kv, page, d = _cache(k_pages, v_pages)
    _int32(copies, "copies", 2)
    if copies.shape[1] != 3 or not copies.is_contiguous():
        raise ValueError("copies: expected a contiguous [n, 3] tensor")
    with _launch(stream, k_pages, v_pages, copies):
        layout = FaPagedLayout(1, 0, H_kv, d, 0, P, page, 0, 0, *(0,) * 12, *k_pages.stride()[:3],
                               *v_pages.stride()[:3], None, 0, 0, 0)
        fa_pages_copy(k_pages, v_pages, copies, layout)
