"""Serving operators of libfa.so: rotary positions, a paged key/value cache, the attention that reads it and
the bookkeeping of its pages.

As in the rest of the binding, nothing is computed here.  Low-level names mirror ``include/fa.h`` (``fa_rotary``,
``fa_paged_append``, ``fa_paged_decode``, ``fa_pages_*``); ``rotary``, ``paged_append``, ``paged_decode`` and ``pages_*``
check the tensors, build the layouts and allocate the outputs, in ``_serving.so`` (csrc/serving_binding.cpp), because a
generation step makes several of these calls and their kernels take a few microseconds each.

A serving step of a batch of sequences, all of it on the device and capturable into a CUDA graph:

    status = pages_extend(page_table, seq_lens, refcounts, page_size, seqs, tokens)    # lengths grow, pages are found
    q = paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q=q, freqs=freqs, tokens=tokens, status=status)
    o, lse = paged_decode(q, k_pages, v_pages, page_table, seq_lens)

``seqs`` are the batch's sequences in their order (the rows of ``page_table``), ``tokens`` what each of them gets in this
step.  Append takes both ``tokens`` and ``status``, so that a sequence that is idle (0 tokens) or whose request was refused
(no page left) keeps its cache as it was; its rows of q are zero, and its rows of o mean nothing.  After the step the host
reads ``status``, makes room for the refused (frees or moves sequences) and gives them the same token again.

Tensors may live on any CUDA device; a call runs on their device, on that device's current stream or on
``stream``.  With ``stream`` the outputs are allocated on it and the inputs are recorded as in use there.
A call on no sequences or no rows returns empty tensors.
"""
from __future__ import annotations

import ctypes
import math
import os

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
               [("cu_seqlens", _VP), ("total", _I32), ("rotary_dim", _I32), ("interleaved", _I32), ("tokens", _VP),
                ("status", _VP)]


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
_ext = None


def _native():
    """The extension module, its functions bound to libfa.so's."""
    global _ext
    if _ext is None:
        import torch  # noqa: F401 (its libraries)
        try:
            from . import _serving
        except ImportError as e:
            from . import build
            what = "does not load with this Python and torch" if os.path.exists(build.EXT) else "is not built"
            raise RuntimeError(f"_serving.so {what} ({e}); run `python -m exact_io_aware_100_b200.build`") from e
        L = _fa.load_library()
        _serving.bind(_fa.FaError, *(ctypes.cast(getattr(L, name), _VP).value for name in (
            "fa_rotary", "fa_paged_append", "fa_paged_decode", "fa_paged_decode_workspace_size", "fa_pages_workspace_size",
            "fa_pages_extend", "fa_pages_fork", "fa_pages_free", "fa_pages_compact", "fa_pages_copy")))
        _ext = _serving
    return _ext


class _On:
    """Makes the caller's ``stream`` (of torch, or a handle) current for a call on `tensors`, which are recorded as in use
    there."""
    __slots__ = ("guards", "tensors", "stream")

    def __init__(self, stream, *tensors):
        import torch
        device = tensors[0].get_device()
        if device < 0:
            raise ValueError("expected a CUDA tensor: the library reads and writes device memory only")
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        self.guards = (torch.cuda.device(device), torch.cuda.stream(stream))
        self.tensors, self.stream = tensors, stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        import torch
        if exc[0] is None and not torch.cuda.is_current_stream_capturing():   # a graph keeps its own memory alive
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        for g in reversed(self.guards):
            g.__exit__(*exc)


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


def rotary(q, k, freqs, positions=None, interleaved: bool = False, magnitude: float = 1.0, out=None, stream=None):
    """(q', k'): q [B, H, N, d] and k [B, H_kv, N, d] (bf16 or float32, any strides; or packed [rows, heads, d]; k may be
    None) with the first 2 * len(freqs) columns of every head turned by the angle position * freqs (fa_rotary).
    positions: int32 [N], [B, N], packed [rows]; None: 0 .. N - 1.  ``out``: a pair to write to, which may be (q, k)."""
    if stream is not None:
        with _On(stream, q, k, freqs, positions, *(out or ())):
            return rotary(q, k, freqs, positions, interleaved, magnitude, out)
    return (_ext or _native()).rotary(q, k, freqs, positions, interleaved, magnitude, out, False)


def rotary_backward(dq, dk, freqs, positions=None, interleaved: bool = False, magnitude: float = 1.0, out=None,
                    stream=None):
    """Gradients of q and k from those of ``rotary``'s outputs: the map's transpose, a turn by the negative angle."""
    if stream is not None:
        with _On(stream, dq, dk, freqs, positions, *(out or ())):
            return rotary_backward(dq, dk, freqs, positions, interleaved, magnitude, out)
    return (_ext or _native()).rotary(dq, dk, freqs, positions, interleaved, magnitude, out, True)


# ----------------------------------------------------------------- the paged cache
def paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q=None, freqs=None, interleaved: bool = False,
                 magnitude: float = 1.0, cu_seqlens=None, out=None, stream=None, tokens=None, status=None):
    """Writes new keys and values (bf16) into the cache k_pages, v_pages [pages, H_kv, page_size, d] (any strides; pages of
    [pages, page_size, H_kv, d] memory are passed as their transpose(1, 2)), and returns q turned (None without q).

    k, v: [B, H_kv, N, d], or packed [rows, H_kv, d] with int32 offsets ``cu_seqlens`` [B + 1].  ``seq_lens`` are the
    lengths after the call: token i of the n of sequence b goes to position seq_lens[b] - n + i.  With ``freqs`` the
    keys, and q [B, H, N, d] (or packed), are turned as by ``rotary`` at those positions.  A token whose position would
    be negative is padding: not written, and zero in the returned q; so are packed rows outside every sequence, which keep
    their values when ``out`` is q itself.

    ``tokens`` (int32 [B]): only the last tokens[b] of sequence b's rows are tokens, the others padding.  ``status`` (int32
    [B], as ``pages_extend`` returns it): a sequence whose entry is not FA_OK has none.  Without them every sequence has n new
    tokens, and one that did not grow by n before the call loses its last cached keys and values to them."""
    if stream is not None:
        with _On(stream, k, v, k_pages, v_pages, page_table, seq_lens, q, freqs, cu_seqlens, out, tokens, status):
            return paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q, freqs, interleaved, magnitude, cu_seqlens,
                                out, None, tokens, status)
    return (_ext or _native()).paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q, freqs, interleaved, magnitude,
                                            cu_seqlens, out, tokens, status)


def paged_decode(q, k_pages, v_pages, page_table, seq_lens, causal: bool = True, scale: float | None = None, stream=None,
                 workspace=None):
    """O, lse of the last N positions q [B, H, N, d] of each sequence against its seq_lens[b] cached keys (bf16; H a
    multiple of the cache's H_kv).  Rows that see no key (an empty sequence) give O = 0, lse = -inf."""
    if stream is not None:
        with _On(stream, q, k_pages, v_pages, page_table, seq_lens, workspace):
            return paged_decode(q, k_pages, v_pages, page_table, seq_lens, causal, scale, None, workspace)
    return (_ext or _native()).paged_decode(q, k_pages, v_pages, page_table, seq_lens, causal, scale, workspace)


# ----------------------------------------------------------------- bookkeeping of pages
def pages_extend(page_table, seq_lens, refcounts, page_size: int, seqs, tokens, stream=None, workspace=None):
    """Sequences ``seqs`` (int32 [n]) grow by ``tokens`` (int32 [n]) positions and get the pages they need: the free ones
    of lowest number, in the order of the requests.  page_table [S, max_pages], seq_lens [S] and refcounts [pages] (int32)
    are updated in place.  Returns status int32 [n]: FA_OK, FA_ERR_WORKSPACE (no page left) or FA_ERR_INVALID; a request
    that is not FA_OK changed nothing (and ``paged_append`` with this status and the same tokens writes nothing for it)."""
    if stream is not None:
        with _On(stream, page_table, seq_lens, refcounts, seqs, tokens, workspace):
            return pages_extend(page_table, seq_lens, refcounts, page_size, seqs, tokens, None, workspace)
    return (_ext or _native()).pages_extend(page_table, seq_lens, refcounts, page_size, seqs, tokens, workspace)


def pages_fork(page_table, seq_lens, refcounts, page_size: int, src, dst, stream=None, workspace=None):
    """The empty sequences ``dst`` (int32 [n]) become copies of ``src``: whole pages are shared, a last page that is not
    full gets a page of its own.  Returns (copies int32 [n, 3], status int32 [n]); ``pages_copy`` with ``copies`` then
    brings the contents over, in each layer's cache."""
    if stream is not None:
        with _On(stream, page_table, seq_lens, refcounts, src, dst, workspace):
            return pages_fork(page_table, seq_lens, refcounts, page_size, src, dst, None, workspace)
    return (_ext or _native()).pages_fork(page_table, seq_lens, refcounts, page_size, src, dst, workspace)


def pages_free(page_table, seq_lens, refcounts, page_size: int, seqs, stream=None) -> None:
    """Sequences ``seqs`` (int32 [n]) become empty; their pages are free once no other sequence holds them."""
    if stream is not None:
        with _On(stream, page_table, seq_lens, refcounts, seqs):
            return pages_free(page_table, seq_lens, refcounts, page_size, seqs)
    (_ext or _native()).pages_free(page_table, seq_lens, refcounts, page_size, seqs)


def pages_compact(page_table, seq_lens, refcounts, page_size: int, stream=None, workspace=None):
    """Moves the pages in use to the lowest numbers.  Returns copies int32 [pages // 2, 3] for ``pages_copy``."""
    if stream is not None:
        with _On(stream, page_table, seq_lens, refcounts, workspace):
            return pages_compact(page_table, seq_lens, refcounts, page_size, None, workspace)
    return (_ext or _native()).pages_compact(page_table, seq_lens, refcounts, page_size, workspace)


def pages_copy(k_pages, v_pages, copies, stream=None) -> None:
    """Copies pages within k_pages, v_pages [pages, H_kv, page_size, d] (any strides) as ``copies`` lists them."""
    if stream is not None:
        with _On(stream, k_pages, v_pages, copies):
            return pages_copy(k_pages, v_pages, copies)
    (_ext or _native()).pages_copy(k_pages, v_pages, copies)
