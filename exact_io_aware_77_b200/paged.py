"""Paged key/value cache: appending rotated rows, and attention over the pages.

Pages are ``[n_pages, H_kv, page_size, d]`` tensors (any strides with a contiguous last dimension),
bf16 or E4M3 codes (``torch.float8_e4m3fn`` or ``torch.uint8``; K = k_scale * code, V = v_scale * code).  Row j of
sequence b is row ``j % page_size`` of page ``page_table[b, j // page_size]``.  ``lengths`` counts the
keys each sequence holds once the new rows are appended, and ``counts`` its new rows where they are
fewer than the batch has: the same tensors serve the append and the attention after it.  Page numbers, lengths and positions are read on the device; one out of
range is never followed, and ``check_status`` reports it.
"""

from __future__ import annotations

import math

import torch
from torch._C import _cuda_getCurrentRawStream as _stream_of
from torch._C import _cuda_getDevice as _current_device

from . import _lib

_BF16, _INT32, _FP32 = torch.bfloat16, torch.int32, torch.float32
_CODES = (torch.float8_e4m3fn, torch.uint8)
_INT_MAX = 0x7fffffff

# The checks below read each property of a tensor once and compare device numbers: a generation step
# takes a few microseconds on the GPU, and the host must not take longer.


def _launch(name, device, *args):
    """Call a library entry point on the current stream of the tensors' device, with that device
    current (the library launches on the current device)."""
    fn, stream = getattr(_lib.load(), name), _stream_of(device)
    if _current_device() == device:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != _lib.FA_OK:
        raise _lib.FAError(name, st)


def _rows(t, what, shape, device):
    """A bf16 tensor of that shape with contiguous d; returns its first three strides."""
    if t.shape != shape or t.dtype is not _BF16 or t.get_device() != device:
        raise ValueError(f"{what} must be a bf16 tensor {tuple(shape)} on cuda:{device}")
    b, h, n, c = t.stride()
    if c != 1:
        raise ValueError(f"{what} must have a contiguous last dimension")
    return b, h, n


def _ints(t, what, shape, device):
    """The address of a contiguous int32 tensor of that shape."""
    if t.shape != shape or t.dtype is not _INT32 or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor {tuple(shape)} on cuda:{device}")
    at = t.data_ptr()
    if at == 0 and t.numel():   # (an address of 0 would stand for an argument left out)
        raise ValueError(f"{what} has no memory")
    return at


def _small(*sizes):
    """Sizes that the library's ints hold (ctypes would pass the low 32 bits of any other)."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX:
        raise ValueError(f"size out of range: {sizes}")


def _first(t, what):
    """Shape, device number (-1 on the host) and first three strides of the tensor that sets a call's."""
    shape, device, stride = t.shape, t.get_device(), t.stride()
    if len(shape) != 4 or device < 0 or t.dtype is not _BF16 or stride[3] != 1:
        raise ValueError(f"{what} must be a bf16 CUDA tensor of four dimensions with a contiguous last one")
    _small(*shape)
    return shape, device, stride[:3]


def _prefix_length(n, prefix_pages, page_size):
    n = int(n)
    if prefix_pages.dim() != 1 or n < 0 or prefix_pages.shape[0] * page_size < n:
        raise ValueError("prefix_pages must be a 1-D tensor whose pages hold prefix_length keys")
    _small(n)
    return n


def _cache(k_pages, v_pages, page_table, B, d, device, k_scale, v_scale):
    """The cache's description as fa_paged_kv bytes, and its K/V heads."""
    shape, dtype = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or shape != v_pages.shape or shape[3] != d or v_pages.dtype is not dtype:
        raise ValueError("k_pages and v_pages must be [n_pages, H_kv, page_size, d] tensors of one type")
    fp8 = dtype is not _BF16
    if fp8 and dtype not in _CODES:
        raise ValueError("pages must be bf16 or E4M3 codes (float8_e4m3fn or uint8)")
    if not fp8 and not k_scale == v_scale == 1.0:
        raise ValueError("k_scale and v_scale are the scales of E4M3 codes: bf16 pages have none")
    kb, kh, kn, kc = k_pages.stride()
    vb, vh, vn, vc = v_pages.stride()
    if kc != 1 or vc != 1:
        raise ValueError("pages must have a contiguous last dimension")
    table_shape = page_table.shape
    if len(table_shape) != 2 or table_shape[0] != B or page_table.dtype is not _INT32:
        raise ValueError(f"page_table must be an int32 tensor [{B}, max_pages]")
    row, column = page_table.stride()
    width = table_shape[1]
    if width > 1 and column != 1:
        raise ValueError("page_table must have contiguous rows")
    if k_pages.get_device() != device or v_pages.get_device() != device or page_table.get_device() != device:
        raise ValueError(f"the pages and the page table must be on cuda:{device}")
    n, H_kv, page_size, _ = shape
    return _lib.PAGED_KV.pack(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kb, kh, kn, vb, vh, vn,
                              max(row, width) if B == 1 else row, n, page_size, width, fp8, k_scale, v_scale), H_kv


def append_kv(k, v, k_pages, v_pages, page_table, lengths, counts=None, q=None, q_out=None, cos=None, sin=None,
              positions=None, sections=None, interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0):
    """Append N new rows per sequence to a paged cache, rotating q and k on the way.

    k, v: bf16 [B, H_kv, N, d]; q (optional): bf16 [B, H, N, d].  ``lengths`` int32 [B] counts each
    sequence's keys after the append; ``counts`` int32 [B] its new rows (the first ones; default
    all N): row i becomes row ``lengths[b] - counts[b] + i``.  Padding rows, and rows of a sequence
    whose place would be negative (an idle slot with length 0), are not written anywhere.

    cos, sin: fp32 [n_angles, rot / 2] tables; without them nothing is rotated.  A row turns by the
    angles of its place in the sequence, or of ``positions`` int32 [B, N]; with several axes (time,
    height and width) ``positions`` is [axes, B, N] and ``sections`` gives the pairs of each axis, in
    order.  Pairs are elements (p, p + rot / 2), or with ``interleaved`` (2p, 2p + 1), of a head's
    first rot elements.

    Returns the rotated q (``q_out`` if given, which may be q itself), or None without q.
    """
    shape, device, k_st = _first(k, "k")
    B, H_kv, N, d = shape
    cache, heads = _cache(k_pages, v_pages, page_table, B, d, device, k_scale, v_scale)
    if heads != H_kv:
        raise ValueError(f"k has {H_kv} heads, the pages {heads}")
    v_st = _rows(v, "v", shape, device)
    H = q_ptr = out_ptr = 0
    q_st = out_st = (0, 0, 0)
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be a tensor [B, H, N, d]")
        H = q.shape[1]
        _small(H)
        q_shape = (B, H, N, d)
        q_st = _rows(q, "q", q_shape, device)
        if q_out is None:
            q_out = torch.empty_like(q)
        out_st = _rows(q_out, "q_out", q_shape, device)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rotation = None
    if cos is not None:
        if sin is None or cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be fp32 tensors [n_angles, rot / 2]")
        for t in (cos, sin):
            if t.dtype is not _FP32 or t.get_device() != device or not t.is_contiguous():
                raise ValueError(f"cos and sin must be contiguous fp32 tensors on cuda:{device}")
        n_angles, pairs = cos.shape
        sections = (pairs,) if sections is None else tuple(sections)
        axes = len(sections)
        if not 1 <= axes <= 4:
            raise ValueError("sections must name 1 to 4 axes")
        if positions is None:
            if axes > 1:
                raise ValueError("several axes need positions")
            pos_ptr = 0
        else:
            pos_ptr = _ints(positions, "positions", (B, N) if axes == 1 and positions.dim() == 2 else (axes, B, N), device)
        rotation = _lib.ROTATION.pack(cos.data_ptr(), sin.data_ptr(), pos_ptr, 2 * pairs, n_angles, axes,
                                      bool(interleaved), *sections, *(0,) * (4 - axes))
    elif sin is not None or positions is not None or sections is not None:
        raise ValueError("a rotation needs cos and sin")
    _launch("fa_kv_append", device, q_ptr, k.data_ptr(), v.data_ptr(), out_ptr, cache,
            _ints(lengths, "lengths", (B,), device), 0 if counts is None else _ints(counts, "counts", (B,), device),
            rotation, B, H, H_kv, N, d, _lib.STRIDES4.pack(*q_st, *k_st, *v_st, *out_st))
    return q_out


def paged_workspace_size(B: int, H: int, H_kv: int, N_q: int, d: int) -> int:
    """Bytes of scratch device memory decode_paged() needs, whatever the lengths are."""
    _small(B, H, H_kv, N_q, d)
    n = _lib.fa_paged_workspace_size(B, H, H_kv, N_q, d)
    if n == 0:
        raise ValueError("invalid shape")
    return n


def _outputs(q, shape, device, out, lse, workspace, need):
    """Output tensors and scratch, allocated where not given, and out's strides."""
    if out is None:
        out = torch.empty_like(q)
    out_st = _rows(out, "out", shape, device)
    if lse is None:
        lse = torch.empty(shape[:3], dtype=_FP32, device=q.device)
    elif (lse.dtype is not _FP32 or lse.numel() != shape[0] * shape[1] * shape[2] or lse.get_device() != device
          or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous fp32 tensor {tuple(shape[:3])} on cuda:{device}")
    if workspace is None:
        workspace = torch.empty(need(), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return out, lse, workspace, out_st


def decode_paged(q, k_pages, v_pages, page_table, lengths, scale: float | None = None, causal: bool = False,
                 window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None, workspace=None,
                 counts=None):
    """O, L for N_q new query rows of each sequence over a paged cache (decode() with lengths of
    their own).

    q: bf16 [B, H, N_q, d]; row i of sequence b stands at position ``lengths[b] - N_q + i``, where
    the causal and window masks apply; with ``counts`` int32 [B], as given to the append, at
    ``lengths[b] - counts[b] + i``, and rows from counts[b] on are padding.  Padding, and rows without
    an allowed key (length 0, or a causal row before the first key), give O = 0 and L = -inf.  Returns O bf16 [B, H, N_q, d] and L fp32
    [B, H, N_q] (``out`` and ``lse`` if given; out may be q itself).
    """
    shape, device, q_st = _first(q, "q")
    B, H, N_q, d = shape
    cache, H_kv = _cache(k_pages, v_pages, page_table, B, d, device, k_scale, v_scale)
    out, lse, workspace, out_st = _outputs(q, shape, device, out, lse, workspace,
                                           lambda: paged_workspace_size(B, H, H_kv, N_q, d))
    _launch("fa_fwd_paged_ragged", device, q.data_ptr(), cache, _ints(lengths, "lengths", (B,), device),
            0 if counts is None else _ints(counts, "counts", (B,), device), out.data_ptr(), lse.data_ptr(), B, H, H_kv, N_q, d, _lib.STRIDES2.pack(*q_st, *out_st),
            1.0 / math.sqrt(d) if scale is None else float(scale), int(bool(causal)),
            max(-1, min(int(window), _INT_MAX)),   # (the library's ints have 32 bits)
            workspace.data_ptr(), workspace.nbytes)
    return out, lse


def shared_workspace_size(B: int, H: int, H_kv: int, N_q: int, d: int, prefix_length: int) -> int:
    """Bytes of scratch device memory decode_shared() needs, whatever the lengths are."""
    _small(B, H, H_kv, N_q, d, prefix_length)
    n = _lib.fa_shared_workspace_size(B, H, H_kv, N_q, d, prefix_length)
    if n == 0:
        raise ValueError("invalid shape")
    return n


def decode_shared(q, k_pages, v_pages, prefix_pages, prefix_length: int, page_table, lengths,
                  scale: float | None = None, causal: bool = False, k_scale: float = 1.0, v_scale: float = 1.0, out=None,
                  lse=None, workspace=None, counts=None):
    """decode_paged() for a batch whose sequences all begin with the same ``prefix_length`` keys, which
    lie in ``prefix_pages`` (int32 page numbers): their part is computed once for the whole batch.

    ``page_table`` and ``lengths`` describe each sequence's own keys, those after the prefix; every row
    attends the whole prefix and its own keys (up to itself with causal).  ``counts`` as in
    decode_paged().  Returns O and L of the
    prefix and the own keys together.
    """
    shape, device, q_st = _first(q, "q")
    B, H, N_q, d = shape
    cache, H_kv = _cache(k_pages, v_pages, page_table, B, d, device, k_scale, v_scale)
    prefix_length = _prefix_length(prefix_length, prefix_pages, k_pages.shape[2])
    pages = _ints(prefix_pages, "prefix_pages", prefix_pages.shape, device)
    out, lse, workspace, out_st = _outputs(
        q, shape, device, out, lse, workspace, lambda: shared_workspace_size(B, H, H_kv, N_q, d, prefix_length))
    _launch("fa_fwd_shared_ragged", device, q.data_ptr(), cache, pages, prefix_length,
            _ints(lengths, "lengths", (B,), device), 0 if counts is None else _ints(counts, "counts", (B,), device),
            out.data_ptr(), lse.data_ptr(), B, H, H_kv, N_q, d, _lib.STRIDES2.pack(*q_st, *out_st),
            1.0 / math.sqrt(d) if scale is None else float(scale), int(bool(causal)), workspace.data_ptr(),
            workspace.nbytes)
    return out, lse
