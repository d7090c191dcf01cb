"""Paged key-value caches: attention of new tokens, appending and page management.

The softmax-attention side of serving a model that mixes such layers with
gated-delta-rule layers; the calls stand beside `decode` and its state pool.
As in the rest of the binding, only arguments are marshalled here
(include/libgdn.h has the contracts) and there is no other implementation.

  attn_decode(q, k_cache, v_cache, page_table, lens, ...) -> out | (out, lse)
  kv_append(k, v, k_cache, v_cache, page_table, lens, ...) -> (k_cache, v_cache)
  pages_copy(pool, src, dst) -> pool
  pages_extend(page_table, lens, refs, add, page_size) -> (page_table, lens, refs, ok)
  pages_fork(page_table, lens, refs, parent, page_size) -> (page_table, lens, refs, src, dst)
  pages_free(page_table, lens, refs, rows, page_size) -> (page_table, lens, refs)
  pages_compact(page_table, refs) -> (page_table, refs, src, dst, n_live)
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

_I32_MIN, _I32_MAX = -(1 << 31), (1 << 31) - 1
_IO = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}
_CACHE = {**_IO, torch.float8_e4m3fn: _lib.GDN_E4M3}
_here = contextlib.nullcontext()


def _on(stream, dev, *tensors):
    """Where a call on tensors of `dev` runs: all of them checked to be there,
    and the device and stream made current, so that memory allocated for the
    call belongs to the stream that uses it."""
    if dev.type != "cuda":
        raise ValueError("GPU tensors are required (libgdn has no CPU path)")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one GPU (%s and %s)" % (dev, t.device))
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, dev))
        return torch.cuda.stream(stream)
    return _here if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _i32(t, name, shape, outside=None):
    """An int32 view or copy of a whole-number tensor.  int64 values outside
    the int32 range become `outside`, or are clamped where it is None."""
    if tuple(t.shape) != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if t.dtype != torch.int32:
        if t.dtype != torch.int64:
            raise ValueError("%s must be int32 or int64" % name)
        if outside is None:
            t = t.clamp(_I32_MIN, _I32_MAX).to(torch.int32)
        else:
            t = torch.where((t < _I32_MIN) | (t > _I32_MAX), outside, t).to(torch.int32)
    return t if t.is_contiguous() else t.contiguous()


def _table(t, rows):
    """A page table as int32 rows with a dense last dimension: (table, row stride)."""
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError("page_table must be [%d, max_pages], got %s" % (rows, tuple(t.shape)))
    if t.dtype != torch.int32 or (t.stride(1) != 1 and t.shape[1] > 1) or (t.stride(0) < t.shape[1] and rows > 1):
        t = _i32(t, "page_table", tuple(t.shape), -1)
    return t, max(t.stride(0), t.shape[1])


def _cache_strides(c, name):
    """Page, token and head strides of a [n_pages, page_size, hkv, d] cache;
    dimensions of one entry get their dense stride."""
    n, page, heads, d = c.shape
    sp, st, sh, sd = c.stride()
    if sd != 1:
        raise ValueError("%s must have a dense last dimension" % name)
    if heads == 1:
        sh = d
    if page == 1:
        st = (heads - 1) * sh + d
    if n == 1:
        sp = (page - 1) * st + (heads - 1) * sh + d
        sp += -sp % 16
    return sp, st, sh


def _caches(io, k_cache, v_cache, k_scale, v_scale, hkv, d):
    """Checks of a key and a value cache and their scales; the cache type's code."""
    if k_cache.dim() != 4 or k_cache.shape[2:] != (hkv, d):
        raise ValueError("k_cache must be [n_pages, page_size, %d, %d], got %s" % (hkv, d, tuple(k_cache.shape)))
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must share shape and dtype")
    if k_cache.shape[1] < 1:
        raise ValueError("page_size must be at least 1")
    if k_cache.dtype != io and k_cache.dtype != torch.float8_e4m3fn:
        raise ValueError("the caches must have the inputs' dtype or float8_e4m3fn, got %s" % k_cache.dtype)
    if k_cache.dtype == torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("float8_e4m3fn caches need k_scale and v_scale")
        k_scale, v_scale = _scale(k_scale, "k_scale", hkv), _scale(v_scale, "v_scale", hkv)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are for float8_e4m3fn caches")
    return _CACHE[k_cache.dtype], k_scale, v_scale


def _scale(t, name, hkv):
    if tuple(t.shape) != (hkv,) or t.dtype != torch.float32:
        raise ValueError("%s must be [%d] float32" % (name, hkv))
    return t if t.is_contiguous() else t.contiguous()


def _rows16(t, name):
    """t as it is where the kernels can read it in place (dense last dimension,
    strides and base multiples of 16 bytes), else a dense copy."""
    unit = 16 // t.element_size()
    s = t.stride()
    if s[-1] != 1 or t.data_ptr() % 16 or any(x % unit or x < 0 for x in s[:-1]):
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def attn_decode_args(q, k_cache, v_cache, page_table, lens, *, scale=None, k_scale=None, v_scale=None,
                     out=None, lse=None):
    """Validate shapes and build the gdn_attn_decode_args struct (device-agnostic).

    Returns (args, keep, out): `keep` holds every tensor whose pointer is in
    args (converted copies included)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, hq, d]")
    if q.dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % q.dtype)
    B, T, hq, d = q.shape
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [n_pages, page_size, hkv, d]")
    n_pages, page, hkv, _ = k_cache.shape
    cache_dtype, k_scale, v_scale = _caches(q.dtype, k_cache, v_cache, k_scale, v_scale, hkv, d)
    q = _rows16(q, "q")
    table, table_stride = _table(page_table, B)
    lens = _i32(lens, "lens", (B,))
    if out is None:
        out = torch.empty((B, T, hq, d), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.data_ptr() % 16:
        raise ValueError("out must be contiguous, 16-byte aligned, with q's shape and dtype")
    if lse is not None and (tuple(lse.shape) != (B, T, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [B, T, hq]")
    a = _lib.AttnDecodeArgs()
    a.batch, a.T, a.hq, a.hkv, a.d = B, T, hq, hkv, d
    a.io_dtype, a.cache_dtype = _IO[q.dtype], cache_dtype
    a.scale = d ** -0.5 if scale is None else float(scale)
    a.q, (a.q_stride_row, a.q_stride_token, a.q_stride_head, _) = q.data_ptr(), q.stride()
    a.k_cache, (a.k_stride_page, a.k_stride_token, a.k_stride_head) = k_cache.data_ptr(), _cache_strides(k_cache, "k_cache")
    a.v_cache, (a.v_stride_page, a.v_stride_token, a.v_stride_head) = v_cache.data_ptr(), _cache_strides(v_cache, "v_cache")
    a.n_pages, a.page_size, a.max_pages = n_pages, page, table.shape[1]
    a.page_table, a.page_table_stride, a.lens = table.data_ptr(), table_stride, lens.data_ptr()
    a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
    a.out, a.lse = out.data_ptr(), _ptr(lse)
    return a, (q, table, lens, k_scale, v_scale), out


def attn_decode(q, k_cache, v_cache, page_table, lens, *, scale=None, k_scale=None, v_scale=None, out=None,
                return_lse=False, workspace=None, stream=None):
    """Softmax attention of each row's newest T tokens over a paged cache.

    q [B, T, hq, d] float32 or bfloat16, 1 <= T <= 64, d in {32, 64, 128, 256};
    k_cache, v_cache [n_pages, page_size, hkv, d] in q's dtype or float8_e4m3fn
    (then with k_scale, v_scale [hkv] float32, the factors of the stored
    values), any page_size, and with heads before tokens in memory where the
    tensor is such a view; page_table [B, max_pages], lens [B] int32 or int64.
    The cache holds the new tokens already (kv_append): token t of row b is
    position lens[b] - T + t and sees the positions up to its own.  Query head
    h reads key-value head h*hkv//hq.  scale None means 1/sqrt(d).

    Rows or tokens that see nothing (lens 0, table entries outside the cache)
    get zeros and lse -inf.  Rows may share pages.  return_lse: also return
    log sum exp of the scores, [B, T, hq] float32, to join the result with
    attention over other keys.  workspace: a uint8 CUDA tensor of at least
    attn_decode_workspace_size bytes for the split over the rows' lengths;
    None allocates one.  Returns out [B, T, hq, d] in q's dtype.
    """
    with _on(stream, q.device, k_cache, v_cache, page_table, lens, k_scale, v_scale, out, workspace):
        lib = _lib.load()
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if return_lse else None
        a, keep, out = attn_decode_args(q, k_cache, v_cache, page_table, lens, scale=scale, k_scale=k_scale,
                                        v_scale=v_scale, out=out, lse=lse)
        need = lib.gdn_attn_decode_workspace_size(ctypes.byref(a))
        if need > 0:
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            elif workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous buffer of at least %d bytes" % need)
            a.workspace, a.workspace_bytes = workspace.data_ptr(), need
        _lib.check(lib.gdn_attn_decode(ctypes.byref(a), _stream()))
        del keep
    return (out, lse) if return_lse else out


def attn_decode_workspace_size(q, k_cache, v_cache, page_table, lens, **kw) -> int:
    """Bytes of device workspace that an attn_decode call with these arguments
    would use (gdn_attn_decode_workspace_size); the values of lens do not matter."""
    a, keep, _ = attn_decode_args(q, k_cache, v_cache, page_table, lens, **kw)
    return int(_lib.load().gdn_attn_decode_workspace_size(ctypes.byref(a)))


def kv_append_args(k, v, k_cache, v_cache, page_table, lens, *, cu_seqlens=None, k_scale=None, v_scale=None):
    """Validate shapes and build the gdn_kv_append_args struct (device-agnostic):
    returns (args, tensors to keep alive)."""
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must share shape and dtype")
    if k.dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % k.dtype)
    B = lens.shape[0] if lens.dim() == 1 else -1
    if B < 0:
        raise ValueError("lens must be [B]")
    if cu_seqlens is None:
        if k.dim() != 4 or k.shape[0] != B:
            raise ValueError("k and v must be [B, T, hkv, d] ([tokens, hkv, d] with cu_seqlens)")
        k, v = (x.reshape(x.shape[0] * x.shape[1], *x.shape[2:]) for x in (k, v))
    else:
        if k.dim() != 3:
            raise ValueError("with cu_seqlens k and v must be [tokens, hkv, d]")
        cu_seqlens = _i32(cu_seqlens, "cu_seqlens", (B + 1,))
    total, hkv, d = k.shape
    cache_dtype, k_scale, v_scale = _caches(k.dtype, k_cache, v_cache, k_scale, v_scale, hkv, d)
    k, v = _rows16(k, "k"), _rows16(v, "v")
    table, table_stride = _table(page_table, B)
    lens = _i32(lens, "lens", (B,))
    a = _lib.KvAppendArgs()
    a.total_tokens, a.batch, a.hkv, a.d = total, B, hkv, d
    a.io_dtype, a.cache_dtype = _IO[k.dtype], cache_dtype
    a.k, (a.k_stride_token, a.k_stride_head, _) = k.data_ptr(), k.stride()
    a.v, (a.v_stride_token, a.v_stride_head, _) = v.data_ptr(), v.stride()
    a.cu_seqlens = _ptr(cu_seqlens)
    a.k_cache, (a.kc_stride_page, a.kc_stride_token, a.kc_stride_head) = k_cache.data_ptr(), _cache_strides(k_cache, "k_cache")
    a.v_cache, (a.vc_stride_page, a.vc_stride_token, a.vc_stride_head) = v_cache.data_ptr(), _cache_strides(v_cache, "v_cache")
    a.n_pages, a.page_size, a.max_pages = k_cache.shape[0], k_cache.shape[1], table.shape[1]
    a.page_table, a.page_table_stride, a.lens = table.data_ptr(), table_stride, lens.data_ptr()
    a.k_scale, a.v_scale = _ptr(k_scale), _ptr(v_scale)
    return a, (k, v, cu_seqlens, table, lens, k_scale, v_scale)


def kv_append(k, v, k_cache, v_cache, page_table, lens, *, cu_seqlens=None, k_scale=None, v_scale=None,
              stream=None):
    """Write new tokens' keys and values into their pages (the caches are
    updated in place).

    k, v: [B, T, hkv, d], T new tokens for every row, or with cu_seqlens
    [B + 1] packed [tokens, hkv, d].  lens [B] counts the new tokens already:
    row b's n tokens go to positions lens[b] - n .. lens[b] - 1 of its pages;
    tokens whose position lies outside the table or whose table entry is
    outside the cache are not written.  Caches, page_table and scales as for
    attn_decode; a float8_e4m3fn cache stores x / scale rounded to nearest
    even and clamped to +-448.  Returns (k_cache, v_cache).
    """
    with _on(stream, k.device, v, k_cache, v_cache, page_table, lens, cu_seqlens, k_scale, v_scale):
        a, keep = kv_append_args(k, v, k_cache, v_cache, page_table, lens, cu_seqlens=cu_seqlens,
                                 k_scale=k_scale, v_scale=v_scale)
        _lib.check(_lib.load().gdn_kv_append(ctypes.byref(a), _stream()))
        del keep
    return k_cache, v_cache


def _page_block(pool):
    """(bytes of a page, bytes from page to page) of a pool [n_pages, ...] whose
    pages are dense blocks, their inner dimensions in any order."""
    if pool.dim() < 1:
        raise ValueError("pool must be [n_pages, ...]")
    inner = 1
    for stride, size in sorted((st, sz) for st, sz in zip(pool.stride()[1:], pool.shape[1:]) if sz != 1):
        if stride != inner:
            raise ValueError("each page of the pool must be one dense block")
        inner *= size
    es = pool.element_size()
    return inner * es, (pool.stride(0) if pool.shape[0] > 1 else inner) * es


def pages_copy(pool, src, dst, *, stream=None):
    """Copy whole pages inside a pool: page dst[i] becomes page src[i].

    pool: any [n_pages, ...] tensor whose pages are dense blocks -- a key or
    value cache, `decode`'s state pool, `conv1d`'s conv_state -- updated in
    place.  src, dst: [n] int32 or int64; pairs with an entry outside
    [0, n_pages) are skipped.  A page that one pair writes and another reads
    or writes is undefined.  Returns pool.
    """
    with _on(stream, pool.device, src, dst):
        nbytes, stride = _page_block(pool)
        n = src.shape[0] if src.dim() == 1 else -1
        if n < 0:
            raise ValueError("src must be [n]")
        src, dst = _i32(src, "src", (n,), -1), _i32(dst, "dst", (n,), -1)
        _lib.check(_lib.load().gdn_pages_copy(pool.data_ptr(), nbytes, stride, pool.shape[0], src.data_ptr(),
                                              dst.data_ptr(), n, _stream()))
    return pool


def pages_args(page_table, lens, refs, page_size, out=None, apart=False, workspace=True):
    """Validate shapes and build the gdn_pages_args struct (device-agnostic):
    returns (args, tensors to keep alive, (page_table, lens, refs) outputs).
    lens None: a call that has no lengths.  apart: the outputs may not be the
    inputs."""
    if page_table.dim() != 2 or page_table.shape[1] < 1:
        raise ValueError("page_table must be [rows, max_pages]")
    if refs.dim() != 1 or refs.shape[0] < 1:
        raise ValueError("refs must be [n_pages]")
    rows, width = page_table.shape
    n = refs.shape[0]
    table, table_stride = _table(page_table, rows)
    refs_in = _i32(refs, "refs", (n,))
    lens_in = None if lens is None else _i32(lens, "lens", (rows,))
    dev = page_table.device
    if out is None:
        to = torch.empty((rows, width), dtype=torch.int32, device=dev)
        lens_to = None if lens is None else torch.empty(rows, dtype=torch.int32, device=dev)
        refs_to = torch.empty(n, dtype=torch.int32, device=dev)
    else:
        to, refs_to = out[0], out[-1]
        lens_to = None if lens is None else out[1]
        for name, t, shape in (("page_table", to, (rows, width)), ("lens", lens_to, (rows,)), ("refs", refs_to, (n,))):
            if t is None:
                continue
            if tuple(t.shape) != shape or t.dtype != torch.int32 or t.device != dev:
                raise ValueError("out's %s must be int32 %s on the inputs' device" % (name, shape))
            if (t.stride(-1) != 1 and t.shape[-1] > 1) or (t.dim() == 2 and rows > 1 and t.stride(0) < width):
                raise ValueError("out's %s must have dense rows" % name)
            given = {"page_table": table, "lens": lens_in, "refs": refs_in}[name]
            same = t.data_ptr() == given.data_ptr() and (t.dim() == 1 or rows == 1 or t.stride(0) == table_stride)
            if _overlap(t, given) and (apart and name != "refs" or not same):
                raise ValueError("out's %s overlaps the input" % name)
    a = _lib.PagesArgs()
    a.rows, a.max_pages, a.n_pages, a.page_size = rows, width, n, int(page_size)
    a.page_table, a.page_table_stride, a.lens, a.refs = table.data_ptr(), table_stride, _ptr(lens_in), refs_in.data_ptr()
    a.page_table_out, a.page_table_out_stride = to.data_ptr(), max(to.stride(0), width)
    a.lens_out, a.refs_out = _ptr(lens_to), refs_to.data_ptr()
    ws = None
    if workspace:
        need = _lib.load().gdn_pages_workspace_size(rows, n)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
    return a, (table, lens_in, refs_in, ws), (to, lens_to, refs_to)


def _overlap(a, b):
    """Whether the memory that two tensors span overlaps."""
    def span(t):
        last = sum((sz - 1) * st for sz, st in zip(t.shape, t.stride())) if t.numel() else -1
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def pages_extend(page_table, lens, refs, add, page_size, *, out=None, stream=None):
    """Grow the rows of a page table by add [rows] tokens, on the device.

    page_table [rows, max_pages], lens [rows], refs [n_pages] (holders of each
    page, 0: free), int32 or int64.  Each row takes the pages it needs from the
    lowest free ones, rows in order; a row is served if its new length fits
    the table and the pages that it and the rows before it need are free (a
    row that needs none always is), others stay as they are.  out: (page_table,
    lens, refs) int32 tensors to write to, which may be the inputs themselves;
    new ones when None.  Returns (page_table, lens, refs, ok [rows] int32).
    """
    with _on(stream, page_table.device, lens, refs, add):
        a, keep, (table, lens_to, refs_to) = pages_args(page_table, lens, refs, page_size, out)
        add = _i32(add, "add", (a.rows,))
        ok = torch.empty(a.rows, dtype=torch.int32, device=add.device)
        _lib.check(_lib.load().gdn_pages_extend(ctypes.byref(a), add.data_ptr(), ok.data_ptr(), _stream()))
        del keep
    return table, lens_to, refs_to, ok


def pages_fork(page_table, lens, refs, parent, page_size, *, out=None, stream=None):
    """Rearrange the rows of a page table: row r becomes what row parent[r] was.

    Rows keep (parent[r] == r), fork (several rows of one parent share its
    pages) or end (parent[r] outside [0, rows): the row is empty and its pages
    are released); all rows read the table as it was.  A part-filled last page
    that others hold too gets its own copy: src[r] is the shared page and
    dst[r] the fresh one, for pages_copy on each cache (-1 where there is
    none; the lowest row keeps a page that every holder has as its part-filled
    last one).  A row for which no page is left ends empty.  out: (page_table,
    lens, refs) int32 tensors; page_table and lens may not be the inputs.
    Returns (page_table, lens, refs, src [rows], dst [rows]).
    """
    with _on(stream, page_table.device, lens, refs, parent):
        a, keep, (table, lens_to, refs_to) = pages_args(page_table, lens, refs, page_size, out, apart=True)
        parent = _i32(parent, "parent", (a.rows,), -1)
        src, dst = torch.empty((2, a.rows), dtype=torch.int32, device=parent.device)
        _lib.check(_lib.load().gdn_pages_fork(ctypes.byref(a), parent.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                              _stream()))
        del keep
    return table, lens_to, refs_to, src, dst


def pages_free(page_table, lens, refs, rows, page_size, *, out=None, stream=None):
    """Release the pages of the rows where rows [n_rows] (bool or uint8) is set:
    they end empty, their table entries -1.  out as in pages_extend.  Returns
    (page_table, lens, refs)."""
    with _on(stream, page_table.device, lens, refs, rows):
        a, keep, to = pages_args(page_table, lens, refs, page_size, out, workspace=False)
        if tuple(rows.shape) != (a.rows,) or rows.dtype not in (torch.bool, torch.uint8):
            raise ValueError("rows must be bool or uint8 [%d]" % a.rows)
        rows = rows.contiguous()
        _lib.check(_lib.load().gdn_pages_free(ctypes.byref(a), rows.data_ptr(), _stream()))
        del keep
    return to


def pages_compact(page_table, refs, *, out=None, stream=None):
    """Move the pages in use to the lowest page numbers, in the table and refs.

    The i-th page in use at or above n_live (the number in use) moves to the
    i-th free page below it; src, dst [n_pages // 2] list the moves for
    pages_copy on each cache (no page is both; -1 past the last).  out:
    (page_table, refs) int32 tensors to write to, which may be the inputs.
    Returns (page_table, refs, src, dst, n_live [1]).
    """
    with _on(stream, page_table.device, refs):
        a, keep, (table, _, refs_to) = pages_args(page_table, None, refs, 1, out)
        src, dst = torch.empty((2, a.n_pages // 2), dtype=torch.int32, device=refs.device)
        n_live = torch.empty(1, dtype=torch.int32, device=refs.device)
        _lib.check(_lib.load().gdn_pages_compact(ctypes.byref(a), src.data_ptr(), dst.data_ptr(), n_live.data_ptr(),
                                                 _stream()))
        del keep
    return table, refs_to, src, dst, n_live
