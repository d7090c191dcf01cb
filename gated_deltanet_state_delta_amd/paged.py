"""Paged key-value caches: attention of new tokens, appending and page management.

The softmax-attention side of serving a model that mixes such layers with
gated-delta-rule layers; the calls stand beside `decode` and its state pool.
As in the rest of the binding, only arguments are marshalled here
(include/libgdn.h has the contracts) and there is no other implementation.

  attn_decode(q, k_cache, v_cache, page_table, lens, ...) -> out | (out, lse)
  kv_append(k, v, k_cache, v_cache, page_table, lens, ...) -> (k_cache, v_cache)
  kv_read(k_cache, v_cache, page_table, lens, tokens, ...) -> (k, v)
  pages_copy(pool, src, dst) -> pool
  pages_extend(page_table, lens, refs, add, page_size) -> (page_table, lens, refs, ok)
  pages_fork(page_table, lens, refs, parent, page_size) -> (page_table, lens, refs, src, dst)
  pages_free(page_table, lens, refs, rows, page_size) -> (page_table, lens, refs)
  pages_compact(page_table, refs) -> (page_table, refs, src, dst, n_live)
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import _lib

_I32_MIN, _I32_MAX = -(1 << 31), (1 << 31) - 1
_IO = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}
_CACHE = {**_IO, torch.float8_e4m3fn: _lib.GDN_E4M3, torch.int8: _lib.GDN_I8}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _short(name, *args):
    """The call by the short way (binding/calls.cpp) on the current device and
    stream, or None where it is not an ordinary one or the module is not there."""
    module = _lib._calls or _lib.short_way()
    if module is None:
        return None
    dev = _current_device()
    return getattr(module, name)(*args, dev, _raw_stream(dev))


def _on(stream, dev, tensors):
    """Where a call on tensors of `dev` runs: checks that all of them are there
    and returns the context that makes the device and stream current (None:
    they are), so that memory allocated for the call belongs to its stream."""
    at = dev.index
    if dev.type != "cuda":
        raise ValueError("GPU tensors are required (libgdn has no CPU path)")
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError("all tensors must be on one GPU (%s and %s)" % (dev, t.device))
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, dev))
        return torch.cuda.stream(stream)
    return None if at == torch.cuda.current_device() else torch.cuda.device(dev)


def _checked(status):
    if status:
        _lib.check(status)


def _library():
    return _lib._lib or _lib.load()


def _i32(t, name, shape, outside=None):
    """An int32 view or copy of a whole-number tensor.  int64 values outside
    the int32 range become `outside`, or are clamped where it is None."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if t.dtype is not torch.int32:
        if t.dtype != torch.int64:
            raise ValueError("%s must be int32 or int64" % name)
        if outside is None:
            t = t.clamp(_I32_MIN, _I32_MAX).to(torch.int32)
        else:
            t = torch.where((t < _I32_MIN) | (t > _I32_MAX), outside, t).to(torch.int32)
    return t if t.is_contiguous() else t.contiguous()


def _table(t, rows):
    """A page table as int32 rows with a dense last dimension: (table, row
    stride, entries of a row)."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError("page_table must be [%d, max_pages], got %s" % (rows, tuple(shape)))
    width = shape[1]
    if t.dtype is torch.int32:
        st, s1 = t.stride()
        if (s1 == 1 or width == 1) and (st >= width or rows == 1):
            return t, (st if st > width else width), width
    return _i32(t, "page_table", tuple(shape), -1), width, width


def _cache_strides(c, shape, name):
    """Page, token and head strides of a [n_pages, page_size, hkv, d] cache;
    dimensions of one entry get their dense stride."""
    n, page, heads, d = shape
    sp, st, sh, sd = c.stride()
    if sd != 1:
        raise ValueError("%s must have a dense last dimension" % name)
    if heads == 1:
        sh = d
    if page == 1:
        st = d
    if n == 1:
        sp = (page - 1) * st + (heads - 1) * sh + d
        sp += -sp % 16
    return sp, st, sh


def _caches(io, k_cache, v_cache, shape, k_scale, v_scale, hkv, d):
    """Checks of a key and a value cache and their scales: (the cache type's
    code, the factors a head (k_scale, v_scale), the block scales (tokens of a
    block, k_scale, v_scale), the K and V strides)."""
    if len(shape) != 4 or shape[2] != hkv or shape[3] != d:
        raise ValueError("k_cache must be [n_pages, page_size, %d, %d], got %s" % (hkv, d, tuple(shape)))
    dtype = k_cache.dtype
    if v_cache.shape != shape or v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must share shape and dtype")
    if shape[1] < 1:
        raise ValueError("page_size must be at least 1")
    blocks = (0, None, None)
    if dtype is torch.float8_e4m3fn or dtype is torch.int8:
        if k_scale is None or v_scale is None:
            raise ValueError("%s caches need k_scale and v_scale" % dtype)
        if k_scale.dim() == 3 or v_scale.dim() == 3 or dtype is torch.int8:
            blocks = (_block_scales(k_scale, v_scale, shape), k_scale, v_scale)
            k_scale = v_scale = None
        else:
            k_scale, v_scale = _scale(k_scale, "k_scale", hkv), _scale(v_scale, "v_scale", hkv)
    elif dtype is not io:
        raise ValueError("the caches must have the inputs' dtype, float8_e4m3fn or int8, got %s" % dtype)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are for 8-bit caches")
    ks = _cache_strides(k_cache, shape, "k_cache")
    vs = _cache_strides(v_cache, shape, "v_cache")
    return _CACHE[dtype], (k_scale, v_scale), blocks, ks, vs


def _scale(t, name, hkv):
    if t.shape != (hkv,) or t.dtype != torch.float32:
        raise ValueError("%s must be [%d] float32" % (name, hkv))
    return t if t.is_contiguous() else t.contiguous()


def _block_scales(k_scale, v_scale, shape):
    """Tokens of a block of the block scales of a cache of this shape."""
    n_pages, page, hkv, _ = shape
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if (t.dim() != 3 or t.shape[0] != n_pages or t.shape[1] != hkv or t.shape[2] < 1 or page % t.shape[2]
                or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError("%s must be contiguous float32 [%d, %d, blocks], blocks dividing page_size %d, got %s %s"
                             % (name, n_pages, hkv, page, t.dtype, tuple(t.shape)))
    if k_scale.shape != v_scale.shape:
        raise ValueError("k_scale and v_scale must share their shape")
    return page // k_scale.shape[2]


def _rows16(t):
    """t as it is where the kernels can read it in place (dense last dimension,
    strides and base multiples of 16 bytes), else a dense copy."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0 and t.shape[-1] % 8 == 0:
        return t
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
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError("q must be [B, T, hq, d]")
    if dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    B, T, hq, d = shape
    cs = k_cache.shape
    if len(cs) != 4:
        raise ValueError("k_cache must be [n_pages, page_size, hkv, d]")
    n_pages, page, hkv, _ = cs
    cache_dtype, factors, blocks, ks, vs = _caches(dtype, k_cache, v_cache, cs, k_scale, v_scale, hkv, d)
    q = _rows16(q)
    table, table_stride, max_pages = _table(page_table, B)
    lens = _i32(lens, "lens", (B,))
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(shape)
    elif out.shape != shape or out.dtype is not dtype or not out.is_contiguous() or out.data_ptr() % 16:
        raise ValueError("out must be contiguous, 16-byte aligned, with q's shape and dtype")
    if lse is not None and (lse.shape != (B, T, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [B, T, hq]")
    # a contiguous tensor's dimensions of one entry may carry any stride
    qs = (T * hq * d, hq * d, d) if q.is_contiguous() else q.stride()
    a = _lib.AttnDecodeArgs(
        B, T, hq, hkv, d, _IO[dtype], cache_dtype, d ** -0.5 if scale is None else float(scale),
        q.data_ptr(), qs[0], qs[1], qs[2], k_cache.data_ptr(), *ks, v_cache.data_ptr(), *vs,
        n_pages, page, max_pages, table.data_ptr(), table_stride, lens.data_ptr(), _ptr(factors[0]), _ptr(factors[1]),
        out.data_ptr(), _ptr(lse), None, 0, blocks[0], _ptr(blocks[1]), _ptr(blocks[2]))
    return a, (q, table, lens, factors, blocks), out


def attn_decode(q, k_cache, v_cache, page_table, lens, *, scale=None, k_scale=None, v_scale=None, out=None,
                return_lse=False, workspace=None, stream=None):
    """Softmax attention of each row's newest T tokens over a paged cache.

    q [B, T, hq, d] float32 or bfloat16, 1 <= T <= 64, d in {32, 64, 128, 256};
    k_cache, v_cache [n_pages, page_size, hkv, d] in q's dtype, float8_e4m3fn
    or int8, any page_size, and with heads before tokens in memory where the
    tensor is such a view.  8-bit caches come with k_scale, v_scale float32, the
    factors of the stored values: [n_pages, hkv, blocks], one for each block of
    page_size / blocks tokens (at most 65536) and head, as kv_append sets them,
    or for float8_e4m3fn [hkv], one for each head.  page_table [B, max_pages], lens [B] int32 or int64.
    The cache holds the new tokens already (kv_append): token t of row b is
    position lens[b] - T + t and sees the positions up to its own.  Query head
    h reads key-value head h*hkv//hq.  scale None means 1/sqrt(d).

    Rows or tokens that see nothing (lens 0, table entries outside the cache),
    or whose scores are all -inf, get zeros and lse -inf; NaN in a query or in a
    key that it sees gives NaN.  Rows may share pages.  return_lse: also return
    log sum exp of the scores, [B, T, hq] float32, to join the result with
    attention over other keys.  workspace: a uint8 CUDA tensor of at least
    attn_decode_workspace_size bytes for the split over the rows' lengths;
    None allocates one.  Returns out [B, T, hq, d] in q's dtype.
    """
    if out is None and workspace is None and stream is None and not return_lse and q.is_cuda:
        got = _short("attn_decode", q, k_cache, v_cache, page_table, lens, scale, k_scale, v_scale)
        if got is not None:
            return got
    dev = q.device
    ctx = _on(stream, dev, (k_cache, v_cache, page_table, lens, k_scale, v_scale, out, workspace))
    if ctx is not None:
        with ctx:
            return attn_decode(q, k_cache, v_cache, page_table, lens, scale=scale, k_scale=k_scale, v_scale=v_scale,
                               out=out, return_lse=return_lse, workspace=workspace)
    lib = _library()
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if return_lse else None
    a, keep, out = attn_decode_args(q, k_cache, v_cache, page_table, lens, scale=scale, k_scale=k_scale,
                                    v_scale=v_scale, out=out, lse=lse)
    need = lib.gdn_attn_decode_workspace_size(byref(a))
    if need > 0:
        if workspace is None:
            workspace = q.new_empty(need // q.element_size())  # (a multiple of 4 bytes)
        elif workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous buffer of at least %d bytes" % need)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need
    _checked(lib.gdn_attn_decode(byref(a), _raw_stream(dev.index)))
    del keep
    return (out, lse) if return_lse else out


def attn_decode_workspace_size(q, k_cache, v_cache, page_table, lens, **kw) -> int:
    """Bytes of device workspace that an attn_decode call with these arguments
    would use (gdn_attn_decode_workspace_size); the values of lens do not matter."""
    a, keep, _ = attn_decode_args(q, k_cache, v_cache, page_table, lens, **kw)
    return int(_library().gdn_attn_decode_workspace_size(byref(a)))


def _tokens(x, shape):
    """[B, T, hkv, d] as rows of tokens one stride apart: x itself where it is dense."""
    if x.is_contiguous():
        return x
    return x.reshape(shape[0] * shape[1], shape[2], shape[3])


def _token_strides(x, hkv, d):
    """Token and head strides of what _tokens gives.  A contiguous tensor's
    dimensions of one entry may carry any stride (a step of a sequence-first
    buffer: T's is that of the steps), so its strides are taken from its shape."""
    return (hkv * d, d) if x.is_contiguous() else x.stride()[-3:-1]


def kv_append_args(k, v, k_cache, v_cache, page_table, lens, *, cu_seqlens=None, k_scale=None, v_scale=None):
    """Validate shapes and build the gdn_kv_append_args struct (device-agnostic):
    returns (args, tensors to keep alive)."""
    shape, dtype = k.shape, k.dtype
    if v.shape != shape or v.dtype is not dtype:
        raise ValueError("k and v must share shape and dtype")
    if dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    if lens.dim() != 1:
        raise ValueError("lens must be [B]")
    B = lens.shape[0]
    if cu_seqlens is None:
        if len(shape) != 4 or shape[0] != B:
            raise ValueError("k and v must be [B, T, hkv, d] ([tokens, hkv, d] with cu_seqlens)")
        total, hkv, d = B * shape[1], shape[2], shape[3]
        k, v = _tokens(k, shape), _tokens(v, shape)
    else:
        if len(shape) != 3:
            raise ValueError("with cu_seqlens k and v must be [tokens, hkv, d]")
        total, hkv, d = shape
        cu_seqlens = _i32(cu_seqlens, "cu_seqlens", (B + 1,))
    cs = k_cache.shape
    cache_dtype, factors, blocks, kcs, vcs = _caches(dtype, k_cache, v_cache, cs, k_scale, v_scale, hkv, d)
    k, v = _rows16(k), _rows16(v)
    table, table_stride, max_pages = _table(page_table, B)
    lens = _i32(lens, "lens", (B,))
    a = _lib.KvAppendArgs(
        total, B, hkv, d, _IO[dtype], cache_dtype, k.data_ptr(), *_token_strides(k, hkv, d),
        v.data_ptr(), *_token_strides(v, hkv, d),
        _ptr(cu_seqlens), k_cache.data_ptr(), *kcs, v_cache.data_ptr(), *vcs, cs[0], cs[1], max_pages,
        table.data_ptr(), table_stride, lens.data_ptr(), _ptr(factors[0]), _ptr(factors[1]), blocks[0], _ptr(blocks[1]),
        _ptr(blocks[2]))
    return a, (k, v, cu_seqlens, table, lens, factors, blocks)


def kv_append(k, v, k_cache, v_cache, page_table, lens, *, cu_seqlens=None, k_scale=None, v_scale=None,
              stream=None):
    """Write new tokens' keys and values into their pages (the caches are
    updated in place).

    k, v: [B, T, hkv, d], T new tokens for every row, or with non-decreasing
    cu_seqlens [B + 1] packed [tokens, hkv, d].  lens [B] counts the new tokens already:
    row b's n tokens go to positions lens[b] - n .. lens[b] - 1 of its pages;
    tokens whose position lies outside the table or whose table entry is
    outside the cache are not written.  Caches, page_table and scales as for
    attn_decode; an 8-bit cache stores x / scale rounded to nearest even and
    clamped to +-448 (float8_e4m3fn) or +-127 (int8).

    Block scales ([n_pages, hkv, blocks]) are updated in place: with a the
    largest finite |x| of a block's new tokens and head, its scale becomes the
    smallest power of two with a <= 448 scale (float8_e4m3fn) or a / 127 (int8),
    not below 2^-126 and, where the row has older tokens in the block, not below
    what it was; older tokens' codes are rounded again where it grew.  The first
    slot of a block starts it anew, so pages need no clearing.  NaN in a token
    makes the scale of an int8 block NaN.  Returns (k_cache, v_cache).
    """
    if stream is None and k.is_cuda:
        if _short("kv_append", k, v, k_cache, v_cache, page_table, lens, cu_seqlens, k_scale, v_scale):
            return k_cache, v_cache
    dev = k.device
    ctx = _on(stream, dev, (v, k_cache, v_cache, page_table, lens, cu_seqlens, k_scale, v_scale))
    if ctx is not None:
        with ctx:
            return kv_append(k, v, k_cache, v_cache, page_table, lens, cu_seqlens=cu_seqlens, k_scale=k_scale,
                             v_scale=v_scale)
    a, keep = kv_append_args(k, v, k_cache, v_cache, page_table, lens, cu_seqlens=cu_seqlens, k_scale=k_scale,
                             v_scale=v_scale)
    _checked(_library().gdn_kv_append(byref(a), _raw_stream(dev.index)))
    del keep
    return k_cache, v_cache


def kv_read_args(k_cache, v_cache, page_table, lens, tokens, *, cu_seqlens=None, dtype=None, k_scale=None,
                 v_scale=None, out=None):
    """Validate shapes and build the gdn_kv_read_args struct (device-agnostic):
    returns (args, tensors to keep alive, (k, v))."""
    cs = k_cache.shape
    if len(cs) != 4:
        raise ValueError("k_cache must be [n_pages, page_size, hkv, d]")
    n_pages, page, hkv, d = cs
    if lens.dim() != 1:
        raise ValueError("lens must be [B]")
    B = lens.shape[0]
    if int(tokens) != tokens or tokens < 0:
        raise ValueError("tokens must be a whole number of at least 0, got %s" % (tokens,))
    tokens = int(tokens)
    if dtype is None:
        dtype = out[0].dtype if out else k_cache.dtype if k_cache.dtype in _IO else torch.bfloat16
    if dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    cache_dtype, factors, blocks, kcs, vcs = _caches(dtype, k_cache, v_cache, cs, k_scale, v_scale, hkv, d)
    if cu_seqlens is None:
        total, shape = B * tokens, (B, tokens, hkv, d)
    else:
        total, shape = tokens, (tokens, hkv, d)
        cu_seqlens = _i32(cu_seqlens, "cu_seqlens", (B + 1,))
    new = out is None
    if new:
        make = torch.empty if B else torch.zeros  # (a batch of no rows is not launched)
        out = tuple(make(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
    else:
        if len(out) != 2 or any(t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.data_ptr() % 16
                                for t in out):
            raise ValueError("out must be two contiguous, 16-byte aligned %s %s" % (dtype, tuple(shape)))
        if out[0].numel() and out[0].data_ptr() == out[1].data_ptr():
            raise ValueError("out's two tensors must be apart")
    table, table_stride, max_pages = _table(page_table, B)
    lens = _i32(lens, "lens", (B,))
    a = _lib.KvReadArgs(
        total, B, hkv, d, _IO[dtype], cache_dtype, out[0].data_ptr(), hkv * d, d, out[1].data_ptr(), hkv * d, d,
        _ptr(cu_seqlens), k_cache.data_ptr(), *kcs, v_cache.data_ptr(), *vcs, n_pages, page, max_pages,
        table.data_ptr(), table_stride, lens.data_ptr(), _ptr(factors[0]), _ptr(factors[1]), blocks[0], _ptr(blocks[1]),
        _ptr(blocks[2]), int(new))
    return a, (cu_seqlens, table, lens, factors, blocks), tuple(out)


def kv_read(k_cache, v_cache, page_table, lens, tokens, *, cu_seqlens=None, dtype=None, k_scale=None, v_scale=None,
            out=None, stream=None):
    """Read tokens back out of their pages: the inverse of kv_append.

    tokens: how many newest tokens of every row, or with non-decreasing
    cu_seqlens [B + 1] the packed total.  Row b's n tokens are those of positions
    lens[b] - n .. lens[b] - 1; positions that hold nothing (below 0, past the
    table, a table entry outside the cache) give zeros.  Caches, page_table and
    scales as for attn_decode; 8-bit values are multiplied by their scale.  dtype
    (None: the caches', bfloat16 for 8-bit ones): of the result, one rounding.
    out: (k, v) to write to; tokens of no row are left as they were there, and
    zeros in new ones.  Returns (k, v): [B, tokens, hkv, d], or [tokens, hkv, d].
    """
    if out is None and stream is None and k_cache.is_cuda:
        io = _IO.get(dtype or k_cache.dtype, _lib.GDN_BF16 if dtype is None else -1)
        got = _short("kv_read", k_cache, v_cache, page_table, lens, tokens, cu_seqlens, io, k_scale, v_scale)
        if got is not None:
            return got
    dev = k_cache.device
    ctx = _on(stream, dev, (v_cache, page_table, lens, cu_seqlens, k_scale, v_scale) + tuple(out or ()))
    if ctx is not None:
        with ctx:
            return kv_read(k_cache, v_cache, page_table, lens, tokens, cu_seqlens=cu_seqlens, dtype=dtype,
                           k_scale=k_scale, v_scale=v_scale, out=out)
    a, keep, out = kv_read_args(k_cache, v_cache, page_table, lens, tokens, cu_seqlens=cu_seqlens, dtype=dtype,
                                k_scale=k_scale, v_scale=v_scale, out=out)
    _checked(_library().gdn_kv_read(byref(a), _raw_stream(dev.index)))
    del keep
    return out


def _page_block(pool):
    """(bytes of a page, bytes from page to page) of a pool [n_pages, ...] whose
    pages are dense blocks, their inner dimensions in any order."""
    if pool.dim() < 1:
        raise ValueError("pool must be [n_pages, ...]")
    inner = 1
    if pool.is_contiguous():
        nbytes = pool.numel() // max(1, pool.shape[0]) * pool.element_size()
        return nbytes, nbytes
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
    dev = pool.device
    ctx = _on(stream, dev, (src, dst))
    if ctx is not None:
        with ctx:
            return pages_copy(pool, src, dst)
    nbytes, stride = _page_block(pool)
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    n = src.shape[0]
    src, dst = _i32(src, "src", (n,), -1), _i32(dst, "dst", (n,), -1)
    _checked(_library().gdn_pages_copy(pool.data_ptr(), nbytes, stride, pool.shape[0], src.data_ptr(), dst.data_ptr(),
                                        n, _raw_stream(dev.index)))
    return pool


def pages_args(page_table, lens, refs, page_size, out=None, apart=False, workspace=True):
    """Validate shapes and build the gdn_pages_args struct (device-agnostic):
    returns (args, tensors to keep alive, (page_table, lens, refs) outputs).
    lens None: a call that has no lengths.  apart: the outputs may not be the
    inputs."""
    shape = page_table.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("page_table must be [rows, max_pages]")
    if refs.dim() != 1 or refs.shape[0] < 1:
        raise ValueError("refs must be [n_pages]")
    if int(page_size) != page_size or not _I32_MIN <= page_size <= _I32_MAX:
        raise ValueError("page_size must be a whole number of 32 bits, got %s" % (page_size,))
    rows, n = shape[0], refs.shape[0]
    table, table_stride, width = _table(page_table, rows)
    refs_in = _i32(refs, "refs", (n,))
    lens_in = None if lens is None else _i32(lens, "lens", (rows,))
    dev = page_table.device
    if out is None:
        to = torch.empty_like(table) if table.is_contiguous() else table.new_empty(rows, width)
        lens_to = None if lens is None else torch.empty_like(lens_in)
        refs_to = torch.empty_like(refs_in)
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
    ws, need = None, 0
    if workspace:
        need = _library().gdn_pages_workspace_size(rows, n)
        ws = refs_in.new_empty(need // 4)
    a = _lib.PagesArgs(rows, width, n, int(page_size), table.data_ptr(), table_stride, _ptr(lens_in), refs_in.data_ptr(),
                       to.data_ptr(), max(to.stride(0), width), _ptr(lens_to), refs_to.data_ptr(), _ptr(ws), need)
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
    dev = page_table.device
    ctx = _on(stream, dev, (lens, refs, add))
    if ctx is not None:
        with ctx:
            return pages_extend(page_table, lens, refs, add, page_size, out=out)
    a, keep, (table, lens_to, refs_to) = pages_args(page_table, lens, refs, page_size, out)
    add = _i32(add, "add", (a.rows,))
    ok = torch.empty_like(add)
    _checked(_library().gdn_pages_extend(byref(a), add.data_ptr(), ok.data_ptr(), _raw_stream(dev.index)))
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
    dev = page_table.device
    ctx = _on(stream, dev, (lens, refs, parent))
    if ctx is not None:
        with ctx:
            return pages_fork(page_table, lens, refs, parent, page_size, out=out)
    a, keep, (table, lens_to, refs_to) = pages_args(page_table, lens, refs, page_size, out, apart=True)
    parent = _i32(parent, "parent", (a.rows,), -1)
    src, dst = torch.empty_like(parent), torch.empty_like(parent)
    _checked(_library().gdn_pages_fork(byref(a), parent.data_ptr(), src.data_ptr(), dst.data_ptr(),
                                        _raw_stream(dev.index)))
    del keep
    return table, lens_to, refs_to, src, dst


def pages_free(page_table, lens, refs, rows, page_size, *, out=None, stream=None):
    """Release the pages of the rows where rows [n_rows] (bool or uint8) is set:
    they end empty, their table entries -1.  out as in pages_extend.  Returns
    (page_table, lens, refs)."""
    dev = page_table.device
    ctx = _on(stream, dev, (lens, refs, rows))
    if ctx is not None:
        with ctx:
            return pages_free(page_table, lens, refs, rows, page_size, out=out)
    a, keep, to = pages_args(page_table, lens, refs, page_size, out, workspace=False)
    if rows.shape != (a.rows,) or rows.dtype not in (torch.bool, torch.uint8):
        raise ValueError("rows must be bool or uint8 [%d]" % a.rows)
    rows = rows.contiguous()
    _checked(_library().gdn_pages_free(byref(a), rows.data_ptr(), _raw_stream(dev.index)))
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
    dev = page_table.device
    ctx = _on(stream, dev, (refs,))
    if ctx is not None:
        with ctx:
            return pages_compact(page_table, refs, out=out)
    a, keep, (table, _, refs_to) = pages_args(page_table, None, refs, 1, out)
    src = refs_to.new_empty(a.n_pages // 2)
    dst, n_live = torch.empty_like(src), refs_to.new_empty(1)
    _checked(_library().gdn_pages_compact(byref(a), src.data_ptr(), dst.data_ptr(), n_live.data_ptr(),
                                           _raw_stream(dev.index)))
    del keep
    return table, refs_to, src, dst, n_live
