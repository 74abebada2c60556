"""Python binding of the attention operators (``include/moe_attn.h``): rotary
positions, appending keys and values to a paged cache, and attention over it.

Argument marshalling and checks only; the operators are the CUDA kernels of
``libmoe_w4a16.so``. Tensors of the wrong type, device or form raise
``ValueError`` before anything is launched; a status of the library raises
``MoeError``.
"""
from __future__ import annotations

import ctypes

import torch

MOE_ATTN_OK = 0
MOE_ATTN_ERR_DEVICE = -6
MOE_ATTN_BF16 = 0
MOE_ATTN_FP16 = 1
MOE_ATTN_ROPE_HALF = 0
MOE_ATTN_ROPE_INTERLEAVED = 1
MOE_ATTN_DEVERR_TIMEOUT = 0x1
MOE_ATTN_DEVERR_RANGE = 0x2

# every symbol include/moe_attn.h declares
EXPORTS_ATTN = (
    "moe_attn_rope_frequencies",
    "moe_attn_rope",
    "moe_attn_workspace_bytes",
    "moe_attn_create",
    "moe_attn_destroy",
    "moe_attn_append",
    "moe_attn_forward",
    "moe_attn_check_device_errors",
)

_DTYPES = {torch.bfloat16: MOE_ATTN_BF16, torch.float16: MOE_ATTN_FP16}
_LAYOUTS = {"half": MOE_ATTN_ROPE_HALF, "interleaved": MOE_ATTN_ROPE_INTERLEAVED}

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class moe_attn_rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class moe_attn_rotation(ctypes.Structure):
    _fields_ = [("freq", _vp), ("rot_dim", _i32), ("layout", _i32), ("magnitude", _f32),
                ("inverse", _i32)]


class moe_attn_config(ctypes.Structure):
    _fields_ = [("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("max_tokens", _i32), ("max_seqs", _i32), ("dtype", _i32),
                ("flags", ctypes.c_uint32)]


class moe_attn_cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("num_pages", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64)]


class moe_attn_batch(ctypes.Structure):
    _fields_ = [("cu_q", _vp), ("kv_len", _vp), ("page_table", _vp), ("table_stride", _i64),
                ("columns", _i32), ("num_seqs", _i32), ("num_tokens", _i32), ("max_q", _i32)]


class moe_attn_scores(ctypes.Structure):
    _fields_ = [("scale", _f32), ("softcap", _f32), ("window", _i32), ("slopes", _vp),
                ("prefix", _vp)]


def _signatures():
    p = ctypes.POINTER
    rows, rot, cache = p(moe_attn_rows), p(moe_attn_rotation), p(moe_attn_cache)
    f64, cfg = ctypes.c_double, p(moe_attn_config)
    return {
        "moe_attn_rope_frequencies": [_i32, f64, f64, _i32, f64, f64, f64, _vp, p(_f32)],
        "moe_attn_rope": [rows, rows, _vp, _i32, _i32, _i32, _i32, rot, _vp],
        "moe_attn_workspace_bytes": [cfg, p(ctypes.c_size_t)],
        "moe_attn_create": [cfg, ctypes.c_int, p(_vp)],
        "moe_attn_destroy": [_vp],
        "moe_attn_append": [_vp, rows, rows, rows, rows, _vp, _vp, _i32, rot, cache, _vp],
        "moe_attn_forward": [_vp, rows, rows, _vp, cache, p(moe_attn_batch), p(moe_attn_scores),
                             _vp],
        "moe_attn_check_device_errors": [_vp, p(ctypes.c_uint32)],
    }


def register(L: ctypes.CDLL) -> None:
    """Give the library's attention functions their argument types."""
    for name, args in _signatures().items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def _by_address(L: ctypes.CDLL, name: str):
    """The function with its structures passed as plain addresses (half the cost
    of the pointers that ctypes makes of them)."""
    fn = L[name]  # a function object of its own
    fn.argtypes = [_vp if issubclass(a, ctypes._Pointer) else a for a in _signatures()[name]]
    fn.restype = ctypes.c_int
    return fn


_library = None


def _lib() -> ctypes.CDLL:
    global _library
    if _library is None:
        from . import lib
        L = lib()
        register(L)
        _library = L
    return _library


def _check(status: int, what: str) -> None:
    if status != MOE_ATTN_OK:
        from . import MoeError
        raise MoeError(status, what)


# the current stream's address without the Stream object around it (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _fill_rows(s, t, heads, dim, dtype, index, what):
    """Describe t [tokens, heads, dim] on device `index` in s; returns its tokens."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what} must be [tokens, {heads}, {dim}], got {list(shape)}")
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{what} must be {dtype} on cuda:{index}, got {t.dtype} on {t.device}")
    token, head, last = t.stride()
    if last != 1 and dim > 1:
        raise ValueError(f"{what} must be contiguous along head_dim")
    s.data = t.data_ptr()
    # the stride of a dimension of one element says nothing
    s.head_stride = head if heads > 1 else dim
    tokens = shape[0]
    s.token_stride = token if tokens > 1 else heads * s.head_stride
    return tokens


def _new_rows(s, tokens, heads, dim, dtype, device, stream):
    """A new tensor [tokens, heads, dim], described in s."""
    t = _empty((tokens, heads, dim), dtype, device, stream)
    s.data = t.data_ptr()
    s.head_stride = dim
    s.token_stride = heads * dim
    return t


def _vector(t, n, dtype, index, what):
    """Address of t, a contiguous vector of n elements on device `index`."""
    if (t.dtype is not dtype or t.get_device() != index or t.dim() != 1 or t.numel() != n or
            not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} on cuda:{index}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """New tensor for a call on `stream`: owned by that stream, where one is given."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        raise ValueError("an output is needed where the stream is a raw address")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _fill_rotation(s, freq, layout, magnitude, inverse, index):
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    n = freq.numel()
    s.freq = _vector(freq, n, torch.int64, index, "freq")
    s.rot_dim = 2 * n
    s.layout = code
    s.magnitude = magnitude
    s.inverse = 1 if inverse else 0


def moe_attn_rope_frequencies(rot_dim, base=10000.0, factor=1.0, by_parts=False,
                              original_len=4096.0, beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freq, magnitude) of rotary positions over rot_dim values of a head.

    freq: int64 [rot_dim / 2] on `device`, turns per position in units of 2^-64.
    factor > 1 stretches the positions for contexts longer than original_len:
    all pairs alike, or (by_parts) those that turn slowly in it, with the
    magnitude 1 + 0.1 log(factor).
    """
    host = torch.empty(max(0, rot_dim // 2), dtype=torch.int64)
    magnitude = _f32(1.0)
    _check(_lib().moe_attn_rope_frequencies(rot_dim, base, factor, 1 if by_parts else 0,
                                            original_len, beta_fast, beta_slow, host.data_ptr(),
                                            ctypes.byref(magnitude)), "moe_attn_rope_frequencies")
    return host.to(device), magnitude.value


def moe_attn_rope(x, positions, freq, out=None, layout="half", magnitude=1.0, inverse=False,
                  stream=None):
    """Rotary positions of x [tokens, heads, head_dim] (bf16 or fp16, any token
    and head strides) at positions int32 [tokens]; out may be x. ``inverse``
    turns the other way: the gradient of x from the gradient of the result."""
    dtype, device = x.dtype, x.device
    code = _DTYPES.get(dtype)
    if code is None or device.type != "cuda" or x.dim() != 3:
        raise ValueError("x must be a bf16 or fp16 CUDA tensor [tokens, heads, head_dim]")
    index = device.index
    tokens, heads, dim = x.shape
    xs, os, rot = moe_attn_rows(), moe_attn_rows(), moe_attn_rotation()
    _fill_rows(xs, x, heads, dim, dtype, index, "x")
    if out is None:
        out = _new_rows(os, tokens, heads, dim, dtype, device, stream)
    elif _fill_rows(os, out, heads, dim, dtype, index, "out") != tokens:
        raise ValueError("x and out differ in tokens")
    _fill_rotation(rot, freq, layout, magnitude, inverse, index)
    args = (xs, os, _vector(positions, tokens, torch.int32, index, "positions"), tokens, heads,
            dim, code, rot, _stream(stream, device))
    if torch.cuda.current_device() == index:
        st = _lib().moe_attn_rope(*args)
    else:
        with torch.cuda.device(device):
            st = _lib().moe_attn_rope(*args)
    if st:
        _check(st, "moe_attn_rope")
    return out


class PagedAttention:
    """Append and attention for layers of one shape: a handle with its
    workspace, usable by every layer of a model on one stream at a time.

    k_pages and v_pages are [pages, kv_heads, page_size, head_dim] (any strides
    with head_dim contiguous, the same for both; 16-byte multiples).
    """

    def __init__(self, q_heads, kv_heads, head_dim, page_size, max_tokens, max_seqs,
                 dtype=torch.bfloat16, device=None):
        if dtype not in _DTYPES:
            raise ValueError("dtype must be torch.bfloat16 or torch.float16")
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.page_size, self.max_tokens, self.max_seqs = page_size, max_tokens, max_seqs
        self.dtype = dtype
        self.handle = None
        self.cfg = moe_attn_config(q_heads, kv_heads, head_dim, page_size, max_tokens, max_seqs,
                                   _DTYPES[dtype], 0)
        self._library = _lib()
        index = torch.cuda.current_device() if device is None else torch.device(device).index or 0
        self.device = torch.device("cuda", index)
        handle = _vp()
        _check(self._library.moe_attn_create(ctypes.byref(self.cfg), index, ctypes.byref(handle)),
               "moe_attn_create")
        self.handle = handle
        # filled anew by every call, and passed by their addresses
        self._q, self._o = moe_attn_rows(), moe_attn_rows()
        self._k, self._v = moe_attn_rows(), moe_attn_rows()
        self._rot, self._cache = moe_attn_rotation(), moe_attn_cache()
        self._batch, self._scores = moe_attn_batch(), moe_attn_scores()
        at = ctypes.addressof
        self._at_q, self._at_o, self._at_k, self._at_v = (at(self._q), at(self._o), at(self._k),
                                                          at(self._v))
        self._at_rot, self._at_cache = at(self._rot), at(self._cache)
        self._at_batch, self._at_scores = at(self._batch), at(self._scores)
        self._append = _by_address(self._library, "moe_attn_append")
        self._forward = _by_address(self._library, "moe_attn_forward")

    def close(self):
        if self.handle is not None and self.handle.value:
            _check(self._library.moe_attn_destroy(self.handle), "moe_attn_destroy")
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t(0)
        _check(self._library.moe_attn_workspace_bytes(ctypes.byref(self.cfg), ctypes.byref(n)),
               "moe_attn_workspace_bytes")
        return n.value

    def check_device_errors(self) -> int:
        """Synchronise; the device error flag bits since the last check (0: none)."""
        flags = ctypes.c_uint32(0)
        st = self._library.moe_attn_check_device_errors(self.handle, ctypes.byref(flags))
        if st != MOE_ATTN_ERR_DEVICE:
            _check(st, "moe_attn_check_device_errors")
        return flags.value

    def _fill_cache(self, k_pages, v_pages):
        c, index = self._cache, self.device.index
        shape, strides = k_pages.shape, k_pages.stride()
        if (len(shape) != 4 or shape[1] != self.kv_heads or shape[2] != self.page_size or
                shape[3] != self.head_dim):
            raise ValueError(f"k_pages must be [pages, {self.kv_heads}, {self.page_size}, "
                             f"{self.head_dim}], got {list(shape)}")
        if v_pages.shape != shape or v_pages.stride() != strides or strides[3] != 1:
            raise ValueError("k_pages and v_pages must have one shape and strides, head_dim "
                             "contiguous")
        dtype = self.dtype
        if (k_pages.dtype is not dtype or v_pages.dtype is not dtype or
                k_pages.get_device() != index or v_pages.get_device() != index):
            raise ValueError(f"the cache must be {dtype} on {self.device}")
        c.k, c.v = k_pages.data_ptr(), v_pages.data_ptr()
        c.num_pages = pages = shape[0]
        c.token_stride = strides[2]
        # the stride of a dimension of one element says nothing
        c.head_stride = strides[1] if self.kv_heads > 1 else self.head_dim
        c.page_stride = (strides[0] if pages > 1 else
                         self.page_size * self.kv_heads * self.head_dim)

    def append(self, q, k, v, positions, slots, k_pages, v_pages, freq, layout="half",
               magnitude=1.0, q_out=None, stream=None):
        """Turn q and k [tokens, heads, head_dim] to their positions (int32) and
        write k and v to their slots (int64; page * page_size + offset, negative:
        not written) of the cache. Returns q_out (new unless given, may be q);
        q None: keys and values only."""
        device, dtype, dim = self.device, self.dtype, self.head_dim
        index = device.index
        T = _fill_rows(self._k, k, self.kv_heads, dim, dtype, index, "k")
        if _fill_rows(self._v, v, self.kv_heads, dim, dtype, index, "v") != T:
            raise ValueError("k and v differ in tokens")
        at_q = at_o = None
        if q is not None:
            at_q, at_o = self._at_q, self._at_o
            if _fill_rows(self._q, q, self.q_heads, dim, dtype, index, "q") != T:
                raise ValueError("q and k differ in tokens")
            if q_out is None:
                q_out = _new_rows(self._o, T, self.q_heads, dim, dtype, device, stream)
            elif _fill_rows(self._o, q_out, self.q_heads, dim, dtype, index, "q_out") != T:
                raise ValueError("q_out and q differ in tokens")
        elif q_out is not None:
            raise ValueError("q_out without q")
        _fill_rotation(self._rot, freq, layout, magnitude, False, index)
        self._fill_cache(k_pages, v_pages)
        st = self._append(self.handle, at_q, at_o, self._at_k, self._at_v,
                          _vector(positions, T, torch.int32, index, "positions"),
                          _vector(slots, T, torch.int64, index, "slots"), T, self._at_rot,
                          self._at_cache, _stream(stream, device))
        if st:
            _check(st, "moe_attn_append")
        return q_out

    def forward(self, q, k_pages, v_pages, page_table, cu_q, kv_len, max_q, scale=None,
                softcap=0.0, window=0, slopes=None, prefix=None, out=None, lse=None,
                return_lse=False, stream=None):
        """Attention of q [tokens, q_heads, head_dim], the last tokens of each
        sequence, over the sequences' keys in the cache.

        cu_q int32 [seqs + 1]: first row of each sequence; kv_len int32 [seqs]:
        its keys, the new ones included; page_table int32 [seqs, columns]; max_q:
        no sequence has more new tokens. scale defaults to 1 / sqrt(head_dim).
        Returns out, or (out, lse) with lse fp32 [tokens, q_heads].
        """
        device, dim = self.device, self.head_dim
        index = device.index
        T = _fill_rows(self._q, q, self.q_heads, dim, self.dtype, index, "q")
        if out is None:
            out = _new_rows(self._o, T, self.q_heads, dim, self.dtype, device, stream)
        elif _fill_rows(self._o, out, self.q_heads, dim, self.dtype, index, "out") != T:
            raise ValueError("q and out differ in tokens")
        b, s = self._batch, self._scores
        table = page_table.shape
        n = kv_len.numel()
        if (len(table) != 2 or table[0] != n or page_table.dtype is not torch.int32 or
                page_table.get_device() != index or
                (page_table.stride(1) != 1 and table[1] > 1)):
            raise ValueError(f"page_table must be int32 [{n}, columns] on {device}, contiguous "
                             "along the columns")
        b.cu_q = _vector(cu_q, n + 1, torch.int32, index, "cu_q")
        b.kv_len = _vector(kv_len, n, torch.int32, index, "kv_len")
        b.page_table = page_table.data_ptr()
        b.columns = columns = table[1]
        b.table_stride = page_table.stride(0) if n > 1 else columns
        b.num_seqs, b.num_tokens, b.max_q = n, T, max_q
        s.scale = dim ** -0.5 if scale is None else scale
        s.softcap, s.window = softcap, window
        s.slopes = None if slopes is None else _vector(slopes, self.q_heads, torch.float32, index,
                                                       "slopes")
        s.prefix = None if prefix is None else _vector(prefix, n, torch.int32, index, "prefix")
        at_lse = None
        if lse is not None:
            if (lse.dtype is not torch.float32 or tuple(lse.shape) != (T, self.q_heads) or
                    not lse.is_contiguous() or lse.get_device() != index):
                raise ValueError(f"lse must be contiguous float32 [{T}, {self.q_heads}] on "
                                 f"{device}")
            at_lse = lse.data_ptr()
        elif return_lse:
            lse = _empty((T, self.q_heads), torch.float32, device, stream)
            at_lse = lse.data_ptr()
        self._fill_cache(k_pages, v_pages)
        st = self._forward(self.handle, self._at_q, self._at_o, at_lse, self._at_cache,
                           self._at_batch, self._at_scores, _stream(stream, device))
        if st:
            _check(st, "moe_attn_forward")
        return (out, lse) if return_lse else out


class PagedKvCache:
    """Pages of one layer's keys and values and the bookkeeping of which
    sequence holds which: slots for new tokens, page tables for attention."""

    def __init__(self, num_pages, kv_heads, page_size, head_dim, dtype=torch.bfloat16,
                 device="cuda"):
        self.k_pages = torch.empty((num_pages, kv_heads, page_size, head_dim), dtype=dtype,
                                   device=device)
        self.v_pages = torch.empty_like(self.k_pages)
        self.page_size = page_size
        self._free = list(range(num_pages - 1, -1, -1))
        self._pages, self._length = {}, {}

    def length(self, seq) -> int:
        return self._length.get(seq, 0)

    def extend(self, seq, tokens):
        """Room for `tokens` more of a sequence: (positions, slots), host lists."""
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        pages, start = self._pages.get(seq, []), self._length.get(seq, 0)
        need = -(-(start + tokens) // self.page_size) - len(pages)
        if need > len(self._free):
            raise RuntimeError(f"the cache is full: {need} pages needed, {len(self._free)} free")
        pages = self._pages.setdefault(seq, pages)
        pages += [self._free.pop() for _ in range(need)]
        self._length[seq] = start + tokens
        positions = list(range(start, start + tokens))
        return positions, [pages[p // self.page_size] * self.page_size + p % self.page_size
                           for p in positions]

    def release(self, seq):
        """Give a sequence's pages back."""
        self._free += reversed(self._pages.pop(seq, []))
        self._length.pop(seq, None)

    def tables(self, seqs):
        """(page_table int32 [seqs, columns], kv_len int32 [seqs]) on the cache's
        device; the columns behind a sequence's pages hold 0 and are not read."""
        columns = max([len(self._pages.get(s, [])) for s in seqs] + [1])
        rows = [self._pages.get(s, []) for s in seqs]
        table = torch.tensor([r + [0] * (columns - len(r)) for r in rows],
                             dtype=torch.int32).reshape(len(rows), columns)
        kv_len = torch.tensor([self.length(s) for s in seqs], dtype=torch.int32)
        return table.to(self.k_pages.device), kv_len.to(self.k_pages.device)
