"""Python binding of the attention operators (``include/moe_attn.h``): rotary
positions, appending keys and values to a paged cache, and attention over it.

Argument marshalling and checks only; the operators are the CUDA kernels of
``libmoe_w4a16.so``. Tensors of the wrong type, device or form, and tensors that
autograd would follow, raise ``ValueError`` before anything is launched; a status
of the library raises ``MoeError``.
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


# The C ABI's structures, for calls by ctypes; the calls below go through csrc/binding.c.
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


_library = None
_native = None  # csrc/binding.c: checks tensors, calls the library


def _lib() -> ctypes.CDLL:
    global _library, _native
    if _library is None:
        from . import lib
        L = lib()
        register(L)
        try:
            from . import _attn_binding
        except ImportError as e:
            raise RuntimeError(
                "the attention operators' Python binding is missing for this interpreter: build it "
                "with `python -m w4a16_routed_expert_router_gb300._build` (it needs the Python "
                "headers)") from e

        def address(name):
            return ctypes.cast(getattr(L, name), ctypes.c_void_p).value

        _attn_binding.setup(address("moe_attn_rope"), address("moe_attn_append"),
                            address("moe_attn_forward"), _check, torch.empty, _raw_stream,
                            _current_device, torch.is_grad_enabled,
                            torch.is_inference_mode_enabled, _increment_version, torch.bfloat16,
                            torch.float16, torch.float32, torch.int32, torch.int64)
        _native, _library = _attn_binding, L
    return _library


def _check(status: int, what: str) -> None:
    if status != MOE_ATTN_OK:
        from . import MoeError
        raise MoeError(status, what)


def _stream_address(index) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's address and the current device without the objects and
# checks around them (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_address)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _increment_versions(tensors):
    for t in tensors:
        torch.autograd.graph.increment_version(t)


# of a list of tensors that were written to
_increment_version = getattr(torch._C, "_increment_version", _increment_versions)


def _layout(layout) -> int:
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    return code


def _on_stream(stream, out, shape, dtype, device):
    """(address of a given stream, output for a call on it: new ones belong to it)."""
    if isinstance(stream, int):
        if out is None:
            raise ValueError("an output is needed where the stream is a raw address")
        return stream, out
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.empty(shape, dtype=dtype, device=device)
    return stream.cuda_stream, out


def _in_use(stream, device, *tensors):
    """Memory of tensors that a call on a given stream works on is not handed out
    again before it is done, though they belong to another."""
    if isinstance(stream, int):  # an address is of the tensors' device, not the current one
        stream = torch.cuda.ExternalStream(stream, device=device)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


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
    turns the other way: the gradient of x from the gradient of the result (autograd
    does not follow this call, and tensors that require a gradient are refused)."""
    if _native is None:
        _lib()
    given = stream
    if stream is not None:
        stream, out = _on_stream(stream, out, x.shape, x.dtype, x.device)
    args = (x, positions, freq, out, _layout(layout), magnitude, inverse, stream)
    done = _native.rope(*args)
    if done is NotImplemented:  # another device is current
        with torch.cuda.device(x.device):
            done = _native.rope(*args)
    if given is not None:
        _in_use(given, x.device, x, positions, freq, out)
    return done


# Handles to be destroyed. That waits for the device, which would end a capture of
# this thread's stream (a collection of garbage comes at any time): they stay here
# until a layer is made or closed outside of one.
_dropped = []


def _destroy_dropped():
    if not _dropped or torch.cuda.is_current_stream_capturing():
        return
    while _dropped:
        library, handle = _dropped.pop()
        _check(library.moe_attn_destroy(handle), "moe_attn_destroy")


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
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError(f"device must be a CUDA device, got {device}")
        index = torch.cuda.current_device() if device.index is None else device.index
        self.device = torch.device("cuda", index)
        _destroy_dropped()
        handle = _vp()
        _check(self._library.moe_attn_create(ctypes.byref(self.cfg), index, ctypes.byref(handle)),
               "moe_attn_create")
        self.handle = handle
        self._layer = _native.layer(handle.value, q_heads, kv_heads, head_dim, page_size, index,
                                    dtype, self.device)

    def close(self):
        if self.handle is not None and self.handle.value:
            _dropped.append((self._library, self.handle))
            self.handle = None
            _destroy_dropped()
        self.handle = None

    def _open(self):
        if self.handle is None:
            raise RuntimeError("this layer has been closed")
        return self._layer

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

    def append(self, q, k, v, positions, slots, k_pages, v_pages, freq, layout="half",
               magnitude=1.0, q_out=None, stream=None):
        """Turn q and k [tokens, heads, head_dim] to their positions (int32) and
        write k and v to their slots (int64; page * page_size + offset, negative:
        not written) of the cache. Returns q_out (new unless given, may be q);
        q None: keys and values only."""
        given = stream
        if stream is not None:
            if q is not None:
                stream, q_out = _on_stream(stream, q_out, q.shape, self.dtype, self.device)
            elif not isinstance(stream, int):
                stream = stream.cuda_stream
        done = _native.append(self._open(), q, k, v, positions, slots, k_pages, v_pages, freq,
                              _layout(layout), magnitude, q_out, stream)
        if given is not None:
            _in_use(given, self.device, q, k, v, positions, slots, k_pages, v_pages, freq, q_out)
        return done

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
        given = stream
        if stream is not None:
            if return_lse and lse is None:
                _, lse = _on_stream(stream, None, q.shape[:2], torch.float32, self.device)
            stream, out = _on_stream(stream, out, q.shape, self.dtype, self.device)
        done = _native.forward(self._open(), q, k_pages, v_pages, page_table, cu_q, kv_len, max_q,
                               scale, softcap, window, slopes, prefix, out, lse, return_lse,
                               stream)
        if given is not None:
            _in_use(given, self.device, q, k_pages, v_pages, page_table, cu_q, kv_len, slopes,
                    prefix, out, lse)
        return done


class PagedKvCache:
    """Pages of one layer's keys and values and the bookkeeping of which
    sequence holds which: slots for new tokens, page tables for attention.

    The bookkeeping is plain Python, for examples and small batches: `tables` makes
    every row anew (3 ms for 64 sequences of 1000 pages). A server keeps its tables
    on the device and adds the pages that are new.
    """

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
