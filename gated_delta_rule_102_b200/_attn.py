"""ctypes binding of libgdn's softmax-attention layer (include/gdn.h): the norm + rotary
+ cache append, the paged attention, the page tables and the row copies. Argument
marshalling and shape checks only; the call goes to the caller's current CUDA stream of
the tensors' device unless ``stream`` is given.

Token-row tensors are [B][T][H][d], or [total][H][d] with ``cu_seqlens`` and ``T_max``;
q, k, v and gate may be slices of one projection (any row and head stride that is a
multiple of 8 elements).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._abi import _BF16, _F32, _I32, GDN_OK, GdnError, lib

GDN_DEVICE_ERR_PAGE = 16
GDN_KV_BF16, GDN_KV_E4M3 = 0, 1


def _i32(x, what: str) -> int:
    """x, if 32 bits hold it: ctypes takes the low 32 bits of any other number without a word."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{what}: {x} does not fit 32 bits")
    return x


class GdnAttnConfig(ctypes.Structure):
    """Mirror of ``gdn_attn_config``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "rotary_dim", "rope_interleaved",
                                              "page_size", "kv_dtype", "window")] + \
               [(n, ctypes.c_float) for n in ("norm_eps", "norm_offset", "rope_scale", "sm_scale", "softcap", "k_scale",
                                              "v_scale")]

    @classmethod
    def make(cls, num_q_heads, num_kv_heads, head_dim, page_size, rotary_dim=0, rope_interleaved=False,
             kv_dtype=torch.bfloat16, window=0, norm_eps=1e-6, norm_offset=0.0, rope_scale=0.0, sm_scale=0.0, softcap=0.0,
             k_scale=0.0, v_scale=0.0) -> "GdnAttnConfig":
        kinds = {torch.bfloat16: GDN_KV_BF16, torch.float8_e4m3fn: GDN_KV_E4M3, GDN_KV_BF16: GDN_KV_BF16,
                 GDN_KV_E4M3: GDN_KV_E4M3}
        if kv_dtype not in kinds:
            raise TypeError(f"kv_dtype: {kv_dtype}, expected torch.bfloat16 or torch.float8_e4m3fn")
        for n, x in (("num_q_heads", num_q_heads), ("num_kv_heads", num_kv_heads), ("head_dim", head_dim),
                     ("rotary_dim", rotary_dim), ("page_size", page_size), ("window", window)):
            _i32(x, n)
        return cls(num_q_heads, num_kv_heads, head_dim, rotary_dim, int(bool(rope_interleaved)), page_size,
                   kinds[kv_dtype], window, norm_eps, norm_offset, rope_scale, sm_scale, softcap, k_scale, v_scale)


class _KvCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("table_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p)]


class _Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _CopyBuffer(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


_declared = False


def _lib() -> ctypes.CDLL:
    global _declared
    L = lib()
    if not _declared:
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        cfg, cache, heads = ctypes.POINTER(GdnAttnConfig), ctypes.POINTER(_KvCache), ctypes.POINTER(_Heads)
        L.gdn_qk_rope_append.argtypes = [cfg, cache, i32, i32, vp, i32, heads, heads, heads] + [vp] * 7
        L.gdn_attn_decode.argtypes = [cfg, cache, i32, i32, vp, i32, heads, heads] + [vp] * 6
        L.gdn_attn_decode_workspace_bytes.argtypes = [cfg, i32, i32]
        L.gdn_attn_decode_workspace_bytes.restype = ctypes.c_size_t
        L.gdn_rope_inv_freq_host.argtypes = [i32, ctypes.c_double, ctypes.c_double, i32, i32, vp, vp]
        L.gdn_pages_reserve.argtypes = [i32, i32, vp, vp, i32, vp, i32, i32, vp, vp, i32, vp, vp]
        L.gdn_pages_fork.argtypes = [i32, i32, vp, vp, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp]
        L.gdn_pages_free.argtypes = [i32, vp, vp, i32, i32, vp, vp, i32, vp, vp]
        L.gdn_pages_compact.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]
        L.gdn_copy_rows.argtypes = [ctypes.POINTER(_CopyBuffer), i32, i32, i32, vp, vp, vp, vp, vp]
        for f in ("gdn_qk_rope_append", "gdn_attn_decode", "gdn_rope_inv_freq_host", "gdn_pages_reserve", "gdn_pages_fork",
                  "gdn_pages_free", "gdn_pages_compact", "gdn_copy_rows"):
            getattr(L, f).restype = i32
        _declared = True
    return L


# The current stream's handle without making a Stream object (2 us of a 5 us call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Call:
    """A marshalled call: the C function, its arguments up to the stream as C values, what
    they point into, and the device they live on."""
    __slots__ = ("name", "fn", "args", "keep", "device", "others")

    def __init__(self, name, args, keep, device):
        declared = getattr(_lib(), name)
        # a handle of its own without argument types: the values below need no conversion at each launch
        self.fn = ctypes.CFUNCTYPE(ctypes.c_int32)(ctypes.cast(declared, ctypes.c_void_p).value)
        self.name, self.keep, self.device = name, keep, device
        self.args = tuple(t(_i32(x, name)) if t is ctypes.c_int32 else
                          (t(x) if t is ctypes.c_void_p else (t() if x is None else x))
                          for t, x in zip(declared.argtypes, args))
        self.others = torch.cuda.device_count() > 1

    def run(self, stream=None) -> None:
        if stream is None:
            stream = _current_stream(self.device.index)
        elif isinstance(stream, torch.cuda.Stream):
            stream = stream.cuda_stream
        if self.others and torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                st = self.fn(*self.args, ctypes.c_void_p(int(stream)))
        else:
            st = self.fn(*self.args, ctypes.c_void_p(stream))
        if st != GDN_OK:
            raise GdnError(st, self.name)


class CallPlan:
    """A call of one of this module's functions with its arguments marshalled once:
    ``CallPlan(gdn_attn_decode, cfg, q, ...)``; ``launch()`` makes the C call with the stored
    pointers on the current stream (or the one given), for loops that run on one set of
    tensors (they must stay in place while the plan is used)."""

    def __init__(self, function, *args, **kwargs):
        marshal = getattr(function, "marshal", None)
        if marshal is None:
            raise TypeError("CallPlan: a function of this module is wanted")
        self._stream = kwargs.pop("stream", None)
        self._call = marshal(*args, **kwargs)

    def launch(self, stream=None) -> None:
        self._call.run(self._stream if stream is None else stream)


def _entry(marshal):
    def decorate(f):
        f.marshal = marshal
        return f
    return decorate


class _Args:
    """Checks tensors of one call: type, device, contiguity, shape."""

    def __init__(self, name):
        self.name, self.device, self.keep = name, None, []

    def _see(self, t, dtypes, what):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch.Tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: dtype {t.dtype}, expected one of {dtypes}")
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a CUDA tensor")
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError(f"{what}: on {t.device}, the call's other tensors are on {self.device}")
        self.keep.append(t)

    def ptr(self, t: Optional[torch.Tensor], dtypes, what, shape=None, at_least=None):
        if t is None:
            return None
        self._see(t, dtypes, what)
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if at_least is not None and t.numel() < at_least:
            raise ValueError(f"{what}: {t.numel()} elements, expected at least {at_least}")
        return t.data_ptr()

    def heads(self, t, what, lead, H, d):
        self._see(t, _BF16, what)
        if tuple(t.shape) != tuple(lead) + (H, d):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(lead) + (H, d)}")
        if d > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        row = t.stride(-3)
        if len(lead) == 2 and lead[0] > 1:
            if lead[1] == 1:
                row = t.stride(0)
            elif t.stride(0) != lead[1] * t.stride(1):
                raise ValueError(f"{what}: the token rows must have one stride")
        rows = 1
        for n in lead:
            rows *= n
        h = _Heads(t.data_ptr(), row if rows > 1 else 0, t.stride(-2) if H > 1 else 0)
        self.keep.append(h)
        return ctypes.byref(h)


def _rows(q, slots, cu_seqlens, T_max):
    """(leading dimensions, B, T, total) of a call's token rows."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("q: expected [B][T][H][d] (or cu_seqlens for packed rows)")
        B, T = q.shape[0], q.shape[1]
        if T_max is not None and T_max != T:
            raise ValueError("T_max: given by q's second dimension")
        return (B, T), B, T, B * T
    if T_max is None:
        raise ValueError("T_max: needed with cu_seqlens")
    if q.dim() != 3:
        raise ValueError("q: expected packed rows [total][H][d]")
    return (q.shape[0],), cu_seqlens.shape[0] - 1, int(T_max), q.shape[0]


def _cache(a: _Args, cfg, k_pages, v_pages, page_table, seq_lens):
    kinds = _BF16 if cfg.kv_dtype == GDN_KV_BF16 else (torch.float8_e4m3fn, torch.uint8)
    if k_pages.dim() != 4:
        raise ValueError("k_pages: expected [num_pages][page_size][Hkv][d]")
    shape = (k_pages.shape[0], cfg.page_size, cfg.num_kv_heads, cfg.head_dim)
    if page_table.dim() != 2:
        raise ValueError("page_table: expected [rows][max_pages]")
    for n in (k_pages.shape[0], *page_table.shape):
        _i32(n, a.name)
    c = _KvCache(a.ptr(k_pages, kinds, "k_pages", shape), a.ptr(v_pages, kinds, "v_pages", shape), k_pages.shape[0],
                 a.ptr(page_table, _I32, "page_table"), page_table.shape[0], page_table.shape[1],
                 a.ptr(seq_lens, _I32, "seq_lens", (page_table.shape[0],)))
    a.keep.append(c)
    return ctypes.byref(c)


def _marshal_append(cfg, q, k, v, q_norm_w, k_norm_w, inv_freq, k_pages, v_pages, page_table, seq_lens, slots, q_out,
                    cu_seqlens=None, T_max=None, err_flag=None) -> _Call:
    a = _Args("gdn_qk_rope_append")
    lead, B, T, total = _rows(q, slots, cu_seqlens, T_max)
    Hq, Hkv, d = cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim
    args = (ctypes.byref(cfg), _cache(a, cfg, k_pages, v_pages, page_table, seq_lens), B, T,
            a.ptr(cu_seqlens, _I32, "cu_seqlens"), total, a.heads(q, "q", lead, Hq, d), a.heads(k, "k", lead, Hkv, d),
            a.heads(v, "v", lead, Hkv, d), a.ptr(q_norm_w, _BF16, "q_norm_w", (d,)), a.ptr(k_norm_w, _BF16, "k_norm_w", (d,)),
            a.ptr(inv_freq, _F32, "inv_freq", (cfg.rotary_dim // 2,)), a.ptr(slots, _I32, "slots", (B,)),
            a.ptr(q_out, _BF16, "q_out", lead + (Hq, d)), a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, (cfg, a.keep), a.device)


@_entry(_marshal_append)
def gdn_qk_rope_append(cfg: GdnAttnConfig, q, k, v, q_norm_w, k_norm_w, inv_freq, k_pages, v_pages, page_table, seq_lens,
                       slots, q_out, cu_seqlens=None, T_max=None, err_flag=None, stream=None) -> None:
    """Norm and rotate the heads of q into q_out and of k into the cache, store v: token t of
    the sequence in slot s goes to position seq_lens[s] + t. q_norm_w, k_norm_w, inv_freq may
    be None (no norm; nothing rotated)."""
    _marshal_append(cfg, q, k, v, q_norm_w, k_norm_w, inv_freq, k_pages, v_pages, page_table, seq_lens, slots, q_out,
                    cu_seqlens, T_max, err_flag).run(stream)


def _marshal_attn(cfg, q, k_pages, v_pages, page_table, seq_lens, slots, out, workspace, gate=None, lse=None,
                  cu_seqlens=None, T_max=None, err_flag=None) -> _Call:
    a = _Args("gdn_attn_decode")
    lead, B, T, total = _rows(q, slots, cu_seqlens, T_max)
    Hq, d = cfg.num_q_heads, cfg.head_dim
    need = attn_decode_workspace_bytes(cfg, B, T)
    if not isinstance(workspace, torch.Tensor) or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace: at least {need} bytes are wanted (attn_decode_workspace)")
    args = (ctypes.byref(cfg), _cache(a, cfg, k_pages, v_pages, page_table, seq_lens), B, T,
            a.ptr(cu_seqlens, _I32, "cu_seqlens"), total, a.heads(q, "q", lead, Hq, d),
            None if gate is None else a.heads(gate, "gate", lead, Hq, d), a.ptr(slots, _I32, "slots", (B,)),
            a.ptr(out, _BF16, "out", lead + (Hq, d)), a.ptr(lse, _F32, "lse", lead + (Hq,)),
            a.ptr(err_flag, _I32, "err_flag", at_least=1),
            a.ptr(workspace, (torch.int32, torch.uint8, torch.int64, torch.float32), "workspace"))
    return _Call(a.name, args, (cfg, a.keep), a.device)


@_entry(_marshal_attn)
def gdn_attn_decode(cfg: GdnAttnConfig, q, k_pages, v_pages, page_table, seq_lens, slots, out, workspace, gate=None,
                    lse=None, cu_seqlens=None, T_max=None, err_flag=None, stream=None) -> None:
    """Attention of the new tokens over the cache, theirs included (append first); out is
    multiplied by sigmoid(gate) when a gate is given. workspace: attn_decode_workspace."""
    _marshal_attn(cfg, q, k_pages, v_pages, page_table, seq_lens, slots, out, workspace, gate, lse, cu_seqlens, T_max,
                  err_flag).run(stream)


def attn_decode_workspace_bytes(cfg: GdnAttnConfig, B: int, T: int) -> int:
    return int(_lib().gdn_attn_decode_workspace_bytes(ctypes.byref(cfg), _i32(B, "B"), _i32(T, "T")))


def attn_decode_workspace(cfg: GdnAttnConfig, B: int, T: int, device) -> torch.Tensor:
    """A zeroed workspace for gdn_attn_decode on `device` (keep one per stream)."""
    return torch.zeros((attn_decode_workspace_bytes(cfg, B, T) + 3) // 4, dtype=torch.int32, device=device)


def gdn_rope_inv_freq_host(rotary_dim: int, theta: float, factor: float = 1.0, yarn: bool = False,
                           original_len: int = 0):
    """(inv_freq [rotary_dim / 2] as a CPU tensor, rope_scale): rotation speeds, optionally
    slowed down for contexts `factor` times the trained length."""
    _i32(rotary_dim, "rotary_dim")
    _i32(original_len, "original_len")
    f = torch.empty(max(rotary_dim // 2, 0), dtype=torch.float32)
    scale = ctypes.c_float()
    st = _lib().gdn_rope_inv_freq_host(rotary_dim, theta, factor, int(yarn), original_len, f.data_ptr(), ctypes.byref(scale))
    if st != GDN_OK:
        raise GdnError(st, "gdn_rope_inv_freq_host")
    return f, scale.value


def _tables(a: _Args, page_table, page_refs):
    if page_table.dim() != 2 or page_refs.dim() != 1:
        raise ValueError("page_table: expected [rows][max_pages]; page_refs: expected [num_pages]")
    return (a.ptr(page_table, _I32, "page_table"), page_table.shape[0], page_table.shape[1],
            a.ptr(page_refs, _I32, "page_refs"), page_refs.shape[0])


def _marshal_reserve(page_size, slots, n_tokens, page_table, seq_lens, page_refs, err_flag=None) -> _Call:
    a = _Args("gdn_pages_reserve")
    table, rows, width, refs, pages = _tables(a, page_table, page_refs)
    counts = n_tokens if isinstance(n_tokens, torch.Tensor) else None
    args = (page_size, slots.shape[0], a.ptr(slots, _I32, "slots"), a.ptr(counts, _I32, "n_tokens", (slots.shape[0],)),
            0 if counts is not None else int(n_tokens), table, rows, width, a.ptr(seq_lens, _I32, "seq_lens", (rows,)),
            refs, pages, a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, a.keep, a.device)


@_entry(_marshal_reserve)
def gdn_pages_reserve(page_size: int, slots, n_tokens, page_table, seq_lens, page_refs, err_flag=None, stream=None) -> None:
    """Give every slot the pages for its next n_tokens tokens (a number, or int32 [n])."""
    _marshal_reserve(page_size, slots, n_tokens, page_table, seq_lens, page_refs, err_flag).run(stream)


def _marshal_fork(page_size, src, dst, page_table, seq_lens, page_refs, copy_src, copy_dst, err_flag=None) -> _Call:
    a = _Args("gdn_pages_fork")
    table, rows, width, refs, pages = _tables(a, page_table, page_refs)
    n = src.shape[0]
    args = (page_size, n, a.ptr(src, _I32, "src"), a.ptr(dst, _I32, "dst", (n,)), table, rows, width,
            a.ptr(seq_lens, _I32, "seq_lens", (rows,)), refs, pages, a.ptr(copy_src, _I32, "copy_src", (n,)),
            a.ptr(copy_dst, _I32, "copy_dst", (n,)), a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, a.keep, a.device)


@_entry(_marshal_fork)
def gdn_pages_fork(page_size: int, src, dst, page_table, seq_lens, page_refs, copy_src, copy_dst, err_flag=None,
                   stream=None) -> None:
    """Make every child slot dst[i] (empty) a copy of src[i]; copy_src, copy_dst (int32 [n])
    get the pages whose data gdn_copy_rows then copies."""
    _marshal_fork(page_size, src, dst, page_table, seq_lens, page_refs, copy_src, copy_dst, err_flag).run(stream)


def _marshal_free(slots, page_table, seq_lens, page_refs, err_flag=None) -> _Call:
    a = _Args("gdn_pages_free")
    table, rows, width, refs, pages = _tables(a, page_table, page_refs)
    args = (slots.shape[0], a.ptr(slots, _I32, "slots"), table, rows, width, a.ptr(seq_lens, _I32, "seq_lens", (rows,)),
            refs, pages, a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, a.keep, a.device)


@_entry(_marshal_free)
def gdn_pages_free(slots, page_table, seq_lens, page_refs, err_flag=None, stream=None) -> None:
    """Release every page of the slots."""
    _marshal_free(slots, page_table, seq_lens, page_refs, err_flag).run(stream)


def _marshal_compact(page_table, page_refs, copy_src, copy_dst, n_copies, remap, err_flag=None) -> _Call:
    a = _Args("gdn_pages_compact")
    table, rows, width, refs, pages = _tables(a, page_table, page_refs)
    args = (table, rows, width, refs, pages, a.ptr(copy_src, _I32, "copy_src", (pages,)),
            a.ptr(copy_dst, _I32, "copy_dst", (pages,)), a.ptr(n_copies, _I32, "n_copies", at_least=1),
            a.ptr(remap, _I32, "remap", (pages,)), a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, a.keep, a.device)


@_entry(_marshal_compact)
def gdn_pages_compact(page_table, page_refs, copy_src, copy_dst, n_copies, remap, err_flag=None, stream=None) -> None:
    """Renumber the pages in use to the front of the pool; gdn_copy_rows with copy_src,
    copy_dst (int32 [num_pages]) and n_dev=n_copies then moves the data."""
    _marshal_compact(page_table, page_refs, copy_src, copy_dst, n_copies, remap, err_flag).run(stream)


def _marshal_copy(buffers: Sequence[torch.Tensor], src_ids, dst_ids, n_dev=None, err_flag=None) -> _Call:
    a = _Args("gdn_copy_rows")
    if not buffers:
        raise ValueError("buffers: at least one is wanted")
    rows = buffers[0].shape[0]
    array = (_CopyBuffer * len(buffers))()
    for i, t in enumerate(buffers):
        base = a.ptr(t, (t.dtype,) if isinstance(t, torch.Tensor) else (), f"buffers[{i}]")
        if t.shape[0] != rows:
            raise ValueError(f"buffers[{i}]: {t.shape[0]} rows, the first buffer has {rows}")
        array[i] = _CopyBuffer(base, t[0].numel() * t.element_size() if rows else 0)
    n = src_ids.shape[0]
    args = (array, len(buffers), rows, n, a.ptr(src_ids, _I32, "src_ids"), a.ptr(dst_ids, _I32, "dst_ids", (n,)),
            a.ptr(n_dev, _I32, "n_dev", at_least=1), a.ptr(err_flag, _I32, "err_flag", at_least=1))
    return _Call(a.name, args, (array, a.keep), a.device)


@_entry(_marshal_copy)
def gdn_copy_rows(buffers: Sequence[torch.Tensor], src_ids, dst_ids, n_dev=None, err_flag=None, stream=None) -> None:
    """Row dst_ids[i] of every buffer (same number of rows) becomes its row src_ids[i];
    negative ids are skipped. n_dev: an int32 CUDA tensor with the number of pairs."""
    _marshal_copy(buffers, src_ids, dst_ids, n_dev, err_flag).run(stream)
