"""GB300-native KV-cache quantisation codec: Python binding of libkvq.so.

The functions here carry the names of the C entry points in include/kvq.h and only
marshal arguments: torch tensors become pointers and pitches, the current CUDA
stream becomes the launch stream, and a non-OK status becomes ``KvqError``.  Every
step of the codec runs in the library's sm_103a kernels; there is no CPU path, and
a missing library raises.

Allocation helpers (``Nvfp4Pool``, ``Packed``) use torch for device memory only.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _abi
from ._abi import (DEV_BAD_BLOCK, DEV_BAD_POS, DEV_BAD_SEQLEN, DEV_BAD_SLOT, DEV_NO_SPACE, DEV_TIMEOUT, FMT_FP8,
                   FMT_FP8_PAGE, FMT_INT4, FMT_NVFP4_TENSOR,
                   FMT_NVFP4, KIND_KEY, KIND_VALUE)

__all__ = [
    "KvqError", "KvPool", "Nvfp4Pool", "Packed", "kvq_quant_scatter", "kvq_restore", "kvq_pack",
    "kvq_unpack", "kvq_encode_residual", "kvq_decode_residual", "kvq_decode_attention",
    "kvq_decode_attention_workspace", "kvq_decode_attention_noalloc", "kvq_attention",
    "kvq_attention_workspace", "kvq_append", "kvq_select_blocks", "kvq_select_blocks_workspace", "kvq_sparse_attention",
    "kvq_sparse_attention_workspace", "kvq_plan_pages", "kvq_storage_bytes", "FMT_FP8_PAGE", "DEV_NO_SPACE",
    "kvq_status_string", "kvq_last_error", "library_path", "FMT_NVFP4", "FMT_INT4", "FMT_FP8", "FMT_NVFP4_TENSOR", "KIND_KEY",
    "KIND_VALUE", "DEV_BAD_SLOT", "DEV_BAD_BLOCK", "DEV_BAD_POS", "DEV_BAD_SEQLEN", "DEV_TIMEOUT",
]


class KvqError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_abi.STATUS_NAMES.get(status, status)}: {detail}")


def library_path() -> str:
    return _abi.LIB_PATH


def _lib():
    return _abi.load()


def _check(status: int) -> None:
    if status != _abi.KVQ_OK:
        raise KvqError(status, _lib().kvq_last_error().decode())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    """The launch stream: the given torch stream, else the current stream of the
    current device (its raw handle, without building a Stream object)."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _view3(t: torch.Tensor, name: str):
    """(ptr, row_pitch, head_pitch) of a bf16 [rows, heads, dim] tensor, inner stride 1."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.size(2) > 1):
        raise ValueError(f"{name} must be [rows, heads, dim] with inner stride 1")
    return t.data_ptr(), st[0], st[1]


def _bf16_in(t: torch.Tensor, name: str):
    p, r, h = _view3(t, name)
    return _abi.Bf16In(p, r, h)


def _bf16_out(t: torch.Tensor, name: str):
    p, r, h = _view3(t, name)
    return _abi.Bf16Out(p, r, h)


# ---------------------------------------------------------------------------
# device memory holders
# ---------------------------------------------------------------------------
@dataclass
class KvPool:
    """Paged K/V planes, slot-major (slot = block * block_size + offset); each plane in
    its own format (fmt for K, v_fmt for V; v_fmt None = the same as fmt).

    NVFP4: codes [slots, H, D/2] u8, bscale [slots, H, D/16] u8 (E4M3), rscale [slots, H] f32.
    FP8:   codes [slots, H, D] u8 (E4M3), rscale [slots, H] f32 (no block scales).
    FP8_PAGE: codes as FP8, rscale [slots / block_size, H] f32, one scale a (block, head)."""

    k_codes: torch.Tensor
    k_bscale: Optional[torch.Tensor]
    k_rscale: torch.Tensor
    v_codes: torch.Tensor
    v_bscale: Optional[torch.Tensor]
    v_rscale: torch.Tensor
    block_size: int
    fmt: int = FMT_NVFP4
    v_fmt: Optional[int] = None

    @classmethod
    def empty(cls, num_slots: int, num_heads: int, head_dim: int, block_size: int = 16,
              device="cuda", fill: Optional[int] = None, fmt: int = FMT_NVFP4,
              v_fmt: Optional[int] = None) -> "KvPool":
        def u8(*shape):
            t = torch.empty(shape, dtype=torch.uint8, device=device)
            return t.fill_(fill) if fill is not None else t

        def f32(*shape):
            t = torch.empty(shape, dtype=torch.float32, device=device)
            if fill is not None:
                t.view(torch.uint8).fill_(fill)
            return t

        def plane(f):
            if f == FMT_FP8:
                return u8(num_slots, num_heads, head_dim), None, f32(num_slots, num_heads)
            if f == FMT_FP8_PAGE:
                return u8(num_slots, num_heads, head_dim), None, f32(num_slots // block_size, num_heads)
            return (u8(num_slots, num_heads, head_dim // 2), u8(num_slots, num_heads, head_dim // 16),
                    f32(num_slots, num_heads))

        return cls(*plane(fmt), *plane(fmt if v_fmt is None else v_fmt), block_size, fmt, v_fmt)

    @property
    def num_slots(self) -> int:
        return self.k_codes.size(0)

    @property
    def num_heads(self) -> int:
        return self.k_codes.size(1)

    @property
    def head_dim(self) -> int:
        return self.k_codes.size(2) * (1 if self.fmt in (FMT_FP8, FMT_FP8_PAGE) else 2)

    def _planes(self):
        return [t for t in (self.k_codes, self.k_bscale, self.k_rscale, self.v_codes, self.v_bscale,
                            self.v_rscale) if t is not None]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._planes())

    def _struct(self) -> _abi.Pool:
        """The C struct of the pool, built once and kept while its planes are the same
        tensors (a plane replaced by another tensor rebuilds it)."""
        kc, kb, kr, vc, vb, vr = (self.k_codes, self.k_bscale, self.k_rscale, self.v_codes, self.v_bscale,
                                  self.v_rscale)
        cached = self.__dict__.get("_c_struct")
        if cached is not None:
            st, t, p, f = cached
            if ((id(kc), id(kb), id(kr), id(vc), id(vb), id(vr)) == t and kc.data_ptr() == p[0]
                    and kr.data_ptr() == p[1] and vc.data_ptr() == p[2] and vr.data_ptr() == p[3]
                    and (kb is None or kb.data_ptr() == p[4]) and (vb is None or vb.data_ptr() == p[5])
                    and (self.block_size, self.fmt, self.v_fmt) == f):
                return st
        bs = lambda t: None if t is None else t.data_ptr()
        for t in self._planes():
            if not t.is_contiguous():
                raise ValueError("pool planes must be contiguous")
        for f, sc, name in ((self.fmt, self.k_rscale, "k_rscale"),
                            (self.fmt if self.v_fmt is None else self.v_fmt, self.v_rscale, "v_rscale")):
            if f == FMT_FP8_PAGE and sc.numel() != self.num_slots // self.block_size * self.num_heads:
                raise ValueError(f"{name} must be [blocks, heads] for FMT_FP8_PAGE")
        st = _abi.Pool(
            _abi.Plane(self.k_codes.data_ptr(), bs(self.k_bscale), self.k_rscale.data_ptr()),
            _abi.Plane(self.v_codes.data_ptr(), bs(self.v_bscale), self.v_rscale.data_ptr()),
            self.num_slots, self.block_size, self.num_heads, self.head_dim, self.fmt,
            0 if self.v_fmt is None else self.v_fmt)
        self.__dict__["_c_struct"] = (
            st, (id(kc), id(kb), id(kr), id(vc), id(vb), id(vr)),
            (kc.data_ptr(), kr.data_ptr(), vc.data_ptr(), vr.data_ptr(), bs(kb), bs(vb)),
            (self.block_size, self.fmt, self.v_fmt))
        return st


Nvfp4Pool = KvPool  # the NVFP4 pool is the default format of KvPool


@dataclass
class Packed:
    """A logical packed tensor [rows, heads, dim] (see kvq_packed in include/kvq.h)."""

    fmt: int
    kind: int
    group_size: int
    rows: int
    heads: int
    dim: int
    codes: torch.Tensor
    meta0: Optional[torch.Tensor]
    meta1: Optional[torch.Tensor] = None
    rscale: Optional[torch.Tensor] = None

    @classmethod
    def empty(cls, fmt: int, kind: int, rows: int, heads: int, dim: int, group_size: int = 64,
              device="cuda") -> "Packed":
        if fmt == FMT_NVFP4_TENSOR:
            bs = (math.ceil(rows / 16), heads, dim) if kind == KIND_KEY else (rows, heads, dim // 16)
            return cls(fmt, kind, 16, rows, heads, dim,
                       torch.empty((rows, heads, dim // 2), dtype=torch.uint8, device=device),
                       torch.empty(bs, dtype=torch.uint8, device=device), None,
                       torch.empty((1,), dtype=torch.float32, device=device))
        if fmt == FMT_FP8:
            return cls(fmt, kind, 0, rows, heads, dim,
                       torch.empty((rows, heads, dim), dtype=torch.uint8, device=device), None, None,
                       torch.empty((rows, heads), dtype=torch.float32, device=device))
        codes = torch.empty((rows, heads, dim // 2), dtype=torch.uint8, device=device)
        if fmt == FMT_NVFP4:
            return cls(fmt, kind, 16, rows, heads, dim, codes,
                       torch.empty((rows, heads, dim // 16), dtype=torch.uint8, device=device),
                       None, torch.empty((rows, heads), dtype=torch.float32, device=device))
        if kind == KIND_KEY:
            ms = (math.ceil(rows / group_size), heads, dim)
        else:
            ms = (rows, heads, math.ceil(dim / group_size))
        return cls(fmt, kind, group_size, rows, heads, dim, codes,
                   torch.empty(ms, dtype=torch.float16, device=device),
                   torch.empty(ms, dtype=torch.float16, device=device), None)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.meta0, self.meta1, self.rscale)
                   if t is not None)

    def _struct(self) -> _abi.Packed:
        """The C struct, built once and kept while the buffers and sizes are the same."""
        bufs = (self.codes, self.meta0, self.meta1, self.rscale)
        key = tuple(None if t is None else (id(t), t.data_ptr()) for t in bufs) + (
            self.fmt, self.kind, self.group_size, self.rows, self.heads, self.dim)
        cached = self.__dict__.get("_c_struct")
        if cached is not None and cached[0] == key:
            return cached[1]
        for t in bufs:
            if t is not None and not t.is_contiguous():
                raise ValueError("packed buffers must be contiguous")
        st = _abi.Packed(self.fmt, self.kind, self.group_size, self.rows, self.heads, self.dim,
                         self.codes.data_ptr(), None if self.meta0 is None else self.meta0.data_ptr(),
                         None if self.meta1 is None else self.meta1.data_ptr(),
                         None if self.rscale is None else self.rscale.data_ptr())
        self.__dict__["_c_struct"] = (key, st)
        return st


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def kvq_quant_scatter(k: Optional[torch.Tensor], v: Optional[torch.Tensor], slot_ids: torch.Tensor,
                      pool: KvPool, dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise + scatter of K/V [T, H, D] bf16 into pool slots slot_ids[T] (int64), in the
    pool's formats (NVFP4, FP8 or FP8_PAGE)."""
    src = k if k is not None else v
    if src is None:
        raise ValueError("k and v are both None")
    if slot_ids.dtype != torch.int64:
        raise TypeError("slot_ids must be int64")
    T = src.size(0)
    kin = _bf16_in(k, "k") if k is not None else None
    vin = _bf16_in(v, "v") if v is not None else None
    ps = pool._struct()
    _check(_lib().kvq_quant_scatter(
        ctypes.byref(kin) if kin is not None else None, ctypes.byref(vin) if vin is not None else None,
        T, _ptr(slot_ids), ctypes.byref(ps), _ptr(dev_status), _stream(stream)))


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """Scratch of one call, allocated on the call's own stream: a block that the allocator hands
    out was freed there, so its former use comes before this one, and its next use after."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _seq_view(t: torch.Tensor, S: int, Tmax: int, name: str):
    """[S, Tmax, H, D] (or [S*Tmax, H, D]) bf16 -> Bf16Out over S*Tmax rows."""
    if t.dim() == 4:
        if t.size(0) != S or t.size(1) != Tmax or (S > 1 and t.stride(0) != Tmax * t.stride(1)):
            raise ValueError(f"{name} must be [S, Tmax, H, D] with sequence stride Tmax*token stride")
        t = t.flatten(0, 1)
    return _bf16_out(t, name)


def kvq_restore(pool: KvPool, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor],
                dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Paged restore into k_out / v_out [S, max_seq_len, H, D] bf16."""
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    ko = _seq_view(k_out, S, max_seq_len, "k_out") if k_out is not None else None
    vo = _seq_view(v_out, S, max_seq_len, "v_out") if v_out is not None else None
    ps = pool._struct()
    _check(_lib().kvq_restore(
        ctypes.byref(ps), _ptr(block_table), S, max_blocks, _ptr(seq_lens), max_seq_len,
        ctypes.byref(ko) if ko is not None else None, ctypes.byref(vo) if vo is not None else None,
        _ptr(dev_status), _stream(stream)))


def kvq_pack(x: torch.Tensor, out: Packed, stream=None) -> Packed:
    xin = _bf16_in(x, "x")
    ps = out._struct()
    _check(_lib().kvq_pack(ctypes.byref(xin), ctypes.byref(ps), _stream(stream)))
    return out


def kvq_unpack(packed: Packed, y: torch.Tensor, stream=None) -> torch.Tensor:
    yo = _bf16_out(y, "y")
    ps = packed._struct()
    _check(_lib().kvq_unpack(ctypes.byref(ps), ctypes.byref(yo), _stream(stream)))
    return y


def kvq_encode_residual(cur: torch.Tensor, prev: torch.Tensor, pos: Optional[torch.Tensor],
                        payload: Packed, pos_out: Optional[torch.Tensor] = None,
                        dev_status: Optional[torch.Tensor] = None, stream=None) -> Packed:
    if pos is not None and pos.dtype != torch.int32:
        raise TypeError("pos must be int32")
    ci, pi = _bf16_in(cur, "cur"), _bf16_in(prev, "prev")
    n = cur.size(0) if pos is None else pos.numel()
    ps = payload._struct()
    pos_ptr = _ptr(pos)
    if pos is not None and pos.numel() == 0:
        pos_ptr = ctypes.c_void_p(prev.data_ptr())  # non-NULL marks "sparse, nothing kept"
    _check(_lib().kvq_encode_residual(
        ctypes.byref(ci), ctypes.byref(pi), cur.size(0), pos_ptr, n, ctypes.byref(ps),
        _ptr(pos_out), _ptr(dev_status), _stream(stream)))
    return payload


def kvq_decode_residual(payload: Packed, pos: Optional[torch.Tensor], prev: torch.Tensor,
                        out: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    if pos is not None and pos.dtype != torch.int32:
        raise TypeError("pos must be int32")
    pi, oo = _bf16_in(prev, "prev"), _bf16_out(out, "out")
    n = prev.size(0) if pos is None else pos.numel()
    ps = payload._struct()
    pos_ptr = _ptr(pos)
    if pos is not None and pos.numel() == 0:
        pos_ptr = ctypes.c_void_p(prev.data_ptr())  # non-NULL marks "sparse, nothing kept"
    _check(_lib().kvq_decode_residual(
        ctypes.byref(ps), pos_ptr, n, ctypes.byref(pi), prev.size(0), ctypes.byref(oo),
        _ptr(dev_status), _stream(stream)))
    return out


def kvq_decode_attention_workspace(num_seqs: int, num_heads: int, num_q_heads: int, head_dim: int,
                                   max_seq_len: int) -> int:
    return int(_lib().kvq_decode_attention_workspace(num_seqs, num_heads, num_q_heads, head_dim, max_seq_len))


def kvq_decode_attention(pool: KvPool, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                         q: torch.Tensor, scale: float, out: torch.Tensor,
                         workspace: Optional[torch.Tensor] = None,
                         dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention of q [S, Hq, D] bf16 over the pool's K/V (decoded in registers)
    into out [S, Hq, D] bf16.  A workspace tensor is allocated when none is given."""
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    qi, oo = _bf16_in(q, "q"), _bf16_out(out, "out")
    Hq = q.size(1)
    if workspace is None:
        need = kvq_decode_attention_workspace(S, pool.num_heads, Hq, pool.head_dim, max_seq_len)
        if need > 0:
            workspace = _workspace(need, q.device, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ps = pool._struct()
    _check(_lib().kvq_decode_attention(
        ctypes.byref(ps), _ptr(block_table), S, max_blocks, _ptr(seq_lens), max_seq_len, ctypes.byref(qi), Hq,
        float(scale), ctypes.byref(oo), _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)))
    return out


def kvq_decode_attention_noalloc(pool: KvPool, block_table: torch.Tensor, seq_lens: torch.Tensor,
                                 max_seq_len: int, q: torch.Tensor, scale: float, out: torch.Tensor,
                                 dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """kvq_decode_attention with the library's built-in split scratch: no workspace and no
    allocation (calls must not overlap on one device)."""
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    qi, oo = _bf16_in(q, "q"), _bf16_out(out, "out")
    ps = pool._struct()
    _check(_lib().kvq_decode_attention_noalloc(
        ctypes.byref(ps), _ptr(block_table), S, max_blocks, _ptr(seq_lens), max_seq_len, ctypes.byref(qi),
        q.size(1), float(scale), ctypes.byref(oo), _ptr(dev_status), _stream(stream)))
    return out


def kvq_attention_workspace(num_seqs: int, num_tokens: int, num_heads: int, num_q_heads: int, head_dim: int,
                            max_query_len: int, max_seq_len: int) -> int:
    return int(_lib().kvq_attention_workspace(num_seqs, num_tokens, num_heads, num_q_heads, head_dim,
                                              max_query_len, max_seq_len))


def _vec(t: Optional[torch.Tensor], dtype, name: str, n: Optional[int] = None):
    """Pointer of a contiguous 1-d tensor of a dtype (and length n); None stays None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous 1-d tensor" + ("" if n is None else f" of {n} entries"))
    return t.data_ptr()


def kvq_attention(pool: KvPool, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                  q: torch.Tensor, query_starts: torch.Tensor, max_query_len: int, scale: float,
                  out: torch.Tensor, *, softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
                  window: int = 0, prefix_lens: Optional[torch.Tensor] = None,
                  key_starts: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the query rows q [T, Hq, D] bf16 (sequence s owns rows query_starts[s] to
    query_starts[s + 1], its last tokens) over the pool's K/V into out [T, Hq, D] bf16; the
    score options are those of kvq_attn_options.  A workspace tensor is allocated when none
    is given."""
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    qi, oo = _bf16_in(q, "q"), _bf16_out(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    T, Hq, D = q.shape
    if D != pool.head_dim:
        raise ValueError(f"q has head_dim {D}, the pool {pool.head_dim}")
    lens = _vec(seq_lens, torch.int32, "seq_lens", S)
    starts = _vec(query_starts, torch.int32, "query_starts", S + 1)
    opts = None
    if softcap != 0.0 or window != 0 or not (alibi_slopes is None and prefix_lens is None and key_starts is None):
        opts = _abi.AttnOptions(float(softcap), _vec(alibi_slopes, torch.float32, "alibi_slopes", Hq), int(window),
                                _vec(prefix_lens, torch.int32, "prefix_lens", S),
                                _vec(key_starts, torch.int32, "key_starts", T))
    if workspace is None:
        need = kvq_attention_workspace(S, T, pool.num_heads, Hq, D, max_query_len, max_seq_len)
        if need > 0:
            workspace = _workspace(need, q.device, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ps = pool._struct()
    _check(_lib().kvq_attention(
        ctypes.byref(ps), block_table.data_ptr(), S, max_blocks, lens, max_seq_len, ctypes.byref(qi), starts, T,
        max_query_len, Hq, float(scale), None if opts is None else ctypes.byref(opts), ctypes.byref(oo),
        _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)))
    return out


def kvq_append(k: Optional[torch.Tensor], v: Optional[torch.Tensor], slot_ids: Optional[torch.Tensor], pool: KvPool, *,
               cos_sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
               interleaved: bool = False, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
               key_bounds: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
               stream=None) -> Optional[torch.Tensor]:
    """K/V [T, H, D] bf16 into pool slots slot_ids [T] (int64), K turned by the angles of its
    positions [T] (int32): cos_sin [num_positions, rot_dim] f32 holds a position's cosines, then its
    sines.  q [T, Hq, D] is turned into q_out (which may be q; returned).  key_bounds
    [blocks, H, 2, D] bf16 keeps the least and largest key of each block (see include/kvq.h)."""
    src = k if k is not None else v if v is not None else q
    if src is None:
        raise ValueError("k, v and q are all None")
    ps = pool._struct()
    T, H, D = src.size(0), ps.num_heads, ps.head_dim
    rows = (T, H, D)
    if (k is not None and k.shape != rows) or (v is not None and v.shape != rows):
        raise ValueError(f"k and v must be [{T}, {H}, {D}]")
    kin = vin = qin = qo = rot = slots = bounds = None
    Hq = 0
    if k is not None:
        kin = ctypes.byref(_bf16_in(k, "k"))
    if v is not None:
        vin = ctypes.byref(_bf16_in(v, "v"))
    if k is not None or v is not None:
        slots = _vec(slot_ids, torch.int64, "slot_ids", T)
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q and q_out come together")
        if q.dim() != 3 or q.shape != q_out.shape or q.size(0) != T or q.size(2) != D:
            raise ValueError(f"q and q_out must be [{T}, query heads, {D}]")
        Hq, qin, qo = q.size(1), ctypes.byref(_bf16_in(q, "q")), ctypes.byref(_bf16_out(q_out, "q_out"))
    if cos_sin is not None:
        if positions is None:
            raise ValueError("cos_sin needs positions")
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous [positions, rot_dim] float32 tensor")
        if cos_sin.size(0) == 0:  # its pointer is null, which means no rotation
            raise ValueError("cos_sin has no positions")
        rot = ctypes.byref(_abi.Rotation(cos_sin.data_ptr(), cos_sin.size(0), cos_sin.size(1), 1 if interleaved else 0,
                                         _vec(positions, torch.int32, "positions", T)))
    elif positions is not None:
        raise ValueError("positions need cos_sin")
    if key_bounds is not None:
        _bounds_shape(key_bounds, ps.num_slots // ps.block_size, H, D)
        bounds = key_bounds.data_ptr()
    _check(_lib().kvq_append(kin, vin, T, slots, ctypes.byref(ps), rot, qin, qo, Hq, bounds, _ptr(dev_status),
                             _stream(stream)))
    return q_out


def _bounds_shape(t: torch.Tensor, blocks: Optional[int], H: Optional[int], D: int) -> None:
    if t.dtype != torch.bfloat16:
        raise TypeError("key_bounds must be bfloat16")
    if (t.dim() != 4 or t.shape != (t.size(0) if blocks is None else blocks, t.size(1) if H is None else H, 2, D)
            or not t.is_contiguous()):
        raise ValueError("key_bounds must be a contiguous [blocks, heads, 2, head_dim] tensor")


def kvq_select_blocks_workspace(num_tokens: int, num_heads: int, max_seq_len: int, block_size: int) -> int:
    return int(_lib().kvq_select_blocks_workspace(num_tokens, num_heads, max_seq_len, block_size))


def kvq_select_blocks(key_bounds: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      block_size: int, q: torch.Tensor, query_starts: torch.Tensor, max_query_len: int,
                      selected: torch.Tensor, *, first_blocks: int = 1, last_blocks: int = 1,
                      workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """The blocks with the highest score bounds for each query row q [T, Hq, D] bf16 and KV head, into
    selected [T, H, topk] int32 (ascending, -1 behind the last), from key_bounds
    [blocks, H, 2, D] bf16 as kvq_append keeps them.  A workspace tensor is allocated when none
    is given."""
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    T, Hq, D = q.shape
    _bounds_shape(key_bounds, None, None, D)
    H = key_bounds.size(1)
    sel = _lists(selected, T, H)
    qi = _bf16_in(q, "q")
    if workspace is None:
        need = kvq_select_blocks_workspace(T, H, max_seq_len, block_size)
        if need > 0:
            workspace = _workspace(need, q.device, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().kvq_select_blocks(
        key_bounds.data_ptr(), key_bounds.size(0), block_size, H, D, block_table.data_ptr(), S, max_blocks,
        _vec(seq_lens, torch.int32, "seq_lens", S), max_seq_len, ctypes.byref(qi),
        _vec(query_starts, torch.int32, "query_starts", S + 1), T, max_query_len, Hq, first_blocks, last_blocks,
        selected.size(2), sel, _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)))
    return selected


def _lists(t: torch.Tensor, T: int, H: int):
    if t.dtype != torch.int32:
        raise TypeError("selected must be int32")
    if t.dim() != 3 or t.shape[:2] != (T, H) or not t.is_contiguous():
        raise ValueError(f"selected must be a contiguous [{T}, {H}, topk] tensor")
    return t.data_ptr()


def kvq_sparse_attention_workspace(num_tokens: int, num_heads: int, num_q_heads: int, head_dim: int, block_size: int,
                                   topk: int) -> int:
    """Bytes that are enough at these sizes and at any smaller num_tokens and topk."""
    return int(_lib().kvq_sparse_attention_workspace(num_tokens, num_heads, num_q_heads, head_dim, block_size, topk))


def kvq_sparse_attention(pool: KvPool, block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                         q: torch.Tensor, query_starts: torch.Tensor, max_query_len: int, selected: torch.Tensor,
                         scale: float, out: torch.Tensor, *, softcap: float = 0.0,
                         workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """kvq_attention over the listed blocks alone: selected [T, H, topk] int32 as kvq_select_blocks
    writes it.  A workspace tensor is allocated when none is given."""
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    qi, oo = _bf16_in(q, "q"), _bf16_out(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ps = pool._struct()
    T, Hq, D = q.shape
    H = ps.num_heads
    if D != ps.head_dim:
        raise ValueError(f"q has head_dim {D}, the pool {ps.head_dim}")
    sel = _lists(selected, T, H)
    topk = selected.size(2)
    if workspace is None:
        need = int(_lib().kvq_sparse_attention_workspace_exact(T, H, Hq, D, pool.block_size, topk))
        if need > 0:
            workspace = _workspace(need, q.device, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().kvq_sparse_attention(
        ctypes.byref(ps), block_table.data_ptr(), S, max_blocks, _vec(seq_lens, torch.int32, "seq_lens", S),
        max_seq_len, ctypes.byref(qi), _vec(query_starts, torch.int32, "query_starts", S + 1), T, max_query_len, Hq,
        sel, topk, float(scale), float(softcap), ctypes.byref(oo), _ptr(workspace), nbytes, _ptr(dev_status),
        _stream(stream)))
    return out


def kvq_plan_pages(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_blocks: torch.Tensor, block_size: int,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, query_starts: torch.Tensor,
                   slot_ids: torch.Tensor, positions: Optional[torch.Tensor], num_used: torch.Tensor,
                   dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Block tables, slot maps and lengths of a step from request lengths (see include/kvq.h):
    block_table [S, max_blocks], seq_lens [S], query_starts [S + 1], slot_ids (int64) and
    positions [max_tokens] and num_used [1] are written."""
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous [S, max_blocks]")
    S, max_blocks = block_table.shape
    i32, n = torch.int32, slot_ids.numel()
    _check(_lib().kvq_plan_pages(
        _vec(cached_lens, i32, "cached_lens", S), _vec(new_lens, i32, "new_lens", S), S,
        _vec(free_blocks, i32, "free_blocks"), free_blocks.numel(), block_size, block_table.data_ptr(), max_blocks,
        _vec(seq_lens, i32, "seq_lens", S), _vec(query_starts, i32, "query_starts", S + 1),
        _vec(slot_ids, torch.int64, "slot_ids"), _vec(positions, i32, "positions", n), n,
        _vec(num_used, i32, "num_used", 1), _ptr(dev_status), _stream(stream)))


def kvq_storage_bytes(fmt: int, kind: int, group_size: int, rows: int, heads: int, dim: int) -> int:
    return int(_lib().kvq_storage_bytes(fmt, kind, group_size, rows, heads, dim))


def kvq_status_string(status: int) -> str:
    return _lib().kvq_status_string(status).decode()


def kvq_last_error() -> str:
    return _lib().kvq_last_error().decode()
