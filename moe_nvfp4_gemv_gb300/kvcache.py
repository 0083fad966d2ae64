"""A paged key/value cache held in 8 bits, and attention over it.

``KvCache8`` wraps the four tensors of a cache -- codes uint8 [num_blocks,
kv_heads, block_size, head_dim] and fp32 scales [num_blocks, kv_heads], keys
and values apart (the formats: include/fp4gemv_decode.h) -- with the calls
of a decode step:

* ``append``: quantises new keys and values into the pages that the block
  table names; a page's scale grows with what it holds;
* ``attend``: attention of each sequence's newest tokens over its pages;
* ``attend_shared``: the same for sequences that begin alike, their beginning
  read and multiplied once;
* ``read``: tokens out of the pages again.

The tensors stay the caller's: copy, share or reset pages as the serving
program likes, between calls on the same stream.  Sequences are given by a
block table (int32 [B, max_blocks], page ids) and their lengths (int32 [B],
new tokens included), both on the device, so a step of any lengths is one
captured graph.  Like the rest of the binding the calls only marshal
arguments; they run on the current stream and raise ``Fp4GemvError`` on a
refused argument.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .fp4gemv import Fp4GemvError, _lib, _marshal, _raw_stream

FORMATS = {"e4m3": 0, "int8": 1}
_F32 = torch.float32
_append = _marshal.kv_append
_attend = _marshal.kv_attention
_attend_sinks = _marshal.kv_attention_sinks
_attend_shared = _marshal.kv_attention_shared
_read = _marshal.kv_read


class _CacheStruct(ctypes.Structure):
    """fp4gemv_kv_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("block_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("format", ctypes.c_int)]


_workspaces: dict = {}  # (device, stream, head_dim): the workspace
_captured: dict = {}    # the same: (capture, its workspace) of the last capture without one of the above


def attention_workspace_bytes(head_dim: int) -> int:
    """Bytes of ``attend``'s workspace on the current device."""
    return int(_lib.fp4gemv_kv_attention_workspace_bytes(head_dim))


def attention_workspace(device: torch.device, head_dim: int, stream: int | None = None) -> torch.Tensor:
    """A zero-filled workspace for ``device`` and one CUDA stream (the current
    one when ``stream`` is None), kept for later calls: calls on one stream
    run one after another and may share it, calls on different streams may
    overlap and each stream has its own.

    While the stream is being captured and has none yet, the capture gets one
    of its own, which its graph clears whenever it runs.  A graph captured on a
    stream that has one uses that one: such graphs may not run at the same time
    as each other or as that stream's calls (give them a ``workspace`` each)."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    current = _raw_stream(index)
    if stream is None:
        stream = current
    key = (index, stream, head_dim)
    ws = _workspaces.get(key)
    if ws is not None:
        return ws
    capture = _lib.fp4gemv_stream_capture_id(stream)
    last = _captured.get(key)
    if capture and last is not None and last[0] == capture:
        return last[1]
    on = contextlib.nullcontext()
    if stream != current:  # (cleared on the stream that it is for)
        on = torch.cuda.stream(torch.cuda.ExternalStream(stream, index) if stream else torch.cuda.default_stream(index))
    with torch.cuda.device(index), on:
        ws = torch.zeros(attention_workspace_bytes(head_dim), dtype=torch.uint8, device=device)
    if capture:
        _captured[key] = (capture, ws)
    else:
        _workspaces[key] = ws
    return ws


class KvCache8:
    """The cache's tensors and their calls.  ``fmt``: "e4m3" or "int8".

    The calls use the tensors' memory as it was given: write into them in
    place; other tensors make another cache."""

    def __setattr__(self, name, value):
        if name in ("k_codes", "v_codes", "k_scale", "v_scale") and name in self.__dict__:
            raise AttributeError(f"{name} is the memory that the calls use: write into it, or make another cache")
        super().__setattr__(name, value)

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 fmt: str = "e4m3"):
        if fmt not in FORMATS:
            raise ValueError(f"fmt must be 'e4m3' or 'int8', not {fmt!r}")
        if k_codes.dim() != 4:
            raise ValueError("codes must be [num_blocks, kv_heads, block_size, head_dim]")
        for name, t, dtype, shape in (("k_codes", k_codes, torch.uint8, k_codes.shape),
                                      ("v_codes", v_codes, torch.uint8, k_codes.shape),
                                      ("k_scale", k_scale, _F32, k_codes.shape[:2]),
                                      ("v_scale", v_scale, _F32, k_codes.shape[:2])):
            if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != k_codes.device:
                raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on the codes' device")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.fmt = fmt
        self.device = k_codes.device
        self._index = k_codes.get_device()
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = k_codes.shape
        self._struct = _CacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                    self.num_blocks, self.kv_heads, self.block_size, self.head_dim, FORMATS[fmt])
        self._handle = ctypes.addressof(self._struct)
        self._sm_scale = 1.0 / math.sqrt(self.head_dim)
        self._scratch = {}  # (batch, q_len, heads): bytes of attend_shared's scratch

    @classmethod
    def allocate(cls, num_blocks: int, kv_heads: int, head_dim: int, block_size: int = 64, fmt: str = "e4m3",
                 device: torch.device | str = "cuda") -> "KvCache8":
        """A cache of zeroed pages."""
        shape = (num_blocks, kv_heads, block_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(shape[:2], dtype=_F32, device=device) for _ in range(2)]
        return cls(*codes, *scales, fmt=fmt)

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               cu_new: torch.Tensor | None = None, pdl: bool = True) -> None:
        """Appends k, v (bf16 or f16 [T, kv_heads, head_dim], heads contiguous,
        any token stride that is a multiple of 8) to B sequences: T / B tokens
        each, or tokens cu_new[b] .. cu_new[b + 1] (int32 [B + 1]) to sequence
        b.  ``seq_lens``: the lengths with the new tokens."""
        status = _append(self._handle, self._index, self.kv_heads, self.head_dim, k, v, block_table, seq_lens, cu_new,
                         pdl)
        if status:
            raise Fp4GemvError(status, "fp4gemv_kv_append")

    def read(self, block_table: torch.Tensor, seq_lens: torch.Tensor, tokens: int | None = None,
             cu: torch.Tensor | None = None, k: torch.Tensor | None = None, v: torch.Tensor | None = None,
             dtype: torch.dtype = torch.bfloat16, pdl: bool = True) -> tuple[torch.Tensor, torch.Tensor]:
        """The last tokens of B sequences out of the cache: (k, v) [T, kv_heads,
        head_dim], code * scale rounded to ``dtype`` (bf16, f16 or fp32).  T / B
        tokens of each, or rows cu[b] .. cu[b + 1] (int32 [B + 1]) of sequence
        b, that end at position seq_lens[b]; rows that ``cu`` does not name stay
        as they are.  ``tokens`` is T; or ``k`` and ``v`` (any token stride that
        is a multiple of 16 bytes, heads contiguous) receive them."""
        if (k is None) != (v is None) or (k is None) == (tokens is None):
            raise ValueError("either tokens, or both k and v")
        if k is None:
            shape = (tokens, self.kv_heads, self.head_dim)
            k, v = (torch.empty(shape, dtype=dtype, device=self.device) for _ in range(2))
        status = _read(self._handle, self._index, self.kv_heads, self.head_dim, block_table, seq_lens, cu, k, v, pdl)
        if status:
            raise Fp4GemvError(status, "fp4gemv_kv_read")
        return k, v

    def attend(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: float | None = None,
               window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, pdl: bool = True, sinks: int = 0) -> torch.Tensor:
        """Attention of q (bf16 or f16 [B, q_len, heads, head_dim], the newest
        q_len tokens of every sequence, already appended; tokens at one stride
        that is a multiple of 8, heads contiguous).  Query i sees tokens up to
        its own position, the last ``window`` of them if that is not 0 and the
        sequence's first ``sinks`` as well; one that sees none gives zeros.  ``sm_scale`` defaults to 1 /
        sqrt(head_dim); ``lse``: fp32 [B, q_len, heads] to receive the natural
        log of the softmax's sums; ``workspace``: uint8, zero-filled once, of
        attention_workspace_bytes(head_dim), the stream's own by default
        (``attention_workspace``; captured calls too).  Returns ``out``."""
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        if workspace is None:
            stream = _raw_stream(self._index)
            workspace = _workspaces.get((self._index, stream, self.head_dim))
            if workspace is None:
                workspace = attention_workspace(self.device, self.head_dim, stream)
        if sm_scale is None:
            sm_scale = self._sm_scale
        if sinks:
            status = _attend_sinks(self._handle, self._index, self.head_dim, q, block_table, seq_lens, sm_scale, window,
                                   out, lse, workspace, pdl, sinks)
            if status:
                raise Fp4GemvError(status, "fp4gemv_kv_attention_sinks")
            return out
        status = _attend(self._handle, self._index, self.head_dim, q, block_table, seq_lens, sm_scale, window, out, lse,
                         workspace, pdl)
        if status:
            raise Fp4GemvError(status, "fp4gemv_kv_attention")
        return out

    def attend_shared(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      prefix_len: torch.Tensor, sm_scale: float | None = None, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      scratch: torch.Tensor | None = None, always: bool = False, pdl: bool = True) -> torch.Tensor:
        """``attend`` of sequences whose first ``prefix_len`` tokens (int32 [1],
        device) are the same: every sequence's row of the block table names
        pages with that beginning, usually the same ones, and what fills whole
        pages of it is read and multiplied once for all.  (In multiples of 128
        tokens, and no further than the first query of the shortest sequence;
        empty sequences do not count.)  Batches of few tokens are attended to one
        by one, which is faster, unless ``always``; how many is judged by the block
        table's width, so cut a table that is much wider than the lengths (a view of
        its first columns, made contiguous), and call ``attend`` for a beginning
        that is short beside the sequences' own tokens.  ``scratch``: uint8, of
        ``shared_scratch_bytes``, allocated for the call by default."""
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        if workspace is None:
            stream = _raw_stream(self._index)
            workspace = _workspaces.get((self._index, stream, self.head_dim))
            if workspace is None:
                workspace = attention_workspace(self.device, self.head_dim, stream)
        if scratch is None:
            sizes = tuple(q.shape[:3])
            nbytes = self._scratch.get(sizes)
            if nbytes is None:
                nbytes = self._scratch[sizes] = self.shared_scratch_bytes(*sizes) if len(sizes) == 3 else 0
            scratch = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        status = _attend_shared(self._handle, self._index, self.head_dim, q, block_table, seq_lens,
                                self._sm_scale if sm_scale is None else sm_scale, 0, out, lse, workspace, pdl,
                                prefix_len, scratch, always)
        if status:
            raise Fp4GemvError(status, "fp4gemv_kv_attention_shared")
        return out

    def shared_scratch_bytes(self, batch: int, q_len: int, heads: int) -> int:
        """Bytes of ``attend_shared``'s scratch on the cache's device (0 for sizes that it refuses)."""
        with torch.cuda.device(self._index):
            return int(_lib.fp4gemv_kv_attention_shared_scratch_bytes(self.kv_heads, self.head_dim, heads, q_len, batch))
