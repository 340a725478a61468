"""The attention sub-layer of a decoding step and of a prompt, on top of the C ABI.

``PagedCache`` wraps two page pools (``gqa_append``, ``gqa_paged_attention``,
``gqa_prompt_attention``); ``AttentionLayer`` puts int4 projections
(``moe.linear``, ``moe.linear_prompt``) around it, and its result is the
``attn`` of ``PackedLayer.decode_batch_block`` and ``PackedLayer.prefill_block``.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib
from .moe import QMatrix, linear, linear_prompt


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


class PagedCache:
    """A paged key-value cache over two pools [n_pages, Hkv, page_size, D] in
    bf16 (any order of heads and positions in memory: pass a transposed view;
    both pools in the same layout).  The pools stay the caller's."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _need(k.dim() == 4 and k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16 and k.shape == v.shape,
              "PagedCache: two bf16 pools [n_pages, Hkv, page_size, D]")
        _need(k.stride() == v.stride() and k.stride(3) == 1, "PagedCache: both pools in one layout, D innermost")
        _need(k.device == v.device, "PagedCache: both pools on one device")
        self.k, self.v = k, v
        self.n_pages, self.Hkv, self.page_size, self.D = k.shape
        # a dimension of size 1 has no stride of its own
        page, head, pos = (s if n > 1 else self.D for s, n in zip(k.stride(), k.shape[:3]))
        self.desc = _lib.gqa_pages(k.data_ptr(), v.data_ptr(), self.n_pages, self.page_size, self.Hkv, self.D, page,
                                   head, pos)
        self._device = k.get_device()
        # where append, attend without a workspace and the projections of a
        # decoding step record errors found on the device (moe_read_device_status)
        self.status = torch.zeros(4, dtype=torch.int32, device=k.device)
        self._at, self._status_at = ctypes.addressof(self.desc), self.status.data_ptr()
        self._scale = 1.0 / math.sqrt(self.D)

    @classmethod
    def empty(cls, n_pages: int, Hkv: int, page_size: int, D: int, device="cuda") -> "PagedCache":
        pool = torch.empty(2, n_pages, Hkv, page_size, D, dtype=torch.bfloat16, device=device)
        return cls(pool[0], pool[1])

    def append(self, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, seq: torch.Tensor,
               index: torch.Tensor, page_table: torch.Tensor, inv_freq: Optional[torch.Tensor], pos_offset: int = 0,
               interleaved: bool = False, q_out: Optional[torch.Tensor] = None, stream=None):
        """Rotate q and k by position index + pos_offset, write k and v to
        position index[t] of sequence seq[t]; returns the rotated q."""
        if stream is not None and q is not None and q_out is None:
            with _lib.on_stream(stream):
                return self.append(q, k, v, seq, index, page_table, inv_freq, pos_offset, interleaved)
        if q_out is None and q is not None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rc = _lib.native().append(self._at, self._device, self._status_at, q, k, v, seq, index, page_table, inv_freq,
                                  pos_offset, interleaved, q_out, _lib.handle(stream))
        if rc:
            raise _lib.MoEError(rc, "gqa_append")
        return q_out

    def workspace(self, B: int, Hq: int, prefix_len: int = 0) -> torch.Tensor:
        """Scratch of attend for up to B rows, Hq heads and prefix_len shared
        positions; calls that may overlap take one each."""
        return torch.zeros(self._workspace_bytes(B, Hq, prefix_len), dtype=torch.uint8, device=self.k.device)

    def _workspace_bytes(self, B: int, Hq: int, prefix_len: int) -> int:
        n = _lib.gqa_paged_workspace_bytes(B, Hq, self.Hkv, self.D, prefix_len)
        if n == 0:
            raise _lib.MoEError(_lib.MOE_ERR_SHAPE, "gqa_paged_workspace_bytes")
        return n

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor,
               prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """out [B, Hq, D]: row b's query attends to the shared prefix (read
        once for all rows), then to the first seq_len[b] positions of
        page_table[b].  scale: 1 / sqrt(D) unless given.  Errors found on the
        device are recorded in the first word of ws, without ws (scratch of the
        call's own is then allocated) in `status`."""
        if stream is not None and (out is None or ws is None):
            with _lib.on_stream(stream):
                return self.attend(q, page_table, seq_len, prefix_pages, prefix_len, scale, out, ws)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        status = None
        if ws is None:
            ws = torch.empty(self._workspace_bytes(q.shape[0], q.shape[1], prefix_len), dtype=torch.uint8,
                             device=self.k.device)
            status = self._status_at
        rc = _lib.native().attend(self._at, self._device, q, page_table, seq_len, prefix_pages, prefix_len,
                                  self._scale if scale is None else scale, out, ws, _lib.handle(stream), status)
        if rc:
            raise _lib.MoEError(rc, "gqa_paged_attention")
        return out


    def prompt_workspace(self, T: int, n_seq: int, Hq: int) -> torch.Tensor:
        """Scratch of attend_prompt for up to T rows of n_seq sequences; calls
        that may overlap take one each."""
        return torch.zeros(self._prompt_bytes(T, n_seq, Hq), dtype=torch.uint8, device=self.k.device)

    def _prompt_bytes(self, T: int, n_seq: int, Hq: int) -> int:
        n = _lib.gqa_prompt_workspace_bytes(T, n_seq, Hq, self.Hkv, self.D)
        if n == 0:
            raise _lib.MoEError(_lib.MOE_ERR_SHAPE, "gqa_prompt_workspace_bytes")
        return n

    def attend_prompt(self, q: torch.Tensor, q_start: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor,
                      prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0, scale: Optional[float] = None,
                      out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """out [T, Hq, D]: causal attention of packed sequences.  Rows
        q_start[b] .. q_start[b + 1] - 1 of q are the last tokens of sequence b,
        whose first seq_len[b] positions are in page_table[b] (their own among
        them): each attends to the shared prefix and its sequence's positions up
        to its own.  scale: 1 / sqrt(D) unless given.  Errors found on the device
        are recorded in the first word of ws, without ws (scratch of the call's own
        is then allocated) in `status`."""
        if stream is not None and (out is None or ws is None):
            with _lib.on_stream(stream):
                return self.attend_prompt(q, q_start, page_table, seq_len, prefix_pages, prefix_len, scale, out, ws)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        status = None
        if ws is None:
            ws = torch.empty(self._prompt_bytes(q.shape[0], seq_len.shape[0], q.shape[1]), dtype=torch.uint8,
                             device=self.k.device)
            status = self._status_at
        rc = _lib.native().attend_prompt(self._at, self._device, q, q_start, page_table, seq_len, prefix_pages,
                                         prefix_len, self._scale if scale is None else scale, out, ws,
                                         _lib.handle(stream), status)
        if rc:
            raise _lib.MoEError(rc, "gqa_prompt_attention")
        return out


class AttentionLayer:
    """int4 projections around a paged cache: qkv [(Hq + 2 Hkv) D, H] and
    out [H, Hq D], both QMatrix (pack_matrix), and the rotation."""

    def __init__(self, qkv: QMatrix, out: QMatrix, Hq: int, Hkv: int, D: int, inv_freq: Optional[torch.Tensor],
                 interleaved: bool = False):
        _need(qkv.rows == (Hq + 2 * Hkv) * D and out.K == Hq * D and out.rows == qkv.K, "AttentionLayer: shapes")
        self.qkv, self.out, self.Hq, self.Hkv, self.D = qkv, out, Hq, Hkv, D
        self.inv_freq, self.interleaved = inv_freq, interleaved

    def project(self, x: torch.Tensor, stream=None, status: Optional[torch.Tensor] = None):
        """Queries, keys and values [T, heads, D] of 1 to 64 tokens (views of one buffer).
        status: as for moe.linear (a cache's `status`, for instance)."""
        return self._split(linear(self.qkv, x, status=status, stream=stream))

    def _split(self, y: torch.Tensor):
        y = y.view(y.shape[0], self.Hq + 2 * self.Hkv, self.D)
        return y[:, :self.Hq], y[:, self.Hq:self.Hq + self.Hkv], y[:, self.Hq + self.Hkv:]

    def decode(self, x: torch.Tensor, cache: PagedCache, seq: torch.Tensor, index: torch.Tensor,
               page_table: torch.Tensor, seq_len: torch.Tensor, ws: torch.Tensor,
               prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0, stream=None) -> torch.Tensor:
        """One step of B rows: x [B, H] (normalised) -> attn [B, H].  Row b's
        new token goes to position index[b] of page table row seq[b]; it
        attends to the prefix and the first seq_len[b] positions of row b
        (seq_len = index + 1 for a plain step; both negative: padding, whose
        attn row means nothing).  1 to 64 rows.  Errors found on the device are
        recorded in cache.status, the attention's in the first word of ws."""
        if stream is not None:
            with _lib.on_stream(stream):
                return self.decode(x, cache, seq, index, page_table, seq_len, ws, prefix_pages, prefix_len)
        qkv = linear(self.qkv, x, status=cache.status)
        q, k, v = self._split(qkv)
        # queries, rotated queries and the attention's output share their place
        cache.append(q, k, v, seq, index, page_table, self.inv_freq, prefix_len, self.interleaved, q_out=q)
        cache.attend(q, page_table, seq_len, prefix_pages, prefix_len, out=q, ws=ws)
        return linear(self.out, qkv[:, :self.Hq * self.D], status=cache.status)

    def prefill(self, x: torch.Tensor, cache: PagedCache, seq: torch.Tensor, index: torch.Tensor,
                q_start: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor,
                prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Packed prompts (or pieces of them): x [T, H] (normalised) -> attn
        [T, H], which PackedLayer.prefill_block takes.  Token t goes to position
        index[t] of page table row seq[t]; rows q_start[b] .. q_start[b + 1] - 1
        are the last tokens of sequence b, of seq_len[b] positions with them
        (attend_prompt; ws is its workspace).  Errors found on the device are
        recorded in cache.status, the attention's in the first word of ws if it is given."""
        if stream is not None:
            with _lib.on_stream(stream):
                return self.prefill(x, cache, seq, index, q_start, page_table, seq_len, prefix_pages, prefix_len, ws)
        qkv = linear_prompt(self.qkv, x, status=cache.status)
        q, k, v = self._split(qkv)
        # queries, rotated queries and the attention's output share their place
        cache.append(q, k, v, seq, index, page_table, self.inv_freq, prefix_len, self.interleaved, q_out=q)
        cache.attend_prompt(q, q_start, page_table, seq_len, prefix_pages, prefix_len, out=q, ws=ws)
        return linear_prompt(self.out, qkv[:, :self.Hq * self.D], status=cache.status)
