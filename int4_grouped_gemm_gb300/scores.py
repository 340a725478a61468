"""What is read from an output head's scores, on top of the C ABI.

``token_logprobs`` gives the log probabilities of given tokens, the entropy and
the most probable alternatives of rows of scores; ``OutputHead`` makes the
scores from hidden states on an int4 head, a piece of the rows at a time.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .moe import QMatrix, linear_prompt, linear_prompt_workspace


class TokenScores(NamedTuple):
    logprob: Optional[torch.Tensor]   # fp32 [T], of the given tokens (None without targets)
    entropy: torch.Tensor             # fp32 [T]
    top_ids: torch.Tensor             # int32 [T, n_top], most probable first, equal scores by lower id
    top_logprobs: torch.Tensor        # fp32 [T, n_top]

    @classmethod
    def empty(cls, T: int, n_top: int, targets: bool = True, device="cuda") -> "TokenScores":
        f = dict(dtype=torch.float32, device=device)
        return cls(torch.empty(T, **f) if targets else None, torch.empty(T, **f),
                   torch.empty(T, n_top, dtype=torch.int32, device=device), torch.empty(T, n_top, **f))

    def rows(self, a: int, b: int) -> "TokenScores":
        return TokenScores(*(None if t is None else t[a:b] for t in self))


def _bytes(T: int, V: int, n_top: int) -> int:
    n = _lib.token_logprobs_workspace_bytes(T, V, n_top)
    if n == 0:
        raise _lib.MoEError(_lib.MOE_ERR_SHAPE, "token_logprobs_workspace_bytes")
    return n


def workspace(T: int, V: int, n_top: int, device="cuda") -> torch.Tensor:
    """Scratch of token_logprobs for up to T rows of V scores; calls that may overlap
    take one each.  Its first word records errors found on the device
    (moe_read_device_status) unless the call is given a status."""
    return torch.zeros(_bytes(T, V, n_top), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, n_top: int = 0,
                   out: Optional[TokenScores] = None, ws: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> TokenScores:
    """Of logits [T, V] (fp32 or bf16): the log probabilities of targets (int32
    [T]; a row with a negative one is padding, its results are left as they
    were in out, and without out NaN, ids -1), the entropy, and the n_top (up to 32)
    most probable tokens.  status: a zeroed int32 device tensor for errors found on
    the device (a target outside the vocabulary); without it they go to the first
    word of ws, or nowhere if ws is not given either."""
    if stream is not None and (out is None or ws is None):
        with _lib.on_stream(stream):
            return token_logprobs(logits, targets, n_top, out, ws, status)
    if ws is None and logits.dim() != 2:
        raise ValueError("token_logprobs: logits [T, V]")
    if out is not None:
        _write(logits, targets, n_top, out, ws, status, stream)
        return out
    rc, *made = _lib.native().scores_new(logits, targets, n_top, ws, status, None)
    if rc:
        raise _lib.MoEError(rc, "token_logprobs")
    return TokenScores._make(made)


def _write(logits, targets, n_top, out, ws, status, stream=None, fill=False):
    """fill: out holds nothing yet."""
    rc = _lib.native().scores(logits, targets, out.logprob, out.entropy, n_top, out.top_ids, out.top_logprobs, ws,
                              status, _lib.handle(stream), fill)
    if rc:
        raise _lib.MoEError(rc, "token_logprobs")


class OutputHead:
    """An int4 output head [V, H] (pack_matrix) and what its scores say."""

    def __init__(self, w: QMatrix, rows: int = 1024):
        """rows: tokens whose fp32 scores are held at a time."""
        if rows < 1:
            raise ValueError("OutputHead: rows >= 1")
        self.w, self.rows = w, rows
        # where logprobs records errors found on the device if it is given no status
        # (moe_read_device_status)
        self.status = torch.zeros(4, dtype=torch.int32, device=w.q.device)

    def logprobs(self, x: torch.Tensor, targets: Optional[torch.Tensor] = None, n_top: int = 0,
                 status: Optional[torch.Tensor] = None, stream=None) -> TokenScores:
        """token_logprobs of x [T, H] (bf16, normalised) times the head, fp32
        scores: the scores of a prompt's tokens are those of the next ones, so
        that targets[t] is the token after token t (negative: padding, whose results
        are NaN, ids -1).  Errors found on the device are recorded in status, a zeroed
        int32 device tensor, or without it in `self.status`."""
        if stream is not None:
            with _lib.on_stream(stream):
                return self.logprobs(x, targets, n_top, status)
        T, V = x.shape[0], self.w.rows
        if targets is not None and targets.shape != (T,):
            raise ValueError(f"OutputHead: targets [{T}], a token for each row of x")
        status = self.status if status is None else status
        n = max(1, min(T, self.rows))
        nbytes = _bytes(n, V, n_top)  # (refuses what there cannot be)
        out = TokenScores.empty(T, n_top, targets is not None, x.device)
        if T == 0:
            return out
        # one piece after another, in the same scratch
        y = torch.empty(n, V, dtype=torch.float32, device=x.device)
        lin_ws = linear_prompt_workspace(self.w, n)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        for a in range(0, T, n):
            b = min(T, a + n)
            linear_prompt(self.w, x[a:b], y[:b - a], ws=lin_ws, status=status)
            _write(y[:b - a], None if targets is None else targets[a:b], n_top, out.rows(a, b), ws, status, fill=True)
        return out
