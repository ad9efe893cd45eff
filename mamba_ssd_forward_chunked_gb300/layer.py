"""The layer around ``ssd_fwd``, for serving: bindings of the calls that
``include/ssd.h`` describes under "The layer around ssd_fwd".

A prompt runs through ``ssd_conv_fwd`` and then ``ssd_fwd`` (or, with a decay
per channel and state, ``ssd_selective_scan``; or, with the delta rule,
``ssd_delta_fwd``); every further token through ``ssd_w4_matvec`` (the
projections), ``ssd_step`` (or the same calls as the prompt) and, for beam
search, ``ssd_beam_select`` and ``ssd_beam_reorder``.  With drafted tokens the
model runs on several at a time, ``ssd_draft_verify`` says how many hold, and
their number is the ``lengths`` with which the states are committed.

As in the rest of the package nothing is computed here: tensors are checked,
outputs that are not given are allocated, and the C entry point of the same
name runs on the current stream (or on ``stream``, which may be a
torch.cuda.Stream or a raw handle, of the tensors' device; the caller orders it
against the work that made the inputs).  Errors raise SSDError before anything
is enqueued.  The checks are compiled (csrc/binding.cpp), because a decoding
loop makes these calls for every layer and token.
"""
from __future__ import annotations

import importlib
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import SSDError


class _NoBinding:
    """In the compiled binding's place where it cannot be loaded: the rest of the
    package needs none of it, and the layer's calls have no other path."""

    def __init__(self, why: ImportError):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"the layer operators need _layer_binding.so, which cannot be loaded ({self._why}): build it "
                          "with `python mamba_ssd_forward_chunked_gb300/build_ext.py`") from self._why


try:
    _binding = importlib.import_module("._layer_binding", __package__)
except ImportError as why:
    _binding = _NoBinding(why)
else:
    _binding.set_error(SSDError)

__all__ = ["ssd_conv_fwd", "ssd_selective_scan", "ssd_step", "ssd_w4_matvec", "ssd_beam_select", "ssd_beam_reorder",
           "ssd_selective_scan_workspace_size", "ssd_beam_select_workspace_size", "w4_pack", "w4_quantize",
           "ssd_delta_fwd", "ssd_delta_workspace_size", "ssd_draft_verify", "ssd_draft_verify_workspace_size"]


def _on(stream, fn, *args):
    """fn(*args) with ``stream`` as the current stream of the tensors' device, so
    that the work runs there and the outputs it allocates belong to it."""
    device = next((t.device for t in args if isinstance(t, torch.Tensor)), None)
    if device is None or device.type != "cuda":
        return fn(*args)  # refused there
    if not hasattr(stream, "cuda_stream"):  # 0, the default stream, is not one for ExternalStream: it would be a new one
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        raise SSDError(1, f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return fn(*args)


# ------------------------------------------------------------------ convolution

def ssd_conv_fwd(u: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                 activation: Optional[str] = "silu", split: Optional[Sequence[int]] = None,
                 ring: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 lengths: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                 new_ring: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
                 stream=None) -> Union[torch.Tensor, Tuple[torch.Tensor, ...]]:
    """The short causal convolution (C: ssd_conv_fwd), for prompts (any length)
    and single tokens (length 1).

    u [B, L, C] float32 or bfloat16, its channels contiguous (a slice of the
    in-projection's output); weight [C, W] (W 2 to 4) and bias [C] float32.
    ``split`` gives the channels of two or three outputs, e.g. (H*64, G*N, G*N)
    for x, Bm and Cm as ssd_fwd takes them; without it there is one output.
    ``ring`` [slots, W, C] is the cache: the inputs of the last tokens, updated
    in place or written to ``new_ring`` (only the rows of this call's sequences).
    ``positions`` [B] int32 are the tokens before this call (0), ``lengths`` [B]
    int32 this call's tokens (L; outputs after them are 0), ``slots`` [B] int32
    the cache rows (the first B; a sequence whose row does not exist is idle)."""
    args = (u, weight, bias, activation, split, ring, positions, lengths, slots, new_ring, out)
    return _binding.conv_fwd(*args) if stream is None else _on(stream, _binding.conv_fwd, *args)


# ------------------------------------------------------------------ selective scan

def ssd_selective_scan_workspace_size(batch: int, seqlen: int, channels: int, dstate: int, ngroups: int) -> int:
    """Bytes of workspace ssd_selective_scan needs for these sizes on the current
    device (0: none)."""
    return _binding.scan_workspace(batch, seqlen, channels, dstate, ngroups)


def ssd_selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                       D: Optional[torch.Tensor] = None, *, z: Optional[torch.Tensor] = None,
                       delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                       init_state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, want_final_state: bool = True,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The recurrence with a decay per channel and state (C:
    ssd_selective_scan), for prompts and single tokens.  Returns (y, final_state).

    u, delta, z [B, L, D] and Bm, Cm [B, L, G, N] share float32 or bfloat16 and
    may be slices of wider rows; A [D, N], D [D], delta_bias [D], init_state and
    final_state [B, D, N] are float32 (N 1 to 64).  final_state may be
    init_state.  ``lengths`` [B] int32: tokens of each sequence."""
    args = (u, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus, init_state, lengths, y, final_state, workspace,
            want_final_state)
    return _binding.selective_scan(*args) if stream is None else _on(stream, _binding.selective_scan, *args)


# ------------------------------------------------------------------ single token

def ssd_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, D: torch.Tensor, weight: torch.Tensor,
             bias: Optional[torch.Tensor], state: torch.Tensor, ring: torch.Tensor, positions: torch.Tensor, *,
             ngroups: int = 1, z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
             dt_softplus: bool = False, slots: Optional[torch.Tensor] = None,
             new_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of a Mamba-2 layer's convolution and recurrence for every
    sequence (C: ssd_step).  Returns y [B, H, 64].

    u [B, H*64 + 2*G*N] (x, B and C before the convolution), z [B, H*64] (the
    gate) and dt [B, H] may be slices of one projection's output; dt may also be
    float32 beside bfloat16 u.  A, D, dt_bias [H], weight [C, W], bias [C] and
    state [slots, H, 64, N] are float32; ring [slots, W, C] has u's type.  ring
    and state are updated in place, or the state goes to ``new_state`` (only the
    rows of this call are written).  ``positions`` [B] int32: tokens before this
    one; ``slots`` [B] int32: cache rows (a row that does not exist: idle)."""
    args = (u, dt, A, D, weight, bias, state, ring, positions, ngroups, z, dt_bias, dt_softplus, slots, new_state, y)
    return _binding.step(*args) if stream is None else _on(stream, _binding.step, *args)


# ------------------------------------------------------------------ delta rule

def ssd_delta_workspace_size(batch: int, seqlen: int, nheads: int, headdim: int, dstate: int, dtype: torch.dtype,
                             ngroups: int = 1) -> int:
    """Bytes of workspace ssd_delta_fwd needs for these sizes on the current
    device (0: none; about 1 GB at most, however large the batch)."""
    return _binding.delta_workspace(batch, seqlen, nheads, headdim, ngroups, dstate, dtype == torch.bfloat16)


def ssd_delta_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                  beta: torch.Tensor, *, scale: Optional[float] = None, dt_bias: Optional[torch.Tensor] = None,
                  dt_softplus: bool = False, beta_sigmoid: bool = False, norm_eps: Optional[float] = None,
                  init_state: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, want_final_state: bool = True,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gated delta rule (C: ssd_delta_fwd), for prompts, a few drafted tokens
    and single tokens.  Returns (y, final_state).

    x [B, L, H, P] (P a multiple of 16), Bm and Cm [B, L, G, N] (N 64, 128 or
    256) share float32 or bfloat16 and may be slices of wider rows; dt and beta
    [B, L, H] have that type or float32.  A, dt_bias [H] and the states
    [slots, H, P, N] are float32.  ``scale`` is 1/sqrt(N) unless given;
    ``norm_eps`` normalises the rows of Bm and Cm.  ``slots`` [B] int32 are the
    rows of the states (the first B; a sequence whose row does not exist is
    idle), ``positions`` [B] int32 the tokens before this call (a sequence at 0
    starts from a state of 0), ``lengths`` [B] int32 this call's tokens (L;
    outputs after them are 0).  final_state may be init_state; with ``slots`` it
    has to be given (or ``want_final_state=False``)."""
    args = (x, dt, A, Bm, Cm, beta, scale, dt_bias, dt_softplus, beta_sigmoid, norm_eps, init_state, slots, positions,
            lengths, y, final_state, workspace, want_final_state)
    return _binding.delta_fwd(*args) if stream is None else _on(stream, _binding.delta_fwd, *args)


# ------------------------------------------------------------------ 4-bit weights

def w4_pack(codes: torch.Tensor) -> torch.Tensor:
    """4-bit codes [n, k] (values 0 to 15, others are refused; a weight is (code - 8) * scale) in the
    order ssd_w4_matvec reads, int32 [ceil(n/16), ceil(k/64), 32, 4].  Done once
    per weight, on any device."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.is_floating_point():
        raise SSDError(1, "codes must be a 2-D tensor of whole numbers")
    n, k = codes.shape
    rows, cols = -(-n // 16), -(-k // 64)
    full = codes.new_full((rows * 16, cols * 64), 8, dtype=torch.int64)
    full[:n, :k] = codes
    if codes.numel() and not 0 <= int(full.min()) <= int(full.max()) <= 15:  # (others would change their neighbours)
        raise SSDError(1, f"codes from {int(full.min())} to {int(full.max())}, expected 0 to 15")
    # [row tile, a, r, column tile, h, c, i, e, p] -> [row tile, column tile, r, c, h, i, e, a, p]
    v = full.view(rows, 2, 8, cols, 2, 4, 2, 2, 2).permute(0, 3, 2, 5, 4, 6, 7, 1, 8)
    e, a, p = torch.meshgrid(*[torch.arange(2, device=codes.device)] * 3, indexing="ij")
    words = (v << (4 * (a + 2 * e) + 16 * p)).sum(dim=(-3, -2, -1))
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    return words.to(torch.int32).reshape(rows, cols, 32, 4)


def w4_quantize(weight: torch.Tensor, group: int = 128) -> Tuple[torch.Tensor, torch.Tensor]:
    """(packed codes, scales) of a weight [n, k] for ssd_w4_matvec: per row and
    group of columns the scale that puts the largest magnitude at 7.  Weights that
    are not finite are refused."""
    if group not in (32, 64, 128):
        raise SSDError(2, f"group {group}, expected 32, 64 or 128")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise SSDError(1, "weight must be a 2-D tensor")
    n, k = weight.shape
    groups = -(-k // group)
    w = weight.new_zeros((n, groups * group), dtype=torch.float32)
    w[:, :k] = weight
    w = w.view(n, groups, group)
    scales = w.abs().amax(-1) / 7.0
    if not bool(torch.isfinite(scales).all()):
        raise SSDError(1, "weight must be finite")
    codes = torch.round(w / torch.where(scales > 0, scales, 1.0)[..., None]).clamp_(-7, 7) + 8
    return w4_pack(codes.view(n, groups * group)[:, :k].to(torch.int64)), scales


def ssd_w4_matvec(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int, *,
                  add: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x W^T (+ add) for a few tokens and a 4-bit W (C: ssd_w4_matvec).

    x [M, k] and add [M, n] float32 or bfloat16 (rows may be strided); ``packed``
    from w4_pack, ``scales`` [n, ceil(k/group)] float32, group 32, 64 or 128.  float32 x, and rows that
    are not 16-byte vectors, take a workspace of 2 bytes for each of x's (or its three parts') values."""
    args = (x, packed, scales, group, add, y, workspace)
    return _binding.w4_matvec(*args) if stream is None else _on(stream, _binding.w4_matvec, *args)


# ------------------------------------------------------------------ beam search

def ssd_beam_select_workspace_size(batch: int, beams: int, vocab: int, k: int) -> int:
    """Bytes of workspace ssd_beam_select needs for these sizes on the current device."""
    return _binding.select_workspace(batch, beams, vocab, k)


def ssd_beam_select(logits: torch.Tensor, scores: torch.Tensor, k: int, *, finished: Optional[torch.Tensor] = None,
                    eos: int = -1, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The k best continuations of every request's beams (C: ssd_beam_select).
    Returns (scores float32, parents int32, tokens int32), each [B, k].

    logits [B, W, V] float32 or bfloat16 (rows may be strided), scores [B, W]
    float32 the beams' log-probabilities, ``finished`` [B, W] bool the beams that
    only go on with ``eos`` at their present score."""
    args = (logits, scores, k, finished, eos, workspace)
    return _binding.beam_select(*args) if stream is None else _on(stream, _binding.beam_select, *args)


def ssd_beam_reorder(states: Sequence[torch.Tensor], parents: torch.Tensor, *,
                     out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> List[torch.Tensor]:
    """Row b*k + i of every state becomes row b*W + parents[b, i] (C:
    ssd_beam_reorder).  ``states``: contiguous tensors of any type with the same
    number of rows B*W; ``parents`` [B, k] int32.  In place without ``out`` (then
    k must be W); otherwise into ``out``, tensors of B*k rows.  Returns the
    reordered tensors."""
    args = (states, parents, out)
    return _binding.beam_reorder(*args) if stream is None else _on(stream, _binding.beam_reorder, *args)


# ------------------------------------------------------------------ drafted tokens

def ssd_draft_verify_workspace_size(batch: int, drafts: int, vocab: int, dtype: torch.dtype, draft_logits: bool) -> int:
    """Bytes of workspace ssd_draft_verify needs for these sizes on the current device."""
    return _binding.verify_workspace(batch, drafts, vocab, dtype == torch.bfloat16, draft_logits)


def ssd_draft_verify(logits: torch.Tensor, draft: torch.Tensor, uniforms: torch.Tensor, *,
                     draft_logits: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                     lengths: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """How many drafted tokens the target's probabilities accept, and the token
    after them (C: ssd_draft_verify).  Returns (tokens [B, T+1] int32: the
    accepted drafts, the drawn token, then -1; accepted [B] int32; log-probabilities
    [B, T+1] float32 of the tokens).

    logits [B, T+1, V] and ``draft_logits`` [B, T, V] float32 or bfloat16 (rows
    may be strided) are the target's and the draft model's; without the latter
    the drafts count as certain.  draft [B, T] int32, uniforms [B, T+1] float32 in
    [0, 1) (one for every draft, the last for the drawn token), ``scale`` [B]
    float32 the inverse temperatures (1), ``lengths`` [B] int32 the drafts of each
    sequence (T)."""
    args = (logits, draft, uniforms, draft_logits, scale, lengths, workspace)
    return _binding.draft_verify(*args) if stream is None else _on(stream, _binding.draft_verify, *args)
