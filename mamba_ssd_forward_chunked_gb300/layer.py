"""The layer around ``ssd_fwd``, for serving: bindings of the calls that
``include/ssd.h`` describes under "The layer around ssd_fwd".

A prompt runs through ``ssd_conv_fwd`` and then ``ssd_fwd`` (or, with a decay
per channel and state, ``ssd_selective_scan``); every further token through
``ssd_w4_matvec`` (the projections), ``ssd_step`` and, for beam search,
``ssd_beam_select`` and ``ssd_beam_reorder``.

As in the rest of the package nothing is computed here: tensors are checked,
outputs that are not given are allocated, and the C entry point of the same
name runs on the current stream (or on ``stream``, which may be a
torch.cuda.Stream or a raw handle; the caller orders it against the work that
made the inputs).  Errors raise SSDError before anything is enqueued.
"""
from __future__ import annotations

import functools
import struct
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import SSD_BF16, SSD_F32, SSDError, lib

__all__ = ["ssd_conv_fwd", "ssd_selective_scan", "ssd_step", "ssd_w4_matvec", "ssd_beam_select", "ssd_beam_reorder",
           "ssd_selective_scan_workspace_size", "ssd_beam_select_workspace_size", "w4_pack", "w4_quantize"]

# The argument structs of include/ssd.h, in native layout.
CONV_ARGS = struct.Struct("@4q8iP2q10P")
SCAN_ARGS = struct.Struct("@3q6i5P10q8PN")
STEP_ARGS = struct.Struct("@3q8i3P3q11P")
W4_ARGS = struct.Struct("@2q4iPq3PqP")
SELECT_ARGS = struct.Struct("@2q6iP2q6PN")
REORDER_MAX = 16
REORDER_ARGS = struct.Struct("@2q4iP%dP%dP%dq" % ((REORDER_MAX,) * 3))

_F32, _I32 = torch.float32, torch.int32
_DTYPES = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without building a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _on_stream(fn):
    """Runs ``fn`` with ``stream`` as the current stream, so that the outputs it
    allocates belong to it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _launch(fn, where: str, args: bytes, dev: int) -> None:
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            code = fn(args, _raw_stream(dev))
    else:
        code = fn(args, _raw_stream(dev))
    if code:
        raise SSDError(code, where)


def _refuse(name, t, dev, dtype, shape, rows):
    if not isinstance(t, torch.Tensor):
        raise SSDError(1, f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise SSDError(1, f"{name} is on {t.device}, the other arguments on cuda:{dev}")
    if t.dtype is not dtype:
        raise SSDError(1, f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise SSDError(1, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise SSDError(1, f"{name} must be contiguous" + (" in its last dimension" if rows else ""))


def _dense(name, t, dev, dtype, shape) -> int:
    """The address of a contiguous tensor of this type and shape (0 for None)."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _refuse(name, t, dev, dtype, shape, False)
    return t.data_ptr()


def _rows(name, t, dev, dtype, shape):
    """The address and strides of a tensor whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(name, t, dev, dtype, shape, True)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        _refuse(name, t, dev, dtype, shape, True)
    return t.data_ptr(), stride


def _first(name, t, dims: int):
    """Device index, dtype code and shape of the tensor the others go by."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise SSDError(1, f"{name} must be a {dims}-D tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise SSDError(2, f"{name} has dtype {t.dtype}, expected float32 or bfloat16")
    dev = t.get_device()
    if dev < 0:
        raise SSDError(1, f"{name} must be a CUDA tensor (got {t.device})")
    return dev, code, t.shape


# ------------------------------------------------------------------ convolution

@_on_stream
def ssd_conv_fwd(u: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                 activation: Optional[str] = "silu", split: Optional[Sequence[int]] = None,
                 ring: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 lengths: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                 new_ring: Optional[torch.Tensor] = None, out: Optional[Sequence[torch.Tensor]] = None,
                 ) -> Union[torch.Tensor, Tuple[torch.Tensor, ...]]:
    """The short causal convolution (C: ssd_conv_fwd), for prompts (any length)
    and single tokens (length 1).

    u [B, L, C] float32 or bfloat16, its channels contiguous (a slice of the
    in-projection's output); weight [C, W] (W 2 to 4) and bias [C] float32.
    ``split`` gives the channels of two or three outputs, e.g. (H*64, G*N, G*N)
    for x, Bm and Cm as ssd_fwd takes them; without it there is one output.
    ``ring`` [slots, W, C] is the cache: the inputs of the last tokens, updated
    in place or written to ``new_ring``.  ``positions`` [B] int32 are the tokens
    before this call (0), ``lengths`` [B] int32 this call's tokens (L; outputs
    after them are 0), ``slots`` [B] int32 the cache rows (the first B; a
    sequence whose row does not exist is idle)."""
    dev, code, shape = _first("u", u, 3)
    B, L, C = shape
    W = weight.shape[1] if isinstance(weight, torch.Tensor) and weight.dim() == 2 else 0
    if activation not in ("silu", None):
        raise SSDError(2, f"activation {activation!r}, expected 'silu' or None")
    parts = (C,) if split is None else tuple(split)
    if not 1 <= len(parts) <= 3 or sum(parts) != C or min(parts) < 1:
        raise SSDError(1, f"split {parts} does not divide {C} channels in one to three parts")
    up, us = _rows("u", u, dev, u.dtype, shape)
    wp = _dense("weight", weight, dev, _F32, (C, W))
    nslots = 0
    if ring is None:
        if new_ring is not None or slots is not None:
            raise SSDError(1, "new_ring and slots belong to a ring")
    else:
        nslots = ring.shape[0] if isinstance(ring, torch.Tensor) and ring.dim() == 3 else 0
    if out is None:
        out = [torch.empty((B, L, n), dtype=u.dtype, device=u.device) for n in parts]
        ptrs = [t.data_ptr() for t in out]
    else:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(parts):
            raise SSDError(1, f"{len(out)} outputs for {len(parts)} parts")
        ptrs = [_dense("out", t, dev, u.dtype, (B, L, n)) for t, n in zip(out, parts)]
    pad = (0,) * (3 - len(parts))
    args = CONV_ARGS.pack(CONV_ARGS.size, B, L, nslots, C, W, code, 1 if activation else 0, len(parts), *parts, *pad,
                          up, us[0], us[1], wp, _dense("bias", bias, dev, _F32, (C,)),
                          _dense("ring", ring, dev, u.dtype, (nslots, W, C)),
                          _dense("new_ring", new_ring, dev, u.dtype, (nslots, W, C)),
                          _dense("positions", positions, dev, _I32, (B,)), _dense("lengths", lengths, dev, _I32, (B,)),
                          _dense("slots", slots, dev, _I32, (B,)), *ptrs, *pad)
    _launch(lib.ssd_conv_fwd, "ssd_conv_fwd", args, dev)
    return out[0] if split is None else tuple(out)


# ------------------------------------------------------------------ selective scan

def _scan_sizes(B, L, D, N, G, code=SSD_F32, softplus=0):
    return (SCAN_ARGS.size, B, L, D, N, G, code, softplus, 0)


def ssd_selective_scan_workspace_size(batch: int, seqlen: int, channels: int, dstate: int, ngroups: int) -> int:
    """Bytes of workspace ssd_selective_scan needs for these sizes (0: none)."""
    return lib.ssd_selective_scan_workspace_size(
        SCAN_ARGS.pack(*_scan_sizes(batch, seqlen, channels, dstate, ngroups), *((0,) * 24)))


@_on_stream
def ssd_selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
                       D: Optional[torch.Tensor] = None, *, z: Optional[torch.Tensor] = None,
                       delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                       init_state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, want_final_state: bool = True,
                       ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The recurrence with a decay per channel and state (C:
    ssd_selective_scan), for prompts and single tokens.  Returns (y, final_state).

    u, delta, z [B, L, D] and Bm, Cm [B, L, G, N] share float32 or bfloat16 and
    may be slices of wider rows; A [D, N], D [D], delta_bias [D], init_state and
    final_state [B, D, N] are float32 (N 1 to 64).  final_state may be
    init_state.  ``lengths`` [B] int32: tokens of each sequence."""
    dev, code, shape = _first("u", u, 3)
    B, L, C = shape
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise SSDError(1, "Bm must be a 4-D tensor")
    G, N = Bm.shape[2], Bm.shape[3]
    dt = u.dtype
    up, us = _rows("u", u, dev, dt, shape)
    dp, ds = _rows("delta", delta, dev, dt, shape)
    zp, zs = _rows("z", z, dev, dt, shape) if z is not None else (0, (0, 0))
    bp, bs = _rows("Bm", Bm, dev, dt, (B, L, G, N))
    cp, cs = _rows("Cm", Cm, dev, dt, (B, L, G, N))
    if G > 1 and (bs[2] != N or cs[2] != N):
        raise SSDError(1, "Bm and Cm must be contiguous over their groups")
    ap = _dense("A", A, dev, _F32, (C, N))
    skip, bias = _dense("D", D, dev, _F32, (C,)), _dense("delta_bias", delta_bias, dev, _F32, (C,))
    ip = _dense("init_state", init_state, dev, _F32, (B, C, N))
    if y is None:
        y = torch.empty(shape, dtype=dt, device=u.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((B, C, N), dtype=_F32, device=u.device)
    sizes = _scan_sizes(B, L, C, N, G, code, 1 if delta_softplus else 0)
    body = (up, dp, zp, bp, cp, us[0], us[1], ds[0], ds[1], zs[0], zs[1], bs[0], bs[1], cs[0], cs[1], ap, skip, bias, ip,
            _dense("final_state", final_state, dev, _F32, (B, C, N)), _dense("y", y, dev, dt, shape),
            _dense("lengths", lengths, dev, _I32, (B,)))
    need = lib.ssd_selective_scan_workspace_size(SCAN_ARGS.pack(*sizes, *body, 0, 0))
    wp = nbytes = 0
    if workspace is not None:
        nbytes = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
        wp = _dense("workspace", workspace, dev, torch.uint8, (nbytes,))
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=u.device)
        wp, nbytes = workspace.data_ptr(), need
    _launch(lib.ssd_selective_scan, "ssd_selective_scan", SCAN_ARGS.pack(*sizes, *body, wp, nbytes), dev)
    return y, final_state


# ------------------------------------------------------------------ single token

@_on_stream
def ssd_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, D: torch.Tensor, weight: torch.Tensor,
             bias: Optional[torch.Tensor], state: torch.Tensor, ring: torch.Tensor, positions: torch.Tensor, *,
             ngroups: int = 1, z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
             dt_softplus: bool = False, slots: Optional[torch.Tensor] = None,
             new_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of a Mamba-2 layer's convolution and recurrence for every
    sequence (C: ssd_step).  Returns y [B, H, 64].

    u [B, H*64 + 2*G*N] (x, B and C before the convolution), z [B, H*64] (the
    gate) and dt [B, H] may be slices of one projection's output; dt may also be
    float32 beside bfloat16 u.  A, D, dt_bias [H], weight [C, W], bias [C] and
    state [slots, H, 64, N] are float32; ring [slots, W, C] has u's type.  ring
    and state are updated in place, or the state goes to ``new_state`` (only the
    rows of this call are written).  ``positions`` [B] int32: tokens before this
    one; ``slots`` [B] int32: cache rows (a row that does not exist: idle)."""
    dev, code, shape = _first("u", u, 2)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise SSDError(1, "state must be a 4-D tensor")
    B, C = shape
    S, H, P, N = state.shape
    if ngroups < 1 or C != H * P + 2 * ngroups * N:
        raise SSDError(1, f"u has {C} channels, expected {H * P + 2 * max(1, ngroups) * N}")
    W = weight.shape[1] if isinstance(weight, torch.Tensor) and weight.dim() == 2 else 0
    up, us = _rows("u", u, dev, u.dtype, shape)
    zp, zs = _rows("z", z, dev, u.dtype, (B, H * P)) if z is not None else (0, (0,))
    tt = _F32 if isinstance(dt, torch.Tensor) and dt.dtype is _F32 else u.dtype
    tp, ts = _rows("dt", dt, dev, tt, (B, H))
    if positions is None:
        raise SSDError(1, "positions must be a torch.Tensor")
    if y is None:
        y = torch.empty((B, H, P), dtype=u.dtype, device=u.device)
    args = STEP_ARGS.pack(STEP_ARGS.size, B, S, H, P, ngroups, N, W, code, _DTYPES[tt], 1 if dt_softplus else 0,
                          up, zp, tp, us[0], zs[0], ts[0], _dense("weight", weight, dev, _F32, (C, W)),
                          _dense("bias", bias, dev, _F32, (C,)), _dense("A", A, dev, _F32, (H,)),
                          _dense("D", D, dev, _F32, (H,)), _dense("dt_bias", dt_bias, dev, _F32, (H,)),
                          _dense("ring", ring, dev, u.dtype, (S, W, C)), _dense("state", state, dev, _F32, (S, H, P, N)),
                          _dense("new_state", new_state, dev, _F32, (S, H, P, N)),
                          _dense("positions", positions, dev, _I32, (B,)), _dense("slots", slots, dev, _I32, (B,)),
                          _dense("y", y, dev, u.dtype, (B, H, P)))
    _launch(lib.ssd_step, "ssd_step", args, dev)
    return y


# ------------------------------------------------------------------ 4-bit weights

def w4_pack(codes: torch.Tensor) -> torch.Tensor:
    """4-bit codes [n, k] (values 0 to 15; a weight is (code - 8) * scale) in the
    order ssd_w4_matvec reads, int32 [ceil(n/16), ceil(k/64), 32, 4].  Done once
    per weight, on any device."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.is_floating_point():
        raise SSDError(1, "codes must be a 2-D tensor of whole numbers")
    n, k = codes.shape
    rows, cols = -(-n // 16), -(-k // 64)
    full = codes.new_full((rows * 16, cols * 64), 8, dtype=torch.int64)
    full[:n, :k] = codes
    # [row tile, a, r, column tile, h, c, i, e, p] -> [row tile, column tile, r, c, h, i, e, a, p]
    v = full.view(rows, 2, 8, cols, 2, 4, 2, 2, 2).permute(0, 3, 2, 5, 4, 6, 7, 1, 8)
    e, a, p = torch.meshgrid(*[torch.arange(2, device=codes.device)] * 3, indexing="ij")
    words = (v << (4 * (a + 2 * e) + 16 * p)).sum(dim=(-3, -2, -1))
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    return words.to(_I32).reshape(rows, cols, 32, 4)


def w4_quantize(weight: torch.Tensor, group: int = 128) -> Tuple[torch.Tensor, torch.Tensor]:
    """(packed codes, scales) of a weight [n, k] for ssd_w4_matvec: per row and
    group of columns the scale that puts the largest magnitude at 7."""
    if group not in (32, 64, 128):
        raise SSDError(2, f"group {group}, expected 32, 64 or 128")
    n, k = weight.shape
    groups = -(-k // group)
    w = weight.new_zeros((n, groups * group), dtype=_F32)
    w[:, :k] = weight
    w = w.view(n, groups, group)
    scales = w.abs().amax(-1) / 7.0
    codes = torch.round(w / torch.where(scales > 0, scales, 1.0)[..., None]).clamp_(-7, 7) + 8
    return w4_pack(codes.view(n, groups * group)[:, :k].to(torch.int64)), scales


@_on_stream
def ssd_w4_matvec(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int, *,
                  add: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W^T (+ add) for a few tokens and a 4-bit W (C: ssd_w4_matvec).

    x [M, k] and add [M, n] float32 or bfloat16 (rows may be strided); ``packed``
    from w4_pack, ``scales`` [n, ceil(k/group)] float32, group 32, 64 or 128."""
    dev, code, shape = _first("x", x, 2)
    M, K = shape
    if not isinstance(scales, torch.Tensor) or scales.dim() != 2:
        raise SSDError(1, "scales must be a 2-D tensor")
    if group not in (32, 64, 128):
        raise SSDError(2, f"group {group}, expected 32, 64 or 128")
    n = scales.shape[0]
    xp, xs = _rows("x", x, dev, x.dtype, shape)
    ap, as_ = _rows("add", add, dev, x.dtype, (M, n)) if add is not None else (0, (0,))
    if y is None:
        y = torch.empty((M, n), dtype=x.dtype, device=x.device)
    args = W4_ARGS.pack(W4_ARGS.size, M, n, K, group, code, xp, xs[0],
                        _dense("packed", packed, dev, _I32, (-(-n // 16), -(-K // 64), 32, 4)),
                        _dense("scales", scales, dev, _F32, (n, -(-K // group))), ap, as_[0],
                        _dense("y", y, dev, x.dtype, (M, n)))
    _launch(lib.ssd_w4_matvec, "ssd_w4_matvec", args, dev)
    return y


# ------------------------------------------------------------------ beam search

def ssd_beam_select_workspace_size(batch: int, beams: int, vocab: int, k: int) -> int:
    """Bytes of workspace ssd_beam_select needs for these sizes."""
    return lib.ssd_beam_select_workspace_size(
        SELECT_ARGS.pack(SELECT_ARGS.size, batch, beams, vocab, k, 0, 0, 0, *((0,) * 10)))


@_on_stream
def ssd_beam_select(logits: torch.Tensor, scores: torch.Tensor, k: int, *, finished: Optional[torch.Tensor] = None,
                    eos: int = -1, workspace: Optional[torch.Tensor] = None,
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The k best continuations of every request's beams (C: ssd_beam_select).
    Returns (scores float32, parents int32, tokens int32), each [B, k].

    logits [B, W, V] float32 or bfloat16 (rows may be strided), scores [B, W]
    float32 the beams' log-probabilities, ``finished`` [B, W] bool the beams that
    only go on with ``eos`` at their present score."""
    dev, code, shape = _first("logits", logits, 3)
    B, W, V = shape
    lp, ls = _rows("logits", logits, dev, logits.dtype, shape)
    sp = _dense("scores", scores, dev, _F32, (B, W))
    fp = _dense("finished", finished, dev, torch.bool, (B, W))
    if k < 1 or k > 64:
        raise SSDError(1 if k < 1 else 2, f"k is {k}, expected 1 to 64")
    best, parents, tokens = torch.empty((3, B, k), dtype=_I32, device=logits.device).unbind(0)
    best = best.view(_F32)
    head = (SELECT_ARGS.size, B, W, V, k, code, eos, 0, lp, ls[0], ls[1], sp, fp, best.data_ptr(), parents.data_ptr(),
            tokens.data_ptr())
    if workspace is None:
        nbytes = lib.ssd_beam_select_workspace_size(SELECT_ARGS.pack(*head, 0, 0))
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=logits.device)
        wp = workspace.data_ptr()
    else:
        nbytes = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
        wp = _dense("workspace", workspace, dev, torch.uint8, (nbytes,))
    _launch(lib.ssd_beam_select, "ssd_beam_select", SELECT_ARGS.pack(*head, wp, nbytes), dev)
    return best, parents, tokens


@_on_stream
def ssd_beam_reorder(states: Sequence[torch.Tensor], parents: torch.Tensor, *,
                     out: Optional[Sequence[torch.Tensor]] = None) -> List[torch.Tensor]:
    """Row b*k + i of every state becomes row b*W + parents[b, i] (C:
    ssd_beam_reorder).  ``states``: contiguous tensors of any type with the same
    number of rows B*W; ``parents`` [B, k] int32.  In place without ``out`` (then
    k must be W); otherwise into ``out``, tensors of B*k rows.  Returns the
    reordered tensors."""
    states = [states] if isinstance(states, torch.Tensor) else list(states)
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        raise SSDError(1, "parents must be a 2-D tensor")
    dev = parents.get_device()
    if dev < 0:
        raise SSDError(1, f"parents must be a CUDA tensor (got {parents.device})")
    B, k = parents.shape
    pp = _dense("parents", parents, dev, _I32, (B, k))
    new = states if out is None else ([out] if isinstance(out, torch.Tensor) else list(out))
    if len(new) != len(states):
        raise SSDError(1, f"{len(new)} outputs for {len(states)} states")
    src, dst, size, beams = [], [], [], 0
    for t, o in zip(states, new):
        if not isinstance(t, torch.Tensor) or t.dim() < 1 or (B and t.shape[0] % B) or (not B and t.shape[0]):
            raise SSDError(1, f"a state must have a multiple of {B} rows")
        w = t.shape[0] // B if B else k
        if beams and w != beams:
            raise SSDError(1, "the states must have the same number of rows")
        beams = w
        src.append(_dense("state", t, dev, t.dtype, t.shape))
        dst.append(_dense("out", o, dev, t.dtype, (B * k, *t.shape[1:])))
        size.append(t.numel() // t.shape[0] * t.element_size() if t.shape[0] else 0)
    for i in range(0, len(states), REORDER_MAX):
        n = min(REORDER_MAX, len(states) - i)
        pad = [0] * (REORDER_MAX - n)
        _launch(lib.ssd_beam_reorder, "ssd_beam_reorder",
                REORDER_ARGS.pack(REORDER_ARGS.size, B, beams, k, n, 0, pp, *src[i:i + n], *pad, *dst[i:i + n], *pad,
                                  *size[i:i + n], *pad), dev)
    return new
