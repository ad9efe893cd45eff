"""What ssd_delta_fwd and ssd_draft_verify refuse, without a GPU: nothing is
enqueued, so any address will do."""
import ctypes

import pytest
import torch

import mamba_ssd_forward_chunked_gb300 as ssd

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
i32, i64, f32, ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class Delta(ctypes.Structure):
    _fields_ = ([("size", i64), ("batch", i64), ("seqlen", i64), ("nslots", i64)]
                + [(n, i32) for n in ("nheads", "headdim", "ngroups", "dstate", "dtype", "gate_dtype", "dt_softplus", "beta_sigmoid")]
                + [("scale", f32), ("norm_eps", f32)] + [(n, ptr) for n in ("x", "Bm", "Cm")]
                + [(n, i64) for n in ("x_batch", "x_token", "B_batch", "B_token", "C_batch", "C_token")]
                + [("dt", ptr), ("beta", ptr)] + [(n, i64) for n in ("dt_batch", "dt_token", "beta_batch", "beta_token")]
                + [(n, ptr) for n in ("A", "dt_bias", "init_state", "final_state", "slots", "positions", "lengths", "y", "workspace")] + [("workspace_bytes", ctypes.c_size_t)])


class Verify(ctypes.Structure):
    _fields_ = ([("size", i64), ("batch", i64)] + [(n, i32) for n in ("drafts", "vocab", "dtype", "reserved")]
                + [("logits", ptr), ("logits_batch", i64), ("logits_row", i64), ("draft_logits", ptr),
                   ("draft_logits_batch", i64), ("draft_logits_row", i64)]
                + [(n, ptr) for n in ("draft", "uniforms", "scale", "lengths", "tokens", "accepted", "logprobs", "workspace")]
                + [("workspace_bytes", ctypes.c_size_t)])


def delta(**change):
    a = dict(size=ctypes.sizeof(Delta), batch=0, seqlen=4, nslots=0, nheads=4, headdim=64, ngroups=2, dstate=64, dtype=1,
             gate_dtype=1, scale=1.0, norm_eps=-1.0)
    a.update(change)
    return ssd.lib.ssd_delta_fwd(ctypes.byref(Delta(**a)), None)


def full(**change):
    """A call with every tensor at an aligned address that is never reached."""
    a = dict(batch=2, nslots=2, **{n: 4096 for n in ("x", "Bm", "Cm", "dt", "beta", "A", "y")})
    a.update(change)
    return delta(**a)


@pytest.mark.parametrize("change,status", [
    (dict(), OK), (dict(size=8), INVALID), (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(nslots=-1), INVALID),
    (dict(nheads=0), INVALID), (dict(headdim=0), INVALID), (dict(ngroups=0), INVALID), (dict(dstate=0), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(gate_dtype=2), UNSUPPORTED), (dict(dtype=0, gate_dtype=1), UNSUPPORTED),
    (dict(gate_dtype=0), OK), (dict(headdim=24), UNSUPPORTED), (dict(headdim=1040), UNSUPPORTED), (dict(headdim=1024), OK),
    (dict(dstate=96), UNSUPPORTED), (dict(dstate=256), OK), (dict(ngroups=3), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(seqlen=(1 << 30) + 1), UNSUPPORTED), (dict(nheads=65536, ngroups=1), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(norm_eps=float("nan")), INVALID),
    (dict(norm_eps=float("inf")), INVALID)])
def test_delta_sizes(change, status):
    assert delta(**change) == status


@pytest.mark.parametrize("change", [
    *[{n: None} for n in ("x", "Bm", "Cm", "dt", "beta", "A", "y")], *[{n: 4097} for n in ("x", "Bm", "Cm", "dt", "beta", "y")],
    *[{n: 4098} for n in ("A", "dt_bias", "slots", "positions", "lengths")], dict(init_state=4104), dict(final_state=4100),
    dict(nslots=1), dict(gate_dtype=0, dt=4098)])
def test_delta_addresses(change):
    assert full(**change) == INVALID


def verify(**change):
    a = dict(size=ctypes.sizeof(Verify), batch=2, drafts=3, vocab=100, dtype=0, workspace_bytes=1 << 20,
             **{n: 4096 for n in ("logits", "draft_logits", "draft", "uniforms", "tokens", "accepted", "logprobs", "workspace")})
    a.update(change)
    return ssd.lib.ssd_draft_verify(ctypes.byref(Verify(**a)), None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), OK), (dict(size=8), INVALID), (dict(batch=-1), INVALID), (dict(drafts=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(drafts=65), UNSUPPORTED),
    (dict(vocab=(1 << 19) + 1), UNSUPPORTED), (dict(workspace_bytes=8), WORKSPACE), (dict(workspace=4104), INVALID),
    *[({n: None}, INVALID) for n in ("logits", "draft", "uniforms", "tokens", "accepted", "logprobs", "workspace")],
    *[({n: 4098}, INVALID) for n in ("logits", "draft_logits", "draft", "uniforms", "scale", "lengths", "tokens", "accepted", "logprobs")]])
def test_verify_arguments(change, status):
    assert verify(**change) == status


def test_verify_workspace_size():
    size = ssd.ssd_draft_verify_workspace_size
    assert size(2, 3, 100, torch.float32, True) == 2 * 7 * 8
    assert size(2, 3, 100, torch.float32, False) == 2 * 4 * 8
    assert size(2, 0, 100, torch.bfloat16, True) == size(2, 0, 100, torch.bfloat16, False) == 2 * 8
    assert size(2, 65, 100, torch.bfloat16, True) == 0 and size(0, 3, 100, torch.bfloat16, True) == 0
    # a row may begin one value after a 16-byte boundary
    assert size(1, 0, 8 * 256, torch.bfloat16, False) == 2 * 8


def test_tensors_are_checked():
    x, dt, A = torch.zeros(1, 2, 4, 64), torch.zeros(1, 2, 4), torch.zeros(4)
    k = torch.zeros(1, 2, 2, 64)
    with pytest.raises(ssd.SSDError, match="x must be a CUDA tensor"):
        ssd.ssd_delta_fwd(x, dt, A, k, k, dt)
    with pytest.raises(ssd.SSDError, match="4-D"):
        ssd.ssd_delta_fwd(x[0], dt, A, k, k, dt)
    with pytest.raises(ssd.SSDError, match="expected float32 or bfloat16"):
        ssd.ssd_delta_fwd(x.double(), dt, A, k, k, dt)
    with pytest.raises(ssd.SSDError, match="x must be a CUDA tensor"):
        ssd.ssd_delta_fwd(x, dt, A, k, k, dt, stream=0)
    with pytest.raises(ssd.SSDError, match="logits must be a CUDA tensor"):
        ssd.ssd_draft_verify(torch.zeros(1, 2, 5), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))
    with pytest.raises(ssd.SSDError, match="3-D"):
        ssd.ssd_draft_verify(torch.zeros(2, 5), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,L,H,G,P,N", [(256, 2048, 32, 16, 128, 128), (65535, 4096, 32, 32, 128, 128), (7, 100000, 64, 1, 64, 64),
                                         (2, 10 ** 6, 256, 256, 1024, 128), (1, 2 ** 30, 8, 8, 64, 128)])
def test_delta_workspace_is_bounded(B, L, H, G, P, N, dtype):
    """2 x 512 MiB, and the states of as many sequences as have 16 chunks in 512 MiB, or of one."""
    record = (2 * (N // 64) + (1 if dtype == torch.bfloat16 else 2)) * 8192 * H
    states = max(1, (512 << 20) // (16 * record)) * H * P * N * 4
    assert 0 < ssd.ssd_delta_workspace_size(B, L, H, P, N, dtype, G) <= 2 * (512 << 20) + states
