"""The layer operators without a GPU: the argument structs against the header,
the packing of 4-bit codes, and the C entry points' refusals (every call here
fails its checks, or has nothing to do, before any CUDA call)."""
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# the argument structs of include/ssd.h, in native layout
REORDER_MAX = 16
CONV_ARGS = struct.Struct("@4q8iP2q10P")
SCAN_ARGS = struct.Struct("@3q6i5P10q8PN")
STEP_ARGS = struct.Struct("@3q8i3P3q11P")
W4_ARGS = struct.Struct("@2q4iPq3PqPPN")
SELECT_ARGS = struct.Struct("@2q6iP2q6PN")
REORDER_ARGS = struct.Struct("@2q4iP%dP%dP%dq" % ((REORDER_MAX,) * 3))
FAKE = 1 << 20  # an aligned address that no call here reads


@pytest.fixture(scope="module")
def ext():
    import __graft_entry__
    __graft_entry__.build()
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def test_struct_sizes_match_the_header(ext, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ["conv", "selective_scan", "step", "w4_matvec", "beam_select", "beam_reorder"]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "ssd.h"\nint main(void){' +
                   "".join(f'printf("%zu\\n", sizeof(ssd_{n}_args));' for n in names) + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [s.size for s in (CONV_ARGS, SCAN_ARGS, STEP_ARGS, W4_ARGS,
                                    SELECT_ARGS, REORDER_ARGS)]
    text = open(os.path.join(ROOT, "include", "ssd.h")).read()
    assert int(re.search(r"#define SSD_REORDER_MAX (\d+)", text).group(1)) == REORDER_MAX


@pytest.mark.parametrize("n,k", [(16, 64), (1, 1), (17, 65), (40, 200)])
def test_pack_puts_every_code_where_the_header_says(ext, n, k):
    g = torch.Generator().manual_seed(n * 1000 + k)
    codes = torch.randint(0, 16, (n, k), generator=g)
    packed = ext.w4_pack(codes)
    assert packed.dtype == torch.int32 and packed.shape == (-(-n // 16), -(-k // 64), 32, 4)
    words = packed.to(torch.int64) & 0xFFFFFFFF
    for row in range(packed.shape[0] * 16):
        for col in range(packed.shape[1] * 64):
            a, r = row % 16 // 8, row % 8
            h, c, i, e, p = col % 64 // 32, col % 32 // 8, col % 8 // 4, col % 4 // 2, col % 2
            got = int(words[row // 16, col // 64, 4 * r + c, 2 * h + i] >> (4 * (a + 2 * e) + 16 * p)) & 15
            assert got == (int(codes[row, col]) if row < n and col < k else 8), (row, col)


def test_quantize_keeps_weights_within_half_a_step(ext):
    g = torch.Generator().manual_seed(3)
    w = torch.randn(24, 150, generator=g)
    w[5, 32:64] = 0.0
    packed, scales = ext.w4_quantize(w, 32)
    assert scales.shape == (24, 5) and float(scales[5, 1]) == 0.0
    words = (packed.to(torch.int64) & 0xFFFFFFFF).view(2, 3, 8, 4, 2, 2)  # row tile, column tile, r, c, h, i
    codes = torch.zeros(32, 192, dtype=torch.int64)
    for a in range(2):
        for e in range(2):
            for p in range(2):
                v = (words >> (4 * (a + 2 * e) + 16 * p)) & 15
                for r in range(8):
                    for c in range(4):
                        for h in range(2):
                            for i in range(2):
                                codes[8 * a + r::16, 32 * h + 8 * c + 4 * i + 2 * e + p::64] = v[:, :, r, c, h, i]
    back = (codes[:24, :150] - 8) * scales.repeat_interleave(32, 1)[:, :150]
    step = scales.repeat_interleave(32, 1)[:, :150]
    assert ((back - w).abs() <= 0.5001 * step + 1e-7).all()


def conv_args(ext, **kw):
    v = dict(size=CONV_ARGS.size, batch=2, seqlen=5, nslots=0, channels=12, width=4, dtype=0, act=1, nout=3,
             c0=4, c1=4, c2=4, u=FAKE, ub=60, ut=12, weight=FAKE, bias=0, ring=0, new_ring=0, positions=0, lengths=0,
             slots=0, o0=FAKE, o1=FAKE, o2=FAKE)
    v.update(kw)
    return CONV_ARGS.pack(*v.values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=8)), (1, dict(batch=-1)), (1, dict(seqlen=-1)), (1, dict(channels=0)), (2, dict(width=1)),
    (2, dict(width=5)), (2, dict(dtype=2)), (2, dict(act=7)), (2, dict(batch=65536)), (1, dict(nout=0)), (1, dict(nout=4)),
    (1, dict(c0=5)), (1, dict(c2=3)), (1, dict(c1=0)), (1, dict(u=0)), (1, dict(u=FAKE + 2)), (1, dict(weight=0)),
    (1, dict(weight=FAKE + 1)), (1, dict(bias=FAKE + 2)), (1, dict(o1=0)), (1, dict(o2=FAKE + 1)),
    (1, dict(slots=FAKE)), (1, dict(new_ring=FAKE)), (1, dict(ring=FAKE, nslots=1)), (1, dict(ring=FAKE + 2, nslots=2)),
    (1, dict(ring=FAKE, nslots=-1)), (0, dict(batch=0)), (0, dict(seqlen=0, u=0, o0=0, o1=0, o2=0)),
    (1, dict(positions=FAKE + 2)), (1, dict(lengths=FAKE + 1)), (1, dict(ring=FAKE, nslots=2, slots=FAKE + 2)),
])
def test_conv_refusals(ext, want, kw):
    assert ext.lib.ssd_conv_fwd(conv_args(ext, **kw), None) == want


def scan_args(ext, **kw):
    v = dict(size=SCAN_ARGS.size, batch=2, seqlen=5, channels=12, dstate=16, ngroups=1, dtype=1, softplus=1,
             reserved=0, u=FAKE, delta=FAKE, z=0, Bm=FAKE, Cm=FAKE, ub=60, ut=12, db=60, dt=12, zb=0, zt=0, Bb=80, Bt=16,
             Cb=80, Ct=16, A=FAKE, D=0, bias=0, init=0, final=0, y=FAKE, lengths=0, ws=0, nbytes=0)
    v.update(kw)
    return SCAN_ARGS.pack(*v.values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=0)), (1, dict(batch=-1)), (1, dict(seqlen=-3)), (1, dict(channels=0)), (1, dict(dstate=0)),
    (2, dict(dstate=65)), (1, dict(ngroups=0)), (2, dict(ngroups=5)), (2, dict(dtype=9)), (2, dict(batch=70000)),
    (1, dict(A=0)), (1, dict(A=FAKE + 2)), (1, dict(u=0)), (1, dict(delta=0)), (1, dict(Bm=0)), (1, dict(Cm=FAKE + 1)),
    (1, dict(y=0)), (1, dict(z=FAKE + 1)), (1, dict(D=FAKE + 1)), (1, dict(bias=FAKE + 1)), (1, dict(init=FAKE + 2)),
    (1, dict(final=FAKE + 2)), (1, dict(lengths=FAKE + 2)), (0, dict(batch=0)), (0, dict(seqlen=0)),
])
def test_scan_refusals(ext, want, kw):
    assert ext.lib.ssd_selective_scan(scan_args(ext, **kw), None) == want


def step_args(ext, **kw):
    v = dict(size=STEP_ARGS.size, batch=2, nslots=2, nheads=4, headdim=64, ngroups=2, dstate=64, width=4, dtype=1,
             dt_dtype=1, softplus=1, u=FAKE, z=0, dt=FAKE, us=512, zs=0, ts=4, weight=FAKE, bias=0, A=FAKE, D=FAKE,
             dt_bias=0, ring=FAKE, state=FAKE, new_state=0, positions=FAKE, slots=0, y=FAKE)
    v.update(kw)
    return STEP_ARGS.pack(*v.values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=1)), (1, dict(batch=-1)), (1, dict(nslots=-1)), (1, dict(nheads=0)), (2, dict(headdim=32)),
    (2, dict(dstate=96)), (2, dict(ngroups=3)), (1, dict(ngroups=0)), (2, dict(width=5)), (2, dict(dtype=3)),
    (2, dict(dtype=0, dt_dtype=1)), (2, dict(batch=65536, nslots=65536)), (1, dict(u=0)), (1, dict(dt=0)),
    (1, dict(dt=FAKE + 1)), (1, dict(z=FAKE + 1)), (1, dict(weight=0)), (1, dict(A=0)), (1, dict(D=0)),
    (1, dict(positions=0)), (1, dict(ring=0)), (1, dict(state=0)), (1, dict(state=FAKE + 8)),
    (1, dict(new_state=FAKE + 4)), (1, dict(y=0)), (1, dict(nslots=1)), (1, dict(bias=FAKE + 1)),
    (1, dict(dt_bias=FAKE + 1)), (1, dict(slots=FAKE + 1)), (0, dict(batch=0)),
])
def test_step_refusals(ext, want, kw):
    assert ext.lib.ssd_step(step_args(ext, **kw), None) == want


def w4_args(ext, **kw):
    v = dict(size=W4_ARGS.size, tokens=1, n=16, k=64, group=32, dtype=1, x=FAKE, xs=64, packed=FAKE, scales=FAKE,
             add=0, adds=0, y=FAKE, ws=0, nbytes=0)
    v.update(kw)
    return W4_ARGS.pack(*v.values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=0)), (1, dict(tokens=-1)), (1, dict(n=0)), (1, dict(k=0)), (2, dict(group=16)), (2, dict(group=0)),
    (2, dict(dtype=4)), (2, dict(tokens=65536)), (1, dict(x=0)), (1, dict(x=FAKE + 1)), (1, dict(packed=0)),
    (1, dict(packed=FAKE + 4)), (1, dict(scales=0)), (1, dict(scales=FAKE + 2)), (1, dict(add=FAKE + 1)), (1, dict(y=0)),
    (0, dict(tokens=0)), (1, dict(dtype=0)), (1, dict(dtype=0, ws=FAKE + 2, nbytes=384)),
    (3, dict(dtype=0, ws=FAKE, nbytes=383)), (1, dict(xs=65, tokens=2)), (1, dict(k=63)), (1, dict(x=FAKE + 2)),
    (3, dict(k=63, ws=FAKE, nbytes=127)),
])
def test_w4_refusals(ext, want, kw):
    assert ext.lib.ssd_w4_matvec(w4_args(ext, **kw), None) == want


def select_args(ext, **kw):
    v = dict(size=SELECT_ARGS.size, batch=2, beams=4, vocab=100, k=4, dtype=0, eos=2, reserved=0, logits=FAKE,
             lb=400, lw=100, scores=FAKE, finished=0, out=FAKE, parents=FAKE, tokens=FAKE, ws=FAKE, nbytes=1 << 30)
    v.update(kw)
    return SELECT_ARGS.pack(*v.values())


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=0)), (1, dict(batch=-1)), (1, dict(beams=0)), (1, dict(vocab=0)), (1, dict(k=0)), (2, dict(k=65)),
    (2, dict(beams=65)), (1, dict(beams=1, vocab=3, k=4)), (2, dict(vocab=1 << 30)), (2, dict(dtype=5)),
    (1, dict(finished=FAKE, eos=-1)), (1, dict(finished=FAKE, eos=100)), (1, dict(logits=0)), (1, dict(logits=FAKE + 2)),
    (1, dict(scores=0)), (1, dict(out=0)), (1, dict(parents=0)), (1, dict(tokens=FAKE + 1)), (1, dict(ws=0)),
    (1, dict(ws=FAKE + 4)), (3, dict(nbytes=1)), (0, dict(batch=0)), (2, dict(batch=65536)),
])
def test_select_refusals(ext, want, kw):
    assert ext.lib.ssd_beam_select(select_args(ext, **kw), None) == want


def reorder_args(ext, **kw):
    n = REORDER_MAX
    v = dict(size=REORDER_ARGS.size, batch=2, beams=4, k=4, count=1, reserved=0, parents=FAKE, src=FAKE,
             dst=2 * FAKE, row=64)
    v.update(kw)
    lists = [[v[key]] + [0] * (n - 1) for key in ("src", "dst", "row")]
    return REORDER_ARGS.pack(*[v[key] for key in ("size", "batch", "beams", "k", "count", "reserved", "parents")],
                                   *lists[0], *lists[1], *lists[2])


@pytest.mark.parametrize("want,kw", [
    (1, dict(size=0)), (1, dict(batch=-1)), (1, dict(beams=0)), (1, dict(k=0)), (2, dict(k=65)), (2, dict(beams=65)),
    (1, dict(count=-1)), (1, dict(count=17)), (1, dict(parents=0)), (1, dict(parents=FAKE + 2)), (1, dict(src=0)),
    (1, dict(dst=0)), (1, dict(row=-1)), (1, dict(dst=FAKE, k=3)), (0, dict(batch=0)), (0, dict(count=0)),
    (2, dict(batch=65536)),
])
def test_reorder_refusals(ext, want, kw):
    assert ext.lib.ssd_beam_reorder(reorder_args(ext, **kw), None) == want


def test_workspace_sizes(ext):
    assert ext.ssd_beam_select_workspace_size(2, 4, 1000, 4) > 0
    assert ext.ssd_beam_select_workspace_size(2, 4, 1000, 65) == 0
    assert ext.ssd_selective_scan_workspace_size(1, 100, 64, 65, 1) == 0


def test_host_tensors_are_refused(ext):
    u = torch.zeros(1, 4, 8)
    with pytest.raises(ext.SSDError, match="CUDA"):
        ext.ssd_conv_fwd(u, torch.zeros(8, 4))
    with pytest.raises(ext.SSDError, match="CUDA"):
        ext.ssd_beam_select(u, torch.zeros(1, 4), 2)
    with pytest.raises(ext.SSDError, match="float32 or bfloat16"):
        ext.ssd_w4_matvec(torch.zeros(1, 64, dtype=torch.float16), u, u, 32)
    with pytest.raises(ext.SSDError, match="2-D"):
        ext.ssd_step(u, u, u, u, u, None, u, u, u)
