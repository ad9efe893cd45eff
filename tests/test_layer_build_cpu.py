"""The compiled binding of the layer operators: the package without it."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "mamba_ssd_forward_chunked_gb300"


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("binding", [None, b"not a module"], ids=["missing", "unusable"])
def test_the_package_without_the_binding(built, tmp_path, binding):
    """What needs only the library is there; the layer's calls say what is missing."""
    there = tmp_path / PACKAGE
    there.mkdir()
    for name in os.listdir(os.path.join(ROOT, PACKAGE)):
        if name.endswith(".py") or name == "libssd_gb300.so":
            shutil.copy(os.path.join(ROOT, PACKAGE, name), there)
    if binding is not None:
        (there / "_layer_binding.so").write_bytes(binding)
    code = f"""
import torch
import {PACKAGE} as ssd
assert ssd.__file__.startswith({str(tmp_path)!r})
assert ssd.ssd_validate_shape(ssd.make_shape(1, 64, 2, 64, 1, 64, 64, torch.float32)) == 0
assert ssd.w4_pack(torch.zeros(3, 5, dtype=torch.int64)).shape == (1, 1, 32, 4)
for call in (lambda: ssd.ssd_conv_fwd(torch.zeros(1, 1, 8), torch.zeros(8, 4)),
             lambda: ssd.ssd_beam_select_workspace_size(1, 1, 10, 1)):
    try:
        call()
    except ImportError as e:
        assert "_layer_binding" in str(e) and "build_ext.py" in str(e), e
    else:
        raise SystemExit("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.fixture
def script(tmp_path, monkeypatch):
    """The build script on files of its own, with compilers that only write their outputs, and an installed torch
    whose version can be set.  Returns (module, set_torch, commands so far)."""
    import __graft_entry__
    mod = __graft_entry__._build_ext_module()
    for name, file in (("OUT", "libssd_gb300.so"), ("BINDING", "_layer_binding.so"), ("BUILD", "objects")):
        monkeypatch.setattr(mod, name, str(tmp_path / file))
    monkeypatch.setattr(mod, "sources", lambda: [])
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(mod.subprocess, "run", run)
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "__init__.py").write_text("")

    class Spec:
        origin = str(torch / "__init__.py")

    class Util:
        find_spec = staticmethod(lambda name: Spec)

    class Importlib:
        util = Util

    def set_torch(version):
        (torch / "version.py").write_text(f"__version__ = {version!r}\n")
        os.utime(torch / "version.py", (1, 1))  # an installation keeps its files' old times
    monkeypatch.setattr(mod, "importlib", Importlib)
    return mod, set_torch, ran


def binding_commands(ran):
    got = sum(any("binding" in word for word in cmd) for cmd in ran)
    ran.clear()
    return got


def test_another_torch_or_python_builds_the_binding_again(script, monkeypatch):
    mod, set_torch, ran = script
    set_torch("2.9.1")
    mod.build()
    assert binding_commands(ran) == 2  # compiled and linked
    mod.build()
    assert binding_commands(ran) == 0
    set_torch("2.11.0")
    mod.build()
    assert binding_commands(ran) == 2
    monkeypatch.setattr(mod.sys, "version", mod.sys.version + " another")
    mod.build()
    assert binding_commands(ran) == 2
    mod.build()
    assert binding_commands(ran) == 0
