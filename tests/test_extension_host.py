"""The extension next to the library: what works without it, and when it is built again (no GPU)."""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "block_causal_linear_rope_b200")

# imports the package of the folder argv[1], calls the library for a block-causal refusal, then each of the extension's
CODE = """
import sys, torch
sys.path.insert(0, sys.argv[1])
if len(sys.argv) > 2: torch.__version__ = sys.argv[2]
import block_causal_linear_rope_b200 as blin
assert blin.__file__.startswith(sys.argv[1])
assert blin.lib.blin_prefill(None, None, None, None, 1, 1, 1, 32, None, None, None, 0, None) == -1
q = torch.zeros(1, 1, 4, 32)
for call in (lambda: blin.rope(q, rope_split=(8, 12, 12), grid=(1, 2, 2)), lambda: blin.decay_prefill(q, q, q, q),
             lambda: blin.decay_step(q, q, q, q, q)):
    try:
        call()
    except ImportError as e:
        print("refused:", e)
    except (TypeError, ValueError) as e:
        print("there:", e)
assert not hasattr(blin._ext, "__wrapped__")
"""


def package(tmp_path, extension):
    pkg = tmp_path / "block_causal_linear_rope_b200"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg / "__init__.py")
    os.symlink(os.path.join(PKG, "libblin.so"), pkg / "libblin.so")
    if extension is not None:
        (pkg / "_blin_torch.so").write_bytes(extension)
    return str(tmp_path)


def run(*args):
    r = subprocess.run([sys.executable, "-c", CODE, *args], capture_output=True, text=True, cwd=args[0], timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.splitlines()


@pytest.mark.parametrize("extension,why", [(None, "missing"), (b"not a library", "does not load")])
def test_the_block_causal_calls_need_no_extension(tmp_path, extension, why):
    lines = run(package(tmp_path, extension))
    assert len(lines) == 3
    for line in lines:
        assert line.startswith("refused:") and why in line and "build.py" in line


def test_an_extension_of_another_torch_is_not_called(tmp_path):
    with open(os.path.join(PKG, "_blin_torch.so"), "rb") as f:
        where = package(tmp_path, f.read())
    assert all(line.startswith("there:") for line in run(where))
    lines = run(where, "1.2.3+cu128")
    assert len(lines) == 3 and all("built for torch" in line and "this is torch 1.2.3" in line for line in lines)


def test_an_extension_that_does_not_tell_its_versions_is_not_called(tmp_path):
    """As one that was built from older sources."""
    src, so = tmp_path / "old.c", tmp_path / "old.so"
    src.write_text('#include <Python.h>\nstatic struct PyModuleDef m = {PyModuleDef_HEAD_INIT, "_blin_torch", 0, -1, 0};\n'
                   "PyMODINIT_FUNC PyInit__blin_torch(void) { return PyModule_Create(&m); }\n")
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], str(src), "-o", str(so)])
    lines = run(package(tmp_path, so.read_bytes()))
    assert len(lines) == 3 and all("refused:" in line and "does not tell" in line for line in lines)


def test_the_extension_is_built_again_for_another_torch(tmp_path, monkeypatch):
    import torch
    spec = importlib.util.spec_from_file_location("_blin_build_under_test", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_blin_torch.so"))
    monkeypatch.setattr(build, "EXT_FOR", str(tmp_path / "b" / "blin_torch.for"))
    runs = []

    def compile(cmd):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build.subprocess, "check_call", compile)
    build.build_ext()
    build.build_ext()
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    build.build_ext()
    build.build_ext()
    assert len(runs) == 2
    build.build_ext(force=True)
    assert len(runs) == 3


def test_the_extension_never_reaches_the_oracle():
    """test_separation looks at the CUDA sources and the library; the same for the C++ source and the extension."""
    import re
    csrc = os.path.join(PKG, "csrc")
    names = [n for n in os.listdir(csrc) if n.endswith((".cpp", ".cc", ".c", ".hpp"))]
    assert names == ["blin_torch.cpp"]
    with open(os.path.join(csrc, names[0])) as f:
        incs = re.findall(r'^\s*#\s*include\s*[<"]([^>"]+)[>"]', f.read(), flags=re.M)
    assert incs and not any("oracle" in i for i in incs)
    ext = os.path.join(PKG, "_blin_torch.so")
    needed = subprocess.run(["readelf", "-d", ext], capture_output=True, text=True).stdout
    syms = subprocess.run(["nm", "-D", ext], capture_output=True, text=True).stdout
    assert "libblin.so" in needed and "oracle" not in needed and syms and "oracle" not in syms
