"""The package without its compiled module, or with one that was built for another torch."""

import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

import split_kv_decode_flashdecoding_b200 as fd

PKG = os.path.dirname(fd.__file__)
PROGRAM = """
import torch
import split_kv_decode_flashdecoding_b200 as fd
info, splits, items = fd.fd_split_plan([700, 3], 2, 1024)
assert len(items) == info["total_items"] > 0
x, n = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
for call in (lambda: fd.fd_prompt_attention(x, x, x, n), lambda: fd.fd_pages_free(n, n, n, n)):
    try:
        call()
    except ImportError as e:
        print(e)
"""


def _builder():
    spec = importlib.util.spec_from_file_location("fd_build", os.path.join(PKG, "build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("module", ["none", "broken", "for another torch"])
def test_what_does_not_need_the_module_runs_without_it(tmp_path, module):
    to = tmp_path / "split_kv_decode_flashdecoding_b200"
    to.mkdir()
    shutil.copy(os.path.join(PKG, "libfd.so"), to)
    program = PROGRAM
    if module == "broken":
        (to / "_fd_binding.so").write_bytes(b"\x7fELF of something else")
    if module == "for another torch":
        shutil.copy(os.path.join(PKG, "_fd_binding.so"), to)
        program = program.replace("import torch\n", "import torch\ntorch.__version__ = '0.1'\n", 1)
    shutil.copy(os.path.join(PKG, "__init__.py"), to)
    r = subprocess.run([sys.executable, "-c", program], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    lines = r.stdout.strip().splitlines()
    assert len(lines) == 2 and all("needs _fd_binding.so" in x and "build.py" in x for x in lines)
    if module == "for another torch":
        assert "this is 0.1" in lines[0]


def test_the_module_is_built_again_for_another_torch(monkeypatch):
    b = _builder()
    b.build_binding()
    assert b.binding_up_to_date()
    monkeypatch.setattr(b, "_torch_version", lambda: "0.1")
    assert not b.binding_up_to_date()


def test_the_module_is_for_this_torch():
    import torch
    assert fd._fd_binding.torch_version == torch.__version__ == _builder()._torch_version()
