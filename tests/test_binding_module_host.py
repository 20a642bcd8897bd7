"""The binding without its extension module: the functions that do not need it work, the
others name what is missing; and a torch of another version asks for a build."""
import os
import shutil
import subprocess
import sys

import sliding_window_attention_fwd_b200 as swa
from sliding_window_attention_fwd_b200 import build

CHILD = r"""
import torch
import sliding_window_attention_fwd_b200 as swa

print(swa.swa_version(), swa.swa_status_string(-1))
try:  # an entry that reaches its argument checks
    swa.swa_forward(torch.zeros(1), torch.zeros(1), torch.zeros(1))
except ValueError as e:
    print("refused:", e)
t = torch.zeros(1)
for call in (lambda: swa.swa_forward_scored(t, t, t),
             lambda: swa.swa_backward_scored(t, t, t, t, t, t),
             lambda: swa.swa_rope_append_paged(t, t, t, t, t, t, t, t, t, 64),
             lambda: swa.swa_decode_shared(t, t, t, t, 0, t, t, 64, 8)):
    try:
        call()
    except ImportError as e:
        print("missing:", "python -m sliding_window_attention_fwd_b200.build" in str(e))
"""


def run_without(tmp_path, module=None):
    """A copy of the package whose extension module is not there (or is `module`)."""
    src = os.path.dirname(build.__file__)
    dst = tmp_path / os.path.basename(src)
    shutil.copytree(src, dst, ignore=shutil.ignore_patterns("*.so", "__pycache__", "csrc"))
    os.symlink(swa.library_path(), dst / "libswa.so")
    if module:
        (dst / os.path.basename(build.calls_path())).write_bytes(module)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path), "CUDA_VISIBLE_DEVICES": ""})
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert lines[0].startswith(str(swa.swa_version())) and lines[1].startswith("refused:")
    assert lines[2:] == ["missing: True"] * 4


def test_without_the_extension_module(tmp_path):
    run_without(tmp_path)


def test_with_one_that_does_not_load(tmp_path):
    run_without(tmp_path, b"not a library")


def test_another_torch_is_stale(monkeypatch):
    import torch

    assert build.torch_version() == torch.__version__
    assert not build.stale()
    monkeypatch.setattr(build, "torch_version", lambda: "0.1")
    assert build.stale()
