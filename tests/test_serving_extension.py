"""The extension through which Python calls the serving operators (CPU): the codec
does without it, and a call that needs it says so."""
import os
import subprocess
import sys

import pytest
import torch

import kv_quantization_tile_b200
from kv_quantization_tile_b200 import _build, hq
from kv_quantization_tile_b200._build import ext_path

PKG = os.path.dirname(os.path.abspath(kv_quantization_tile_b200.__file__))


@pytest.fixture
def bare(tmp_path):
    """A copy of the package with its library and without the extension."""
    to = tmp_path / "kv_quantization_tile_b200"
    to.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py") or name == "libhq.so":
            os.symlink(os.path.join(PKG, name), to / name)
    return to


def python(package, code):
    return subprocess.run([sys.executable, "-c", code], cwd=package.parent, capture_output=True, text=True,
                          env={**os.environ, "PYTHONPATH": str(package.parent)})


USE = """
import torch
from kv_quantization_tile_b200 import hq
assert hq.hq_version() >= 100 and hq.hq_tile_bound_words(256, "E8", 4.0) > 0
table, x = hq.rope_table(64, device="cpu"), torch.zeros(1, 1, 64)
for call in (lambda: hq.hq_rope(x, torch.zeros(1, dtype=torch.int64), table, x),
             lambda: hq.hq_attention_merge(x, x[..., 0], x, x[..., 0], x)):
    try:
        call()
    except ImportError as e:
        assert "g.build()" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_the_codec_does_without_the_extension(bare):
    r = python(bare, USE)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_an_extension_that_does_not_load_counts_as_missing(bare):
    (bare / os.path.basename(ext_path())).write_bytes(b"not a library")
    r = python(bare, USE)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_an_extension_for_another_torch_is_neither_loaded_nor_kept(bare, monkeypatch):
    ours = ext_path()
    assert os.path.samefile(hq._hq_torch.__file__, ours)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    theirs = ext_path()
    assert theirs != ours and _build.stale()  # built again for the torch that is there
    os.symlink(ours, bare / os.path.basename(theirs))
    r = python(bare, USE)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr
    os.symlink(ours, bare / os.path.basename(ours))
    r = python(bare, USE)
    assert r.returncode != 0 and "CUDA tensors only" in r.stderr  # loaded: it looks at the tensors
