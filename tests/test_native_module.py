"""The CPython module of the binding's small calls: what works without it, and when it is built again. No GPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, types
name = "paged_kv_attention_28_gb300._pycall"
if {version!r}:
    fake = types.ModuleType(name)
    fake.torch_version = {version!r}
    fake.linear = lambda *a: 0
    sys.modules[name] = fake
else:
    sys.modules[name] = None  # (importing it raises)
import torch
import paged_kv_attention_28_gb300 as package
if {version!r}:
    package._pycall = fake
from paged_kv_attention_28_gb300 import binding as b
# what needs the library alone
assert b.decode_num_splits(4, 2048, 32, 8, 128, 16, 32) == 32 and b.status_string(0)
assert b.decode_weights_workspace_size(1, 4, 8, 8, 64, 16) > 0
x, pool, i = torch.zeros(2, 64), torch.zeros(4, 2, 16, 64), torch.zeros(1, 4, dtype=torch.int32)
for old in (lambda: b.decode_paged(x.view(1, 2, 64), pool, pool, i, i[0, :1], 0.1), lambda: b.flat_gemm(x, x),
            lambda: b.prefill_paged_chunk(x.view(1, 1, 2, 64), pool, pool, i, i[0, :1], 0.1)):
    try:
        old()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("host tensors were taken")
# what goes through the module says why it cannot
for new in (lambda: b.linear(x, x), lambda: b.cache_evict(pool, pool, i, i[0, :1], x, i, 16),
            lambda: b.qk_norm_rope_append(x.view(1, 1, 2, 64), x, x, pool, pool, i, i[0, :1])):
    try:
        new()
    except ImportError as e:
        assert "_pycall.so" in str(e) and "--force" in str(e) and {version!r} in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


@pytest.fixture(scope="module")
def build():
    from paged_kv_attention_28_gb300 import build as m
    m.build(quiet=True)
    return m


@pytest.mark.parametrize("version", ["", "1.0.3"])
def test_older_calls_need_the_library_alone(build, version):
    """The module missing, or built for another PyTorch."""
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(version=version)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_a_module_of_another_pytorch_is_stale(build, monkeypatch, tmp_path):
    assert not build._module_is_stale()
    built_for = tmp_path / "version"
    monkeypatch.setattr(build, "PYCALL_FOR", str(built_for))
    assert build._module_is_stale()  # unknown
    built_for.write_text("1.0.3")
    assert build._module_is_stale()
    built_for.write_text(build._torch_version())
    assert not build._module_is_stale()
    import torch
    assert build._torch_version().split("+")[0] == torch.__version__.split("+")[0]


def test_a_module_that_cannot_be_built_leaves_the_library(build, monkeypatch, tmp_path, capsys):
    module = tmp_path / "_pycall.so"
    monkeypatch.setattr(build, "PYCALL", str(module))
    monkeypatch.setattr(build, "PYCALL_FOR", str(tmp_path / "version"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    before = os.path.getmtime(build.LIB)
    for cxx in ("false", "/nonexistent/g++"):
        for age in (10 ** 9, 0):
            module.write_text("older than its sources, or of an unknown PyTorch")
            os.utime(module, (os.path.getmtime(module) - age,) * 2)
            monkeypatch.setenv("CXX", cxx)
            assert build.build(quiet=True) == build.LIB
            assert "was not built" in capsys.readouterr().err
            assert module.exists() == (age == 0) and os.path.getmtime(build.LIB) == before
