"""The library and the native module of the attention half are built and loaded each for itself (no GPU)."""
import os
import subprocess
import sys

import pytest

from quantized_routed_expert_02_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def built():
    build.build()


def test_the_experts_load_without_the_native_module():
    code = """
import sys
sys.modules["quantized_routed_expert_02_gb300._binding"] = None  # importing it raises, as a module of another PyTorch does
from quantized_routed_expert_02_gb300 import moeq4k as m
assert m.moe_workspace_bytes(1, 2048, 128, 8, 768) > 0 and callable(m.moe_ffn) and callable(m.moe_layer)
assert m.moe_attention_workspace_bytes(32, 4, 128) > 0
for f in (m.moe_add_rmsnorm, m.moe_rope_append, m.moe_attention_paged):
    try:
        f(1, out=2)
    except RuntimeError as e:
        assert "_binding" in str(e) and f.__name__ in str(e)
    else:
        raise AssertionError("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_another_pytorch_asks_for_another_module(monkeypatch):
    assert build.up_to_date()
    monkeypatch.setattr(build, "torch_version", lambda: "0.0 /elsewhere/torch/__init__.py")
    assert not build.up_to_date() and not build.binding_up_to_date() and build.library_up_to_date()


def test_without_pytorch_the_library_alone_is_wanted(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "torch_version", lambda: None)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "none.so"))
    monkeypatch.setattr(build, "nvcc", lambda: pytest.fail("nothing is to be compiled"))
    assert build.up_to_date() and build.build() == build.LIB


def test_a_module_that_does_not_compile_leaves_the_library(monkeypatch, tmp_path):
    """The library is linked before the module's compiler error is raised."""
    broken = tmp_path / "binding.cpp"
    broken.write_text("#error no headers\n")
    small = tmp_path / "small.cu"
    small.write_text("extern \"C\" int small() { return 1; }\n")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "BINDING_SRC", str(broken))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "binding_for"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "_sources", lambda: [str(small)])
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_the_module_follows_the_pytorch_it_was_built_for():
    assert build.torch_version().split()[0] in open(build.BINDING_FOR).read()
