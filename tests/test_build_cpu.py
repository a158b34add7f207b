"""What the build makes, and when: the C ABI's library stands alone, and a binding built against another Python or
PyTorch is neither kept nor loaded."""
import importlib.util

import pytest

from latent_moe_layer_gb300 import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """The build in an empty place, its compilers replaced by notes of what ran."""
    ran = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_experts.so"))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "experts_binding.txt"))
    monkeypatch.setattr(build, "_build_library", lambda force, verbose: ran.append("library") or "lib")

    def binding():
        ran.append("binding")
        (tmp_path / "_experts.so").write_text("")
        (tmp_path / "experts_binding.txt").write_text(build.binding_key())
    monkeypatch.setattr(build, "_build_binding", binding)
    return ran


def test_the_library_needs_neither_pytorch_nor_its_compiler(made, monkeypatch):
    assert build.build(binding=False) == "lib" and made == ["library"]
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == "lib" and made == ["library"] * 2


def test_a_binding_of_another_pytorch_or_python_is_built_again(made, monkeypatch):
    pytest.importorskip("torch")
    build.build()
    assert made.count("binding") == 1 and build.binding_matches()
    build.build()
    assert made.count("binding") == 1
    monkeypatch.setattr(build, "_torch_release", lambda base: "version = 0.0")
    assert not build.binding_matches()
    build.build()
    assert made.count("binding") == 2 and build.binding_matches()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-000")
    assert not build.binding_matches()
    build.build()
    assert made.count("binding") == 3 and build.binding_matches()


def test_a_binding_of_another_pytorch_is_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    from latent_moe_layer_gb300 import experts
    build.build()
    monkeypatch.setattr(experts, "_native", None)
    monkeypatch.setattr(build, "_torch_release", lambda base: "version = 0.0")
    with pytest.raises(ImportError, match="another Python or PyTorch"):
        experts.native()
