"""What the build makes, and what it does without the Python headers."""
import ctypes
import os
import subprocess
import sys
import sysconfig

import pytest

from w4a16_routed_expert_router_gb300 import _build

ROOT = os.path.dirname(_build.PKG)


def test_the_binding_is_named_after_its_interpreter():
    assert _build.build_binding()
    assert os.path.exists(_build.BINDING)
    assert os.path.basename(_build.BINDING) == "_attn_binding" + sysconfig.get_config_var(
        "EXT_SUFFIX")


def test_the_library_builds_without_python_headers(monkeypatch, tmp_path, capsys):
    _build.build()
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_attn_binding.so"))
    assert _build.python_headers() is None
    assert _build.build() == _build.LIB
    assert "no Python headers" in capsys.readouterr().err
    assert not os.path.exists(_build.BINDING)
    ctypes.CDLL(_build.LIB).moe_w4a16_status_string


def test_a_binding_that_does_not_compile_is_an_error(monkeypatch, tmp_path):
    bad = tmp_path / "binding.c"
    bad.write_text("not C\n")
    monkeypatch.setattr(_build, "BINDING_SRC", str(bad))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_attn_binding.so"))
    with pytest.raises(RuntimeError, match="binding.c failed"):
        _build.build_binding()


def test_attention_says_what_is_missing():
    code = ("import sys; sys.modules['w4a16_routed_expert_router_gb300._attn_binding'] = None\n"
            "import w4a16_routed_expert_router_gb300 as moe\n"
            "moe.lib().moe_w4a16_status_string(0)\n"
            "try:\n    moe.moe_attn_rope_frequencies(8, device='cpu')\n"
            "except RuntimeError as e:\n    print('said:', e)\n")
    _build.build()
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0 and "said: the attention operators' Python binding" in out.stdout
