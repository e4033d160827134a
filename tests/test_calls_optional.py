"""The package and its build without the compiled calls (_calls.so): every entry
point stays, the helpers take their Python path."""

import importlib.util
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "fine_grained_block_fp8q_amd")

USE = """
    import sys, warnings
    sys.path.insert(0, sys.argv[1])
    import torch
    import unittest.mock as um
    import fine_grained_block_fp8q_amd as fq
    assert fq.abi_version() == 3
    i8, u8, f32, bf16 = torch.int8, torch.uint8, torch.float32, torch.bfloat16
    t = lambda s, d: torch.zeros(s, dtype=d)
    seen = []
    with um.patch.object(fq, "_stream", lambda st, d: None), \\
            um.patch.object(fq, "_invoke", lambda f, a, wh: seen.append(wh)), \\
            warnings.catch_warnings(record=True) as w:
        warnings.simplefilter("always")
        q, s = fq.quantize_token_i8(t((4, 100), bf16))
        assert q.shape == (4, 112) and s.shape == (4,)
        a, sa, wq, ws = t((4, 64), i8), t(4, f32), t((10, 64), i8), t(10, f32)
        assert fq.gemm_i8(a, sa, wq, ws).dtype is f32
        assert fq.gemm_i8_gated(a, sa, wq, ws, act="gelu_tanh").shape == (4, 5)
        e = t((4, 128), u8), t((1, 4), f32)
        h, gu = fq.gemm_gated(*e, t((256, 128), u8), t((2, 1), f32), save_gate_up=True)
        assert h.shape == (4, 128) and gu.shape == (4, 256)
        fq.grouped_gemm_gated(*e, t(3, torch.int32), t((2, 256, 128), u8), t((2, 2, 1), f32))
        r = fq.gated_backward(t((4, 128), bf16), t((4, 256), bf16), tokens=False)
        assert r[0].shape == (4, 256) and r[2] is None
        try:
            fq.gemm_i8(a, sa, t((10, 80), i8), ws)
            raise SystemExit("not refused")
        except ValueError:
            pass
    names = ["quantize_token_i8", "gemm_i8", "gemm_i8_gated", "gemm_gated", "grouped_gemm_gated",
             "gated_backward"]
    assert seen == ["fp8q_" + n for n in names], seen
    said = [str(x.message) for x in w if issubclass(x.category, RuntimeWarning)]
    assert len(said) == 1 and "compiled calls" in said[0], said
    print("used")
"""


@pytest.mark.parametrize("calls", ["absent", "unloadable"])
def test_package_without_the_compiled_calls(tmp_path, calls):
    pkg = tmp_path / "fine_grained_block_fp8q_amd"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "libfp8q.so"), pkg / "libfp8q.so")
    if calls == "unloadable":
        (pkg / "_calls.so").write_bytes(b"not a module")
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(USE), str(tmp_path)], cwd=tmp_path,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("used"), r.stderr


@pytest.mark.parametrize("lacks", ["torch", "g++"])
def test_build_without_what_the_compiled_calls_need(tmp_path, monkeypatch, capsys, lacks):
    spec = importlib.util.spec_from_file_location("_build_of_the_test", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    stale = tmp_path / "_calls.so"
    stale.write_bytes(b"of another torch")
    monkeypatch.setattr(b, "LIB_CALLS", str(stale))
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)    # its import fails
    else:
        monkeypatch.setattr(shutil, "which", lambda name: None)
    b._build_calls(False)
    assert not stale.exists() and f"{lacks} not found" in capsys.readouterr().out
