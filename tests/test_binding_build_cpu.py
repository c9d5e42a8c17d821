"""What works without _binding.so, and when it is built."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "rwkv_linear_attention_wkv_b200"


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


WITHOUT = f"import sys; sys.modules['{PACKAGE}._binding'] = None\n"


def test_everything_imports_without_it():
    got = python(WITHOUT + f"""
import warnings
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    from {PACKAGE} import *
    from {PACKAGE}.autograd import gated_delta_rule, norm_gate, wkv
assert len(told) == 1 and "build.py" in str(told[0].message), told
assert wkv_gdr_forward and wkv_norm_gate_backward
""")
    assert got.returncode == 0, got.stderr


def test_without_it_calls_go_the_long_way():
    # (which refuses a host tensor; a missing extension would be another error)
    got = python(WITHOUT + f"""
import warnings; warnings.simplefilter("ignore")
import torch, {PACKAGE} as W
x, g, S = torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 3), torch.zeros(1, 3, 64, 64)
for call in (lambda: W.wkv_gdr_forward(x, x, x, g, g), lambda: W.wkv_gdr_forward_checkpointed(x, x, x, g, g),
             lambda: W.wkv_gdr_backward(x, x, x, g, g, x, S),
             lambda: W.wkv_gdr_decode_step(x[0], x[0], x[0], g[0], g[0], S),
             lambda: W.wkv_norm_gate_forward(x, act="none"),
             lambda: W.wkv_norm_gate_backward(x, None, x, act="none")):
    try:
        call()
        raise SystemExit("not refused")
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
""")
    assert got.returncode == 0, got.stderr


def test_one_of_another_torch_is_not_used():
    got = python(f"""
import warnings, torch
import {PACKAGE}._binding as b
assert b.torch_version == torch.__version__
b.torch_version = "0.0"
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    from {PACKAGE} import gdr
assert len(told) == 1 and gdr._binding is not b
""")
    assert got.returncode == 0, got.stderr


@pytest.fixture
def build(monkeypatch):
    spec = importlib.util.spec_from_file_location("_wkv_build", os.path.join(ROOT, PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    ran = []
    monkeypatch.setattr(b.subprocess, "check_call", lambda cmd: ran.append(cmd))
    monkeypatch.setattr(b.os, "replace", lambda *a: None)
    monkeypatch.setattr(b, "up_to_date", lambda: True)
    return b, ran


def test_build_makes_it(build, tmp_path):
    b, ran = build
    b.BINDING = str(tmp_path / "none.so")
    b.build()
    assert len(ran) == 1 and b.BINDING_SOURCE in ran[0]


def test_another_torch_rebuilds_it(build, monkeypatch):
    b, ran = build
    monkeypatch.setattr(b, "torch_version", lambda: "0.0.1", raising=False)
    b.build_binding()
    assert len(ran) == 1 and b.BINDING_SOURCE in ran[0]
