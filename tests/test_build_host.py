"""The build on a host without torch, and the paged calls where only the C library was built."""
import os
import subprocess
import sys

import pytest

import global_gqa_b200 as g3

NO_TORCH = "import sys; sys.modules['torch'] = None; "


@pytest.fixture(scope="module", autouse=True)
def built():
    from global_gqa_b200 import build
    build.build()


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=g3.ROOT, capture_output=True, text=True, timeout=600)


def test_build_without_torch_builds_the_library_alone():
    r = python(NO_TORCH + "import runpy; sys.argv = ['build']; runpy.run_module('global_gqa_b200.build', run_name='__main__')")
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().endswith("libg3attn.so") and "_paged.so" in r.stderr


def test_library_loads_without_torch():
    r = python(NO_TORCH + "import global_gqa_b200 as g; print(g.paged_decode_workspace_size(128) > 0, sorted(set(g.header_functions()) - set(dir(g.lib()))) == [] )")
    assert r.returncode == 0 and r.stdout.startswith("True"), r.stderr


def test_paged_calls_without_the_quick_module_take_the_ordinary_way(monkeypatch):
    import torch
    monkeypatch.setattr(g3, "_quick", None)
    monkeypatch.setattr(g3, "HERE", os.path.join(g3.ROOT, "nonexistent"))
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="_paged.so is missing"), pytest.raises(ValueError, match="CUDA"):
        g3.page_map(i32, i32, i32[:, None], i32, i32, 16, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        g3.page_bounds(torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), i32[:, None], i32, i32, None, None)
    assert g3._quick is g3._Ordinary  # and says so once


def test_a_warning_that_is_an_error_stops_one_call_only(monkeypatch):
    import warnings

    import torch
    monkeypatch.setattr(g3, "_quick", None)
    monkeypatch.setattr(g3, "HERE", os.path.join(g3.ROOT, "nonexistent"))
    i32 = torch.zeros(2, dtype=torch.int32)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning):
            g3.page_map(i32, i32, i32[:, None], i32, i32, 16, 4, 8)
        with pytest.raises(ValueError, match="CUDA"):
            g3.page_map(i32, i32, i32[:, None], i32, i32, 16, 4, 8)
