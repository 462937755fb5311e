"""What the compiled part of the attention binding may break: itself.  The C library is linked
before it and without torch, and the scans import and run where it is missing or does not load."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "selective_state_space_s6_amd")

USE = """
import selective_state_space_s6_amd as m
assert m.ssm_s6_scan_fwd_workspace_size(1, 64, 16, 4) >= 0 and callable(m.ssd_chunk_scan_fwd)
assert set(m.__all__) <= set(dir(m))
assert m.ssm_paged_attn_decode_fwd_workspace_size(4, 8, 2, 64, 8, 16) > 0 and m.SSM_KV_F8E4M3 == 2
for call in (lambda: m.ssm_kv_pages_step(None, None, None, None, None, page_size=1, n_tokens=1),
             lambda: m.ssm_paged_attn_decode_fwd(None, None, None, None, None, scale=1.0)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and "_attn_bind" in str(e), e
    else:
        raise AssertionError("nothing raised")
print("fine")
"""


@pytest.mark.parametrize("there", [None, b"", b"not a library"], ids=["missing", "empty", "unreadable"])
def test_the_scans_import_without_the_attention_binding(tmp_path, there):
    to = tmp_path / "selective_state_space_s6_amd"
    to.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py"):
            shutil.copy(os.path.join(PKG, f), to)
    os.symlink(os.path.join(PKG, "libssmscan.so"), to / "libssmscan.so")
    if there is not None:
        (to / "_attn_bind.so").write_bytes(there)
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py with its compilers noted instead of run."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.HERE, mod.LIB, mod.BIND = str(tmp_path), str(tmp_path / "lib.so"), str(tmp_path / "bind.so")
    mod.ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        mod.ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        done = Done()
        if mod.fails(cmd):
            done.returncode = 1
        else:
            open(out, "w").close()
        return done
    mod.fails = lambda cmd: False
    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod


def test_the_library_is_linked_before_the_binding(build):
    build.fails = lambda cmd: cmd[0] == "g++"
    with pytest.raises(RuntimeError, match="bind_attn"):
        build.build(verbose=False)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    build.fails = lambda cmd: False
    assert build.build(verbose=False) == build.LIB and os.path.exists(build.BIND)


def test_the_library_needs_no_torch(build, monkeypatch, capsys):
    there = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else there(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)          # importing it raises
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    assert all("g++" not in c[0] for c in build.ran) and "torch" in capsys.readouterr().out
