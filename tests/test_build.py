"""What is built when, and what works without the marshalling module of the prompt side.  The compilers are stand-ins
that write their output file and a line to a log."""
import importlib.util
import os
import shutil
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "paged_kv_cache_17_gb300"


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """The build script over a folder of its own, with stand-in compilers; builder.ran() are the files made since
    the last call."""
    spec = importlib.util.spec_from_file_location("pkv_build_test", os.path.join(ROOT, PACKAGE, "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    log = tmp_path / "log"
    for name in ("nvcc", "cxx"):
        exe = tmp_path / name
        exe.write_text(f'''#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && out="$2"; shift; done
echo "$out" >> {log}
[ -z "$FAIL_{name}" ] && echo made > "$out"
''')
        exe.chmod(exe.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "cxx"))
    m.OUT_DIR = str(tmp_path / "_lib")
    m.LIB, m.BIND = os.path.join(m.OUT_DIR, "libpkv.so"), os.path.join(m.OUT_DIR, "_pkv_prompt.so")
    m.BOUND_TO = m.BIND + ".bound_to"

    def ran():
        made = log.read_text().split() if log.exists() else []
        log.write_text("")
        return {os.path.basename(x).split(".tmp")[0] for x in made}

    m.ran = ran
    return m


def test_everything_once(builder):
    assert builder.build() == builder.LIB
    made = builder.ran()
    assert {"libpkv.so", "_pkv_prompt.so", "prompt_bind.o", "prefill_tc.o"} <= made and len(made) == len(builder.SOURCES) + 3
    builder.build()
    assert builder.ran() == set()
    builder.build(force=True)
    assert builder.ran() == made


def test_binding_is_made_again_for_another_torch(builder, monkeypatch):
    builder.build()
    builder.ran()
    monkeypatch.setattr(builder, "_bound_to", lambda: "another torch")
    builder.build()
    assert builder.ran() == {"prompt_bind.o", "_pkv_prompt.so"}
    builder.build()
    assert builder.ran() == set()


def test_library_alone_where_the_headers_are_missing(builder, monkeypatch, tmp_path, capsys):
    builder.build()
    builder.ran()
    monkeypatch.setattr(builder.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert builder.build(force=True) == builder.LIB
    made = builder.ran()
    assert "libpkv.so" in made and not {"_pkv_prompt.so", "prompt_bind.o"} & made
    assert not os.path.exists(builder.BIND)  # what was there may be bound to something else
    assert "Python.h" in capsys.readouterr().err
    builder.build()
    assert builder.ran() == set()


def test_library_is_in_place_when_the_binding_fails(builder, monkeypatch):
    monkeypatch.setenv("FAIL_cxx", "1")
    with pytest.raises(RuntimeError, match="prompt_bind"):
        builder.build()
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.BIND)


def test_failure_of_a_kernel_is_raised(builder, monkeypatch):
    monkeypatch.setenv("FAIL_nvcc", "1")
    with pytest.raises(RuntimeError):
        builder.build()
    assert not os.path.exists(builder.LIB)


@pytest.mark.parametrize("left", [None, "not a library"], ids=["missing", "not loadable"])
def test_import_without_the_binding(tmp_path, left):
    """The decode side imports, and the prompt side's calls say what is missing."""
    import __graft_entry__

    __graft_entry__.build()
    src, dst = os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE
    (dst / "_lib").mkdir(parents=True)
    for f in os.listdir(src):
        if f.endswith(".py"):
            shutil.copy(os.path.join(src, f), dst / f)
    shutil.copy(os.path.join(src, "_lib", "libpkv.so"), dst / "_lib" / "libpkv.so")
    if left is not None:
        (dst / "_lib" / "_pkv_prompt.so").write_text(left)
    code = f"""
import torch, {PACKAGE} as pkv
assert pkv.__file__.startswith({str(tmp_path)!r})
assert pkv.version() > 0 and len(pkv.rope_inv_freq(64)[0]) == 32 and callable(pkv.paged_decode_attention)
t = torch.zeros(1)
for call in (lambda: pkv.paged_prefill_attention(t, t, t, t, t, t, 1.0), lambda: pkv.paged_kv_gather(t, t, t, t, t, t),
             lambda: pkv.qk_norm_rope_append(t, t, t, t, t, t, t)):
    try:
        call()
    except ImportError as e:
        assert "_build" in str(e)
    else:
        raise SystemExit("no error")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr
