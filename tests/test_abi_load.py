"""Loading the library: one built from other sources is refused with an error
that says what to do, and nothing of it is kept."""

import os
import re
import subprocess

import pytest

from helpers import ROOT, mx


def build_stub(path, names, version):
    src = path / "stub.c"
    src.write_text("".join(f"int {n}(void) {{ return {version}; }}\n" for n in names))
    so = path / "libstub.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    return str(so)


@pytest.fixture
def load(monkeypatch, tmp_path):
    m = mx()
    monkeypatch.setattr(m, "_lib", None)

    def run(names, version):
        monkeypatch.setattr(m, "LIB_PATH", build_stub(tmp_path, names, version))
        return m.lib()

    return run


def test_a_library_without_a_declared_call_is_out_of_date(load):
    """As one built before the call was added: the version is the same."""
    m = mx()
    names = [n for n in m.SIGNATURES if n != "mx_rmsnorm_slab"]
    with pytest.raises(m.MXError, match=r"out of date \(no mx_rmsnorm_slab\); run __graft_entry__.build"):
        load(names, m.MX_ABI_VERSION)
    assert m._lib is None


def test_a_library_of_another_version_is_out_of_date(load):
    m = mx()
    with pytest.raises(m.MXError, match="out of date .ABI version 11"):
        load(list(m.SIGNATURES), 11)
    assert m._lib is None


def test_a_whole_library_loads_and_the_version_is_the_headers(load):
    m = mx()
    assert load(list(m.SIGNATURES), m.MX_ABI_VERSION) is m._lib
    text = open(os.path.join(ROOT, "include", "mx.h")).read()
    assert int(re.search(r"#define MX_ABI_VERSION (\d+)", text).group(1)) == m.MX_ABI_VERSION
