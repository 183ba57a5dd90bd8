"""The C++ module behind the cache and attention calls: its first use by several threads, and which build is taken."""

import os
import threading
import time

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_topk_gb300 as tks  # noqa: E402
from sparse_attention_topk_gb300 import _build, attention  # noqa: E402

# A stand-in for the module: calls before it has been pointed at a library are errors, as in the real one.
STAND_IN = """
import time
ready = False
def set_library(error, *addresses):
    global ready
    time.sleep(0.05)
    assert len(addresses) == 4 and all(addresses)
    ready = True
def write(*args):
    if not ready:
        raise TypeError("the library is not set")
"""


def test_first_calls_of_several_threads(monkeypatch, tmp_path):
    path = tmp_path / "tks_binding_stand_in.py"
    path.write_text(STAND_IN)
    builds = []

    def build_binding(force=False):
        builds.append(threading.get_ident())
        time.sleep(0.05)
        return str(path)

    monkeypatch.setattr(_build, "build_binding", build_binding)
    monkeypatch.setattr(attention, "_binding", None)
    tks.load()
    failed, begin = [], threading.Barrier(8)

    def call(i):
        try:
            begin.wait()
            time.sleep(0.02 * i)  # (some come while the first builds, some while it points the module at the library)
            tks.cache_write(None, None, None, None, None)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(builds) == 1


def test_another_library_is_taken_up(monkeypatch, tmp_path):
    """A library taken into use before the first call, or after it, is the one that the calls go to."""
    path = tmp_path / "tks_binding_stand_in.py"
    path.write_text("to = []\ndef set_library(error, *addresses): to.append(addresses)\ndef write(*args): pass\n")
    monkeypatch.setattr(_build, "build_binding", lambda force=False: str(path))
    monkeypatch.setattr(attention, "_binding", None)
    lib = tks.load()

    class Other:
        def __getattr__(self, name):
            return getattr(lib, "tks_status_string")

    try:
        attention.bound(Other())
        tks.cache_write(None, None, None, None, None)
        to = attention._binding.to
        assert len(to) == 1 and len(set(to[0])) == 1
        attention.bound(lib)
        assert len(to) == 2 and len(set(to[1])) == 4
    finally:
        attention.bound(lib)


def test_a_build_for_another_torch_or_abi_is_not_taken(monkeypatch):
    assert os.path.exists(_build.build_binding()) and _build._binding_up_to_date()
    for where, name, other in ((torch, "__version__", "0.0.0"), (torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)):
        with monkeypatch.context() as m:
            m.setattr(where, name, other)
            assert not _build._binding_up_to_date()
    assert _build._binding_up_to_date()


def test_builds_side_by_side_have_files_of_their_own(monkeypatch, tmp_path):
    made = []

    class Compiler:
        returncode = 1

        def __init__(self, cmd):
            made.append(cmd[cmd.index("-o") + 1])

        def wait(self):
            return 1 if len(made) > 2 else 0

    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(_build.subprocess, "Popen", Compiler)
    a, b = _build.start_binding(force=True), _build.start_binding(force=True)
    assert made[0] != made[1]
    assert _build.finish_binding(a) == _build.finish_binding(b) and os.listdir(tmp_path) == [os.path.basename(_build.binding_path())]
    with pytest.raises(_build.subprocess.CalledProcessError):  # a build that fails leaves nothing behind
        _build.finish_binding(_build.start_binding(force=True))
    assert len(os.listdir(tmp_path)) == 1
