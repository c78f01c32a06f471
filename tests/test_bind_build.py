"""The compiled Python side of the pool operators (_bind) belongs to one torch, one Python and one machine: it is
built anew for another, and its absence says what to do."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def build():
    from speculative_decode_persistent_gb300 import build as b
    b.build()
    return b


def _stale(b):
    return b._bind_stale([])


def test_built_once(build):
    assert not _stale(build)
    at = os.path.getmtime(build.BIND)
    build.build()
    assert os.path.getmtime(build.BIND) == at


def test_another_torch_python_or_machine(build, monkeypatch):
    for mod, name, value in ((build.importlib.metadata, "version", lambda n: "0.0"), (build.sysconfig, "get_config_var", lambda n: "other"),
                             (build.platform, "machine", lambda: "other"), (build.importlib.util, "find_spec", lambda n: None)):
        with monkeypatch.context() as m:
            m.setattr(mod, name, value)
            assert _stale(build)
        assert not _stale(build)
    monkeypatch.setattr(build, "BIND_KEY", build.BIND_KEY + ".none")
    assert _stale(build)


def test_a_missing_module_says_what_to_do(build):
    code = ("import sys; sys.modules['speculative_decode_persistent_gb300._bind'] = None\n"
            "import speculative_decode_persistent_gb300.mk\n"
            "import speculative_decode_persistent_gb300.ops")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode and "build()" in r.stderr.splitlines()[-1]


def test_a_torch_without_package_data(build, monkeypatch):
    def none(name):
        raise build.importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(build.importlib.metadata, "version", none)
    assert len(build._bind_key().splitlines()) == 4
