"""The C++ part of the Python binding is used only where it was compiled for the
library's version and signatures and for this torch (no GPU needed)."""
import subprocess
from types import SimpleNamespace

import pytest

import __graft_entry__ as entry
import combine_topk_ids_02_amd as moe


def other(n, value):
    """built_for() of a module like the right one, with its n-th part another."""
    moe.lib()
    found = list(moe._fast.built_for())
    found[n] = value
    return lambda: tuple(found)


@pytest.fixture
def built():
    moe.lib()
    if moe._fast is None:
        pytest.skip("not built, or built after the package was imported")


def loaded_with(monkeypatch, module):
    """The package's state after a first lib() that finds this module."""
    monkeypatch.setattr(moe, "_lib", None)
    monkeypatch.setattr(moe, "_fast", module)
    monkeypatch.setattr(moe, "_address", module.address)
    moe.lib()
    return moe._fast, moe._address


@pytest.mark.parametrize("n, value", [(0, moe.ABI_VERSION - 1), (1, "2.0.0"), (2, "pippippfpippp"),
                                      (3, ""), (4, "pppqppppp"), (5, "piipppqpppppq")])
def test_a_module_for_something_else_is_not_used(built, monkeypatch, n, value):
    bound = []
    module = SimpleNamespace(built_for=other(n, value), bind=lambda *a: bound.append(a),
                             address=moe._fast.address)
    assert loaded_with(monkeypatch, module) == (None, None)
    assert not bound


def test_a_module_that_does_not_say_is_not_used(built, monkeypatch):
    bound = []
    module = SimpleNamespace(bind=lambda *a: bound.append(a), address=moe._fast.address)
    assert loaded_with(monkeypatch, module) == (None, None)
    assert not bound


def test_the_module_that_fits_is_used(built, monkeypatch):
    module = moe._fast
    assert loaded_with(monkeypatch, module) == (module, module.address)
    assert len(module.built_for()) == 2 + len(moe._FAST_CALLS)


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, "g++"), OSError("no g++")])
def test_a_failed_build_leaves_no_older_module(monkeypatch, tmp_path, error):
    def fails(cmd):
        raise error

    older = tmp_path / "_binding.so"
    older.write_bytes(b"older")
    monkeypatch.setattr(entry, "BINDING_LIB", str(older))
    monkeypatch.setattr(entry, "_run", fails)
    entry.build_binding()
    assert not older.exists()
    entry.build_binding()  # nor does it need one
