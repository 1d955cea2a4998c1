"""A device-side wait that gave up is told by Seq: by check() and, at the latest, by close().  The library is a
stand-in whose status word is set, so that no wait has to run out."""
import ctypes

import pytest

import mixed_precision_refinement_gb300 as zs
from mixed_precision_refinement_gb300 import seq as binding


class Library:
    def __init__(self, status):
        self.status, self.destroyed = status, 0

    def zsolve_seq_check(self, seq):
        status, self.status = self.status, zs.ZSOLVE_OK  # as the library: told once
        return status

    def zsolve_seq_last_error(self, seq):
        return b"a bounded device-side wait gave up"

    def zsolve_strerror(self, status):
        return b"timeout"

    def zsolve_seq_destroy(self, seq):
        self.destroyed += 1


@pytest.fixture
def make(monkeypatch):
    made = []

    def _make(status):
        lib = Library(status)
        monkeypatch.setattr(binding, "_lib", lib)
        s = zs.Seq.__new__(zs.Seq)
        s.seq = ctypes.c_void_p(1)
        made.append(s)
        return s, lib

    yield _make
    for s in made:
        s.seq = None  # nothing of the stand-in reaches the library


def test_check_raises_once(make):
    s, lib = make(zs.ZSOLVE_ETIMEOUT)
    with pytest.raises(zs.ZsolveError) as e:
        s.check()
    assert e.value.status == zs.ZSOLVE_ETIMEOUT
    s.check()
    s.close()
    assert lib.destroyed == 1 and s.seq is None


@pytest.mark.parametrize("block", [False, True])
def test_close_raises_and_releases(make, block):
    s, lib = make(zs.ZSOLVE_ETIMEOUT)
    with pytest.raises(zs.ZsolveError):
        if block:
            with s:
                pass
        else:
            s.close()
    assert lib.destroyed == 1 and s.seq is None
    s.close()  # again: nothing left to release
    assert lib.destroyed == 1


def test_an_exception_of_the_block_goes_on(make):
    s, lib = make(zs.ZSOLVE_ETIMEOUT)
    with pytest.raises(KeyError):
        with s:
            raise KeyError
    assert lib.destroyed == 1


@pytest.mark.parametrize("status", [zs.ZSOLVE_OK, zs.ZSOLVE_ECUDA])
def test_close_without_a_give_up(make, status):
    s, lib = make(status)
    s.close()
    assert lib.destroyed == 1
    s, lib = make(zs.ZSOLVE_ETIMEOUT)
    s.__del__()  # the collector's: silent
    assert lib.destroyed == 1
