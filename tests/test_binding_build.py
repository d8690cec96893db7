"""The binding's marshalling module: built for the interpreter that loads it, and not needed."""
import importlib.machinery
import os

import numpy as np
import pytest

import session_decode_step_gb300 as kd
import test_branching_host as host
from session_decode_step_gb300 import build as kbuild


@pytest.fixture
def lib():
    kbuild.build()
    return kd.lib()


@pytest.fixture
def through_ctypes(lib, monkeypatch):
    monkeypatch.setattr(kd, "_call", kd._CtypesCalls)
    return lib


def test_named_for_the_interpreter(lib, monkeypatch):
    assert kbuild.CALL == kd.CALL_PATH
    assert kbuild.CALL.name == "_kdcall" + importlib.machinery.EXTENSION_SUFFIXES[0] != "_kdcall.so"
    monkeypatch.setattr(kd, "_call", None)
    assert kbuild.CALL.exists() and kd._fast().__file__ == str(kbuild.CALL)


def test_another_interpreters_module_is_not_loaded(lib, monkeypatch, tmp_path):
    """Only files of other names beside the library: the calls go through ctypes."""
    for name in ("_kdcall.so", "_kdcall.cpython-299-any.so"):
        (tmp_path / name).write_bytes(b"not to be loaded")
    monkeypatch.setattr(kd, "CALL_PATH", tmp_path / kd.CALL_PATH.name)
    monkeypatch.setattr(kd, "_call", None)
    assert kd._fast() is kd._CtypesCalls


@pytest.mark.parametrize("missing", ["_cc", "_python_headers"])
def test_builds_without_a_compiler_or_headers(lib, monkeypatch, tmp_path, missing):
    monkeypatch.setattr(kbuild, missing, lambda: None)
    monkeypatch.setattr(kbuild, "CALL", tmp_path / kbuild.CALL.name)
    when = kbuild.LIB.stat().st_mtime_ns
    assert kbuild.build() == kbuild.LIB and not kbuild.CALL.exists()
    kbuild.CALL.write_bytes(b"of older sources")
    os.utime(kbuild.CALL, (1, 1))
    kbuild.build()
    assert not kbuild.CALL.exists()  # nothing out of date stays
    assert kbuild.LIB.stat().st_mtime_ns == when  # and the library is not built again for it


def test_the_module_alone_is_built_again(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(kbuild, "CALL", tmp_path / kbuild.CALL.name)
    when = kbuild.LIB.stat().st_mtime_ns
    kbuild.build()
    assert kbuild.CALL.exists() and kbuild.LIB.stat().st_mtime_ns == when


def test_ctypes_checks_planes(through_ctypes):
    host.test_binding_checks_plane_sizes()


def test_ctypes_refuses_the_same(through_ctypes):
    host.test_binding_refuses_what_it_cannot_pass(through_ctypes)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kind", [list, tuple, lambda v: np.array(v, np.int32), lambda v: np.array(v, np.int64),
                                  lambda v: np.array(v, ">i4")])
def test_ctypes_takes_the_same_arrays(through_ctypes, kind, q8):
    host.test_binding_takes_host_arrays_of_any_kind(through_ctypes, kind, q8)


BAD = [
    lambda: host.bound_window([0], [0], cap=2 ** 31),
    lambda: host.bound_window([0], [0], cap=2 ** 70),
    lambda: host.bound_window([0], [0], cap="8"),
    lambda: host.bound_window([2 ** 40], [0]),
    lambda: host.bound_window([0, 1], [[0], [1], [2]]),
    lambda: host.bound_window([0], [64]),
    lambda: kd.kd_attn_window_append_decode(*[None] * 5, [0], [0], 4, 2, 64, 8, 64, 16, 4, None, 4096),
    lambda: kd.kd_beam_select(None, 1, 2, 100, None, 4, None, None, None, np.zeros(4), ld=2 ** 64),
    lambda: kd.kd_beam_select(np.zeros(4), 1, 2, 100, None, 4, None, None, None, None),
    lambda: kd.kd_beam_select(np.zeros(4), 1, 20, 100, None, 4, np.zeros(4), np.zeros(4), np.zeros(4), np.zeros(4)),
    lambda: kd.kd_kv_reorder(3, [0], [1], [5], 2, 4, 2, 64),
    lambda: kd.kd_kv_reorder([], [0], [1], [5], 2, 4, 2, 64),
    lambda: kd.kd_kv_reorder([np.zeros(2 * 4 * 2 * 64 * 12, np.uint8)], [0], [1], [5], 2, 4, 2, 64),
    lambda: kd.kd_kv_reorder([np.zeros(2 * 4 * 2 * 64 * 8, np.uint8)], [0], [1], [5], 2, 4, 2, 64, window=-1),
    lambda: kd.kd_kv_reorder([np.zeros(2 * 4 * 2 * 64 * 8, np.uint8)], [0, 1], [1, 0], [5], 2, 4, 2, 64),
    lambda: kd.kd_kv_reorder([np.zeros(2 * 4 * 2 * 64 * 8, np.uint8)], [0], [1], [5], 2, 2 ** 31, 2, 64),
]


@pytest.mark.parametrize("bad", BAD)
def test_both_raise_alike(lib, monkeypatch, bad):
    raised = []
    for call in (None, kd._CtypesCalls):
        monkeypatch.setattr(kd, "_call", call)
        with pytest.raises(Exception) as e:
            bad()
        raised.append(e)
    a, b = raised
    assert a.type is b.type, (a.value, b.value)
    if a.type in (kd.KdError, ValueError):
        assert str(a.value) == str(b.value)


@pytest.mark.gpu
def test_both_give_the_same(kdlib, monkeypatch):
    torch = pytest.importorskip("torch")
    import test_gpu_beam as beam
    import test_gpu_window as win
    got = []
    for call in (None, kd._CtypesCalls):
        monkeypatch.setattr(kd, "_call", call)
        res = [win.Case(q8, 3, 8, 2, 128, 300, [5, 130, 299], 100, 4).run(kd) for q8 in (False, True)]
        rng = np.random.default_rng(1)
        res += beam.Call(kd, rng.standard_normal((8, 700)).astype(np.float32), 4, 5, scores=-rng.random(8), pad=4).run()
        planes = [torch.arange(2 * 4 * 2 * 40 * w, device="cuda", dtype=torch.int16).view(2, 4, 2, 40, w) for w in (64, 4)]
        kd.kd_kv_reorder(planes, [0, 1, 2], [1, 2, 0], [40, 30, 7], 2, 4, 2, 40, window=20, sinks=3)
        got.append(res + [p.cpu().numpy() for p in planes])
    for a, b in zip(*got):
        assert np.array_equal(a, b)
