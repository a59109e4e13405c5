"""Edges of the rotary and eviction calls that need no GPU: alignment of slices
of larger tensors, frequencies, and how the library and its Python module are
built."""
import ctypes
import math
import os
from decimal import Decimal, localcontext

import numpy as np
import pytest

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import _lib
from paged_kv_decode_append_gb300 import build as pkv_build
from paged_kv_decode_append_gb300.api import CacheDesc

FAKE = 0x10000  # aligned, never dereferenced on these paths
EINVAL, EWORKSPACE = pkv.api.EINVAL, pkv.api.EWORKSPACE


def test_alignment_of_slices():
    """Layers of one state begin on 4 bytes unless slots is a multiple of 4, lse of
    some of the tokens too (the refusal of the workspace comes next)."""
    d = CacheDesc(64, 16, 1, 128, 1)

    def mass(out=FAKE, pos=FAKE, lse=FAKE, slots=65):
        return _lib.load().pkv_attn_mass(ctypes.byref(d), FAKE, FAKE, FAKE, lse, FAKE, 4, FAKE, 2, 8, 9, 0.1, None, None, out,
                                         pos, slots, None, 0, None, None)

    for at in (4, 8, 12):
        assert mass(out=FAKE + at) == mass(pos=FAKE + at) == mass(lse=FAKE + at) == EWORKSPACE
        assert mass(out=FAKE + at, slots=64) == mass(pos=FAKE + at, slots=64) == EINVAL
    for at in (1, 2, 3, 6):
        assert mass(out=FAKE + at) == mass(pos=FAKE + at) == mass(lse=FAKE + at) == EINVAL
    assert mass(pos=None) == EWORKSPACE


def test_apply_refuses_scores_between_words():
    """Scores and positions off a 4-byte boundary, which no load may take."""
    one = (ctypes.c_void_p * 1)(FAKE)

    def apply(mass=FAKE, pos=FAKE, slots=65):
        return _lib.load().pkv_evict_apply(ctypes.byref(CacheDesc(64, 16, 1, 128, 1)), 1, one, one, FAKE, 4, FAKE, FAKE, FAKE, 4,
                                           mass, pos, slots, FAKE, FAKE, 2, None, None)

    for at in (1, 2, 3):
        for slots in (64, 65):
            assert apply(mass=FAKE + at, slots=slots) == apply(pos=FAKE + at, slots=slots) == EINVAL


def turns_of(*args, **kw):
    """Frequencies in turns per token of 64-bit floats."""
    f, _ = pkv.rope_freqs(*args, device="cpu", **kw)
    return f.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64


@pytest.mark.parametrize("rot,base", [(16, 1e4), (64, 1e4), (128, 5e5)])
@pytest.mark.parametrize("scaling", ["parts", "turns"])
def test_pairs_of_at_most_low_turns_are_stretched(rot, base, scaling):
    """g / factor where a pair makes at most `low` turns, g where at least `high`,
    for lengths at which all pairs, some or none make them.  Either frequency is
    made of a few roundings of 2^-53, magnified by at most ln(base) < 14, and
    becomes a whole number of 2^-64, which is off by half of one: together their
    ratio is off by 2^-46 of itself and 2^-64 / g at most."""
    low, high, factor = 2.0, 16.0, 8.0
    plain = turns_of(rot, base)
    for length in (1.0, 6.0, 2 * math.pi * low, 12.6, 13.0, 30.0, 100.0, 1e3, 1e5, 1e9):
        made = length * plain
        got = turns_of(rot, base, scaling=scaling, factor=factor, low=low, high=high, orig_len=length) / plain
        off = 2.0 ** -46 + 2.0 ** -64 / plain
        slow, fast = made <= low * (1 - 1e-9), made >= high * (1 + 1e-9)
        assert (np.abs(got - 1 / factor) <= off)[slow].all() and (np.abs(got - 1.0) <= off)[fast].all()
        assert (got >= 1 / factor - off).all() and (got <= 1 + off).all()
        assert length > 7 or slow.all()


@pytest.mark.parametrize("rot,base", [(16, 150000000), (64, 10000), (128, 1000000), (256, 500000)])
@pytest.mark.parametrize("scaling,factor", [("plain", 1), ("linear", 3), ("linear", 8), ("ntk", 4), ("ntk", 7)])
def test_frequencies_against_60_digits(rot, base, scaling, factor):
    """Within 2^-53 turns per token: with g radians, the power is off by two steps of
    2^-53 and by the exponent's rounding, |ln g| of them, two pi, the two divisions
    and a changed base by one each, in all (6 + |ln g|) g 2^-53 / (2 pi) at most,
    which is largest at g = 1; and by half of 2^-64."""
    f, _ = pkv.rope_freqs(rot, float(base), scaling=scaling, factor=float(factor), device="cpu")
    with localcontext() as digits:
        digits.prec = 60
        turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        b = base * (Decimal(factor) ** (Decimal(rot) / (rot - 2)) if scaling == "ntk" else 1)
        for i, got in enumerate(f.numpy().view(np.uint64).tolist()):
            want = b ** (Decimal(-2 * i) / rot) / turn / (factor if scaling == "linear" else 1)
            assert abs(Decimal(got) / 2 ** 64 - want) <= Decimal(2) ** -53


def fail():
    raise ImportError("no torch with CUDA here")


@pytest.mark.parametrize("job", ["missing", "compile", "link"])
def test_the_library_is_built_where_its_python_module_cannot_be(tmp_path, monkeypatch, capfd, job):
    here = str(tmp_path)
    for name, value in (("HERE", here), ("BUILD_DIR", os.path.join(here, "_build")), ("LIB_PATH", os.path.join(here, "libpkv.so")),
                        ("CUDA_SOURCES", []), ("CXX_SOURCES", ["pkv_pool.cc"])):
        monkeypatch.setattr(pkv_build, name, value)
    ok, no = ["true", "-o", None], ["false", "-o", None]
    monkeypatch.setattr(pkv_build, "_module_job",
                        {"missing": fail, "compile": lambda: (no[:1], list(ok)), "link": lambda: (ok[:1], list(no))}[job])
    assert not pkv_build.up_to_date()
    assert pkv_build.build() == pkv_build.LIB_PATH and os.path.getsize(pkv_build.LIB_PATH) > 0 and pkv_build.up_to_date()
    assert "pkv_torch was not built" in capfd.readouterr().err and not os.path.exists(pkv_build.module_path())
    with pytest.raises((ImportError, RuntimeError)):  # asked for by name: why not
        pkv_build.build_module()


def test_a_module_of_another_torch_or_python_is_not_taken(monkeypatch):
    import sysconfig

    import torch

    pkv_build.build()
    path = pkv_build.build_module()
    assert pkv_build.module_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert pkv_build.module_path() != path and not pkv_build.module_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".other.so")
        assert pkv_build.module_path() != path and not pkv_build.module_up_to_date()
    assert _lib.calls().__file__ == path
