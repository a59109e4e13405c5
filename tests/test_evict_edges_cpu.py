"""Edges of the rotary and eviction calls that need no GPU: alignment of slices
of larger tensors, frequencies, and how the library and its Python module are
built."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import _lib
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
