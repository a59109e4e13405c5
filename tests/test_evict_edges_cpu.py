"""Edges of the rotary and eviction calls that need no GPU: alignment of slices
of larger tensors, frequencies, and how the library and its Python module are
built."""
import ctypes

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
