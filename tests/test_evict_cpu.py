"""Refusals of the rotary and eviction calls, which come back before any CUDA
call (no GPU), frequencies, and the plain implementations of their GPU tests."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import _lib
from paged_kv_decode_append_gb300 import workloads as wl
from paged_kv_decode_append_gb300.api import CacheDesc

import evict_ref as ref

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p(0x10004)
OK, EINVAL, EUNSUPPORTED = pkv.api.OK, pkv.api.EINVAL, pkv.api.EUNSUPPORTED
EWORKSPACE = pkv.api.EWORKSPACE
NAN = float("nan")


def test_rope_refusals():
    def rope(q=FAKE, k=FAKE, pos=FAKE, T=4, hq=8, hk=2, D=128, freqs=FAKE, rot=128, pairing=0, a=1.0, qo=FAKE, ko=FAKE):
        return _lib.load().pkv_rope(q, k, pos, T, hq, hk, D, freqs, rot, pairing, a, qo, ko, None)

    assert rope(D=96, rot=64) == EUNSUPPORTED and rope(rot=24) == EUNSUPPORTED
    assert rope(rot=144) == EINVAL and rope(rot=0) == EINVAL and rope(rot=-16) == EINVAL
    assert rope(pairing=2) == EINVAL and rope(a=NAN) == EINVAL and rope(a=math.inf) == EINVAL
    assert rope(q=None) == EINVAL and rope(ko=None) == EINVAL and rope(q=None, qo=None, k=None, ko=None) == EINVAL
    assert rope(T=-1) == EINVAL and rope(hq=0) == EINVAL and rope(hk=0) == EINVAL and rope(hk=-1) == EINVAL
    assert rope(pos=None) == EINVAL and rope(freqs=None) == EINVAL
    assert rope(q=ODD) == EINVAL and rope(k=ODD) == EINVAL and rope(qo=ODD) == EINVAL and rope(ko=ODD) == EINVAL
    assert rope(T=0) == OK


def test_rope_append_refusals():
    d = CacheDesc(64, 16, 2, 128, 1)

    def append(desc=d, kc=FAKE, vc=FAKE, q=FAKE, k=FAKE, v=FAKE, T=4, indptr=FAKE, freqs=FAKE, rot=64, pairing=1, a=1.0,
               table=FAKE, width=4, lens=FAKE, batch=2, hq=8, qo=FAKE):
        return _lib.load().pkv_rope_append(ctypes.byref(desc), kc, vc, q, k, v, T, indptr, None, None, freqs, rot, pairing, a,
                                           table, width, lens, batch, hq, qo, None, None)

    assert append(desc=CacheDesc(64, 16, 2, 96, 1)) == EUNSUPPORTED and append(desc=CacheDesc(1, 16, 2, 64, 1)) == EINVAL
    assert append(rot=40) == EUNSUPPORTED and append(rot=256) == EINVAL and append(pairing=-1) == EINVAL
    assert append(T=4, indptr=None) == EINVAL and append(q=None) == EINVAL and append(qo=None) == EINVAL
    assert append(kc=None) == EINVAL and append(v=None) == EINVAL and append(k=None) == EINVAL and append(lens=None) == EINVAL
    assert append(kc=ODD) == EINVAL and append(v=ODD) == EINVAL and append(q=ODD) == EINVAL and append(qo=ODD) == EINVAL
    assert append(table=None) == EINVAL and append(freqs=None) == EINVAL and append(a=NAN) == EINVAL
    assert append(width=0) == EINVAL and append(batch=-1) == EINVAL and append(T=-1) == EINVAL and append(hq=0) == EINVAL
    assert append(batch=0) == OK and append(T=0) == OK


def test_mass_refusals():
    d = CacheDesc(64, 16, 2, 128, 1)

    def mass(desc=d, kc=FAKE, q=FAKE, indptr=FAKE, lse=FAKE, table=FAKE, width=4, lens=FAKE, batch=2, hq=8, T=9, scale=0.1,
             out=FAKE, pos=None, slots=64, ws=FAKE, ws_bytes=1 << 40):
        return _lib.load().pkv_attn_mass(ctypes.byref(desc), kc, q, indptr, lse, table, width, lens, batch, hq, T, scale, None,
                                         None, out, pos, slots, ws, ws_bytes, None, None)

    assert mass(desc=CacheDesc(64, 16, 2, 96, 1)) == EUNSUPPORTED and mass(desc=CacheDesc(64, 4, 2, 128, 1)) == EUNSUPPORTED
    assert mass(hq=7) == EINVAL and mass(hq=258) == EUNSUPPORTED and mass(batch=1025) == EUNSUPPORTED
    assert mass(T=-1) == EINVAL and mass(T=1 << 28) == EUNSUPPORTED and mass(width=0) == EINVAL and mass(slots=0) == EINVAL
    assert mass(indptr=None) == EINVAL and mass(scale=NAN) == EINVAL
    assert mass(kc=None) == EINVAL and mass(q=None) == EINVAL and mass(lse=None) == EINVAL and mass(out=None) == EINVAL
    assert mass(table=None) == EINVAL and mass(lens=None) == EINVAL
    assert mass(kc=ODD) == EINVAL and mass(q=ODD) == EINVAL and mass(out=ODD) == EINVAL and mass(pos=ODD) == EINVAL
    assert mass(ws=None) == EWORKSPACE and mass(ws_bytes=16) == EWORKSPACE
    assert mass(batch=0) == OK and mass(T=0) == OK
    assert pkv.pkv_mass_workspace_size(2, 9, 4, 8, d) >= 256 and pkv.pkv_mass_workspace_size(2, 9, 4, 7, d) == 0


def test_plan_refusals():
    def plan(mass=FAKE, pos=FAKE, layers=1, batch=2, hk=2, slots=64, lens=FAKE, budgets=FAKE, sink=0, recent=0, moves=FAKE,
             most=32, num=FAKE, rows=FAKE):
        return _lib.load().pkv_evict_plan(mass, pos, layers, batch, hk, slots, lens, None, budgets, sink, recent, moves, most,
                                          num, rows, None, None)

    assert plan(layers=0) == EINVAL and plan(batch=-1) == EINVAL and plan(hk=0) == EINVAL and plan(slots=0) == EINVAL
    assert plan(sink=-1) == EINVAL and plan(recent=-1) == EINVAL and plan(most=0) == EINVAL
    assert plan(slots=(1 << 19) + 1) == EUNSUPPORTED and plan(layers=1 << 20, batch=1 << 10, hk=4) == EUNSUPPORTED
    assert plan(mass=None) == EINVAL and plan(pos=None) == EINVAL and plan(lens=None) == EINVAL and plan(budgets=None) == EINVAL
    assert plan(moves=None) == EINVAL and plan(num=None) == EINVAL and plan(rows=None) == EINVAL
    assert plan(mass=ODD) == EINVAL and plan(pos=ODD) == EINVAL and plan(moves=ODD) == EINVAL
    assert plan(batch=0) == OK


def test_apply_refusals():
    one = (ctypes.c_void_p * 1)(0x10000)
    odd = (ctypes.c_void_p * 1)(0x10008)
    none = (ctypes.c_void_p * 1)(0)

    def apply(desc=CacheDesc(64, 16, 2, 128, 1), layers=1, k=one, v=one, moves=FAKE, most=4, num=FAKE, rows=FAKE, table=FAKE,
              width=4, slots=64, lens=FAKE, gone=FAKE, batch=2):
        return _lib.load().pkv_evict_apply(ctypes.byref(desc), layers, k, v, moves, most, num, rows, table, width, FAKE, FAKE,
                                           slots, lens, gone, batch, None, None)

    assert apply(desc=CacheDesc(64, 16, 2, 96, 1)) == EUNSUPPORTED and apply(layers=0) == EINVAL
    assert apply(layers=129) == EUNSUPPORTED and apply(k=None) == EINVAL and apply(v=odd) == EINVAL and apply(k=none) == EINVAL
    assert apply(moves=None) == EINVAL and apply(moves=ODD) == EINVAL and apply(num=None) == EINVAL and apply(rows=None) == EINVAL
    assert apply(table=None) == EINVAL and apply(most=0) == EINVAL and apply(width=0) == EINVAL and apply(slots=0) == EINVAL
    assert apply(lens=None) == EINVAL and apply(batch=-1) == EINVAL and apply(batch=0) == OK


def test_the_binding_refuses_host_tensors():
    x, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        pkv.pkv_rope(f, None, x, x)
    with pytest.raises(ValueError):
        pkv.pkv_rope(None, None, x, x)
    with pytest.raises(ValueError):
        pkv.pkv_evict_plan(f[None], x, x, x, x, 0, 0)
    with pytest.raises(ValueError):
        pkv.pkv_attn_mass(torch.zeros(2, 16, 1, 64), f, f, x[None], x, 1.0, f)


def turns(radians):
    return np.asarray(radians) / (2 * math.pi) * 2.0 ** 64


def freqs(*args, **kw):
    f, a = pkv.rope_freqs(*args, device="cpu", **kw)
    return f.numpy().view(np.uint64).astype(np.float64), a


def test_frequencies():
    """Against the formulas in 64 bits: a few roundings of 2^-53 in the powers
    (the exponent's product by ln(base) below 14 magnifies them to 2^-49), and
    half a unit of 2^-64 where the frequency becomes a whole number of them."""
    i = np.arange(32)
    g = 1e6 ** (-2.0 * i / 64)

    def near(f, radians):
        return (np.abs(f - turns(radians)) <= 0.5 + 2.0 ** -46 * turns(radians)).all()

    f, a = freqs(64, 1e6)
    assert a == 1.0 and near(f, g)
    f, a = freqs(64, 1e6, scaling="linear", factor=8.0)
    assert a == 1.0 and near(f, g / 8)
    f, a = freqs(64, 1e4, scaling="ntk", factor=4.0)
    assert near(f, (1e4 * 4 ** (64 / 62)) ** (-2.0 * i / 64))
    f, a = freqs(64, 1e4, scaling="turns", factor=8.0, low=1.0, high=4.0, orig_len=8192)
    g = 1e4 ** (-2.0 * i / 64)
    n = 8192 * g / (2 * math.pi)
    want = np.where(n >= 4, g, np.where(n <= 1, g / 8, g / 8 + (g - g / 8) * (n - 1) / 3))
    assert near(f, want) and a == 1.0
    f, a = freqs(64, 1e4, scaling="parts", factor=16.0, low=1.0, high=32.0, orig_len=4096)
    assert a == np.float32(0.1 * math.log(16) + 1)
    at = [64 * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(1e4)) for t in (32.0, 1.0)]
    lo, hi = math.floor(at[0]), math.ceil(at[1])
    part = np.clip((i - lo) / (hi - lo), 0, 1)
    assert near(f, g / 16 * part + g * (1 - part)) and 0 < part.sum() < 32


def test_frequency_refusals():
    for kw in (dict(rot_dim=0), dict(rot_dim=3), dict(base=1.0), dict(base=math.inf), dict(base=NAN),
               dict(scaling="linear", factor=0.5), dict(scaling="ntk", rot_dim=2, factor=2.0),
               dict(scaling="parts", factor=2.0, low=2.0, high=1.0, orig_len=10.0), dict(scaling="turns", factor=2.0),
               dict(scaling="turns", factor=NAN, orig_len=10.0), dict(scaling="parts", factor=2.0, orig_len=math.inf)):
        with pytest.raises(pkv.PkvError):
            pkv.rope_freqs(**{**dict(rot_dim=64, device="cpu"), **kw})
    with pytest.raises(ValueError):
        pkv.rope_freqs(64, scaling="none", device="cpu")
    assert _lib.load().pkv_rope_freqs(64, 1e4, 0, 1.0, 1.0, 2.0, 1.0, None, None) == EINVAL
    assert _lib.load().pkv_rope_freqs(64, 1e4, 5, 1.0, 1.0, 2.0, 1.0, (ctypes.c_uint64 * 32)(), None) == EINVAL


def test_plain_rotation():
    f = pkv.rope_freqs(16, 100.0, device="cpu")[0].numpy().view(np.uint64)
    x = np.random.default_rng(0).standard_normal((3, 2, 64))
    for inter in (False, True):
        y, size = ref.rotate(x, [0, 5, -7], f, inter, 1.5)
        assert np.array_equal(y[..., 16:], x[..., 16:]) and np.allclose(y[0, :, :16], 1.5 * x[0, :, :16])
        a, b = (x[1, 0, 4], x[1, 0, 5]) if inter else (x[1, 0, 2], x[1, 0, 10])
        z = complex(a, b) * 1.5 * np.exp(1j * 5 * 100.0 ** (-4 / 16))
        got = (y[1, 0, 4], y[1, 0, 5]) if inter else (y[1, 0, 2], y[1, 0, 10])
        assert abs(complex(*got) - z) < 1e-12
        back, _ = ref.rotate(y, [0, -5, 7], f, inter, 1 / 1.5)
        assert np.allclose(back, x)


def test_plain_mass():
    """Weights of a row add up to its queries and heads; the plan's choice."""
    case = wl.mixed_step(5, [4, 3], [20, 0], 4, 2, 64, 8, wl.HND)
    for b in range(2):
        lo, n, L = int(case.qo_indptr[b]), int(np.diff(case.qo_indptr)[b]), int(case.cache_seqlens[b])
        for pool, new in ((case.k_cache, case.k_new),):
            pos = np.arange(L, L + n)
            wl.scatter_tokens(pool, case.layout, 8, case.block_table[b, pos // 8], pos % 8, new[lo:lo + n])
        lse = torch.zeros(case.q.shape[:2], dtype=torch.float64)
        lse[lo:lo + n] = ref.lse_of(case, b, lo, n, L)
        got, tol = ref.mass_row(case, b, lo, n, L, lse)
        assert np.allclose(got.sum(1), 2 * n) and (tol > 0).all() and (tol < 1e-2).all()
    m = np.array([1, 5, 5, NAN, 2, 7, 5, 0], np.float32)
    pos = np.array([9, 1, 2, 0, 10, 12, 13, 3], np.int32)
    # keep 4 of 8: the newest of 14 (slot 6) and position 0 (slot 3) first, then 7 and the first 5
    assert ref.plan_row(m, pos, 8, 6, 4, 1, 1) == [(5, 0), (6, 2)]
    assert ref.plan_row(m, pos, 8, 6, 8, 1, 1) == [] and ref.plan_row(m, pos, 8, 6, -1, 0, 0) == []
    assert ref.plan_row(m, pos, 8, 6, 1, 0, 0) == [(5, 0)] and ref.plan_row(m, pos, 8, 6, 0, 0, 0) == []
