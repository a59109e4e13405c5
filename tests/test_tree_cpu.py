"""Refusals of the tree and table calls, which come back before any CUDA call
(no GPU), and the plain implementations their GPU tests are held to."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import _lib
from paged_kv_decode_append_gb300 import workloads as wl
from paged_kv_decode_append_gb300.api import CacheDesc

import tree_ref as ref

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p(0x10004)
OK, EINVAL, EUNSUPPORTED = pkv.api.OK, pkv.api.EINVAL, pkv.api.EUNSUPPORTED
EWORKSPACE = pkv.api.EWORKSPACE


def attn(desc, batch=2, hq=8, total_q=40, nodes=32, words=1, ws=FAKE, ws_bytes=1 << 40, q=FAKE, k_new=FAKE,
         v_new=FAKE, scale=0.1, max_blocks=4, mask=FAKE, out=FAKE):
    return _lib.load().pkv_tree_attn(ctypes.byref(desc), FAKE, FAKE, q, k_new, v_new, FAKE, mask, words, FAKE,
                                     max_blocks, FAKE, batch, hq, total_q, nodes, scale, out, None, ws, ws_bytes, None, None)


def test_attention_refusals():
    d = CacheDesc(64, 16, 2, 128, 1)
    assert attn(CacheDesc(64, 16, 2, 96, 1)) == EUNSUPPORTED   # head dim
    assert attn(CacheDesc(64, 4, 2, 128, 1)) == EUNSUPPORTED   # page below 8
    assert attn(CacheDesc(1, 16, 2, 128, 1)) == EINVAL
    assert attn(d, hq=7) == EINVAL                             # Hq % Hkv
    assert attn(d, hq=258) == EUNSUPPORTED                     # 129 heads per kv head
    assert attn(d, nodes=0) == EINVAL
    assert attn(d, nodes=257, words=8) == EUNSUPPORTED
    assert attn(d, nodes=33) == EINVAL                         # one word of mask
    assert attn(d, words=9) == EUNSUPPORTED
    assert attn(d, words=0) == EINVAL
    assert attn(d, q=None) == EINVAL
    assert attn(d, mask=None) == EINVAL
    assert attn(d, k_new=None) == EINVAL                       # one of the pair
    assert attn(d, out=ODD) == EINVAL
    assert attn(d, scale=float("nan")) == EINVAL
    assert attn(d, ws=None) == EWORKSPACE
    assert attn(d, ws_bytes=16) == EWORKSPACE
    assert attn(d, batch=0) == OK
    assert attn(d, total_q=0) == OK
    assert attn(d, batch=1025) == EUNSUPPORTED
    assert attn(d, total_q=-1) == EINVAL
    assert attn(d, total_q=1 << 28) == EUNSUPPORTED            # total_q * Hq
    assert attn(d, max_blocks=0) == EINVAL


def test_workspace_size():
    d = CacheDesc(65536, 16, 8, 128, 0)
    n = pkv.pkv_tree_workspace_size(64, 4096, 2049, 32, 64, d)
    assert n >= 256
    assert pkv.pkv_tree_workspace_size(1025, 4096, 2049, 32, 64, d) == 0
    assert pkv.pkv_tree_workspace_size(64, 4096, 2049, 30, 64, d) == 0
    assert pkv.pkv_tree_workspace_size(64, 4096, 2049, 32, 257, d) == 0


def test_build_refusals():
    def build(batch=2, total=9, nodes=8, mask=FAKE, words=1, parents=FAKE):
        return _lib.load().pkv_tree_build(parents, FAKE, FAKE, batch, total, nodes, mask, words, None, None, None)

    assert build(nodes=0) == EINVAL and build(nodes=257, words=8) == EUNSUPPORTED
    assert build(nodes=33) == EINVAL and build(words=9) == EUNSUPPORTED and build(words=0) == EINVAL
    assert build(batch=-1) == EINVAL and build(total=-1) == EINVAL
    assert build(mask=None) == EINVAL and build(parents=None) == EINVAL
    assert build(batch=0) == OK and build(total=0) == OK


def test_accept_refusals():
    def accept(batch=2, total=9, nodes=8, path=FAKE, max_path=4, length=FAKE, draft=FAKE):
        return _lib.load().pkv_tree_accept(FAKE, draft, FAKE, None, FAKE, FAKE, batch, total, nodes, path, max_path,
                                           length, None, None, None, None)

    assert accept(nodes=0) == EINVAL and accept(nodes=257) == EUNSUPPORTED and accept(max_path=0) == EINVAL
    assert accept(path=None) == EINVAL and accept(length=None) == EINVAL and accept(draft=None) == EINVAL
    assert accept(batch=-1) == EINVAL and accept(batch=0) == OK


def test_commit_refusals():
    one = (ctypes.c_void_p * 1)(0x10000)
    odd = (ctypes.c_void_p * 1)(0x10008)
    none = (ctypes.c_void_p * 1)(0)

    def commit(desc=CacheDesc(64, 16, 2, 128, 1), layers=1, k=one, v=one, path=FAKE, max_path=4, batch=2, max_blocks=4):
        return _lib.load().pkv_tree_commit(ctypes.byref(desc), layers, k, v, path, max_path, FAKE, FAKE, max_blocks,
                                           FAKE, batch, None, None)

    assert commit(desc=CacheDesc(64, 16, 2, 96, 1)) == EUNSUPPORTED
    assert commit(layers=0) == EINVAL and commit(layers=129) == EUNSUPPORTED
    assert commit(k=None) == EINVAL and commit(v=odd) == EINVAL and commit(k=none) == EINVAL
    assert commit(max_path=0) == EINVAL and commit(max_path=257) == EUNSUPPORTED and commit(path=None) == EINVAL
    assert commit(max_blocks=0) == EINVAL and commit(batch=-1) == EINVAL and commit(batch=0) == OK


def test_table_refusals():
    def update(pool=FAKE, pages=64, P=16, table=FAKE, width=4, held=FAKE, batch=2, slots=None, tokens=0):
        return _lib.load().pkv_table_update(pool, pages, P, table, width, held, FAKE, FAKE, batch, None, slots, None,
                                            tokens, None, None)

    assert update(pages=1) == EINVAL and update(P=0) == EINVAL and update(width=0) == EINVAL
    assert update(P=24) == EUNSUPPORTED and update(P=512) == EUNSUPPORTED and update(batch=1025) == EUNSUPPORTED
    assert update(batch=-1) == EINVAL and update(tokens=-1) == EINVAL
    assert update(pool=None) == EINVAL and update(table=None) == EINVAL and update(held=None) == EINVAL
    assert update(slots=ODD, tokens=4) == EINVAL and update(batch=0) == OK
    lib = _lib.load()
    assert lib.pkv_device_pool_bytes(1) == 0 and lib.pkv_device_pool_bytes(9) == 4 * (16 + 8)
    assert lib.pkv_device_pool_init(None, 1 << 20, 9, None) == EINVAL
    assert lib.pkv_device_pool_init(FAKE, 95, 9, None) == EINVAL
    assert lib.pkv_device_pool_init(FAKE, 1 << 20, 1, None) == EINVAL


def test_pools_past_32_bit_ring_indices_are_refused():
    lib = _lib.load()
    most = 1 << 30
    assert lib.pkv_device_pool_bytes(most) == 4 * (16 + most - 1)
    for pages in (most + 1, 2 ** 31 - 1):
        assert lib.pkv_device_pool_bytes(pages) == 0
        assert lib.pkv_device_pool_init(FAKE, 1 << 40, pages, None) == EUNSUPPORTED
        assert lib.pkv_table_update(FAKE, pages, 16, FAKE, 4, FAKE, FAKE, FAKE, 2, None, None, None, 0, None,
                                    None) == EUNSUPPORTED


def test_the_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.pkv_tree_build(x, x, x, 4)
    with pytest.raises(ValueError):
        pkv.pkv_tree_accept(x, x, x, None, x, x, 4)
    with pytest.raises(ValueError):
        pkv.pkv_table_update(x, x, x, x, x, 16)
    with pytest.raises(ValueError):
        pkv.LayerCaches([], [])
    with pytest.raises(ValueError):
        pkv.LayerCaches([torch.zeros(2, 8, 1, 64)], [torch.zeros(2, 8, 1, 64)])


def test_plain_attention_against_torch():
    case = wl.mixed_step(5, [4, 3], [20, 0], 4, 2, 64, 8, wl.HND)
    seen = [ref.ancestor_bits(p) for p in ([-1, 0, 0, 2], [-1, -1, 1])]
    out, lse, tol = ref.attention(case, seen)
    for b in range(2):
        lo, hi, L = int(case.qo_indptr[b]), int(case.qo_indptr[b + 1]), int(case.cache_seqlens[b])
        k, v = ref.row_kv(case, b, hi - lo, True)
        full = np.concatenate([np.ones((hi - lo, L), bool), seen[b]], 1)
        got = torch.nn.functional.scaled_dot_product_attention(
            case.q[lo:hi].double().transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1),
            v.repeat_interleave(2, 1).transpose(0, 1), attn_mask=torch.as_tensor(full)).transpose(0, 1)
        assert np.abs(got.numpy() - out[lo:hi]).max() < 1e-12
    assert np.isfinite(lse).all() and (tol > 0).all()


def test_plain_walks():
    assert ref.ancestor_bits([-1, 0, 0, 2]).astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]]
    assert ref.pack([ref.ancestor_bits([-1, 0, 1])], 2).tolist() == [[1, 0], [3, 0], [7, 0]]
    # children 1 and 2 both carry the target's token: the first is taken
    assert ref.accept([-1, 0, 0, 1], [5, 6, 6, 7], [6, 7, 9, 8], 5, 9) == ([0, 1, 3], 8)
    assert ref.accept([-1, 0], [5, 6], [6, 7], 4, 9) == ([], 4)
    assert ref.accept([-1, 0], [5, 6], [6, 7], None, 1) == ([0], 6)
    pool = ref.TablePool(5, 2, 3, 4)
    indptr, slots, pos, failed = pool.update([0, 3], [5, 1])
    assert indptr.tolist() == [0, 5, 6] and slots.tolist() == [4, 5, 6, 7, 8, 15] and pos.tolist() == [0, 1, 2, 3, 4, 3]
    assert not failed and pool.free == [4]
    assert pool.update([-1, 4], [0, 8])[3] == {1: "pool"}
    assert pool.free == [4, 1, 2] and math.isclose(pool.held[1], 1)
