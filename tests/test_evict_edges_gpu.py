"""Edges of the rotary and eviction calls (GPU): sizes at which parts of a kernel
have nothing to do, slices of larger tensors, large scores, and the calls next
to the attention calls they stand beside."""
import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv

import test_evict_gpu as base

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (256, 8, 2)])
def test_mass_of_rows_of_one_tile(D, Hq, Hkv):
    """One key tile and one query for each of many rows and heads: only one of the
    warps that issue MMAs has any to issue for a query tile."""
    lens = np.random.default_rng(D).integers(0, 128, 500)
    case, lse = base.mass_case(31, [1] * 500, lens, Hq, Hkv, D, 16)
    first = base.run_mass(case, lse)
    assert first[3] == 0
    base.check_mass(case, lse, first)
    ws = pkv.mass_workspace(500, 500, case.max_blocks, Hq, pkv.cache_desc(case.k_cache), DEV)
    for _ in range(50):
        again = base.run_mass(case, lse, ws=ws)
        assert again[3] == 0 and base.same_bits(again[1], first[1])
