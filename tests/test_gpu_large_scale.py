"""A scale that takes q, but no score, beyond 32 bits' range: q of some units,
a scale of 1e38, keys of 0 or with four channels of some 4e-39.

A score (up to 15) is rounded by at most 3 x 2^-24 of itself and a weight by
another 2^-22, so an output is within 2 (3 x 15 x 2^-24 + 2^-22) max |v| < 3e-5
of the 64-bit one; helpers.TOL for 16-bit pools.
"""
import numpy as np
import pytest
import torch

from helpers import TOL
from test_gpu_sparse import attend_by_hand, batch, keys

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402


@pytest.mark.parametrize("dtype,small", [("f32", 4e-39), ("bf16", 4e-39), ("f32", 0.0), ("bf16", 0.0), ("f16", 0.0)])
@pytest.mark.parametrize("g", [1, 4])
@pytest.mark.parametrize("k", [20, 1100])
def test_large_scale(native, dtype, small, g, k):
    bs, hkv, d, scale = 8, 2, 128, 1e38
    lens = [1200 * bs - 3 if k > 1024 else 30 * bs - 3]
    tables, nb = batch(lens, bs, k)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1) * small, keys((nb, hkv, bs, d), dtype, 2)
    kp[..., 4:] = 0
    q = keys((1, g * hkv, d), dtype, 3) * 4
    sel = np.tile(np.arange(k, dtype=np.int32) + 2, (1, hkv, 1))
    every = np.tile(np.arange(-(-lens[0] // bs), dtype=np.int32), (1, hkv, 1))
    args = [x.cuda() for x in (q, kp, vp, torch.from_numpy(tables), torch.tensor(lens, dtype=torch.int32))]
    for out, chosen in ((P.pkv_paged_attention_decode_sparse(*args, torch.from_numpy(sel).cuda(), scale), sel),
                        (P.pkv_paged_attention_decode(*args, scale), every)):
        want = attend_by_hand(q, kp, vp, tables, lens, chosen, scale)
        tol = 3e-5 if dtype == "f32" else TOL[dtype] * want.abs().clamp(min=1)
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert P.pkv_device_status(clear=True) == 0
