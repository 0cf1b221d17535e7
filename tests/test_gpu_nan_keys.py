"""NaN in a key or a value reaches the output it belongs to, and no other: a NaN
key every channel of its KV head's rows, a NaN value its channel."""
import math

import numpy as np
import pytest
import torch

from helpers import TOL
from test_gpu_sparse import attend_by_hand, batch, keys

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16", "e4m3"])
@pytest.mark.parametrize("g", [1, 4])
@pytest.mark.parametrize("form", ["sparse", "long list", "dense", "partitions"])
@pytest.mark.parametrize("at", [0, 7, 150, 238])
def test_nan(native, dtype, g, form, at):
    bs, hkv, d = 8, 3, 128
    k = 1100 if form == "long list" else 30
    lens = [k * bs - 1, 21]
    tables, nb = batch(lens, bs, k)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1), keys((nb, hkv, bs, d), dtype, 2)
    raw = lambda p: p.view(torch.uint8) if dtype == "e4m3" else p  # noqa: E731
    nan = 0x7F if dtype == "e4m3" else math.nan
    clean = kp.clone(), vp.clone()
    raw(kp)[tables[0, at // bs], 0, at % bs, 5] = nan
    raw(vp)[tables[0, at // bs], 1, at % bs, 9] = nan
    q = keys((2, g * hkv, d), "f16" if dtype == "e4m3" else dtype, 3)
    sel = np.full((2, hkv, k), -1, dtype=np.int32)
    sel[0] = np.arange(k)
    sel[1, :, :3] = np.arange(3)
    args = [x.cuda() for x in (q, kp, vp, torch.from_numpy(tables), torch.tensor(lens, dtype=torch.int32))]
    size = 64 if form == "partitions" else 0
    if form in ("sparse", "long list"):
        args.append(torch.from_numpy(sel).cuda())
        out = P.pkv_paged_attention_decode_sparse_fp8(*args, d ** -0.5, 1.0, 1.0) if dtype == "e4m3" else \
            P.pkv_paged_attention_decode_sparse(*args, d ** -0.5)
    else:
        out = P.pkv_paged_attention_decode_fp8(*args, d ** -0.5, 1.0, 1.0, partition_tokens=size) if dtype == "e4m3" \
            else P.pkv_paged_attention_decode(*args, d ** -0.5, partition_tokens=size)
    out = out.cpu().double()
    want = attend_by_hand(q, *(p.float() for p in clean), tables, lens, sel, d ** -0.5)
    want[0, :g] = math.nan
    want[0, g:2 * g, 9] = math.nan
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    ok = ~torch.isnan(want)
    tol = TOL["f16" if dtype == "e4m3" else dtype]
    assert bool(((out - want).abs()[ok] <= tol * want.abs().clamp(min=1)[ok]).all())
    assert P.pkv_device_status(clear=True) == 0
