"""Batches large enough for the kernels that serve them: block-sparse decode of
more rows than the GPU has SMs (three-warp CTAs), block selection over more
sequences than a warp numbers at a time (128), and selections whose border lies
inside the error of 32-bit scores.

Selections are compared for equality.  Attention: scores of head_dim 128 of
N(0, 1) inputs are off by at most 128 x 2^-24 x sum |q k| / sqrt(128) < 1e-4, so
an output by less than 2e-4 max |v| (5 at most here) = 1e-3 at worst; over the
many rows the mean error is that of rounding, below 1e-5.
"""
import math

import numpy as np
import pytest
import torch

from helpers import DT
from test_gpu_sparse import batch, bounds_of, check_select, choose, keys, spoil

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def attend(q, kp, vp, tables, lens, sel, scale):
    """All rows at once, in 64 bits on the device."""
    B, hq, d = q.shape
    hkv, bs = kp.shape[1], kp.shape[2]
    sel = sel.long()
    phys = tables.long()[:, None, :].expand(-1, hkv, -1).gather(2, sel.clamp(min=0)).clamp(min=0)
    token = sel[..., None] * bs + torch.arange(bs, device="cuda")
    live = ((sel >= 0)[..., None] & (token < lens.long()[:, None, None, None])).flatten(2)
    head = torch.arange(hkv, device="cuda")[None, :, None].expand_as(phys)
    k, v = (p.float()[phys, head].double().flatten(2, 3).masked_fill(~live[..., None], 0) for p in (kp, vp))
    s = q.double().view(B, hkv, -1, d) @ k.transpose(2, 3) * scale
    w = torch.softmax(s.masked_fill(~live[:, :, None], -math.inf), -1)
    return torch.nan_to_num(w, nan=0.0).matmul(v).view(B, hq, d)  # an empty list: zeros


@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 1), ("bf16", 128, 4), ("bf16", 64, 2), ("bf16", 64, 8),
                                       ("f16", 128, 2), ("f16", 128, 8), ("f16", 64, 4), ("e4m3", 128, 1),
                                       ("e4m3", 128, 2), ("e4m3", 128, 4), ("e4m3", 128, 8)])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("num_seqs,hkv,k", [(50, 3, 30), (149, 1, 13), (75, 2, 1), (297, 1, 5), (130, 5, 9)])
def test_sparse_decode_of_many_rows(dtype, d, g, bs, num_seqs, hkv, k):
    """150 rows (clusters of two where the lists are long), 149, 297 and 650."""
    rng = np.random.default_rng(num_seqs + bs + g)
    lens = [int(n) for n in rng.integers(0, 2 * k * bs, num_seqs)]
    lens[:6] = [0, 1, bs - 1, bs, bs + 1, 2 * k * bs]
    tables, nb = batch(lens, bs, d + g + k)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1), keys((nb, hkv, bs, d), dtype, 2)
    spoil(kp, tables, lens, bs)
    spoil(vp, tables, lens, bs)
    q = keys((num_seqs, g * hkv, d), "f16" if dtype == "e4m3" else dtype, 3)
    sel = choose(lens, bs, hkv, k, k)
    sel[7] = -1  # a sequence with nothing selected
    args = [x.cuda() for x in (q, kp, vp, torch.from_numpy(tables), torch.tensor(lens, dtype=torch.int32),
                               torch.from_numpy(sel))]
    got = P.pkv_paged_attention_decode_sparse_fp8(*args, d ** -0.5, 1.0, 1.0) if dtype == "e4m3" else \
        P.pkv_paged_attention_decode_sparse(*args, d ** -0.5)
    want = attend(*args, d ** -0.5)
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all()) and float(err.max()) <= 1e-3 and float(err.mean()) <= 1e-5
    empty = torch.from_numpy((sel >= 0).sum(-1) == 0).repeat_interleave(g, 1).cuda()
    assert bool((got[empty] == 0).all())


@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("f16", 64, 1), ("e4m3", 128, 8), ("f32", 64, 2)])
@pytest.mark.parametrize("num_seqs", [127, 128, 129, 256, 300])
def test_select_over_many_sequences(dtype, d, g, num_seqs):
    """Runs of sequences with nothing to choose, across the borders at 128."""
    bs, hkv, k = 8, 2, 6
    rng = np.random.default_rng(num_seqs)
    for kind in ("mixed", "none around 128", "only the last", "only the first", "none"):
        lens = rng.integers(0, 60 * bs, num_seqs)
        short = rng.integers(0, k * bs + 1, num_seqs)
        at = np.arange(num_seqs)
        if kind == "mixed":
            few = rng.random(num_seqs) < 0.5
        elif kind == "none around 128":
            few = (at > 90) & (at < 170)
        elif kind == "only the last":
            few, lens[-1] = at < num_seqs - 1, 59 * bs + 1
        elif kind == "only the first":
            few, lens[0] = at > 0, 59 * bs + 1
        else:
            few = at >= 0
        lens = [int(n) for n in np.where(few, short, lens)]
        tables, nb = batch(lens, bs, num_seqs)
        bounds = bounds_of(nb, hkv, d, dtype, g)
        q = keys((num_seqs, g * hkv, d), "f16" if dtype == "e4m3" else dtype, 5)
        check_select(q, bounds, tables, lens, k, bs, 1, 2)


@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("bf16", 64, 1), ("f16", 128, 8), ("f16", 64, 2),
                                       ("e4m3", 128, 1), ("e4m3", 128, 4), ("f32", 128, 4)])
@pytest.mark.parametrize("blocks", [300, 4000])
@pytest.mark.parametrize("tiny", [2.0 ** -2, 2.0 ** -5, 2.0 ** -8, 2.0 ** -12])
def test_select_where_large_channels_cancel(dtype, d, g, blocks, tiny):
    """Half of the channels are large and cancel exactly, the others are `tiny`
    of them: from scores spread over many times the assumed error of 32-bit
    sums (2^-14 of sum |q| max |bound|) to scores all within it.  The border
    then lies among 300 blocks ranked in shared memory, or 4000 of which more
    than 512 go to the radix selection.

    The 32-bit scores (they lie at the start of the workspace) keep to that
    error: it is an assumption on how tensor cores align a sum, measured here."""
    bs, hkv, k = 8, 2, 20
    lens = [blocks * bs - 5, 7]
    tables, nb = batch(lens, bs, blocks)
    rng = np.random.default_rng(int(1 / tiny) + d + g)
    pt, io = (torch.float8_e4m3fn, torch.float16) if dtype == "e4m3" else (DT[dtype], DT[dtype])
    top = 240.0 if dtype == "e4m3" else 1000.0
    t, L = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.empty(P.pkv_select_workspace_size(2, hkv, tables.shape[1]), dtype=torch.uint8, device="cuda")
    for trial in range(3):
        # q > 0 everywhere, so a score is q.hi: pairs of channels +x and -x with equal q cancel
        q = torch.from_numpy(rng.uniform(0.5, 2.0, (2, g * hkv, d)).astype(np.float32)).to(io)
        # in order, the sum first grows to its largest; else in a random one
        large = torch.from_numpy(rng.permutation(d)[:d // 2].copy()) if trial else torch.arange(d // 2)
        a, b = large[:d // 4], large[d // 4:]
        q[..., b] = q[..., a]
        hi = torch.from_numpy(rng.standard_normal((nb, hkv, d), dtype=np.float32)) * (top * tiny / 4)
        x = torch.from_numpy(rng.uniform(-top, top, (nb, hkv, d // 4)).astype(np.float32)).to(pt).float()
        hi[..., a], hi[..., b] = x, -x
        hi = hi.to(pt).float()
        bounds = torch.stack([hi - 1, hi], 2).to(pt)  # the lower bounds are not used
        check_select(q, bounds, tables, lens, k, bs, 1, 2)
        P.pkv_block_select(q.cuda(), bounds.cuda(), t, L, k, bs, 1, 2, workspace=ws)
        scores = ws[:2 * hkv * tables.shape[1] * 4].view(torch.float32).view(2, hkv, -1)[0, :, :blocks].cpu().double()
        for h in range(hkv):
            heads, b = q[0, h * g:(h + 1) * g].double(), bounds[tables[0].astype(np.int64), h].float().double()
            err = (scores[h] - (b[:, 1] @ heads.T).amax(-1)).abs().max()
            assert float(err) <= float(heads.sum(-1).max() * b.abs().max()) * 2.0 ** -14, float(err)
