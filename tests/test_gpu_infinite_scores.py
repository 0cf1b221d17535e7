"""Scores of -inf: infinite keys, keys at the type's lowest value whose product
with q overflows, a scale that overflows a score.  A token that scores -inf has
weight 0, wherever it comes first (a warp's first chunk, a partition, the whole
first tile); a row of nothing else gives zeros.

The expectation is the softmax in 64 bits with those tokens' weights set to 0.
Tolerance: helpers.TOL; scores of finite tokens are those of N(0, 1) inputs (or
all zero), the -inf tokens add nothing to sums.
"""
import math

import numpy as np
import pytest
import torch

from helpers import DT, TOL

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402

TYPES = {**DT, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def make(kind, dtype, g, n, bs, gone, d=128, hkv=2, seed=0):
    """One sequence of n tokens: q, pools, table, scale; the tokens `gone`
    score -inf for every head (kind "lowest": for the even heads only)."""
    rng = np.random.default_rng(seed)
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    nblk = -(-n // bs)
    order = rng.permutation(nblk + 2)[:nblk]
    io = torch.float16 if dtype == "e4m3" else DT[dtype]
    q = normal(1, g * hkv, d).abs() + 0.5
    k, v = normal(nblk * bs, hkv, d), normal(nblk * bs, hkv, d)
    scale, dead = d ** -0.5, torch.ones(g * hkv, dtype=torch.bool)
    gone = torch.as_tensor(gone)
    if kind == "infinite":
        k[gone] = -math.inf
    elif kind == "lowest":
        k[gone] = torch.finfo(DT[dtype]).min
        q[:, 1::2] *= 1e-36  # scores of some -1e4: the weights of those heads come out 0 all the same, but finite
        dead[1::2] = False
    else:  # q.k is 0 or at most -100: times 1e38 beyond 32 bits
        k.zero_()
        k[gone] = -4.0
        scale = 1e38
    pool = lambda x: x.view(nblk, bs, hkv, d).transpose(1, 2).to(TYPES[dtype])  # noqa: E731
    kp, vp = (torch.zeros(nblk + 2, hkv, bs, d).to(TYPES[dtype]) for _ in range(2))
    for p, x in ((kp, k), (vp, v)):
        raw = torch.uint8 if dtype == "e4m3" else p.dtype
        p.view(raw)[order] = pool(x).contiguous().view(raw)
    return q.to(io), kp, vp, torch.from_numpy(order.astype(np.int32))[None], scale, gone, dead


def attend(q, kp, vp, table, scale, gone, tokens):
    """64-bit softmax over the given tokens, those of `gone` left out."""
    hkv, bs, d = kp.shape[1:]
    g = q.shape[1] // hkv
    tokens = torch.as_tensor(np.setdiff1d(np.asarray(list(tokens)), gone.numpy()))
    out = torch.zeros(q.shape[1], d, dtype=torch.float64)
    if not tokens.numel():
        return out
    blk, r = table[0].long()[tokens // bs], tokens % bs
    for h in range(hkv):
        k, v = (p.float()[blk, h, r].double() for p in (kp, vp))
        out[h * g:(h + 1) * g] = torch.softmax(q[0, h * g:(h + 1) * g].double() @ k.T * scale, -1) @ v
    return out


def close(got, want, dtype):
    tol = TOL["f16" if dtype == "e4m3" else dtype] * want.abs().clamp(min=1)
    assert bool(((got.cpu().double() - want).abs() <= tol).all()), float((got.cpu().double() - want).abs().max())


KINDS = [("infinite", "f32"), ("infinite", "bf16"), ("infinite", "f16"), ("lowest", "f32"), ("lowest", "bf16"),
         ("scale", "f32"), ("scale", "bf16"), ("scale", "f16"), ("scale", "e4m3")]


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("bs,k", [(8, 40), (16, 40), (32, 40), (8, 1100)])  # the last: beyond the cluster kernel's list
def test_sparse(kind, dtype, g, bs, k):
    n = 1200 * bs - 3 if k > 1024 else 60 * bs - 3
    blocks = np.sort(np.random.default_rng(k).permutation(-(-n // bs))[:k])
    # the tokens of the first blocks of the list, of one in its middle and of its last
    dead = [*blocks[:k // 8 + 1], blocks[k // 2], blocks[-1]]
    gone = [t for j in dead for t in range(j * bs, min(n, (j + 1) * bs))]
    q, kp, vp, table, scale, gone, _ = make(kind, dtype, g, n, bs, gone)
    sel = torch.from_numpy(np.tile(blocks.astype(np.int32), (1, 2, 1)))
    args = (q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    call = lambda s: P.pkv_paged_attention_decode_sparse_fp8(*args, s.cuda(), scale, 1.0, 1.0) if dtype == "e4m3" \
        else P.pkv_paged_attention_decode_sparse(*args, s.cuda(), scale)  # noqa: E731
    tokens = [t for j in blocks for t in range(j * bs, min(n, (j + 1) * bs))]
    close(call(sel)[0], attend(q, kp, vp, table, scale, gone, tokens), dtype)
    nothing = torch.full_like(sel, -1)
    nothing[..., :3] = torch.tensor(np.sort(dead[:3]).astype(np.int32))
    got = call(nothing)[0].cpu()  # every selected token scores -inf
    heads = torch.arange(2 * g) % 2 == 0 if kind == "lowest" else torch.ones(2 * g, dtype=torch.bool)
    assert bool((got[heads] == 0).all()) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("g", [1, 4])
@pytest.mark.parametrize("partition", [0, 256])
def test_dense(kind, dtype, g, partition):
    """The decode over every token: a first tile, a whole partition, the last tokens."""
    bs, n = 16, 3000
    q, kp, vp, table, scale, gone, _ = make(kind, dtype, g, n, bs, [*range(400), *range(1024, 1280), 2998, 2999])
    args = (q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), scale)
    got = P.pkv_paged_attention_decode_fp8(*args, 1.0, 1.0, partition_tokens=partition) if dtype == "e4m3" else \
        P.pkv_paged_attention_decode(*args, partition_tokens=partition)
    close(got[0], attend(q, kp, vp, table, scale, gone, range(n)), dtype)
    short = (*args[:4], torch.tensor([390], dtype=torch.int32).cuda(), scale)
    got = P.pkv_paged_attention_decode_fp8(*short, 1.0, 1.0, partition_tokens=partition) if dtype == "e4m3" else \
        P.pkv_paged_attention_decode(*short, partition_tokens=partition)
    heads = slice(0, None, 2) if kind == "lowest" else slice(None)
    assert bool((got[0, heads] == 0).all()) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("kind,dtype", [("infinite", "bf16"), ("infinite", "f16"), ("scale", "f16"), ("scale", "bf16")])
@pytest.mark.parametrize("stage_v", [False, True])
def test_prefill(kind, dtype, stage_v):
    bs, n, g = 16, 400, 4
    q1, kp, vp, table, scale, gone, _ = make(kind, dtype, g, n, bs, range(200))
    rows = torch.stack([q1[0]] * n)
    got = P.pkv_paged_attention_prefill(rows.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                        torch.tensor([n], dtype=torch.int32).cuda(),
                                        torch.tensor([0, n], dtype=torch.int32).cuda(), n, scale, stage_v=stage_v)
    for i in (0, 1, 127, 128, 199, 200, 201, 255, 256, 330, 399):
        close(got[i], attend(q1, kp, vp, table, scale, gone, range(i + 1)), dtype)
