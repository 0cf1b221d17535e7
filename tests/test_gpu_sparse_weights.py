"""What the weights of block-sparse decode keep when they enter P.V: weights far
below the largest one, weights with low bits, values at the ends of their type.

Scores here lie in two channels (q is 0 elsewhere, scale 1) and are exact in 32
bits.  A weight is then 2^(x - m) with x = score times log2(e) in 32 bits: x, m
and their difference are each rounded by at most 2^-24 max|x|, and ex2 and the
factor that joins partial sums by 2^-22 each, so a weight is off by at most
    W = 3 ln2 2^-24 max|x| + 2 x 2^-22
of itself; the normalised one by twice that, and by the roundings of the sums.
Tensor cores align the 16 products and the sum of a step to the largest of them
and drop bits below 2^-23 of it: at most 17 x 2^-23 of a chunk's sum of |w v|.
Running sums and joins round by 2^-24 a chunk, for some chunks and 16 joins.
"""
import math

import numpy as np
import pytest
import torch

from helpers import DT

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402

TYPES = {**DT, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def case(scores, values, dtype, bs, g=1, d=128, base=None):
    """One sequence, one KV head: token t scores scores[t] + 8 base[t] for every head."""
    n = len(scores)
    nblk = -(-n // bs)
    k, v = torch.zeros(nblk * bs, d), torch.zeros(nblk * bs, d)
    k[:n, 5], v[:n] = torch.as_tensor(scores, dtype=torch.float32), values.float()
    if base is not None:
        k[:n, 77] = base
    order = torch.from_numpy(np.random.default_rng(n).permutation(nblk + 1)[:nblk])
    pools = []
    for x in (k, v):
        p = torch.zeros(nblk + 1, 1, bs, d).to(TYPES[dtype])
        raw = torch.uint8 if dtype == "e4m3" else p.dtype
        p.view(raw)[order] = x.view(nblk, 1, bs, d).to(p.dtype).view(raw)
        pools.append(p)
    q = torch.zeros(1, g, d, dtype=torch.float16 if dtype == "e4m3" else DT[dtype])
    q[..., 5], q[..., 77] = 1, 8
    return q, *pools, order.to(torch.int32)[None], torch.tensor([n], dtype=torch.int32)


def run(c, dtype):
    q, kp, vp, t, n = (x.cuda() for x in c)
    bs, nblk = kp.shape[2], t.shape[1]
    sel = torch.arange(nblk, dtype=torch.int32, device="cuda").view(1, 1, nblk)
    if dtype == "e4m3":
        return P.pkv_paged_attention_decode_sparse_fp8(q, kp, vp, t, n, sel, 1.0, 1.0, 1.0).cpu().double()[0]
    return P.pkv_paged_attention_decode_sparse(q, kp, vp, t, n, sel, 1.0).cpu().double()[0]


def weights(c):
    """64-bit softmax weights of the tokens, their values, and max |x|."""
    _, kp, vp, t, n = c
    n, bs = int(n), kp.shape[2]
    tok = torch.arange(n)
    k, v = (p.float()[t[0].long()[tok // bs], 0, tok % bs].double() for p in (kp, vp))
    s = k[:, 5] + 8 * k[:, 77]
    return torch.softmax(s, 0), v, float(s.abs().max()) * math.log2(math.e)


def bound(x_max, n):
    w = 3 * math.log(2) * 2.0 ** -24 * x_max + 2 * 2.0 ** -22
    return 2 * w + 17 * 2.0 ** -23 + (n / 16 + 16) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3", "f32"])
@pytest.mark.parametrize("gap", [10, 13, 16, 18, 20])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_weights_far_below_a_sink(dtype, gap, bs):
    """One token takes all but e^-gap of the weight and its value is 0: the
    output is made of the small weights alone and keeps its relative precision.
    (In the sink's own chunk a weight may be off by 2^-40 of the sink's, 2^-11
    of itself at a gap of 20: 15 tokens of 719 or more, 1e-5 of the output.)"""
    g = torch.Generator().manual_seed(gap)
    n = 90 * bs - 1
    scores = (torch.randint(-8, 9, (n,), generator=g) / 8).tolist()  # exact in every type
    at = n // 3
    values = torch.randn(n, 128, generator=g)
    values[at] = 0
    scores[at] = gap
    c = case(scores, values, dtype, bs, g=4 if dtype == "f32" else 8)
    w, v, x_max = weights(c)
    got = run(c, dtype)
    tol = (bound(x_max, n) + 15 / n * 2.0 ** -40 * math.exp(gap + 2)) * (w @ v.abs())
    err = (got - w @ v).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3", "f32"])
def test_low_bits_of_weights(dtype):
    """Values of 1: the output is the sum of the weights as they enter P.V over
    their 32-bit sum: 1 up to the roundings of two sums of 16.  One weight is 1
    and the others at least 1/4, so what tensor cores drop is at most 17 x 2^-23
    of 1 in a sum of 4.75 or more, below 2^-21; the 32-bit sum and the joins add
    12 roundings.  Weights that kept 16 bits only would show up to 2^-17."""
    worst = 0.0
    for i in range(64):  # 15 weights of 2^-x around one of 1: every pattern of low bits
        low = -float(torch.tensor((i + 1) / 50).to(TYPES[dtype]).float())
        got = run(case([0.0] + [low] * 15, torch.ones(16, 128), dtype, 16), dtype)
        worst = max(worst, float((got - 1).abs().max()))
    assert worst <= 2.0 ** -21 + 12 * 2.0 ** -24, worst


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3", "f32"])
@pytest.mark.parametrize("bs", [8, 32])
def test_scores_of_thousands(dtype, bs):
    """Scores around 2048 and -2048: the former share all the weight."""
    g = torch.Generator().manual_seed(1)
    n = 20 * bs - 3
    scores = (torch.randint(-8, 9, (n,), generator=g) / 8).tolist()
    values = torch.randn(n, 128, generator=g)
    base = torch.where(torch.rand(n, generator=g) < 0.5, 256.0, -256.0)
    c = case(scores, values, dtype, bs, g=2, base=base)
    w, v, x_max = weights(c)
    err = (run(c, dtype) - w @ v).abs()
    assert bool((err <= bound(x_max, n) * (w @ v.abs())).all()), float(err.max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
def test_largest_values(dtype):
    """A value row of the type's largest numbers, and columns of nothing else:
    the output is finite and as precise as elsewhere.  bf16 values reach the
    end of 32 bits' range themselves: up to 256 tokens of equal weight fit."""
    g = torch.Generator().manual_seed(2)
    top = torch.finfo(TYPES[dtype]).max
    n = 150
    values = torch.randn(n, 128, generator=g)
    values[70] = top
    values[:, 3], values[:, 4] = top, -top
    for scores in (torch.zeros(n), torch.arange(n) % 16 / 4, torch.arange(n).clamp(max=8)):
        c = case(scores.tolist(), values, dtype, 16, g=4)
        w, v, x_max = weights(c)
        got = run(c, dtype)
        assert bool(torch.isfinite(got).all())
        err = (got - w @ v).abs()
        assert bool((err <= bound(x_max, n) * (w @ v.abs())).all()), float((err / (w @ v.abs())).max())
