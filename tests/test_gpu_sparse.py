"""GPU parity of block bounds, block selection and block-sparse decode against
plain implementations in 64 bits.

Bounds and selections are exact (a bound is one of the keys; the ranking is
that of 64-bit sums), so they are compared for equality.  Attention: the
weights enter P.V within 2^-16 of their value, and a score of head_dim 128 of
N(0, 1) inputs is off by at most 128 x 2^-24 x sum |q k| / sqrt(128), about
1e-4 in the exponent, so an output differs from the 64-bit one by less than
(2 x 1e-4 + 2^-16) max |v| < 2e-3 (fp32 pools: 32-bit products throughout,
1e-5), the bounds of helpers.TOL.
"""
import math

import numpy as np
import pytest
import torch

from helpers import DT, TOL, Case

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def batch(lens, bs, seed, guard=2):
    """Tables of a scattered pool; returns (tables [B, maxb], blocks in the pool)."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + guard
    order = rng.permutation(nb)
    tables = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    return tables, nb


def keys(shape, dtype, seed):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32))
    return x.to(torch.float8_e4m3fn) if dtype == "e4m3" else x.to(DT[dtype])


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

def bounds_by_hand(pool, tables, lens, new, out, bs):
    out, p = out.clone(), pool.double()
    touched = set()
    for b, (n, m) in enumerate(zip(lens, new)):
        for j in range((n - m) // bs, -(-n // bs)) if m else ():
            rows = p[tables[b, j], :, :min(bs, n - j * bs)]
            out[tables[b, j], :, 0] = rows.amin(1).to(out.dtype) if out.dtype != torch.float8_e4m3fn else \
                rows.amin(1).float().to(out.dtype)
            out[tables[b, j], :, 1] = rows.amax(1).to(out.dtype) if out.dtype != torch.float8_e4m3fn else \
                rows.amax(1).float().to(out.dtype)
            touched.add(int(tables[b, j]))
    return out, touched


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128), ("f16", 64), ("f16", 128),
                                     ("e4m3", 128)])
@pytest.mark.parametrize("bs,hkv", [(8, 1), (16, 8), (32, 3)])
def test_bounds(dtype, d, bs, hkv):
    lens = [0, 1, 2, bs - 1, bs, bs + 1, 3 * bs, 100, 5 * bs + 7]
    tables, nb = batch(lens, bs, bs + hkv)
    pool = keys((nb, hkv, bs, d), dtype, d + bs)
    for b, n in enumerate(lens):  # rows behind the last token hold NaN
        if n % bs:
            pool.view(torch.uint8 if dtype == "e4m3" else pool.dtype)[tables[b, n // bs], :, n % bs:] = \
                0x7F if dtype == "e4m3" else math.nan
    start = keys((nb, hkv, 2, d), dtype, 1)
    dev = [torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")]
    for new in (None, [min(n, 1) for n in lens], lens, [min(n, bs) for n in lens], [n // 2 for n in lens]):
        got = start.cuda()
        t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        P.pkv_block_bounds(pool.cuda(), *dev, got, new_tokens=t, max_new_tokens=1 if new is None else max(max(new), 1))
        want, _ = bounds_by_hand(pool, tables, lens, [min(n, 1) for n in lens] if new is None else new, start, bs)
        assert torch.equal(got.cpu().float(), want.float())


def test_bounds_of_nan_and_infinite_keys():
    lens, bs = [20], 16
    tables, nb = batch(lens, bs, 0)
    for dtype in ("f32", "bf16", "f16"):
        pool = keys((nb, 1, bs, 64), dtype, 3)
        pool[tables[0, 0], 0, 5, 7] = math.nan
        pool[tables[0, 0], 0, 9, 8] = -math.inf
        pool[tables[0, 1], 0, 0, 9] = math.inf
        got = torch.zeros(nb, 1, 2, 64, dtype=DT[dtype], device="cuda")
        P.pkv_block_bounds(pool.cuda(), torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           got, torch.tensor([20], dtype=torch.int32).cuda(), 20)
        a, b = got[tables[0, 0], 0].cpu(), got[tables[0, 1], 0].cpu()
        assert torch.isnan(a[:, 7]).all() and not torch.isnan(a[:, :7]).any()
        assert a[0, 8] == -math.inf and b[1, 9] == math.inf


def test_bounds_refuses_bad_rows_on_the_device():
    lens, bs = [20, 33], 16
    tables, nb = batch(lens, bs, 0)
    pool, start = keys((nb, 2, bs, 64), "bf16", 3).cuda(), keys((nb, 2, 2, 64), "bf16", 4).cuda()
    t = torch.from_numpy(tables).cuda()

    def call(lens, new, tab=t, mx=64):
        got = start.clone()
        P.pkv_block_bounds(pool, tab, torch.tensor(lens, dtype=torch.int32).cuda(), got,
                           torch.tensor(new, dtype=torch.int32).cuda(), mx)
        return got, P.pkv_device_status(clear=True)

    want = call([20, 0], [20, 0])[0]
    for lens2, new in (([20, 33], [20, 34]), ([20, 33], [20, -1]), ([20, 49], [20, 1]), ([20, -1], [20, 0])):
        got, status = call(lens2, new)
        assert status == -1 and torch.equal(bits(got), bits(want))
    got, status = call([20, 33], [4, 33], mx=4)  # more new tokens than announced
    assert status == -1
    bad = t.clone()
    bad[1, 2] = nb
    got, status = call([20, 33], [20, 1], bad)
    assert status == -8 and torch.equal(bits(got), bits(want))


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def select_by_hand(q, bounds, tables, lens, k, bs, first, last):
    B, hq, d = q.shape
    hkv = bounds.shape[1]
    q = q.double().view(B, hkv, hq // hkv, d).numpy()
    bounds = bounds.double().numpy()
    out = np.full((B, hkv, k), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        nblk = -(-int(n) // bs)
        if nblk <= k:
            out[b, :, :nblk] = np.arange(nblk)
            continue
        for g in range(hkv):
            lo, hi = bounds[tables[b, :nblk], g, 0], bounds[tables[b, :nblk], g, 1]
            with np.errstate(invalid="ignore"):
                s = (np.minimum(q[b, g], 0)[:, None] * lo + np.maximum(q[b, g], 0)[:, None] * hi).sum(-1)
            s = s.max(0)  # NaN of any head stays
            j = np.arange(nblk)
            forced = (j < first) | (j >= nblk - last)
            rank = np.where(np.isnan(s), np.inf, s)
            # forced first, then NaN, then the score; equal ones by index
            order = sorted(range(nblk), key=lambda i: (not forced[i], not np.isnan(s[i]), -rank[i], i))
            out[b, g] = np.sort(np.array(order[:k]))
    return out


def check_select(q, bounds, tables, lens, k, bs, first, last):
    want = select_by_hand(q, bounds, tables, lens, k, bs, first, last)
    got = P.pkv_block_select(q.cuda(), bounds.cuda(), torch.from_numpy(tables).cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), k, bs, first, last).cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def bounds_of(nb, hkv, d, dtype, seed, rows=8):
    x = keys((nb, hkv, rows, d), "f16" if dtype == "e4m3" else dtype, seed).float()
    both = torch.stack([x.amin(2), x.amax(2)], 2)
    return both.to(torch.float8_e4m3fn) if dtype == "e4m3" else both.to(DT[dtype])


@pytest.mark.parametrize("dtype,d,g", [("f32", 64, 1), ("f32", 128, 4), ("f32", 128, 8), ("bf16", 64, 8),
                                       ("bf16", 128, 4), ("bf16", 128, 1), ("f16", 128, 2), ("f16", 64, 4),
                                       ("e4m3", 128, 1), ("e4m3", 128, 4), ("e4m3", 128, 8)])
@pytest.mark.parametrize("bs", [8, 32])
def test_select(dtype, d, g, bs):
    hkv, k = 2, 12
    lens = [0, 1, bs, k * bs - 1, k * bs, k * bs + 1, 13 * bs, 40 * bs + 3, 300 * bs, 517 * bs - 2]
    tables, nb = batch(lens, bs, d + g)
    bounds = bounds_of(nb, hkv, d, dtype, g)
    q = keys((len(lens), g * hkv, d), "f16" if dtype == "e4m3" else dtype, 5)
    for first, last in ((1, 2), (0, 0), (0, 12), (5, 7)):
        check_select(q, bounds, tables, lens, k, bs, first, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["zero q", "equal", "few values", "outlier"])
def test_select_ties(dtype, kind):
    """Ties far beyond what shared memory ranks (512): the lower index wins."""
    bs, hkv, g, d, k = 16, 2, 4, 128, 70
    lens = [3000 * bs - 5, 700 * bs, 100 * bs]
    tables, nb = batch(lens, bs, 1)
    rng = np.random.default_rng(3)
    io = torch.float16 if dtype == "e4m3" else DT[dtype]
    pt = torch.float8_e4m3fn if dtype == "e4m3" else DT[dtype]
    q = torch.from_numpy(rng.integers(-2, 3, (3, g * hkv, d)).astype(np.float32))
    x = torch.from_numpy(rng.integers(-3, 4, (nb, hkv, 2, d)).astype(np.float32))
    bounds = torch.stack([x.amin(2), x.amax(2)], 2)
    if kind == "zero q":
        q.zero_()
    elif kind == "equal":
        bounds[:] = bounds[:1]
    elif kind == "outlier":  # one block far above the rest, which are equal
        bounds[:] = bounds[:1]
        bounds[tables[0, 1500]] *= 64
        bounds[tables[1, 3]] *= 64
    check_select(q.to(io), bounds.to(pt), tables, lens, k, bs, 1, 2)


def test_select_close_scores():
    """Scores that differ by less than 32 bits resolve: the 64-bit order."""
    bs, d, k = 8, 64, 16
    lens = [900 * bs]
    tables, nb = batch(lens, bs, 2)
    bounds = torch.zeros(nb, 1, 2, d)
    rng = np.random.default_rng(0)
    tiny = torch.from_numpy(rng.permutation(nb).astype(np.float32)) * 2.0 ** -30
    bounds[:, 0, :, 0] = 1000.0
    bounds[:, 0, :, 1] = tiny[:, None]
    check_select(torch.ones(1, 1, d), bounds, tables, lens, k, bs, 0, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_select_with_nan_and_infinities(dtype):
    bs, hkv, g, d, k = 16, 1, 2, 64, 20
    lens = [600 * bs, 64 * bs]
    tables, nb = batch(lens, bs, 4)
    bounds = bounds_of(nb, hkv, d, dtype, 6)
    q = keys((2, g, d), dtype, 7)
    bounds[tables[0, 17], 0, :, 3] = math.nan
    bounds[tables[0, 400], 0, 1, 5] = math.inf
    bounds[tables[0, 401], 0, 0, 5] = -math.inf
    bounds[tables[1, 30], 0, 0, 0] = -math.inf
    check_select(q, bounds, tables, lens, k, bs, 1, 1)
    q[1, 0, 2] = math.inf  # a whole row of infinities and NaN
    check_select(q, bounds, tables, lens, k, bs, 1, 1)
    q[1] = math.nan
    check_select(q, bounds, tables, lens, k, bs, 1, 1)


def test_select_tiny_values():
    """Products below 32 bits' range: ranked in 64."""
    bs, d, k = 16, 64, 10
    lens = [200 * bs]
    tables, nb = batch(lens, bs, 5)
    for dtype, f in (("f32", 1e-30), ("bf16", 1e-30), ("bf16", 1e-20)):
        bounds = bounds_of(nb, 1, d, dtype, 8) * f
        check_select(keys((1, 1, d), dtype, 9) * f, bounds, tables, lens, k, bs, 1, 1)


def test_select_large_values():
    """Products beyond 32 bits: every candidate is ranked in 64."""
    bs, d, k = 16, 64, 10
    lens = [200 * bs]
    tables, nb = batch(lens, bs, 5)
    bounds = bounds_of(nb, 1, d, "f32", 8) * 1e30
    check_select(keys((1, 1, d), "f32", 9) * 1e20, bounds, tables, lens, k, bs, 1, 1)


def test_select_long_context():
    bs, d, k = 8, 64, 256
    lens = [140000 * bs - 3, 5]  # a bitmap of more than 16 KB
    tables, nb = batch(lens, bs, 6)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(nb, 1, 2, d, generator=g, device="cuda")
    bounds = torch.stack([x.amin(2), x.amax(2)], 2).to(torch.bfloat16)
    q = torch.randn(2, 2, d, generator=g, device="cuda").to(torch.bfloat16)
    t = torch.from_numpy(tables).cuda()
    got = P.pkv_block_select(q, bounds, t, torch.tensor(lens, dtype=torch.int32).cuda(), k, bs, 1, 2)[0, 0]
    b = bounds[t[0].long(), 0].double()
    s = (b[:, 0] @ q[0].double().clamp(max=0).T + b[:, 1] @ q[0].double().clamp(min=0).T).amax(1)
    s[:1] = math.inf
    s[-2:] = math.inf
    want = s.sort(dim=0, descending=True, stable=True).indices[:k].sort().values
    assert torch.equal(got.long(), want)


def test_select_bad_lengths_and_blocks():
    bs, k = 16, 4
    lens = [20 * bs, 10 * bs]
    tables, nb = batch(lens, bs, 7)
    bounds, q = bounds_of(nb, 1, 64, "bf16", 1).cuda(), keys((2, 2, 64), "bf16", 2).cuda()
    t = torch.from_numpy(tables).cuda()
    ok = P.pkv_block_select(q, bounds, t, torch.tensor(lens, dtype=torch.int32).cuda(), k, bs)
    for n in (-1, 20 * bs + 1):
        got = P.pkv_block_select(q, bounds, t, torch.tensor([lens[0], n], dtype=torch.int32).cuda(), k, bs)
        assert P.pkv_device_status(clear=True) == -1
        assert torch.equal(got[0], ok[0]) and bool((got[1] == -1).all())
    t[1, 5] = nb + 9
    P.pkv_block_select(q, bounds, t, torch.tensor(lens, dtype=torch.int32).cuda(), k, bs)
    assert P.pkv_device_status(clear=True) == -8


# ---------------------------------------------------------------------------
# attention over the selection
# ---------------------------------------------------------------------------

def attend_by_hand(q, k_pool, v_pool, tables, lens, selected, scale):
    B, hq, d = q.shape
    hkv, bs = k_pool.shape[1], k_pool.shape[2]
    g = hq // hkv
    q, k_pool, v_pool = q.double(), k_pool.double(), v_pool.double()
    out = torch.zeros(B, hq, d, dtype=torch.float64)
    for b in range(B):
        for h in range(hkv):
            rows = [(tables[b, j], r) for j in selected[b, h] if j >= 0 for r in range(bs) if j * bs + r < lens[b]]
            if not rows:
                continue
            blk, r = (torch.tensor([int(x[i]) for x in rows]) for i in (0, 1))
            w = torch.softmax(q[b, h * g:(h + 1) * g] @ k_pool[blk, h, r].T * scale, -1)
            out[b, h * g:(h + 1) * g] = w @ v_pool[blk, h, r]
    return out


def choose(lens, bs, hkv, k, seed):
    """Ascending random selections of 0 .. k blocks; some hold the last block, some do not."""
    rng = np.random.default_rng(seed)
    out = np.full((len(lens), hkv, k), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        nblk = -(-int(n) // bs)
        for h in range(hkv):
            m = int(rng.integers(0, min(k, nblk) + 1)) if h else min(k, nblk)
            out[b, h, :m] = np.sort(rng.permutation(nblk)[:m])
    return out


def spoil(pool, tables, lens, bs):
    """NaN behind every sequence's last token."""
    raw = pool.view(torch.uint8) if pool.element_size() == 1 else pool
    for b, n in enumerate(lens):
        if n % bs:
            raw[tables[b, n // bs], :, n % bs:] = 0x7F if pool.element_size() == 1 else math.nan


@pytest.mark.parametrize("dtype,d,g", [("f32", 64, 1), ("f32", 128, 4), ("bf16", 128, 1), ("bf16", 128, 4),
                                       ("bf16", 64, 8), ("f16", 128, 8), ("f16", 64, 2), ("e4m3", 128, 1),
                                       ("e4m3", 128, 2), ("e4m3", 128, 4), ("e4m3", 128, 8)])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("k", [1, 5, 40])
def test_sparse_decode(dtype, d, g, bs, k):
    hkv = 3
    lens = [0, 1, bs - 1, bs, 2 * bs + 1, 7 * bs + 3, 50 * bs - 1, 33 * bs]
    tables, nb = batch(lens, bs, d + g + k)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1), keys((nb, hkv, bs, d), dtype, 2)
    spoil(kp, tables, lens, bs)
    spoil(vp, tables, lens, bs)
    q = keys((len(lens), g * hkv, d), "f16" if dtype == "e4m3" else dtype, 3)
    sel = choose(lens, bs, hkv, k, k)
    args = (q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(tables).cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), torch.from_numpy(sel).cuda(), d ** -0.5)
    if dtype == "e4m3":
        got = P.pkv_paged_attention_decode_sparse_fp8(*args, 0.5, 0.25)
        want = attend_by_hand(q, kp.float(), vp.float(), tables, lens, sel, d ** -0.5 * 0.5) * 0.25
        tol = TOL["f16"]
    else:
        got = P.pkv_paged_attention_decode_sparse(*args)
        want = attend_by_hand(q, kp, vp, tables, lens, sel, d ** -0.5)
        tol = TOL[dtype]
    err = (got.cpu().double() - want).abs()
    assert bool(torch.isfinite(got).all()) and bool((err <= tol * want.abs().clamp(min=1)).all()), float(err.max())
    empty = torch.from_numpy((sel >= 0).sum(-1) == 0).repeat_interleave(g, 1)
    assert bool((got.cpu()[empty] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "f32"])
def test_long_lists(dtype):
    """More selected blocks than a CTA lists in shared memory (1024)."""
    bs, hkv, g, d, k = 8, 2, 4, 128, 1500
    lens = [1600 * bs - 3, 1025 * bs, 40]
    tables, nb = batch(lens, bs, 2)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1), keys((nb, hkv, bs, d), dtype, 2)
    q = keys((3, g * hkv, d), "f16" if dtype == "e4m3" else dtype, 3)
    sel = choose(lens, bs, hkv, k, 5)
    args = (q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(tables).cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), torch.from_numpy(sel).cuda(), d ** -0.5)
    got = P.pkv_paged_attention_decode_sparse_fp8(*args, 1.0, 1.0) if dtype == "e4m3" else \
        P.pkv_paged_attention_decode_sparse(*args)
    f = (lambda t: t.float()) if dtype == "e4m3" else (lambda t: t)
    want = attend_by_hand(q, f(kp), f(vp), tables, lens, sel, d ** -0.5)
    tol = TOL["f16" if dtype == "e4m3" else dtype]
    assert bool(((got.cpu().double() - want).abs() <= tol * want.abs().clamp(min=1)).all())


@pytest.mark.parametrize("dtype,g", [("bf16", 4), ("f16", 1), ("f32", 2)])
def test_every_block_selected_is_dense_decode(dtype, g):
    case = Case([700, 1, 0, 64, 333], 2 * g, 2, 128, 16, dtype, seed=3)
    d = case.device()
    nblk = [-(-int(n) // 16) for n in case.lens]
    sel = np.full((5, 2, 50), -1, dtype=np.int32)
    for b, n in enumerate(nblk):
        sel[b, :, :n] = np.arange(n)
    got = P.pkv_paged_attention_decode_sparse(d["q"], d["k_pool"], d["v_pool"], d["block_tables"], d["seq_lens"],
                                              torch.from_numpy(sel).cuda(), case.scale)
    want = torch.from_numpy(case.oracle())
    assert bool(((got.cpu().double() - want).abs() <= TOL[dtype] * want.abs().clamp(min=1)).all())


def test_large_scores_and_extreme_values():
    """Scores of some thousands, a value row of the type's largest numbers."""
    bs, d = 16, 128
    lens = [20 * bs]
    tables, nb = batch(lens, bs, 3)
    for dtype in ("bf16", "f16"):
        kp, vp = keys((nb, 1, bs, d), dtype, 1) * 30, keys((nb, 1, bs, d), dtype, 2)
        q = keys((1, 4, d), dtype, 3) * 30
        sel = np.arange(0, 20, 2, dtype=np.int32)[None, None]
        got = P.pkv_paged_attention_decode_sparse(q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(tables).cuda(),
                                                  torch.tensor(lens, dtype=torch.int32).cuda(),
                                                  torch.from_numpy(sel).cuda(), d ** -0.5)
        want = attend_by_hand(q, kp, vp, tables, lens, sel, d ** -0.5)
        # a score: 128 x 2^-24 x 900 x 128 x 0.64 / 11.3 = 0.05 in the exponent, on the weights of the few largest
        assert bool(torch.isfinite(got).all()) and float((got.cpu().double() - want).abs().max()) <= 2 * 0.05 * 5


def test_bad_selections_end_the_list_and_are_recorded():
    bs, d, hkv = 16, 64, 1
    lens = [10 * bs - 3]
    tables, nb = batch(lens, bs, 3)
    kp, vp = keys((nb, hkv, bs, d), "bf16", 1), keys((nb, hkv, bs, d), "bf16", 2)
    q = keys((1, 2, d), "bf16", 3)
    dev = (q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(tables).cuda(),
           torch.tensor(lens, dtype=torch.int32).cuda())

    def run(sel, t=None):
        a = dev if t is None else (*dev[:3], t, dev[4])
        out = P.pkv_paged_attention_decode_sparse(*a, torch.tensor([[sel]], dtype=torch.int32).cuda(), 0.125)
        return out, P.pkv_device_status(clear=True)

    good, status = run([2, 5, -1, -1])
    assert status == 0
    want = attend_by_hand(q, kp, vp, tables, lens, np.array([[[2, 5]]]), 0.125)
    assert float((good.cpu().double() - want).abs().max()) <= TOL["bf16"] * 4
    assert torch.equal(run([2, 5, -1, 7])[0], good)          # nothing behind the end is read
    for sel in ([2, 5, 5, 7], [2, 5, 4, 7], [2, 5, 10, -1], [2, 5, 1 << 30, -1]):
        got, status = run(sel)
        assert status == -1 and torch.equal(got, good), sel
    got, status = run([-5, 3, 4, 5])
    assert status == 0 and bool((got == 0).all())
    bad = torch.from_numpy(tables).cuda()
    bad[0, 5] = -7
    assert run([2, 5, -1, -1], bad)[1] == -8
    out = P.pkv_paged_attention_decode_sparse(*dev[:4], torch.tensor([10 * bs + 1], dtype=torch.int32).cuda(),
                                              torch.tensor([[[0, 1]]], dtype=torch.int32).cuda(), 0.125)
    assert P.pkv_device_status(clear=True) == -1 and bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_wait_that_runs_out(dtype):
    """A CTA whose first copies are left out: its waits give up, the call ends
    with a status, the other rows and the next call are right."""
    bs, hkv, d = 16, 4, 128
    lens = [40 * bs, 33 * bs]
    tables, nb = batch(lens, bs, 3)
    kp, vp = keys((nb, hkv, bs, d), dtype, 1), keys((nb, hkv, bs, d), dtype, 2)
    q = keys((2, 2 * hkv, d), "f16" if dtype == "e4m3" else dtype, 3)
    sel = choose(lens, bs, hkv, 30, 1)
    args = (q.cuda(), kp.cuda(), vp.cuda(), torch.from_numpy(tables).cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda(), torch.from_numpy(sel).cuda(), d ** -0.5)
    call = (lambda: P.pkv_paged_attention_decode_sparse_fp8(*args, 1.0, 1.0)) if dtype == "e4m3" else \
        (lambda: P.pkv_paged_attention_decode_sparse(*args))
    want = call().clone()
    P.pkv_debug_stall_decode(0)
    try:
        got = call()
        assert P.pkv_device_status(clear=True) == -6
    finally:
        P.pkv_debug_stall_decode(-1)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, 2:], want[0, 2:])  # CTA 0 serves sequence 0, KV head 0
    assert torch.equal(call(), want)


def test_offsets_beyond_32_bits():
    """Blocks at the end of pools of more than 2^32 bytes (and bounds of more
    than 2^29 values), through every operator."""
    bs, hkv, g, d, nb, k = 16, 8, 2, 128, 280000, 6
    kp, vp = (torch.empty(nb, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bounds = torch.empty(nb, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
    assert kp.numel() > 1 << 32
    lens = [30 * bs - 5, 40]
    ids = torch.tensor(np.random.default_rng(1).permutation(200)[:33] + nb - 200)
    tables = torch.full((2, 30), -1, dtype=torch.int32)
    tables[0], tables[1, :3] = ids[:30], ids[30:]
    t, L = tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    n = sum(lens)
    x = keys((n, hkv * (g + 2), d), "bf16", 3).cuda()
    pos = torch.tensor([p for m in lens for p in range(m)], dtype=torch.int32)
    slot = torch.tensor([int(tables[b, p // bs]) * bs + p % bs for b, m in enumerate(lens) for p in range(m)])
    inv, _ = P.pkv_rope_frequencies(d)
    hq = g * hkv
    q = P.pkv_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos.cuda(), inv, slot.to(torch.int32).cuda(),
                          kp, vp)
    P.pkv_block_bounds(kp, t, L, bounds, L, max(lens))
    q = q[[lens[0] - 1, n - 1]].contiguous()
    sel = P.pkv_block_select(q, bounds, t, L, k, bs, 1, 1)
    out = P.pkv_paged_attention_decode_sparse(q, kp, vp, t, L, sel, d ** -0.5)
    # the same in a pool of 200 blocks
    small = [p[nb - 200:].contiguous() for p in (kp, vp)]
    st = torch.where(tables >= 0, tables - (nb - 200), tables)
    blank = torch.zeros(200, hkv, 2, d, dtype=torch.bfloat16)
    want_b, _ = bounds_by_hand(small[0].cpu(), st.numpy(), lens, lens, blank, bs)
    used = (ids - (nb - 200)).long()
    assert torch.equal(bounds[nb - 200:].cpu()[used].float(), want_b[used].float())
    want_s = select_by_hand(q.cpu(), want_b, st.numpy(), lens, k, bs, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want_s)
    ref = attend_by_hand(q.cpu(), small[0].cpu(), small[1].cpu(), st.numpy(), lens, want_s, d ** -0.5)
    assert bool(((out.cpu().double() - ref).abs() <= TOL["bf16"] * ref.abs().clamp(min=1)).all())
    rows = slot - (nb - 200) * bs
    assert torch.equal(small[1].transpose(1, 2).reshape(-1, hkv, d)[rows.cuda()].view(torch.int16),
                       x[:, hq + hkv:].contiguous().view(torch.int16))


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_steps_of_a_long_context(dtype):
    """Prompts written with rotation, bounds kept up, then decode steps that
    select and attend: each stage against its own definition on the state the
    stage before left on the device."""
    bs, hq, hkv, d, k = 16, 4, 2, 128, 6
    prompts, steps = [300, 17, 512], 5
    io = torch.float16 if dtype == "e4m3" else DT[dtype]
    cap = [n + steps for n in prompts]
    tables, nb = batch(cap, bs, 9)
    t = torch.from_numpy(tables).cuda()
    inv, factor = P.pkv_rope_frequencies(d, 10000.0, "yarn", 4.0, 256)
    pool = torch.zeros(nb, hkv, bs, d, device="cuda").to(torch.float8_e4m3fn if dtype == "e4m3" else io)
    kp, vp, bounds = pool, pool.clone(), torch.zeros(nb, hkv, 2, d, device="cuda").to(pool.dtype)
    g = torch.Generator(device="cuda").manual_seed(4)
    scales = (0.25, 0.5)

    def append(pos, seq):
        n = len(pos)
        x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").to(io)
        slots = torch.tensor([int(tables[s, p // bs]) * bs + p % bs for p, s in zip(pos, seq)], dtype=torch.int32)
        a = (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], torch.tensor(pos, dtype=torch.int32).cuda(), inv,
             slots.cuda(), kp, vp)
        return P.pkv_rope_append_fp8(*a, *scales, factor=factor) if dtype == "e4m3" else \
            P.pkv_rope_append(*a, factor=factor)

    append([p for n in prompts for p in range(n)], [s for s, n in enumerate(prompts) for _ in range(n)])
    new = torch.tensor(prompts, dtype=torch.int32).cuda()
    P.pkv_block_bounds(kp, t, new, bounds, new, max(prompts))
    for step in range(steps):
        lens = [n + step + 1 for n in prompts]
        q = append([n - 1 for n in lens], range(len(prompts)))
        L = torch.tensor(lens, dtype=torch.int32).cuda()
        P.pkv_block_bounds(kp, t, L, bounds)
        want, _ = bounds_by_hand(kp.cpu(), tables, lens, lens, torch.zeros_like(bounds).cpu(), bs)
        assert torch.equal(bounds.cpu().float(), want.float())
        sel = P.pkv_block_select(q, bounds, t, L, k, bs, 1, 2)
        by_hand = select_by_hand(q.cpu(), bounds.cpu().float(), tables, lens, k, bs, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), by_hand)
        if dtype == "e4m3":
            out = P.pkv_paged_attention_decode_sparse_fp8(q, kp, vp, t, L, sel, d ** -0.5, *scales)
            ref = attend_by_hand(q.cpu(), kp.cpu().float(), vp.cpu().float(), tables, lens, by_hand,
                                 d ** -0.5 * scales[0]) * scales[1]
        else:
            out = P.pkv_paged_attention_decode_sparse(q, kp, vp, t, L, sel, d ** -0.5)
            ref = attend_by_hand(q.cpu(), kp.cpu(), vp.cpu(), tables, lens, by_hand, d ** -0.5)
        tol = TOL["f16" if dtype == "e4m3" else dtype]
        assert bool(((out.cpu().double() - ref).abs() <= tol * ref.abs().clamp(min=1)).all())


def test_captured_steps_share_no_hidden_state():
    """Two captured graphs with workspaces of their own, replayed on two
    streams at once and in turns, give what single calls give."""
    bs, hkv, g, d, k = 16, 2, 4, 128, 24
    graphs, wants, outs = [], [], []
    sets = []
    for i in range(2):
        lens = [2000 + 700 * i, 900, 16 * 24]
        tables, nb = batch(lens, bs, i)
        kp, vp = (keys((nb, hkv, bs, d), "bf16", 10 * i + j).cuda() for j in (1, 2))
        bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
        q, t = keys((3, g * hkv, d), "bf16", i + 5).cuda(), torch.from_numpy(tables).cuda()
        L = torch.tensor(lens, dtype=torch.int32).cuda()
        sel = torch.empty(3, hkv, k, dtype=torch.int32, device="cuda")
        out = torch.empty(3, g * hkv, d, device="cuda")
        ws1 = torch.empty(P.pkv_select_workspace_size(3, hkv, t.shape[1]), dtype=torch.uint8, device="cuda")
        need = P.pkv_sparse_workspace_size(3, g * hkv, hkv, d, k, bs, torch.bfloat16)
        ws2 = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

        def step(kp=kp, vp=vp, bounds=bounds, q=q, t=t, L=L, sel=sel, out=out, ws1=ws1, ws2=ws2):
            P.pkv_block_bounds(kp, t, L, bounds, L, 4096)
            P.pkv_block_select(q, bounds, t, L, k, bs, selected=sel, workspace=ws1)
            P.pkv_paged_attention_decode_sparse(q, kp, vp, t, L, sel, d ** -0.5, out=out, workspace=ws2)

        sets.append((kp, vp, bounds, q, t, L, sel, ws1, ws2))
        step()
        wants.append(out.clone())
        outs.append(out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        graphs.append((graph, side))
        bounds.zero_()
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)
