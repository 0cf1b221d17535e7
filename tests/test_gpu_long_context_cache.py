"""PagedKVCache with a rotation and key bounds: prompts through write_chunk,
decode steps over every block and over selected ones, forks with
copy-on-write.  The expectation keeps every token's K and V, rotated in 64
bits and rounded as the pool rounds them, outside the cache.

Tolerance: a key rounded to the pool's type from a 32-bit value may differ from
the one rounded from 64 bits by one step (eps) where the two straddle a
rounding border, as q may; a score then moves by at most eps sum |q k| scale of
few channels, far below helpers.TOL for 16-bit pools; for fp32 pools rotations
are within 4e-7 of (|a| + |b|), so scores move by 1e-5 at most and outputs by
2e-5 max |v|: 1e-4.
"""
import numpy as np
import pytest
import torch

from helpers import DT

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402
from paged_kv_cache_406_b200.cache import PagedKVCache, Rope  # noqa: E402

HQ, HKV, D, BS = 8, 2, 128, 16
TOLS = {"bf16": 2e-2, "f16": 4e-3, "f32": 1e-4}


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def rotate(x, pos, rope):
    """64-bit rotation, half layout."""
    x, inv = x.double().cpu(), rope.inv_freq.cpu()
    ang = torch.as_tensor(pos, dtype=torch.float64)[:, None] * inv
    c, s = (ang.cos() * rope.factor)[:, None], (ang.sin() * rope.factor)[:, None]
    h = inv.numel()
    y = x.clone()
    y[..., :h], y[..., h:2 * h] = x[..., :h] * c - x[..., h:2 * h] * s, x[..., :h] * s + x[..., h:2 * h] * c
    return y


class Mirror:
    """Every sequence's K and V as the pool should hold them."""

    def __init__(self, dtype, rope):
        self.dtype, self.rope, self.k, self.v = DT[dtype], rope, {}, {}

    def put(self, seq, k, v):
        n = self.k[seq].shape[0] if seq in self.k else 0
        k = rotate(k, range(n, n + k.shape[0]), self.rope).to(self.dtype).double()
        v = v.cpu().double()
        self.k[seq] = torch.cat([self.k[seq], k]) if n else k
        self.v[seq] = torch.cat([self.v[seq], v]) if n else v

    def attend(self, seq, q, scale, blocks=None):
        k, v = self.k[seq], self.v[seq]
        q = rotate(q[None], [k.shape[0] - 1], self.rope).to(self.dtype).double()[0]
        out = torch.empty(HQ, D, dtype=torch.float64)
        for h in range(HKV):
            rows = torch.arange(k.shape[0])
            if blocks is not None:
                rows = rows[torch.isin(rows // BS, blocks[h])]
            w = torch.softmax(q[h * 4:h * 4 + 4] @ k[rows, h].T * scale, -1)
            out[h * 4:h * 4 + 4] = w @ v[rows, h]
        return out

    def select(self, seq, q, k_sel, first, last):
        k = self.k[seq]
        q = rotate(q[None], [k.shape[0] - 1], self.rope).to(self.dtype).double()[0]
        nblk = -(-k.shape[0] // BS)
        picked, margin = [], []
        for h in range(HKV):
            if nblk <= k_sel:
                picked.append(torch.arange(nblk))
                margin.append(float("inf"))
                continue
            lo = torch.stack([k[j * BS:(j + 1) * BS, h].amin(0) for j in range(nblk)])
            hi = torch.stack([k[j * BS:(j + 1) * BS, h].amax(0) for j in range(nblk)])
            g = q[h * 4:h * 4 + 4]
            s = (g.clamp(max=0) @ lo.T + g.clamp(min=0) @ hi.T).amax(0)
            s[:first] = s[nblk - last:] = float("inf")
            order = s.sort(descending=True, stable=True)
            picked.append(order.indices[:k_sel].sort().values)
            margin.append(float(order.values[k_sel - 1] - order.values[k_sel]))
        return picked, margin


@pytest.mark.parametrize("dtype,rot,scaling", [("bf16", 128, "plain"), ("f16", 64, "yarn"), ("f32", 128, "linear")])
def test_steps(dtype, rot, scaling):
    rope = Rope(*P.pkv_rope_frequencies(rot, 10000.0, scaling, 4.0 if scaling != "plain" else 1.0, 256))
    cache = PagedKVCache(160, HKV, D, BS, DT[dtype], 64, rope=rope, key_bounds=True,
                         free_order=np.random.default_rng(0).permutation(160).astype(np.int32))
    mirror = Mirror(dtype, rope)
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    scale, prompts = D ** -0.5, [400, 37, 1]
    for s, n in enumerate(prompts):
        cache.add(s, n)
    total = sum(prompts)
    q, k, v = rand(total, HQ, D), rand(total, HKV, D), rand(total, HKV, D)
    cache.write_chunk([0, 1, 2], prompts, q, k, v)
    at = 0
    for s, n in enumerate(prompts):
        mirror.put(s, k[at:at + n], v[at:at + n])
        at += n
    cache.fork(0, 3)
    mirror.k[3], mirror.v[3] = mirror.k[0], mirror.v[0]
    ids = [0, 1, 2, 3]
    sparse_checked = 0
    for step in range(20):  # 1 -> 21 tokens: block borders and copy-on-write on the way
        q, k, v = rand(4, HQ, D), rand(4, HKV, D), rand(4, HKV, D)
        few = 8 if step % 2 else None
        out = cache.decode_step(ids, q, k, v, scale, max_selected=few, n_first=1, n_last=2).cpu().double()
        for i, s in enumerate(ids):
            mirror.put(s, k[i:i + 1], v[i:i + 1])
            blocks = None
            if few:
                blocks, margin = mirror.select(s, q[i], few, 1, 2)
                if min(margin) < 0.05:  # a rounding of q or K may decide otherwise
                    continue
                sparse_checked += 1
            want = mirror.attend(s, q[i], scale, blocks)
            err = (out[i] - want).abs().max()
            assert float(err) <= TOLS[dtype] * max(1.0, float(want.abs().max())), (step, s, float(err))
    assert sparse_checked >= 20


def test_selecting_every_block_is_the_dense_step():
    rope = Rope(*P.pkv_rope_frequencies(128))
    caches = [PagedKVCache(64, HKV, D, BS, torch.bfloat16, 32, rope=rope, key_bounds=b) for b in (False, True)]
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(300, HQ, D), rand(300, HKV, D), rand(300, HKV, D)
    for c in caches:
        c.add(0, 300)
        c.write_chunk([0], [300], q, k, v)
    q, k, v = rand(1, HQ, D), rand(1, HKV, D), rand(1, HKV, D)
    dense = caches[0].decode_step([0], q, k, v, D ** -0.5).clone()
    sparse = caches[1].decode_step([0], q, k, v, D ** -0.5, max_selected=32)
    # two kernels' 32-bit sums of the same products; weights rounded to 2^-16 at worst
    assert float((dense - sparse).abs().max()) <= 1e-4
    assert torch.equal(caches[0].k_pool.view(torch.int16)[caches[0].alloc.block_tables([0], 32)[0][0, :18]],
                       caches[1].k_pool.view(torch.int16)[caches[1].alloc.block_tables([0], 32)[0][0, :18]])


def test_queries_over_a_cached_prompt():
    """A prompt found whole by prefix caching: its rows are in the pool, only
    the query is rotated, and the attention is the one behind the append."""
    rope = Rope(*P.pkv_rope_frequencies(128))
    cache = PagedKVCache(32, HKV, D, BS, torch.bfloat16, 16, rope=rope)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    tokens = np.arange(6 * BS) % 50
    assert cache.add_cached(0, tokens) == 0
    q = rand(6 * BS, HQ, D)
    turned, tables, lens, start = cache.write_chunk([0], [6 * BS], q, rand(6 * BS, HKV, D), rand(6 * BS, HKV, D))
    assert cache.add_cached(1, tokens) == 6 * BS
    last = torch.tensor([6 * BS - 1], dtype=torch.int32, device="cuda")
    again = cache.rotate(q[-1:], last)
    assert torch.equal(again, turned[-1:])
    t, n = cache.alloc.block_tables([1], 16)
    want = P.pkv_paged_attention_decode(turned[-1:].contiguous(), cache.k_pool, cache.v_pool, tables, lens, D ** -0.5)
    got = P.pkv_paged_attention_decode(again, cache.k_pool, cache.v_pool, torch.from_numpy(t).cuda(),
                                       torch.from_numpy(n).cuda(), D ** -0.5)
    assert torch.equal(got, want)
    back = cache.rotate(again.float(), last, undo=True)
    # one rounding to bf16 of each rotated channel, and 32-bit rotations
    size = q[-1:].float().abs()
    assert bool(((back - q[-1:].float()).abs() <= 2.0 ** -8 * 2 * (size + size.roll(D // 2, -1))).all())
    with pytest.raises(ValueError):
        PagedKVCache(4, HKV, D, BS, torch.bfloat16, 4).rotate(again, last)


def test_e4m3_cache_and_bounds_refreshed():
    cache = PagedKVCache(64, HKV, D, BS, torch.float8_e4m3fn, 32, k_scale=0.25, v_scale=0.25, key_bounds=True,
                         rope=Rope(*P.pkv_rope_frequencies(64), interleaved=True))
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cache.add(5, 200)
    q, tables, lens, start = cache.write_chunk([5], [200], rand(200, HQ, D), rand(200, HKV, D), rand(200, HKV, D))
    assert q.dtype == torch.float16 and start.tolist() == [0, 200] and lens.tolist() == [200]
    kept = cache.bounds.clone()
    cache.bounds.view(torch.uint8).zero_()
    cache.refresh_bounds([5])
    assert torch.equal(cache.bounds.view(torch.uint8), kept.view(torch.uint8))
    step = (rand(1, HQ, D), rand(1, HKV, D), rand(1, HKV, D))
    out = cache.decode_step([5], *step, D ** -0.5, max_selected=13).clone()  # every block of 201 tokens
    again = PagedKVCache(64, HKV, D, BS, torch.float8_e4m3fn, 32, k_scale=0.25, v_scale=0.25, k_pool=cache.k_pool,
                         v_pool=cache.v_pool)
    t, n = cache.alloc.block_tables([5], 32)
    at = torch.tensor([200], dtype=torch.int32, device="cuda")
    q = P.pkv_rope(step[0], at, cache.rope.inv_freq, interleaved=True)
    dense = P.pkv_paged_attention_decode_fp8(q.to(torch.float16), again.k_pool, again.v_pool,
                                             torch.from_numpy(t).cuda(), torch.from_numpy(n).cuda(), D ** -0.5, 0.25,
                                             0.25)
    # q rounded to bf16 first here: half a step 2^-9 of each channel moves a score by about 2^-9 and an output likewise
    assert float((out - dense).abs().max()) <= 0.05


def test_refusals():
    plain = PagedKVCache(8, HKV, D, BS, torch.bfloat16, 4)
    plain.add(0, 3)
    x = torch.zeros(1, HKV, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, HQ, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        plain.decode_step([0], q, x, x, 0.1, max_selected=2)
    assert plain.alloc.seq_len(0) == 3  # nothing reserved
    with pytest.raises(ValueError):
        plain.refresh_bounds([0])
    with pytest.raises(ValueError):
        plain.write_chunk([0], [4], q, x, x)
    with pytest.raises(ValueError):
        plain.write_chunk([0], [2], q, x, x)
    bounded = PagedKVCache(8, HKV, D, BS, torch.bfloat16, 4, key_bounds=True)
    bounded.add(0, 3)
    for kw in (dict(max_selected=0), dict(max_selected=2, n_first=2, n_last=1), dict(max_selected=4, n_first=-1)):
        with pytest.raises(ValueError):
            bounded.decode_step([0], q, x, x, 0.1, **kw)
    with pytest.raises(ValueError):
        PagedKVCache(8, HKV, D, BS, torch.bfloat16, 4, rope=Rope(torch.ones(4, device="cuda")))
    with pytest.raises(ValueError):
        PagedKVCache(8, HKV, D, BS, torch.bfloat16, 4, rope=Rope(*P.pkv_rope_frequencies(2 * D)))
    with pytest.raises(ValueError):
        bounded.decode_step_host(np.array([0]), q.cpu(), x.cpu(), x.cpu(), 0.1)
    assert bounded.alloc.seq_len(0) == 3
