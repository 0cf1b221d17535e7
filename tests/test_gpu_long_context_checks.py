"""Calls of the rotating and block-sparse entry points that are refused, and what
a refused call leaves behind: nothing."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402
from paged_kv_cache_406_b200.cache import PagedKVCache, Rope  # noqa: E402

HKV, D, BS = 2, 128, 16


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def step_inputs(dtype, n=2, hq=8):
    return tuple(torch.ones(n, h, D, dtype=dtype, device="cuda") for h in (hq, HKV, HKV))


BAD = {  # a change of (q, k, v, scale, keywords), and the error
    "3 heads a group": (lambda q, k, v: (q[:, :6].contiguous(), k, v), {}, P.PagedKVError),
    "16 heads a group": (lambda q, k, v: (torch.cat([q] * 4, 1), k, v), {}, P.PagedKVError),
    "7 query heads": (lambda q, k, v: (q[:, :7].contiguous(), k, v), {}, P.PagedKVError),
    "head_dim": (lambda q, k, v: (q[..., :64].contiguous(), k, v), {}, ValueError),
    "KV heads": (lambda q, k, v: (q, k[:, :1].contiguous(), v), {}, ValueError),
    "rows": (lambda q, k, v: (q[:1], k, v), {}, ValueError),
    "rows of v": (lambda q, k, v: (q, k, torch.cat([v, v])), {}, ValueError),
    "dims": (lambda q, k, v: (q, k[0], v), {}, ValueError),
    "type of q": (lambda q, k, v: (q.double(), k, v), {}, TypeError),
    "type of k": (lambda q, k, v: (q, k.double(), v), {}, TypeError),
    "types of k and v": (lambda q, k, v: (q, k, v.float() if v.dtype != torch.float32 else v.half()), {}, TypeError),
    "strided channels": (lambda q, k, v: (torch.cat([q, q], -1)[..., ::2], k, v), {}, ValueError),
    "misaligned": (lambda q, k, v: (torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape), k, v), {},
                   ValueError),
    "scale": (lambda q, k, v: (q, k, v), {"scale": math.nan}, ValueError),
    "out's shape": (lambda q, k, v: (q, k, v), {"out": (1, 8, D)}, ValueError),
    "out's type": (lambda q, k, v: (q, k, v), {"out": torch.float16}, ValueError),
    "out misaligned": (lambda q, k, v: (q, k, v), {"out": "odd"}, ValueError),
}


@pytest.mark.parametrize("what", list(BAD))
@pytest.mark.parametrize("pool,rope,bounds,max_selected", [
    (torch.bfloat16, True, True, 4), (torch.bfloat16, True, False, None), (torch.float16, False, True, 4),
    (torch.float16, False, True, None), (torch.float8_e4m3fn, True, True, 4), (torch.float8_e4m3fn, False, True, 4),
    (torch.float32, True, True, 4)])
def test_a_refused_step_reserves_and_writes_nothing(what, pool, rope, bounds, max_selected):
    change, kw, error = BAD[what]
    cache = PagedKVCache(12, HKV, D, BS, pool, 6, rope=Rope(*P.pkv_rope_frequencies(D)) if rope else None,
                         key_bounds=bounds)
    rows = torch.float16 if pool == torch.float8_e4m3fn else pool
    for p in (cache.k_pool, cache.v_pool):
        p.view(torch.uint8).fill_(9)
    cache.add(0, 5)
    cache.add(1, 16)  # the next token opens a block
    free = cache.stats()
    kw = dict(kw)
    if "out" in kw:
        kw["out"] = torch.empty(2 * 8 * D + 1, device="cuda")[1:].view(2, 8, D) if kw["out"] == "odd" else \
            torch.empty(kw["out"], device="cuda") if isinstance(kw["out"], tuple) else \
            torch.empty(2, 8, D, dtype=kw["out"], device="cuda")
    args = change(*step_inputs(rows))
    if pool == torch.float32 and what == "16 heads a group":
        args = (torch.cat(list(step_inputs(rows)[:1]) * 2, 1), *args[1:])  # fp32 pools: 8 are too many already
    scale = kw.pop("scale", 0.1)
    with pytest.raises(error):
        cache.decode_step([0, 1], *args, scale, max_selected=max_selected, **kw)
    assert cache.alloc.seq_len(0) == 5 and cache.alloc.seq_len(1) == 16 and cache.stats() == free
    for p in (cache.k_pool, cache.v_pool):
        assert bool((p.view(torch.uint8) == 9).all())
    good = cache.decode_step([0, 1], *step_inputs(rows), 0.1, max_selected=max_selected)
    assert good.shape == (2, 8, D) and cache.alloc.seq_len(1) == 17
    with pytest.raises(error):  # as well behind a step of the same sizes
        cache.decode_step([0, 1], *args, scale, max_selected=max_selected, **kw)
    assert cache.alloc.seq_len(0) == 6 and cache.alloc.seq_len(1) == 17


def test_a_step_from_views_of_one_projection():
    """Rotating caches take rows whose token stride is free, on the device or on
    the host; the checks refuse none of them."""
    caches = [PagedKVCache(12, HKV, D, BS, torch.bfloat16, 6, rope=Rope(*P.pkv_rope_frequencies(D)), key_bounds=True)
              for _ in range(3)]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 12, D, generator=g, device="cuda").to(torch.bfloat16)
    parts = (x[:, :8], x[:, 8:10], x[:, 10:])
    outs = []
    for c, rows in zip(caches, (parts, [t.contiguous() for t in parts], [t.cpu() for t in parts])):
        for p in (c.k_pool, c.v_pool):
            p.zero_()
        c.add(0, 5)
        c.add(1, 16)
        c.refresh_bounds([0, 1])
        outs.append(c.decode_step([0, 1], *rows, 0.1, max_selected=4).clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    mine = torch.empty(2, 8, D, device="cuda")
    for c in caches:  # the same step into a tensor of the caller's, behind one of the same sizes
        assert c.decode_step([0, 1], *parts, 0.1, max_selected=4, out=mine) is mine
        outs.append(mine.clone())
    assert torch.equal(outs[3], outs[4]) and torch.equal(outs[3], outs[5])
    one = caches[0].decode_step([1], x[1:, :8], x[1:, 8:10], x[1:, 10:], 0.1, max_selected=np.int64(4))
    assert one.shape == (1, 8, D)


def test_partition_sizes_and_rows_on_the_host():
    cache = PagedKVCache(12, HKV, D, BS, torch.bfloat16, 6, rope=Rope(*P.pkv_rope_frequencies(D)))
    cache.add(0, 5)
    q, k, v = step_inputs(torch.bfloat16, 1)
    for size in (-16, 8, 24):
        with pytest.raises(P.PagedKVError):
            cache.decode_step([0], q, k, v, 0.1, partition_tokens=size)
    assert cache.alloc.seq_len(0) == 5
    # host rows are copied first: an odd stride there is no stride on the device
    wide = torch.ones(2, 12 * D + 1, dtype=torch.bfloat16)[:, :-1].view(2, 12, D)
    cache.add(1, 5)
    out = cache.decode_step([0, 1], wide[:, :8], wide[:, 8:10], wide[:, 10:], 0.1)
    assert out.shape == (2, 8, D) and cache.alloc.seq_len(0) == 6


def test_no_tokens_of_any_stride():
    """A tensor without elements has no stride to refuse (torch gives some zeros)."""
    inv, _ = P.pkv_rope_frequencies(64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 1, 1, device="cuda")[:0].expand(0, 4, 64)
    assert x.stride() == (0, 0, 0) or x.stride(1) == 0
    assert P.pkv_rope(x, none, inv).shape == (0, 4, 64)
    pools = [torch.zeros(1, 4, 8, 64, device="cuda") for _ in range(2)]
    assert P.pkv_rope_append(x, x, x, none, inv, none, *pools).shape == (0, 4, 64)
