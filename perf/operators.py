"""Cases of the operators around a paged decode step with rotary positions and
block-sparse attention, their plain forms and their exact values.

    rope     rotary positions applied to heads, or their transpose (the gradient)
    append   q rotated, K rotated on its way into the paged pool, V beside it
    bounds   per-channel minimum and maximum of the keys of each touched block
    select   the blocks of each (sequence, KV head) with the highest score bound
    sparse   decode attention over the selected blocks

``run`` computes a case in elementary torch operations, or with ``own`` set by
the library's entry points.  ``prepare`` makes what a serving loop holds
before the call; ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _rope(name, n, heads, d, rot, interleaved, transpose, dtype, far):
    return {"name": name, "op": "rope", "n": n, "heads": heads, "d": d, "rot": rot, "interleaved": interleaved,
            "transpose": transpose, "dtype": dtype, "far": far}


def _append(name, n, hq, hkv, d, bs, rot, interleaved, src, pool, fused, pad, far, scaled):
    return {"name": name, "op": "append", "n": n, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "rot": rot,
            "interleaved": interleaved, "src": src, "pool": pool, "fused": fused, "pad": pad, "far": far,
            "scaled": scaled}


def _bounds(name, b, lo, hi, new, hkv, d, bs, pool):
    return {"name": name, "op": "bounds", "b": b, "lo": lo, "hi": hi, "new": new, "hkv": hkv, "d": d, "bs": bs,
            "pool": pool}


def _select(name, b, lo, hi, k, first, last, hq, hkv, d, bs, pool):
    return {"name": name, "op": "select", "b": b, "lo": lo, "hi": hi, "k": k, "first": first, "last": last,
            "hq": hq, "hkv": hkv, "d": d, "bs": bs, "pool": pool}


def _sparse(name, b, lo, hi, k, hq, hkv, d, bs, pool):
    return {"name": name, "op": "sparse", "b": b, "lo": lo, "hi": hi, "k": k, "hq": hq, "hkv": hkv, "d": d,
            "bs": bs, "pool": pool}


def listed():
    return [
        # the query heads of one decode step of 64 sequences (32 heads of 128): launch latency
        _rope("rope decode q", 64, 32, 128, 128, False, False, "bf16", 4096),
        # the gradient of a prefill's query rotation, half of each head rotated in neighbouring pairs
        _rope("rope prefill gradient", 8192, 32, 128, 64, True, True, "f16", 131072),
        # one decode step of the Llama-3-8B-shaped layer (32 / 8 heads): one token per sequence
        _append("append decode", 64, 32, 8, 128, 16, 128, False, "bf16", "bf16", False, 0, 4096, "none"),
        # 16 prompt chunks of 512 tokens out of a fused projection, positions scaled for a long context
        _append("append prompt chunks", 8192, 32, 8, 128, 16, 128, False, "bf16", "bf16", True, 0, 131072, "blend"),
        # an odd number of tokens with padding rows into an 8-bit cache, three quarters of each head rotated
        _append("append e4m3 odd", 2051, 32, 8, 128, 16, 96, False, "f16", "e4m3", True, 37, 32768, "linear"),
        # upkeep of the block bounds after a decode step's append: the last block of each sequence
        _bounds("bounds decode", 64, 512, 4096, 1, 8, 128, 16, "bf16"),
        # upkeep after 16 prompts of up to 4096 tokens were written (every block)
        _bounds("bounds prompts", 16, 2049, 4095, 4096, 8, 128, 32, "f16"),
        # a few chats of some thousand tokens: launch latency and the selection itself
        _select("select few", 4, 4001, 8191, 64, 1, 4, 32, 8, 128, 16, "bf16"),
        # a batch of long contexts: the reading of the bounds
        _select("select batch", 64, 8193, 32767, 128, 1, 4, 32, 8, 128, 16, "bf16"),
        # two documents of up to 128K tokens in an 8-bit cache, 8 query heads per KV head
        _select("select documents", 2, 65537, 131071, 256, 1, 8, 64, 8, 128, 16, "e4m3"),
        # the batch's attention over 64 blocks (1024 tokens) of each context
        _sparse("sparse batch", 64, 4097, 16383, 64, 32, 8, 128, 16, "bf16"),
        # the two documents' attention over 256 blocks (4096 tokens)
        _sparse("sparse documents", 2, 65537, 131071, 256, 64, 8, 128, 16, "e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    return {k: v for k, v in _drawn(rng).items() if k != "name"}


def _drawn(rng):
    op = rng.choice(["rope", "append", "bounds", "select", "sparse"])
    d = rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 32])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        dtype = rng.choice(["f32", "bf16", "f16"])
        rot = rng.choice([d, d, d // 2, d // 4, d - 4, 20])
        heads = rng.randint(1, 40)
        n = min(_log(rng, 1, 8192), 8192 * 32 * 128 // (heads * d))
        return _rope("", n // 2 + 1 if dtype == "f32" else n, heads, d, rot, rng.random() < 0.5, rng.random() < 0.3,
                     dtype, _log(rng, 256, 1 << 20))
    pool = rng.choice(["f32", "bf16", "bf16", "f16", "e4m3"])
    if op == "append":
        src = pool if pool != "e4m3" else rng.choice(["f32", "bf16", "f16"])
        n = _log(rng, 1, 4096)
        return _append("", n, hkv * rng.choice([1, 2, 4]), hkv, d, bs, rng.choice([d, d, d // 2, d - 4, 20]),
                       rng.random() < 0.4, src, pool, rng.random() < 0.5, rng.randint(0, n // 8),
                       _log(rng, 256, 1 << 20), rng.choice(["none", "linear", "blend"]))
    d = 128 if pool == "e4m3" else d
    g = rng.choice([1, 2, 4, 8]) if pool != "f32" else rng.choice([1, 2, 4])
    b = _log(rng, 1, 48)
    cap = 64 * 16384 // b  # tokens of the longest sequence: a batch no larger than the listed ones
    if op == "bounds":
        hi = _log(rng, 1, min(cap // 32, 4096))
        new = rng.choice([1, 1, _log(rng, 1, hi), hi])
        return _bounds("", b, rng.randint(0, hi), hi, new, hkv, d, bs, pool)
    hi = _log(rng, 1, min(cap // (4 if pool == "f32" else 2), 131072, 8192 * bs))
    k = _log(rng, 8, 256)
    if op == "select":
        hi = max(hi, 3 * k * bs)  # something to choose from
    lo = rng.randint(0, hi)
    if op == "select":
        return _select("", b, lo, hi, k, rng.randint(0, 2), rng.randint(0, 5), hkv * g, hkv, d, bs, pool)
    return _sparse("", b, lo, hi, min(k, (896 if pool == "f32" else 1792) // bs), hkv * g, hkv, d, bs, pool)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _lens(c):
    """Lengths spread evenly from lo to hi."""
    b = c["b"]
    return [c["hi"] if b == 1 else c["lo"] + (c["hi"] - c["lo"]) * i // (b - 1) for i in range(b)]


def _blocks(c, lens=None):
    return [-(-n // c["bs"]) for n in (lens or _lens(c))]


def _normal(shape, dtype, g):
    kind = torch.float32 if dtype == "e4m3" else DTYPES[dtype]
    return torch.randn(shape, generator=g, device="cuda", dtype=kind).to(DTYPES[dtype])


def _frequencies(rot, scaled):
    """inv_freq in float64 and the attention factor."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if scaled == "linear":
        return f / 8, 1.0
    if scaled == "blend":  # long wavelengths slowed down by 16, short ones kept, a ramp between
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * keep + f / 16 * (1 - keep), 0.1 * math.log(16.0) + 1
    return f, 1.0


def _batch(c, rng, g):
    """Shuffled lengths and block tables of a scattered pool."""
    lens = _lens(c)
    rng.shuffle(lens)
    need = _blocks(c, lens)
    width, total = max(1, max(need)), max(1, sum(need))
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    fill = torch.tensor(need, device="cuda")
    j = torch.arange(width, device="cuda")
    used = j[None, :] < fill[:, None]
    first = torch.cumsum(fill, 0) - fill
    at = (first[:, None] + j[None, :]).clamp(max=total - 1)
    tables = torch.where(used, order[at], torch.full_like(order[at], -1)).contiguous()
    return lens, need, total, tables, torch.tensor(lens, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "op": c["op"]}
    if c["op"] in ("rope", "append"):
        inv, factor = _frequencies(c["rot"], c.get("scaled", "none"))
        s["inv_freq"], s["factor"] = inv.cuda(), factor
        s["positions"] = torch.randint(0, c["far"], (c["n"],), generator=g, device="cuda", dtype=torch.int32)
    if c["op"] == "rope":
        s["x"] = _normal((c["n"], c["heads"], c["d"]), c["dtype"], g)
        return s
    if c["op"] == "append":
        n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
        if c["fused"]:  # views of one projection's output
            x = _normal((n, hq + 2 * hkv, d), c["src"], g)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        else:
            s["q"] = _normal((n, hq, d), c["src"], g)
            s["k"], s["v"] = _normal((n, hkv, d), c["src"], g), _normal((n, hkv, d), c["src"], g)
        nb = -(-(n + n // 4 + 1) // c["bs"]) + 1  # the last block stays free
        slots = torch.randperm((nb - 1) * c["bs"], generator=g, device="cuda")[:n].to(torch.int32)
        if c["pad"]:
            slots[torch.randperm(n, generator=g, device="cuda")[:c["pad"]]] = -1
        s["slots"] = slots
        shape = (nb, hkv, c["bs"], d)
        s["k_pool"], s["v_pool"] = _normal(shape, c["pool"], g), _normal(shape, c["pool"], g)
        return s
    lens, need, total, s["tables"], s["lens"] = _batch(c, rng, g)
    hkv, d, bs = c["hkv"], c["d"], c["bs"]
    io = "f16" if c["pool"] == "e4m3" else c["pool"]
    if c["op"] == "bounds":
        s["k_pool"] = _normal((total, hkv, bs, d), c["pool"], g)
        s["bounds"] = torch.zeros((total, hkv, 2, d), device="cuda").to(DTYPES[c["pool"]])
        s["new"] = torch.tensor([min(n, c["new"]) for n in lens], dtype=torch.int32, device="cuda")
        return s
    s["q"] = _normal((c["b"], c["hq"], d), io, g)
    if c["op"] == "select":
        bounds = torch.empty((total, hkv, 2, d), device="cuda", dtype=DTYPES[c["pool"]])
        kind = "f32" if c["pool"] == "f32" else "f16" if c["pool"] == "e4m3" else c["pool"]
        step = max(1, (1 << 27) // (hkv * bs * d))
        for a in range(0, total, step):  # bounds of blocks of normal keys around a mean of their own
            n = min(step, total - a)
            keys = _normal((n, hkv, bs, d), kind, g) + _normal((n, hkv, 1, d), kind, g) / 2
            bounds[a:a + n, :, 0], bounds[a:a + n, :, 1] = keys.amin(2).to(bounds.dtype), keys.amax(2).to(bounds.dtype)
        s["bounds"] = bounds
        return s
    pools = []
    for _ in range(2):
        if c["pool"] == "e4m3":
            p = torch.empty((total, hkv, bs, d), device="cuda", dtype=DTYPES["e4m3"])
            step = max(1, (1 << 27) // (hkv * bs * d))
            for a in range(0, total, step):
                p[a:a + step] = _normal((min(step, total - a), hkv, bs, d), "f16", g).to(p.dtype)
        else:
            p = _normal((total, hkv, bs, d), c["pool"], g)
        pools.append(p)
    s["k_pool"], s["v_pool"] = pools
    # an ascending random choice of each context's blocks, the first and the last among them
    width = max(1, max(need))
    r = torch.rand((c["b"], hkv, width), generator=g, device="cuda")
    fill = torch.tensor(need, device="cuda")[:, None, None]
    j = torch.arange(width, device="cuda")
    r = torch.where((j == 0) | (j == fill - 1), r + 2, r)
    r = torch.where(j < fill, r, torch.full_like(r, -1))
    k = min(c["k"], width)
    value, at = torch.topk(r, k, dim=-1)
    at = torch.where(value >= 0, at, torch.full_like(at, 1 << 30)).sort(-1).values
    sel = torch.full((c["b"], hkv, c["k"]), -1, dtype=torch.int32, device="cuda")
    sel[..., :k] = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32)
    s["selected"] = sel
    s["scale"] = d ** -0.5
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _rotate(x, positions, inv_freq, factor, interleaved, transpose=False):
    """x [n, heads, d] in float32 with its first 2 * len(inv_freq) channels rotated."""
    ang = positions.double()[:, None] * inv_freq[None, :]
    cos, sin = (ang.cos() * factor).float()[:, None, :], (ang.sin() * factor).float()[:, None, :]
    if transpose:
        sin = -sin
    rot = 2 * inv_freq.numel()
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _narrow(x, dtype):
    """float32 values rounded to dtype; e4m3 saturates."""
    if dtype == torch.float8_e4m3fn:
        x = x.clamp(-448, 448)
    return x.to(dtype)


def _plain_rope(s):
    c = s["case"]
    y = _rotate(s["x"], s["positions"], s["inv_freq"], s["factor"], c["interleaved"], c["transpose"])
    return y.to(s["x"].dtype)


def _plain_append(s):
    c = s["case"]
    pool = DTYPES[c["pool"]]
    q = _rotate(s["q"], s["positions"], s["inv_freq"], s["factor"], c["interleaved"])
    k = _narrow(_rotate(s["k"], s["positions"], s["inv_freq"], s["factor"], c["interleaved"]), pool)
    v = _narrow(s["v"].float(), pool)
    kp, vp = s["k_pool"], s["v_pool"]
    skip = (s["slots"] < 0)
    spare = torch.full_like(s["slots"], kp.shape[0] * c["bs"] - 1)  # a free slot, which keeps its value
    slot = torch.where(skip, spare, s["slots"]).long()
    blk, off = slot // c["bs"], slot % c["bs"]
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[kp.element_size()]
    for p, rows in ((kp, k), (vp, v)):
        p, rows = p.view(raw), rows.view(raw)
        p[blk, :, off] = torch.where(skip[:, None, None], p[blk, :, off], rows)
    return {"q": q.to(torch.float16 if c["pool"] == "e4m3" else pool), "k_pool": kp, "v_pool": vp}


def _plain_bounds(s):
    c = s["case"]
    bs, lens, new = c["bs"], s["lens"].long(), s["new"].long()
    window = (c["new"] + bs - 2) // bs + 1
    j = torch.div(lens - new, bs, rounding_mode="floor")[:, None] + torch.arange(window, device="cuda")
    touched = (j * bs < lens[:, None]) & (new > 0)[:, None]
    phys = s["tables"].long().gather(1, j.clamp(0, s["tables"].shape[1] - 1))
    phys = torch.where(touched, phys, torch.zeros_like(phys))
    keys = s["k_pool"][phys].float()  # [b, window, hkv, bs, d]
    row = j[..., None] * bs + torch.arange(bs, device="cuda")
    live = (row < lens[:, None, None])[:, :, None, :, None]
    lo = keys.masked_fill(~live, math.inf).amin(3)
    hi = keys.masked_fill(~live, -math.inf).amax(3)
    both = torch.stack([lo, hi], 3).to(s["bounds"].dtype)
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[both.element_size()]
    whole = s["bounds"].view(raw)
    whole = torch.cat([whole, whole[:1]])
    whole[torch.where(touched, phys, torch.full_like(phys, whole.shape[0] - 1))] = both.view(raw)
    return whole[:-1].view(s["bounds"].dtype)


def _plain_select(s):
    c = s["case"]
    hkv, d, k = c["hkv"], c["d"], c["k"]
    fill = torch.div(s["lens"].long() + c["bs"] - 1, c["bs"], rounding_mode="floor")
    b = s["bounds"][s["tables"].long().clamp(min=0)].double()  # [b, width, hkv, 2, d]
    q = s["q"].double().view(c["b"], hkv, -1, d).transpose(2, 3)
    lo, hi = b[..., 0, :].transpose(1, 2), b[..., 1, :].transpose(1, 2)
    score = (lo @ q.clamp(max=0) + hi @ q.clamp(min=0)).amax(-1)  # [b, hkv, width]
    j = torch.arange(score.shape[-1], device="cuda")
    fill = fill[:, None, None]
    score = torch.where((j < c["first"]) | (j >= fill - c["last"]), torch.full_like(score, math.inf), score)
    score = torch.where(j < fill, score, torch.full_like(score, -math.inf))
    at = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    at = torch.where(at < fill, at, torch.full_like(at, 1 << 30)).sort(-1).values
    sel = torch.full((c["b"], hkv, k), -1, dtype=torch.int32, device="cuda")
    sel[..., :at.shape[-1]] = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32)
    return sel


def _gathered(s, dtype):
    """K, V [b, hkv, k * bs, d] of the selected blocks and which of their rows hold tokens."""
    c = s["case"]
    sel = s["selected"].long()
    have = sel >= 0
    phys = s["tables"].long()[:, None, :].expand(-1, c["hkv"], -1).gather(2, sel.clamp(min=0)).clamp(min=0)
    head = torch.arange(c["hkv"], device="cuda")[None, :, None].expand_as(phys)
    token = sel[..., None] * c["bs"] + torch.arange(c["bs"], device="cuda")
    live = (have[..., None] & (token < s["lens"].long()[:, None, None, None])).flatten(2)
    k = s["k_pool"][phys, head].to(dtype).flatten(2, 3)
    v = s["v_pool"][phys, head].to(dtype).flatten(2, 3).masked_fill(~live[..., None], 0)
    return k, v, live


def _plain_sparse(s):
    c = s["case"]
    k, v, live = _gathered(s, torch.float32)
    q = s["q"].float().view(c["b"], c["hkv"], -1, c["d"])
    score = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~live[:, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(live[:, :, None, :], (score - top).exp(), torch.zeros_like(score))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.view(c["b"], c["hq"], c["d"])


def _own(s):
    import paged_kv_cache_406_b200 as P

    c, op = s["case"], s["op"]
    if op == "rope":
        return P.pkv_rope(s["x"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], factor=s["factor"],
                          transpose=c["transpose"])
    if op == "append":
        how = {"interleaved": c["interleaved"], "factor": s["factor"]}
        args = (s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_pool"], s["v_pool"])
        q = P.pkv_rope_append_fp8(*args, 1.0, 1.0, **how) if c["pool"] == "e4m3" else P.pkv_rope_append(*args, **how)
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "bounds":
        return P.pkv_block_bounds(s["k_pool"], s["tables"], s["lens"], s["bounds"], new_tokens=s["new"],
                                  max_new_tokens=c["new"])
    if op == "select":
        return P.pkv_block_select(s["q"], s["bounds"], s["tables"], s["lens"], c["k"], c["bs"], n_first=c["first"],
                                  n_last=c["last"])
    args = (s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["selected"], s["scale"])
    if c["pool"] == "e4m3":
        return P.pkv_paged_attention_decode_sparse_fp8(*args, 1.0, 1.0)
    return P.pkv_paged_attention_decode_sparse(*args)


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "bounds": _plain_bounds, "select": _plain_select,
            "sparse": _plain_sparse}[state["op"]](state)


# ----------------------------------------------------------------------------
# what one pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    d = c["d"]
    if c["op"] == "rope":
        x = c["n"] * c["heads"] * d
        return {"bytes": 2 * x * BYTES[c["dtype"]] + 4 * c["n"] + 4 * c["rot"],
                "flops": 3 * c["n"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        qo = 2 if c["pool"] == "e4m3" else BYTES[c["pool"]]
        live = c["n"] - c["pad"]
        b = c["n"] * c["hq"] * d * (BYTES[c["src"]] + qo)
        b += live * 2 * c["hkv"] * d * (BYTES[c["src"]] + BYTES[c["pool"]])
        return {"bytes": b + 8 * c["n"] + 4 * c["rot"], "flops": 3 * c["rot"] * (c["n"] * c["hq"] + live * c["hkv"])}
    lens, need = _lens(c), _blocks(c)
    es = BYTES[c["pool"]]
    if c["op"] == "bounds":
        rows = blocks = 0
        for n in lens:
            new = min(n, c["new"])
            if new:
                a = (n - new) // c["bs"]
                blocks += -(-n // c["bs"]) - a
                rows += n - a * c["bs"]
        return {"bytes": (rows + 2 * blocks) * c["hkv"] * d * es + 4 * blocks + 8 * c["b"],
                "flops": 2 * rows * c["hkv"] * d}
    io = 2 if c["pool"] == "e4m3" else es
    if c["op"] == "select":
        b = sum(need) * (c["hkv"] * 2 * d * es + 4) + c["b"] * (c["hq"] * d * io + 4 + 4 * c["hkv"] * c["k"])
        return {"bytes": b, "flops": 2 * d * c["hq"] * sum(need)}
    rows = chosen = 0
    for n, m in zip(lens, need):
        k = min(c["k"], m)
        chosen += k
        rows += max(0, k * c["bs"] - (m * c["bs"] - n))  # the last block, perhaps not full, is among them
    b = rows * c["hkv"] * 2 * d * es + chosen * (4 + 4 * c["hkv"]) + c["b"] * c["hq"] * d * (io + 4)
    return {"bytes": b, "flops": 4 * rows * c["hq"] * d}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _turned(x, positions, inv_freq, factor, interleaved, transpose=False):
    """Rotation as a product of complex numbers."""
    rot = 2 * inv_freq.numel()
    ang = torch.outer(positions.double(), inv_freq) * (-1 if transpose else 1)
    turn = torch.polar(torch.full_like(ang, factor), ang)[:, None, :]
    head = x[..., :rot].double()
    pairs = head.unflatten(-1, (rot // 2, 2)) if interleaved else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:].double()], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return _turned(s["x"], s["positions"], s["inv_freq"], s["factor"], c["interleaved"], c["transpose"])
    if c["op"] == "append":
        how = (s["positions"], s["inv_freq"], s["factor"], c["interleaved"])
        live = (s["slots"] >= 0).nonzero().flatten()
        at = s["slots"][live].long()
        got = {"q": _turned(s["q"], *how)}
        for name, rows in (("k_pool", _turned(s["k"], *how)), ("v_pool", s["v"].double())):
            pool = s[name].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])  # a row for each slot
            pool[at] = rows[live]
            got[name] = pool.view(-1, c["bs"], c["hkv"], c["d"]).transpose(1, 2).contiguous()
        return got
    if c["op"] == "bounds":
        got = s["bounds"].double()
        lens, new, tables = s["lens"].tolist(), s["new"].tolist(), s["tables"].tolist()
        ids, fills = [], []
        for n, m, t in zip(lens, new, tables):
            for j in range((n - m) // c["bs"], -(-n // c["bs"])) if m else ():
                ids.append(t[j])
                fills.append(min(c["bs"], n - j * c["bs"]))
        for f in sorted(set(fills)):
            i = torch.tensor([x for x, y in zip(ids, fills) if y == f], device="cuda")
            keys = s["k_pool"][i][:, :, :f].double()
            got[i] = torch.stack([keys.min(2).values, keys.max(2).values], 2)
        return got
    if c["op"] == "select":
        return None
    out = torch.zeros((c["b"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    g = c["hq"] // c["hkv"]
    lens, sel = s["lens"].tolist(), s["selected"].cpu()
    for i, n in enumerate(lens):
        for h in range(c["hkv"]):
            js = sel[i, h][sel[i, h] >= 0].long().cuda()
            if not js.numel() or not n:
                continue
            phys = s["tables"][i].long()[js]
            rows = (js[:, None] * c["bs"] + torch.arange(c["bs"], device="cuda")).flatten() < n
            k = s["k_pool"][phys, h].double().flatten(0, 1)[rows]
            v = s["v_pool"][phys, h].double().flatten(0, 1)[rows]
            w = torch.softmax(s["q"][i, h * g:(h + 1) * g].double() @ k.T * s["scale"], -1)
            out[i, h * g:(h + 1) * g] = w @ v
    return out
