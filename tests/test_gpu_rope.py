"""GPU parity of the rotary operators against the formula in 64 bits.

Tolerances.  The reduced angle is rounded to 32 bits (at most 2^-25 of half a
turn: 2 pi 2^-26 = 9.4e-8 rad) and sincospif is within 2 units of 2^-24: sine
and cosine are within 2.2e-7, so y = x_a c - x_b s is within
(|x_a| + |x_b|) factor (2.2e-7 + 2 x 2^-24) < 4e-7 (|x_a| + |x_b|) factor
before its one rounding, which adds eps / 2 of |y| (f16 below 2^-14: 2^-25;
e4m3: 2^-4 of |y|, below 2^-6 half of 2^-9, in units of the scale).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import paged_kv_cache_406_b200 as P  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FAR = [0, 1, 2, 511, 4095, 131071, (1 << 20) + 1, -5, (1 << 31) - 1]


@pytest.fixture(autouse=True)
def _clean_status(native):
    P.pkv_device_status(clear=True)
    yield
    assert P.pkv_device_status(clear=True) == 0, "a kernel recorded a device error"


def formula(x, pos, inv, factor, interleaved, transpose=False):
    """(y, |x_a| + |x_b|) in 64 bits."""
    x, rot = x.double(), 2 * inv.numel()
    ang = pos.double()[:, None] * inv
    c, s = (factor * ang.cos())[:, None], (factor * ang.sin())[:, None] * (-1 if transpose else 1)
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    xa, xb = x[..., a], x[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    mag[..., a] = mag[..., b] = xa.abs() + xb.abs()
    return y, mag


def close(got, want, mag, factor, dtype):
    half = torch.finfo(dtype).eps / 2
    tol = 4e-7 * abs(factor) * mag
    tol = tol + half * (want.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)
    tol = torch.where(mag == 0, torch.zeros_like(tol), tol)  # channels that pass through are the same
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def inputs(n, heads, d, rot, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g).to(DT[dtype]).cuda()
    far = torch.tensor(FAR, dtype=torch.int64)
    pos = far[torch.randint(0, len(FAR), (n,), generator=g)] if n < len(FAR) else torch.cat(
        [far, torch.randint(0, 1 << 17, (n - len(FAR),), generator=g)])
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return x, pos.to(torch.int32).cuda(), inv.cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,d,rot", [
    (1, 1, 64, 64), (1, 32, 128, 128), (64, 32, 128, 128), (77, 5, 128, 64), (33, 3, 64, 20),   # halves of 10 channels
    (9, 7, 80, 80), (130, 1, 128, 2), (40, 2, 128, 126), (12, 2, 512, 512), (5, 3, 24, 24), (700, 1, 8, 4),
])
def test_rope(dtype, interleaved, n, heads, d, rot):
    x, pos, inv = inputs(n, heads, d, rot, dtype, n + d)
    for transpose, factor in ((False, 1.0), (True, 1.25)):
        got = P.pkv_rope(x, pos, inv, interleaved=interleaved, factor=factor, transpose=transpose)
        assert got.dtype == x.dtype and got.shape == x.shape
        close(got, *formula(x, pos, inv, factor, interleaved, transpose), factor, x.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_in_place_and_strided(dtype):
    x, pos, inv = inputs(50, 12, 64, 48, dtype)
    want = P.pkv_rope(x, pos, inv)
    view = x[:, 3:9]  # heads 3 .. 8 of a wider projection
    out = torch.full_like(x, 7.0)
    P.pkv_rope(view, pos, inv, out=out[:, 1:7])
    assert torch.equal(out[:, 1:7], want[:, 3:9])
    assert bool((out[:, :1] == 7).all()) and bool((out[:, 7:] == 7).all())
    y = x.clone()
    assert P.pkv_rope(y[:, 3:9], pos, inv, out=y[:, 3:9]).data_ptr() == y[:, 3:9].data_ptr()
    assert torch.equal(y[:, 3:9], want[:, 3:9]) and torch.equal(y[:, :3], x[:, :3]) and torch.equal(y[:, 9:], x[:, 9:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_transpose_is_the_gradient(interleaved):
    """Against autograd of the formula in 64 bits, and against differences:
    y is linear in x, so (y(x + u) - y(x - u)) / 2 = y(u) up to rounding."""
    x, pos, inv = inputs(20, 3, 64, 44, "f32", 4)
    dy, _, _ = inputs(20, 3, 64, 44, "f32", 5)
    leaf = x.double().requires_grad_()
    ang = pos.double()[:, None] * inv
    c, s = ang.cos()[:, None] * 1.5, ang.sin()[:, None] * 1.5
    a, b = (slice(0, 44, 2), slice(1, 44, 2)) if interleaved else (slice(0, 22), slice(22, 44))
    parts = leaf[..., a] * c - leaf[..., b] * s, leaf[..., a] * s + leaf[..., b] * c
    loss = (parts[0] * dy[..., a].double()).sum() + (parts[1] * dy[..., b].double()).sum() + \
        (leaf[..., 44:] * dy[..., 44:].double()).sum()
    loss.backward()
    dx = P.pkv_rope(dy, pos, inv, interleaved=interleaved, factor=1.5, transpose=True)
    _, mag = formula(dy, pos, inv, 1.5, interleaved, True)
    close(dx, leaf.grad, mag, 1.5, torch.float32)

    u, _, _ = inputs(20, 3, 64, 44, "f32", 6)
    up = P.pkv_rope(x + u, pos, inv, interleaved=interleaved, factor=1.5).double()
    down = P.pkv_rope(x - u, pos, inv, interleaved=interleaved, factor=1.5).double()
    diff = ((up - down) / 2 * dy.double()).sum()
    # x + u and x - u are rounded (2^-24 of each), each y is within 4e-7 * 1.5 (|x_a| + |x_b|) and 2^-24
    size = (x.abs() + u.abs()).double()
    pair = size.clone()
    pair[..., a] = pair[..., b] = size[..., a] + size[..., b]
    tol = ((4e-7 + 4 * 2.0 ** -24) * 1.5 * pair * dy.abs().double()).sum()
    assert abs(float(diff - (dx.double() * u.double()).sum())) <= float(2 * tol)


def test_undoing_a_rotation():
    x, pos, inv = inputs(30, 4, 128, 128, "f32", 9)
    back = P.pkv_rope(P.pkv_rope(x, pos, inv), pos, inv, transpose=True)
    _, mag = formula(x, pos, inv, 1.0, False)
    assert bool(((back - x).double().abs() <= 4 * 4e-7 * mag).all())


def slots_for(n, nb, bs, pad, seed):
    rng = np.random.default_rng(seed)
    s = rng.permutation(nb * bs)[:n].astype(np.int32)
    s[rng.permutation(n)[:pad]] = -1
    return torch.from_numpy(s)


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


@pytest.mark.parametrize("dtype,d,bs,hq,hkv,rot,interleaved,n,pad,fused", [
    ("bf16", 128, 16, 32, 8, 128, False, 64, 0, False),
    ("bf16", 128, 16, 32, 8, 128, False, 301, 9, True),
    ("f16", 128, 32, 8, 8, 64, True, 1, 0, False),
    ("f16", 64, 8, 14, 2, 62, False, 45, 45, True),       # every row a padding row
    ("f32", 64, 8, 3, 3, 20, False, 19, 3, True),
    ("f32", 128, 16, 4, 1, 128, True, 33, 0, False),
    ("bf16", 64, 32, 0, 4, 64, False, 21, 2, False),      # keys and values only
])
def test_rope_append(dtype, d, bs, hq, hkv, rot, interleaved, n, pad, fused):
    x, pos, inv = inputs(n, hq + 2 * hkv, d, rot, dtype, n)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-n // bs) + 3
    slots = slots_for(n, nb, bs, pad, n)
    kp = torch.randn(nb, hkv, bs, d).to(DT[dtype]).cuda()
    vp = torch.randn(nb, hkv, bs, d).to(DT[dtype]).cuda()
    k0, v0 = kp.clone(), vp.clone()
    got = P.pkv_rope_append(q, k, v, pos, inv, slots.cuda(), kp, vp, interleaved=interleaved, factor=1.1)
    close(got, *formula(q, pos, inv, 1.1, interleaved), 1.1, x.dtype)
    wk, mag = formula(k, pos, inv, 1.1, interleaved)
    rows = lambda p: p.transpose(1, 2).reshape(nb * bs, hkv, d)  # noqa: E731
    live = (slots >= 0).nonzero().flatten().cuda()
    at = slots.cuda().long()[live]
    close(rows(kp)[at], wk[live], mag[live], 1.1, x.dtype)
    assert torch.equal(bits(rows(vp)[at]), bits(v[live].contiguous()))
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(bits(rows(kp)[rest]), bits(rows(k0)[rest]))
    assert torch.equal(bits(rows(vp)[rest]), bits(rows(v0)[rest]))


@pytest.mark.parametrize("src,d,bs,rot,interleaved,n,pad", [
    ("f16", 128, 16, 128, False, 64, 0), ("bf16", 128, 8, 96, True, 77, 5), ("f32", 128, 32, 128, False, 5, 0),
    ("f16", 64, 16, 44, False, 31, 1), ("f32", 64, 8, 20, True, 18, 0),
])
def test_rope_append_fp8(src, d, bs, rot, interleaved, n, pad):
    hq, hkv, ks, vs = 8, 4, 1 / 32, 1 / 16
    x, pos, inv = inputs(n, hq + 2 * hkv, d, rot, src, n)
    x[:, -1] *= 40  # beyond 448 / 16: saturates
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    nb = -(-n // bs) + 2
    slots = slots_for(n, nb, bs, pad, n + 1)
    kp = torch.randint(0, 120, (nb, hkv, bs, d), dtype=torch.uint8).cuda()
    vp = torch.randint(0, 120, (nb, hkv, bs, d), dtype=torch.uint8).cuda()
    k0, v0 = kp.clone(), vp.clone()
    got = P.pkv_rope_append_fp8(q, k, v, pos, inv, slots.cuda(), kp, vp, ks, vs, interleaved=interleaved)
    assert got.dtype == torch.float16
    wq, mag = formula(q, pos, inv, 1.0, interleaved)
    tol = 4e-7 * mag + 2.0 ** -11 * (wq.abs() + 4e-7 * mag) + 2.0 ** -25
    assert bool(((got.double() - wq).abs() <= tol).all())
    wk, mag = formula(k, pos, inv, 1.0, interleaved)
    rows = lambda p: p.transpose(1, 2).reshape(nb * bs, hkv, d)  # noqa: E731
    live = (slots >= 0).nonzero().flatten().cuda()
    at = slots.cuda().long()[live]
    for pool, want, m, s in ((kp, wk, mag, ks), (vp, v.double(), torch.zeros_like(mag), vs)):
        code = rows(pool)[at].view(torch.float8_e4m3fn).double()
        want, m = (want / s)[live].clamp(-448, 448), m[live] / s
        tol = 4e-7 * m + 2.0 ** -4 * (want.abs() + 4e-7 * m) + 2.0 ** -10
        assert bool(((code - want).abs() <= tol).all())
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(rows(kp)[rest], rows(k0)[rest]) and torch.equal(rows(vp)[rest], rows(v0)[rest])


def test_values_are_the_unrotated_append_s(native):
    """V codes and the channels beyond rot_dim of K equal pkv_kv_append_fp8's."""
    n, hkv, d, bs = 24, 4, 128, 16
    x, pos, inv = inputs(n, 3 * hkv, d, 64, "bf16", 3)
    q, k, v = (x[:, i * hkv:(i + 1) * hkv].contiguous() for i in range(3))
    slots = slots_for(n, 4, bs, 0, 1).cuda()
    pools = [torch.zeros(4, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(4)]
    P.pkv_rope_append_fp8(q, k, v, pos, inv, slots, pools[0], pools[1], 0.25, 0.5)
    P.pkv_kv_append_fp8(k, v, slots, pools[2], pools[3], 0.25, 0.5)
    assert torch.equal(pools[1], pools[3]) and torch.equal(pools[0][..., 64:], pools[2][..., 64:])


def test_slot_outside_the_pool_is_recorded():
    x, pos, inv = inputs(3, 3, 64, 64, "bf16")
    pools = [torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([5, 16, 3], dtype=torch.int32, device="cuda")  # 16: one past the last
    P.pkv_rope_append(x[:, :1], x[:, 1:2], x[:, 2:], pos, inv, slots, *pools)
    assert P.pkv_device_status(clear=True) == -8
    assert torch.equal(pools[1][0, 0, 5], x[0, 2]) and torch.equal(pools[1][0, 0, 3], x[2, 2])
    assert int((pools[1].abs().sum(-1) > 0).sum()) == 2


def test_refusals_of_the_binding():
    x, pos, inv = inputs(4, 6, 64, 64, "bf16")
    with pytest.raises(ValueError):
        P.pkv_rope(x.transpose(1, 2), pos, inv)           # channels not packed
    with pytest.raises(ValueError):
        P.pkv_rope(x, pos[:3], inv)
    with pytest.raises(TypeError):
        P.pkv_rope(x, pos.long(), inv)
    with pytest.raises(TypeError):
        P.pkv_rope(x, pos, inv.float())
    with pytest.raises(TypeError):
        P.pkv_rope(x.to(torch.float64), pos, inv)
    with pytest.raises(ValueError):
        P.pkv_rope(x, pos.cpu(), inv)
    kp = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        P.pkv_rope(x, pos, inv, out=x[:2])
    with pytest.raises(TypeError):
        P.pkv_rope_append(x[:, :2], x[:, 2:4], x[:, 4:], pos, inv, s, kp.half(), kp.half())
    q = x[:, :2].contiguous()
    with pytest.raises(ValueError):                       # q_out must not be q
        P.pkv_rope_append(q, x[:, 2:4], x[:, 4:], pos, inv, s, kp, kp.clone(), q_out=q)
    with pytest.raises(TypeError):
        P.pkv_rope_append_fp8(q, x[:, 2:4], x[:, 4:], pos, inv, s, kp, kp.clone(), 1.0, 1.0)


def test_capture_replay_and_another_stream():
    x, pos, inv = inputs(40, 8, 128, 128, "bf16", 2)
    kp, vp = (torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = slots_for(40, 8, 16, 0, 2).cuda()
    q_out = torch.empty(40, 4, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: P.pkv_rope_append(x[:, :4], x[:, 4:6], x[:, 6:], pos, inv, slots, kp, vp, q_out=q_out)  # noqa: E731
    want = call().clone()
    wk = kp.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    q_out.zero_()
    kp.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, want) and torch.equal(kp, wk)
    x.mul_(-1)  # new contents of the captured buffers
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, -want) and torch.equal(kp, -wk)


def test_one_token_of_a_strided_tensor():
    """A single token's stride may be anything, an odd one among them."""
    base, pos, inv = inputs(1, 12, 64, 64, "bf16", 3)
    odd = torch.empty(1 * 777 + 12 * 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 12, 64), (777, 64, 1))
    odd.copy_(base)
    assert torch.equal(P.pkv_rope(odd, pos, inv), P.pkv_rope(base, pos, inv))
    pools = [torch.zeros(1, 3, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    slot = torch.tensor([4], dtype=torch.int32, device="cuda")
    a = P.pkv_rope_append(odd[:, :6], odd[:, 6:9], odd[:, 9:], pos, inv, slot, pools[0], pools[1])
    b = P.pkv_rope_append(base[:, :6].contiguous(), base[:, 6:9].contiguous(), base[:, 9:].contiguous(), pos, inv, slot,
                          pools[2], pools[3])
    assert torch.equal(a, b) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_numpy_scalars_and_no_tokens():
    x, pos, inv = inputs(2, 4, 64, 64, "f32")
    want = P.pkv_rope(x, pos, inv, factor=0.5)
    assert torch.equal(P.pkv_rope(x, pos, inv, interleaved=np.bool_(False), factor=np.float32(0.5)), want)
    assert P.pkv_rope(x[:0], pos[:0], inv).shape == (0, 4, 64)
    kp = torch.zeros(1, 1, 8, 64, device="cuda")
    got = P.pkv_rope_append(x[:0, :2], x[:0, 2:3], x[:0, 3:], pos[:0], inv, pos[:0], kp, kp.clone())
    assert got.shape == (0, 2, 64) and not bool(kp.any())
