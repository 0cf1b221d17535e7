"""Rotary and block-sparse entry points on the host: frequencies against their
formulas, workspace sizes, and refusals (no call here reaches a launch)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_406_b200 import _native as N

FAKE = 1 << 20  # an aligned non-null address; every call below fails validation before using it


def _freq(native, rot, base, kind=0, orig=0, scale=1.0, slow=1.0, fast=32.0):
    out = (ctypes.c_double * max(1, rot // 2))()
    factor = ctypes.c_float(0)
    sc = N.pkv_rope_scaling_t(kind, orig, scale, slow, fast)
    rc = native.pkv_rope_frequencies(rot, base, ctypes.byref(sc), out, ctypes.byref(factor))
    return rc, np.array(out), factor.value


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (2, 10000.0), (20, 1e6)])
def test_plain_and_linear_frequencies(native, rot, base):
    rc, f, factor = _freq(native, rot, base)
    want = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    assert rc == 0 and factor == 1.0
    np.testing.assert_allclose(f, want, rtol=1e-14)
    rc, g, factor = _freq(native, rot, base, 1, scale=8.0)
    assert rc == 0 and factor == 1.0
    np.testing.assert_allclose(g, want / 8, rtol=1e-14)
    out = (ctypes.c_double * (rot // 2))()
    fac = ctypes.c_float(0)
    assert native.pkv_rope_frequencies(rot, base, None, out, ctypes.byref(fac)) == 0  # no scaling: plain
    assert np.array_equal(np.array(out), f) and fac.value == 1.0


def test_scaled_base_keeps_the_shortest_and_stretches_the_longest_wave(native):
    _, plain, _ = _freq(native, 128, 10000.0)
    rc, f, factor = _freq(native, 128, 10000.0, 2, scale=4.0)
    assert rc == 0 and factor == 1.0 and f[0] == 1.0
    # base * s^(R / (R - 2)) turns base^(-(R - 2) / R) into base^(-(R - 2) / R) / s
    assert math.isclose(f[-1], plain[-1] / 4.0, rel_tol=1e-12)


def test_bands(native):
    orig, s, slow, fast = 8192, 8.0, 1.0, 4.0
    _, plain, _ = _freq(native, 128, 500000.0)
    rc, f, factor = _freq(native, 128, 500000.0, 3, orig, s, slow, fast)
    assert rc == 0 and factor == 1.0
    kinds = set()
    for p, got in zip(plain, f):
        turns = orig * p / (2 * math.pi)
        if turns <= slow:
            want, kind = p / s, "slow"
        elif turns >= fast:
            want, kind = p, "fast"
        else:
            keep = (turns - slow) / (fast - slow)
            want, kind = p * keep + p / s * (1 - keep), "blend"
        kinds.add(kind)
        assert math.isclose(got, want, rel_tol=1e-12)
    assert kinds == {"slow", "fast", "blend"}


def test_yarn(native):
    orig, s, slow, fast, rot, base = 4096, 16.0, 1.0, 32.0, 128, 10000.0
    _, plain, _ = _freq(native, rot, base)
    rc, f, factor = _freq(native, rot, base, 4, orig, s, slow, fast)
    assert rc == 0 and math.isclose(factor, 0.1 * math.log(16) + 1, rel_tol=2.0 ** -24)

    def pair(turns):  # base^(-2 i / rot) * orig = 2 pi turns, solved for i
        return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))

    a, b = math.floor(pair(fast)), math.ceil(pair(slow))
    for i, (p, got) in enumerate(zip(plain, f)):
        keep = 1 - min(1.0, max(0.0, (i - a) / (b - a)))
        assert math.isclose(got, p * keep + p / s * (1 - keep), rel_tol=1e-12)
    assert f[a] == plain[a] and f[b] != plain[b]


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=3), dict(rot=-2), dict(base=1.0), dict(base=float("nan")), dict(kind=1, scale=0.5),
    dict(kind=1, scale=float("inf")), dict(kind=2, rot=2, scale=2.0), dict(kind=3, scale=2.0, orig=0),
    dict(kind=4, scale=2.0, orig=4096, slow=4.0, fast=4.0), dict(kind=4, scale=2.0, orig=4096, slow=0.0),
])
def test_frequency_refusals(native, kw):
    a = dict(rot=64, base=10000.0)
    a.update(kw)
    assert _freq(native, a.pop("rot"), a.pop("base"), **a)[0] == N.PKV_ERR_INVALID_ARG


def test_unknown_scaling_is_unsupported(native):
    assert _freq(native, 64, 10000.0, 9, scale=2.0)[0] == N.PKV_ERR_UNSUPPORTED
    import paged_kv_cache_406_b200 as P
    with pytest.raises(ValueError):
        P.pkv_rope_frequencies(64, scaling="other", device="cpu")
    f, factor = P.pkv_rope_frequencies(64, 10000.0, "yarn", 16.0, 4096, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and factor > 1


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), N.PKV_ERR_UNSUPPORTED),
    (dict(dtype=N.PKV_FP8_E4M3), N.PKV_ERR_UNSUPPORTED),
    (dict(d=100), N.PKV_ERR_UNSUPPORTED),
    (dict(d=520), N.PKV_ERR_UNSUPPORTED),
    (dict(rot=0), N.PKV_ERR_INVALID_ARG),
    (dict(rot=63), N.PKV_ERR_INVALID_ARG),
    (dict(rot=130), N.PKV_ERR_INVALID_ARG),
    (dict(n=-1), N.PKV_ERR_INVALID_ARG),
    (dict(h=0), N.PKV_ERR_INVALID_ARG),
    (dict(il=2), N.PKV_ERR_INVALID_ARG),
    (dict(tr=-1), N.PKV_ERR_INVALID_ARG),
    (dict(factor=float("inf")), N.PKV_ERR_INVALID_ARG),
    (dict(x=0), N.PKV_ERR_INVALID_ARG),
    (dict(x=FAKE + 8), N.PKV_ERR_INVALID_ARG),
    (dict(pos=0), N.PKV_ERR_INVALID_ARG),
    (dict(f=FAKE + 4), N.PKV_ERR_INVALID_ARG),
    (dict(xs=8 * 128 - 8), N.PKV_ERR_INVALID_ARG),      # tokens would overlap
    (dict(xs=8 * 128 + 4), N.PKV_ERR_INVALID_ARG),      # not a multiple of 16 bytes
    (dict(x=FAKE, out=FAKE, xs=8 * 256), N.PKV_ERR_INVALID_ARG),  # in place with another stride
])
def test_rope_refusals(native, kw, code):
    a = dict(x=FAKE, xs=8 * 128, pos=FAKE, f=FAKE, n=4, h=8, d=128, rot=128, il=0, factor=1.0, tr=0, dtype=N.PKV_BF16,
             out=2 * FAKE, os=8 * 128)
    a.update(kw)
    rc = native.pkv_rope(a["x"], a["xs"], a["pos"], a["f"], a["n"], a["h"], a["d"], a["rot"], a["il"], a["factor"],
                         a["tr"], a["dtype"], a["out"], a["os"], None)
    assert rc == code, native.pkv_last_error_string()


APPEND = [
    (dict(dtype=9), N.PKV_ERR_UNSUPPORTED),
    (dict(d=96), N.PKV_ERR_UNSUPPORTED),
    (dict(bs=12), N.PKV_ERR_UNSUPPORTED),
    (dict(hkv=0), N.PKV_ERR_INVALID_ARG),
    (dict(nb=0), N.PKV_ERR_INVALID_ARG),
    (dict(rot=129), N.PKV_ERR_INVALID_ARG),
    (dict(ks=1024 + 2), N.PKV_ERR_INVALID_ARG),
    (dict(vs=512), N.PKV_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), N.PKV_ERR_INVALID_ARG),
    (dict(q=0), N.PKV_ERR_INVALID_ARG),
    (dict(qo=0), N.PKV_ERR_INVALID_ARG),
    (dict(slots=0), N.PKV_ERR_INVALID_ARG),
    (dict(kp=FAKE + 4), N.PKV_ERR_INVALID_ARG),
    (dict(factor=float("nan")), N.PKV_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", APPEND + [(dict(dtype=N.PKV_FP8_E4M3), N.PKV_ERR_UNSUPPORTED)])
def test_rope_append_refusals(native, kw, code):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, f=FAKE, slots=FAKE, n=3, qo=FAKE, kp=FAKE,
             vp=FAKE, nb=8, hq=32, hkv=8, d=128, bs=16, rot=128, factor=1.0, dtype=N.PKV_BF16)
    a.update(kw)
    rc = native.pkv_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["f"], a["slots"], a["n"],
                                a["qo"], a["kp"], a["vp"], a["nb"], a["hq"], a["hkv"], a["d"], a["bs"], a["rot"], 0,
                                a["factor"], a["dtype"], None)
    assert rc == code, native.pkv_last_error_string()


@pytest.mark.parametrize("kw,code", APPEND + [(dict(k_scale=0.0), N.PKV_ERR_INVALID_ARG),
                                              (dict(v_scale=float("inf")), N.PKV_ERR_INVALID_ARG)])
def test_rope_append_fp8_refusals(native, kw, code):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, f=FAKE, slots=FAKE, n=3, qo=FAKE, kp=FAKE,
             vp=FAKE, nb=8, hq=32, hkv=8, d=128, bs=16, rot=128, factor=1.0, dtype=N.PKV_F16, k_scale=0.5, v_scale=0.5)
    a.update(kw)
    rc = native.pkv_rope_append_fp8(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["dtype"], a["pos"], a["f"],
                                    a["slots"], a["n"], a["qo"], a["kp"], a["vp"], a["nb"], a["hq"], a["hkv"], a["d"],
                                    a["bs"], a["rot"], 0, a["factor"], a["k_scale"], a["v_scale"], None)
    assert rc == code, native.pkv_last_error_string()


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), N.PKV_ERR_UNSUPPORTED),
    (dict(dtype=N.PKV_FP8_E4M3, d=64), N.PKV_ERR_UNSUPPORTED),
    (dict(bs=24), N.PKV_ERR_UNSUPPORTED),
    (dict(mx=-1), N.PKV_ERR_INVALID_ARG),
    (dict(new=None, mx=0), N.PKV_ERR_INVALID_ARG),
    (dict(maxb=1 << 21), N.PKV_ERR_INVALID_ARG),
    (dict(B=-1), N.PKV_ERR_INVALID_ARG),
    (dict(lens=0), N.PKV_ERR_INVALID_ARG),
    (dict(bounds=FAKE + 8), N.PKV_ERR_INVALID_ARG),
])
def test_bounds_refusals(native, kw, code):
    a = dict(kp=FAKE, t=FAKE, lens=FAKE, new=FAKE, mx=16, B=2, nb=8, hkv=8, d=128, maxb=4, bs=16, dtype=N.PKV_BF16,
             bounds=FAKE)
    a.update(kw)
    rc = native.pkv_block_bounds(a["kp"], a["t"], a["lens"], a["new"], a["mx"], a["B"], a["nb"], a["hkv"], a["d"],
                                 a["maxb"], a["bs"], a["dtype"], a["bounds"], None)
    assert rc == code, native.pkv_last_error_string()


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), N.PKV_ERR_UNSUPPORTED),
    (dict(hq=24), N.PKV_ERR_UNSUPPORTED),
    (dict(hq=30), N.PKV_ERR_INVALID_ARG),
    (dict(K=0), N.PKV_ERR_INVALID_ARG),
    (dict(first=-1), N.PKV_ERR_INVALID_ARG),
    (dict(first=5, last=4), N.PKV_ERR_INVALID_ARG),     # more than max_selected
    (dict(ws=FAKE + 16), N.PKV_ERR_INVALID_ARG),
    (dict(ws_bytes=100), N.PKV_ERR_INVALID_ARG),
    (dict(q=FAKE + 4), N.PKV_ERR_INVALID_ARG),
    (dict(sel=0), N.PKV_ERR_INVALID_ARG),
    (dict(maxb=(1 << 20) + 1, bs=8), N.PKV_ERR_INVALID_ARG),
])
def test_select_refusals(native, kw, code):
    a = dict(q=FAKE, bounds=FAKE, t=FAKE, lens=FAKE, B=2, hq=32, hkv=8, d=128, nb=64, maxb=64, bs=16, K=8, first=1,
             last=2, dtype=N.PKV_BF16, ws=FAKE, ws_bytes=1 << 30, sel=FAKE)
    a.update(kw)
    rc = native.pkv_block_select(a["q"], a["bounds"], a["t"], a["lens"], a["B"], a["hq"], a["hkv"], a["d"], a["nb"],
                                 a["maxb"], a["bs"], a["K"], a["first"], a["last"], a["dtype"], a["ws"], a["ws_bytes"],
                                 a["sel"], None)
    assert rc == code, native.pkv_last_error_string()


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), N.PKV_ERR_UNSUPPORTED),
    (dict(dtype=N.PKV_FP8_E4M3), N.PKV_ERR_UNSUPPORTED),  # has its own form
    (dict(dtype=N.PKV_F32, hq=64), N.PKV_ERR_UNSUPPORTED),
    (dict(hq=24), N.PKV_ERR_UNSUPPORTED),
    (dict(K=0), N.PKV_ERR_INVALID_ARG),
    (dict(scale=float("nan")), N.PKV_ERR_INVALID_ARG),
    (dict(ws_bytes=64, K=2000), N.PKV_ERR_INVALID_ARG),     # a long list needs a workspace,
    (dict(ws=None, K=2000), N.PKV_ERR_INVALID_ARG),
    (dict(ws=FAKE + 16, K=2000), N.PKV_ERR_INVALID_ARG),
    (dict(ws_bytes=64, dtype=N.PKV_F32), N.PKV_ERR_INVALID_ARG),  # and so do fp32 pools
    (dict(sel=0), N.PKV_ERR_INVALID_ARG),
    (dict(out=FAKE + 4), N.PKV_ERR_INVALID_ARG),
    (dict(nb=1 << 27), N.PKV_ERR_INVALID_ARG),           # more than 2^31 token rows
])
def test_sparse_decode_refusals(native, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, t=FAKE, lens=FAKE, sel=FAKE, K=8, B=2, hq=32, hkv=8, d=128, nb=64, maxb=64, bs=16,
             scale=0.1, dtype=N.PKV_BF16, ws=FAKE, ws_bytes=1 << 30, out=FAKE)
    a.update(kw)
    rc = native.pkv_paged_attention_decode_sparse(
        a["q"], a["k"], a["v"], a["t"], a["lens"], a["sel"], a["K"], a["B"], a["hq"], a["hkv"], a["d"], a["nb"],
        a["maxb"], a["bs"], a["scale"], a["dtype"], a["ws"], a["ws_bytes"], a["out"], None)
    assert rc == code, native.pkv_last_error_string()


def test_sparse_decode_fp8_refusals(native):
    def call(d=128, ks=0.5, vs=0.5):  # a list of 2000 blocks: a workspace is needed
        return native.pkv_paged_attention_decode_sparse_fp8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2000, 2, 32, 8, d, 64,
                                                            64, 16, 0.1, ks, vs, FAKE, 16, FAKE, None)
    assert call(d=64) == N.PKV_ERR_UNSUPPORTED
    assert call(ks=0.0) == N.PKV_ERR_INVALID_ARG
    assert call(vs=float("nan")) == N.PKV_ERR_INVALID_ARG
    assert call() == N.PKV_ERR_INVALID_ARG  # workspace too small


def test_empty_calls_are_no_ops(native):
    assert native.pkv_rope(None, 0, None, None, 0, 8, 128, 128, 0, 1.0, 0, N.PKV_BF16, None, 0, None) == 0
    assert native.pkv_rope_append(None, 0, None, 0, None, 0, None, None, None, 0, None, None, None, 8, 32, 8, 128, 16,
                                  128, 0, 1.0, N.PKV_BF16, None) == 0
    assert native.pkv_block_bounds(None, None, None, None, 1, 0, 8, 8, 128, 4, 16, N.PKV_BF16, None, None) == 0
    assert native.pkv_block_select(None, None, None, None, 0, 32, 8, 128, 8, 4, 16, 4, 1, 1, N.PKV_BF16, None, 0, None,
                                   None) == 0
    assert native.pkv_paged_attention_decode_sparse(None, None, None, None, None, None, 4, 0, 32, 8, 128, 8, 4, 16, 0.1,
                                                    N.PKV_BF16, None, 0, None, None) == 0


def test_workspace_sizes(native):
    out = ctypes.c_size_t(0)
    assert native.pkv_select_workspace_size(64, 8, 2048, ctypes.byref(out)) == 0 and out.value >= 64 * 8 * 2048 * 12
    assert native.pkv_select_workspace_size(0, 8, 2048, ctypes.byref(out)) == 0
    assert native.pkv_select_workspace_size(1, 0, 2048, ctypes.byref(out)) == N.PKV_ERR_INVALID_ARG
    assert native.pkv_sparse_workspace_size(64, 32, 8, 128, 64, 16, N.PKV_BF16, ctypes.byref(out)) == 0 and out.value == 0
    assert native.pkv_sparse_workspace_size(64, 32, 8, 128, 64, 16, N.PKV_F32, ctypes.byref(out)) == 0 and out.value > 0
    assert native.pkv_sparse_workspace_size(64, 32, 8, 128, 1025, 16, N.PKV_BF16, ctypes.byref(out)) == 0 and out.value > 0
    assert native.pkv_sparse_workspace_size(64, 30, 8, 128, 64, 16, N.PKV_BF16, ctypes.byref(out)) == N.PKV_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    import paged_kv_cache_406_b200 as P
    x, pos, f = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        P.pkv_rope(x, pos, f)
    with pytest.raises(ValueError):
        P.pkv_block_bounds(torch.zeros(2, 1, 8, 64), pos[None], pos[:1], torch.zeros(2, 1, 2, 64))
