"""Tensor-level binding of the rotary and block-sparse entry points.

As in ``binding.py`` every function has the name of the C entry point it
calls, checks its tensors and forwards pointers, sizes and the stream that is
current on the tensors' device; the tensors of a call lie on one device, which
need not be the current one.  A decode step's calls are short, so each function
checks everything in one expression first and looks for what is wrong only
where that fails.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _native as N
from ._native import check, lib
from .binding import _DTYPES, _dtype_code

_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}


def _issue(fn, dev: int, *args) -> None:
    """One library call on ``dev`` and the stream current there."""
    stream = _raw_stream(dev)
    if dev == _current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc:
        check(rc)


def _device(t: torch.Tensor, name: str) -> int:
    """The index of a CUDA tensor's device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _on(t: torch.Tensor, name: str, dev: int, dtype=None) -> None:
    """Checks that a tensor is packed, on device ``dev`` and of ``dtype``."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.is_contiguous() and (
            dtype is None or t.dtype == dtype):
        return
    if _device(t, name) != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the other tensors are on device {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _rows(t: torch.Tensor, name: str, dev: int, dtype=None):
    """Checks ``[n_tokens, heads, head_dim]`` with packed heads; returns its
    sizes and the token stride."""
    if _device(t, name) != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the other tensors are on device {dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [n_tokens, heads, head_dim]")
    n, heads, d = t.shape
    s0, s1, s2 = t.stride()
    if t.numel() and ((s2 != 1 and d > 1) or (s1 != d and heads > 1)):
        raise ValueError(f"the heads and channels of {name} must be packed (only the token stride is free)")
    return n, heads, d, s0 if n > 1 else heads * d


_I32, _F64 = torch.int32, torch.float64
_FLOATS = {torch.float32: N.PKV_F32, torch.bfloat16: N.PKV_BF16, torch.float16: N.PKV_F16}


def _packed(s, d: int, heads: int) -> bool:
    """Whether a stride leaves only the token's free."""
    return s[2] == 1 and (s[1] == d or heads == 1)


def _positions(positions: torch.Tensor, inv_freq: torch.Tensor, n: int, dev: int) -> int:
    _on(positions, "positions", dev, torch.int32)
    _on(inv_freq, "inv_freq", dev, torch.float64)
    if positions.numel() != n:
        raise ValueError("positions must hold one position per token")
    return 2 * inv_freq.numel()


def _pools(k_pool: torch.Tensor, v_pool: torch.Tensor, dev: int):
    _on(k_pool, "k_pool", dev)
    _on(v_pool, "v_pool", dev, k_pool.dtype)
    if k_pool.dim() != 4 or k_pool.shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must both be [num_blocks, num_kv_heads, block_size, head_dim]")
    return k_pool.shape


def pkv_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain", scale: float = 1.0,
                         original_positions: int = 0, slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """``(inv_freq, factor)``: float64 frequencies ``[rot_dim / 2]`` on
    ``device`` and the factor of sines and cosines.  ``scaling`` for contexts
    longer than ``original_positions``: "plain", "linear", "base", "bands" or
    "yarn" (the formulas are beside the C declaration)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    factor = ctypes.c_float(0)
    sc = N.pkv_rope_scaling_t(_SCALINGS[scaling], int(original_positions), float(scale), float(slow), float(fast))
    check(lib().pkv_rope_frequencies(rot_dim, float(base), ctypes.byref(sc), out, ctypes.byref(factor)))
    return torch.tensor(list(out), dtype=torch.float64, device=device), factor.value


class _Rotation(torch.autograd.Function):
    """pkv_rope of a tensor that requires a gradient: the transposed map takes
    the gradient back, by another call (so it can be differentiated in turn)."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, interleaved, factor, transpose):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = interleaved, factor, transpose
        return pkv_rope(x, positions, inv_freq, interleaved, factor, transpose)

    @staticmethod
    def backward(ctx, grad):
        interleaved, factor, transpose = ctx.how
        return pkv_rope(grad.contiguous(), *ctx.saved_tensors, interleaved, factor, not transpose), *(None,) * 5


def pkv_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
             factor: float = 1.0, transpose: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotates the first ``2 * len(inv_freq)`` channels of every head of ``x``
    ``[n_tokens, heads, head_dim]`` (float32, bfloat16 or float16; any token
    stride) by ``positions * inv_freq``; returns ``out`` (``x`` itself for in
    place).  ``transpose`` applies the transposed map, which takes the
    gradient of the result to that of ``x``; autograd calls it where ``x``
    requires a gradient (``out`` must then be None; ``inv_freq`` gets none)."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise RuntimeError("pkv_rope with out records no gradient, and x requires one: call it under torch.no_grad()")
        return _Rotation.apply(x, positions, inv_freq, interleaved, factor, transpose)
    code = _FLOATS.get(x.dtype)
    n, heads, d = x.shape if x.dim() == 3 else (0, 0, 0)
    dev, st = x.get_device(), x.stride()
    if not (n and code is not None and dev >= 0 and _packed(st, d, heads) and positions.dtype == _I32
            and positions.get_device() == dev and positions.is_contiguous() and positions.numel() == n
            and inv_freq.dtype == _F64 and inv_freq.get_device() == dev and inv_freq.is_contiguous()):
        dev = _device(x, "x")
        n, heads, d, stride = _rows(x, "x", dev)
        _positions(positions, inv_freq, n, dev)
        if code is None:
            raise TypeError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    else:
        stride = st[0] if n > 1 else heads * d
    rot = 2 * inv_freq.numel()
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ostride = heads * d
    else:
        on, oheads, od, ostride = _rows(out, "out", dev, x.dtype)
        if (on, oheads, od) != (n, heads, d):
            raise ValueError("out has the wrong shape")
    _issue(lib().pkv_rope, dev, x.data_ptr(), stride, positions.data_ptr(), inv_freq.data_ptr(), n, heads, d, rot,
           bool(interleaved), float(factor), bool(transpose), code, out.data_ptr(), ostride)
    return out


def _append_args(q, k, v, positions, inv_freq, slot_mapping, k_pool, v_pool, q_out, q_dtype):
    """What the rotating appends pass on, checked."""
    dtype, dev = k.dtype, k.get_device()
    ks, vs, qs = k.stride(), v.stride(), q.stride()
    if not (k.dim() == q.dim() == 3 and k_pool.dim() == 4):
        raise ValueError("q, k, v must be [n_tokens, heads, head_dim], the pools [num_blocks, num_kv_heads, "
                         "block_size, head_dim]")
    n, hkv, d = k.shape
    nq, hq, dq = q.shape
    nb, ph, bs, pd = k_pool.shape
    if not (n and dev >= 0 and dtype in _FLOATS and nq == n and dq == d and ph == hkv and pd == d
            and v.shape == k.shape and v_pool.shape == k_pool.shape and q.dtype == dtype and v.dtype == dtype
            and v_pool.dtype == k_pool.dtype and q.get_device() == dev and v.get_device() == dev
            and k_pool.get_device() == dev and v_pool.get_device() == dev and k_pool.is_contiguous()
            and v_pool.is_contiguous() and _packed(ks, d, hkv) and _packed(vs, d, hkv) and _packed(qs, d, hq)
            and positions.dtype == _I32 and positions.get_device() == dev and positions.is_contiguous()
            and positions.numel() == n and slot_mapping.dtype == _I32 and slot_mapping.get_device() == dev
            and slot_mapping.is_contiguous() and slot_mapping.numel() == n and inv_freq.dtype == _F64
            and inv_freq.get_device() == dev and inv_freq.is_contiguous()):
        dev = _device(k, "k")
        strides = []
        for t, name in ((k, "k"), (v, "v"), (q, "q")):
            tn, th, td, stride = _rows(t, name, dev, dtype)
            if tn != n or td != d or (name == "v" and th != hkv):
                raise ValueError("q, k and v differ in tokens, head_dim or (k, v) heads")
            strides.append(stride)
        ks, vs, qs = ((x,) for x in strides)
        _pools(k_pool, v_pool, dev)
        if ph != hkv or pd != d:
            raise ValueError(f"q, k, v must be [n_tokens, heads, {pd}] with {ph} heads in k and v")
        _positions(positions, inv_freq, n, dev)
        _on(slot_mapping, "slot_mapping", dev, _I32)
        if slot_mapping.numel() != n:
            raise ValueError("slot_mapping must hold one slot per new token")
        if dtype not in _FLOATS:
            raise TypeError(f"q, k, v must be float32, bfloat16 or float16, got {dtype}")
    elif n == 1:  # a token's stride is anything
        ks = vs = (hkv * d,)
        qs = (hq * d,)
    if q_out is None:
        q_out = torch.empty_like(q, dtype=q_dtype, memory_format=torch.contiguous_format)
    else:
        _on(q_out, "q_out", dev, q_dtype)
        if q_out.shape != q.shape:
            raise ValueError("q_out has the wrong shape")
        if n and q_out.data_ptr() == q.data_ptr():
            raise ValueError("q_out must not be q")
    return (dev, q.data_ptr(), qs[0], k.data_ptr(), ks[0], v.data_ptr(), vs[0]), positions.data_ptr(), \
        inv_freq.data_ptr(), slot_mapping.data_ptr(), n, q_out, k_pool.data_ptr(), v_pool.data_ptr(), \
        (nb, hq, hkv, d, bs, 2 * inv_freq.numel())


def pkv_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                    inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                    interleaved: bool = False, factor: float = 1.0,
                    q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """:func:`pkv_kv_append` with the rotation of :func:`pkv_rope` on the way:
    K rotated and V as it is into their slots (``slot < 0`` = padding), q
    rotated into ``q_out``, which is returned.  q, k, v ``[n_tokens, heads,
    head_dim]`` may be views of one projection's output.  Like every call that
    writes or reads a pool it records no gradient."""
    if k_pool.dtype != k.dtype:
        raise TypeError(f"k is {k.dtype}, the pools are {k_pool.dtype}")
    rows, pos, inv, slots, n, q_out, kp, vp, sizes = _append_args(q, k, v, positions, inv_freq, slot_mapping, k_pool,
                                                                  v_pool, q_out, k.dtype)
    _issue(lib().pkv_rope_append, *rows, pos, inv, slots, n, q_out.data_ptr(), kp, vp, *sizes,
           bool(interleaved), float(factor), _FLOATS[k.dtype])
    return q_out


def pkv_rope_append_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                        inv_freq: torch.Tensor, slot_mapping: torch.Tensor, k_pool: torch.Tensor,
                        v_pool: torch.Tensor, k_scale: float, v_scale: float, interleaved: bool = False,
                        factor: float = 1.0, q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """:func:`pkv_rope_append` into e4m3 pools (x / scale rounded once to its
    code); the returned q is float16."""
    if k_pool.dtype not in _E4M3:
        raise TypeError(f"the pools must hold e4m3 codes, got {k_pool.dtype}")
    rows, pos, inv, slots, n, q_out, kp, vp, sizes = _append_args(q, k, v, positions, inv_freq, slot_mapping, k_pool,
                                                                  v_pool, q_out, torch.float16)
    _issue(lib().pkv_rope_append_fp8, *rows, _FLOATS[k.dtype], pos, inv, slots, n, q_out.data_ptr(), kp, vp, *sizes,
           bool(interleaved), float(factor), float(k_scale), float(v_scale))
    return q_out


def _batch(block_tables: torch.Tensor, seq_lens: torch.Tensor, dev: int):
    b, shape = seq_lens.numel(), block_tables.shape
    if not (len(shape) == 2 and shape[0] == b and block_tables.dtype == _I32 and seq_lens.dtype == _I32
            and block_tables.get_device() == dev and seq_lens.get_device() == dev and block_tables.is_contiguous()
            and seq_lens.is_contiguous()):
        _on(block_tables, "block_tables", dev, _I32)
        _on(seq_lens, "seq_lens", dev, _I32)
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq] and seq_lens [num_seqs]")
    return b, shape[1]


def pkv_block_bounds(k_pool: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, bounds: torch.Tensor,
                     new_tokens: Optional[torch.Tensor] = None, max_new_tokens: int = 1) -> torch.Tensor:
    """Rewrites, in ``bounds`` ``[num_blocks, num_kv_heads, 2, head_dim]`` (the
    pool's dtype), the smallest and largest key of every block that holds one
    of the last ``new_tokens`` tokens of a sequence (int32 ``[num_seqs]``;
    None: one each); returns ``bounds``."""
    dev = _device(k_pool, "k_pool")
    _on(k_pool, "k_pool", dev)
    if k_pool.dim() != 4:
        raise ValueError("k_pool must be [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = k_pool.shape
    _on(bounds, "bounds", dev, k_pool.dtype)
    if tuple(bounds.shape) != (nb, hkv, 2, d):
        raise ValueError(f"bounds must be [{nb}, {hkv}, 2, {d}]")
    b, maxb = _batch(block_tables, seq_lens, dev)
    if new_tokens is not None:
        _on(new_tokens, "new_tokens", dev, torch.int32)
        if new_tokens.numel() != b:
            raise ValueError("new_tokens must be [num_seqs]")
    _issue(lib().pkv_block_bounds, dev, k_pool.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
           None if new_tokens is None else new_tokens.data_ptr(), int(max_new_tokens), b, nb, hkv, d, maxb, bs,
           _dtype_code(k_pool), bounds.data_ptr())
    return bounds


@functools.lru_cache(maxsize=256)
def pkv_select_workspace_size(num_seqs: int, num_kv_heads: int, max_blocks_per_seq: int) -> int:
    """Workspace bytes of :func:`pkv_block_select`."""
    out = ctypes.c_size_t(0)
    check(lib().pkv_select_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq, ctypes.byref(out)))
    return out.value


def pkv_block_select(q: torch.Tensor, bounds: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     max_selected: int, block_size: int, n_first: int = 1, n_last: int = 2,
                     selected: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The blocks each (sequence, KV head) attends over: ``selected`` int32
    ``[num_seqs, num_kv_heads, max_selected]``, ascending logical block
    indices, -1 behind the last - the first ``n_first`` and last ``n_last``
    blocks and the best-scored of the others (see the C declaration)."""
    dev = _device(bounds, "bounds")
    _on(bounds, "bounds", dev)
    if bounds.dim() != 4 or bounds.shape[2] != 2:
        raise ValueError("bounds must be [num_blocks, num_kv_heads, 2, head_dim]")
    nb, hkv, _, d = bounds.shape
    b, maxb = _batch(block_tables, seq_lens, dev)
    _on(q, "q", dev, torch.float16 if bounds.dtype in _E4M3 else bounds.dtype)
    if q.dim() != 3 or q.shape[0] != b or q.shape[2] != d:
        raise ValueError(f"q must be [{b}, num_q_heads, {d}]")
    if selected is None:
        selected = seq_lens.new_empty((b, hkv, max_selected))
    else:
        _on(selected, "selected", dev, torch.int32)
        if tuple(selected.shape) != (b, hkv, max_selected):
            raise ValueError("selected has the wrong shape")
    if workspace is None:
        ws_bytes = pkv_select_workspace_size(b, hkv, maxb)  # a multiple of 256
        workspace = seq_lens.new_empty(ws_bytes // 4)
    else:
        _on(workspace, "workspace", dev, torch.uint8)
        ws_bytes = workspace.numel()
    _issue(lib().pkv_block_select, dev, q.data_ptr(), bounds.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
           b, q.shape[1], hkv, d, nb, maxb, int(block_size), int(max_selected), int(n_first),
           int(n_last), _dtype_code(bounds), workspace.data_ptr(), ws_bytes, selected.data_ptr())
    return selected


@functools.lru_cache(maxsize=256)
def pkv_sparse_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_selected: int,
                              block_size: int, dtype: torch.dtype) -> int:
    """Workspace bytes of the block-sparse decode over pools of ``dtype`` (0
    where it needs none)."""
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; expected float32, bfloat16, float16 or e4m3 codes")
    out = ctypes.c_size_t(0)
    check(lib().pkv_sparse_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_selected, block_size,
                                          _DTYPES[dtype], ctypes.byref(out)))
    return out.value


def _sparse(fn, q, k_pool, v_pool, block_tables, seq_lens, selected, tail, q_dtype, out, workspace):
    dev = _device(k_pool, "k_pool")
    nb, hkv, bs, d = _pools(k_pool, v_pool, dev)
    b, maxb = _batch(block_tables, seq_lens, dev)
    _on(q, "q", dev, q_dtype)
    if q.dim() != 3 or q.shape[0] != b or q.shape[2] != d:
        raise ValueError(f"q must be [{b}, num_q_heads, {d}]")
    _on(selected, "selected", dev, torch.int32)
    if selected.dim() != 3 or selected.shape[:2] != (b, hkv):
        raise ValueError(f"selected must be [{b}, {hkv}, max_selected]")
    hq, k = q.shape[1], selected.shape[2]
    if out is None:
        out = torch.empty_like(q, dtype=torch.float32)  # q is packed
    else:
        _on(out, "out", dev, torch.float32)
        if tuple(out.shape) != (b, hq, d):
            raise ValueError("out has the wrong shape")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _on(workspace, "workspace", dev, torch.uint8)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
    else:
        ws_bytes = pkv_sparse_workspace_size(b, hq, hkv, d, k, bs, k_pool.dtype)  # 0 or a multiple of 256
        if ws_bytes:
            workspace = seq_lens.new_empty(ws_bytes // 4)
            ws_ptr = workspace.data_ptr()
    _issue(fn, dev, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
           selected.data_ptr(), k, b, hq, hkv, d, nb, maxb, bs, *tail, ws_ptr, ws_bytes, out.data_ptr())
    return out


def pkv_paged_attention_decode_sparse(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                      block_tables: torch.Tensor, seq_lens: torch.Tensor, selected: torch.Tensor,
                                      scale: float, out: Optional[torch.Tensor] = None,
                                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """:func:`pkv_paged_attention_decode` over the tokens of the selected
    blocks only (``selected`` as :func:`pkv_block_select` returns it); float32
    ``[num_seqs, num_q_heads, head_dim]``, zeros for an empty selection."""
    return _sparse(lib().pkv_paged_attention_decode_sparse, q, k_pool, v_pool, block_tables, seq_lens, selected,
                   (float(scale), _dtype_code(k_pool)), k_pool.dtype, out, workspace)


def pkv_paged_attention_decode_sparse_fp8(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                          block_tables: torch.Tensor, seq_lens: torch.Tensor, selected: torch.Tensor,
                                          scale: float, k_scale: float, v_scale: float,
                                          out: Optional[torch.Tensor] = None,
                                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The same over e4m3 pools (q float16)."""
    if k_pool.dtype not in _E4M3:
        raise TypeError(f"the pools must hold e4m3 codes, got {k_pool.dtype}")
    return _sparse(lib().pkv_paged_attention_decode_sparse_fp8, q, k_pool, v_pool, block_tables, seq_lens, selected,
                   (float(scale), float(k_scale), float(v_scale)), torch.float16, out, workspace)


__all__ = ["pkv_rope_frequencies", "pkv_rope", "pkv_rope_append", "pkv_rope_append_fp8", "pkv_block_bounds",
           "pkv_select_workspace_size", "pkv_block_select", "pkv_sparse_workspace_size",
           "pkv_paged_attention_decode_sparse", "pkv_paged_attention_decode_sparse_fp8"]
