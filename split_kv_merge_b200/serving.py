"""Serving operators around the attention calls: rotary positions and the cache append.  Argument
checks and marshalling; the work runs in the library's kernels."""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import Optional

import numpy as np

from . import (AppendParams, BF16, E4M3, F32, I8, PagedParams, PagedScaledParams, Plan, PromptParams, Rope,
               RopeParams, _check, _index_ptr, _kv_append, _prompt_fwd, _ROPE, _ROPE_SCALING, _rope_apply,
               _rope_frequencies, _scaled_fwd, plan_paged_scaled, plan_prompt)

_NULL = nullcontext()


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on(dev, **tensors) -> None:
    """Every given tensor lives on the CUDA device ``dev``."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _cache_code(dtype):
    import torch
    return {torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3, torch.uint8: E4M3, torch.int8: I8}.get(dtype)


def _index(name: str, t, n: Optional[int] = None) -> None:
    import torch
    if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous()
                          or (n is not None and t.shape[0] != n)):
        raise ValueError(f"{name} must be a contiguous int32 vector" + ("" if n is None else f" of {n} entries"))


def _device(dev):
    """Context that makes ``dev`` current for the launch (a no-op when it already is)."""
    import torch
    _need(dev.type == "cuda", "tensors must be on a CUDA device")
    return _NULL if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream(stream, dev) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream(dev).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(stream, dev):
    """Context in which outputs are allocated for work on ``stream``, so that their memory is not
    handed out again before that work is done."""
    if stream is None:
        return _NULL
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _rope(rope_dim: int, rope_theta: float, rope_layout: str, inv_freq, mscale: float):
    """(skv_rope, the frequency array it points to -- keep it until the call returns)."""
    _need(rope_layout in _ROPE, f"rope_layout must be one of {sorted(_ROPE)}")
    if inv_freq is None or rope_dim == 0:
        return Rope(rope_dim, _ROPE[rope_layout], rope_theta, None, mscale), None
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    _need(f.shape == (rope_dim // 2,), f"inv_freq must hold rope_dim / 2 = {rope_dim // 2} frequencies")
    return Rope(rope_dim, _ROPE[rope_layout], rope_theta, f.__array_interface__["data"][0], mscale), f


def rope_frequencies(rope_dim: int, rope_theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_context: float = 8192, low: Optional[float] = None, high: Optional[float] = None):
    """skv_rope_frequencies: (inv_freq float64 [rope_dim / 2], mscale) of the base ``rope_theta``, stretched
    for long contexts by ``scaling``: "linear" (positions divided by ``factor``), "ntk" (a larger base),
    "yarn" or "bands" (pairs that turn fewer than ``low`` times in ``original_context`` positions are
    stretched, those that turn more than ``high`` times kept, a ramp between; 1 and 32 by default for
    "yarn", which also gives an mscale, 1 and 4 for "bands").  Pass both on to ``rope_apply`` or
    ``paged_kv_append``."""
    _need(scaling in _ROPE_SCALING, f"scaling must be one of {sorted(_ROPE_SCALING)}")
    lo = 1.0 if low is None else low
    hi = (4.0 if scaling == "bands" else 32.0) if high is None else high
    f, m = np.zeros(max(1, rope_dim // 2)), ctypes.c_float(1.0)
    _check(_rope_frequencies(rope_dim, rope_theta, _ROPE_SCALING[scaling], factor, original_context, lo, hi,
                             f.ctypes.data, ctypes.byref(m)), "skv_rope_frequencies")
    return f, float(m.value)


def _rows3(name: str, t, rows: int, dim: int) -> None:
    _need(t.dim() == 3 and t.shape[0] == rows and t.shape[2] == dim and (t.stride(2) == 1 or t.numel() == 0),
          f"{name} must be [{rows}, heads, {dim}] with contiguous heads, got {tuple(t.shape)}")


def rope_apply(q, k, positions, *, rope_dim: Optional[int] = None, rope_theta: float = 10000.0,
               rope_layout: str = "interleaved", inv_freq=None, mscale: float = 1.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None):
    """skv_rope_apply: rotary positions of q [tokens, Hq, D] and k [tokens, Hk, D] (either may be None; bf16
    or float32, any token / head strides), ``positions`` int32 [tokens] on the device.  The first
    ``rope_dim`` (default D) values of a head turn, the others are copied.  ``inv_freq`` (float64, host)
    replaces rope_theta^(-2p/rope_dim).  ``q_out=q`` / ``k_out=k`` rotates in place; ``inverse`` turns
    back (and takes gradients through the rotation).  Returns (q_out, k_out)."""
    import torch
    x = q if q is not None else k
    _need(x is not None, "one of q and k is needed")
    _need(x.dim() == 3, "q and k are [tokens, heads, head_dim]")
    dev, tokens, dim, dtype = x.device, x.shape[0], x.shape[2], x.dtype
    _need(dtype in (torch.bfloat16, torch.float32), "q and k must be bfloat16 or float32")
    _on(dev, q=q, k=k, positions=positions, q_out=q_out, k_out=k_out)
    _index("positions", positions, tokens)
    with _device(dev):
        with _on_stream(stream, dev):
            if q is not None and q_out is None:
                q_out = torch.empty(q.shape, dtype=dtype, device=dev)
            if k is not None and k_out is None:
                k_out = torch.empty(k.shape, dtype=dtype, device=dev)
        args = [None] * 4
        strides = [(0, 0)] * 4
        for i, (name, t, like) in enumerate((("q", q, q), ("q_out", q_out, q), ("k", k, k), ("k_out", k_out, k))):
            if like is None:
                _need(t is None, f"{name} without its input")
                continue
            _rows3(name, t, tokens, dim)
            _need(t.dtype == dtype and t.shape == like.shape, f"{name} must have the dtype and shape of its input")
            args[i], strides[i] = t.data_ptr(), t.stride()[:2]
        desc, keep = _rope(dim if rope_dim is None else rope_dim, rope_theta, rope_layout, inv_freq, mscale)
        p = RopeParams(*args, *strides, positions.data_ptr(), tokens, 0 if q is None else q.shape[1],
                       0 if k is None else k.shape[1], dim, F32 if dtype == torch.float32 else BF16, int(inverse), desc)
        _check(_rope_apply(ctypes.byref(p), _stream(stream, dev)), "skv_rope_apply")
    del keep
    return q_out, k_out


def _scales(k_cache, k_scale, v_scale, num_pages: int):
    """Tokens that share a scale in the scale tensors [num_pages, blocks per page, Hk] float32."""
    import torch
    page, hk = k_cache.shape[1], k_cache.shape[2]
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _need(t.dim() == 3 and t.dtype == torch.float32 and t.shape[0] >= num_pages and t.shape[2] == hk
              and t.shape[1] > 0 and page % t.shape[1] == 0 and t.shape[1] == k_scale.shape[1],
              f"{name} must be float32 [num_pages, blocks per page, {hk}] with whole blocks of tokens")
    return page // k_scale.shape[1]


def paged_kv_append(k, v, k_cache, v_cache, append_indptr, kv_indptr, kv_indices, kv_last_page_len, *, k_scale=None,
                    v_scale=None, kv_scale: float = 1.0, q=None, q_out=None, positions=None, rope_dim: int = 0,
                    rope_theta: float = 10000.0, rope_layout: str = "interleaved", inv_freq=None, mscale: float = 1.0,
                    num_pages: Optional[int] = None, status=None, stream=None):
    """skv_paged_kv_append: new keys and values k, v [rows, Hk, D] bf16 into the paged cache.  Request r's
    new tokens are rows append_indptr[r] .. append_indptr[r+1] and become its last positions; the page
    table (device int32) describes the requests after the append.  Caches [num_pages, P, Hk, D]: bf16;
    float8_e4m3fn with the per-tensor ``kv_scale``; or float8_e4m3fn / int8 with ``k_scale`` /
    ``v_scale`` float32 [num_pages, P / block, Hk], one scale for each block of tokens and head, which
    the call updates.  ``rope_dim`` > 0 rotates the keys (and ``q`` [rows, Hq, D]) on the way, at the
    tokens' positions or at ``positions``.  Returns q_out (None without q)."""
    import torch
    _need(k.dim() == 3 and k_cache.dim() == 4, "k is [rows, Hk, D], the caches [num_pages, P, Hk, D]")
    dev, rows, hk, dim = k.device, k.shape[0], k.shape[1], k.shape[2]
    code = _cache_code(k_cache.dtype)
    _need(code is not None and v_cache.dtype == k_cache.dtype, "caches must both be bfloat16, float8_e4m3fn or int8")
    _need(k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16, "k and v must be bfloat16")
    _on(dev, v=v, k_cache=k_cache, v_cache=v_cache, append_indptr=append_indptr, kv_indptr=kv_indptr,
        kv_indices=kv_indices, kv_last_page_len=kv_last_page_len, k_scale=k_scale, v_scale=v_scale, q=q, q_out=q_out,
        positions=positions, status=status)
    _rows3("k", k, rows, dim)
    _rows3("v", v, rows, dim)
    _need(v.shape[1] == hk and k_cache.shape[2:] == (hk, dim) and v_cache.shape == k_cache.shape
          and k_cache.stride(3) == 1 and v_cache.stride(3) == 1, "the caches must be [num_pages, P, Hk, D] like k and v")
    batch = append_indptr.shape[0] - 1
    _index("append_indptr", append_indptr)
    _index("kv_indptr", kv_indptr, batch + 1)
    _index("kv_indices", kv_indices)
    _index("kv_last_page_len", kv_last_page_len, batch)
    _index("positions", positions, rows)
    pages = k_cache.shape[0] if num_pages is None else num_pages
    _need(0 <= pages <= k_cache.shape[0], "num_pages is more than the cache holds")
    block = 0
    if k_scale is not None or v_scale is not None:
        _need(k_scale is not None and v_scale is not None, "k_scale and v_scale come together")
        block = _scales(k_cache, k_scale, v_scale, pages)
    with _device(dev):
        if q is not None:
            if q_out is None:
                with _on_stream(stream, dev):
                    q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            for name, t in (("q", q), ("q_out", q_out)):
                _rows3(name, t, rows, dim)
                _need(t.dtype == torch.bfloat16 and t.shape == q.shape, f"{name} must be bfloat16 [rows, Hq, D]")
        else:
            _need(q_out is None, "q_out without q")
        desc, keep = _rope(rope_dim, rope_theta, rope_layout, inv_freq, mscale)
        none3 = (0, 0, 0)
        p = AppendParams(k.data_ptr(), v.data_ptr(), k.stride()[:2], v.stride()[:2], k_cache.data_ptr(),
                         v_cache.data_ptr(), k_cache.stride()[:3], v_cache.stride()[:3], code, kv_scale, block,
                         k_scale.data_ptr() if block else None, v_scale.data_ptr() if block else None,
                         k_scale.stride() if block else none3, v_scale.stride() if block else none3,
                         append_indptr.data_ptr(), kv_indptr.data_ptr(), _index_ptr(kv_indices),
                         _index_ptr(kv_last_page_len), None if positions is None else positions.data_ptr(), batch, rows,
                         pages, k_cache.shape[1], hk, dim, desc, None if q is None else q.data_ptr(),
                         None if q is None else q_out.data_ptr(), (0, 0) if q is None else q.stride()[:2],
                         (0, 0) if q is None else q_out.stride()[:2], 0 if q is None else q.shape[1],
                         None if status is None else status.data_ptr())
        _check(_kv_append(ctypes.byref(p), _stream(stream, dev)), "skv_paged_kv_append")
    del keep
    return q_out


def _dev_i32(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(dev)


def paged_attention_scaled(q, k_cache, v_cache, k_scale, v_scale, qo_indptr_h, kv_indptr_h, kv_indices,
                           kv_last_page_len_h, *, sm_scale: Optional[float] = None, causal: bool = False,
                           policy="balanced", param: int = 0, split_page_start=None, o_dtype=None,
                           num_pages: Optional[int] = None, kv_indptr=None, kv_last_page_len=None,
                           plan: Optional[Plan] = None, status=None, stream=None, o_out=None, lse_out=None):
    """GQA attention over a paged 8-bit cache with block scales (skv_paged_attn_scaled_fwd): q [total_q, Hq, D]
    bf16, caches [num_pages, P, Hk, D] float8_e4m3fn or int8, ``k_scale`` / ``v_scale`` float32
    [num_pages, P / block, Hk], as ``paged_kv_append`` writes them.  ``causal``: a request's query tokens are
    its last positions and each sees keys up to its own.  Host page-table shape arrays (``*_h``) feed
    the planner; ``plan`` (``plan_paged_scaled`` with the same ``causal``) and device copies ``kv_indptr`` /
    ``kv_last_page_len`` may be kept over the layers of a step.
    Returns (o, lse, extras) with extras = {"plan", "o_part", "lse_part"}."""
    import torch
    _need(q.dim() == 3 and k_cache.dim() == 4, "q is [total_q, Hq, D], the caches [num_pages, P, Hk, D]")
    dev, total_q, hq, dim = q.device, q.shape[0], q.shape[1], q.shape[2]
    hk, page = k_cache.shape[2], k_cache.shape[1]
    code = _cache_code(k_cache.dtype)
    _need(q.dtype == torch.bfloat16 and q.is_contiguous(), "q must be contiguous bfloat16")
    _need(code in (E4M3, I8) and v_cache.dtype == k_cache.dtype, "caches must both be float8_e4m3fn or int8")
    _need(v_cache.shape == k_cache.shape and k_cache.shape[3] == dim and k_cache.stride(3) == 1
          and v_cache.stride(3) == 1, "the caches must be [num_pages, P, Hk, D] with the head_dim of q")
    _need(len(qo_indptr_h) > 0 and total_q >= int(qo_indptr_h[-1]), "q has fewer rows than qo_indptr names")
    pages = k_cache.shape[0] if num_pages is None else num_pages
    _need(0 <= pages <= k_cache.shape[0], "num_pages is more than the cache holds")
    block = _scales(k_cache, k_scale, v_scale, pages)
    batch = len(qo_indptr_h) - 1
    _on(dev, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, kv_indices=kv_indices,
        kv_indptr=kv_indptr, kv_last_page_len=kv_last_page_len, status=status, o_out=o_out, lse_out=lse_out)
    _index("kv_indices", kv_indices)
    _index("kv_indptr", kv_indptr, batch + 1)
    _index("kv_last_page_len", kv_last_page_len, batch)
    for name, t, shape in (("o_out", o_out, (total_q, hq, dim)), ("lse_out", lse_out, (total_q, hq))):
        _need(t is None or (tuple(t.shape) == shape and t.is_contiguous()), f"{name} must be contiguous {shape}")
    _need(lse_out is None or lse_out.dtype == torch.float32, "lse_out must be float32")
    out_dtype = o_out.dtype if o_out is not None else (o_dtype or torch.float32)
    _need(out_dtype in (torch.float32, torch.bfloat16), "outputs are float32 or bfloat16")
    with _device(dev), _on_stream(stream, dev):
        if plan is None:
            plan = plan_paged_scaled(qo_indptr_h, kv_indptr_h, kv_last_page_len_h, page, hq, hk, dim, causal, policy,
                                     param, split_page_start)
        if plan.device is None:
            plan.to(dev)
        if kv_indptr is None:
            kv_indptr = _dev_i32(kv_indptr_h, dev)
        if kv_last_page_len is None:
            kv_last_page_len = _dev_i32(kv_last_page_len_h, dev)
        o = torch.empty(total_q, hq, dim, dtype=out_dtype, device=dev) if o_out is None else o_out
        lse = torch.empty(total_q, hq, dtype=torch.float32, device=dev) if lse_out is None else lse_out
        n_part = plan.info.num_partial_rows
        o_part = torch.empty(n_part, hq, dim, dtype=torch.float32, device=dev) if n_part else None
        lse_part = torch.empty(n_part, hq, dtype=torch.float32, device=dev) if n_part else None
        base = PagedParams(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_cache.stride()[:3],
                           v_cache.stride()[:3], kv_indptr.data_ptr(), _index_ptr(kv_indices),
                           _index_ptr(kv_last_page_len), batch, total_q, pages, page, hq, hk, dim,
                           dim ** -0.5 if sm_scale is None else sm_scale, o.data_ptr(),
                           BF16 if out_dtype == torch.bfloat16 else F32, lse.data_ptr(),
                           o_part.data_ptr() if n_part else None, lse_part.data_ptr() if n_part else None,
                           None if status is None else status.data_ptr(), code, 1.0)
        p = PagedScaledParams(base, k_scale.data_ptr(), v_scale.data_ptr(), k_scale.stride(), v_scale.stride(), block)
        _check(_scaled_fwd(ctypes.byref(p), plan.device.data_ptr(), ctypes.byref(plan.info), _stream(stream, dev)),
               "skv_paged_attn_scaled_fwd")
    return o, lse, {"plan": plan, "o_part": o_part, "lse_part": lse_part}


def prompt_attention(q, k, v, qo_indptr_h, kv_indptr_h=None, *, causal: bool = True, sm_scale: Optional[float] = None,
                     o_dtype=None, plan: Optional[Plan] = None, status=None, stream=None, o_out=None, lse_out=None):
    """Attention over packed prompts (skv_prompt_attn_fwd): q [total_q, Hq, D], k, v [total_kv, Hk, D] bf16, any
    token / head strides; sequence r has query rows qo_indptr_h[r] .. and key rows kv_indptr_h[r] ..
    (default: the same rows).  ``causal``: its query tokens are its last positions.  ``plan``
    (``plan_prompt`` with the same ``causal``) may be kept over the layers of a step.  Rows of outputs given as
    ``o_out`` / ``lse_out`` behind the last sequence are left as they are.
    Returns (o, lse, extras) with extras = {"plan", "o_part", "lse_part"}."""
    import torch
    _need(q.dim() == 3 and k.dim() == 3, "q is [total_q, Hq, D], k and v are [total_kv, Hk, D]")
    dev, total_q, hq, dim = q.device, q.shape[0], q.shape[1], q.shape[2]
    total_kv, hk = k.shape[0], k.shape[1]
    _need(q.dtype == torch.bfloat16 and k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16,
          "q, k and v must be bfloat16")
    _rows3("q", q, total_q, dim)
    _rows3("k", k, total_kv, dim)
    _rows3("v", v, total_kv, dim)
    _need(v.shape[1] == hk, "k and v must have the same heads")
    _on(dev, k=k, v=v, status=status, o_out=o_out, lse_out=lse_out)
    _need(len(qo_indptr_h) > 0 and total_q >= int(qo_indptr_h[-1]), "q has fewer rows than qo_indptr names")
    _need(total_kv >= int((qo_indptr_h if kv_indptr_h is None else kv_indptr_h)[-1]),
          "k and v have fewer rows than kv_indptr names")
    for name, t, shape in (("o_out", o_out, (total_q, hq, dim)), ("lse_out", lse_out, (total_q, hq))):
        _need(t is None or (tuple(t.shape) == shape and t.is_contiguous()), f"{name} must be contiguous {shape}")
    _need(lse_out is None or lse_out.dtype == torch.float32, "lse_out must be float32")
    out_dtype = o_out.dtype if o_out is not None else (o_dtype or torch.float32)
    _need(out_dtype in (torch.float32, torch.bfloat16), "outputs are float32 or bfloat16")
    with _device(dev), _on_stream(stream, dev):
        if plan is None:
            plan = plan_prompt(qo_indptr_h, kv_indptr_h, hq, hk, dim, causal)
        if plan.device is None:
            plan.to(dev)
        o = torch.empty(total_q, hq, dim, dtype=out_dtype, device=dev) if o_out is None else o_out
        lse = torch.empty(total_q, hq, dtype=torch.float32, device=dev) if lse_out is None else lse_out
        n_part = plan.info.num_partial_rows
        o_part = torch.empty(n_part, hq, dim, dtype=torch.float32, device=dev) if n_part else None
        lse_part = torch.empty(n_part, hq, dtype=torch.float32, device=dev) if n_part else None
        p = PromptParams(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride()[:2], k.stride()[:2], v.stride()[:2], total_q,
                         total_kv, hq, hk, dim, dim ** -0.5 if sm_scale is None else sm_scale, o.data_ptr(),
                         BF16 if out_dtype == torch.bfloat16 else F32, lse.data_ptr(),
                         o_part.data_ptr() if n_part else None, lse_part.data_ptr() if n_part else None,
                         None if status is None else status.data_ptr())
        _check(_prompt_fwd(ctypes.byref(p), plan.device.data_ptr(), ctypes.byref(plan.info), _stream(stream, dev)),
               "skv_prompt_attn_fwd")
    return o, lse, {"plan": plan, "o_part": o_part, "lse_part": lse_part}
