"""Serving operators around the paged attention calls: rotary positions, the cache append, attention
over a block-scaled 8-bit cache and over packed prompts.

The signatures and what they mean stand here; arguments are checked, outputs allocated and the C ABI
called by the extension module built from ``csrc/binding.cpp``.  It needs torch and is loaded by the
first call; planning and ``rope_frequencies`` do without.

The calls record nothing for autograd: their results have no history, whatever their inputs require.  Tensors
that they write in place count as modified."""
from __future__ import annotations

import ctypes
from typing import Optional

import numpy as np

from . import (BF16, F32, Plan, SkvError, _check, _ROPE, _ROPE_SCALING, _rope_frequencies, plan_paged_scaled, plan_prompt,
               prompt_key, scaled_key)

_ext = None
_O_CODE = {}


def _load():
    """The extension module (on the first call)."""
    global _ext
    import torch

    try:
        from . import _serving
    except ImportError as e:
        raise ImportError(f"the serving operators' extension is not there (run split_kv_merge_b200/build.py where torch "
                          f"is installed): {e}") from e
    _O_CODE.update({None: F32, torch.float32: F32, torch.bfloat16: BF16})
    _serving.set_error(SkvError)
    _ext = _serving
    return _ext


def _bad(what: str):
    raise ValueError(what)


def _on_stream(stream, tensor):
    """Context in which a call runs on ``stream`` and allocates from it (so that its memory is not handed out
    again before the stream's work is done)."""
    import torch
    dev = tensor.device
    if dev.type != "cuda":
        _bad("tensors must be on a CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != dev:
        _bad(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _layout(rope_layout: str) -> int:
    code = _ROPE.get(rope_layout)
    if code is None:
        _bad(f"rope_layout must be one of {sorted(_ROPE)}")
    return code


def _frequencies(inv_freq):
    return None if inv_freq is None else np.ascontiguousarray(inv_freq, dtype=np.float64)


def rope_frequencies(rope_dim: int, rope_theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_context: float = 8192, low: Optional[float] = None, high: Optional[float] = None):
    """skv_rope_frequencies: (inv_freq float64 [rope_dim / 2], mscale) of the base ``rope_theta``, stretched
    for long contexts by ``scaling``: "linear" (positions divided by ``factor``), "ntk" (a larger base),
    "yarn" or "bands" (pairs that turn fewer than ``low`` times in ``original_context`` positions are
    stretched, those that turn more than ``high`` times kept, a ramp between; 1 and 32 by default for
    "yarn", which also gives an mscale, 1 and 4 for "bands").  Pass both on to ``rope_apply`` or
    ``paged_kv_append``."""
    if scaling not in _ROPE_SCALING:
        _bad(f"scaling must be one of {sorted(_ROPE_SCALING)}")
    lo = 1.0 if low is None else low
    hi = (4.0 if scaling == "bands" else 32.0) if high is None else high
    f, m = np.zeros(max(0, rope_dim // 2)), ctypes.c_float(1.0)
    _check(_rope_frequencies(rope_dim, rope_theta, _ROPE_SCALING[scaling], factor, original_context, lo, hi,
                             f.ctypes.data, ctypes.byref(m)), "skv_rope_frequencies")
    return f, float(m.value)


def rope_apply(q, k, positions, *, rope_dim: Optional[int] = None, rope_theta: float = 10000.0,
               rope_layout: str = "interleaved", inv_freq=None, mscale: float = 1.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None):
    """skv_rope_apply: rotary positions of q [tokens, Hq, D] and k [tokens, Hk, D] (either may be None; bf16
    or float32, any token / head strides), ``positions`` int32 [tokens] on the device.  The first
    ``rope_dim`` (default D) values of a head turn, the others are copied.  ``inv_freq`` (float64, host)
    replaces rope_theta^(-2p/rope_dim).  ``q_out=q`` / ``k_out=k`` rotates in place; ``inverse`` turns
    back, and is the rotation's transpose for any ``mscale``: what the backward method of a caller's own
    autograd function applies to the gradient.  Returns (q_out, k_out)."""
    if stream is not None:
        with _on_stream(stream, positions):
            return rope_apply(q, k, positions, rope_dim=rope_dim, rope_theta=rope_theta, rope_layout=rope_layout,
                              inv_freq=inv_freq, mscale=mscale, inverse=inverse, q_out=q_out, k_out=k_out)
    return (_ext or _load()).rope_apply(q, k, positions, rope_dim, rope_theta, _layout(rope_layout),
                                        _frequencies(inv_freq), mscale, inverse, q_out, k_out)


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
    if stream is not None:
        with _on_stream(stream, k):
            return paged_kv_append(k, v, k_cache, v_cache, append_indptr, kv_indptr, kv_indices, kv_last_page_len,
                                   k_scale=k_scale, v_scale=v_scale, kv_scale=kv_scale, q=q, q_out=q_out,
                                   positions=positions, rope_dim=rope_dim, rope_theta=rope_theta,
                                   rope_layout=rope_layout, inv_freq=inv_freq, mscale=mscale, num_pages=num_pages,
                                   status=status)
    return (_ext or _load()).paged_kv_append(k, v, k_cache, v_cache, append_indptr, kv_indptr, kv_indices,
                                             kv_last_page_len, k_scale, v_scale, kv_scale, q, q_out, positions,
                                             rope_dim, rope_theta, _layout(rope_layout), _frequencies(inv_freq), mscale,
                                             num_pages, status)


def _o_code(o_dtype) -> int:
    code = _O_CODE.get(o_dtype)
    if code is None:
        _bad("outputs are float32 or bfloat16")
    return code


def _same(plan: Plan, made_for: tuple):
    if plan.made_for is not None and plan.made_for != made_for:
        _bad("the plan was made for other requests: their lengths, heads, page size and causal must be the call's")


def _dev_i32(a, like):
    import torch
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(like.device)


def paged_attention_scaled(q, k_cache, v_cache, k_scale, v_scale, qo_indptr_h, kv_indptr_h, kv_indices,
                           kv_last_page_len_h, *, sm_scale: Optional[float] = None, causal: bool = False,
                           policy="balanced", param: int = 0, split_page_start=None, o_dtype=None,
                           num_pages: Optional[int] = None, kv_indptr=None, kv_last_page_len=None,
                           plan: Optional[Plan] = None, status=None, stream=None, o_out=None, lse_out=None):
    """GQA attention over a paged 8-bit cache with block scales (skv_paged_attn_scaled_fwd): q [total_q, Hq, D]
    bf16, caches [num_pages, P, Hk, D] float8_e4m3fn or int8, ``k_scale`` / ``v_scale`` float32
    [num_pages, P / block, Hk], as ``paged_kv_append`` writes them.  ``causal``: a request's query tokens are
    its last positions and each sees keys up to its own.  Host page-table shape arrays (``*_h``) feed
    the planner; ``plan`` (``plan_paged_scaled`` of the same lengths, heads and ``causal``, which are compared; without
    ``causal`` the last pages may have filled since) and device copies ``kv_indptr`` / ``kv_last_page_len`` may be
    kept over the layers of a step.
    Returns (o, lse, extras) with extras = {"plan", "workspace"} (the split partials' buffer)."""
    if stream is not None:
        with _on_stream(stream, q):
            return paged_attention_scaled(q, k_cache, v_cache, k_scale, v_scale, qo_indptr_h, kv_indptr_h, kv_indices,
                                          kv_last_page_len_h, sm_scale=sm_scale, causal=causal, policy=policy,
                                          param=param, split_page_start=split_page_start, o_dtype=o_dtype,
                                          num_pages=num_pages, kv_indptr=kv_indptr, kv_last_page_len=kv_last_page_len,
                                          plan=plan, status=status, o_out=o_out, lse_out=lse_out)
    ext = _ext or _load()
    if q.dim() != 3 or k_cache.dim() != 4 or q.shape[0] < qo_indptr_h[-1]:
        _bad("q is [total_q, Hq, D] with the rows qo_indptr names, the caches are [num_pages, P, Hk, D]")
    if plan is None:
        plan = plan_paged_scaled(qo_indptr_h, kv_indptr_h, kv_last_page_len_h, k_cache.shape[1], q.shape[1],
                                 k_cache.shape[2], q.shape[2], causal, policy, param, split_page_start)
    else:
        _same(plan, scaled_key(qo_indptr_h, kv_indptr_h, kv_last_page_len_h, causal, k_cache.shape[1], q.shape[1],
                               k_cache.shape[2], q.shape[2]))
    if kv_indices is None or kv_indices.numel() < kv_indptr_h[-1]:
        _bad("kv_indices must hold every page id that kv_indptr names")
    if plan.device is None:
        plan.to(q.device)
    if kv_indptr is None:
        kv_indptr = _dev_i32(kv_indptr_h, q)
    if kv_last_page_len is None:
        kv_last_page_len = _dev_i32(kv_last_page_len_h, q)
    if kv_indptr.numel() != len(qo_indptr_h):
        _bad("qo_indptr and kv_indptr must name the same requests")
    o, lse, ws = ext.paged_attention_scaled(q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                                            kv_last_page_len, plan.device, ctypes.addressof(plan.info), sm_scale,
                                            _o_code(o_dtype), o_out, lse_out, num_pages, status)
    return o, lse, {"plan": plan, "workspace": ws}


def prompt_attention(q, k, v, qo_indptr_h, kv_indptr_h=None, *, causal: bool = True, sm_scale: Optional[float] = None,
                     o_dtype=None, plan: Optional[Plan] = None, status=None, stream=None, o_out=None, lse_out=None):
    """Attention over packed prompts (skv_prompt_attn_fwd): q [total_q, Hq, D], k, v [total_kv, Hk, D] bf16, any
    token / head strides; sequence r has query rows qo_indptr_h[r] .. and key rows kv_indptr_h[r] ..
    (default: the same rows).  ``causal``: its query tokens are its last positions.  ``plan``
    (``plan_prompt`` of the same lengths, heads and ``causal``, which are compared) may be kept over the layers of
    a step.  Rows of outputs given as ``o_out`` / ``lse_out`` behind the last sequence are left as they are.
    Returns (o, lse, extras) with extras = {"plan", "workspace"} (the partials' buffer)."""
    if stream is not None:
        with _on_stream(stream, q):
            return prompt_attention(q, k, v, qo_indptr_h, kv_indptr_h, causal=causal, sm_scale=sm_scale,
                                    o_dtype=o_dtype, plan=plan, status=status, o_out=o_out, lse_out=lse_out)
    ext = _ext or _load()
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] < qo_indptr_h[-1] or \
            k.shape[0] < (qo_indptr_h if kv_indptr_h is None else kv_indptr_h)[-1]:
        _bad("q is [total_q, Hq, D], k and v are [total_kv, Hk, D] with the rows qo_indptr and kv_indptr name")
    if plan is None:
        plan = plan_prompt(qo_indptr_h, kv_indptr_h, q.shape[1], k.shape[1], q.shape[2], causal)
    else:
        _same(plan, prompt_key(qo_indptr_h, kv_indptr_h, causal, q.shape[1], k.shape[1], q.shape[2]))
    if plan.device is None:
        plan.to(q.device)
    o, lse, ws = ext.prompt_attention(q, k, v, plan.device, ctypes.addressof(plan.info), sm_scale, _o_code(o_dtype),
                                      o_out, lse_out, status)
    return o, lse, {"plan": plan, "workspace": ws}
