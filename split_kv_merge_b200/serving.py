"""Serving operators around the paged attention calls: rotary positions, the cache append, attention
over a block-scaled 8-bit cache and over packed prompts.  Argument checks and marshalling; the work runs
in the library's kernels.

A call costs the host about as much as the smallest kernels run, so parameter blocks are packed with
``struct`` (layouts taken from the ctypes structures) and tensor properties are read once."""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import numpy as np

from . import (AppendParams, BF16, E4M3, F32, I8, PagedScaledParams, Plan, PromptParams, RopeParams, SkvError,
               _check, _index_ptr, _lib, _ROPE, _ROPE_SCALING, _rope_frequencies, plan_paged_scaled, plan_prompt)


def _packer(cls) -> struct.Struct:
    """``struct`` layout of a ctypes structure, its fields (nested ones and arrays too) in order."""
    fmt, at = ["="], 0
    code = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_double: "d", ctypes.c_void_p: "Q"}

    def walk(c, base):
        nonlocal at
        for name, kind in c._fields_:
            offset = base + getattr(c, name).offset
            if isinstance(kind, type) and issubclass(kind, ctypes.Structure):
                walk(kind, offset)
                continue
            n, item = (kind._length_, kind._type_) if isinstance(kind, type) and issubclass(kind, ctypes.Array) else (1, kind)
            fmt.append(f"{offset - at}x{n}{code[item]}")
            at = offset + n * ctypes.sizeof(item)

    walk(cls, 0)
    fmt.append(f"{ctypes.sizeof(cls) - at}x")
    return struct.Struct("".join(fmt))


_pack_rope, _pack_append = _packer(RopeParams).pack, _packer(AppendParams).pack
_pack_scaled, _pack_prompt = _packer(PagedScaledParams).pack, _packer(PromptParams).pack


def _entry(name: str, args: int):
    """The C function taking ``args`` addresses (a second prototype beside the binding's own)."""
    return ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * args)((name, _lib))


_addressof, _char = ctypes.addressof, ctypes.c_char
_call_rope, _call_append = _entry("skv_rope_apply", 2), _entry("skv_paged_kv_append", 2)
_call_scaled, _call_prompt = _entry("skv_paged_attn_scaled_fwd", 4), _entry("skv_prompt_attn_fwd", 4)

torch = _bf16 = _f32 = _i32 = _cache_codes = _raw_stream = _cuda_device = _contiguous = None


def _init() -> None:
    """Imports torch on the first call (planning alone needs numpy only)."""
    global torch, _bf16, _f32, _i32, _cache_codes, _raw_stream, _cuda_device, _contiguous
    import torch as t
    _bf16, _f32, _i32, _contiguous = t.bfloat16, t.float32, t.int32, t.contiguous_format
    _cache_codes = {t.bfloat16: BF16, t.float8_e4m3fn: E4M3, t.uint8: E4M3, t.int8: I8}
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or \
        (lambda i: t.cuda.current_stream(i).cuda_stream)
    _cuda_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t


def _bad(what: str):
    raise ValueError(what)


def _device_index(t) -> int:
    i = t.get_device()
    if i < 0:
        _bad("tensors must be on a CUDA device")
    return i


def _index(name: str, t, n: int, dev: int) -> int:
    """Address of a contiguous int32 vector of n entries (n < 0: any) on the device."""
    if t.dtype is not _i32 or t.dim() != 1 or (n >= 0 and t.numel() != n) or not t.is_contiguous():
        _bad(f"{name} must be a contiguous int32 vector" + ("" if n < 0 else f" of {n} entries"))
    if t.get_device() != dev:
        _bad(f"{name} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr() or _index_ptr(t)


def _rows(name: str, t, dtype, rows: int, dim: int, dev: int):
    """(heads, address, token stride, head stride) of a [rows, heads, dim] tensor."""
    try:
        n, heads, d = t.shape
    except ValueError:
        n = heads = d = -1
    if n != rows or d != dim or t.dtype is not dtype or t.get_device() != dev:
        _bad(f"{name} must be a {dtype} tensor [{rows}, heads, {dim}] on cuda:{dev}, got {t.dtype} {tuple(t.shape)} "
             f"on {t.device}")
    s0, s1, s2 = t.stride()
    if s2 != 1 and n * heads * d:
        _bad(f"{name} must have contiguous heads")
    return heads, t.data_ptr(), s0, s1


def _like(t, heads: int):
    """A new tensor of t's shape and dtype, and its (heads, address, token stride, head stride)."""
    out = torch.empty_like(t, memory_format=_contiguous)
    d = t.shape[2]
    return out, (heads, out.data_ptr(), heads * d, d)


class _Launch:
    """Makes the tensors' device current for a call, and a given stream current for its allocations (so
    that their memory is not handed out again before the stream's work is done)."""
    __slots__ = ("contexts",)

    def __init__(self, dev: int, stream):
        self.contexts = []
        if _cuda_device() != dev:
            self.contexts.append(torch.cuda.device(dev))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = int(getattr(stream, "cuda_stream", stream))
                stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
            if stream.device.index != dev:
                _bad(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _elsewhere(dev: int, stream) -> bool:
    return stream is not None or _cuda_device() != dev


def _freqs(rope_dim: int, rope_layout: str, inv_freq):
    """(layout code, address of the frequencies or 0, the array to keep until the call returns)."""
    layout = _ROPE.get(rope_layout)
    if layout is None:
        _bad(f"rope_layout must be one of {sorted(_ROPE)}")
    if inv_freq is None or rope_dim <= 0:
        return layout, 0, None
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.ndim != 1 or 2 * f.size != rope_dim:
        _bad(f"inv_freq must hold rope_dim / 2 = {rope_dim // 2} frequencies")
    if f.flags.writeable:  # the address, by the quicker way where the array allows it
        return layout, _addressof(_char.from_buffer(f)), f
    return layout, f.__array_interface__["data"][0], f


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


_NO_ROWS = (0, 0, 0, 0)


def rope_apply(q, k, positions, *, rope_dim: Optional[int] = None, rope_theta: float = 10000.0,
               rope_layout: str = "interleaved", inv_freq=None, mscale: float = 1.0, inverse: bool = False,
               q_out=None, k_out=None, stream=None):
    """skv_rope_apply: rotary positions of q [tokens, Hq, D] and k [tokens, Hk, D] (either may be None; bf16
    or float32, any token / head strides), ``positions`` int32 [tokens] on the device.  The first
    ``rope_dim`` (default D) values of a head turn, the others are copied.  ``inv_freq`` (float64, host)
    replaces rope_theta^(-2p/rope_dim).  ``q_out=q`` / ``k_out=k`` rotates in place; ``inverse`` turns
    back (and takes gradients through the rotation).  Returns (q_out, k_out)."""
    if torch is None:
        _init()
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        _bad("q or k is needed, [tokens, heads, head_dim]")
    dtype = x.dtype
    if dtype is not _bf16 and dtype is not _f32:
        _bad("q and k must be bfloat16 or float32")
    dev = _device_index(x)
    if _elsewhere(dev, stream):
        with _Launch(dev, stream):
            return rope_apply(q, k, positions, rope_dim=rope_dim, rope_theta=rope_theta, rope_layout=rope_layout,
                              inv_freq=inv_freq, mscale=mscale, inverse=inverse, q_out=q_out, k_out=k_out)
    tokens, _, dim = x.shape
    at = _index("positions", positions, tokens, dev)
    hq = hk = 0
    qi = qo = ki = ko = _NO_ROWS
    if q is not None:
        qi = _rows("q", q, dtype, tokens, dim, dev)
        hq = qi[0]
        if q_out is None:
            q_out, qo = _like(q, hq)
        else:
            qo = _rows("q_out", q_out, dtype, tokens, dim, dev)
    if k is not None:
        ki = _rows("k", k, dtype, tokens, dim, dev)
        hk = ki[0]
        if k_out is None:
            k_out, ko = _like(k, hk)
        else:
            ko = _rows("k_out", k_out, dtype, tokens, dim, dev)
    if qo[0] != hq or ko[0] != hk or (q is None and q_out is not None) or (k is None and k_out is not None):
        _bad("q_out and k_out must have the shapes of q and k")
    rope_dim = dim if rope_dim is None else rope_dim
    layout, freq, keep = _freqs(rope_dim, rope_layout, inv_freq)
    code = _call_rope(_pack_rope(qi[1], qo[1], ki[1], ko[1], qi[2], qi[3], qo[2], qo[3], ki[2], ki[3], ko[2], ko[3], at,
                                 tokens, hq, hk, dim, F32 if dtype is _f32 else BF16, 1 if inverse else 0, rope_dim,
                                 layout, rope_theta, freq, mscale), _raw_stream(dev))
    if code:
        raise SkvError(code, "skv_rope_apply")
    return q_out, k_out


def _caches(k_cache, v_cache, dim: int, num_pages, dev: int):
    """(dtype code, pages, page size, Hk, page / slot / head strides of K and V) of a pair of caches."""
    code = _cache_codes.get(k_cache.dtype)
    if code is None or v_cache.dtype is not k_cache.dtype:
        _bad("caches must both be bfloat16, float8_e4m3fn or int8")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        _bad("the caches must both be [num_pages, P, Hk, D]")
    held, page, hk, d = shape
    ks, vs = k_cache.stride(), v_cache.stride()
    if d != dim or ks[3] != 1 or vs[3] != 1:
        _bad(f"the caches must be [num_pages, P, Hk, {dim}] with contiguous heads")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        _bad(f"the caches must be on cuda:{dev}")
    pages = held if num_pages is None else num_pages
    if not 0 <= pages <= held:
        _bad("num_pages is more than the cache holds")
    return code, pages, page, hk, ks, vs


def _scales(k_scale, v_scale, pages: int, page: int, hk: int, dev: int) -> int:
    """Tokens that share a scale in the scale tensors [num_pages, blocks per page, Hk] float32."""
    if k_scale is None or v_scale is None:
        _bad("k_scale and v_scale come together")
    shape = k_scale.shape
    if len(shape) != 3 or v_scale.shape != shape or k_scale.dtype is not _f32 or v_scale.dtype is not _f32 \
            or k_scale.get_device() != dev or v_scale.get_device() != dev:
        _bad(f"k_scale and v_scale must be float32 [num_pages, blocks per page, {hk}] on cuda:{dev}")
    n, blocks, heads = shape
    if n < pages or heads != hk or blocks < 1 or page % blocks:
        _bad(f"k_scale and v_scale must be float32 [num_pages, blocks per page, {hk}] with whole blocks of tokens")
    return page // blocks


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
    if torch is None:
        _init()
    if k.dim() != 3:
        _bad("k and v are [rows, Hk, D]")
    dev = _device_index(k)
    if _elsewhere(dev, stream):
        with _Launch(dev, stream):
            return paged_kv_append(k, v, k_cache, v_cache, append_indptr, kv_indptr, kv_indices, kv_last_page_len,
                                   k_scale=k_scale, v_scale=v_scale, kv_scale=kv_scale, q=q, q_out=q_out,
                                   positions=positions, rope_dim=rope_dim, rope_theta=rope_theta,
                                   rope_layout=rope_layout, inv_freq=inv_freq, mscale=mscale, num_pages=num_pages,
                                   status=status)
    rows, _, dim = k.shape
    ki, vi = _rows("k", k, _bf16, rows, dim, dev), _rows("v", v, _bf16, rows, dim, dev)
    code, pages, page, hk, ks, vs = _caches(k_cache, v_cache, dim, num_pages, dev)
    if ki[0] != hk or vi[0] != hk:
        _bad(f"k, v and the caches must have the same heads, got {ki[0]}, {vi[0]} and {hk}")
    batch = append_indptr.numel() - 1
    if batch < 0:
        _bad("append_indptr must be a contiguous int32 vector")
    block, kp, vp, kss, vss = 0, 0, 0, _NO_ROWS, _NO_ROWS
    if k_scale is not None or v_scale is not None:
        block = _scales(k_scale, v_scale, pages, page, hk, dev)
        kp, vp, kss, vss = k_scale.data_ptr(), v_scale.data_ptr(), k_scale.stride(), v_scale.stride()
    qi = qo = _NO_ROWS
    if q is not None:
        qi = _rows("q", q, _bf16, rows, dim, dev)
        if q_out is None:
            q_out, qo = _like(q, qi[0])
        else:
            qo = _rows("q_out", q_out, _bf16, rows, dim, dev)
    if qo[0] != qi[0] or (q is None and q_out is not None):
        _bad("q_out must have the shape of q")
    layout, freq, keep = _freqs(rope_dim, rope_layout, inv_freq)
    ret = _call_append(_pack_append(
        ki[1], vi[1], ki[2], ki[3], vi[2], vi[3], k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0],
        vs[1], vs[2], code, kv_scale, block, kp, vp, kss[0], kss[1], kss[2], vss[0], vss[1], vss[2],
        _index("append_indptr", append_indptr, batch + 1, dev), _index("kv_indptr", kv_indptr, batch + 1, dev),
        _index("kv_indices", kv_indices, -1, dev), _index("kv_last_page_len", kv_last_page_len, batch, dev),
        0 if positions is None else _index("positions", positions, rows, dev), batch, rows, pages, page, hk, dim,
        rope_dim, layout, rope_theta, freq, mscale, qi[1], qo[1], qi[2], qi[3], qo[2], qo[3], qi[0],
        0 if status is None else _index("status", status, -1, dev)), _raw_stream(dev))
    if ret:
        raise SkvError(ret, "skv_paged_kv_append")
    return q_out


def _outputs(q, total_q: int, hq: int, dim: int, o_dtype, o_out, lse_out, dev: int):
    """(o, its dtype code, lse), allocated unless given."""
    if o_out is None:
        dtype = o_dtype or _f32
        if dtype is _bf16:
            o = torch.empty_like(q, memory_format=_contiguous)
        else:
            o = q.new_empty((total_q, hq, dim), dtype=dtype)
    else:
        o, dtype = o_out, o_out.dtype
        if tuple(o.shape) != (total_q, hq, dim) or not o.is_contiguous() or o.get_device() != dev:
            _bad(f"o_out must be contiguous [{total_q}, {hq}, {dim}] on cuda:{dev}")
    if dtype is not _f32 and dtype is not _bf16:
        _bad("outputs are float32 or bfloat16")
    if lse_out is None:
        lse = q.new_empty((total_q, hq), dtype=_f32)
    else:
        lse = lse_out
        if tuple(lse.shape) != (total_q, hq) or not lse.is_contiguous() or lse.get_device() != dev or lse.dtype is not _f32:
            _bad(f"lse_out must be contiguous float32 [{total_q}, {hq}] on cuda:{dev}")
    return o, BF16 if dtype is _bf16 else F32, lse


def _workspace(q, plan: Plan, hq: int, dim: int):
    """(buffer for the plan's split partials, addresses of o_part and lse_part in it)."""
    n = plan.info.num_partial_rows
    if n == 0:
        return None, 0, 0
    ws = q.new_empty(n * hq * (dim + 1), dtype=_f32)
    return ws, ws.data_ptr(), ws.data_ptr() + 4 * n * hq * dim


def _dev_i32(a, like):
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
    the planner; ``plan`` (``plan_paged_scaled`` with the same ``causal``) and device copies ``kv_indptr`` /
    ``kv_last_page_len`` may be kept over the layers of a step.
    Returns (o, lse, extras) with extras = {"plan", "workspace"} (the split partials' buffer)."""
    if torch is None:
        _init()
    if q.dim() != 3:
        _bad("q is [total_q, Hq, D]")
    dev = _device_index(q)
    if _elsewhere(dev, stream):
        with _Launch(dev, stream):
            return paged_attention_scaled(q, k_cache, v_cache, k_scale, v_scale, qo_indptr_h, kv_indptr_h, kv_indices,
                                          kv_last_page_len_h, sm_scale=sm_scale, causal=causal, policy=policy,
                                          param=param, split_page_start=split_page_start, o_dtype=o_dtype,
                                          num_pages=num_pages, kv_indptr=kv_indptr, kv_last_page_len=kv_last_page_len,
                                          plan=plan, status=status, o_out=o_out, lse_out=lse_out)
    total_q, hq, dim = q.shape
    if q.dtype is not _bf16 or not q.is_contiguous():
        _bad("q must be contiguous bfloat16")
    code, pages, page, hk, ks, vs = _caches(k_cache, v_cache, dim, num_pages, dev)
    if code == BF16:
        _bad("caches must both be float8_e4m3fn or int8")
    block = _scales(k_scale, v_scale, pages, page, hk, dev)
    batch = len(qo_indptr_h) - 1
    if batch < 0 or total_q < qo_indptr_h[batch]:
        _bad("q has fewer rows than qo_indptr names")
    if plan is None:
        plan = plan_paged_scaled(qo_indptr_h, kv_indptr_h, kv_last_page_len_h, page, hq, hk, dim, causal, policy, param,
                                 split_page_start)
    if plan.device is None:
        plan.to(q.device)
    if kv_indptr is None:
        kv_indptr = _dev_i32(kv_indptr_h, q)
    if kv_last_page_len is None:
        kv_last_page_len = _dev_i32(kv_last_page_len_h, q)
    o, o_code, lse = _outputs(q, total_q, hq, dim, o_dtype, o_out, lse_out, dev)
    ws, o_part, lse_part = _workspace(q, plan, hq, dim)
    kss, vss = k_scale.stride(), v_scale.stride()
    ret = _call_scaled(_pack_scaled(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
        _index("kv_indptr", kv_indptr, batch + 1, dev), _index("kv_indices", kv_indices, -1, dev),
        _index("kv_last_page_len", kv_last_page_len, batch, dev), batch, total_q, pages, page, hq, hk, dim,
        dim ** -0.5 if sm_scale is None else sm_scale, o.data_ptr(), o_code, lse.data_ptr(), o_part, lse_part,
        0 if status is None else _index("status", status, -1, dev), code, 1.0, k_scale.data_ptr(), v_scale.data_ptr(),
        kss[0], kss[1], kss[2], vss[0], vss[1], vss[2], block), _index("plan", plan.device, -1, dev),
        ctypes.addressof(plan.info), _raw_stream(dev))
    if ret:
        raise SkvError(ret, "skv_paged_attn_scaled_fwd")
    return o, lse, {"plan": plan, "workspace": ws}


def prompt_attention(q, k, v, qo_indptr_h, kv_indptr_h=None, *, causal: bool = True, sm_scale: Optional[float] = None,
                     o_dtype=None, plan: Optional[Plan] = None, status=None, stream=None, o_out=None, lse_out=None):
    """Attention over packed prompts (skv_prompt_attn_fwd): q [total_q, Hq, D], k, v [total_kv, Hk, D] bf16, any
    token / head strides; sequence r has query rows qo_indptr_h[r] .. and key rows kv_indptr_h[r] ..
    (default: the same rows).  ``causal``: its query tokens are its last positions.  ``plan``
    (``plan_prompt`` with the same ``causal``) may be kept over the layers of a step.  Rows of outputs given as
    ``o_out`` / ``lse_out`` behind the last sequence are left as they are.
    Returns (o, lse, extras) with extras = {"plan", "workspace"} (the partials' buffer)."""
    if torch is None:
        _init()
    if q.dim() != 3 or k.dim() != 3:
        _bad("q is [total_q, Hq, D], k and v are [total_kv, Hk, D]")
    dev = _device_index(q)
    if _elsewhere(dev, stream):
        with _Launch(dev, stream):
            return prompt_attention(q, k, v, qo_indptr_h, kv_indptr_h, causal=causal, sm_scale=sm_scale,
                                    o_dtype=o_dtype, plan=plan, status=status, o_out=o_out, lse_out=lse_out)
    total_q, hq, dim = q.shape
    total_kv = k.shape[0]
    qi, ki = _rows("q", q, _bf16, total_q, dim, dev), _rows("k", k, _bf16, total_kv, dim, dev)
    vi = _rows("v", v, _bf16, total_kv, dim, dev)
    hk = ki[0]
    if vi[0] != hk:
        _bad("k and v must have the same heads")
    if len(qo_indptr_h) < 1 or total_q < qo_indptr_h[-1]:
        _bad("q has fewer rows than qo_indptr names")
    if total_kv < (qo_indptr_h if kv_indptr_h is None else kv_indptr_h)[-1]:
        _bad("k and v have fewer rows than kv_indptr names")
    if plan is None:
        plan = plan_prompt(qo_indptr_h, kv_indptr_h, hq, hk, dim, causal)
    if plan.device is None:
        plan.to(q.device)
    o, o_code, lse = _outputs(q, total_q, hq, dim, o_dtype, o_out, lse_out, dev)
    ws, o_part, lse_part = _workspace(q, plan, hq, dim)
    ret = _call_prompt(_pack_prompt(
        qi[1], ki[1], vi[1], qi[2], qi[3], ki[2], ki[3], vi[2], vi[3], total_q, total_kv, hq, hk, dim,
        dim ** -0.5 if sm_scale is None else sm_scale, o.data_ptr(), o_code, lse.data_ptr(), o_part, lse_part,
        0 if status is None else _index("status", status, -1, dev)), _index("plan", plan.device, -1, dev),
        ctypes.addressof(plan.info), _raw_stream(dev))
    if ret:
        raise SkvError(ret, "skv_prompt_attn_fwd")
    return o, lse, {"plan": plan, "workspace": ws}
