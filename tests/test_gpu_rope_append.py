"""GPU parity of rotary positions and the cache append against the float64 oracle.

Tolerances.  Rotation: |x'| <= |a| + |b| for a pair (a, b); fp32 cos and sin are within 2 ulp (2^-23)
of their angle's, the fp32 angle within 2^-25 of its own, the two products and their sum round by
2^-24 each: together below 2^-21 (|a| + |b|) m.  A bf16 result adds half a step, 2^-8 |x'|.
Codes: half a step of the format (e4m3: 2^-4 |x| for normal values, 2^-10 scales below; int8: half a
scale) on top of the rotation's error; the scale itself is one division of a value with that error:
2^-21 of the sum of the head's largest pair."""
import numpy as np
import pytest
import torch

import oracle.serving as OS
import split_kv_merge_b200 as skv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
QMAX = {"e4m3": 448.0, "i8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).to(DEV)


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


def _pair_size(x, rope_dim, layout):
    """|a| + |b| of every value's pair (|x| outside the rotated part)."""
    s = np.abs(x).copy()
    if rope_dim:
        a, b = OS.pair_columns(layout, rope_dim)
        both = np.abs(x[..., a]) + np.abs(x[..., b])
        s[..., a], s[..., b] = both, both
    return s


def _check_rotated(got, x, pos, f, layout, mscale, inverse, dtype, where):
    want = OS.rotate(x, pos, f, layout, mscale, inverse)
    tol = _pair_size(x, 2 * len(f), layout) * 2.0 ** -21 * mscale
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(_f64(got) - want)
    assert np.all(err <= tol + 1e-30), (where, float((err - tol).max()))
    rest = _f64(got)[..., 2 * len(f):]
    assert np.array_equal(rest, x[..., 2 * len(f):])


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,d,rope", [(1, 1, 1, 64, 64), (17, 5, 1, 128, 128), (33, 8, 2, 128, 48),
                                                 (7, 3, 0, 72, 64), (5, 0, 2, 8, 0), (300, 64, 8, 128, 128),
                                                 (9, 2, 2, 256, 256), (3, 1, 1, 1024, 32), (6, 2, 1, 24, 16)])
def test_rope(layout, dtype, tokens, hq, hk, d, rope):
    rng = np.random.default_rng(tokens + d)
    x = [torch.from_numpy(rng.standard_normal((tokens, h, d)).astype(np.float32)).to(dtype).to(DEV) if h else None
         for h in (hq, hk)]
    pos = rng.integers(-5, 200000, tokens)
    f = 10000.0 ** (-np.arange(rope // 2) * 2.0 / max(1, rope))
    for inverse in (False, True):
        out = skv.rope_apply(*x, _i32(pos), rope_dim=rope, rope_layout=layout, mscale=1.25, inverse=inverse)
        for t, o in zip(x, out):
            assert (o is None) == (t is None)
            if o is not None:
                _check_rotated(o, _f64(t), pos, f, layout, 1.25, inverse, dtype, (layout, inverse))


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_rope_far_positions_and_frequencies(layout):
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 2 ** 20 + 3, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31, 99999999])
    q = torch.from_numpy(rng.standard_normal((len(pos), 2, 64)).astype(np.float32)).to(DEV)
    f, m = skv.rope_frequencies(64, 500000.0, "yarn", 16.0, 4096)
    f[:4] = [2.5, 7.0, -0.3, 0.0]            # several turns a position, backwards, none
    o, _ = skv.rope_apply(q, None, _i32(pos), rope_layout=layout, inv_freq=f, mscale=m)
    _check_rotated(o, _f64(q), pos, f, layout, m, False, torch.float32, layout)


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_rope_strided_in_place_and_inverse(layout):
    rng = np.random.default_rng(6)
    qkv = _bf16(rng, 50, 12, 64)
    before = qkv.clone()
    pos = rng.integers(0, 5000, 50)
    q, k = qkv[:, :8], qkv[:, 8:10]
    f = 10000.0 ** (-np.arange(16) / 16.0)
    want = skv.rope_apply(q, k, _i32(pos), rope_dim=32, rope_layout=layout)
    got = skv.rope_apply(q, k, _i32(pos), rope_dim=32, rope_layout=layout, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 10:], before[:, 10:])
    _check_rotated(q, _f64(before[:, :8]), pos, f, layout, 1.0, False, torch.bfloat16, layout)
    # the transpose: <R x, y> = <x, R^T y> in float32
    x, y = (torch.from_numpy(rng.standard_normal((50, 3, 64)).astype(np.float32)).to(DEV) for _ in range(2))
    rx, _ = skv.rope_apply(x, None, _i32(pos), rope_layout=layout, mscale=1.3)
    ry, _ = skv.rope_apply(y, None, _i32(pos), rope_layout=layout, mscale=1.3, inverse=True)
    lhs, rhs = (rx.double() * y.double()).sum(-1), (x.double() * ry.double()).sum(-1)
    bound = 2.0 ** -20 * 1.3 * (x.double().norm(dim=-1) * y.double().norm(dim=-1)) * 2
    assert bool(torch.all((lhs - rhs).abs() <= bound))


def test_rope_copies_without_positions():
    """The C entry needs no positions when nothing turns."""
    import ctypes
    x = _bf16(np.random.default_rng(3), 9, 3, 64)
    out = torch.zeros_like(x)
    p = skv.RopeParams(q=x.data_ptr(), q_out=out.data_ptr(), q_stride=x.stride()[:2], q_out_stride=out.stride()[:2],
                       num_tokens=9, num_q_heads=3, head_dim=64, dtype=skv.BF16, rope=skv.Rope(0, 0, 1e4, None, 1.0))
    assert skv._rope_apply(ctypes.byref(p), torch.cuda.current_stream().cuda_stream) == skv.OK
    torch.cuda.synchronize()
    assert torch.equal(out, x)


def test_rope_no_tokens():
    q, _ = skv.rope_apply(torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), None, _i32([]))
    assert q.shape == (0, 4, 64)


# ------------------------------------------------------------------------------------- append
class Case:
    """A cache with earlier tokens in it, new tokens for some requests, and rows behind the last."""

    def __init__(self, seed, old, new, page, block, cache, hk, d, hq=0, pad=3, offset_views=False):
        rng = np.random.default_rng(seed)
        self.old, self.new, self.page, self.block, self.cache, self.hk, self.d = old, new, page, block, cache, hk, d
        total = [o + n for o, n in zip(old, new)]
        n_pages = [-(-t // page) for t in total]
        self.kv_indptr = np.concatenate([[0], np.cumsum(n_pages)])
        self.last = np.array([t - (p - 1) * page if p else 1 for t, p in zip(total, n_pages)])
        self.num_pages = int(self.kv_indptr[-1]) + 2
        self.kv_indices = rng.permutation(self.num_pages)[:self.kv_indptr[-1]]
        self.append_indptr = np.concatenate([[0], np.cumsum(new)])
        rows = int(self.append_indptr[-1]) + pad
        self.k, self.v = _bf16(rng, rows, hk, d), _bf16(rng, rows, hk, d)
        self.k *= torch.exp(torch.randn(rows, hk, 1, generator=torch.Generator().manual_seed(seed)).to(DEV)).bfloat16()
        self.q = _bf16(rng, rows, hq, d) if hq else None
        shape = (self.num_pages, page, hk, d)
        self.k_scale = self.v_scale = None
        if cache == "bf16":
            self.k_cache, self.v_cache = _bf16(rng, *shape), _bf16(rng, *shape)
        else:
            codes = [torch.from_numpy(rng.integers(1, 120, shape).astype(np.uint8) | (rng.integers(0, 2, shape) << 7).astype(np.uint8))
                     for _ in range(2)]
            self.k_cache, self.v_cache = (c.to(DEV).view(CODE[cache]) for c in codes)
            if block:
                self.k_scale, self.v_scale = (torch.from_numpy(np.exp(rng.standard_normal((self.num_pages, page // block, hk))
                                              - 4).astype(np.float32)).to(DEV) for _ in range(2))
        self.rows = OS.append_rows(self.append_indptr, self.kv_indptr, self.kv_indices, self.last, page)

    def run(self, **kw):
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = skv.paged_kv_append(self.k, self.v, self.k_cache, self.v_cache, _i32(self.append_indptr),
                                  _i32(self.kv_indptr), _i32(self.kv_indices), _i32(self.last), k_scale=self.k_scale,
                                  v_scale=self.v_scale, q=self.q, status=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def bits(self):
        raw = lambda t: t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy().copy()  # noqa: E731
        return raw(self.k_cache), raw(self.v_cache)

    def scales(self):
        return [None if s is None else _f64(s).copy() for s in (self.k_scale, self.v_scale)]


def _check_append(c, before, before_scales, rope=0, layout="halves", mscale=1.0, positions=None, kv_scale=1.0):
    assert int(c.status.item()) == 0
    n = len(c.rows)
    pos = np.array([p for _, p, _, _ in c.rows]) if positions is None else positions[:n]
    f = 10000.0 ** (-np.arange(rope // 2) * 2.0 / max(1, rope))
    k = _f64(c.k)[:n]
    want = {"k": OS.rotate(k, pos, f, layout, mscale) if rope else k, "v": _f64(c.v)[:n]}
    noise = {"k": _pair_size(k, rope, layout) * 2.0 ** -21 * mscale if rope else np.zeros_like(k), "v": np.zeros_like(k)}
    after, after_scales = c.bits(), c.scales()
    written = np.zeros((c.num_pages, c.page), bool)
    for _, _, page, slot in c.rows:
        written[page, slot] = True
    for i, name in enumerate("kv"):
        x, e = want[name], noise[name]
        if c.cache == "bf16":
            assert np.array_equal(after[i][~written], before[i][~written]), name
            got = _f64(c.k_cache if name == "k" else c.v_cache)
            for t, (_, _, page, slot) in enumerate(c.rows):
                assert np.all(np.abs(got[page, slot] - x[t]) <= 2.0 ** -8 * np.abs(x[t]) + 1.01 * e[t]), (name, t)
            continue
        step = lambda v, s: np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) if c.cache == "e4m3" else 0.5 * s  # noqa: E731
        got = OS.decode(after[i], c.cache)
        if not c.block:
            assert np.array_equal(after[i][~written], before[i][~written]), name
            for t, (_, _, page, slot) in enumerate(c.rows):
                y = np.clip(x[t], -448 * kv_scale, 448 * kv_scale)
                assert np.all(np.abs(got[page, slot] * kv_scale - y) <= step(y, kv_scale) * (1 + 2.0 ** -20) + 1.1 * e[t]), (name, t)
            continue
        old_values = OS.decode(before[i], c.cache) * np.repeat(before_scales[i], c.block, axis=1)[..., None]
        values, scales = OS.append_blocks(x, old_values, before_scales[i], c.rows, c.block, QMAX[c.cache])
        changed = scales != before_scales[i]
        spread = e.max() / QMAX[c.cache]
        assert np.all(np.abs(after_scales[i] - scales) <= 2.0 ** -22 * scales + spread), name
        # the other slots of a block with earlier tokens are re-encoded where the scale grew; all else keeps its bits
        first = {}
        for r, p, page, slot in c.rows:
            first.setdefault((page, slot // c.block), slot)
        same = ~written
        for (page, b), slot in first.items():
            if slot % c.block and changed[page, b].any():
                same[page, b * c.block:(b + 1) * c.block] = False
        assert np.array_equal(after[i][same], before[i][same]), name
        full = got * np.repeat(after_scales[i], c.block, axis=1)[..., None]
        s = np.repeat(after_scales[i], c.block, axis=1)[..., None]
        for (page, b), slot in first.items():
            mine = np.arange(c.page) // c.block == b
            if slot % c.block == 0:                          # a new block: its other slots hold nothing
                mine &= written[page]
            err = np.abs(full[page, mine] - values[page, mine])
            tol = step(values[page, mine], s[page, mine]) * (1 + 2.0 ** -18) + 2.0 ** -20 * QMAX[c.cache] * s[page, mine] + 1.1 * e.max()
            assert np.all(err <= tol), (name, page, b, float((err - tol).max()))


SHAPES = [  # page, block
    ("bf16", 16, 0), ("bf16", 1, 0), ("e4m3", 16, 0), ("e4m3", 16, 16), ("i8", 16, 16), ("i8", 16, 4), ("e4m3", 1, 1),
    ("e4m3", 64, 64), ("i8", 256, 256), ("i8", 48, 24)]


@pytest.mark.parametrize("cache,page,block", SHAPES)
@pytest.mark.parametrize("hk,d,hq", [(2, 64, 8), (5, 128, 0), (8, 128, 64)])
def test_append(cache, page, block, hk, d, hq):
    c = Case(7 + page, [0, 5, 16, 300, 0, 31, 255, 40], [1, 1, 17, 40, 0, 2, 70, 0], page, block, cache, hk, d, hq)
    before, before_scales = c.bits(), c.scales()
    tail = len(c.rows)
    q_before = None if c.q is None else c.q.clone()
    q_out = None if c.q is None else torch.full_like(c.q, 7.0)
    c.run(rope_dim=d, rope_layout="halves", mscale=1.1, kv_scale=0.03, q_out=q_out)
    _check_append(c, before, before_scales, d, "halves", 1.1, kv_scale=0.03)
    if hq:
        pos = np.array([p for _, p, _, _ in c.rows])
        f = 10000.0 ** (-np.arange(d // 2) * 2.0 / d)
        _check_rotated(q_out[:tail], _f64(q_before)[:tail], pos, f, "halves", 1.1, False, torch.bfloat16, "q")
        assert bool(torch.all(q_out[tail:] == 7.0)) and torch.equal(c.q, q_before)


@pytest.mark.parametrize("cache,page,block", [("bf16", 16, 0), ("i8", 32, 32), ("e4m3", 32, 8)])
@pytest.mark.parametrize("layout,rope", [("interleaved", 64), ("interleaved", 16), ("halves", 0)])
def test_append_layouts_and_positions(cache, page, block, layout, rope):
    c = Case(31, [3, 0, 100], [4, 9, 33], page, block, cache, 3, 64, 6)
    before, before_scales = c.bits(), c.scales()
    pos = np.random.default_rng(2).integers(0, 100000, c.k.shape[0])
    c.run(rope_dim=rope, rope_layout=layout, positions=_i32(pos))
    _check_append(c, before, before_scales, rope, layout, positions=pos)


@pytest.mark.parametrize("cache,block", [("bf16", 0), ("e4m3", 64), ("i8", 16)])
def test_append_long_prompts(cache, block):
    """Windows of several rows: blocks that begin in one window and end in the next."""
    c = Case(9, [10, 0, 63], [9000, 4000, 6001], 64, block, cache, 2, 64, 2)
    before, before_scales = c.bits(), c.scales()
    c.run(rope_dim=0)
    _check_append(c, before, before_scales)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_append_scale_growth_and_repeats(cache):
    """Tokens appended one by one to one block: the scale only grows; the same call again changes nothing."""
    c = Case(12, [0], [16], 16, 16, cache, 2, 64, pad=0)
    rows_k, rows_v = c.k.clone(), c.v.clone()
    top = 0.0
    for t in range(16):
        step = Case(12, [t], [1], 16, 16, cache, 2, 64, pad=0)
        step.k_cache, step.v_cache, step.k_scale, step.v_scale = c.k_cache, c.v_cache, c.k_scale, c.v_scale
        step.kv_indices, step.num_pages = c.kv_indices, c.num_pages
        step.rows = OS.append_rows(step.append_indptr, step.kv_indptr, step.kv_indices, step.last, 16)
        step.k, step.v = rows_k[t:t + 1], rows_v[t:t + 1]
        before, before_scales = step.bits(), step.scales()
        step.run()
        _check_append(step, before, before_scales)
        again, again_scales = step.bits(), step.scales()
        step.run()
        assert all(np.array_equal(a, b) for a, b in zip(again, step.bits()))
        assert all(np.array_equal(a, b) for a, b in zip(again_scales, step.scales()))
        page = int(c.kv_indices[0])
        now = _f64(c.k_scale)[page, 0]
        assert np.all(now >= top)
        top = now


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_append_zero_and_tiny_rows(cache):
    c = Case(13, [0, 4], [5, 3], 16, 16, cache, 2, 64)
    c.k[:5] = 0.0
    c.v[:5] = 1e-38
    for s in (c.k_scale, c.v_scale):
        s[int(c.kv_indices[1])] = 0.0               # earlier tokens of the second request: all zero
    c.run(rope_dim=64)
    page = int(c.kv_indices[0])
    assert bool(torch.all(c.k_scale[page] == 0)) and bool(torch.all(c.k_cache.view(torch.uint8)[page, :5] & 0x7F == 0))
    # 1e-38 / qmax is below 2^-126: held as zero
    assert bool(torch.all(c.v_scale[page] == 0)) and bool(torch.all(c.v_cache.view(torch.uint8)[page, :5] & 0x7F == 0))
    assert bool(torch.all(torch.isfinite(c.k_scale)))


def test_append_values_that_are_not_finite_stay_in_their_block():
    c, clean = (Case(14, [0, 0], [40, 20], 16, 16, "e4m3", 2, 64) for _ in range(2))
    c.k[3, 0, 5], c.v[20, 1, 0] = float("nan"), float("inf")
    c.run()
    clean.run()
    a, b = c.bits(), clean.bits()
    for i, t, h in ((0, 3, 0), (1, 20, 1)):
        _, _, page, slot = c.rows[t]
        bad = np.zeros(a[i].shape[:3], bool)
        bad[page, :, h] = True
        assert np.array_equal(a[i][~bad], b[i][~bad])
    _, _, page, slot = c.rows[3]
    assert a[0][page, slot, 0, 5] & 0x7F == 0x7F       # a NaN stays one


def test_append_bad_pages_and_short_requests():
    for cache, block in (("bf16", 0), ("i8", 16)):
        c = Case(15, [5, 0, 0], [3, 20, 4], 16, block, cache, 2, 64, 4)
        c.kv_indices = c.kv_indices.copy()
        c.kv_indices[1] = c.num_pages + 9              # the second request's first page
        before, before_scales = c.bits(), c.scales()
        c.run()
        assert int(c.status.item()) == skv.DEV_PAGE_OOB
        keep = [r for r in c.rows if not (r[0] == 1 and r[1] < 16)]
        after = c.bits()
        touched = np.zeros((c.num_pages, 16), bool)
        for _, _, page, slot in keep:
            touched[page, slot] = True
        if block:                                      # the first request's block: its scale may have grown
            touched[int(c.kv_indices[0])] = True
        for i in range(2):
            assert np.array_equal(after[i][~touched], before[i][~touched])
            assert not np.array_equal(after[i][touched], before[i][touched])
        c = Case(16, [0, 0], [5, 6], 16, block, cache, 2, 64, 4)
        c.last = np.array([4, 6])                      # shorter than its new tokens
        before = c.bits()
        c.run()
        assert int(c.status.item()) == skv.DEV_PLAN_BAD
        page = int(c.kv_indices[0])
        assert np.array_equal(c.bits()[0][page], before[0][page])


@pytest.mark.parametrize("cache,block", [("bf16", 0), ("e4m3", 16)])
def test_append_captured_and_replayed_with_other_lengths(cache, block):
    """One graph over padded rows; the batch's lengths change on the device between replays."""
    c = Case(17, [0, 20, 33], [1, 1, 1], 16, block, cache, 2, 64, 4, pad=6)
    ip, ki, ix, la = _i32(c.append_indptr), _i32(c.kv_indptr), _i32(c.kv_indices), _i32(c.last)
    q_out = torch.zeros_like(c.q)
    call = lambda: skv.paged_kv_append(c.k, c.v, c.k_cache, c.v_cache, ip, ki, ix, la, k_scale=c.k_scale,  # noqa: E731
                                       v_scale=c.v_scale, q=c.q, q_out=q_out, rope_dim=64)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for seed, old, new in ((18, [0, 20, 33], [1, 1, 1]), (19, [1, 17, 30], [1, 4, 2]), (20, [0, 1, 2], [0, 0, 1])):
        other = Case(seed, old, new, 16, block, cache, 2, 64, 4, pad=9 - sum(new))
        pages = -(-(np.array(old) + np.array(new)) // 16)
        assert np.all(pages <= np.diff(c.kv_indptr))
        # same pages as the captured batch, fewer of them in use
        other.kv_indices = np.concatenate([c.kv_indices[c.kv_indptr[r]:c.kv_indptr[r] + pages[r]] for r in range(3)])
        other.num_pages = c.num_pages
        other.rows = OS.append_rows(other.append_indptr, other.kv_indptr, other.kv_indices, other.last, 16)
        other.k_cache, other.v_cache, other.k_scale, other.v_scale = c.k_cache, c.v_cache, c.k_scale, c.v_scale
        before, before_scales = c.bits(), c.scales()
        for dst, src in ((ip, other.append_indptr), (ki, other.kv_indptr), (la, other.last)):
            dst.copy_(_i32(src))
        ix[:len(other.kv_indices)] = _i32(other.kv_indices)
        c.k.copy_(other.k)
        c.v.copy_(other.v)
        graph.replay()
        torch.cuda.synchronize()
        other.k, other.v = c.k, c.v
        other.status = torch.zeros(1, dtype=torch.int32)
        _check_append(other, before, before_scales, 64, "interleaved")


def test_append_on_another_stream_and_strided_inputs():
    rng = np.random.default_rng(21)
    c = Case(22, [3, 0], [20, 50], 16, 16, "i8", 2, 128, 4, pad=0)
    rows = c.k.shape[0]
    qkv = _bf16(rng, rows, 8, 128)
    c.q, c.k, c.v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    # K and V halves of one allocation, scales as slices of one
    both = torch.zeros(c.num_pages, 16, 2, 2, 128, dtype=torch.int8, device=DEV)
    both[:, :, 0], both[:, :, 1] = c.k_cache, c.v_cache
    c.k_cache, c.v_cache = both[:, :, 0], both[:, :, 1]
    scales = torch.stack([c.k_scale, c.v_scale], dim=-1).contiguous()
    c.k_scale, c.v_scale = scales[..., 0], scales[..., 1]
    before = tuple(x.contiguous().view(torch.uint8).cpu().numpy().copy() for x in (c.k_cache, c.v_cache))
    before_scales = c.scales()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    c.run(rope_dim=128, stream=stream)
    c.k_cache, c.v_cache = c.k_cache.contiguous(), c.v_cache.contiguous()
    _check_append(c, before, before_scales, 128, "interleaved")


def test_rows_past_32_bit_offsets():
    """Tokens 8.4 million values apart, read, turned in place and appended (bf16 pages as far apart)."""
    rng = np.random.default_rng(16)
    n, hk, d, page = 260, 2, 128, 16
    far = torch.zeros(n * 8_400_000, dtype=torch.bfloat16, device=DEV)
    x = torch.from_numpy(rng.standard_normal((n, hk, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    spread = far.as_strided((n, hk, d), (8_400_000, d, 1))
    spread.copy_(x)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    want, _ = skv.rope_apply(x, None, pos)
    got, _ = skv.rope_apply(spread, None, pos)
    assert torch.equal(got, want)
    pages = -(-n // page)
    table = [torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([0, n], [0, pages], list(range(pages))[::-1], [n - (pages - 1) * page])]
    dense = [torch.zeros(pages, page, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    skv.paged_kv_append(x, x, *dense, *table, rope_dim=d)
    cache = [far[at:].as_strided((pages, page, hk, d), (130_000_000, 512, 128, 1)) for at in (1024, 1024 + 256)]
    skv.paged_kv_append(spread, x, *cache, *table, rope_dim=d)
    for a, b in zip(dense, cache):
        assert torch.equal(a, b)
    skv.rope_apply(spread, None, pos, q_out=spread)
    assert torch.equal(spread, want)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("growth", [1.0, 1.07, 1.5])
def test_a_block_filled_token_by_token_against_its_tokens(cache, growth):
    """Each token `growth` times the last: a token's error is the sum of one rounding for every scale that it was held
    at (int8: half of it; e4m3: 2^-4 of the value as it then was, or half the subnormal step 2^-9 of the scale).  The
    scale is amax / qmax to 2^-22, each product of a re-encoding to 2^-24."""
    n, hk, d, page = 32, 2, 64, 32
    rng = np.random.default_rng(23)
    x = [torch.from_numpy((rng.standard_normal((n, hk, d)) * growth ** np.arange(n)[:, None, None]).astype(np.float32))
         .to(torch.bfloat16).to(DEV) for _ in range(2)]
    codes = [torch.zeros(1, page, hk, d, dtype=CODE[cache], device=DEV) for _ in range(2)]
    scales = [torch.zeros(1, 1, hk, device=DEV) for _ in range(2)]
    want, bound, held = [_f64(t) for t in x], [np.zeros((n, hk, d)) for _ in x], [np.zeros(hk) for _ in x]
    raised = 0
    for t in range(n):
        skv.paged_kv_append(x[0][t:t + 1], x[1][t:t + 1], *codes, _i32([0, 1]), _i32([0, 1]), _i32([0]), _i32([t + 1]),
                            k_scale=scales[0], v_scale=scales[1])
        for i in range(2):
            s = _f64(scales[i])[0, 0]
            grew = s > held[i]
            raised += int(grew.sum()) if t else 0
            live = np.zeros((n, hk, 1), bool)
            live[t], live[:t] = True, grew[:, None]
            step = 0.5 * s[:, None] if cache == "i8" else np.maximum(2.0 ** -4 * (np.abs(want[i]) + bound[i]), 2.0 ** -10 * s[:, None])
            noise = 2.0 ** -21 * (np.abs(want[i]) + bound[i])
            bound[i] += np.where(live, np.broadcast_to(step, bound[i].shape) + noise, 0.0)
            held[i] = s
            got = OS.decode(codes[i].view(torch.uint8).cpu().numpy()[0], cache) * s[:, None]
            err = np.abs(got[:t + 1] - want[i][:t + 1])
            assert np.all(err <= bound[i][:t + 1]), (t, i, float((err / bound[i][:t + 1]).max()))
    top = [np.maximum.accumulate(np.abs(w).max(axis=2), axis=0) for w in want]
    assert raised == sum(int((m[1:] > m[:-1]).sum()) for m in top) > 0       # a scale grows with its block's largest value
