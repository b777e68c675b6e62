"""GPU parity of attention over a paged 8-bit cache with block scales against the float64 oracle.

Tolerances.  Scores: D products of f16 codes and bf16 queries are exact, their fp32 sum is off by at
most D 2^-23 of the sum of magnitudes M, the two scalings round by 2^-24 each: e_s = (D + 4) 2^-23 M.
LSE: e_s, the hardware exponential's 2^-22, a sum of at most L terms (L 2^-24).  O: weights move by
twice that, their f16 rounding by 2^-11 of themselves (2^-25 for the smallest; the largest
is at least 1), the divisor's by 2^-11 at most; a bf16 output adds half a step, 2^-8 |O|."""
import numpy as np
import pytest
import torch

import oracle.serving as OS
import split_kv_merge_b200 as skv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CODE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


class Case:
    def __init__(self, seed, lengths, q_lens, hq, hk, d, page, block, cache, extra=2, poison=True, spread=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hk, self.d, self.page, self.block, self.cache = hq, hk, d, page, block, cache
        self.lengths = np.asarray(lengths)
        n_pages = -(-self.lengths // page)
        self.kv_indptr = np.concatenate([[0], np.cumsum(n_pages)])
        self.last = np.where(n_pages > 0, self.lengths - (n_pages - 1) * page, 1)
        self.qo_indptr = np.concatenate([[0], np.cumsum(q_lens)])
        self.num_pages = int(self.kv_indptr[-1]) + extra
        self.kv_indices = rng.permutation(self.num_pages)[:self.kv_indptr[-1]]
        shape = (self.num_pages, page, hk, d)
        self.scale = [(np.exp(spread * rng.standard_normal((self.num_pages, page // block, hk))) *
                       (0.01 if cache == "i8" else 0.004)).astype(np.float32) for _ in range(2)]
        if cache == "i8":
            self.code = [rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8) for _ in range(2)]
        else:
            self.code = [(rng.integers(0, 0x7F, shape) | (rng.integers(0, 2, shape) << 7)).astype(np.uint8) for _ in range(2)]
        if poison:  # what no request sees: NaN codes (the lowest for int8), NaN scales
            seen = np.zeros((self.num_pages, page), bool)
            for r, n in enumerate(self.lengths):
                for t in range(n):
                    seen[self.kv_indices[self.kv_indptr[r] + t // page], t % page] = True
            live = seen.reshape(self.num_pages, page // block, block).any(axis=2)
            for i in range(2):
                self.code[i][~seen] = 0x80 if cache == "i8" else 0x7F
                self.scale[i][~live] = np.nan
        q = rng.standard_normal((int(self.qo_indptr[-1]), hq, d)).astype(np.float32)
        self.q = torch.from_numpy(q).to(torch.bfloat16).to(DEV)

    def device(self):
        k, v = (torch.from_numpy(c).to(DEV).view(CODE[self.cache]) for c in self.code)
        ks, vs = (torch.from_numpy(s).to(DEV) for s in self.scale)
        return k, v, ks, vs

    def values(self, i, r):
        n = int(self.lengths[r])
        t = np.arange(n)
        page, slot = self.kv_indices[self.kv_indptr[r] + t // self.page], t % self.page
        return OS.decode(self.code[i][page, slot], self.cache) * self.scale[i][page, slot // self.block].astype(np.float64)[..., None]

    def oracle(self, causal, sm_scale, requests=None):
        q = self.q.double().cpu().numpy()
        return OS.packed_attention(q, lambda r: self.values(0, r), lambda r: self.values(1, r), self.qo_indptr,
                                   self.lengths, self.hk, causal, sm_scale, requests)


def _run(c, causal, tensors=None, **kw):
    k, v, ks, vs = c.device() if tensors is None else tensors
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse, ex = skv.paged_attention_scaled(c.q, k, v, ks, vs, c.qo_indptr, c.kv_indptr, _i32(c.kv_indices), c.last,
                                            causal=causal, num_pages=c.num_pages, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0, skv.status_str(int(status.item()))
    return o, lse, ex


def _check(c, o, lse, causal, sm_scale=None, requests=None, where=""):
    sm_scale = c.d ** -0.5 if sm_scale is None else sm_scale
    O, LSE, A, M = c.oracle(causal, sm_scale, requests)
    rows = ~np.isnan(LSE).all(axis=1)
    O, LSE, A, M = O[rows], LSE[rows], A[rows], M[rows]
    got, glse = o.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    assert np.array_equal(np.isneginf(glse), np.isneginf(LSE)), where
    empty = np.isneginf(LSE)
    assert np.all(got[empty] == 0)
    L = max(1, int(c.lengths.max()))
    e = (c.d + 4) * 2.0 ** -23 * M + 2.0 ** -22 + L * 2.0 ** -24
    err = np.abs(np.where(empty, 0, glse - np.where(empty, 0, LSE)))
    assert np.all(err <= e + 2.0 ** -23 * np.abs(np.where(empty, 0, LSE))), (where, float(err.max()))
    vmax = max((np.abs(c.values(1, r)).max() for r in range(len(c.lengths)) if c.lengths[r]), default=0.0)
    tol = A * (2.0 ** -10 + 2 * e[..., None]) + L * 2.0 ** -25 * vmax
    if o.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O)
    err = np.abs(got - O)
    assert np.all(err <= tol), (where, float((err / np.maximum(tol, 1e-30)).max()))


LENGTHS = [0, 1, 16, 17, 31, 33, 300, 1000, 65]


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (64, 8, 128), (5, 1, 128), (12, 3, 64), (4, 4, 128), (32, 16, 64),
                                     (40, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("policy,param", [("none", 0), ("fixed", 3), ("balanced", 0)])
def test_heads_and_splits(cache, hq, hk, d, policy, param):
    c = Case(hq + d, LENGTHS, [1] * len(LENGTHS), hq, hk, d, 16, 16, cache)
    o, lse, ex = _run(c, False, policy=policy, param=param)
    assert ex["plan"].info.kernel == 5
    _check(c, o, lse, False)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("page,block", [(1, 1), (16, 1), (16, 4), (24, 12), (64, 64), (256, 32), (7, 7)])
def test_pages_and_blocks(cache, page, block):
    c = Case(page, [5, 0, 129, 257, 700], [1, 1, 2, 1, 3], 8, 4, 64, page, block, cache)
    for causal in (False, True):
        o, lse, _ = _run(c, causal, policy="balanced", o_dtype=torch.bfloat16)
        _check(c, o, lse, causal)


@pytest.mark.parametrize("hq,hk,d", [(8, 8, 128), (32, 8, 128), (8, 1, 64), (24, 1, 64), (6, 2, 128)])
@pytest.mark.parametrize("q_lens", [[4, 4, 4, 4, 4], [1, 0, 7, 40, 2], [130, 1, 1, 3, 64]])
def test_several_query_tokens_causal(hq, hk, d, q_lens):
    """Mixed query lengths, some requests shorter than their query tokens (rows that see no key)."""
    c = Case(3, [4, 9, 3, 200, 1], q_lens, hq, hk, d, 16, 16, "i8")
    for policy in ("none", "balanced"):
        o, lse, _ = _run(c, True, policy=policy)
        _check(c, o, lse, True, where=policy)


def test_explicit_splits_and_empty_splits():
    c = Case(4, [200, 64], [2, 1], 8, 2, 64, 16, 16, "e4m3")
    o, lse, ex = _run(c, True, policy="explicit", split_page_start=[[0, 0, 5, 13], [0, 4, 4]])
    assert ex["plan"].info.num_partial_rows == 8
    _check(c, o, lse, True)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_rising_scores_and_extreme_scales(cache):
    """Each block's K scale larger than the last (the running maximum is raised again and again), V scales
    over many binades, a zero block and queries with one dominant element."""
    c = Case(5, [1500], [1], 16, 2, 128, 16, 16, cache, poison=False)
    order = c.kv_indices
    c.scale[0][order, 0] = (np.linspace(0.05, 3.0, len(order))[:, None] * (0.01 if cache == "i8" else 0.003)).astype(np.float32)
    c.scale[1][order, 0] = (2.0 ** np.random.default_rng(1).integers(-20, 4, (len(order), 2))).astype(np.float32)
    c.code[0][order[3]], c.scale[0][order[3]] = 0, 0.0
    c.code[1][order[4]], c.scale[1][order[4]] = 0, 0.0
    c.q[0, 3] *= 2.0 ** -30
    c.q[0, 4, 1:] *= 2.0 ** -20
    o, lse, _ = _run(c, False, policy="fixed", param=2)
    _check(c, o, lse, False)


@pytest.mark.parametrize("cache,block", [("e4m3", 16), ("i8", 16), ("i8", 4)])
def test_negative_softmax_scale_and_large_queries(cache, block):
    c = Case(15, [70, 300], [2, 1], 16, 2, 128, 16, block, cache)
    c.q *= 512.0
    o, lse, _ = _run(c, True, sm_scale=-0.0003)
    _check_scaled(c, o, lse, -0.0003)


def _check_scaled(c, o, lse, sm_scale):
    """As _check, with the score magnitudes taken at |sm_scale|."""
    q = c.q.double().cpu().numpy()
    args = (lambda r: c.values(0, r), lambda r: c.values(1, r), c.qo_indptr, c.lengths, c.hk, True)
    O, LSE, A, _ = OS.packed_attention(q, *args, sm_scale)
    M = OS.packed_attention(np.abs(q), lambda r: np.abs(c.values(0, r)), args[1], *args[2:], abs(sm_scale))[3]
    e = (c.d + 4) * 2.0 ** -23 * M + 2.0 ** -22 + 300 * 2.0 ** -24
    assert np.all(np.abs(lse.cpu().numpy() - LSE) <= e + 2.0 ** -23 * np.abs(LSE))
    vmax = max(np.abs(c.values(1, r)).max() for r in range(2))
    assert np.all(np.abs(o.cpu().numpy() - O) <= A * (2.0 ** -10 + 2 * e[..., None]) + 300 * 2.0 ** -25 * vmax)


def test_zero_scales_everywhere():
    c = Case(6, [40, 3], [1, 1], 8, 2, 64, 16, 16, "i8", poison=False)
    c.scale[0][:], c.scale[1][:] = 0.0, 0.0
    o, lse, _ = _run(c, False)
    assert bool(torch.all(o == 0))
    assert np.allclose(lse.cpu().numpy(), np.log([[40.0], [3.0]]), atol=1e-5)


@pytest.mark.parametrize("cache,page,block", [("e4m3", 16, 16), ("i8", 16, 16), ("e4m3", 12, 4), ("i8", 12, 4)])
def test_subnormal_scales_count_as_zero(cache, page, block):
    c = Case(7, [40, 100, 3], [1, 2, 1], 8, 2, 64, page, block, cache, poison=False)
    k, v, ks, vs = c.device()
    outs = []
    for tiny in (1e-39, 0.0):
        ks[::3], vs[::2] = tiny, tiny                      # whole pages, beside others of ordinary scales
        outs.append(_run(c, False, (k, v, ks, vs))[:2])
    assert bool(torch.isfinite(outs[0][0]).all()) and bool(torch.isfinite(outs[0][1]).all())
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("cache,block", [("i8", 16), ("e4m3", 4)])
def test_append_and_attention_past_32_bit_offsets(cache, block):
    """Pages 1.2e9 bytes apart: the same results as in a dense cache."""
    rng = np.random.default_rng(15)
    hq, hk, d, page, pages, n = 8, 2, 64, 16, 3, 45
    far = torch.zeros(2 * 1_200_000_000 + (1 << 16), dtype=torch.uint8, device=DEV)
    spread = lambda at: far[at:].as_strided((pages, page, hk, d), (1_200_000_000, 256, 64, 1)).view(CODE[cache])  # noqa: E731
    results = []
    k, v, q = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV) for h in (hk, hk, hq))
    ids = _i32([2, 0, 1])
    for dense in (True, False):
        kc, vc = ((torch.zeros(pages, page, hk, d, dtype=CODE[cache], device=DEV) for _ in range(2)) if dense else
                  (spread(0), spread(128)))
        ks, vs = (torch.zeros(pages, page // block, hk, device=DEV) for _ in range(2))
        skv.paged_kv_append(k, v, kc, vc, _i32([0, n]), _i32([0, 3]), ids, _i32([n - 32]), k_scale=ks, v_scale=vs,
                            rope_dim=d)
        o, lse, _ = skv.paged_attention_scaled(q, kc, vc, ks, vs, [0, n], [0, 3], ids, [n - 32], causal=True)
        results.append((o, lse, ks, vs, kc.view(torch.uint8).contiguous(), vc.view(torch.uint8).contiguous()))
    assert int(results[0][4].ne(0).sum()) > 0.9 * n * hk * d
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_strided_caches_scales_and_outputs_given():
    c = Case(7, [100, 33, 0, 250], [1, 2, 1, 1], 16, 4, 128, 16, 8, "e4m3")
    k, v, ks, vs = c.device()
    both = torch.zeros(c.num_pages, 4, 2, 16, 128, dtype=torch.uint8, device=DEV)  # heads outside, K | V side by side
    both[:, :, 0] = k.view(torch.uint8).permute(0, 2, 1, 3)
    both[:, :, 1] = v.view(torch.uint8).permute(0, 2, 1, 3)
    kk, vv = (both[:, :, i].permute(0, 2, 1, 3).view(torch.float8_e4m3fn) for i in range(2))
    sc = torch.stack([ks, vs], -1).permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    o = torch.full((5, 16, 128), 9.0, device=DEV)
    lse = torch.full((5, 16), 9.0, device=DEV)
    got = _run(c, True, (kk, vv, sc[..., 0], sc[..., 1]), o_out=o, lse_out=lse)
    assert got[0] is o and got[1] is lse
    _check(c, o, lse, True)
    plain, plse, _ = _run(c, True)
    assert torch.equal(plain, o) and torch.equal(plse, lse)


def test_repeated_calls_other_streams_and_two_at_once():
    cases = [Case(8 + i, [700, 90 + i, 2000], [1, 1, 1], 32, 8, 128, 16, 16, "e4m3") for i in range(2)]
    tensors = [c.device() for c in cases]
    first = [_run(c, False, t) for c, t in zip(cases, tensors)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    ix = [_i32(c.kv_indices) for c in cases]
    for _ in range(5):
        again = []
        for c, t, s, i in zip(cases, tensors, streams, ix):
            s.wait_stream(torch.cuda.current_stream())
            again.append(skv.paged_attention_scaled(c.q, *t, c.qo_indptr, c.kv_indptr, i, c.last, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_replayed():
    c = Case(11, [500, 64], [2, 2], 16, 2, 64, 32, 32, "i8")
    k, v, ks, vs = c.device()
    plan = skv.plan_paged_scaled(c.qo_indptr, c.kv_indptr, c.last, 32, 16, 2, 64, causal=True).to(DEV)
    ki, la, ix = _i32(c.kv_indptr), _i32(c.last), _i32(c.kv_indices)
    call = lambda: skv.paged_attention_scaled(c.q, k, v, ks, vs, c.qo_indptr, c.kv_indptr, ix, c.last, causal=True,  # noqa: E731
                                              kv_indptr=ki, kv_last_page_len=la, plan=plan)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse, _ = call()
    for _ in range(2):
        c.q.copy_(torch.randn_like(c.q.float()).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        _check(c, o, lse, True)


def test_bad_page_id_sets_status():
    c = Case(12, [100, 50], [1, 1], 8, 2, 64, 16, 16, "i8", poison=False)
    k, v, ks, vs = c.device()
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        ids = c.kv_indices.copy()
        ids[2] = bad
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, lse, _ = skv.paged_attention_scaled(c.q, k, v, ks, vs, c.qo_indptr, c.kv_indptr, _i32(ids), c.last, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == skv.DEV_PAGE_OOB
        _check_second_request(c, o, lse)


def _check_second_request(c, o, lse):
    O, LSE, _, _ = c.oracle(False, c.d ** -0.5, [1])
    assert np.abs(o[1].cpu().numpy() - O[1]).max() < 1e-2 * max(1.0, np.abs(O[1]).max())
    assert np.abs(lse[1].cpu().numpy() - LSE[1]).max() < 1e-3


def test_batch_shape_sampled():
    rng = np.random.default_rng(2)
    c = Case(13, rng.integers(1024, 8193, 64), [1] * 64, 64, 8, 128, 16, 16, "e4m3", poison=False)
    o, lse, ex = _run(c, True, o_dtype=torch.bfloat16)
    assert ex["plan"].info.num_merge_rows > 0
    order = np.argsort(c.lengths)
    _check(c, o, lse, True, requests=[int(order[0]), int(order[-1]), 17])


def test_append_then_attend():
    """A request built by prompts and single steps through paged_kv_append, attended after every step; the
    cache it reads is what append wrote, so the attention is exact for the stored values, and within
    the quantisation of the float64 attention over the tokens themselves."""
    rng = np.random.default_rng(14)
    hq, hk, d, page = 16, 4, 128, 16
    pages, order = 12, rng.permutation(12)
    for cache in ("e4m3", "i8"):
        k_cache, v_cache = (torch.zeros(pages, page, hk, d, dtype=CODE[cache], device=DEV) for _ in range(2))
        k_scale, v_scale = (torch.zeros(pages, 1, hk, device=DEV) for _ in range(2))
        keys, vals, length = [], [], 0
        for n in (37, 1, 1, 4, 60, 1):
            k, v, q = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
                       for h in (hk, hk, hq))
            length += n
            np_ = -(-length // page)
            ip, ki, la = np.array([0, n]), np.array([0, np_]), np.array([length - (np_ - 1) * page])
            q_rot = skv.paged_kv_append(k, v, k_cache, v_cache, _i32(ip), _i32(ki), _i32(order[:np_]), _i32(la),
                                        k_scale=k_scale, v_scale=v_scale, q=q, rope_dim=d, rope_layout="halves")
            o, lse, _ = skv.paged_attention_scaled(q_rot, k_cache, v_cache, k_scale, v_scale, ip, ki, _i32(order[:np_]), la,
                                                   causal=True)
            pos = np.arange(length - n, length)
            f = 10000.0 ** (-np.arange(d // 2) * 2.0 / d)
            keys.append(OS.rotate(k.double().cpu().numpy(), pos, f, "halves"))
            vals.append(v.double().cpu().numpy())
            K, V = np.concatenate(keys), np.concatenate(vals)
            O, LSE, _, _ = OS.packed_attention(OS.rotate(q.double().cpu().numpy(), pos, f, "halves"), lambda r: K,
                                               lambda r: V, ip, [length], hk, True, d ** -0.5)
            rel = np.linalg.norm(o.cpu().numpy() - O) / np.linalg.norm(O)
            # e4m3 is off by 2^-4 of a value at most, int8 by half a 127th of its block's largest (about 4 sigma)
            assert rel < (2.0 ** -4 if cache == "e4m3" else 4 / 127), (cache, length, rel)


def _check_visible(c, o, lse, causal, where=""):
    """As _check, with every bound taken from the keys that the row itself sees.  A weight times its V scale, w, is
    held in 11 bits (2^-11 of itself; a 2^-39th of the row's largest where it is less than a 2^-28th of that), the
    divisor is the sum of the exact weights; int8 codes carry a bias of 128 whose sum over 32 tokens comes out again
    in fp32 (34 additions of 2^-23 twice: 2^-10 of the sum of w, in units of one code)."""
    q = c.q.double().cpu().numpy()
    qmax, g, sm = (127.0 if c.cache == "i8" else 448.0), c.hq // c.hk, c.d ** -0.5
    for r, L in enumerate(c.lengths):
        k, v, t = c.values(0, r), c.values(1, r), np.arange(int(L))
        page = c.kv_indices[c.kv_indptr[r] + t // c.page]
        vs = c.scale[1][page, t % c.page // c.block].astype(np.float64)
        n = int(c.qo_indptr[r + 1] - c.qo_indptr[r])
        for i in range(n):
            seen = int(L) - n + i + 1 if causal else int(L)
            row = int(c.qo_indptr[r]) + i
            for h in range(c.hq):
                kk, vv, w = k[:seen, h // g], v[:seen, h // g], vs[:seen, h // g]
                s = sm * (kk @ q[row, h])
                M = sm * (np.abs(kk) @ np.abs(q[row, h])).max()
                want = np.log(np.exp(s - s.max()).sum()) + s.max()
                p = np.exp(s - want)
                e = (c.d + 4) * 2.0 ** -23 * M + 2.0 ** -22 + seen * 2.0 ** -24
                assert abs(float(lse[row, h]) - want) <= e + 2.0 ** -23 * abs(want), (where, r, i, h)
                tol = (p @ np.abs(vv)) * (2.0 ** -11 + 2.0 ** -20 + 2 * e + seen * 2.0 ** -23)
                tol = tol + seen * 2.0 ** -39 * (p * w).max() * qmax + (2.0 ** -10 * (p @ w) if c.cache == "i8" else 0.0)
                if o.dtype == torch.bfloat16:
                    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(p @ vv)
                err = np.abs(o[row, h].double().cpu().numpy() - p @ vv)
                assert np.all(err <= tol), (where, r, i, h, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 8), (12, 4)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (16, 2, 128), (2, 2, 128)])
def test_a_hidden_block_of_large_values_leaves_the_others_alone(cache, page, block, hq, hk, d):
    """The last token begins a block whose V scale is 2^k of the others'.  The first query token does not see it, nor
    may its result lose a bit to it."""
    for k in (0, 12, 18, 22, 26, 40):
        c = Case(31 + k, [2 * page + 1, 1 + block, 5 * page + 1], [2, 2, 2], hq, hk, d, page, block, cache, spread=0.3)
        for r, n in enumerate(c.lengths):
            at = int(n) - 1
            c.scale[1][c.kv_indices[c.kv_indptr[r] + at // page], at % page // block] *= np.float32(2.0 ** k)
        o, lse, _ = _run(c, True)
        _check_visible(c, o, lse, True, where=k)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("page,block", [(16, 16), (12, 4)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (16, 1, 128)])
def test_an_unattended_block_of_large_values_leaves_the_others_alone(cache, page, block, hq, hk, d):
    """Every other block has a V scale 2^k of its neighbour's and scores that leave it a weight of 2^-2k."""
    for k in (10, 18, 22, 26, 40):
        c = Case(41 + k, [3 * page + 5], [1], hq, hk, d, page, block, cache, poison=False, spread=0.3)
        small = np.zeros((c.num_pages, page // block), bool)
        for t in range(0, int(c.lengths[0]), block):
            small[c.kv_indices[t // page], t % page // block] = t // block % 2 == 0
        c.q[:] = 1.0
        c.code[0][:] = 64 if cache == "i8" else 0x38          # 64 and 1.0: all keys alike
        unit = 64.0 if cache == "i8" else 1.0
        c.scale[0][:] = 0.0                                    # large values: score 0
        c.scale[0][small] = 2 * k * np.log(2.0) / (d ** 0.5 * unit)   # small ones: 2 k ln 2
        c.scale[1][~small] *= np.float32(2.0 ** k)
        o, lse, _ = _run(c, False)
        _check_visible(c, o, lse, False, where=k)


@pytest.mark.parametrize("policy,param", [("none", 0), ("balanced", 0)])
def test_a_plan_without_causal_serves_last_pages_that_fill(policy, param):
    c = Case(51, [700, 35, 1201], [1, 2, 1], 16, 4, 128, 16, 16, "i8", poison=False)
    plan = skv.plan_paged_scaled(c.qo_indptr, c.kv_indptr, c.last, 16, 16, 4, 128, False, policy, param)
    for step in range(3):                      # last pages of 12, 3 and 1 tokens, then of two more each
        o, lse, _ = _run(c, False, plan=plan)
        _check_visible(c, o, lse, False, where=step)
        fresh = _run(c, False, policy=policy, param=param)
        assert torch.equal(o, fresh[0]) and torch.equal(lse, fresh[1])
        c.last, c.lengths = c.last + 2, c.lengths + 2
    c.last, c.lengths = c.last - 4, c.lengths - 4
    plan = skv.plan_paged_scaled(c.qo_indptr, c.kv_indptr, c.last, 16, 16, 4, 128, True, policy, param)
    _run(c, True, plan=plan)
    c.last = c.last + 1
    with pytest.raises(ValueError, match="plan was made for"):
        _run(c, True, plan=plan)
