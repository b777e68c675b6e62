"""GPU parity of packed prompt attention against the float64 oracle.

Tolerances.  Scores: products of bf16 are exact, their fp32 sum of D terms is off by at most D 2^-23
of the sum of magnitudes M, the scaling rounds: e_s = (D + 4) 2^-23 M.  LSE: e_s, the hardware
exponential's 2^-22, a sum of at most L terms (L 2^-24), its own rounding.  O: weights move by twice
e_s; rounded to bf16 they move by 2^-8 of themselves in the product and at most as much in the
divisor (the sum of the rounded ones); L fp32 additions; a bf16 output adds half a step, 2^-8 |O|."""
import numpy as np
import pytest
import torch

import oracle.serving as OS
import split_kv_merge_b200 as skv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Case:
    def __init__(self, seed, q_lens, kv_lens, hq, hk, d, pad=0, boost=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hk, self.d = hq, hk, d
        self.qo = np.concatenate([[0], np.cumsum(q_lens)])
        self.kv = np.concatenate([[0], np.cumsum(kv_lens)])
        make = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.q, self.k, self.v = make(int(self.qo[-1]) + pad, hq), make(int(self.kv[-1]) + pad, hk), make(int(self.kv[-1]) + pad, hk)
        self.q *= boost

    def oracle(self, causal, sm_scale=None, requests=None):
        q, k, v = (t.double().cpu().numpy() for t in (self.q, self.k, self.v))
        rows = lambda x, r: x[self.kv[r]:self.kv[r + 1]]  # noqa: E731
        return OS.packed_attention(q[:self.qo[-1]], lambda r: rows(k, r), lambda r: rows(v, r), self.qo, np.diff(self.kv),
                                   self.hk, causal, self.d ** -0.5 if sm_scale is None else sm_scale, requests)

    def run(self, causal, **kw):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, lse, ex = skv.prompt_attention(self.q, self.k, self.v, self.qo, self.kv, causal=causal, status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0, skv.status_str(int(status.item()))
        return o, lse, ex

    def check(self, o, lse, causal, sm_scale=None, requests=None, where=""):
        O, LSE, A, M = self.oracle(causal, sm_scale, requests)
        rows = np.flatnonzero(~np.isnan(LSE).all(axis=1))
        O, LSE, A, M = O[rows], LSE[rows], A[rows], M[rows]
        got, glse = o.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
        empty = np.isneginf(LSE)
        assert np.array_equal(np.isneginf(glse), empty), where
        assert np.all(got[empty] == 0), where
        L = max(1, int(np.diff(self.kv).max()))
        e = (self.d + 4) * 2.0 ** -23 * M + 2.0 ** -22 + L * 2.0 ** -24
        want = np.where(empty, 0, LSE)
        err = np.abs(np.where(empty, 0, glse) - want)
        assert np.all(err <= e + 2.0 ** -23 * np.abs(want)), (where, float(err.max()))
        tol = A * (2.0 ** -7 + 2 * e[..., None] + L * 2.0 ** -23) + 1e-30
        if o.dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(O)
        err = np.abs(got - O)
        assert np.all(err <= tol), (where, float((err / tol).max()), np.argwhere(err > tol)[:3])


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 128), (8, 2, 64), (4, 4, 128), (5, 1, 64), (12, 4, 128), (32, 8, 128), (16, 1, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_prompts(hq, hk, d, causal):
    lens = [1, 130, 0, 64, 300, 128, 129, 17]
    c = Case(hq + d, lens, lens, hq, hk, d)
    for dtype in (torch.float32, torch.bfloat16):
        o, lse, ex = c.run(causal, o_dtype=dtype)
        assert ex["plan"].info.kernel == 6 and ex["plan"].info.num_merge_rows == 0
        c.check(o, lse, causal, where=str(dtype))


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 128), (3, 3, 64), (6, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_more_or_fewer_keys_than_queries(hq, hk, d, causal):
    """Prompts taken in chunks, and sequences whose first query tokens see no key at all."""
    c = Case(5, [1, 7, 260, 3, 200, 129, 5], [1, 500, 700, 0, 100, 1, 1024], hq, hk, d)
    o, lse, _ = c.run(causal)
    c.check(o, lse, causal)


@pytest.mark.parametrize("hq,hk", [(4, 1), (3, 1)])
def test_cut_along_the_keys(hq, hk):
    """Few query tokens over many keys: partials and a merge."""
    c = Case(6, [100, 1, 300], [9000, 6000, 20], hq, hk, 128)
    for causal in (True, False):
        o, lse, ex = c.run(causal)
        assert ex["plan"].info.max_splits > 4 and ex["plan"].info.num_merge_rows >= 101
        c.check(o, lse, causal)
        ob, lb, _ = c.run(causal, o_dtype=torch.bfloat16)
        assert torch.equal(ob, o.to(torch.bfloat16)) and torch.equal(lb, lse)


@pytest.mark.parametrize("hq,hk,sms", [(4, 2, 20), (3, 1, 16)])
def test_uneven_rounds_are_cut(hq, hk, sms):
    """More items than CTAs, but no full round of them: the shortest are cut, the others stay whole."""
    c = Case(9, [1500], [4100], hq, hk, 128)
    plan = skv.plan_prompt(c.qo, c.kv, hq, hk, 128, True, sms)
    assert 0 < plan.info.num_merge_rows < 1500 and plan.info.num_ctas <= sms
    o, lse, _ = c.run(True, plan=plan)
    c.check(o, lse, True)


def test_other_sequences_never_reach_a_result():
    """NaN and infinite keys and values of one sequence stay in it, wherever its neighbours' tiles end."""
    for hq, hk in ((4, 2), (3, 3)):
        clean = Case(7, [60, 200, 5, 77], [60, 200, 5, 77], hq, hk, 64, pad=70)
        o0, l0, _ = clean.run(True)
        clean.k[60:260], clean.v[60:260] = float("nan"), float("inf")
        clean.k[342:], clean.v[342:] = float("nan"), float("nan")          # rows behind the last sequence
        clean.q[60:260] = float("nan")
        o1, l1, _ = clean.run(True)
        keep = torch.ones(342, dtype=torch.bool, device=DEV)
        keep[60:260] = False
        assert torch.equal(o0[:342][keep], o1[:342][keep]) and torch.equal(l0[:342][keep], l1[:342][keep])
        assert bool(torch.isnan(o1[60:260]).all())


def test_rows_behind_the_last_sequence_are_left():
    c = Case(8, [33, 90], [33, 90], 4, 2, 128, pad=150)
    o, lse = torch.full((273, 4, 128), 5.0, device=DEV), torch.full((273, 4), 5.0, device=DEV)
    c.run(True, o_out=o, lse_out=lse)
    c.check(o, lse, True)
    assert bool(torch.all(o[123:] == 5.0)) and bool(torch.all(lse[123:] == 5.0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_on_16_byte_addresses(dtype):
    """Results at an address that is a multiple of 16 bytes but not of 32."""
    c = Case(21, [33, 200], [33, 200], 4, 2, 64)
    want, lse, _ = c.run(True, o_dtype=dtype)
    flat = torch.zeros(233 * 4 * 64 + 32, dtype=dtype, device=DEV)
    out = flat[16 // flat.element_size():][:233 * 4 * 64].view(233, 4, 64)
    assert out.data_ptr() % 32 == 16
    c.run(True, o_out=out)
    assert torch.equal(out, want) and int(flat.ne(0).sum()) == int(want.ne(0).sum())


def test_slices_of_one_projection():
    rng = np.random.default_rng(9)
    qkv = torch.from_numpy(rng.standard_normal((321, 16, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    c = Case(9, [200, 121], [200, 121], 8, 4, 128)
    c.q, c.k, c.v = qkv[:, :8], qkv[:, 8:12], qkv[:, 12:]
    o, lse, _ = c.run(True)
    c.check(o, lse, True)
    # heads outside tokens, one KV head whose head stride is never used
    c = Case(10, [150], [150], 2, 1, 64)
    c.q = c.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    c.k = c.k.expand(-1, 1, -1).as_strided((150, 1, 64), (64, 3, 1))
    o, lse, _ = c.run(True)
    c.check(o, lse, True)


@pytest.mark.parametrize("boost", [8.0, 60.0])
def test_large_scores_and_scales(boost):
    """Scores far apart: the running maximum is raised again and again, rows with one dominant key."""
    c = Case(11, [500], [900], 4, 2, 128, boost=boost)
    c.k[600:] *= 3.0
    for causal in (True, False):
        o, lse, _ = c.run(causal, sm_scale=0.2)
        c.check(o, lse, causal, sm_scale=0.2)


def test_dominant_key_returns_its_value():
    c = Case(12, [40], [300], 2, 1, 128)
    c.k[:] = 0.0
    c.q[:] = 1.0
    c.k[123] = 8.0
    o, _, _ = c.run(False, sm_scale=1.0)
    assert torch.equal(o.cpu(), c.v[123].float().expand(40, 2, 128).cpu())


def test_repeats_streams_and_capture():
    c = Case(13, [400, 700, 50], [400, 900, 50], 8, 2, 128)
    o, lse, ex = c.run(True)
    plan = ex["plan"]
    for _ in range(3):
        o2, l2, _ = c.run(True, plan=plan)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    other = Case(14, [300, 20], [300, 4000], 3, 3, 64)
    want = other.run(True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = []
        for case, s in zip((c, other), streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append(skv.prompt_attention(case.q, case.k, case.v, case.qo, case.kv, stream=s))
        torch.cuda.synchronize()
        assert torch.equal(got[0][0], o) and torch.equal(got[1][0], want[0]) and torch.equal(got[1][1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg, _ = skv.prompt_attention(c.q, c.k, c.v, c.qo, c.kv, plan=plan)
    c.q.copy_(torch.randn_like(c.q.float()).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    c.check(og, lg, True)


def test_no_rows_and_no_keys():
    c = Case(15, [0, 0], [0, 5], 4, 2, 64)
    o, lse, _ = c.run(True)
    assert o.shape == (0, 4, 64)
    c = Case(16, [5, 130], [0, 0], 4, 2, 64)
    for causal in (True, False):
        o, lse, _ = c.run(causal)
        assert bool(torch.all(o == 0)) and bool(torch.all(torch.isneginf(lse)))


def test_rows_past_32_bit_offsets():
    """Tokens 8.4 million values apart."""
    c = Case(19, [260], [260], 4, 2, 128)
    want, lse, _ = c.run(True)
    for name, h in (("q", 4), ("k", 2), ("v", 2)):
        x = getattr(c, name)
        far = torch.empty(260 * 8_400_000, dtype=torch.bfloat16, device=DEV).as_strided((260, h, 128), (8_400_000, 128, 1))
        setattr(c, name, far.copy_(x))
        o, l2, _ = c.run(True)
        assert torch.equal(o, want) and torch.equal(l2, lse)
        setattr(c, name, x)


def test_long_prompt_sampled():
    """One 5000-token prompt: the heads of the first group against the oracle."""
    c = Case(17, [5000], [5000], 32, 8, 128)
    o, lse, _ = c.run(True, o_dtype=torch.bfloat16)
    s = Case(17, [1], [1], 4, 1, 128)
    rows = np.r_[0:3, 126:130, 2500:2503, 4990:5000]
    for r in rows:                       # row r alone: its last position over the first r + 1 keys
        s.qo, s.kv = np.array([0, 1]), np.array([0, r + 1])
        s.q, s.k, s.v = c.q[r:r + 1, :4], c.k[:r + 1, :1], c.v[:r + 1, :1]
        s.check(o[r:r + 1, :4], lse[r:r + 1, :4], True, where=int(r))


def test_a_serving_step():
    """Prompts rotated, attended and appended; then single steps over the cache they left: every output against
    the float64 attention over the tokens themselves."""
    rng = np.random.default_rng(18)
    hq, hk, d, page = 8, 2, 128, 16
    f, mscale = skv.rope_frequencies(d, 10000.0, "bands", 4.0, 64)
    lens = np.array([50, 7, 129])
    rope = dict(rope_dim=d, rope_layout="interleaved", inv_freq=f, mscale=mscale)
    make = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)  # noqa: E731
    n_max = -(-(lens + 3) // page)
    base = np.concatenate([[0], np.cumsum(n_max)])
    order = rng.permutation(int(base[-1]))
    k_cache, v_cache = (torch.zeros(int(base[-1]), page, hk, d, dtype=torch.int8, device=DEV) for _ in range(2))
    k_scale, v_scale = (torch.zeros(int(base[-1]), 1, hk, device=DEV) for _ in range(2))
    K, V = [np.zeros((0, hk, d))] * 3, [np.zeros((0, hk, d))] * 3
    now = np.zeros(3, int)
    for step in range(4):
        n = lens if step == 0 else np.ones(3, int)
        ip = np.concatenate([[0], np.cumsum(n)])
        T = int(ip[-1])
        q, k, v = make(T, hq), make(T, hk), make(T, hk)
        pos = np.concatenate([np.arange(now[r], now[r] + n[r]) for r in range(3)])
        now = now + n
        pages = -(-now // page)
        ki = np.concatenate([[0], np.cumsum(pages)])
        ix = np.concatenate([order[base[r]:base[r] + pages[r]] for r in range(3)])
        la = now - (pages - 1) * page
        q_rot = skv.paged_kv_append(k, v, k_cache, v_cache, i32(ip), i32(ki), i32(ix), i32(la), k_scale=k_scale,
                                    v_scale=v_scale, q=q, **rope)
        if step == 0:
            qr, kr = skv.rope_apply(q, k, i32(pos), **rope)
            assert torch.equal(qr, q_rot)
            o, lse, _ = skv.prompt_attention(qr, kr, v, ip)
        else:
            o, lse, _ = skv.paged_attention_scaled(q_rot, k_cache, v_cache, k_scale, v_scale, ip, ki, i32(ix), la, causal=True)
        kn, vn, qn = (OS.rotate(k.double().cpu().numpy(), pos, f, "interleaved", mscale), v.double().cpu().numpy(),
                      OS.rotate(q.double().cpu().numpy(), pos, f, "interleaved", mscale))
        K = [np.concatenate([K[r], kn[ip[r]:ip[r + 1]]]) for r in range(3)]
        V = [np.concatenate([V[r], vn[ip[r]:ip[r + 1]]]) for r in range(3)]
        O, _, _, _ = OS.packed_attention(qn, lambda r: K[r], lambda r: V[r], ip, now, hk, True, d ** -0.5)
        rel = np.linalg.norm(o.cpu().numpy() - O) / np.linalg.norm(O)
        # bf16 rotated rows and weights (2^-8 each) in the prompt; half a 127th of about 4 sigma in the int8 cache
        assert rel < (2.0 ** -6 if step == 0 else 4 / 127), (step, rel)


def test_two_captured_steps_side_by_side():
    """Two graphs of a whole step (append, rotation, both attentions) replayed on two streams at once."""
    lens, page, hq, hk, d = np.array([37, 130]), 16, 8, 2, 128
    n, pages = int(lens.sum()), -(-lens // page)
    qo, ki, la = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(pages)]), lens - (pages - 1) * page
    i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)  # noqa: E731
    qo_d, ki_d, ids, la_d = i32(qo), i32(ki), i32(np.arange(ki[-1])), i32(la)
    pos = i32(np.concatenate([np.arange(x) for x in lens]))
    scaled = skv.plan_paged_scaled(qo, ki, la, page, hq, hk, d, True).to(DEV)
    packed = skv.plan_prompt(qo, None, hq, hk, d, True).to(DEV)

    def make(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = [torch.randn(n, h, d, device=DEV, generator=g).bfloat16() for h in (hq, hk, hk)]
        x += [torch.zeros(int(ki[-1]), page, hk, d, dtype=torch.int8, device=DEV) for _ in range(2)]
        return x + [torch.zeros(int(ki[-1]), 2, hk, device=DEV) for _ in range(2)]

    def step(q, k, v, kc, vc, ks, vs):
        qr = skv.paged_kv_append(k, v, kc, vc, qo_d, ki_d, ids, la_d, k_scale=ks, v_scale=vs, q=q, rope_dim=d)
        _, kr = skv.rope_apply(None, k, pos)
        a = skv.paged_attention_scaled(qr, kc, vc, ks, vs, qo, ki, ids, la, causal=True, plan=scaled, kv_indptr=ki_d,
                                       kv_last_page_len=la_d)
        b = skv.prompt_attention(qr, kr, v, qo, plan=packed)
        return a[0], a[1], b[0], b[1]

    sets = [make(1), make(2)]
    want = [[t.clone() for t in step(*s)] for s in sets]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in sets], [], []
    for s, stream in zip(sets, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            outs.append(step(*s))
    for _ in range(10):
        for s in sets:
            for t in s[3:]:
                t.zero_()
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for x, y in zip(o, w):
                assert torch.equal(x, y)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 128), (3, 3, 64), (1, 1, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", [([300], [300]), ([40, 7], [260, 300])])
def test_keys_of_one_value_return_it(hq, hk, d, q_lens, kv_lens):
    """Every key of a KV head has the same V, and a few scores of a row within the 2^8 by which the running maximum may
    lag outweigh the others: the weights' rounding, to 2^-8 each, has to come out again in the divisor.  What is
    left is fp32: L products and additions in the numerator, L additions in the divisor (2^-24 each; twice that for the
    tensor cores' sums), the reciprocal, its product and a merge."""
    for seed, boost in ((22, 1.0), (23, 3.0), (24, 6.0)):
        c = Case(seed, q_lens, kv_lens, hq, hk, d, boost=boost)
        c.v[:] = c.v[:1].clone()
        for causal in (True, False):
            o, lse, _ = c.run(causal)
            want = c.v[0].double().repeat_interleave(hq // hk, dim=0)[None]
            tol = want.abs() * (3 * 300 + 8) * 2.0 ** -24
            err = (o.double() - want).abs()
            assert bool(torch.all(err <= tol)), (boost, causal, float((err / tol).max()))
            c.check(o, lse, causal)


def test_keys_of_one_value_over_cut_keys():
    c = Case(25, [60], [6000], 4, 1, 128, boost=4.0)
    c.v[:] = c.v[:1].clone()
    o, lse, ex = c.run(True)
    assert ex["plan"].info.max_splits > 1
    want = c.v[0].double().expand(60, 4, 128)
    assert bool(torch.all((o.double() - want).abs() <= want.abs() * (3 * 6000 + 16) * 2.0 ** -24))
