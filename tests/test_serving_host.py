"""Rotary frequencies and the argument checks of skv_rope_apply and skv_paged_kv_append, without a
GPU: every refusal returns before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import oracle.serving as OS
import split_kv_merge_b200 as skv

PTR = 0x10000  # never dereferenced: a refused call launches nothing


def _rope_params(**kw):
    rope = dict(dim=64, layout=0, theta=10000.0, inv_freq_h=None, mscale=1.0)
    rope.update({k[5:]: v for k, v in kw.items() if k.startswith("rope_")})
    p = dict(q=PTR, q_out=2 * PTR, k=3 * PTR, k_out=4 * PTR, q_stride=(512, 64), q_out_stride=(512, 64),
             k_stride=(128, 64), k_out_stride=(128, 64), positions=5 * PTR, num_tokens=3, num_q_heads=8, num_k_heads=2,
             head_dim=64, dtype=skv.BF16, inverse=0)
    p.update({k: v for k, v in kw.items() if not k.startswith("rope_")})
    return skv.RopeParams(rope=skv.Rope(**rope), **p)


def _append_params(**kw):
    rope = dict(dim=64, layout=1, theta=10000.0, inv_freq_h=None, mscale=1.0)
    rope.update({k[5:]: v for k, v in kw.items() if k.startswith("rope_")})
    p = dict(k=PTR, v=PTR, k_row_stride=(128, 64), v_row_stride=(128, 64), k_cache=PTR, v_cache=PTR,
             k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), kv_dtype=skv.BF16, kv_scale=1.0, block_tokens=0,
             k_scale=PTR, v_scale=PTR, k_scale_stride=(2, 2, 1), v_scale_stride=(2, 2, 1), append_indptr=PTR,
             kv_indptr=PTR, kv_indices=PTR, kv_last_page_len=PTR, positions=None, batch=2, num_rows=5, num_pages=9,
             page_size=16, num_kv_heads=2, head_dim=64, q=PTR, q_out=2 * PTR, q_stride=(512, 64),
             q_out_stride=(512, 64), num_q_heads=8, status=None)
    p.update({k: v for k, v in kw.items() if not k.startswith("rope_")})
    return skv.AppendParams(rope=skv.Rope(**rope), **p)


@pytest.mark.parametrize("change,code", [
    (dict(num_tokens=-1), skv.ERR_INVALID), (dict(num_q_heads=-1), skv.ERR_INVALID), (dict(head_dim=0), skv.ERR_INVALID),
    (dict(head_dim=68), skv.ERR_UNSUPPORTED), (dict(head_dim=2048), skv.ERR_UNSUPPORTED),
    (dict(dtype=skv.E4M3), skv.ERR_UNSUPPORTED), (dict(rope_dim=-16), skv.ERR_INVALID),
    (dict(rope_dim=80), skv.ERR_INVALID), (dict(rope_dim=24), skv.ERR_UNSUPPORTED),
    (dict(head_dim=512, rope_dim=512), skv.ERR_UNSUPPORTED), (dict(rope_layout=2), skv.ERR_INVALID),
    (dict(rope_theta=0.0), skv.ERR_INVALID), (dict(rope_theta=math.inf), skv.ERR_INVALID),
    (dict(rope_mscale=0.0), skv.ERR_INVALID), (dict(rope_mscale=math.nan), skv.ERR_INVALID),
    (dict(q=None), skv.ERR_INVALID), (dict(k_out=None), skv.ERR_INVALID), (dict(positions=None), skv.ERR_INVALID),
    (dict(q=PTR + 2), skv.ERR_ALIGNMENT), (dict(q_stride=(516, 64)), skv.ERR_ALIGNMENT),
    (dict(k_stride=(-128, 64)), skv.ERR_INVALID), (dict(q_out=PTR, q_out_stride=(1024, 64)), skv.ERR_INVALID),
    (dict(num_tokens=0), skv.OK), (dict(num_q_heads=0, num_k_heads=0), skv.OK),
])
def test_rope_apply_refusals(change, code):
    assert skv._rope_apply(ctypes.byref(_rope_params(**change)), None) == code


def test_rope_apply_refuses_frequencies_that_are_not_finite():
    f = np.ones(32)
    f[7] = np.nan
    assert skv._rope_apply(ctypes.byref(_rope_params(rope_inv_freq_h=f.ctypes.data)), None) == skv.ERR_INVALID


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), skv.ERR_INVALID), (dict(page_size=0), skv.ERR_INVALID), (dict(num_kv_heads=0), skv.ERR_INVALID),
    (dict(head_dim=96), skv.ERR_UNSUPPORTED), (dict(kv_dtype=skv.F32), skv.ERR_UNSUPPORTED),
    (dict(kv_dtype=skv.I8), skv.ERR_UNSUPPORTED), (dict(kv_dtype=skv.E4M3, kv_scale=0.0), skv.ERR_INVALID),
    (dict(kv_dtype=skv.E4M3, kv_scale=math.nan), skv.ERR_INVALID),
    (dict(kv_dtype=skv.E4M3, kv_scale=1e-40), skv.ERR_INVALID), (dict(block_tokens=16), skv.ERR_INVALID),
    (dict(kv_dtype=skv.I8, block_tokens=5), skv.ERR_INVALID), (dict(kv_dtype=skv.I8, block_tokens=-1), skv.ERR_INVALID),
    (dict(kv_dtype=skv.I8, block_tokens=512, page_size=512), skv.ERR_UNSUPPORTED),
    (dict(kv_dtype=skv.I8, block_tokens=16, k_scale=None), skv.ERR_INVALID),
    (dict(kv_dtype=skv.I8, block_tokens=16, v_scale_stride=(2, -2, 1)), skv.ERR_INVALID),
    (dict(kv_dtype=skv.I8, block_tokens=16, k_stride=(2048, 128, 72)), skv.ERR_ALIGNMENT),
    (dict(rope_dim=40), skv.ERR_UNSUPPORTED), (dict(rope_layout=-1), skv.ERR_INVALID), (dict(k=None), skv.ERR_INVALID),
    (dict(v_row_stride=(128, 60)), skv.ERR_ALIGNMENT), (dict(append_indptr=None), skv.ERR_INVALID),
    (dict(kv_indices=None), skv.ERR_INVALID), (dict(k_cache=PTR + 8), skv.ERR_ALIGNMENT),
    (dict(v_stride=(-2048, 128, 64)), skv.ERR_INVALID), (dict(q=None), skv.ERR_INVALID),
    (dict(q_out=PTR, q_out_stride=(520, 64)), skv.ERR_INVALID), (dict(num_rows=0), skv.OK), (dict(batch=0), skv.OK),
])
def test_append_refusals(change, code):
    assert skv._kv_append(ctypes.byref(_append_params(**change)), None) == code


@pytest.mark.parametrize("change", [dict(q_out_stride=(0, 64)), dict(q_out_stride=(512, 0)), dict(k_out_stride=(128, 0))])
def test_rotated_rows_need_places_of_their_own(change):
    assert skv._rope_apply(ctypes.byref(_rope_params(**change)), None) == skv.ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(q_out_stride=(0, 64)), dict(k_stride=(0, 128, 64)), dict(v_stride=(2048, 0, 64)), dict(k_stride=(2048, 128, 0)),
    dict(kv_dtype=skv.I8, block_tokens=8, k_scale_stride=(0, 2, 1)),
    dict(kv_dtype=skv.I8, block_tokens=8, v_scale_stride=(4, 0, 1)),
    dict(kv_dtype=skv.E4M3, block_tokens=8, v_scale_stride=(4, 2, 0))])
def test_appended_rows_and_scales_need_places_of_their_own(change):
    assert skv._kv_append(ctypes.byref(_append_params(**change)), None) == skv.ERR_INVALID


def test_null_params():
    assert skv._rope_apply(None, None) == skv.ERR_INVALID
    assert skv._kv_append(None, None) == skv.ERR_INVALID


def test_python_checks():
    torch = pytest.importorskip("torch")
    x, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (lambda: skv.rope_apply(x, None, pos),                         # not on a CUDA device
                lambda: skv.rope_apply(None, None, pos), lambda: skv.rope_apply(x.half(), None, pos),
                lambda: skv.rope_apply(x, None, pos.long()), lambda: skv.rope_apply(x, None, pos[:2]),
                lambda: skv.rope_frequencies(64, scaling="cubic")):
        with pytest.raises(ValueError):
            bad()
    cache, ip = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(k_scale=torch.zeros(4, 1, 2)), dict(q=torch.zeros(3, 4, 32)), dict(num_pages=5),
               dict(positions=pos[:1]), dict()):
        with pytest.raises(ValueError):
            skv.paged_kv_append(x, x, cache, cache, ip, ip, ip, ip[:1], **kw)


def _wavelength_turns(f, context):
    return context * f / (2 * math.pi)


def test_rope_frequencies():
    dim, theta, ctx, factor = 128, 10000.0, 4096, 8.0
    plain = np.array([theta ** (-2 * i / dim) for i in range(dim // 2)])
    f, m = skv.rope_frequencies(dim, theta)
    assert m == 1.0 and np.allclose(f, plain, rtol=1e-14, atol=0)
    f, _ = skv.rope_frequencies(dim, theta, "linear", factor)
    assert np.allclose(f, plain / factor, rtol=1e-14, atol=0)
    # a larger base that leaves the fastest pair and divides the slowest by the factor
    f, _ = skv.rope_frequencies(dim, theta, "ntk", factor)
    assert f[0] == 1.0 and np.isclose(f[-1], plain[-1] / factor, rtol=1e-12)
    for name, low, high in (("yarn", 1.0, 32.0), ("bands", 1.0, 4.0)):
        f, m = skv.rope_frequencies(dim, theta, name, factor, ctx)
        assert np.isclose(m, 0.1 * math.log(factor) + 1 if name == "yarn" else 1.0, rtol=1e-6)
        turns = _wavelength_turns(plain, ctx)
        kept, stretched = turns > high * 1.2, turns < low / 1.2   # a pair of the ramp's rounding either side
        assert kept.any() and stretched.any()
        assert np.allclose(f[kept], plain[kept], rtol=1e-14) and np.allclose(f[stretched], plain[stretched] / factor)
        assert np.all(np.diff(f) < 0) and np.all(f <= plain) and np.all(f >= plain / factor * (1 - 1e-12))
    i = int(np.argmin(np.abs(_wavelength_turns(plain, ctx) - 2.0)))
    kept = (_wavelength_turns(plain, ctx)[i] - 1) / 3
    assert np.isclose(skv.rope_frequencies(dim, theta, "bands", factor, ctx)[0][i],
                      plain[i] * (kept + (1 - kept) / factor), rtol=1e-12)


@pytest.mark.parametrize("args", [(63,), (0,), (64, 1.0), (64, 1e4, 9), (64, 1e4, 1, 0.5), (2, 1e4, 2, 2.0),
                                  (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096, 4.0, 4.0), (64, math.nan)])
def test_rope_frequencies_refusals(args):
    full = list(args) + [1e4, 0, 1.0, 4096.0, 1.0, 32.0][len(args) - 1:]
    assert skv._rope_frequencies(*full, None, None) == skv.ERR_INVALID


def test_oracle_rotation_is_a_rotation():
    """The oracle's rotation against complex multiplication, and its reduction of far angles."""
    rng = np.random.default_rng(3)
    x, pos, f = rng.standard_normal((5, 2, 24)), [0, 1, -7, 12345, 2 ** 30 + 1], np.array([1.0, 0.37, 1e-3, 2.5, 0.01, 7e-5, 0.2, 3.0])
    for layout in ("interleaved", "halves"):
        a, b = OS.pair_columns(layout, 16)
        y = OS.rotate(x, pos, f, layout, 1.5)
        z = (x[..., a] + 1j * x[..., b]) * 1.5 * np.exp(1j * np.remainder(np.outer(pos, f).astype(np.longdouble), 2 * np.pi).astype(float))[:, None]
        assert np.allclose(y[:4, :, a], z.real[:4], atol=1e-10) and np.allclose(y[:4, :, b], z.imag[:4], atol=1e-10)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(OS.rotate(y, pos, f, layout, 1 / 1.5, inverse=True), x, atol=1e-12)


def c_layout(pairs):
    """Sizes and field offsets of C structs of include/splitkv.h, compiled with gcc, against ctypes."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "splitkv.h"', "int main(void) {"]
    for cls, name in pairs:
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        lines += [f'  printf("%zu %zu\\n", offsetof({name}, {f}), sizeof((({name}*)0)->{f}));' for f, _ in cls._fields_]
    d = os.path.join(root, "_build", "c_tests")
    os.makedirs(d, exist_ok=True)
    src, exe = os.path.join(d, "serving_layout.c"), os.path.join(d, "serving_layout")
    with open(src, "w") as f:
        f.write("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    want = []
    for cls, _ in pairs:
        want.append(str(ctypes.sizeof(cls)))
        want += [f"{getattr(cls, f).offset} {getattr(cls, f).size}" for f, _ in cls._fields_]
    return got, want


def test_struct_layouts():
    import shutil
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    got, want = c_layout([(skv.Rope, "skv_rope"), (skv.RopeParams, "skv_rope_params"),
                          (skv.AppendParams, "skv_append_params")])
    assert got == want


def _plan_scaled(**kw):
    a = dict(batch=2, qo=[0, 1, 2], kv=[0, 3, 5], last=[4, 16], page=16, hq=8, hk=2, d=64, causal=0, policy=0, param=0)
    a.update(kw)
    arrays = [None if a[k] is None else np.asarray(a[k], dtype=np.int32) for k in ("qo", "kv", "last")]
    info, plan = skv.PlanInfo(), np.zeros(4096, np.int32)
    code = skv._plan_scaled(a["batch"], *[skv._ptr_i32(x) for x in arrays], a["page"], a["hq"], a["hk"], a["d"],
                            a["causal"], a["policy"], a["param"], None, None, skv._ptr_i32(plan), plan.size,
                            ctypes.byref(info))
    return code, plan, info


@pytest.mark.parametrize("change,code", [
    (dict(), skv.OK), (dict(batch=-1), skv.ERR_INVALID), (dict(qo=None), skv.ERR_INVALID), (dict(kv=None), skv.ERR_INVALID),
    (dict(qo=[1, 2, 3]), skv.ERR_INVALID), (dict(qo=[0, 2, 1]), skv.ERR_INVALID), (dict(kv=[0, 3, 2]), skv.ERR_INVALID),
    (dict(last=[17, 1]), skv.ERR_INVALID), (dict(hq=7), skv.ERR_INVALID), (dict(hk=0), skv.ERR_INVALID),
    (dict(d=96), skv.ERR_UNSUPPORTED), (dict(policy=9), skv.ERR_INVALID), (dict(policy=1, param=0), skv.ERR_INVALID),
    (dict(hq=131072, hk=65536), skv.ERR_UNSUPPORTED), (dict(page=0), skv.ERR_INVALID),
])
def test_plan_scaled_refusals(change, code):
    assert _plan_scaled(**change)[0] == code


@pytest.mark.parametrize("hq,hk,q_len,tile", [(8, 8, 1, 8), (64, 8, 1, 1), (32, 8, 4, 4), (64, 8, 4, 2), (40, 2, 3, 1),
                                              (6, 2, 9, 5), (24, 1, 2, 1)])
def test_plan_scaled_items(hq, hk, q_len, tile):
    """Every (query token, key page) of a request is in one item; causal limits count from the item's first token."""
    for causal in (0, 1):
        code, plan, info = _plan_scaled(qo=[0, q_len, 2 * q_len], hq=hq, hk=hk, causal=causal, policy=2, param=148)
        assert code == skv.OK and info.kernel == 5 and info.q_tile == tile
        seen = np.zeros((2 * q_len, 5), int)
        for r, q0, n, p0, p1, _, _, limit in plan[:8 * info.num_work].reshape(-1, 8):
            assert n <= tile
            seen[q0:q0 + n, [0, 3][r] + p0:[0, 3][r] + p1] += 1
            assert limit == ([36, 32][r] - q_len + q0 - r * q_len + 1 if causal else 1 << 30)
        assert np.all(seen[:q_len, :3] == 1) and np.all(seen[q_len:, 3:] == 1) and seen.sum() == 5 * q_len


def _scaled_params(**kw):
    base = dict(q=PTR, k_cache=PTR, v_cache=PTR, k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), kv_indptr=PTR,
                kv_indices=PTR, kv_last_page_len=PTR, batch=2, total_q=2, num_pages=5, page_size=16, num_qo_heads=8,
                num_kv_heads=2, head_dim=64, sm_scale=0.1, o=PTR, o_dtype=skv.F32, lse=PTR, o_part=PTR, lse_part=PTR,
                status=None, kv_dtype=skv.I8, kv_scale=1.0)
    top = dict(k_scale=PTR, v_scale=PTR, k_scale_stride=(2, 2, 1), v_scale_stride=(2, 2, 1), block_tokens=16)
    for k, v in kw.items():
        (base if k in base else top)[k] = v
    return skv.PagedScaledParams(base=skv.PagedParams(**base), **top)


@pytest.mark.parametrize("change,code", [
    (dict(kv_dtype=skv.BF16), skv.ERR_UNSUPPORTED), (dict(head_dim=32), skv.ERR_UNSUPPORTED),
    (dict(num_qo_heads=7), skv.ERR_INVALID), (dict(o_dtype=skv.E4M3), skv.ERR_UNSUPPORTED),
    (dict(block_tokens=0), skv.ERR_INVALID), (dict(block_tokens=5), skv.ERR_INVALID), (dict(q=None), skv.ERR_INVALID),
    (dict(k_scale=None), skv.ERR_INVALID), (dict(v_scale_stride=(-2, 2, 1)), skv.ERR_INVALID),
    (dict(k_stride=(2048, 128, 72)), skv.ERR_ALIGNMENT), (dict(v_stride=(-2048, 128, 64)), skv.ERR_INVALID),
    (dict(v_cache=PTR + 8), skv.ERR_ALIGNMENT), (dict(q=PTR + 2), skv.ERR_ALIGNMENT),
    (dict(o_part=None), skv.ERR_WORKSPACE), (dict(kv_indices=None), skv.ERR_INVALID), (dict(batch=-1), skv.ERR_INVALID),
    (dict(num_qo_heads=64), skv.ERR_INVALID),           # a plan for another group
])
def test_scaled_fwd_refusals(change, code):
    _, plan, info = _plan_scaled(qo=[0, 4, 8], policy=1, param=2)
    assert info.num_partial_rows > 0
    p = _scaled_params(**change)
    assert skv._scaled_fwd(ctypes.byref(p), PTR, ctypes.byref(info), None) == code


def test_plans_run_only_on_their_own_call():
    _, _, info = _plan_scaled()
    assert skv._paged_fwd(ctypes.byref(_scaled_params(kv_dtype=skv.BF16).base), PTR, ctypes.byref(info), None) == skv.ERR_INVALID
    other = skv.plan_paged([0, 1, 2], [0, 3, 5], [4, 16], 16, 8, 2, 64, "none").info
    assert skv._scaled_fwd(ctypes.byref(_scaled_params()), PTR, ctypes.byref(other), None) == skv.ERR_INVALID
    assert skv._scaled_fwd(None, PTR, ctypes.byref(info), None) == skv.ERR_INVALID


def test_scaled_struct_layout():
    import shutil
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    got, want = c_layout([(skv.PagedScaledParams, "skv_paged_scaled_params")])
    assert got == want


def _plan_prompt(qo, kv, hq=4, hk=2, d=64, causal=1, sms=148, batch=None):
    q = None if qo is None else np.asarray(qo, np.int32)
    k = None if kv is None else np.asarray(kv, np.int32)
    info, plan = skv.PlanInfo(), np.zeros(1 << 20, np.int32)
    code = skv._plan_prompt(len(qo) - 1 if batch is None else batch, skv._ptr_i32(q), skv._ptr_i32(k), hq, hk, d, causal,
                            sms, skv._ptr_i32(plan), plan.size, ctypes.byref(info))
    return code, plan, info


@pytest.mark.parametrize("args,kw,code", [
    (([0, 5], None), {}, skv.OK), (([0], None), {}, skv.OK), (([0, 0, 0], [0, 4, 4]), {}, skv.OK),
    (([0, 5], None), dict(batch=-1), skv.ERR_INVALID), ((None, None), dict(batch=1), skv.ERR_INVALID),
    (([1, 5], None), {}, skv.ERR_INVALID), (([0, 5, 3], None), {}, skv.ERR_INVALID),
    (([0, 5], [0, -1]), {}, skv.ERR_INVALID), (([0, 5], [2, 5]), {}, skv.ERR_INVALID),
    (([0, 5], None), dict(hq=5), skv.ERR_INVALID), (([0, 5], None), dict(hk=0), skv.ERR_INVALID),
    (([0, 5], None), dict(d=80), skv.ERR_UNSUPPORTED), (([0, 5], None), dict(sms=-1), skv.ERR_INVALID),
    (([0, 5], None), dict(hq=131072, hk=2), skv.ERR_UNSUPPORTED),
])
def test_plan_prompt_refusals(args, kw, code):
    assert _plan_prompt(*args, **kw)[0] == code


def _covers(hq, hk, causal, q_lens, kv_lens, sms=148):
    """Each (query token, head) meets each key tile that it sees in exactly one item; its partial rows and merge
    items agree; the CTAs' lists hold every item once."""
    kv_lens = q_lens if kv_lens is None else kv_lens
    qo, kv = (np.concatenate([[0], np.cumsum(x)]) for x in (q_lens, kv_lens))
    code, plan, info = _plan_prompt(qo, kv, hq, hk, 64, causal, sms)
    assert code == skv.OK and info.kernel == 6
    items = plan[:16 * info.num_work].reshape(-1, 16)
    merges = plan[16 * info.num_work:16 * info.num_work + 4 * info.num_merge_rows].reshape(-1, 4)
    lists = plan[info.cta_offset:info.cta_offset + info.num_ctas + 1]
    assert lists[0] == 0 and lists[-1] == info.num_work and np.all(np.diff(lists) >= 1) and info.num_ctas <= sms
    merged = {int(m[0]): (int(m[1]), int(m[2])) for m in merges}
    tiles = -(-max(max(kv_lens), 1) // 128)
    met = np.zeros((int(qo[-1]), hq, tiles), int)
    written = np.zeros((max(1, info.num_partial_rows), hq), int)
    direct = np.zeros((int(qo[-1]), hq), int)
    for w in items:
        q0a, q0b, na, nb, ha, hb, la, lb, kv0, kv_len, t0, t1, part, stride, is_causal, _ = (int(v) for v in w)
        r = int(np.searchsorted(qo, q0a, side="right")) - 1
        assert (kv0, kv_len, is_causal) == (kv[r], kv_lens[r], causal) and ha // (hq // hk) == hb // (hq // hk)
        for q0, n, h, lim in ((q0a, na, ha, la), (q0b, nb, hb, lb)):
            assert 0 <= n <= 128 and q0 + n <= qo[r + 1] or n == 0
            for i in range(n):
                tok = q0 + i
                assert lim + i == kv_lens[r] - q_lens[r] + (tok - qo[r]) + 1
                met[tok, h, t0:t1] += 1
                if part < 0:
                    direct[tok, h] += 1
                else:
                    row = part + (tok - q0a) * stride
                    written[row, h] += 1
                    first, count = merged[tok]
                    assert first <= row < first + count and count == stride
    for tok in range(int(qo[-1])):
        r = int(np.searchsorted(qo, tok, side="right")) - 1
        sees = min(kv_lens[r], kv_lens[r] - q_lens[r] + tok - qo[r] + 1) if causal else kv_lens[r]
        need = -(-max(0, sees) // 128)
        assert np.all(met[tok, :, :need] == 1) and met[tok].max(initial=0) <= 1
        assert np.all(direct[tok] == (0 if tok in merged else 1))
    if info.num_partial_rows:
        assert np.all(written == 1)
        assert sum(c for _, c in merged.values()) == info.num_partial_rows
    return items, lists


@pytest.mark.parametrize("hq,hk", [(4, 2), (3, 1), (5, 5), (8, 1)])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 300, 0, 128, 129], None), ([5, 64, 700], [4000, 20, 900]),
                                            ([100], [30000]), ([7, 3], [0, 2])])
def test_plan_prompt_covers_every_pair_once(hq, hk, causal, q_lens, kv_lens):
    _covers(hq, hk, causal, q_lens, kv_lens)


@pytest.mark.parametrize("hq,hk,q_lens,kv_lens,sms", [(4, 2, [1500], [3600], 20), (3, 1, [1500], [5100], 16),
                                                      (32, 8, [1024], [4000], 100), (2, 1, [900, 700], [4000, 3000], 12)])
def test_plan_prompt_evens_out_uneven_rounds(hq, hk, q_lens, kv_lens, sms):
    """Where whole items leave CTAs one item short, some are cut along the keys, and the longest list shrinks."""
    items, lists = _covers(hq, hk, 1, q_lens, kv_lens, sms)
    whole = len({(int(w[0]), int(w[4])) for w in items})
    assert sms < whole < len(items)
    tiles = items[:, 11] - items[:, 10]
    load = np.array([tiles[a:b].sum() for a, b in zip(lists[:-1], lists[1:])])
    assert load.max() <= 1.15 * tiles.sum() / sms


def _prompt_params(**kw):
    p = dict(q=PTR, k=PTR, v=PTR, q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), total_q=300, total_kv=9000,
             num_qo_heads=4, num_kv_heads=2, head_dim=64, sm_scale=0.1, o=PTR, o_dtype=skv.F32, lse=PTR, o_part=PTR,
             lse_part=PTR, status=None)
    p.update(kw)
    return skv.PromptParams(**p)


@pytest.mark.parametrize("change,code", [
    (dict(total_q=-1), skv.ERR_INVALID), (dict(num_qo_heads=5), skv.ERR_INVALID), (dict(num_kv_heads=0), skv.ERR_INVALID),
    (dict(head_dim=32), skv.ERR_UNSUPPORTED), (dict(o_dtype=skv.I8), skv.ERR_UNSUPPORTED),
    (dict(sm_scale=0.0), skv.ERR_INVALID), (dict(sm_scale=-1.0), skv.ERR_INVALID), (dict(sm_scale=math.inf), skv.ERR_INVALID),
    (dict(q=None), skv.ERR_INVALID), (dict(v=None), skv.ERR_INVALID), (dict(o=None), skv.ERR_INVALID),
    (dict(k=PTR + 2), skv.ERR_ALIGNMENT), (dict(q_stride=(260, 64)), skv.ERR_ALIGNMENT),
    (dict(k_stride=(128, 0)), skv.ERR_INVALID), (dict(v_stride=(-128, 64)), skv.ERR_INVALID),
    (dict(k_stride=(1 << 38, 64)), skv.ERR_UNSUPPORTED), (dict(o_part=None), skv.ERR_WORKSPACE), (dict(total_q=0), skv.OK),
])
def test_prompt_fwd_refusals(change, code):
    _, _, info = _plan_prompt([0, 100], [0, 9000])
    assert info.num_partial_rows > 0
    assert skv._prompt_fwd(ctypes.byref(_prompt_params(**change)), PTR, ctypes.byref(info), None) == code


def test_prompt_fwd_needs_its_own_plan():
    _, _, info = _plan_scaled()
    assert skv._prompt_fwd(ctypes.byref(_prompt_params()), PTR, ctypes.byref(info), None) == skv.ERR_INVALID
    assert skv._prompt_fwd(ctypes.byref(_prompt_params()), PTR, None, None) == skv.ERR_INVALID
    _, _, info = _plan_prompt([0, 5], None)
    assert skv._prompt_fwd(ctypes.byref(_prompt_params()), None, ctypes.byref(info), None) == skv.ERR_INVALID
    assert skv._scaled_fwd(ctypes.byref(_scaled_params()), PTR, ctypes.byref(info), None) == skv.ERR_INVALID
    with pytest.raises(ValueError):
        skv.plan_prompt([0, 5], [0, 5, 6], 4, 2, 64)


def test_a_kept_plan_serves_the_requests_it_was_made_for():
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(9, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    for plan, qo, kv, causal in ((skv.plan_prompt([0, 8], None, 4, 2, 64), [0, 9], None, True),
                                 (skv.plan_prompt([0, 9], None, 8, 2, 64), [0, 9], None, True),
                                 (skv.plan_prompt([0, 9], [0, 8], 4, 2, 64), [0, 9], None, True),
                                 (skv.plan_prompt([0, 9], None, 4, 2, 64), [0, 9], None, False),
                                 (skv.plan_prompt([0, 9], None, 4, 2, 64), [0, 4, 9], None, True)):
        with pytest.raises(ValueError, match="plan was made for"):
            skv.prompt_attention(q, k, k, qo, kv, causal=causal, plan=plan)
    cache, scale = torch.zeros(3, 16, 2, 64, dtype=torch.int8), torch.zeros(3, 1, 2)
    for plan, qo, causal in ((skv.plan_paged_scaled([0, 1], [0, 2], [5], 16, 4, 2, 64), [0, 2], False),
                             (skv.plan_paged_scaled([0, 1], [0, 2], [5], 16, 8, 2, 64), [0, 1], False),
                             (skv.plan_paged_scaled([0, 1], [0, 2], [5], 8, 4, 2, 64), [0, 1], False),
                             (skv.plan_paged_scaled([0, 1], [0, 2], [5], 16, 4, 2, 64), [0, 1], True)):
        with pytest.raises(ValueError, match="plan was made for"):
            skv.paged_attention_scaled(q, cache, cache, scale, scale, qo, [0, 2], None, [5], causal=causal, plan=plan)


def test_prompt_struct_layout():
    import shutil
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    got, want = c_layout([(skv.PromptParams, "skv_prompt_params")])
    assert got == want


def test_a_kept_plan_is_compared_by_every_length():
    """Equal totals are not equal requests: other borders between them, or another length in the last page."""
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(9, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    for made, qo, kv in ((([0, 4, 9], None), [0, 8, 9], None), (([0, 4, 9], [0, 4, 9]), [0, 4, 9], [0, 5, 9]),
                         (([0, 4, 9], None), [0, 4, 9], [0, 8, 9])):
        for causal in (True, False):
            with pytest.raises(ValueError, match="plan was made for"):
                skv.prompt_attention(q, k, k, qo, kv, causal=causal, plan=skv.plan_prompt(*made, 4, 2, 64, causal))
    cache, scale = torch.zeros(3, 16, 2, 64, dtype=torch.int8), torch.zeros(3, 1, 2)
    call = lambda plan, qo, ki, la, causal: skv.paged_attention_scaled(  # noqa: E731
        q, cache, cache, scale, scale, qo, ki, None, la, causal=causal, plan=plan)
    for made, now, causal in ((([0, 1, 3], [0, 1, 3], [5, 5]), ([0, 2, 3], [0, 1, 3], [5, 5]), False),
                              (([0, 1, 2], [0, 1, 3], [5, 5]), ([0, 1, 2], [0, 2, 3], [5, 5]), False),
                              (([0, 1, 2], [0, 1, 3], [5, 5]), ([0, 1, 2], [0, 1, 3], [5, 6]), True),
                              (([0, 1, 2], [0, 1, 3], [6, 4]), ([0, 1, 2], [0, 1, 3], [5, 5]), True)):
        with pytest.raises(ValueError, match="plan was made for"):
            call(skv.plan_paged_scaled(*made, 16, 4, 2, 64, causal), *now, causal)


def test_a_kept_plan_serves_equal_lengths_however_they_are_held():
    """The comparison passes (these tensors are then refused for not being on a GPU)."""
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(9, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    as_tensor = lambda a: torch.tensor(a)  # noqa: E731
    plan = skv.plan_prompt([0, 4, 9], None, 4, 2, 64)
    plan.device = torch.zeros(1, dtype=torch.int32)
    for hold in (list, tuple, np.asarray, as_tensor):
        for kv in (None, hold([0, 4, 9])):
            with pytest.raises(ValueError, match="CUDA device"):
                skv.prompt_attention(q, k, k, hold([0, 4, 9]), kv, plan=plan)
    cache, scale = torch.zeros(3, 16, 2, 64, dtype=torch.int8), torch.zeros(3, 1, 2)
    ids = torch.arange(3, dtype=torch.int32)
    for causal, last in ((True, [5, 5]), (False, [5, 5]), (False, [5, 6])):   # not causal: the last page may fill
        plan = skv.plan_paged_scaled([0, 1, 2], [0, 1, 3], [5, 5], 16, 4, 2, 64, causal)
        plan.device = torch.zeros(1, dtype=torch.int32)
        with pytest.raises(ValueError, match="CUDA device"):
            skv.paged_attention_scaled(q, cache, cache, scale, scale, np.array([0, 1, 2]), [0, 1, 3], ids, last,
                                       causal=causal, plan=plan)


@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_scaled_fwd_refuses_a_softmax_scale_that_is_not_finite(scale):
    _, _, info = _plan_scaled(qo=[0, 4, 8], policy=1, param=2)
    assert skv._scaled_fwd(ctypes.byref(_scaled_params(sm_scale=scale)), PTR, ctypes.byref(info), None) == skv.ERR_INVALID


def test_scaled_attention_needs_every_page_id_that_the_table_names():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache, scale = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 1, 2)
    plan = skv.plan_paged_scaled([0, 1, 2], [0, 1, 3], [5, 5], 16, 4, 2, 64)
    plan.device = torch.zeros(1, dtype=torch.int32)
    for n, why in ((2, "kv_indices"), (0, "kv_indices"), (3, "CUDA device"), (4, "CUDA device")):
        for kept in (plan, None):
            with pytest.raises(ValueError, match=why):
                skv.paged_attention_scaled(q, cache, cache, scale, scale, [0, 1, 2], [0, 1, 3],
                                           torch.zeros(n, dtype=torch.int32), [5, 5], plan=kept)
    with pytest.raises(ValueError, match="kv_indices"):
        skv.paged_attention_scaled(q, cache, cache, scale, scale, [0, 1, 2], [0, 1, 3], None, [5, 5], plan=plan)


@pytest.mark.parametrize("change,code", [
    (dict(q_out_stride=(512, 56)), skv.ERR_INVALID),                            # heads of 64 values, 56 apart
    (dict(q_out_stride=(448, 64)), skv.ERR_INVALID),                            # tokens of 8 x 64, 448 apart
    (dict(q_out_stride=(64, 128)), skv.ERR_INVALID),                            # 3 tokens inside 2 heads' distance
    (dict(k_out_stride=(120, 64)), skv.ERR_INVALID), (dict(k_out_stride=(1 << 62, 1 << 62)), skv.ERR_INVALID),
])
def test_rotated_rows_may_not_overlap(change, code):
    assert skv._rope_apply(ctypes.byref(_rope_params(**change)), None) == code


@pytest.mark.parametrize("change", [
    dict(k_stride=(2048, 64, 64)), dict(k_stride=(1920, 128, 64)), dict(v_stride=(2048, 128, 48)),
    dict(v_stride=(64, 1024, 512)), dict(q_out_stride=(496, 64)), dict(k_stride=(1 << 61, 1 << 61, 64)),
    dict(kv_dtype=skv.I8, block_tokens=8, k_scale_stride=(3, 2, 1)),
    dict(kv_dtype=skv.I8, block_tokens=8, v_scale_stride=(4, 1, 1)),
    dict(kv_dtype=skv.E4M3, block_tokens=4, v_scale_stride=(2, 18, 3))])
def test_appended_rows_and_scales_may_not_overlap(change):
    assert skv._kv_append(ctypes.byref(_append_params(**change)), None) == skv.ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(), dict(k_stride=(4096, 256, 128), v_stride=(4096, 256, 128)),         # K and V side by side
    dict(k_stride=(2048, 64, 1024)), dict(k_stride=(64, 1152, 576)),            # heads, or pages, innermost
    dict(kv_dtype=skv.I8, block_tokens=8, k_scale_stride=(8, 4, 2), v_scale_stride=(1, 18, 9))])
def test_layouts_with_places_of_their_own_are_checked_on(change):
    """These layouts pass: the call goes on to the next refusal (a misaligned q)."""
    p = dict(dict(k_scale_stride=(4, 2, 1), v_scale_stride=(4, 2, 1)), **change)
    assert skv._kv_append(ctypes.byref(_append_params(q=PTR + 2, **p)), None) == skv.ERR_ALIGNMENT
