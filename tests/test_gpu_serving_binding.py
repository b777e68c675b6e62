"""What the serving calls leave behind them on the Python side: version counters, histories, errors."""
import numpy as np
import pytest
import torch

import split_kv_merge_b200 as skv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


def test_tensors_written_in_place_count_as_modified():
    q = torch.randn(5, 4, 64, device=DEV, requires_grad=True)
    pos = _i32(np.arange(5))
    x = q * 1.0
    y = (x * x).sum()                                        # keeps x for its backward pass
    before = x._version
    skv.rope_apply(x, None, pos, q_out=x)
    assert x._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    k = torch.randn(5, 2, 64, device=DEV, dtype=torch.bfloat16)
    cache = [torch.zeros(1, 16, 2, 64, dtype=torch.int8, device=DEV) for _ in range(2)]
    scale = [torch.zeros(1, 1, 2, device=DEV) for _ in range(2)]
    out = torch.empty(5, 4, 64, device=DEV, dtype=torch.bfloat16)
    written = (*cache, *scale, out)
    before = [t._version for t in written]
    table = _i32([0, 5]), _i32([0, 1]), _i32([0]), _i32([5])
    skv.paged_kv_append(k, k, *cache, *table, k_scale=scale[0], v_scale=scale[1], q=out.clone(), q_out=out, rope_dim=64)
    assert all(t._version > b for t, b in zip(written, before)) and k._version == 0
    o, lse = torch.empty(5, 4, 64, device=DEV), torch.empty(5, 4, device=DEV)
    skv.paged_attention_scaled(out, *cache, *scale, [0, 5], [0, 1], table[2], [5], causal=True, o_out=o, lse_out=lse)
    assert o._version == 1 and lse._version == 1
    skv.prompt_attention(out, k, k, [0, 5], o_out=o, lse_out=lse)
    assert o._version == 2 and lse._version == 2 and cache[0]._version == before[0] + 1


def test_inference_tensors_are_written_as_they_are():
    with torch.inference_mode():
        x = torch.randn(3, 2, 64, device=DEV)
        want, _ = skv.rope_apply(x, None, _i32([0, 1, 2]))
        skv.rope_apply(x, None, _i32([0, 1, 2]), q_out=x)
        assert torch.equal(x, want)
    y = x.clone()
    skv.rope_apply(y, None, _i32([0, 1, 2]), q_out=y)
    skv.rope_apply(x, None, _i32([0, 1, 2]), q_out=x)       # an inference tensor outside inference mode
    assert torch.equal(x, y)


class _Rope(torch.autograd.Function):
    """The way a training program takes gradients through the rotation."""

    @staticmethod
    def forward(ctx, x, pos):
        ctx.save_for_backward(pos)
        return skv.rope_apply(x, None, pos, rope_dim=32, mscale=1.5)[0]

    @staticmethod
    def backward(ctx, g):
        return skv.rope_apply(g.contiguous(), None, *ctx.saved_tensors, rope_dim=32, mscale=1.5, inverse=True)[0], None


def test_no_history_and_the_gradient_by_the_inverse():
    x = torch.randn(7, 3, 64, device=DEV, requires_grad=True)
    pos = _i32([0, 1, 5, 100, 7, 3, 2])
    out, _ = skv.rope_apply(x, None, pos, rope_dim=32, mscale=1.5)
    assert not out.requires_grad and x._version == 0
    w = torch.randn(7, 3, 64, device=DEV)
    (_Rope.apply(x, pos) * w).sum().backward()
    z = x.detach().double().requires_grad_()
    angle = pos.double()[:, None] * (10000.0 ** (-torch.arange(16, device=DEV).double() / 16))
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = z[..., 0:32:2], z[..., 1:32:2]
    turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2) * 1.5
    (torch.cat([turned, z[..., 32:]], -1) * w.double()).sum().backward()
    # fp32 cos, sin, products and their sum: 2^-21 of the pair's |a| + |b|
    size = torch.cat([(w[..., 0:32:2].abs() + w[..., 1:32:2].abs()).repeat_interleave(2, -1) * 1.5, w[..., 32:].abs()], -1)
    assert bool(torch.all((x.grad.double() - z.grad).abs() <= size.double() * 2.0 ** -21))


def test_running_out_of_memory_is_torchs_error():
    """An output of 8.7 TB: torch's allocator refuses it, and nothing is launched."""
    tokens = 1 << 20
    x = torch.zeros(1, 1, 64, device=DEV, dtype=torch.bfloat16).expand(tokens, 65000, 64)
    with pytest.raises(torch.OutOfMemoryError):
        skv.rope_apply(x, None, torch.zeros(tokens, dtype=torch.int32, device=DEV))


def test_a_flag_without_a_truth_value_raises_its_own_error():
    x = torch.zeros(2, 1, 64, device=DEV)
    with pytest.raises(RuntimeError, match="ambiguous"):
        skv.rope_apply(x, None, _i32([0, 1]), inverse=torch.zeros(2))
