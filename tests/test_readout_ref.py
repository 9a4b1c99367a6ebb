"""The float64 attention that the readout tests compare with: its gradients against autograd and
central differences, its rows without keys, and that its bounds are not loose enough to pass a mistake."""
import math

import pytest
import torch

import readout_ref as R


def make(lens, Hq, Hkv, seed=0, dtype=torch.float64):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    return [torch.randn(T, h, 128, generator=g, dtype=torch.float64).to(dtype) for h in (Hq, Hkv, Hkv, Hq)]


def dense(q, k, v, lens):
    G = q.shape[1] // k.shape[1]
    outs, a = [], 0
    for n in lens:
        x, y, z = (t[a:a + n].transpose(0, 1) for t in (q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)))
        outs.append(torch.nn.functional.scaled_dot_product_attention(x, y, z, is_causal=True).transpose(0, 1))
        a += n
    return torch.cat(outs)


@pytest.mark.parametrize("lens,Hq,Hkv", [([7, 1, 0, 12], 4, 2), ([33], 3, 1)])
def test_gradients_match_autograd_and_differences(lens, Hq, Hkv):
    q, k, v, g = make(lens, Hq, Hkv)
    ref = R.packed(q, k, v, lens, d_o=g)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = dense(*leaves, [n for n in lens if n])
    assert torch.allclose(o, ref["o"], atol=1e-12)
    grads = torch.autograd.grad(o, leaves, g)
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert torch.allclose(got, ref[name], atol=1e-11), name
    eps = 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(leaves[i].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(5 + i))
        args = [[x + s * eps * d if j == i else x for j, x in enumerate((q, k, v))] for s in (1, -1)]
        diff = sum(s * (R.packed(*a, lens)["o"] * g).sum().item() for s, a in zip((1, -1), args)) / (2 * eps)
        assert diff == pytest.approx((ref[name] * d).sum().item(), rel=1e-6, abs=1e-7)


def test_rows_without_keys():
    q, k, v, _ = make([3], 2, 2)
    f = R.attend(q.transpose(0, 1), k.transpose(0, 1)[:, :0], v.transpose(0, 1)[:, :0],
                 torch.ones(3, 0, dtype=torch.bool), 0.1, torch.float32)
    assert not f["o"].any() and (f["lse"] == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bounds_catch_a_missing_key(dtype):
    """Leaving out one key of the last row is outside the bounds."""
    lens = [40]
    q, k, v, g = (x.to(dtype) for x in make(lens, 2, 1))
    ref = R.packed(q, k, v, lens, d_o=g)
    R.check(ref["o"].to(dtype), ref, "o")
    bad = ref["o"].clone()
    x = lambda t: t.transpose(0, 1).repeat_interleave(2 // t.shape[1], dim=0)
    mask = torch.ones(40, 40, dtype=torch.bool).tril()
    mask[39, 5] = False
    bad[39] = R.attend(x(q), x(k), x(v), mask, 1 / math.sqrt(128), dtype)["o"][:, 39]
    with pytest.raises(AssertionError):
        R.check(bad.to(dtype), ref, "o")
