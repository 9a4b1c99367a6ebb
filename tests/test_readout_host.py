"""What the readout's Python side hands to the library, and what it refuses before that: on the CPU, with tensors that say
they are on a device and the library's calls replaced by recorders (no GPU needed)."""
import pytest
import torch

from hierarchical_kv_routing_tok_b200 import _capi as C
from hierarchical_kv_routing_tok_b200 import build as B
from hierarchical_kv_routing_tok_b200 import readout as RO

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """[(name, positional arguments without the stream)] of the library's calls; nothing runs."""
    B.build()
    out = []
    monkeypatch.setattr(RO, "_launch", lambda fn, device, *args: out.append((fn.__name__, args)))
    monkeypatch.setattr(RO, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    return out


def fused(T=9, Hq=4, Hkv=2, dtype=BF16):
    q, k, v = torch.randn(T, Hq + 2 * Hkv, 128).to(dtype).split([Hq, Hkv, Hkv], dim=1)
    return q, k, v, torch.tensor([0, T], dtype=torch.int32)


def heads(T=9, Hq=4, Hkv=2, dtype=BF16):
    q, k, v = (torch.randn(h, T, 128).to(dtype).transpose(0, 1) for h in (Hq, Hkv, Hkv))
    return q, k, v, torch.tensor([0, T], dtype=torch.int32)


def repack(how):
    """Pack and unpack hooks that keep values and change strides, as activation offload does."""
    def pack(t):
        return t.detach().clone(memory_format=torch.contiguous_format)

    def unpack(t):
        if how == "dense" or t.dim() != 3:
            return t
        wide = torch.zeros(t.shape[0] + 1, t.shape[1] + 3, t.shape[2], dtype=t.dtype)
        wide[:-1, 1:-2] = t
        return wide[:-1, 1:-2]
    return torch.autograd.graph.saved_tensors_hooks(pack, unpack)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", [fused, heads])
@pytest.mark.parametrize("how", ["dense", "wide"])
def test_backward_describes_the_tensors_it_gets(calls, dtype, layout, how):
    q, k, v, cu = layout(dtype=dtype)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    with repack(how):
        o, _ = RO.packed_attention(*leaves, cu, softmax_scale=0.25)
    seen = []
    real = RO._bwd

    def bwd(cfg, q, k, v, *args, **kw):
        seen.extend([q, k, v])
        return real(cfg, q, k, v, *args, **kw)

    with pytest.MonkeyPatch.context() as m:
        m.setattr(RO, "_bwd", bwd)
        torch.autograd.grad(o, leaves, torch.ones_like(o))
    name, args = calls[-1]
    cfg = args[0]
    assert name == "packed_attn_bwd" and abs(cfg.softmax_scale - 0.25) < 1e-7
    got = [(cfg.q_stride_t, cfg.q_stride_h), (cfg.k_stride_t, cfg.k_stride_h), (cfg.v_stride_t, cfg.v_stride_h)]
    assert got == [t.stride()[:2] for t in seen]
    assert list(args[1:4]) == [t.data_ptr() for t in seen]


@pytest.mark.parametrize("T,Hkv", [(9, 2), (1, 2), (9, 1), (0, 2)])
def test_config_and_tensors_agree(calls, T, Hkv):
    """A configuration with the tensors that it was made from, and written by hand with contiguous strides left out."""
    q, k, v, cu = fused(T, 4, Hkv)
    o, lse = RO.packed_attn_fwd(RO.make_packed_config(q, k, v, cu), q, k, v, cu)
    RO.packed_attn_bwd(RO.make_packed_config(q, k, v, cu), q, k, v, cu, o, lse, o)
    q, k, v = (x.contiguous() for x in (q, k, v))
    cfg = C.PackedConfig(4, Hkv, 128, 1, T, dtype=C.HGA_BF16)
    RO.packed_attn_fwd(cfg, q, k, v, cu)
    assert [n for n, _ in calls] == ["packed_attn_fwd", "packed_attn_bwd", "packed_attn_fwd"]


WRONG = {
    "fewer rows": lambda q, k, v, cu: (q[:8], k[:8], v[:8], cu),
    "short k": lambda q, k, v, cu: (q, k[:8], v, cu),
    "heads of q": lambda q, k, v, cu: (q[:, :2], k, v, cu),
    "heads of v": lambda q, k, v, cu: (q, k, v[:, :1], cu),
    "dense q": lambda q, k, v, cu: (q.contiguous(), k, v, cu),
    "dense k": lambda q, k, v, cu: (q, k.contiguous(), v, cu),
    "dense v": lambda q, k, v, cu: (q, k, v.contiguous(), cu),
    "float32": lambda q, k, v, cu: (q.float(), k.float(), v.float(), cu),
    "dtype of k": lambda q, k, v, cu: (q, k.half(), v, cu),
    "more bounds": lambda q, k, v, cu: (q, k, v, torch.zeros(5, dtype=torch.int32)),
    "fewer bounds": lambda q, k, v, cu: (q, k, v, cu[:1]),
    "int64 bounds": lambda q, k, v, cu: (q, k, v, cu.long()),
    "strided bounds": lambda q, k, v, cu: (q, k, v, torch.zeros(4, dtype=torch.int32)[::2]),
    "off a boundary": lambda q, k, v, cu: (q, k, torch.zeros(9 * 1024 + 1, dtype=BF16)[1:].view(9, 8, 128)[:, :2], cu),
}


@pytest.mark.parametrize("what", WRONG)
def test_tensors_that_are_not_the_configurations_are_refused(calls, what):
    q, k, v, cu = fused()
    cfg = RO.make_packed_config(q, k, v, cu)
    o, lse = torch.zeros(9, 4, 128, dtype=BF16), torch.zeros(4, 9)
    args = WRONG[what](q, k, v, cu)
    with pytest.raises(ValueError):
        RO.packed_attn_fwd(cfg, *args)
    with pytest.raises(ValueError):
        RO.packed_attn_bwd(cfg, *args, o, lse, o)
    assert not calls


def ints(max_seqs, max_pages, n_pages):
    return [torch.zeros(s, dtype=torch.int32) for s in ((max_seqs, max_pages), (max_seqs,), (n_pages,))]


@pytest.mark.parametrize("shape,expand", [((1, 6), (3, 6)), ((2, 1), (2, 6)), ((1, 1), (3, 6))], ids=["layers", "pages", "both"])
def test_expanded_pools_are_refused(calls, shape, expand):
    """Layers or pages of one memory, which the library would take for contiguous ones and step behind the pool."""
    pool = torch.zeros(*shape, 2, 16, 128, dtype=BF16).expand(*expand, 2, 16, 128)
    with pytest.raises(ValueError, match="must not share memory"):
        RO.PagedKVCache(pool, pool, *ints(2, 3, expand[1]))


def test_pools_of_one_layer_or_page_may_have_any_stride(calls):
    for shape in ((1, 6), (3, 1), (1, 1)):
        pools = [torch.zeros(*shape, 2, 16, 128, dtype=BF16) for _ in range(2)]
        pools = [x.as_strided(x.shape, [0 if n == 1 else s for n, s in zip(x.shape, x.stride())]) for x in pools]
        RO.PagedKVCache(*pools, *ints(2, 3, shape[1]))


@pytest.mark.parametrize("which", range(3))
def test_forward_mode_is_refused(calls, which):
    import torch.autograd.forward_ad as fw
    q, k, v, cu = fused(dtype=F32)
    with fw.dual_level():
        x = [q, k, v]
        RO.packed_attention(*x, cu)                    # nothing to derive: as outside
        x[which] = fw.make_dual(x[which], torch.ones_like(x[which]))
        del calls[:]
        with pytest.raises(RuntimeError):
            RO.packed_attention(*x, cu)
        with torch.no_grad(), pytest.raises(RuntimeError):
            RO.packed_attention(*x, cu)


def cache(Hkv=2):
    return RO.PagedKVCache(*(torch.zeros(2, 6, Hkv, 16, 128, dtype=BF16) for _ in range(2)), *ints(2, 3, 6))


def test_attend_has_no_backward(calls):
    """A q that requires a gradient: values as ever, and an error where a gradient would be left out."""
    import torch.autograd.forward_ad as fw
    c, rows = cache(), torch.zeros(1, dtype=torch.int32)
    q = torch.randn(1, 4, 128, dtype=BF16)
    o, lse = c.attend(0, q, rows)
    assert not o.requires_grad and not lse.requires_grad
    q.requires_grad_()
    for grad in (True, False):
        with torch.set_grad_enabled(grad):
            o, lse = c.attend(0, q, rows)
        assert o.requires_grad == grad and not lse.requires_grad
        assert calls[-1][1][6] == q.data_ptr()
    o, _ = c.attend(0, q, rows)
    with pytest.raises(RuntimeError, match="no backward pass"):
        o.float().sum().backward()
    assert q.grad is None
    out, lse = torch.zeros(1, 4, 128, dtype=BF16), torch.zeros(1, 4)
    for _ in range(3):
        a, b = c.attend(0, q, rows, o=out, lse=lse)
        assert a is out and b is lse and not a.requires_grad
    with fw.dual_level(), pytest.raises(RuntimeError):
        c.attend(0, fw.make_dual(q.detach(), torch.ones_like(q)), rows)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("grad", [False, True])
def test_workspace_of_packed_attention(calls, given, grad):
    """A given workspace goes to forward and backward and is never cleared; without one each call has its own, cleared."""
    from hierarchical_kv_routing_tok_b200 import new_workspace
    x = [t.detach().requires_grad_(grad) for t in fused()[:3]]
    cu = fused()[3]
    ws = new_workspace(RO.make_packed_config(*x, cu), "cpu") if given else None
    o, _ = RO.packed_attention(*x, cu, workspace=ws)
    if grad:
        torch.autograd.grad(o, x, torch.ones_like(o))
    assert len(calls) == 1 + grad
    for _, args in calls:
        assert args[0].flags == C.HGA_PACKED_FILL_TAIL | (0 if given else C.HGA_PACKED_CLEAR_STATUS)
        assert not given or args[-1] == ws.data_ptr()
    with pytest.raises(ValueError):
        RO.packed_attention(*x, cu, workspace=torch.zeros(16, dtype=torch.uint8))


@pytest.mark.parametrize("scale", [0, 0.0, -1.0, float("nan"), 1e-50, -1e-50, 1e-46, float("inf"), 1e39, 3e38])
def test_scales_that_float32_cannot_hold_are_refused(calls, scale):
    """0 means the default to the library: no other number may become it."""
    q, k, v, cu = fused()
    c = cache()
    with pytest.raises((ValueError, C.HGAError)):
        RO.packed_attention(q, k, v, cu, softmax_scale=scale)
    del calls[:]
    with pytest.raises((ValueError, C.HGAError)):
        c.attend(0, q[:1].contiguous(), torch.zeros(1, dtype=torch.int32), softmax_scale=scale)
        C.paged_attn(*calls[0][1])                     # (the library's own check, before any launch)
    c.attend(0, q[:1].contiguous(), torch.zeros(1, dtype=torch.int32), softmax_scale=1e-44)
    assert calls[-1][1][4] > 0
