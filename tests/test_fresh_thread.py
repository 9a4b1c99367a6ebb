"""Calls from a thread that has made no CUDA call yet (a server's worker, autograd's own thread): the library needs nothing
that an earlier call of the thread would have left there."""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hga():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_kv_routing_tok_b200 as H
    H.load()
    return H


def in_fresh_thread(fn):
    errors = []

    def work():
        try:
            fn()
        except Exception as e:                         # noqa: BLE001 (raised again below)
            errors.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


def randn(*shape, dtype):
    return torch.randn(*shape, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[9, 40, 2, 6], [3000, 2000]], ids=["few tiles", "list"])
def test_packed_attention(hga, dtype, lens):
    T = sum(lens)
    q, k, v, d_o = (randn(T, h, 128, dtype=dtype) for h in (8, 2, 2, 8))
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    cfg = hga.make_packed_config(q, k, v, cu)
    ws = hga.new_workspace(cfg, "cuda")
    o, lse = hga.packed_attn_fwd(cfg, q, k, v, cu, workspace=ws)
    grads = hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, workspace=ws)
    new = [torch.zeros_like(x) for x in (o, lse, *grads)]
    in_fresh_thread(lambda: hga.packed_attn_fwd(cfg, q, k, v, cu, *new[:2], workspace=ws))
    in_fresh_thread(lambda: hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, *new[2:], workspace=ws))
    for a, b in zip(new, (o, lse, *grads)):
        assert torch.equal(a, b)
    assert hga.read_status(ws) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cache(hga, dtype):
    cache = hga.PagedKVCache.new(1, 8, 16, 2, 2, 64, dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rows, k, cu = i32([0, 1]), randn(30, 2, 128, dtype=dtype), i32([0, 20, 30])
    cache.write(0, k, k, cu, rows, cache.reserve(rows, i32([20, 10])))
    q = randn(2, 8, 128, dtype=dtype)
    o, lse = cache.attend(0, q, rows)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    in_fresh_thread(lambda: cache.attend(0, q, rows, o=o2, lse=lse2))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    page = i32([6]), i32([7])
    in_fresh_thread(lambda: cache.copy_pages(*page))
    in_fresh_thread(lambda: cache.free(rows))
    assert cache.status() == 0


def routed(hga, dtype):
    B, Hq, Hkv, H, S = 1, 4, 2, 512, 128
    q, kh, vh, ks, vs = (randn(B, h, n, 128, dtype=dtype) for h, n in ((Hq, S), (Hkv, H), (Hkv, H), (Hkv, S), (Hkv, S)))
    cfg = hga.make_config(q, kh, 4, 8)
    ws = hga.new_workspace(cfg, "cuda")
    gs, cs = hga.build_summaries(cfg, kh)
    _, gi = hga.route(cfg, q, gs, cs, workspace=ws)
    return cfg, ws, (q, kh, vh, ks, vs, gi)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_routed_attention(hga, dtype):
    cfg, ws, x = routed(hga, dtype)
    o, lse = hga.attn_fwd(cfg, *x, workspace=ws)
    d_o = torch.randn_like(o)
    grads = hga.attn_bwd(cfg, *x, o, lse, d_o, workspace=ws)
    new = [torch.zeros_like(t) for t in (o, lse, *grads)]
    in_fresh_thread(lambda: hga.attn_fwd(cfg, *x, *new[:2], workspace=ws))
    in_fresh_thread(lambda: hga.attn_bwd(cfg, *x, o, lse, d_o, *new[2:], workspace=ws))
    for a, b in zip(new, (o, lse, *grads)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd_thread(hga, dtype):
    """The first backward passes of a process, in autograd's thread, with memory from the allocator's cache: in a process of
    its own."""
    code = f"""
import torch, hierarchical_kv_routing_tok_b200 as H
d = torch.{'bfloat16' if dtype is BF16 else 'float32'}
x = [torch.empty(1 << 18, device='cuda') for _ in range(8)]
del x
q, k, v = (torch.randn(57, h, 128, device='cuda').to(d).requires_grad_() for h in (8, 2, 2))
cu = torch.tensor([0, 9, 49, 51, 57], dtype=torch.int32, device='cuda')
o, _ = H.packed_attention(q, k, v, cu)
for g in torch.autograd.grad(o, (q, k, v), torch.randn_like(o)):
    assert torch.isfinite(g).all()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_threads_at_once(hga, dtype):
    """Forward, backward and decoding from two threads, each with its own stream, tensors and cache."""
    work = []
    for lens in ([9, 40, 2, 6], [1500, 700]):
        q, k, v = (randn(sum(lens), h, 128, dtype=dtype).requires_grad_() for h in (8, 2, 2))
        cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        cache = hga.PagedKVCache.new(1, 256, 16, 2, len(lens), 2048, dtype)
        rows = torch.arange(len(lens), dtype=torch.int32, device="cuda")
        add = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cache.write(0, k.detach(), v.detach(), cu, rows, cache.reserve(rows, add))
        new, d_o = randn(len(lens), 8, 128, dtype=dtype), torch.randn_like(q)

        def step(q=q, k=k, v=v, cu=cu, cache=cache, rows=rows, new=new, d_o=d_o):
            o, lse = hga.packed_attention(q, k, v, cu)
            return [o.detach(), lse, *torch.autograd.grad(o, (q, k, v), d_o), *cache.attend(0, new, rows)]

        work.append((step, torch.cuda.Stream()))
    want = [step() for step, _ in work]
    torch.cuda.synchronize()
    errors = []

    def run(i):
        try:
            step, stream = work[i]
            with torch.cuda.stream(stream):
                for _ in range(40):
                    got = step()
                    stream.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except BaseException as e:                     # noqa: BLE001 (raised again below)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]
