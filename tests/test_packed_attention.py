"""Causal attention over packed sequences (hga_packed_attn_fwd / _bwd) on the GPU against the float64
reference, with the bounds of readout_ref."""
import math

import pytest
import torch

import readout_ref as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def hga():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_kv_routing_tok_b200 as H
    H.load()
    return H


def ends(lens):
    e = [0]
    for n in lens:
        e.append(e[-1] + n)
    return torch.tensor(e, dtype=torch.int32, device="cuda")


def rows(gen, T, heads, layout, dtype):
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    if layout == "fused":
        return list(mk(T, sum(heads), 128).split(heads, dim=1))
    if layout == "heads":
        return [mk(h, T, 128).transpose(0, 1) for h in heads]
    if layout == "wide":                   # rows of a wider buffer, every tensor at another offset
        return [mk(T, h + 2, 136)[:, 1:h + 1, 8:] for h in heads]
    return [mk(T, h, 128) for h in heads]


def make(lens, Hq, Hkv, dtype, layout="tokens", tail=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + tail
    q, k, v = rows(gen, T, [Hq, Hkv, Hkv], layout, dtype)
    d_o = torch.randn(T, Hq, 128, generator=gen, device="cuda").to(dtype)
    return q, k, v, d_o


def run(hga, q, k, v, d_o, cu, scale=None):
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o, lse = hga.packed_attention(*leaves, cu, softmax_scale=scale)
    dq, dk, dv = torch.autograd.grad(o, leaves, d_o)
    return {"o": o.detach(), "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def check_all(got, ref):
    for name in ("o", "lse", "dq", "dk", "dv"):
        R.check(got[name], ref, name)


LENS = [[1], [2, 1], [63, 64, 65], [127, 0, 128, 1, 129], [300], [0, 0, 5], [255, 257, 33], [513, 2, 700]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(hga, dtype, lens):
    q, k, v, d_o = make(lens, 8, 2, dtype)
    check_all(run(hga, q, k, v, d_o, ends(lens)), R.packed(q, k, v, lens, d_o=d_o))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (2, 1), (3, 1), (5, 1), (6, 1), (7, 1), (8, 1), (12, 1), (16, 1), (6, 2),
                                    (32, 8), (40, 1)])
def test_heads(hga, dtype, Hq, Hkv):
    lens = [150, 1, 0, 77, 260]
    q, k, v, d_o = make(lens, Hq, Hkv, dtype, seed=Hq)
    check_all(run(hga, q, k, v, d_o, ends(lens)), R.packed(q, k, v, lens, d_o=d_o))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["fused", "heads", "wide"])
def test_layouts_and_tail(hga, dtype, layout):
    lens = [129, 70, 3]
    q, k, v, d_o = make(lens, 4, 2, dtype, layout, tail=9)
    for x in (q, k, v, d_o):               # rows of no sequence: whatever they hold
        x[sum(lens):] = math.nan
    check_all(run(hga, q, k, v, d_o, ends(lens)),
              R.packed(*(x.nan_to_num() for x in (q, k, v)), lens, d_o=d_o.nan_to_num()))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_ragged(hga, dtype):
    lens = [2100, 40, 1025, 1, 333]
    q, k, v, d_o = make(lens, 4, 1, dtype, "fused", tail=100)
    check_all(run(hga, q, k, v, d_o, ends(lens)), R.packed(q, k, v, lens, d_o=d_o))


def test_many_sequences(hga):
    """More sequences than the plan keeps in shared memory."""
    lens = [(7 * i) % 4 for i in range(5000)]
    q, k, v, d_o = make(lens, 2, 1, BF16)
    got = run(hga, q, k, v, d_o, ends(lens))
    starts = ends(lens).tolist()
    for i in list(range(40)) + [2500, 4094, 4095, 4096, 4097, 4998, 4999]:
        a, b = starts[i], starts[i + 1]
        if a < b:
            ref = R.packed(q[a:b], k[a:b], v[a:b], [b - a], d_o=d_o[a:b])
            for name in ("o", "dq", "dk", "dv"):
                R.check(got[name][a:b], ref, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.02, 0.5])
def test_scale(hga, dtype, scale):
    lens = [200, 31]
    q, k, v, d_o = make(lens, 4, 2, dtype, seed=3)
    check_all(run(hga, q, k, v, d_o, ends(lens), scale), R.packed(q, k, v, lens, scale=scale, d_o=d_o))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sequences_do_not_mix(hga, dtype):
    """NaN and infinities in one sequence change no bit of the others."""
    lens = [100, 61, 190, 5]
    q, k, v, d_o = make(lens, 4, 2, dtype)
    clean = run(hga, q, k, v, d_o, ends(lens))
    for x, bad in ((q, math.nan), (k, math.inf), (v, -math.inf), (d_o, math.nan)):
        x[100:161] = bad
    got = run(hga, q, k, v, d_o, ends(lens))
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[100:161] = False
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[name][keep], clean[name][keep]), name
    assert torch.equal(got["lse"][:, keep], clean["lse"][:, keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (2, 2)])
@pytest.mark.parametrize("at", [0, 63, 130, 299])
def test_non_finite_value_reaches_only_later_rows(hga, dtype, Hq, Hkv, at):
    """v of token `at` not finite: rows before it keep their bits, rows from it on get inf / nan there."""
    lens = [10, 300, 4]
    q, k, v, _ = make(lens, Hq, Hkv, dtype, seed=at)
    cu = ends(lens)
    clean, lse0 = hga.packed_attention(q, k, v, cu)
    v[10 + at, 0, 5] = math.inf
    v[10 + at, 0, 77] = math.nan
    o, lse = hga.packed_attention(q, k, v, cu)
    assert torch.equal(lse, lse0)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[10 + at:310, :Hq // Hkv, 5] = True
    hit[10 + at:310, :Hq // Hkv, 77] = True
    assert torch.equal(o[~hit], clean[~hit])
    assert (o[10 + at:310, :Hq // Hkv, 5] == math.inf).all()
    assert o[10 + at:310, :Hq // Hkv, 77].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_scores(hga, dtype):
    """Scores of several thousand: the running maximum keeps the sums finite."""
    lens = [400]
    q, k, v, d_o = make(lens, 2, 1, dtype)
    q *= 64
    k *= 32
    o, lse = hga.packed_attention(q, k, v, ends(lens))
    ref = R.packed(q, k, v, lens)
    assert torch.isfinite(o).all()
    R.check(o, ref, "o")
    R.check(lse, ref, "lse")


def test_given_outputs_keep_their_tail(hga):
    """Outputs that the caller gives: rows of no sequence are left as they were."""
    for dtype in (F32, BF16):
        lens = [70, 0, 59]
        q, k, v, d_o = make(lens, 4, 2, dtype, tail=21)
        cu, n = ends(lens), sum(lens)
        cfg = hga.make_packed_config(q, k, v, cu)
        ws = torch.zeros(hga._capi.packed_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        o, dq, dk, dv = (torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for x in (q, q, k, v))
        lse = torch.full((4, n + 21), 7.0, device="cuda")
        hga.packed_attn_fwd(cfg, q, k, v, cu, o, lse, ws)
        hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, dq, dk, dv, ws)
        ref = R.packed(q, k, v, lens, d_o=d_o)
        for name, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            assert (x[n:] == 7).all(), name
            x[n:] = 0
            R.check(x, ref, name)
        assert (lse[:, n:] == 7).all()
        assert hga.read_status(ws) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [[1, 5, 9], [0, 6, 5], [0, 4, 99], [0, -3, 9]], ids=str)
def test_invalid_bounds_are_recorded(hga, dtype, bad):
    """A cu_seqlens that is not valid computes nothing and is recorded."""
    q, k, v, d_o = make([9], 4, 2, dtype)
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    cfg = hga.make_packed_config(q, k, v, cu)
    ws = torch.zeros(hga._capi.packed_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    o, lse = hga.packed_attn_fwd(cfg, q, k, v, cu, workspace=ws)
    assert hga.read_status(ws) == hga._capi.HGA_ERR_ARG
    assert not o.any() and (lse == -math.inf).all()
    grads = hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, workspace=ws)
    assert hga.read_status(ws) == hga._capi.HGA_ERR_ARG
    assert not any(g.any() for g in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty(hga, dtype):
    for T, cu in ((0, [0]), (0, [0, 0, 0]), (6, [0]), (6, [0, 0])):
        q, k, v, d_o = make([T], 4, 2, dtype)
        got = run(hga, q, k, v, d_o, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert not got["o"].any() and not got["dq"].any() and not got["dk"].any() and not got["dv"].any()
        assert (got["lse"] == -math.inf).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_reproducible_on_another_stream_and_in_a_graph(hga, dtype):
    lens = [260, 1, 129, 64]
    q, k, v, d_o = make(lens, 8, 2, dtype)
    cu = ends(lens)
    want = run(hga, q, k, v, d_o, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(hga, q, k, v, d_o, cu)
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    cfg = hga.make_packed_config(q, k, v, cu)
    ws = torch.zeros(hga._capi.packed_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(want["o"]), torch.zeros_like(want["lse"])
    dq, dk, dv = (torch.zeros_like(want[n]) for n in ("dq", "dk", "dv"))

    def step():
        hga.packed_attn_fwd(cfg, q, k, v, cu, o, lse, ws)
        hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, dq, dk, dv, ws)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    # the graph follows the tensors' content: other lengths, other values
    lens2 = [3, 300, 0, 140]
    cu.copy_(ends(lens2))
    q.copy_(q.flip(0))
    for _ in range(2):
        for x in (o, dq, dk, dv):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref = R.packed(q, k, v, lens2, d_o=d_o)
        for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            R.check(x[:443], {n: ref[n][:443], "e_" + n: ref["e_" + n][:443]}, n)
    assert hga.read_status(ws) == 0


def test_gradient_against_differences(hga):
    """Directional derivatives of the float32 forward: a central difference of step h of a loss computed from
    float32 outputs is off by h^2 f'''/6 and by the outputs' error over h; with |direction| = 1, h = 0.05 the
    float64 reference's own difference shows the first, the output bounds give the second."""
    lens = [90, 33]
    q, k, v, d_o = make(lens, 4, 2, F32)
    cu = ends(lens)
    got = run(hga, q, k, v, d_o, cu)
    h = 0.05
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(got[name].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
        d /= d.norm()
        loss, exact, err = [], [], 0.0
        for s in (1, -1):
            args = [x + s * h * d if j == i else x for j, x in enumerate((q, k, v))]
            ref = R.packed(*args, lens)
            exact.append((ref["o"] * d_o.double()).sum().item())
            err += (ref["e_o"] * d_o.double().abs()).sum().item()
            loss.append((hga.packed_attention(*args, cu)[0].double() * d_o.double()).sum().item())
        along = (got[name].double() * d.double()).sum().item()
        truncation = abs((exact[0] - exact[1]) / (2 * h) - (R.packed(q, k, v, lens, d_o=d_o)[name] * d.double()).sum().item())
        assert abs((loss[0] - loss[1]) / (2 * h) - along) <= truncation + err / (2 * h) + 1e-6


def test_broadcast_gradient(hga):
    """d_o of a sum (stride 0) and k, v that feed two calls: gradients add up."""
    lens = [65, 20]
    q, k, v, _ = make(lens, 4, 2, F32)
    cu = ends(lens)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o1, _ = hga.packed_attention(*leaves, cu)
    o2, _ = hga.packed_attention(*leaves, cu)
    (o1.sum() + o2.sum()).backward()
    once = run(hga, q, k, v, torch.ones_like(q), cu)
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(x.grad, 2 * once[n])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd_in_a_graph(hga, dtype):
    """Forward and backward through autograd, captured while an eager graph of the same leaves is alive: refused where it
    was made on the default stream, and right where on the capture's."""
    lens = [200, 1, 99]
    q, k, v, d_o = make(lens, 4, 2, dtype)
    cu = ends(lens)
    leaves = [x.requires_grad_() for x in (q, k, v)]
    side = torch.cuda.Stream()
    alive = hga.packed_attention(*leaves, cu)          # an eager graph that stays
    want = torch.autograd.grad(hga.packed_attention(*leaves, cu)[0], leaves, d_o)
    side.wait_stream(torch.cuda.current_stream())
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            hga.packed_attention(*leaves, cu)
    for a, b in zip(torch.autograd.grad(alive[0], leaves, d_o), want):
        assert torch.equal(a, b)
    del alive
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        alive = hga.packed_attention(*leaves, cu)
        torch.autograd.grad(hga.packed_attention(*leaves, cu)[0], leaves, d_o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = torch.autograd.grad(hga.packed_attention(*leaves, cu)[0], leaves, d_o)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        late = torch.autograd.grad(alive[0], leaves, d_o)
    torch.cuda.synchronize()
    for a, b in zip(late, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_seqs,tail", [(1, 0), (30, 3), (31, 0), (31, 70), (32, 0), (32, 9), (33, 5)])
def test_number_of_sequences(hga, dtype, n_seqs, tail):
    """Few tiles of up to 31 sequences are found by the kernels themselves, others by a list: one result."""
    lens = [(37 * i * i + 11 * i) % 23 if i % 3 else 0 for i in range(n_seqs - 1)] + [130]
    q, k, v, d_o = make(lens, 2, 1, dtype, tail=tail)
    check_all(run(hga, q, k, v, d_o, ends(lens)), R.packed(q, k, v, lens, d_o=d_o))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_seqs", [3, 40])
def test_bad_bounds_fill_everything(hga, dtype, n_seqs):
    lens = [9] * n_seqs
    q, k, v, d_o = make(lens, 2, 1, dtype)
    for bad in (lambda c: c[0].fill_(1), lambda c: c[2].fill_(5), lambda c: c[-1].fill_(q.shape[0] + 1),
                lambda c: c.fill_(-1)):
        cu = ends(lens)
        bad(cu)
        o, lse = hga.packed_attention(q, k, v, cu)
        assert not o.any() and (lse == -float("inf")).all()
        cfg = hga.make_packed_config(q, k, v, cu)
        ws = torch.zeros(hga._capi.packed_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        dq, dk, dv = hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, workspace=ws)
        assert not dq.any() and not dk.any() and not dv.any()
        assert hga.read_status(ws) == hga._capi.HGA_ERR_ARG


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("which", ["q", "k", "v", "qv"])
def test_gradients_of_some_inputs(hga, dtype, which):
    lens = [70, 5, 200]
    q, k, v, d_o = make(lens, 4, 2, dtype)
    cu = ends(lens)
    want = run(hga, q, k, v, d_o, cu)
    x = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
    for n in which:
        x[n].requires_grad_()
    o, lse = hga.packed_attention(x["q"], x["k"], x["v"], cu)
    assert not lse.requires_grad
    o.backward(d_o)
    for n in "qkv":
        if n in which:
            assert torch.equal(x[n].grad, want["d" + n])
        else:
            assert x[n].grad is None


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shared_workspace_in_two_graphs(hga, dtype):
    """Two captured problems over one workspace, replayed in turn, one of each kind of work list."""
    probs, graphs, outs = [], [], []
    for seed, lens in ((0, [33, 20]), (1, [5] * 40 + [300])):
        q, k, v, _ = make(lens, 8, 2, dtype, seed=seed)
        probs.append((q, k, v, ends(lens)))
    cfgs = [hga.make_packed_config(*p) for p in probs]
    ws = torch.zeros(max(hga._capi.packed_workspace_size(c) for c in cfgs), dtype=torch.uint8, device="cuda")
    want = [hga.packed_attention(*p) for p in probs]
    torch.cuda.synchronize()
    for c, p in zip(cfgs, probs):
        outs.append((torch.full_like(p[0], 7), torch.full((8, p[0].shape[0]), 7.0, device="cuda")))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            hga.packed_attn_fwd(c, *p, *outs[-1], workspace=ws)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i][0].fill_(7)
        graphs[i].replay()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    assert hga.read_status(ws) == 0


def test_two_at_once(hga):
    """Two problems on two streams, each with its own workspace, over and over."""
    probs = []
    for seed, lens in ((0, [700, 3, 128]), (1, [1, 400, 77, 512])):
        q, k, v, d_o = make(lens, 8, 2, BF16, seed=seed)
        probs.append((q, k, v, d_o, ends(lens)))
    want = [run(hga, *p) for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (s, p) in enumerate(zip(streams, probs)):
            with torch.cuda.stream(s):
                got[i].append(run(hga, *p))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for n in want[i]:
                assert torch.equal(g[n], want[i][n]), n


def test_more_than_2_31_elements(hga):
    """Offsets beyond 32 bits: the last sequences of 530,000 packed rows of 32 heads."""
    lens = [1000] * 529 + [513, 487]
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, d_o = (torch.randn(T, 32, 128, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    k, v = (torch.randn(T, 1, 128, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    assert q.numel() > 2 ** 31
    got = run(hga, q, k, v, d_o, ends(lens))
    for a, b in ((T - 487, T), (T - 1000, T - 487), (0, 1000)):
        ref = R.packed(q[a:b], k[a:b], v[a:b], [b - a], d_o=d_o[a:b])
        for name in ("o", "dq", "dk", "dv"):
            R.check(got[name][a:b], ref, name)


@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 2, [300, 65]), (4, 4, [2000] * 12)], ids=["paired", "single"])
def test_expired_wait_is_recorded(hga, Hq, Hkv, lens):
    """A wait limit shorter than a tile's load: the kernels give up, say so and return, and the next call is exact."""
    q, k, v, d_o = make(lens, Hq, Hkv, BF16)
    cu = ends(lens)
    cfg = hga.make_packed_config(q, k, v, cu)
    ws = torch.zeros(hga._capi.packed_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    want = run(hga, q, k, v, d_o, cu)
    short = hga.make_packed_config(q, k, v, cu, wait_limit_ns=1)
    hga.packed_attn_fwd(short, q, k, v, cu, workspace=ws)
    assert hga.read_status(ws) == hga._capi.HGA_ERR_TIMEOUT
    o, lse = hga.packed_attn_fwd(cfg, q, k, v, cu, workspace=ws)
    assert hga.read_status(ws) == 0
    hga.packed_attn_bwd(short, q, k, v, cu, o, lse, d_o, workspace=ws)
    assert hga.read_status(ws) == hga._capi.HGA_ERR_TIMEOUT
    got = run(hga, q, k, v, d_o, cu)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_rounding_kept_for_the_backward(hga):
    """o + o_lo is the output to twice the digits, and brings the gradients of short sequences nearer."""
    lens = [5, 3, 2, 7, 1, 4] * 40
    q, k, v, d_o = make(lens, 8, 2, BF16)
    cu = ends(lens)
    cfg = hga.make_packed_config(q, k, v, cu)
    lo = torch.empty_like(q)
    o, lse = hga.packed_attn_fwd(cfg, q, k, v, cu, o_lo=lo)
    ref = R.packed(q, k, v, lens, d_o=d_o)
    assert (lo.abs().float() <= o.abs().float() * 2 ** -8 + 1e-30).all()
    off = []
    for x in (None, lo):
        dq, dk, dv = hga.packed_attn_bwd(cfg, q, k, v, cu, o, lse, d_o, o_lo=x)
        for n, g in (("dq", dq), ("dk", dk), ("dv", dv)):
            R.check(g, ref, n)
        off.append([((g.double() - ref[n]).norm() / ref[n].norm()).item() for n, g in (("dq", dq), ("dk", dk))])
    assert off[1][0] < off[0][0] and off[1][1] < off[0][1]


def test_refusals(hga):
    q, k, v, d_o = make([9], 4, 2, BF16)
    cu = ends([9])
    for args in ((q.half(), k.half(), v.half(), cu), (q, k.float(), v, cu), (q, k, v[:8], cu), (q[:, :3], k, v, cu),
                 (q, k, v, cu.long()), (q, k, v, cu.cpu()), (q.cpu(), k, v, cu), (q[..., :64], k, v, cu),
                 (q, k[:, :1].expand(-1, 2, -1), v, cu), (q.transpose(1, 2).contiguous().transpose(1, 2), k, v, cu)):
        with pytest.raises((ValueError, RuntimeError)):
            hga.packed_attention(*args)
    cfg = hga.make_packed_config(q, k, v, cu)
    with pytest.raises(ValueError):
        hga.packed_attn_fwd(cfg, q, k, v, cu, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        hga.packed_attn_fwd(cfg, q, k, v, cu, o=torch.empty_like(q))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["fused", "heads", "wide"])
@pytest.mark.parametrize("pin", [False, True])
def test_saved_tensors_on_the_host(hga, dtype, layout, pin):
    """Tensors kept on the host between the passes come back with other strides: the same gradients."""
    lens = [129, 0, 70, 3]
    q, k, v, d_o = make(lens, 4, 2, dtype, layout, tail=9)
    want = run(hga, q, k, v, d_o, ends(lens))
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    with torch.autograd.graph.save_on_cpu(pin_memory=pin):
        o, _ = hga.packed_attention(*leaves, ends(lens))
    for got, n in zip(torch.autograd.grad(o, leaves, d_o), ("dq", "dk", "dv")):
        assert torch.equal(got, want[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [0, 1, 63, 130, 299])
def test_largest_numbers_of_the_type(hga, dtype, at):
    """The type's largest and lowest values in v and k of token `at`: finite numbers, which no row before it sees and no
    product with 0 makes infinite.  q and d_o are 0 in those dims, so that scores, dP and delta are what they were."""
    lens, big = [10, 300, 4], torch.finfo(dtype).max
    q, k, v, d_o = make(lens, 4, 2, dtype, seed=at)
    cu, dims = ends(lens), [5, 77]
    q[..., dims] = 0
    d_o[..., dims] = 0
    clean = run(hga, q, k, v, d_o, cu)
    for x in (k, v):
        x[10 + at, 0, 5], x[10 + at, 0, 77] = big, -big
    got = run(hga, q, k, v, d_o, cu)
    ref = R.packed(q, k, v, lens, d_o=d_o)
    # sums in float32 before their last factor: infinite, of the right sign, where they pass the largest float32.  dq =
    # scale (sum ds k): one term of it, ds big, is all that counts here, and dq itself may be less (the scale is 0.088).
    # o = (sum p v) / sum p: in bf16 p is relative to a maximum that is up to 2^8 too small, in float32 p is at most 1; an
    # infinite o makes delta, and with it the sequence's gradients, undefined.
    def over(n, factor):
        x = ref[n].abs() * factor > 0.99 * torch.finfo(F32).max
        assert torch.equal(got[n][x & got[n].isinf()].sign().double(), ref[n][x & got[n].isinf()].sign())
        return x
    assert torch.equal(got["lse"], clean["lse"])
    for n, factor in (("o", 1 if dtype == F32 else 2 ** 8), ("dq", math.sqrt(128)))[:2 if dtype == F32 else 1]:
        hit = torch.zeros_like(got[n], dtype=torch.bool)
        hit[10 + at:310, :2, dims] = True
        assert torch.equal(got[n][~hit], clean[n][~hit]), n
        big_sum = over(n, factor)
        assert (hit | ~big_sum).all() and torch.isfinite(got[n][~big_sum]).all() and not got[n].isnan().any()
        big_sum &= got[n].isinf()
        R.check(got[n].masked_fill(big_sum, 0), {n: ref[n].masked_fill(big_sum, 0), "e_" + n: ref["e_" + n]}, n)
    if dtype == F32:
        for n in ("dk", "dv"):
            assert torch.equal(got[n], clean[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_seqs", [3, 40])
def test_status_of_packed_attention(hga, dtype, n_seqs):
    """With a workspace of the caller's, what forward and backward record can be read, and the results are the same."""
    lens = [9] * n_seqs
    q, k, v, d_o = make(lens, 4, 2, dtype)
    cu = ends(lens)
    want = run(hga, q, k, v, d_o, cu)
    ws = hga.new_workspace(hga.make_packed_config(q, k, v, cu), "cuda")
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o, lse = hga.packed_attention(*leaves, cu, workspace=ws)
    assert hga.read_status(ws) == 0 and torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])
    for g, n in zip(torch.autograd.grad(o, leaves, d_o, retain_graph=True), ("dq", "dk", "dv")):
        assert torch.equal(g, want[n])
    assert hga.read_status(ws) == 0
    bad = cu.clone()
    bad[-1] += 1
    for x in (q, leaves[0]):                           # without and with a graph
        o, lse = hga.packed_attention(x, k, v, bad, workspace=ws)
        hga.packed_attention(q, k, v, cu, workspace=ws)      # (a later call clears nothing)
        assert hga.read_status(ws) == hga._capi.HGA_ERR_ARG
        assert not o.any() and (lse == -math.inf).all()
    dq, = torch.autograd.grad(o, leaves[:1], d_o)
    assert hga.read_status(ws) == hga._capi.HGA_ERR_ARG and not dq.any()
    assert hga.read_status(ws) == 0


def test_norms_of_the_errors(hga):
    """bf16, sequences of up to 128 tokens (one tile on the diagonal each), errors over norms.  Rounding a result to bf16 takes
    r = 1.66e-3 (uniform in half a step, over a normal distribution's mantissas: 1.5e-3 to 1.7e-3).  o and dv: rounded, from
    operands rounded once (P), so at most sqrt(2) r = 2.35e-3, with 6 % for the distribution of P.  dq and dk: dS keeps
    what its rounding took, so r, and the rest (o + o_lo in delta, 2^-17; exp, 2^-22) far below: the limit is half way to the
    sqrt(2) r of a dS without it."""
    lens = [128, 64, 127, 33, 100, 2, 90, 128, 77]
    q, k, v, d_o = make(lens, 32, 8, BF16)
    got, ref = run(hga, q, k, v, d_o, ends(lens)), R.packed(q, k, v, lens, d_o=d_o)
    for n, limit in (("o", 2.5e-3), ("dq", 2.0e-3), ("dk", 2.0e-3), ("dv", 2.5e-3)):
        e = ((got[n].double() - ref[n]).norm() / ref[n].norm()).item()
        assert 1e-3 < e <= limit, (n, e)
