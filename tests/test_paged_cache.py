"""The paged K/V cache (hga_pages_*, hga_paged_attn) on the GPU: its integers against a plain Python model,
its contents against the tokens that were put in, its attention against float64 with the bounds of
readout_ref."""
import math
import random
import threading

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """The cache as the header describes it, in Python lists; content[row] lists token ids."""

    def __init__(self, n_pages, page, max_seqs, max_pages):
        self.page, self.cap, self.n_pages = page, max_pages * page, n_pages
        self.table = [[] for _ in range(max_seqs)]
        self.len = [0] * max_seqs
        self.ref = [0] * n_pages
        self.content = [[] for _ in range(max_seqs)]

    def pages(self, n):
        return -(-n // self.page)

    def take(self, need):
        free = [i for i, r in enumerate(self.ref) if r == 0]
        return free[:need] if len(free) >= need else None

    def reserve(self, rows, add):
        bad = len(set(rows)) < len(rows) or any(
            not 0 <= r < len(self.len) or a < 0 or self.len[r] + a > self.cap for r, a in zip(rows, add))
        if bad:
            return [-1] * len(rows), -1
        need = [self.pages(self.len[r] + a) - self.pages(self.len[r]) for r, a in zip(rows, add)]
        ids = self.take(sum(need))
        if ids is None:
            return [-1] * len(rows), -8
        pos = []
        for r, a, k in zip(rows, add, need):
            self.table[r] += ids[:k]
            for i in ids[:k]:
                self.ref[i] = 1
            ids = ids[k:]
            pos.append(self.len[r])
            self.len[r] += a
        return pos, 0

    def fork(self, src, dst):
        n = len(self.len)
        if any(not 0 <= d < n or self.len[d] for d in dst) or len(set(dst)) < len(dst) or any(
                not 0 <= s < n or s in dst for s in src):
            return -1
        ids = self.take(sum(self.len[s] % self.page != 0 for s in src))
        if ids is None:
            return -8
        for s, d in zip(src, dst):
            full = self.len[s] // self.page
            self.table[d] = self.table[s][:full]
            for i in self.table[d]:
                self.ref[i] += 1
            if self.len[s] % self.page:
                i = ids.pop(0)
                self.ref[i] = 1
                self.table[d].append(i)
            self.len[d] = self.len[s]
            self.content[d] = list(self.content[s])
        return 0

    def free(self, rows):
        if len(set(rows)) < len(rows) or any(not 0 <= r < len(self.len) for r in rows):
            return -1
        for r in rows:
            for i in self.table[r]:
                self.ref[i] -= 1
            self.table[r], self.len[r], self.content[r] = [], 0, []
        return 0

    def compact(self):
        n = sum(r > 0 for r in self.ref)
        to = dict(zip([i for i in range(n, self.n_pages) if self.ref[i]], [i for i in range(n) if not self.ref[i]]))
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = [[to.get(i, i) for i in t] for t in self.table]
        return n

    def same(self, cache):
        assert cache.seq_len.tolist() == self.len
        assert cache.ref_count.tolist() == self.ref
        for t, got in zip(self.table, cache.page_table.tolist()):
            assert got[:len(t)] == t


def tokens(ids, Hkv, dtype, which):
    """K or V rows of token ids: distinct small whole numbers, exact in bf16."""
    x = torch.tensor(ids, device="cuda", dtype=torch.float64).view(-1, 1, 1)
    h = torch.arange(Hkv, device="cuda", dtype=torch.float64).view(1, -1, 1)
    d = torch.arange(128, device="cuda", dtype=torch.float64).view(1, 1, -1)
    return ((x * 7 + h * 31 + d * 3 + 101 * which) % 251).to(dtype)


def check_content(cache, model, layers):
    for r, ids in enumerate(model.content):
        if ids:
            pages = torch.tensor(model.table[r], device="cuda")
            for layer in range(layers):
                for which, pool in enumerate((cache.k_pool, cache.v_pool)):
                    got = pool[layer, pages].transpose(1, 2).flatten(0, 1)[:len(ids)]
                    want = tokens([i + 1000 * layer for i in ids], cache.cfg.Hkv, cache.dtype, which)
                    assert torch.equal(got, want), (r, layer, which)


def append(cache, model, rows, add, fresh, layers):
    want_pos, code = model.reserve(rows, add)
    pos = cache.reserve(i32(rows), i32(add))
    assert pos.tolist() == want_pos
    cu = [0]
    new = []
    for r, a in zip(rows, add):
        cu.append(cu[-1] + a if a > 0 else cu[-1])
        ids = [next(fresh) for _ in range(max(a, 0))]
        new += ids
        if code == 0:
            model.content[r] += ids
    for layer in range(layers):
        k, v = (tokens([i + 1000 * layer for i in new], cache.cfg.Hkv, cache.dtype, w) for w in (0, 1))
        cache.write(layer, k, v, i32(cu), i32(rows), pos)
    return code


@pytest.mark.parametrize("dtype,page,Hkv", [(BF16, 16, 2), (BF16, 64, 1), (F32, 32, 2), (BF16, 128, 3)])
def test_random_life(hga, dtype, page, Hkv):
    """A long random run of every call, full and refused ones among them, against the model after each."""
    rng = random.Random(page)
    layers, n_pages, seqs, max_pages = 2, 40, 9, 7
    cache = hga.PagedKVCache.new(layers, n_pages, page, Hkv, seqs, max_pages * page, dtype)
    cache.k_pool.fill_(math.nan)
    cache.v_pool.fill_(math.nan)
    model = Model(n_pages, page, seqs, max_pages)
    fresh = iter(range(10 ** 6))
    seen = set()
    for step in range(120):
        op = rng.choice(["append"] * 4 + ["fork", "fork", "free", "compact"])
        if op == "append":
            rows = rng.sample(range(seqs), rng.randint(1, 4))
            add = [rng.choice([0, 1, 1, rng.randint(1, 3 * page)]) for _ in rows]
            if rng.random() < 0.1:
                rows[-1] = rng.choice([rows[0], -1, seqs])
            code = append(cache, model, rows, add, fresh, layers)
        elif op == "fork":
            empty = [r for r in range(seqs) if model.len[r] == 0]
            dst = rng.sample(empty, min(len(empty), rng.randint(0, 3))) + ([rng.randrange(seqs)] if rng.random() < 0.2 else [])
            src = [rng.randrange(seqs) for _ in dst]
            code = model.fork(src, dst)
            cache.fork(i32(src), i32(dst))
        elif op == "free":
            rows = rng.sample(range(seqs), rng.randint(0, 4))
            if rng.random() < 0.2 and rows:
                rows.append(rng.choice([rows[0], seqs + 3]))
            code = model.free(rows)
            cache.free(i32(rows))
        else:
            code = 0
            assert cache.compact().item() == model.compact()
        assert cache.status() == code, (step, op)
        seen.add((op, code))
        model.same(cache)
        check_content(cache, model, layers)
    assert {("append", -1), ("fork", -1), ("free", -1), ("fork", 0), ("compact", 0)} <= seen
    # more pages than the pool has: refused whole; then as many as it has
    rows = list(range(seqs))
    model.free(rows)
    cache.free(i32(rows))
    assert append(cache, model, rows, [max_pages * page] * seqs, fresh, layers) == cache.status() == -8
    assert append(cache, model, rows[:6], [max_pages * page] * 5 + [(n_pages - 5 * max_pages) * page], fresh, layers) == 0
    assert append(cache, model, rows[6:7], [1], fresh, layers) == cache.status() == -8
    model.same(cache)
    check_content(cache, model, layers)


def dense(cache, rows, q, layer=0, scale=None):
    """Reference outputs and bounds of attend(): {o, e_o, lse, e_lse}."""
    n, Hq, _ = q.shape
    Hkv = cache.cfg.Hkv
    out = {"o": torch.zeros(n, Hq, 128, dtype=torch.float64, device="cuda"),
           "lse": torch.full((n, Hq), -math.inf, dtype=torch.float64, device="cuda")}
    out.update({"e_" + k: torch.zeros_like(v) for k, v in list(out.items())})
    lens, table = cache.seq_len.tolist(), cache.page_table.tolist()
    for i, r in enumerate(rows):
        L = lens[r]
        if L:
            ids = torch.tensor(table[r][:-(-L // cache.cfg.page)], device="cuda")
            k, v = (p[layer, ids].transpose(0, 1).flatten(1, 2)[:, :L].repeat_interleave(Hq // Hkv, 0)
                    for p in (cache.k_pool, cache.v_pool))
            f = R.attend(q[i][:, None], k, v, torch.ones(1, L, dtype=torch.bool, device="cuda"),
                         scale or 1 / math.sqrt(128), q.dtype)
            for x in ("o", "e_o", "lse", "e_lse"):
                out[x][i] = f[x][:, 0]
    return out


def filled(hga, lens, page, Hkv, dtype, seed=0, layers=1, spare=5, room=0):
    """A cache whose row i has lens[i] random tokens in pages scattered over the pool; every place that holds
    no token is NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    width = max(need + [1]) + room
    cache = hga.PagedKVCache.new(layers, n_pages, page, Hkv, len(lens), width * page, dtype)
    cache.k_pool.fill_(math.nan)
    cache.v_pool.fill_(math.nan)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").int().tolist()
    table = torch.zeros(len(lens), width, dtype=torch.int32)
    for r, (n, k) in enumerate(zip(lens, need)):
        mine, ids = ids[:k], ids[k:]
        table[r, :k] = torch.tensor(mine, dtype=torch.int32)
        for pool in (cache.k_pool, cache.v_pool):
            x = torch.full((layers, k * page, Hkv, 128), math.nan, device="cuda", dtype=dtype)
            x[:, :n] = torch.randn(layers, n, Hkv, 128, generator=gen, device="cuda").to(dtype)
            if k:
                pool[:, torch.tensor(mine, device="cuda")] = x.view(layers, k, page, Hkv, 128).transpose(2, 3)
        cache.ref_count[mine] = 1
    cache.page_table.copy_(table)
    cache.seq_len.copy_(i32(lens))
    return cache, gen


def attend_and_check(cache, q, rows, layer=0, scale=None):
    o, lse = cache.attend(layer, q, i32(rows), softmax_scale=scale)
    ref = dense(cache, rows, q, layer, scale)
    R.check(o, ref, "o")
    R.check(lse, ref, "lse")
    assert cache.status() == 0
    return o, lse


DECODE_LENS = [[1], [0], [16], [0, 1, 15, 17, 64, 65, 127, 0], [1000], [513, 2, 2047, 0, 90], [3000, 1], [5, 64, 128, 4097]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", DECODE_LENS, ids=str)
def test_attend_lengths(hga, dtype, page, lens):
    cache, gen = filled(hga, lens, page, 2, dtype, seed=len(lens))
    q = torch.randn(len(lens), 8, 128, generator=gen, device="cuda").to(dtype)
    attend_and_check(cache, q, list(range(len(lens))))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (128, 1), (8, 8), (32, 8), (10, 5)])
def test_attend_heads(hga, dtype, Hq, Hkv):
    lens = [700, 33, 0, 1]
    cache, gen = filled(hga, lens, 32, Hkv, dtype, seed=Hq)
    q = torch.randn(4, Hq, 128, generator=gen, device="cuda").to(dtype)
    attend_and_check(cache, q, [0, 1, 2, 3])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_one_long_sequence(hga, dtype):
    """All CTAs on one pair, and the join of all of their parts."""
    cache, gen = filled(hga, [50001], 64, 1, dtype)
    q = torch.randn(1, 4, 128, generator=gen, device="cuda").to(dtype)
    attend_and_check(cache, q, [0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_rows_scale_strides_layers(hga, dtype):
    """Rows in any order and more than once, a scale, strided queries, another layer."""
    lens = [100, 0, 257, 31]
    cache, gen = filled(hga, lens, 16, 2, dtype, layers=3)
    wide = torch.randn(6, 7, 128, generator=gen, device="cuda").to(dtype)
    rows = [2, 0, 0, 3, 1, 2]
    attend_and_check(cache, wide[:, 1:5], rows, layer=2, scale=0.3)
    a, _ = attend_and_check(cache, wide[:1, :4].expand(1, 4, 128), [2], layer=1)
    b, _ = cache.attend(1, wide[:, :4], i32(rows))
    R.check(b, dense(cache, rows, wide[:, :4], 1), "o")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_queries(hga, dtype):
    lens = [(37 * i) % 90 for i in range(700)]
    cache, gen = filled(hga, lens, 16, 1, dtype)
    q = torch.randn(700, 2, 128, generator=gen, device="cuda").to(dtype)
    attend_and_check(cache, q, list(range(700)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_pools(hga, dtype):
    """K and V in one allocation, a page's layers side by side."""
    layers, P, Hkv, page = 2, 12, 2, 16
    whole = torch.full((P, 2, layers, Hkv, page, 128), math.nan, device="cuda", dtype=dtype)
    k, v = (whole[:, i].transpose(0, 1) for i in (0, 1))
    cache = hga.PagedKVCache(k, v, *(torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((4, 6), (4,), (P,))))
    model = Model(P, page, 4, 6)
    fresh = iter(range(10 ** 6))
    assert append(cache, model, [1, 3], [50, 17], fresh, layers) == 0
    model.fork([1, 3], [0, 2])
    cache.fork(i32([1, 3]), i32([0, 2]))
    model.free([1])
    cache.free(i32([1]))
    assert cache.compact().item() == model.compact()
    assert cache.status() == 0
    model.same(cache)
    check_content(cache, model, layers)
    q = torch.randn(3, 4, 128, device="cuda").to(dtype) / 64
    attend_and_check(cache, q, [0, 2, 3], layer=1)


def test_copy_pages(hga):
    cache, _ = filled(hga, [64, 64, 64], 16, 2, BF16, layers=2, spare=8)
    before = cache.k_pool.clone(), cache.v_pool.clone()
    src, dst = [3, 3, 0, 7], [1, 9, 12, 5]
    cache.copy_pages(i32(src), i32(dst))
    for pool, old in zip((cache.k_pool, cache.v_pool), before):
        want = old.clone()
        want[:, dst] = old[:, src]
        assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    after = cache.k_pool.clone()
    for s, d in (([1, 2], [4, 4]), ([1, 2], [2, 5]), ([1], [20]), ([-1], [3]), ([1], [-1])):
        cache.copy_pages(i32(s), i32(d))
        assert cache.status() == hga._capi.HGA_ERR_ARG, (s, d)
    assert torch.equal(cache.k_pool.view(torch.int16), after.view(torch.int16))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_integers_are_recorded(hga, dtype):
    """Page ids, lengths and rows outside their ranges are never followed: the tokens are left out."""
    cache, gen = filled(hga, [200, 130, 40], 16, 2, dtype)
    q = torch.randn(3, 8, 128, generator=gen, device="cuda").to(dtype)
    good = dense(cache, [0, 1, 2], q)
    cache.page_table[1, 3] = 10 ** 6
    cache.page_table[1, 5] = -7
    o, lse = cache.attend(0, q, i32([0, 1, 2]))
    assert cache.status() == hga._capi.HGA_ERR_ARG
    for i in (0, 2):
        R.check(o[i], {"o": good["o"][i], "e_o": good["e_o"][i]}, "o")
    assert torch.isfinite(o).all()
    keep = [i for i in range(130) if i // 16 not in (3, 5)]
    ids = cache.page_table[1].long()
    k, v = (torch.stack([p[0, ids[t // 16], :, t % 16] for t in keep], 1).repeat_interleave(4, 0)
            for p in (cache.k_pool, cache.v_pool))
    f = R.attend(q[1][:, None], k, v, torch.ones(1, len(keep), dtype=torch.bool, device="cuda"), 1 / math.sqrt(128), dtype)
    R.check(o[1], {"o": f["o"][:, 0], "e_o": f["e_o"][:, 0]}, "o")
    o, lse = cache.attend(0, q, i32([0, 99, -1]))
    assert cache.status() == hga._capi.HGA_ERR_ARG
    assert not o[1:].any() and (lse[1:] == -math.inf).all()
    cache.seq_len[2] = 10 ** 7
    o, lse = cache.attend(0, q, i32([0, 0, 2]))
    assert cache.status() == hga._capi.HGA_ERR_ARG
    assert not o[2].any()
    # the page moves refuse what they cannot follow, and change nothing
    ints = [x.clone() for x in (cache.page_table, cache.seq_len, cache.ref_count)]
    for call in (lambda: cache.reserve(i32([2]), i32([1])), lambda: cache.free(i32([2])), lambda: cache.free(i32([0, 1])),
                 lambda: cache.reserve(i32([0]), i32([-1])), lambda: cache.reserve(i32([0]), i32([10 ** 9]))):
        call()
        assert cache.status() == hga._capi.HGA_ERR_ARG
        for x, y in zip(ints, (cache.page_table, cache.seq_len, cache.ref_count)):
            assert torch.equal(x, y)


def test_refused_reserve_writes_nothing(hga):
    """A write with the positions of a refused reserve touches no byte of the pools."""
    cache, _ = filled(hga, [16, 16], 16, 1, BF16, spare=1, room=1)
    before = cache.k_pool.clone()
    pos = cache.reserve(i32([0, 1]), i32([1, 1]))                    # two pages, one free
    assert pos.tolist() == [-1, -1]
    assert cache.status() == hga._capi.HGA_ERR_PAGES
    x = torch.ones(2, 1, 128, device="cuda", dtype=BF16)
    cache.write(0, x, x, i32([0, 1, 2]), i32([0, 1]), pos)
    assert cache.status() == 0
    # positions behind the sequence's length are refused as well
    cache.write(0, x, x, i32([0, 1, 2]), i32([0, 1]), i32([16, 10 ** 8]))
    assert cache.status() == hga._capi.HGA_ERR_ARG
    assert torch.equal(cache.k_pool.view(torch.int16), before.view(torch.int16))


def test_generation_matches_the_prompt(hga):
    """A prompt's attention, its K/V into the cache, then token by token from a CUDA graph of the whole decode
    step: every new token's output is the packed attention's row of the longer sequence; a fork goes on from
    the same prefix."""
    Hq, Hkv, page, steps = 8, 2, 16, 40
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens = [33, 1, 100]
    total = [n + steps for n in lens]
    qkv = [torch.randn(n, Hq + 2 * Hkv, 128, generator=gen, device="cuda").to(BF16) for n in total]
    cache = hga.PagedKVCache.new(1, 64, page, Hkv, 4, 256)
    packed = torch.cat([x[:n] for x, n in zip(qkv, lens)])
    q, k, v = packed.split([Hq, Hkv, Hkv], dim=1)
    cu = i32([0, 33, 34, 134])
    rows = i32([0, 1, 2])
    o, _ = hga.packed_attention(q, k, v, cu)
    R.check(o, R.packed(q, k, v, lens), "o")
    cache.write(0, k, v, cu, rows, cache.reserve(rows, i32(lens)))
    x = torch.empty(3, Hq + 2 * Hkv, 128, device="cuda", dtype=BF16)
    out, lse = torch.empty(3, Hq, 128, device="cuda", dtype=BF16), torch.empty(3, Hq, device="cuda")
    one, cu1 = i32([1, 1, 1]), i32([0, 1, 2, 3])

    def step():
        pos = cache.reserve(rows, one)
        cache.write(0, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu1, rows, pos)
        cache.attend(0, x[:, :Hq], rows, o=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [t.clone() for t in (cache.page_table, cache.seq_len, cache.ref_count)]
    x.zero_()
    with torch.cuda.stream(side):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((cache.page_table, cache.seq_len, cache.ref_count), state):
        t.copy_(old)                                   # the first run was for warming up
    got = []
    for i in range(steps):
        x.copy_(torch.stack([s[n + i] for s, n in zip(qkv, lens)]))
        graph.replay()
        got.append(out.clone())
    assert cache.status() == 0
    assert cache.seq_len.tolist() == total + [0]
    got = torch.stack(got, 1)
    for r, s in enumerate(qkv):
        ref = R.packed(*s.split([Hq, Hkv, Hkv], dim=1), [total[r]])
        R.check(got[r], {n: ref[n][lens[r]:] for n in ("o", "e_o")}, "o")
    cache.fork(i32([2]), i32([3]))
    cache.free(i32([2]))
    a = torch.randn(1, Hq, 128, generator=gen, device="cuda").to(BF16)
    attend_and_check(cache, a, [3])
    k, v = (t.transpose(0, 1).double().repeat_interleave(4, 0) for t in qkv[2].split([Hq, Hkv, Hkv], dim=1)[1:])
    f = R.attend(a[0][:, None], k, v, torch.ones(1, total[2], dtype=torch.bool, device="cuda"), 1 / math.sqrt(128), BF16)
    R.check(cache.attend(0, a, i32([3]))[0][0], {"o": f["o"][:, 0], "e_o": f["e_o"][:, 0]}, "o")


def test_more_than_2_31_elements(hga):
    """A pool of more than 2^31 elements: pages at its end are written, attended, forked and moved."""
    page, Hkv, P = 64, 8, 33000
    cache = hga.PagedKVCache.new(1, P, page, Hkv, 3, 4 * page)
    assert cache.k_pool.numel() > 2 ** 31
    cache.ref_count[:P - 6] = 1                        # only the last six pages are free
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = 150
    k, v = (torch.randn(n, Hkv, 128, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    row = i32([1])
    cache.write(0, k, v, i32([0, n]), row, cache.reserve(row, i32([n])))
    assert cache.status() == 0
    assert cache.page_table[1, :3].tolist() == [P - 6, P - 5, P - 4]
    q = torch.randn(2, 32, 128, generator=gen, device="cuda", dtype=BF16)
    attend_and_check(cache, q, [1, 1])
    cache.fork(row, i32([2]))
    assert cache.page_table[2, :3].tolist() == [P - 6, P - 5, P - 3]
    a, _ = cache.attend(0, q, i32([1, 2]))
    attend_and_check(cache, q, [2, 1])
    cache.ref_count[100:200] = 0
    assert cache.compact().item() == P - 6 - 100 + 4
    assert cache.page_table[2, :3].max().item() < 200
    b, _ = cache.attend(0, q, i32([1, 2]))
    assert cache.status() == 0 and torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_expired_wait_is_recorded(hga, dtype):
    cache, gen = filled(hga, [999, 3000, 5, 0, 1200], 64, 2, dtype)
    q = torch.randn(5, 8, 128, generator=gen, device="cuda").to(dtype)
    rows = i32([0, 1, 2, 3, 4])
    want, _ = cache.attend(0, q, rows)
    cache.cfg.wait_limit_ns = 1
    cache.attend(0, q, rows)
    assert cache.status() == hga._capi.HGA_ERR_TIMEOUT
    cache.cfg.wait_limit_ns = 0
    for _ in range(3):
        got, _ = cache.attend(0, q, rows)
        assert torch.equal(got, want)
    assert cache.status() == 0


def test_reserve_of_more_than_2_31_pages(hga):
    """The pages asked for add up beyond 32 bits: refused, nothing changed."""
    n, P = 2100, 1 << 20
    cache = hga.PagedKVCache.new(1, P, 16, 1, n, 16 * (P + 64))
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    pos = cache.reserve(rows, torch.full_like(rows, 16 * (P + 64)))
    assert cache.status() == hga._capi.HGA_ERR_PAGES
    assert (pos == -1).all() and not cache.seq_len.any() and not cache.ref_count.any()
    assert cache.reserve(rows, torch.full_like(rows, 17)).eq(0).all()
    assert cache.status() == 0 and cache.ref_count.sum().item() == 2 * n


def test_two_caches_at_once(hga):
    """Attention over two caches on two streams, over and over."""
    both = [filled(hga, lens, 32, 2, BF16, seed=i) for i, lens in enumerate(([2000, 17, 640], [5, 3000]))]
    qs = [torch.randn(len(c.seq_len), 8, 128, generator=g, device="cuda").to(BF16) for c, g in both]
    rows = [i32(list(range(len(c.seq_len)))) for c, _ in both]
    want = [c.attend(0, q, r)[0] for (c, _), q, r in zip(both, qs, rows)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both[i][0].attend(0, qs[i], rows[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_is_reproducible(hga, dtype):
    lens = [999, 3000, 5, 0, 1200]
    cache, gen = filled(hga, lens, 64, 2, dtype)
    q = torch.randn(5, 8, 128, generator=gen, device="cuda").to(dtype)
    a, b = cache.attend(0, q, i32([0, 1, 2, 3, 4]))
    for _ in range(20):
        c, d = cache.attend(0, q, i32([0, 1, 2, 3, 4]))
        assert torch.equal(a, c) and torch.equal(b, d)


def test_extreme_scores(hga):
    for dtype in (F32, BF16):
        cache, gen = filled(hga, [700], 32, 1, dtype)
        q = torch.randn(1, 4, 128, generator=gen, device="cuda").to(dtype) * 512
        attend_and_check(cache, q, [0])


def test_refusals(hga):
    cache, _ = filled(hga, [20, 30], 16, 2, BF16)
    q = torch.zeros(2, 4, 128, device="cuda", dtype=BF16)
    rows = i32([0, 1])
    for call in (lambda: cache.attend(1, q, rows), lambda: cache.attend(-1, q, rows), lambda: cache.attend(0, q.float(), rows),
                 lambda: cache.attend(0, q, i32([0])), lambda: cache.attend(0, q, rows.long()),
                 lambda: cache.attend(0, q, rows.cpu()), lambda: cache.attend(0, q[:, :3], rows),
                 lambda: cache.fork(rows, i32([0])), lambda: cache.reserve(rows, i32([1])),
                 lambda: cache.write(0, q[:, :2], q[:, :2], i32([0, 1]), rows, rows),
                 lambda: cache.write(0, q, q, i32([0, 1, 2]), rows, rows),
                 lambda: hga.PagedKVCache.new(1, 4, 24, 2, 2, 64),
                 lambda: hga.PagedKVCache(cache.k_pool, cache.v_pool[:, :3], cache.page_table, cache.seq_len, cache.ref_count),
                 lambda: hga.PagedKVCache(cache.k_pool.transpose(2, 3), cache.v_pool.transpose(2, 3), cache.page_table,
                                          cache.seq_len, cache.ref_count)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def big_cache(hga, n_pages):
    pools = [torch.empty(1, n_pages, 1, 16, 128, device="cuda", dtype=BF16) for _ in range(2)]
    return hga.PagedKVCache(*pools, i32([[0]]), i32([0]), torch.zeros(n_pages, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("n_pages", [380_000, 385_024, 393_150, 393_200, 393_217, 1 << 20])
def test_copy_pages_of_large_pools(hga, n_pages):
    """The list of destinations seen (a bit per page) at and around 48 KB of shared memory."""
    cache = big_cache(hga, n_pages)
    src, dst = [n_pages - 1, 5, 5], [7, n_pages - 2, 0]
    cache.k_pool[:, src] = 3
    cache.v_pool[:, src] = 4
    cache.copy_pages(i32(src), i32(dst))
    assert cache.status() == 0
    assert (cache.k_pool[:, dst] == 3).all() and (cache.v_pool[:, dst] == 4).all()
    cache.copy_pages(i32([1, 2]), i32([n_pages - 1, n_pages - 1]))
    assert cache.status() == hga._capi.HGA_ERR_ARG


def test_copy_pages_from_two_threads(hga):
    """Pools of different sizes, copied from two threads at once: no call takes the other's limit of shared memory."""
    caches = [big_cache(hga, n) for n in (400_000, 900_000)]
    streams, errors = [torch.cuda.Stream() for _ in caches], []
    src, dst = i32([1]), i32([2])
    torch.cuda.synchronize()

    def work(cache, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(3000):
                    cache.copy_pages(src, dst)
        except Exception as e:                         # noqa: BLE001 (whatever it is, the test fails with it)
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(caches, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert [c.status() for c in caches] == [0, 0]


@pytest.mark.parametrize("cu", [[0, 3, 9], [0, 5, 3, 6], [2, 1, 6], [0, 7], [-1, 6]], ids=str)
def test_write_with_bounds_of_rows_that_are_not_there(hga, cu):
    """Bounds that decrease or pass the rows: recorded, and no byte outside the rows' reserved places is touched."""
    n = len(cu) - 1
    cache, _ = filled(hga, [0] * n + [40], 16, 2, BF16, spare=2 * n, room=2)
    rows = i32(list(range(n)))
    pos = cache.reserve(rows, i32([20] * n))
    assert cache.status() == 0
    own = {p for r in range(n) for p in cache.page_table[r, :2].tolist()}
    others = [p for p in range(cache.cfg.n_pages) if p not in own]
    before = cache.k_pool[:, others].clone()
    x = torch.ones(6, 2, 128, device="cuda", dtype=BF16)
    cache.write(0, x, x, i32(cu), rows, pos)
    assert cache.status() == hga._capi.HGA_ERR_ARG
    assert torch.equal(cache.k_pool[:, others].view(torch.int16), before.view(torch.int16))
    cache.write(0, x, x, i32([0] * n + [6]), rows, pos)
    cache.write(0, x, x, i32([1] + [4] * n), rows, pos)          # rows before the first and behind the last entry's: no one's
    assert cache.status() == 0


def test_compact_with_bad_integers(hga):
    """Rows that are in order follow their pages, whatever the others hold; what is not in order stays and is recorded."""
    cache, gen = filled(hga, [100, 200, 40, 90], 16, 2, BF16, spare=30)
    q = torch.randn(2, 4, 128, generator=gen, device="cuda").to(BF16)
    rows = i32([0, 3])
    want, _ = cache.attend(0, q, rows)
    cache.page_table[1, 2] = 10 ** 6
    cache.page_table[1, 3] = -4
    cache.seq_len[2] = -9
    used = int((cache.ref_count > 0).sum())
    stale = cache.page_table[2].clone()
    assert cache.compact().item() == used
    assert cache.status() == hga._capi.HGA_ERR_ARG
    assert cache.page_table[1, 2:4].tolist() == [10 ** 6, -4] and cache.seq_len[2].item() == -9
    assert torch.equal(cache.page_table[2], stale)
    assert (cache.ref_count[:used] > 0).all() and not cache.ref_count[used:].any()
    got, _ = cache.attend(0, q, rows)
    assert cache.status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1), (16, 1), (40, 2)])
def test_attend_rounds_its_output_only(hga, Hq, Hkv):
    """bf16: p is the sum of two bf16 numbers (of which what is left is 2^-16 at most), scores and sums are in float32 (below 1e-5 for these): the error is
    that of rounding the exact output, 1.6e-3 of the norm, where a p of one number would add as much again."""
    lens = [1000, 33, 5000, 2]
    cache, gen = filled(hga, lens, 64, Hkv, BF16, seed=Hq)
    q = torch.randn(4, Hq, 128, generator=gen, device="cuda").to(BF16)
    o, _ = cache.attend(0, q, i32([0, 1, 2, 3]))
    ref = dense(cache, [0, 1, 2, 3], q)["o"]
    rounding = (ref.to(BF16).double() - ref).norm() / ref.norm()
    assert (o.double() - ref).norm() / ref.norm() <= rounding + 2e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1), (16, 1), (20, 1), (8, 2)])
def test_attended_values_that_are_not_finite(hga, dtype, Hq, Hkv):
    """Infinities and NaN in v of cached tokens: the query heads that attend them get them, with their sign, in their dim, and
    nothing else changes."""
    lens = [1, 20, 700, 64]
    cache, gen = filled(hga, lens, 16, Hkv, dtype, seed=Hq)
    q = torch.randn(4, Hq, 128, generator=gen, device="cuda").to(dtype)
    rows = i32([0, 1, 2, 3])
    clean, lse = cache.attend(0, q, rows)
    for r, t in ((0, 0), (1, 19), (2, 100), (2, 699)):
        page = cache.page_table[r, t // 16].long()
        for d, x in ((5, math.inf), (77, -math.inf), (90, math.nan)):
            cache.v_pool[0, page, 0, t % 16, d] = x
    got, lse2 = cache.attend(0, q, rows)
    assert cache.status() == 0 and torch.equal(lse, lse2)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[:3, :Hq // Hkv, [5, 77, 90]] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert (got[:3, :Hq // Hkv, 5] == math.inf).all() and (got[:3, :Hq // Hkv, 77] == -math.inf).all()
    assert got[:3, :Hq // Hkv, 90].isnan().all()
