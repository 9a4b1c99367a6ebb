"""Measured cases of the dense readout: causal attention over packed prompts (forward, and with its
gradients), attention of one new token over a paged K/V cache, and the page moves of that cache
(append, fork and free, compact).

``run`` computes a case in its plain form, elementary torch operations in 32 bits; with ``own`` set it
makes the calls a user makes of ``hierarchical_kv_routing_tok_b200``.  Layouts: packed rows
[tokens, heads, 128]; pools [layers, pages, KV heads, page, 128]; a cache's integers (page table, lengths,
page reference counts) are one int32 buffer.  A case's sequence lengths are a text of comma-separated
numbers.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one short question to a small layer: all latency
        {"name": "prompt 37 tokens", "op": "prompt", "dtype": "bf16", "hq": 8, "hkv": 2, "lens": "37", "tail": 0,
         "layout": "tokens"},
        # the readout of one 16K-token context by the 32/8-head layer
        {"name": "prompt 16K", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "lens": "16384", "tail": 0,
         "layout": "fused"},
        # the tiny float32 layer trained on a few packed snippets, one of a single token, one empty
        {"name": "train tiny f32", "op": "train", "dtype": "f32", "hq": 4, "hkv": 1, "lens": "256,1,0,77,641",
         "tail": 5, "layout": "tokens"},
        # a packed 16K-token training batch: documents of very different lengths, rows left over at the end
        {"name": "train packed 16K", "op": "train", "dtype": "bf16", "hq": 32, "hkv": 8,
         "lens": "8192,2049,1,811,300,64,3517,129,1000,47,263", "tail": 11, "layout": "fused"},
        # one chat a few pages long: the latency of a decode step
        {"name": "decode one chat", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "lens": "513", "page": 64},
        # a served batch, every request at another length (one not begun), small pages
        {"name": "decode batch of 48", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "page": 16,
         "lens": "1,7901,640,4096,333,0,2050,5121,17,900,6143,129,3000,1024,77,2511,8000,45,1999,700,256,3601,1100,"
                 "2,4801,1500,60,970,7001,430,2222,31,1801,5550,128,640,3333,95,2048,1201,6502,15,880,4100,510,2700,"
                 "64,1301"},
        # two requests at the evaluation length: the cache's bandwidth
        {"name": "decode 2 x 131K", "op": "decode", "dtype": "bf16", "hq": 32, "hkv": 8, "lens": "131071,130000",
         "page": 64},
        # two beams that each branch twice, and the branches dropped again
        {"name": "fork 2 beams", "op": "fork", "dtype": "bf16", "hkv": 8, "page": 16, "layers": 2, "pages": 256,
         "lens": "700,333", "ways": 2},
        # a served batch that branches four ways over all layers
        {"name": "fork 24 x 4", "op": "fork", "dtype": "bf16", "hkv": 8, "page": 64, "layers": 4, "pages": 1024,
         "lens": "1000,130,65,1999,700,256,1601,1100,2,801,1500,60,970,1,430,222,31,1801,550,129,640,333,95,2047",
         "ways": 4},
        # a pool after a long run of requests of which a half has ended
        {"name": "compact 4096 pages", "op": "compact", "dtype": "bf16", "hkv": 8, "page": 64, "layers": 2,
         "pages": 4096, "seqs": 96, "fill": 0.5},
        # the decode step's append: one token for each of 64 requests
        {"name": "append 64 x 1", "op": "append", "dtype": "bf16", "hkv": 8, "page": 64, "pages": 2048,
         "lens": ",".join(str(37 * i % 1900) for i in range(64)), "add": ",".join(["1"] * 64), "layout": "tokens"},
        # packed prompts written into the cache after their attention
        {"name": "append prompts 16K", "op": "append", "dtype": "bf16", "hkv": 8, "page": 64, "pages": 2048,
         "lens": "0,100,0,0,5000,63", "add": "8192,1,1200,4097,2045,849", "layout": "fused"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "train", "decode", "decode", "fork", "compact", "append"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    hkv = rng.choice([1, 2, 4, 8])
    if op in ("prompt", "train"):
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
        hq = hkv * (32 // hkv) if hq > 32 else hq
        longest = 16384 if op == "prompt" and dtype == "bf16" else 8192 if dtype == "bf16" else 1500
        total = _log_int(rng, 1, longest)
        lens, left = [], total
        for _ in range(rng.randint(0, 11)):
            if left > 1:
                lens.append(min(left - 1, _log_int(rng, 1, left)))
                left -= lens[-1]
        lens.append(left)
        if rng.random() < 0.3:
            lens.append(0)
        rng.shuffle(lens)
        return {"op": op, "dtype": dtype, "hq": hq, "hkv": hkv, "lens": ",".join(map(str, lens)),
                "tail": rng.choice([0, 0, rng.randint(1, 150)]), "layout": rng.choice(["tokens", "fused", "heads"])}
    if op == "decode":
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        n = _log_int(rng, 1, 96)
        longest = _log_int(rng, 40, min(131072, 1 << 20 if n < 3 else 200000 // n))
        lens = [rng.choice([0, 1, longest]) if rng.random() < 0.1 else _log_int(rng, 1, longest) for _ in range(n)]
        lens[rng.randrange(n)] = longest
        return {"op": op, "dtype": dtype, "hq": hq, "hkv": hkv, "lens": ",".join(map(str, lens)),
                "page": rng.choice([16, 32, 64, 128])}
    page = rng.choice([16, 32, 64, 128])
    if op == "compact":
        return {"op": op, "dtype": dtype, "hkv": hkv, "page": page, "layers": rng.randint(1, 2),
                "pages": _log_int(rng, 8, 2000), "seqs": rng.randint(1, 64), "fill": round(rng.uniform(0.1, 1.0), 3)}
    n = _log_int(rng, 1, 40)
    lens = [_log_int(rng, 1, 2000) if rng.random() < 0.9 else 0 for _ in range(n)]
    if op == "fork":
        ways = rng.randint(1, 4)
        need = sum(-(-x // page) for x in lens) + ways * n
        return {"op": op, "dtype": dtype, "hkv": hkv, "page": page, "layers": rng.randint(1, 4),
                "pages": need + rng.randint(1, 60), "lens": ",".join(map(str, lens)), "ways": ways}
    add = [1 if rng.random() < 0.5 else _log_int(rng, 1, 400) for _ in range(n)]
    need = sum(-(-(x + a) // page) for x, a in zip(lens, add))
    return {"op": op, "dtype": dtype, "hkv": hkv, "page": page, "pages": need + rng.randint(1, 60),
            "lens": ",".join(map(str, lens)), "add": ",".join(map(str, add)),
            "layout": rng.choice(["tokens", "fused", "heads"])}


# ------------------------------------------------------------------------------------------- inputs
def _ints(text):
    return [int(x) for x in text.split(",")]


def _ends(lens):
    e = [0]
    for x in lens:
        e.append(e[-1] + x)
    return e


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _rows(gen, T, heads, layout, dtype):
    """[T, h, 128] tensors, one for each of `heads`: separate, slices of one fused projection, or
    transposed views of head-major tensors."""
    if layout == "fused":
        return list(_randn(gen, T, sum(heads), D, dtype=dtype).split(heads, dim=1))
    if layout == "heads":
        return [_randn(gen, h, T, D, dtype=dtype).transpose(0, 1) for h in heads]
    return [_randn(gen, T, h, D, dtype=dtype) for h in heads]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(gen, case, lens, rows, width, layers):
    """Pools and integers of a cache whose first sequences have `lens` tokens in pages taken at random."""
    page, n_pages = case["page"], case["pages"]
    pools = [_randn(gen, layers, n_pages, case["hkv"], page, D, dtype=DTYPES[case["dtype"]]) for _ in range(2)]
    ints = torch.zeros(rows * width + rows + n_pages, dtype=torch.int32, device="cuda")
    counts = torch.tensor([-(-x // page) for x in lens], device="cuda")
    used = int(counts.sum())
    ids = torch.randperm(n_pages, generator=gen, device="cuda")[:used].to(torch.int32)
    col = torch.arange(width, device="cuda")
    table, seq_len, ref = _views(ints, rows, width)
    table[:len(lens)][col < counts[:, None]] = ids
    seq_len[:len(lens)] = _i32(lens)
    ref[ids.long()] = 1
    return {"k_pool": pools[0], "v_pool": pools[1], "ints": ints, "ints0": ints.clone(), "rows": rows, "width": width,
            "page": page}


def _views(ints, rows, width):
    return ints[:rows * width].view(rows, width), ints[rows * width:rows * (width + 1)], ints[rows * (width + 1):]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op}
    if op in ("prompt", "train"):
        lens = _ints(case["lens"])
        ends = _ends(lens)
        T = ends[-1] + case["tail"]
        q, k, v = _rows(gen, T, [case["hq"], case["hkv"], case["hkv"]], case["layout"], dtype)
        # keys of one 64-token chunk share an offset, as the repository's other inputs have it
        k += 0.5 * _randn(gen, -(-T // 64), case["hkv"], D, dtype=dtype).repeat_interleave(64, dim=0)[:T]
        s.update(q=q, k=k, v=v, cu=_i32(ends), ends=ends)
        if op == "train":
            s["d_o"] = _randn(gen, T, case["hq"], D, dtype=dtype)
            s.update({n: s[n].detach().requires_grad_() for n in ("q", "k", "v")})
        return s
    if op == "decode":
        lens, page = _ints(case["lens"]), case["page"]
        width = max(1, max(-(-x // page) for x in lens))
        n_pages = sum(-(-x // page) for x in lens) + 3
        s.update(_cache(gen, dict(case, pages=n_pages), lens, len(lens), width, 1))
        s["q"] = _randn(gen, len(lens), case["hq"], D, dtype=dtype)
        s["slots"] = torch.arange(len(lens), dtype=torch.int32, device="cuda")
        return s
    if op == "fork":
        lens, ways, page = _ints(case["lens"]), case["ways"], case["page"]
        n = len(lens)
        s.update(_cache(gen, case, lens, n * (ways + 1), max(1, max(-(-x // page) for x in lens)), case["layers"]))
        s["src"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(ways)
        s["dst"] = torch.arange(n, n * (ways + 1), dtype=torch.int32, device="cuda")
        # pages that the branches share, and those copied for them, in the order of the branches
        s["part"] = [i for i in range(n * ways) if lens[i // ways] % page]
        s["part"] = torch.tensor(s["part"], dtype=torch.long, device="cuda")
        return s
    if op == "compact":
        n, page = case["seqs"], case["page"]
        used = max(n, int(case["pages"] * case["fill"])) if case["pages"] >= n else case["pages"]
        n = min(n, used)
        per = used // n
        lens = [max(1, page * (per + (1 if i < used - per * n else 0)) - i % page) for i in range(n)]
        s.update(_cache(gen, case, lens, n, per + 1, case["layers"]))
        ref = _views(s["ints"], n, per + 1)[2]
        s["used"] = used
        s["moved"] = int((ref[used:] > 0).sum())
        return s
    lens, add, page = _ints(case["lens"]), _ints(case["add"]), case["page"]
    ends = _ends(add)
    s.update(_cache(gen, case, lens, len(lens), max(-(-(x + a) // page) for x, a in zip(lens, add)), 1))
    s["k"], s["v"] = _rows(gen, ends[-1], [case["hkv"], case["hkv"]], case["layout"], dtype)
    s.update(cu=_i32(ends), add=_i32(add), total=ends[-1], slots=torch.arange(len(lens), dtype=torch.int32, device="cuda"))
    s["need"] = sum(-(-(x + a) // page) - -(-x // page) for x, a in zip(lens, add))
    return s


# ------------------------------------------------------------------------------------------- passes
def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _plain_prompt, "train": _plain_train, "decode": _plain_decode, "fork": _plain_fork,
            "compact": _plain_compact, "append": _plain_append}[state["op"]](state)


def _run_own(s):
    import hierarchical_kv_routing_tok_b200 as H
    op = s["op"]
    if op == "prompt":
        return H.packed_attention(s["q"], s["k"], s["v"], s["cu"])
    if op == "train":
        o, _ = H.packed_attention(s["q"], s["k"], s["v"], s["cu"])
        dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["d_o"])
        return o.detach(), dq, dk, dv
    if "cache" not in s:              # the handle that a serving program keeps beside the cache's tensors
        table, seq_len, ref = _views(s["ints"], s["rows"], s["width"])
        s["cache"] = H.PagedKVCache(s["k_pool"], s["v_pool"], table, seq_len, ref)
    cache = s["cache"]
    if op == "decode":
        return cache.attend(0, s["q"], s["slots"])
    s["ints"].copy_(s["ints0"])       # the same step again: from the same state
    if op == "fork":
        cache.fork(s["src"], s["dst"])
        shared = s["ints"].clone()
        cache.free(s["dst"])
        return s["k_pool"], s["v_pool"], shared, s["ints"]
    if op == "compact":
        cache.compact()
        return s["k_pool"], s["v_pool"], s["ints"]
    pos = cache.reserve(s["slots"], s["add"])
    cache.write(0, s["k"], s["v"], s["cu"], s["slots"], pos)
    return s["k_pool"], s["v_pool"], s["ints"], pos


def _plain_prompt(s):
    return _forward(s["q"], s["k"], s["v"], s["ends"])


def _heads(x, a, b, groups):
    """Rows a..b of x as [heads, b - a, 128] in 32 bits, each KV head repeated for its query heads."""
    return x[a:b].transpose(0, 1).float().repeat_interleave(groups, dim=0)


def _forward(q, k, v, ends):
    T, hq, _ = q.shape
    o = torch.zeros(T, hq, D, dtype=q.dtype, device=q.device)
    lse = torch.full((hq, T), -math.inf, device=q.device)
    G = hq // k.shape[1]
    for a, b in zip(ends, ends[1:]):               # each packed sequence is a softmax of its own
        if a < b:
            p = _heads(q, a, b, 1) @ _heads(k, a, b, G).transpose(1, 2)
            pos = torch.arange(b - a, device=q.device)
            p.mul_(SCALE).masked_fill_(pos[None, :] > pos[:, None], -math.inf)
            m = p.amax(dim=2, keepdim=True)
            p.sub_(m).exp_()
            l = p.sum(dim=2, keepdim=True)
            o[a:b] = ((p @ _heads(v, a, b, G)) / l).transpose(0, 1).to(q.dtype)
            lse[:, a:b] = (m + l.log())[:, :, 0]
    return o, lse


def _plain_train(s):
    q, k, v, d_o = (s[n].detach() for n in ("q", "k", "v", "d_o"))
    hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    o = torch.zeros_like(q, memory_format=torch.contiguous_format)
    dq, dk, dv = (torch.zeros_like(x, memory_format=torch.contiguous_format) for x in (q, k, v))
    for a, b in zip(s["ends"], s["ends"][1:]):
        if a < b:
            n = b - a
            qs, ks, vs, gs = _heads(q, a, b, 1), _heads(k, a, b, G), _heads(v, a, b, G), _heads(d_o, a, b, 1)
            pos = torch.arange(n, device=q.device)
            p = qs @ ks.transpose(1, 2)
            p.mul_(SCALE).masked_fill_(pos[None, :] > pos[:, None], -math.inf)
            p.sub_(p.amax(dim=2, keepdim=True)).exp_()
            p.div_(p.sum(dim=2, keepdim=True))
            os = p @ vs
            ds = gs @ vs.transpose(1, 2)
            ds.sub_((gs * os).sum(dim=2, keepdim=True)).mul_(p).mul_(SCALE)
            o[a:b] = os.transpose(0, 1).to(q.dtype)
            dq[a:b] = (ds @ ks).transpose(0, 1).to(q.dtype)
            dk[a:b] = (ds.transpose(1, 2) @ qs).view(hkv, G, n, D).sum(1).transpose(0, 1).to(q.dtype)
            dv[a:b] = (p.transpose(1, 2) @ gs).view(hkv, G, n, D).sum(1).transpose(0, 1).to(q.dtype)
    return o, dq, dk, dv


def _plain_decode(s):
    table, seq_len, _ = _views(s["ints"], s["rows"], s["width"])
    q = s["q"]
    n, hq, _ = q.shape
    hkv = s["k_pool"].shape[2]
    rows = s["slots"].long()
    ids, length = table[rows].long(), seq_len[rows]
    k = s["k_pool"][0][ids].transpose(1, 2).reshape(n, hkv, -1, D).float()
    v = s["v_pool"][0][ids].transpose(1, 2).reshape(n, hkv, -1, D).float()
    p = (q.float() * SCALE).view(n, hkv, hq // hkv, D) @ k.transpose(2, 3)
    out = torch.arange(p.shape[3], device=q.device) >= length[:, None]
    p.masked_fill_(out[:, None, None], -math.inf)
    m = p.amax(dim=3, keepdim=True)
    p.sub_(m.clamp_min(-1e30)).exp_()              # a sequence without tokens: all zeros
    l = p.sum(dim=3, keepdim=True)
    o = (p @ v) / l.clamp_min(1e-30)
    return o.reshape(n, hq, D).to(q.dtype), (m + l.log()).reshape(n, hq)


def _plain_fork(s):
    s["ints"].copy_(s["ints0"])
    table, seq_len, ref = _views(s["ints"], s["rows"], s["width"])
    src, dst = s["src"].long(), s["dst"].long()
    length, page = seq_len[src], s["page"]
    full = length // page
    col = torch.arange(s["width"], device=src.device)
    t = table[src]
    ref.index_add_(0, t.reshape(-1).long(), (col < full[:, None]).reshape(-1).int())
    part = s["part"]                               # branches whose last page is begun: it is copied
    new = torch.argsort((ref > 0).int(), stable=True)[:part.numel()]
    at = full[part].long()
    old = t[part, at].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, new] = pool[:, old]
    t[part, at] = new.int()
    ref[new] = 1
    keep = col < (length + page - 1)[:, None] // page
    table[dst] = torch.where(keep, t, table[dst])
    seq_len[dst] = length
    shared = s["ints"].clone()
    ref.index_add_(0, t.reshape(-1).long(), -keep.reshape(-1).int())
    seq_len[dst] = 0
    return s["k_pool"], s["v_pool"], shared, s["ints"]


def _plain_compact(s):
    s["ints"].copy_(s["ints0"])
    table, seq_len, ref = _views(s["ints"], s["rows"], s["width"])
    taken = ref > 0
    ids = torch.arange(ref.numel(), device=ref.device)
    below = ids < taken.sum()
    src = torch.argsort((~(taken & ~below)).int(), stable=True)[:s["moved"]]
    dst = torch.argsort((~(~taken & below)).int(), stable=True)[:s["moved"]]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, dst] = pool[:, src]
    to = ids.int()
    to[src] = dst.int()
    col = torch.arange(s["width"], device=ref.device)
    table.copy_(torch.where(col < ((seq_len + s["page"] - 1) // s["page"])[:, None], to[table.long()], table))
    ref[dst] = ref[src]
    ref[src] = 0
    return s["k_pool"], s["v_pool"], s["ints"]


def _plain_append(s):
    s["ints"].copy_(s["ints0"])
    table, seq_len, ref = _views(s["ints"], s["rows"], s["width"])
    rows, page = s["slots"].long(), s["page"]
    pos = seq_len[rows]
    end = pos + s["add"]
    col = torch.arange(s["width"], device=rows.device)
    fresh = (col >= ((pos + page - 1) // page)[:, None]) & (col < ((end + page - 1) // page)[:, None])
    new = torch.argsort((ref > 0).int(), stable=True)[:s["need"]]
    t = table[rows]
    nth = (fresh.reshape(-1).cumsum(0) - 1).clamp(0, max(0, s["need"] - 1)).view_as(fresh)
    table[rows] = torch.where(fresh, new[nth].int(), t) if s["need"] else t
    ref[new] = 1
    seq_len[rows] = end
    token = torch.arange(s["total"], device=rows.device)
    which = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    p = pos[which] + token - s["cu"][which]
    at = table[rows[which], (p // page).long()].long()
    for pool, new_rows in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
        pool[0].transpose(1, 2)[at, (p % page).long()] = new_rows
    return s["k_pool"], s["v_pool"], s["ints"], pos


# -------------------------------------------------------------------------------- work and exact values
def work(case):
    esz = 4 if case["dtype"] == "f32" else 2
    op, hkv = case["op"], case["hkv"]
    if op in ("prompt", "train"):
        lens, hq = _ints(case["lens"]), case["hq"]
        T, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
        if op == "prompt":
            return {"bytes": T * D * esz * (2 * hq + 2 * hkv) + 4 * hq * T, "flops": 4 * D * hq * pairs}
        # q, k, v, d_o read, o, dq, dk, dv written; two products forward, five backward
        return {"bytes": T * D * esz * (4 * hq + 4 * hkv), "flops": 14 * D * hq * pairs}
    if op == "decode":
        lens, hq = _ints(case["lens"]), case["hq"]
        return {"bytes": sum(lens) * hkv * D * esz * 2 + len(lens) * hq * (2 * D * esz + 4),
                "flops": 4 * D * hq * sum(lens)}
    page = hkv * case["page"] * D * esz * 2        # K and V of one page of one layer
    if op == "fork":
        lens, ways = _ints(case["lens"]), case["ways"]
        part = sum(1 for x in lens if x % case["page"])
        # each begun page is read once and written for each branch
        ints = 4 * sum(-(-x // case["page"]) for x in lens) * (1 + 2 * ways)
        return {"bytes": part * (1 + ways) * page * case["layers"] + ints, "flops": 0}
    if op == "compact":
        # pages in use are spread at random: a used page lies behind the used part with probability 1 - fill
        used = case["pages"] * case["fill"]
        return {"bytes": 2 * used * (1 - case["fill"]) * page * case["layers"] + 8 * case["pages"], "flops": 0}
    return {"bytes": 2 * sum(_ints(case["add"])) * hkv * D * esz * 2, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "train"):
        return _exact_packed(s, op == "train")
    if op == "decode":
        return _exact_decode(s)
    if op == "append":
        return _exact_append(s)
    return None                                    # page moves compute no numbers


def _exact_packed(s, train):
    q, k, v = (s[n].detach().double() for n in ("q", "k", "v"))
    T, hq, _ = q.shape
    G = hq // k.shape[1]
    o, dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=x.device) for x in (q, q, k, v))
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=q.device)
    for a, b in zip(s["ends"], s["ends"][1:]):
        for h in range(hq):
            # a band of rows at a time: row i of the sequence sees its keys 0..i
            for r in range(a, b, 4096):
                e = min(b, r + 4096)
                z = (q[r:e, h] @ k[a:e, h // G].T) / math.sqrt(D)
                z += torch.full_like(z, -math.inf).triu(r - a + 1)
                lse[h, r:e] = torch.logsumexp(z, dim=1)
                w = torch.exp(z - lse[h, r:e, None])
                o[r:e, h] = w @ v[a:e, h // G]
                if train:
                    g = s["d_o"][r:e, h].double()
                    dw = g @ v[a:e, h // G].T
                    dz = w * (dw - (w * dw).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[r:e, h] = dz @ k[a:e, h // G]
                    dk[a:e, h // G] += dz.T @ q[r:e, h]
                    dv[a:e, h // G] += w.T @ g
    return (o, dq, dk, dv) if train else (o, lse)


def _exact_decode(s):
    table, seq_len, _ = _views(s["ints"], s["rows"], s["width"])
    n, hq, _ = s["q"].shape
    o = torch.zeros(n, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(seq_len.tolist()):
        if length:
            ids = table[i, :-(-length // s["page"])].long()
            k, v = (s[p][0, ids].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :length] for p in ("k_pool", "v_pool"))
            z = torch.einsum("hgd,hld->hgl", s["q"][i].double().view(k.shape[0], -1, D), k) / math.sqrt(D)
            lse[i] = torch.logsumexp(z, dim=2).flatten()
            o[i] = torch.einsum("hgl,hld->hgd", torch.softmax(z, dim=2), v).reshape(hq, D)
    return o, lse


def _exact_append(s):
    table, seq_len, ref = _views(s["ints"], s["rows"], s["width"])
    free = iter((ref == 0).nonzero().flatten().tolist())
    pos, add = seq_len.tolist(), s["add"].tolist()
    t, page, begin = table.tolist(), s["page"], s["cu"].tolist()
    for i in range(len(pos)):
        for c in range(-(-pos[i] // page), -(-(pos[i] + add[i]) // page)):
            t[i][c] = next(free)
        p = torch.arange(pos[i], pos[i] + add[i], device="cuda")
        at = torch.tensor(t[i], device="cuda")[p // page]
        for pool, x in (("k_pool", "k"), ("v_pool", "v")):
            s[pool][0][at, :, p % page] = s[x][begin[i]:begin[i + 1]]
    return s["k_pool"], s["v_pool"], None, None
