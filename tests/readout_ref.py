"""Plain float64 attention over packed and cached sequences, with the error that a kernel may make.

The bounds follow the kernels' arithmetic.  u is the unit roundoff of the type (half a step): products
and sums are in float32 (u32 = 2^-24, one rounding per term in any order: n u32 sum |terms|), the
probabilities and dS enter the second product rounded to the type, outputs are rounded once.
  score      es  = 129 u32 scale sum |q||k|                      (128 products, one scaling)
  p          rho = 2 max(es) + 16 u32 + n u32                    (relative: its score, the row's lse, exp, sum)
  o          sum p |v| (u + rho + n u32) + u |o|
  delta      sum |do| (error of o) + 129 u32 sum |do||o|
  dP         129 u32 sum |do||v|
  dS         p (e_dP + e_delta) + |dS| (rho + u)
  dQ, dK     scale sum e_dS |k| (|q|) + n u32 scale sum |dS||k| + u |result|;  dV like o
"""
import math

import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, mask, scale, dtype):
    """q [h, n, D], k, v [h, m, D] (already one per query head), mask [n, m] True where attended.
    Returns a dict of o, lse and bounds; rows without a key give 0 and -inf."""
    q, k, v = (x.double() for x in (q, k, v))
    u, m = unit(dtype), k.shape[1]
    s = scale * (q @ k.transpose(1, 2))
    es = 129 * U32 * scale * (q.abs() @ k.abs().transpose(1, 2))
    s = torch.where(mask, s, -math.inf)
    es = torch.where(mask, es, 0.0).amax(dim=2, keepdim=True) if m else torch.zeros(*s.shape[:2], 1, device=s.device)
    lse = torch.logsumexp(s, dim=2, keepdim=True) if m else torch.full_like(es, -math.inf)
    p = torch.where(mask, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)), 0.0)
    o = p @ v
    rho = 2 * es + (16 + m) * U32
    absv = p @ v.abs()
    return {"p": p, "o": o, "lse": lse[..., 0], "rho": rho, "e_o": absv * (u * (dtype != torch.float32) + rho + m * U32)
            + u * o.abs(), "e_lse": (es + (16 + m) * U32)[..., 0] + 4 * U32 * lse[..., 0].abs().nan_to_num(posinf=0.0)}


def attend_bwd(q, k, v, mask, scale, d_o, dtype):
    """Adds dq, dk, dv (per query head) and their bounds."""
    f = attend(q, k, v, mask, scale, dtype)
    q, k, v, g = (x.double() for x in (q, k, v, d_o))
    n, m = q.shape[1], k.shape[1]
    u = unit(dtype)
    ur = u if dtype != torch.float32 else 0.0          # roundings of p and dS before the second product
    p, rho = f["p"], f["rho"]
    dp = g @ v.transpose(1, 2)
    delta = (g * f["o"]).sum(dim=2, keepdim=True)
    e_delta = (g.abs() * (f["e_o"] + 129 * U32 * f["o"].abs())).sum(dim=2, keepdim=True)
    e_dp = 129 * U32 * (g.abs() @ v.abs().transpose(1, 2))
    ds = p * (dp - delta)
    e_ds = p * (e_dp + e_delta) + ds.abs() * (rho + ur + 4 * U32)
    f["dq"] = scale * (ds @ k)
    f["e_dq"] = scale * ((e_ds + m * U32 * ds.abs()) @ k.abs()) + u * f["dq"].abs()
    f["dk"] = scale * (ds.transpose(1, 2) @ q)
    f["e_dk"] = scale * ((e_ds + 8 * n * U32 * ds.abs()).transpose(1, 2) @ q.abs())
    f["dv"] = p.transpose(1, 2) @ g
    f["e_dv"] = (p * (rho + ur + 8 * n * U32)).transpose(1, 2) @ g.abs()
    return f


def packed(q, k, v, lens, scale=None, d_o=None):
    """The whole packed batch: {name: value, "e_" + name: bound} in the layouts of the library; rows of no
    sequence are zeros (lse: -inf) with bound 0."""
    T, Hq, D = q.shape
    Hkv, G, dtype = k.shape[1], q.shape[1] // k.shape[1], q.dtype
    scale = scale or 1.0 / math.sqrt(D)
    z = lambda h: torch.zeros(T, h, D, dtype=torch.float64, device=q.device)
    out = {"o": z(Hq), "lse": torch.full((Hq, T), -math.inf, dtype=torch.float64, device=q.device),
           "dq": z(Hq), "dk": z(Hkv), "dv": z(Hkv)}
    out.update({"e_" + n: torch.zeros_like(x) for n, x in list(out.items())})
    a = 0
    for n in lens:
        b = a + n
        if n:
            h = lambda x, r: x[a:b].transpose(0, 1).repeat_interleave(r, dim=0)
            mask = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
            args = (h(q, 1), h(k, G), h(v, G), mask, scale)
            f = attend(*args, dtype) if d_o is None else attend_bwd(*args, h(d_o, 1), dtype)
            for x in ("lse", "e_lse"):
                out[x][:, a:b] = f[x]
            for x in ("o", "e_o") + (("dq", "e_dq") if d_o is not None else ()):
                out[x][a:b] = f[x].transpose(0, 1)
            if d_o is not None:                        # the KV head's gradient: the sum over its query heads
                for x in ("dk", "dv", "e_dk", "e_dv"):
                    out[x][a:b] = f[x].view(Hkv, G, n, D).sum(1).transpose(0, 1)
        a = b
    if d_o is not None:
        for x in ("dk", "dv"):
            out["e_" + x] += unit(dtype) * out[x].abs()
    return out


def check(got, ref, name):
    """|got - ref| <= bound everywhere, equal where ref is not finite."""
    want, e = ref[name], ref["e_" + name]
    got = got.double()
    assert got.shape == want.shape, name
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{name}: non-finite values differ"
    over = torch.where(fin, (got - want).abs() - 1.0001 * e - 1e-30, -1.0)
    worst = over.amax().item() if over.numel() else -1.0
    assert worst <= 0, f"{name}: {int((over > 0).sum())} values off by up to {worst:.3e} more than they may be"
