"""Plain 64-bit references of decay attention and the group norm (torch on the
CPU, from the definitions), with the magnitude of every output: the same sums
with each term replaced by its absolute value.

Tolerances.  An output entry is a sum of terms; in any order of summation its
rounding error is at most (number of roundings a term passes) x 2^-24 x the
entry's magnitude.

  fp32: a term passes at most 256 + 64 additions of its two contractions and a
        few products, and its decay factor carries the rounding of a sum of log
        decays: 2^-24 x (about 330) = 2e-5.
  bf16: each term has one operand rounded to bf16 (2^-9), the result is rounded
        once more (2^-9): 2^-8, doubled to 2^-7 where a gradient sums two such
        paths.  States keep fp32's bound: their products are formed from
        operands kept to 24 bits.
  The 2-norm of the error, where roundings add like independent ones: one bf16
        rounding is 1.7e-3 on average, three together below 3e-3: 5e-3.  fp32:
        2^-24 x sqrt(330) x a few: 1e-5.
  dlog_decay is a suffix sum of differences dq_i.q_i - dk_i.k_i whose common
        pairs cancel: its entries carry the roundings of that sum's terms, so
        its magnitude is that sum's.
"""
from __future__ import annotations

import torch

EPS32 = 2e-5
EPS16 = 2.0 ** -7
NORM32 = 1e-5
NORM16 = 5e-3


def attn(q, k, v, g, h0=None, lengths=None, dout=None, dh_last=None):
    """Outputs (and with dout the gradients) as a dict of (value, magnitude)."""
    d = torch.float64
    q, k, v, g = (t.detach().cpu().to(d) for t in (q, k, v, g))
    B, L, H, dv = v.shape
    Hk, dk = q.shape[2], q.shape[3]
    head = torch.arange(H) // max(1, H // max(1, Hk))
    q, k = q[:, :, head], k[:, :, head]
    zero = torch.zeros(B, H, dk, dv, dtype=d)
    h0_ = zero if h0 is None else h0.detach().cpu().to(d)
    n = [L] * B if lengths is None else [min(max(int(x), 0), L) for x in lengths.cpu()]
    live = torch.tensor([[t < n[b] for t in range(L)] for b in range(B)]).reshape(B, L)
    m = live[:, :, None, None]
    q, k, v = (torch.where(m, t, torch.zeros((), dtype=d)) for t in (q, k, v))
    a = torch.where(live[:, :, None], torch.exp(g), torch.ones((), dtype=d))[..., None, None]
    S, SA = [h0_], [h0_.abs()]
    for t in range(L):
        up = k[:, t, :, :, None] * v[:, t, :, None, :]
        S.append(S[-1] * a[:, t] + up)
        SA.append(SA[-1] * a[:, t] + up.abs())
    read = lambda s, x: (s * x[..., None]).sum(-2)  # noqa: E731
    o = torch.stack([read(S[t + 1], q[:, t]) for t in range(L)], 1) if L else v.clone()
    oa = torch.stack([read(SA[t + 1], q[:, t].abs()) for t in range(L)], 1) if L else v.clone()
    out = {"o": (o, oa), "h_last": (S[L], SA[L])}
    if dout is None:
        return out
    do = torch.where(m, dout.detach().cpu().to(d), torch.zeros((), dtype=d))
    P = zero if dh_last is None else dh_last.detach().cpu().to(d)
    G, GA = P.clone(), P.abs()
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    qa, ka, va = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, ga = torch.zeros_like(g), torch.zeros_like(g)
    suffix = (S[L].abs() * P.abs()).sum((-1, -2))
    suffix = torch.maximum(suffix, (SA[L] * GA).sum((-1, -2)))
    for t in range(L - 1, -1, -1):
        w = do[:, t, :, None, :] * q[:, t, :, :, None]
        G, GA = G + w, GA + w.abs()
        dq[:, t] = (S[t + 1] * do[:, t, :, None, :]).sum(-1)
        qa[:, t] = (SA[t + 1] * do[:, t, :, None, :].abs()).sum(-1)
        dkk[:, t] = (G * v[:, t, :, None, :]).sum(-1)
        ka[:, t] = (GA * v[:, t, :, None, :].abs()).sum(-1)
        dvv[:, t] = read(G, k[:, t])
        va[:, t] = read(GA, k[:, t].abs())
        suffix = suffix + (qa[:, t] * q[:, t].abs()).sum(-1) + (ka[:, t] * k[:, t].abs()).sum(-1)
        G, GA = G * a[:, t], GA * a[:, t]
        on = live[:, t, None]
        dg[:, t] = torch.where(on, (S[t] * G).sum((-1, -2)), torch.zeros((), dtype=d))
        ga[:, t] = torch.where(on, suffix, torch.zeros((), dtype=d))
    fold = lambda x: torch.where(m, x, torch.zeros((), dtype=d)).reshape(  # noqa: E731
        B, L, Hk, H // Hk if Hk else 1, dk).sum(3)
    out.update(dq=(fold(dq), fold(qa)), dk=(fold(dkk), fold(ka)),
               dv=(torch.where(m, dvv, torch.zeros((), dtype=d)), torch.where(m, va, torch.zeros((), dtype=d))),
               dlog_decay=(dg, ga), dh0=(G, GA))
    return out


def norm(x, groups, weight=None, bias=None, z=None, act=None, gate_first=False, rms=False, eps=1e-5,
         dy=None):
    """y (and with dy the gradients) as a dict of (value, magnitude).  The
    magnitude of a normalized value is |u - mean| r + |mean| r (the difference's
    operands); of a gradient the sum of its terms' sizes."""
    d = torch.float64
    f = lambda t: None if t is None else t.detach().cpu().to(d)  # noqa: E731
    x, w, b, z, dy = f(x), f(weight), f(bias), f(z), f(dy)
    shape, C = x.shape, x.shape[-1]
    w = torch.ones(C, dtype=d) if w is None else w
    b = torch.zeros(C, dtype=d) if b is None else b
    x = x.reshape(-1, C)
    z = None if z is None else z.reshape(-1, C)
    cut = (x.shape[0], groups, C // groups)
    sig = torch.sigmoid
    gate = None if z is None else z * sig(z)
    u = (x * gate if gate_first else x).reshape(cut)
    mean = torch.zeros(cut[:2] + (1,), dtype=d) if rms else u.mean(-1, keepdim=True)
    r = ((u - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    n, na = (u - mean) * r, (u.abs() + mean.abs()) * r
    n, na = n.reshape(-1, C), na.reshape(-1, C)
    a, aa = n * w + b, na * w.abs() + b.abs()
    if act == "silu":
        y, ya = a * sig(a), aa * (1 + aa * 0.25)
    elif z is not None and not gate_first:
        y, ya = a * gate, aa * gate.abs() * (1 + z.abs())
    else:
        y, ya = a, aa
    out = {"y": (y.reshape(shape), ya.reshape(shape))}
    if dy is None:
        return out
    dy = dy.reshape(-1, C)
    ds = lambda t: sig(t) * (1 + t * (1 - sig(t)))  # noqa: E731
    if act == "silu":
        da, daa = dy * ds(a), dy.abs() * (1 + aa)
    elif z is not None and not gate_first:
        da, daa = dy * gate, dy.abs() * gate.abs() * (1 + z.abs())
    else:
        da, daa = dy, dy.abs()
    out["dweight"] = ((da * n).sum(0), (daa * na).sum(0))
    out["dbias"] = (da.sum(0), daa.sum(0))
    dn, dna = (da * w).reshape(cut), (daa * w.abs()).reshape(cut)
    ng, nga = n.reshape(cut), na.reshape(cut)
    du = dn - ng * (dn * ng).mean(-1, keepdim=True)
    dua = dna + nga * (dna * nga).mean(-1, keepdim=True)
    if not rms:
        du, dua = du - dn.mean(-1, keepdim=True), dua + dna.mean(-1, keepdim=True)
    du, dua = (du * r).reshape(-1, C), (dua * r).reshape(-1, C)
    if z is not None and gate_first:
        out["dz"] = (du * x * ds(z), dua * x.abs() * (1 + z.abs()))
        du, dua = du * gate, dua * gate.abs() * (1 + z.abs())
    elif z is not None:
        out["dz"] = (dy * a * ds(z), dy.abs() * aa * (1 + z.abs()))
    out["dx"] = (du, dua)
    for name in ("dx", "dz"):
        if name in out:
            out[name] = tuple(t.reshape(shape) for t in out[name])
    return out


def check(name, got, ref, bf16, norm=True):
    """|got - ref| <= eps x magnitude for every entry, and the 2-norm's bound
    (with many entries; `norm` False leaves it out)."""
    value, mag = ref
    got = got.detach().cpu().to(torch.float64)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    err = (got - value).abs()
    bound = (EPS16 if bf16 else EPS32) * mag + 1e-30
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(k) for k in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d entries outside; first %s: got %g, reference %g, magnitude %g"
                             % (name, int(bad.sum()), bad.numel(), i, got[i], value[i], mag[i]))
    if norm and value.numel() >= 64 and float(value.norm()) > 1e-3 * float(mag.norm()):
        rel = float((got - value).norm() / value.norm())
        assert rel <= (NORM16 if bf16 else NORM32), "%s: relative error %.3g" % (name, rel)
