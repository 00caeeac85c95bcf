"""Plain 64-bit references (torch on the CPU, from the definitions) of the packed
scan, the short convolution and the residual rms norm, with the magnitude of every
output: the same sums with each term replaced by its absolute value.

Tolerances.  u = 2^-24 is half a step of fp32, 2^-8 of bf16, 2^-4 of e4m3, all
relative to the value.  An output entry is a sum of terms; its error is at most
(roundings that a term passes) x u x its magnitude, in any order.

  scan    A term is the input of one token, carried over at most L others.  A step
          rounds the exponent's product, relative to its size |z| <= 2 here (2 u),
          the exp (1 ulp: 2 u), the product and the sum (2 u), and where a chunk's
          summary is joined the same once more: 8 u a step.  In front and behind:
          the input factor, C's product, the sum over 16 states, D, the gate's
          exp, reciprocal and products: below 64 u.  So (8 L + 64) u.
          ZOH's factor (a - 1) / A loses 2 u / |z|, taken only above |z| = 0.03
          (fp32 inputs) or 2^-13 (bf16): 67 u or 2^-10 more.
          A gradient passes the recurrence twice (the state's and the adjoint's)
          and a sum over at most `sums` tokens or channels: (16 L + 128 + sums) u.
          With ZOH its factors' direct forms lose up to 4 u / z^2, down to
          |z| = 1/16 (fp32) or 1/64 (bf16): 2^-14 or 2^-10 more.
  conv    Four products and sums, the bias, silu (exp, reciprocal, three products,
          whose argument's error reaches the exp times its size, below 16 here):
          48 u of the magnitude; sums over n tokens: n u more.
  norm    s, a sum over C squares (C / 16 + 16 additions a lane and across lanes),
          the root, two products: halved by the root: (C / 16 + 32) u.
  Each ends with one rounding to the output's type.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
D = torch.float64


def f64(t):
    return None if t is None else t.detach().cpu().to(D)


def check(name, got, value, magnitude, eps, kind=torch.float32):
    """|got - value| <= eps x magnitude + one rounding of the value to `kind`."""
    got, value = f64(got), value.to(D)
    assert got.shape == value.shape, (name, got.shape, value.shape)
    bound = eps * magnitude + HALF[kind] * (value.abs() + eps * magnitude) + 1e-38
    bad = ~((got - value).abs() <= bound)
    if bad.any():
        i = tuple(int(k) for k in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d outside; first %s: got %g, reference %g, bound %g"
                             % (name, int(bad.sum()), bad.numel(), i, got[i], value[i], bound[i]))


# ---------------------------------------------------------------------------
# packed scan
# ---------------------------------------------------------------------------

def scan_eps(L, zoh, low):
    return (8 * L + 64) * U32 + ((2.0 ** -10 if low else 67 * U32) if zoh else 0)


def grad_eps(L, zoh, low, sums=0):
    return (16 * L + 128 + sums) * U32 + ((2.0 ** -10 if low else 2.0 ** -14) if zoh else 0)


def _zoh(z, A, dl):
    """(exp(z) - 1) / A, and its limit."""
    return torch.where(A != 0, torch.expm1(z) / torch.where(A != 0, A, torch.ones_like(A)), dl.expand_as(z))


def scan(x, delta, A, B, C, offsets, Dskip=None, h0=None, slots=None, resume=None, zoh=False, bias=None, softplus=False,
         z=None, dy=None, dh_last=None):
    """Values and magnitudes: dict name -> (value, magnitude).  y is NaN at tokens of no
    sequence; h_last has an entry per sequence (None where its slot is out of range)."""
    x, delta, A, B, C, Dskip, h0, bias, z, dy, dh_last = map(f64, (x, delta, A, B, C, Dskip, h0, bias, z, dy, dh_last))
    off = [int(v) for v in offsets.cpu()]
    S, (T, dim), N = len(off) - 1, x.shape, A.shape[1]
    place = list(range(S)) if slots is None else [int(v) for v in slots.cpu()]
    taken = [True] * S if resume is None else [bool(v) for v in resume.cpu()]
    if bias is not None:
        delta = delta + bias
    if softplus:
        delta = torch.clamp(delta, min=0) + torch.log1p(torch.exp(-delta.abs()))
    Dk = torch.zeros(dim, dtype=D) if Dskip is None else Dskip
    y, ym = torch.full((T, dim), float("nan"), dtype=D), torch.zeros(T, dim, dtype=D)
    zero = torch.zeros(dim, N, dtype=D)
    last, states = [], {}
    for s in range(S):
        ok = h0 is not None and taken[s] and 0 <= place[s] < h0.shape[0]
        h = h0[place[s]] if ok else zero
        hm = h.abs()
        for t in range(off[s], off[s + 1]):
            states[t] = (h, hm)
            dl = delta[t][:, None]
            a = torch.exp(dl * A)
            f = _zoh(dl * A, A, dl) if zoh else dl
            u = f * B[t] * x[t][:, None]
            h, hm = a * h + u, a * hm + u.abs()
            y[t] = h @ C[t] + Dk * x[t]
            ym[t] = hm @ C[t].abs() + (Dk * x[t]).abs()
        last.append((h, hm))
    if z is not None:
        g = z * torch.sigmoid(z)
        y, ym = y * g, ym * g.abs() * (1 + z.abs())
    out = {"y": (y, ym), "h_last": (torch.stack([v for v, _ in last]) if S else torch.zeros(0, dim, N, dtype=D),
                                    torch.stack([m for _, m in last]) if S else torch.zeros(0, dim, N, dtype=D)),
           "states": states}
    if dy is None:
        return out
    shapes = {"dx": x.shape, "ddelta": x.shape, "dA": A.shape, "dB": B.shape, "dC": C.shape, "dD": (dim,),
              "dh0": (S, dim, N)}
    v = {k: torch.zeros(s, dtype=D) for k, s in shapes.items()}
    m = {k: torch.zeros(s, dtype=D) for k, s in shapes.items()}
    for s in range(S):
        p = zero if dh_last is None else dh_last[s]
        pm = p.abs()
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            h, hm = states[t]
            dl, dyt, ut = delta[t][:, None], dy[t][:, None], x[t][:, None]
            e = dl * A
            a = torch.exp(e)
            f = _zoh(e, A, dl) if zoh else dl.expand_as(e)
            u = f * B[t] * ut
            p, pm = p + dyt * C[t], pm + (dyt * C[t]).abs()
            v["dC"][t], m["dC"][t] = (dyt * (a * h + u)).sum(0), (dyt.abs() * (a * hm + u.abs())).sum(0)
            v["dB"][t], m["dB"][t] = (p * f * ut).sum(0), (pm * (f * ut).abs()).sum(0)
            v["dx"][t] = (p * f * B[t]).sum(1) + Dk * dy[t]
            m["dx"][t] = (pm * (f * B[t]).abs()).sum(1) + (Dk * dy[t]).abs()
            fd = a if zoh else torch.ones_like(e)
            v["ddelta"][t] = (p * a * h * A + p * fd * B[t] * ut).sum(1)
            m["ddelta"][t] = (pm * a * hm * A.abs() + pm * (fd * B[t] * ut).abs()).sum(1)
            # d f / d A: Delta^2 (1/2 + z/3 + ...)
            fa = dl * dl * torch.where(e.abs() < 1e-3, 0.5 + e / 3 + e * e / 8,
                                       (e * a - torch.expm1(e)) / torch.where(e == 0, torch.ones_like(e), e * e)) if zoh else 0 * e
            v["dA"] += p * a * h * dl + p * fa * B[t] * ut
            m["dA"] += pm * a * hm * dl.abs() + pm * (fa * B[t] * ut).abs()
            v["dD"] += dy[t] * x[t]
            m["dD"] += (dy[t] * x[t]).abs()
            p, pm = p * a, pm * a
        v["dh0"][s], m["dh0"][s] = p, pm
    out.update({k: (v[k], m[k]) for k in v})
    return out


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------

CONV_EPS = 48 * U32


def conv(x, weight, bias, spans, act, windows=None, dy=None):
    """x (tokens, channels); spans: (first, end) of every sequence; windows: their inputs
    before, (channels, K - 1) each or None.  y is NaN at tokens of no sequence."""
    x, w, b, dy = f64(x), f64(weight), f64(bias), f64(dy)
    T, (C, K) = x.shape[0], w.shape
    b = torch.zeros(C, dtype=D) if b is None else b
    y, ym = torch.full((T, C), float("nan"), dtype=D), torch.zeros(T, C, dtype=D)
    dx, dxm = torch.zeros(T, C, dtype=D), torch.zeros(T, C, dtype=D)
    dw, dwm, db, dbm = (torch.zeros(s, dtype=D) for s in ((C, K), (C, K), (C,), (C,)))
    moved = []
    for i, (lo, hi) in enumerate(spans):
        win = torch.zeros(C, K - 1, dtype=D) if windows is None or windows[i] is None else f64(windows[i])
        line = torch.cat([win.t(), x[lo:hi]])
        n = hi - lo
        a = b + sum(w[:, k] * line[k:k + n] for k in range(K))
        am = b.abs() + sum((w[:, k] * line[k:k + n]).abs() for k in range(K))
        g = torch.sigmoid(a)
        y[lo:hi] = a * g if act else a
        ym[lo:hi] = am * (1 + a.abs()) if act else am
        moved.append(line[n:].t())
        if dy is None:
            continue
        d = dy[lo:hi]
        da = d * g * (1 + a * (1 - g)) if act else d
        dam = d.abs() * (1 + am) if act else d.abs()
        db += da.sum(0)
        dbm += dam.sum(0)
        dl, dlm = torch.zeros_like(line), torch.zeros_like(line)
        for k in range(K):
            dl[k:k + n] += w[:, k] * da
            dlm[k:k + n] += (w[:, k]).abs() * dam
            dw[:, k] += (da * line[k:k + n]).sum(0)
            dwm[:, k] += (dam * line[k:k + n].abs()).sum(0)
        dx[lo:hi], dxm[lo:hi] = dl[K - 1:], dlm[K - 1:]
    return {"y": (y, ym), "moved": moved, "dx": (dx, dxm), "dweight": (dw, dwm), "dbias": (db, dbm)}


# ---------------------------------------------------------------------------
# residual and norm
# ---------------------------------------------------------------------------

def norm_eps(C):
    return (C / 16 + 32) * U32


def norm(x, residual, weight, eps, dy=None, dsum=None, total=None):
    """y and s; with dy the gradients, from the kept `total`."""
    x, residual, weight, dy, dsum, total = map(f64, (x, residual, weight, dy, dsum, total))
    C = x.shape[-1]
    w = torch.ones(C, dtype=D) if weight is None else weight
    s = x if residual is None else x + residual
    r = (s.square().sum(-1, keepdim=True) / C + eps).rsqrt()
    out = {"y": (s * r * w, (s * r * w).abs()), "sum": (s, s.abs())}
    if dy is None:
        return out
    s = total
    r = (s.square().sum(-1, keepdim=True) / C + eps).rsqrt()
    n, dn = s * r, dy * w
    mean, meanm = (dn * n).sum(-1, keepdim=True) / C, (dn * n).abs().sum(-1, keepdim=True) / C
    ds, dsm = r * (dn - n * mean), r * (dn.abs() + n.abs() * meanm)
    if dsum is not None:
        ds, dsm = ds + dsum, dsm + dsum.abs()
    flat = lambda t: t.reshape(-1, C).sum(0)  # noqa: E731
    return dict(out, dx=(ds, dsm), dweight=(flat(dy * n), flat((dy * n).abs())))


def to_e4m3(q):
    """Nearest e4m3 value (ties to even) of q, |q| <= 448."""
    unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(q / unit) * unit
