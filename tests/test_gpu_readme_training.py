"""The training lines of README.md, run as they stand, in both types; every gradient
against the 64-bit definition (layer_ref) on the inputs that the lines give it."""
import os

import pytest
import torch

import layer_ref as R
import selective_state_space_83_amd as ssm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def training_lines():
    lines = open(README).read().splitlines()
    first = next(i for i, line in enumerate(lines) if line.startswith("hs = torch.empty(ssm.packed_states_shape("))
    return lines[first:lines.index("```", first)]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_training_lines(dtype):
    gen = torch.Generator().manual_seed(31)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    lengths, dim, N, K = [19, 0, 1, 44, 8], 96, 16, 4
    tokens = sum(lengths)
    offsets = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    row = lambda w: n(tokens, w).to(dtype).cuda()  # noqa: E731
    v = {"ssm": ssm, "torch": torch, "tokens": tokens, "dim": dim, "N": N, "offsets": offsets, "x": row(dim), "u": row(dim),
         "B": row(N), "C": row(N), "dy": row(dim), "residual": row(dim), "dtotal": row(dim), "D": n(dim).cuda(),
         "A": -torch.arange(1, N + 1.0).repeat(dim, 1).cuda() / 4, "cw": 0.5 * n(dim, K).cuda(), "cb": 0.1 * n(dim).cuda(),
         "weight": (1 + 0.1 * n(dim)).cuda(), "delta": (0.1 * torch.rand(tokens, dim, generator=gen)).to(dtype).cuda()}
    grads = []
    for line in training_lines():
        exec(line, v)
        if line.startswith("grads = "):
            grads.append(v["grads"])
    torch.cuda.synchronize()
    scan, conv, norm = grads
    want = R.scan(v["u"], v["delta"], v["A"], v["B"], v["C"], offsets, v["D"], dy=v["dy"])
    R.check("y", v["y"], *want["y"], R.scan_eps(max(lengths), False, dtype == BF16), dtype)
    for k in ("dx", "ddelta", "dA", "dB", "dC", "dD"):
        sums = tokens if k in ("dA", "dD") else dim if k in ("dB", "dC") else 0
        R.check(k, scan[k], *want[k], R.grad_eps(max(lengths), False, dtype == BF16, sums))
    spans = [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]
    want = R.conv(v["x"], v["cw"], v["cb"], spans, True, dy=scan["dx"].to(dtype))
    R.check("conv dx", conv["dx"], *want["dx"], R.CONV_EPS, dtype)
    for k in ("dweight", "dbias"):
        R.check("conv " + k, conv[k], *want[k], R.CONV_EPS + tokens * R.U32)
    s = R.f64(v["x"]) + R.f64(v["residual"])
    want = R.norm(v["x"], v["residual"], v["weight"], 1e-5, v["dy"], v["dtotal"], s)
    R.check("norm dx", norm["dx"], *want["dx"], 4 * R.norm_eps(dim), dtype)
    R.check("norm dweight", norm["dweight"], *want["dweight"], 2 * R.norm_eps(dim) + tokens * R.U32)


def test_a_layer_trained_in_bf16():
    """Norm, convolution and scan behind one another: every call's gradients, down to the
    norm's weight, are the definition's on what the call before it left."""
    gen = torch.Generator().manual_seed(32)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    lengths, dim, N, K = [33, 5, 0, 70], 128, 16, 4
    tokens = sum(lengths)
    offsets = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    spans = [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]
    row = lambda w: n(tokens, w).to(BF16).cuda()  # noqa: E731
    x, res, B, C, dout, dtotal = row(dim), row(dim), row(N), row(N), row(dim), row(dim)
    w, cw, cb = (1 + 0.1 * n(dim)).cuda(), 0.5 * n(dim, K).cuda(), 0.1 * n(dim).cuda()
    A, delta = -torch.arange(1, N + 1.0).repeat(dim, 1).cuda() / 4, (0.1 * torch.rand(tokens, dim, generator=gen)).to(BF16).cuda()
    y, total = ssm.add_rms_norm(x, res, w)
    u = ssm.short_conv(y, cw, cb, offsets)
    hs = torch.empty(ssm.packed_states_shape(tokens, dim, N), device="cuda")
    ssm.packed_scan(u, delta, A, B, C, offsets, h_saved=hs)
    g = ssm.packed_scan_bwd(u, delta, A, B, C, offsets, dout, hs, want_dD=False)
    du = g["dx"].to(BF16)
    c = ssm.short_conv_bwd(y, cw, du, cb, offsets)
    m = ssm.add_rms_norm_bwd(x, c["dx"], w, dsum=dtotal, residual=res)
    torch.cuda.synchronize()
    want = R.scan(u, delta, A, B, C, offsets, dy=dout)
    R.check("du", g["dx"], *want["dx"], R.grad_eps(max(lengths), False, True))
    R.check("dA", g["dA"], *want["dA"], R.grad_eps(max(lengths), False, True, tokens))
    want = R.conv(y, cw, cb, spans, True, dy=du)
    R.check("dy", c["dx"], *want["dx"], R.CONV_EPS, BF16)
    s = R.f64(x) + R.f64(res)
    want = R.norm(x, res, w, 1e-5, c["dx"], dtotal, s)
    R.check("dx", m["dx"], *want["dx"], 4 * R.norm_eps(dim), BF16)
    R.check("dweight", m["dweight"], *want["dweight"], 2 * R.norm_eps(dim) + tokens * R.U32)
    rounded = R.norm(x, res, w, 1e-5, c["dx"], dtotal, total)["dweight"][0]
    with pytest.raises(AssertionError):   # not those of the rounded sum
        R.check("rounded", rounded, *want["dweight"], 2 * R.norm_eps(dim) + tokens * R.U32)
