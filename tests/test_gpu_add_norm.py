"""The residual's addition with the rms norm on the GPU against its 64-bit definition:
types, widths, layouts, the 8-bit output and gradients."""
import pytest
import torch

import layer_ref as R
import selective_state_space_83_amd as ssm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, None), (BF16, None), (F32, F32), (BF16, BF16), (BF16, F32)]
WIDTHS = [1, 3, 8, 31, 64, 100, 128, 255, 256, 500, 512, 1000, 1024, 1536, 2048, 2560, 4096, 4097, 5120, 8192, 16384, 16392, 20001]


def make(rows, C, dtype, residual, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(8000 + seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return {"x": (scale * n(rows, C)).to(dtype).cuda(), "weight": (1 + 0.2 * n(C)).cuda(), "dy": n(rows, C).to(dtype).cuda(),
            "residual": None if residual is None else (2 * scale * n(rows, C)).to(residual).cuda(),
            "dsum": None if residual is None else n(rows, C).to(residual).cuda()}


def check(t, eps=1e-5, weight=True):
    w = t["weight"] if weight else None
    y, total = ssm.add_rms_norm(t["x"], t["residual"], w, eps=eps)
    g = ssm.add_rms_norm_bwd(total, t["dy"], w, dsum=t["dsum"], eps=eps)
    torch.cuda.synchronize()
    want = R.norm(t["x"], t["residual"], w, eps, t["dy"], t["dsum"], total)
    C, dt = t["x"].shape[-1], t["x"].dtype
    e = R.norm_eps(C)
    R.check("y", y, *want["y"], e, dt)
    if t["residual"] is None:
        assert total is t["x"]
    else:
        assert total.dtype == t["residual"].dtype
        R.check("total", total, *want["sum"], R.U32, total.dtype)
    assert ("dresidual" in g) == (total.dtype != dt)
    rows = t["x"].numel() // C
    R.check("dx", g["dx"], *want["dx"], 4 * e, dt)
    if "dresidual" in g:
        R.check("dresidual", g["dresidual"], *want["dx"], 4 * e, F32)
    R.check("dweight", g["dweight"], *want["dweight"], 2 * e + rows * R.U32)
    return y, total, g


def check_8bit(t, block, eps=1e-5):
    """The scales, and q within one rounding of y / scale."""
    q, scale, total = ssm.add_rms_norm_8bit(t["x"], t["residual"], t["weight"], eps=eps, block=block)
    torch.cuda.synchronize()
    want, mag = R.norm(t["x"], t["residual"], t["weight"], eps)["y"]
    C = t["x"].shape[-1]
    size = block or C
    assert q.dtype == torch.float8_e4m3fn and scale.shape == t["x"].shape[:-1] + (-(-C // size),)
    e = R.norm_eps(C)
    top = torch.stack([p.abs().amax(-1) for p in want.split(size, -1)], -1) / 448
    top = torch.where(top > 0, top.clamp(min=2.0 ** -126), torch.ones_like(top))
    R.check("scale", scale, top, top, 2 * e + 2 * R.U32)
    got, s = q.float().cpu().double(), scale.cpu().double().repeat_interleave(size, -1)[..., :C]
    # half a step of e4m3: 2^-4 of the value, 2^-10 below 2^-6
    v = want / s
    bound = torch.maximum(2.0 ** -4 * v.abs(), torch.tensor(2.0 ** -10, dtype=R.D)) * (1 + 4 * e) + 4 * e * v.abs() + 1e-30
    assert ((got - v).abs() <= bound).all()
    # nearest: away from the middle of two values it is the one the definition names
    near = R.to_e4m3(v.clamp(-448, 448))
    differ = got != near
    lo, hi = R.to_e4m3((v * (1 - 8 * e)).clamp(-448, 448)), R.to_e4m3((v * (1 + 8 * e)).clamp(-448, 448))
    assert not (differ & (lo == hi)).any()
    assert float(got.abs().max()) <= 448
    return q, scale, total


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(C, types):
    check(make(5, C, *types, seed=C))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_widths_8bit(C, types):
    t = make(5, C, *types, seed=C)
    for block in (0, 32, 128, 256):
        check_8bit(t, block)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 63, 300, 2100, 9001])
def test_rows(rows, types):
    t = make(rows, 192, *types, seed=rows)
    check(t)
    check_8bit(t, 64)
    check_8bit(t, 0)
    check(t, weight=False)


def test_rows_dealt_several_to_a_lane():
    """Enough rows that a lane walks several, widths of each dealing."""
    for C in (8, 64, 512, 520, 2560):
        t = make(max(300, (1 << 21) // C), C, BF16, F32, seed=C)
        check(t)
        check_8bit(t, 32)


@pytest.mark.parametrize("types", TYPES)
def test_strided_rows(types):
    """Slices of wider rows, on and off 16 bytes; a (batch, L, channels) view; broadcasts."""
    for off in (0, 1, 8):
        t = make(24, 3 * 64 + 16, *types, seed=off)
        for n in ("x", "residual", "dy", "dsum"):
            if t[n] is not None:
                t[n] = t[n][:, off:off + 128]
        t["weight"] = t["weight"][:128].contiguous()
        y, total, g = check(t)
        check_8bit(t, 32)
        check_8bit(t, 0)
        u = {k: v if v is None or v.dim() == 1 else v.unflatten(0, (4, 6)) for k, v in t.items()}
        y3, _ = ssm.add_rms_norm(u["x"], u["residual"], u["weight"])
        assert torch.equal(y3.flatten(0, 1), y)
        q3, s3, _ = ssm.add_rms_norm_8bit(u["x"], u["residual"], u["weight"], block=64)
        assert q3.shape == (4, 6, 128) and s3.shape == (4, 6, 2)
    t["x"] = t["x"][:1].expand(24, 128)
    check(t)


@pytest.mark.parametrize("residual", [BF16, F32])
@pytest.mark.parametrize("C", [512, 500, 20000])
def test_the_sum_in_the_residuals_place(C, residual):
    t = make(33, C, BF16, residual, seed=C)
    y, total = ssm.add_rms_norm(t["x"], t["residual"], t["weight"])
    q, s, total8 = ssm.add_rms_norm_8bit(t["x"], t["residual"], t["weight"], block=32)
    r1, r2 = t["residual"].clone(), t["residual"].clone()
    y1, same = ssm.add_rms_norm(t["x"], r1, t["weight"], total=r1)
    q2, s2, same2 = ssm.add_rms_norm_8bit(t["x"], r2, t["weight"], block=32, total=r2)
    assert same is r1 and torch.equal(y1, y) and torch.equal(r1, total)
    assert same2 is r2 and torch.equal(q2.float(), q.float()) and torch.equal(s2, s) and torch.equal(r2, total8)
    none = ssm.add_rms_norm(t["x"], t["residual"], t["weight"], want_total=False)
    assert none[1] is None and torch.equal(none[0], y)


def test_magnitudes():
    """Large, small, zero and non-finite rows."""
    for scale in (1e-12, 1e15):
        t = make(6, 256, F32, F32, seed=5, scale=scale)
        t["dsum"] = None
        check(t, eps=0.0 if scale > 1 else 1e-5)
        check_8bit(t, 64, eps=0.0 if scale > 1 else 1e-5)
    x = torch.zeros(3, 256, device="cuda")
    y, _ = ssm.add_rms_norm(x)
    q, s, _ = ssm.add_rms_norm_8bit(x, block=64)
    assert (y == 0).all() and (q.float() == 0).all() and (s == 1).all()
    t = make(6, 256, F32, F32, seed=6)
    clean, _ = ssm.add_rms_norm(t["x"], t["residual"], t["weight"])
    cq, cs, _ = ssm.add_rms_norm_8bit(t["x"], t["residual"], t["weight"], block=32)
    t["x"][2, 5] = float("nan")
    t["residual"][4, 100] = float("inf")
    y, _ = ssm.add_rms_norm(t["x"], t["residual"], t["weight"])
    q, s, _ = ssm.add_rms_norm_8bit(t["x"], t["residual"], t["weight"], block=32)
    keep = [0, 1, 3, 5]
    assert torch.isnan(y[2]).all() and torch.isnan(y[4, 100]) and torch.equal(y[keep], clean[keep])
    assert torch.isnan(q[2].float()).all() and torch.isnan(q[4].float()[100])
    assert torch.equal(q[keep].float(), cq[keep].float()) and torch.equal(s[keep], cs[keep])


def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(3)
    t = make(5, 48, F32, F32, seed=8)
    _, total, g = check(t)
    for name, gn in (("x", "dx"), ("residual", "dx"), ("weight", "dweight")):
        d = torch.randn(t[name].shape, generator=gen).double()

        def loss(e):
            u = {k: v.cpu().double() for k, v in t.items()}
            u[name] = u[name] + e * d
            o = R.norm(u["x"], u["residual"], u["weight"], 1e-5)
            return float((o["y"][0] * u["dy"]).sum() + (o["sum"][0] * u["dsum"]).sum())

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = g[gn].cpu().double() * d
        # the kept sum is rounded once (2^-24); the differences' own error about 1e-9
        assert abs(float(terms.sum()) - want) <= (16 * R.norm_eps(48) + 1e-7) * float(terms.abs().sum()), name


def test_gradients_asked_for():
    t = make(700, 96, BF16, F32, seed=9)
    full = ssm.add_rms_norm_bwd(t["residual"], t["dy"], t["weight"], dsum=t["dsum"])
    some = ssm.add_rms_norm_bwd(t["residual"], t["dy"], t["weight"], dsum=t["dsum"], want_dweight=False)
    again = ssm.add_rms_norm_bwd(t["residual"], t["dy"], t["weight"], dsum=t["dsum"])
    assert set(some) == {"dx", "dresidual"} and torch.equal(some["dx"], full["dx"])
    assert all(torch.equal(full[k], again[k]) for k in full)
    alone = ssm.add_rms_norm_bwd(t["residual"], t["dy"], t["weight"])
    zero = ssm.add_rms_norm_bwd(t["residual"], t["dy"], t["weight"], dsum=torch.zeros_like(t["dsum"]))
    assert torch.equal(alone["dresidual"], zero["dresidual"])


def test_offsets_past_32_bits():
    far = 3 << 29
    u = make(3, 64, F32, F32, seed=12)
    bufs = {k: torch.empty(far * 2 + 64, device="cuda").as_strided((3, 64), (far, 1)).copy_(u[k]) for k in ("x", "residual", "dy")}
    a, b = check(u), check(dict(u, **bufs))
    assert torch.equal(a[0], b[0]) and torch.equal(a[2]["dx"], b[2]["dx"])


def test_graph_replays():
    t = make(100, 256, BF16, F32, seed=13)

    def body():
        y, total = ssm.add_rms_norm(t["x"], t["residual"], t["weight"])
        q, s, _ = ssm.add_rms_norm_8bit(t["x"], t["residual"], t["weight"], block=64)
        g = ssm.add_rms_norm_bwd(total, t["dy"], t["weight"], dsum=t["dsum"])
        return [y, total, q.view(torch.uint8), s] + [g[n] for n in sorted(g)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = body()
    for i in range(4):
        u = make(100, 256, BF16, F32, seed=300 + i)
        for n in t:
            t[n].copy_(u[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for a, b in zip(got, body()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_empty():
    x = torch.zeros(0, 64, device="cuda")
    assert ssm.add_rms_norm(x)[0].shape == (0, 64)
    g = ssm.add_rms_norm_bwd(x, x)
    assert (g["dweight"] == 0).all()
    q, s, _ = ssm.add_rms_norm_8bit(x, block=32)
    assert q.shape == (0, 64) and s.shape == (0, 2)


def test_binding_refuses():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for args, kw in [((x.cpu(),), {}), ((x.half(),), {}), ((x.t(),), {}), ((x, x[:2]), {}), ((x.bfloat16(), x.half()), {}),
                     ((x, x.bfloat16()), {}), ((x, None, w[:3]), {}), ((x, None, w.bfloat16()), {}), ((x,), dict(eps=-1.0)),
                     ((x,), dict(eps=float("nan"))), ((x,), dict(y=x)), ((x, x.clone()), dict(total=x)), ((x,), dict(total=x.clone())),
                     ((x, x.clone()), dict(total=x.bfloat16())), ((x,), dict(y=x.bfloat16()))]:
        with pytest.raises(ValueError):
            ssm.add_rms_norm(*args, **kw)
    for block in (16, 48, 512, -32):
        with pytest.raises(ValueError):
            ssm.add_rms_norm_8bit(x, block=block)
    for args, kw in [((x, x[:2]), {}), ((x.bfloat16(), x), {}), ((x, x), dict(dsum=x.bfloat16())), ((x, x), dict(weight=w[:2]))]:
        with pytest.raises(ValueError):
            ssm.add_rms_norm_bwd(*args, **kw)
