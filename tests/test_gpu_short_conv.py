"""The short convolution on the GPU against its 64-bit definition: lengths, windows in
slots, strides, types, taps, single tokens and gradients."""
import pytest
import torch

import layer_ref as R
import selective_state_space_83_amd as ssm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LENGTHS = {"one token": [1], "one": [45], "ones": [1] * 40, "twos": [2] * 21, "empty ends": [0, 0, 5, 0, 12, 1, 0, 2, 0],
           "at tile ends": [30, 3, 62, 1, 2, 31], "long": [301, 5], "none": [0, 0]}


def make(lengths, C, K, dtype, seed=0, start=0, tail=0, slots=0, sliced=0):
    """Inputs; `start` and `tail` tokens of no sequence around them, as NaN; `slots`: windows
    in a cache of so many entries, half of the sequences resumed; `sliced`: columns before x
    in wider rows."""
    gen = torch.Generator().manual_seed(6000 + seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    S, T = len(lengths), start + sum(lengths) + tail
    cuts = [start]
    for v in lengths:
        cuts.append(cuts[-1] + v)
    live = torch.zeros(T, dtype=torch.bool)
    live[start:cuts[-1]] = True
    t = {"live": live, "spans": list(zip(cuts[:-1], cuts[1:])), "offsets": torch.tensor(cuts, dtype=torch.int32, device="cuda")}
    for k in ("x", "dy"):
        v = n(T, C)
        v[~live] = float("nan")
        wide = torch.full((T, C + sliced * 2), float("nan"))
        wide[:, sliced:sliced + C] = v
        t[k] = wide.to(dtype).cuda()[:, sliced:sliced + C]
    t["weight"], t["bias"] = n(C, K).cuda(), n(C).cuda()
    t["state"] = t["slots"] = t["resume"] = None
    if slots:
        t["state"] = n(slots, C, K - 1).cuda()
        t["slots"] = torch.randperm(slots, generator=gen)[:S].to(torch.int32).cuda()
        t["resume"] = (torch.rand(S, generator=gen) < 0.5).cuda()
    return t


def windows(t):
    if t["state"] is None:
        return None
    n = t["state"].shape[0]
    return [t["state"][int(p)] if bool(r) and 0 <= int(p) < n else None for p, r in zip(t["slots"], t["resume"])]


def check(t, act="silu", bias=True):
    b = t["bias"] if bias else None
    want = R.conv(t["x"], t["weight"], b, t["spans"], act == "silu", windows(t))
    y = torch.full(t["x"].shape, 7.5, dtype=t["x"].dtype, device="cuda")
    cache = None if t["state"] is None else t["state"].clone()
    ssm.short_conv(t["x"], t["weight"], b, offsets=t["offsets"], act=act, state=cache, slots=t["slots"], resume=t["resume"], y=y)
    torch.cuda.synchronize()
    live = t["live"]
    R.check("y", y.cpu()[live], want["y"][0][live], want["y"][1][live], R.CONV_EPS, y.dtype)
    assert (y.cpu()[~live] == 7.5).all()
    if cache is not None:
        left = set(range(cache.shape[0]))
        for p, w in zip(t["slots"].tolist(), want["moved"]):
            if 0 <= p < cache.shape[0]:
                left.discard(p)
                assert torch.equal(cache[p].cpu().double(), w)   # inputs, not rounded
        rest = sorted(left)
        assert torch.equal(cache[rest], t["state"][rest])
    return y


def check_gradients(t, act="silu", bias=True):
    b = t["bias"] if bias else None
    want = R.conv(t["x"], t["weight"], b, t["spans"], act == "silu", None, dy=t["dy"])
    g = ssm.short_conv_bwd(t["x"], t["weight"], t["dy"], b, offsets=t["offsets"], act=act)
    torch.cuda.synchronize()
    n = sum(h - l for l, h in t["spans"])
    R.check("dx", g["dx"], want["dx"][0], want["dx"][1], R.CONV_EPS, t["x"].dtype)
    for k in ("dweight", "dbias"):
        assert g[k].dtype == F32
        R.check(k, g[k], want[k][0], want[k][1], R.CONV_EPS + n * R.U32)
    return g


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_lengths(name, dtype, K):
    lengths = LENGTHS[name]
    for C in (24, 30):   # rows on 16 bytes, and off them
        check(make(lengths, C, K, dtype, seed=K))
        t = make(lengths, C, K, dtype, seed=10 + K, start=5, tail=30, slots=len(lengths) + 3 if K > 1 else 0)
        check(t)
        check_gradients(t)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [1, 7, 8, 64, 255, 256, 513, 1024])
def test_channels(C, dtype):
    lengths = [40, 0, 3, 90]
    t = make(lengths, C, 4, dtype, seed=C, slots=5, tail=1)
    check(t)
    check_gradients(t)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("sliced", [1, 8])
def test_strided_rows_without_bias_or_act(dtype, act, sliced):
    lengths = [33, 64]
    for K in (2, 4):
        t = make(lengths, 72, K, dtype, seed=30, sliced=sliced, slots=3)
        check(t, act, bias=False)
        check_gradients(t, act, bias=False)
    t = make(lengths, 72, 4, dtype, seed=31)
    t["x"] = t["x"][:1].expand(97, 72)
    check(t, act)
    check_gradients(t, act)


def test_windows_of_sequences_that_begin_at_every_place_of_a_tile():
    """The window is read by one tile only, wherever the sequence begins."""
    for first in range(26, 34):
        for K in (2, 3, 4):
            check(make([first, 200], 64, K, F32, seed=first, slots=2))
            check(make([first, 1, 2, 100], 64, K, BF16, seed=first, slots=4))


def test_slots_outside_the_cache():
    t = make([20, 30, 10], 64, 4, F32, seed=40, slots=5)
    t["slots"] = torch.tensor([3, -1, 5], dtype=torch.int32, device="cuda")
    t["resume"][:] = True
    check(t)


def test_padding_batch_of_equal_lengths():
    """(batch, L, channels) without offsets: every row a sequence."""
    t = make([50, 50, 50], 48, 4, BF16, seed=41, slots=3)
    y = check(t)
    cache = t["state"].clone()
    y3 = ssm.short_conv(t["x"].unflatten(0, (3, 50)), t["weight"], t["bias"], state=cache, slots=t["slots"], resume=t["resume"])
    assert torch.equal(y3.flatten(0, 1), y)
    g = check_gradients(t)
    g3 = ssm.short_conv_bwd(t["x"].unflatten(0, (3, 50)), t["weight"], t["dy"].unflatten(0, (3, 50)), t["bias"])
    assert torch.equal(g3["dx"].flatten(0, 1), g["dx"]) and torch.equal(g3["dweight"], g["dweight"])
    cache = t["state"].clone()
    y0 = ssm.short_conv(t["x"].new_empty(3, 0, 48), t["weight"], t["bias"], state=cache, slots=t["slots"], resume=t["resume"])
    assert y0.shape == (3, 0, 48)
    kept = t["state"].clone()
    kept[t["slots"].long()] *= t["resume"].float()[:, None, None]
    assert torch.equal(cache, kept)


def test_a_nan_stays_where_its_taps_reach():
    for K in (1, 2, 3, 4):
        t = make([60, 40], 64, K, F32, seed=42 + K)
        y = check(t)
        g = check_gradients(t)
        u = dict(t, x=t["x"].clone())
        u["x"][59] = float("nan")
        y2 = ssm.short_conv(u["x"], t["weight"], t["bias"], offsets=t["offsets"])
        assert torch.equal(y2[:59], y[:59]) and torch.isnan(y2[59]).all() and torch.equal(y2[60:], y[60:])
        u["x"] = t["x"].clone()
        u["x"][20] = float("inf")
        y2 = ssm.short_conv(u["x"], t["weight"], t["bias"], offsets=t["offsets"])
        keep = [i for i in range(100) if not 20 <= i < 20 + K]
        assert torch.equal(y2[keep], y[keep])
        dy = t["dy"].clone()
        dy[60] = float("nan")
        g2 = ssm.short_conv_bwd(t["x"], t["weight"], dy, t["bias"], offsets=t["offsets"])
        keep = [i for i in range(100) if i != 60]
        assert torch.equal(g2["dx"][keep], g["dx"][keep])


def test_silu_at_the_ends():
    x = torch.tensor([-1e30, -200.0, -88.0, 0.0, 88.0, 1e30], device="cuda").view(6, 1)
    w, off = torch.ones(1, 1, device="cuda"), torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    y = ssm.short_conv(x, w, offsets=off)
    g = ssm.short_conv_bwd(x, w, torch.ones_like(x), offsets=off)
    assert torch.isfinite(y).all() and torch.isfinite(g["dx"]).all()
    xd = x.double()
    assert torch.allclose(y.double(), torch.where(xd > -300, xd * torch.sigmoid(xd), 0 * xd), rtol=1e-6, atol=1e-30)


def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(9)
    for act in (None, "silu"):
        t = make([19, 0, 24], 12, 4, F32, seed=50)
        g = ssm.short_conv_bwd(t["x"], t["weight"], t["dy"], t["bias"], offsets=t["offsets"], act=act)
        for name, gn in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias")):
            d = torch.randn(t[name].shape, generator=gen).double()

            def loss(e):
                u = {k: t[k].cpu().double() for k in ("x", "weight", "bias")}
                u[name] = u[name] + e * d
                y = R.conv(u["x"], u["weight"], u["bias"], t["spans"], act == "silu")["y"][0]
                return float((y * t["dy"].cpu().double()).sum())

            want = (loss(1e-5) - loss(-1e-5)) / 2e-5
            terms = g[gn].cpu().double() * d
            # 43 terms a sum at most, the differences' own error about 1e-10 of the terms
            assert abs(float(terms.sum()) - want) <= (R.CONV_EPS * 4 + 43 * R.U32 + 1e-8) * float(terms.abs().sum()), (act, gn)


def test_gradients_asked_for():
    t = make([70, 58], 96, 4, F32, seed=51)
    args = (t["x"], t["weight"], t["dy"], t["bias"])
    full = ssm.short_conv_bwd(*args, offsets=t["offsets"])
    some = ssm.short_conv_bwd(*args, offsets=t["offsets"], want_dweight=False, want_dbias=False)
    one = ssm.short_conv_bwd(*args, offsets=t["offsets"], want_dweight=False)
    again = ssm.short_conv_bwd(*args, offsets=t["offsets"])
    torch.cuda.synchronize()
    assert set(some) == {"dx"} and torch.equal(some["dx"], full["dx"])
    assert set(one) == {"dx", "dbias"} and torch.equal(one["dbias"], full["dbias"])
    assert all(torch.equal(full[k], again[k]) for k in full)


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step(K, dtype):
    for batch, C, sliced in ((1, 1, 0), (5, 67, 0), (9, 256, 4), (6, 256, 1)):
        t = make([1] * batch, C, K, dtype, seed=60 + K, slots=batch + 2, sliced=sliced)
        t["resume"][:] = True
        if batch > 1:
            t["slots"][1] = -1
            t["slots"][2] = batch + 2
        for act in (None, "silu"):
            want = R.conv(t["x"], t["weight"], t["bias"], t["spans"], act, windows(t))
            cache = t["state"].clone()
            y = ssm.short_conv_step(cache, t["x"], t["weight"], t["bias"], act=act, slots=t["slots"])
            R.check("y", y, want["y"][0], want["y"][1], R.CONV_EPS, dtype)
            kept = {int(p): w for p, w in zip(t["slots"], want["moved"])}
            for p in range(batch + 2):
                assert torch.equal(cache[p].cpu().double(), kept.get(p, t["state"][p].cpu().double()))


def test_prompt_then_tokens():
    """Bit for bit what one call over all tokens gives: each output is the same sum."""
    t = make([40, 25], 64, 4, F32, seed=70, slots=4)
    whole = check(t)
    cache = t["state"].clone()
    rows = list(range(33)) + list(range(40, 58))
    off = torch.tensor([0, 33, 51], dtype=torch.int32, device="cuda")
    y = ssm.short_conv(t["x"][rows], t["weight"], t["bias"], offsets=off, state=cache, slots=t["slots"], resume=t["resume"])
    assert torch.equal(y, whole[rows])
    for i in range(7):
        y = ssm.short_conv_step(cache, t["x"][[33 + i, 58 + i]], t["weight"], t["bias"], slots=t["slots"])
        assert torch.equal(y, whole[[33 + i, 58 + i]])


def test_offsets_past_32_bits():
    wide = 1 << 26
    t = make([60, 30], 64, 4, BF16, seed=71, slots=2)
    far = {k: torch.empty(90 * wide, dtype=BF16, device="cuda").as_strided((90, 64), (wide, 1)).copy_(t[k]) for k in ("x", "dy")}
    y, g = check(t), check_gradients(t)
    u = dict(t, **far)
    assert torch.equal(check(u), y) and torch.equal(check_gradients(u)["dx"], g["dx"])


def test_graph_replays():
    t = make([90, 0, 35, 1], 128, 4, BF16, seed=80, slots=6)
    cache = t["state"].clone()

    def body():
        y = ssm.short_conv(t["x"], t["weight"], t["bias"], offsets=t["offsets"], state=cache, slots=t["slots"], resume=t["resume"])
        g = ssm.short_conv_bwd(t["x"], t["weight"], t["dy"], t["bias"], offsets=t["offsets"])
        y1 = ssm.short_conv_step(cache, t["x"][:4], t["weight"], t["bias"], slots=t["slots"])
        return [y, y1] + [g[k] for k in sorted(g)]

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
        w = make([90, 0, 35, 1], 128, 4, BF16, seed=81 + i)
        t["x"].copy_(w["x"])
        t["dy"].copy_(w["dy"])
        cut = torch.randint(0, 127, (3,), generator=torch.Generator().manual_seed(i)).sort().values
        t["offsets"][1:4] = cut.to(torch.int32).cuda()
        cache.copy_(t["state"])
        graph.replay()
        torch.cuda.synchronize()
        got, state = [o.clone() for o in outs], cache.clone()
        cache.copy_(t["state"])
        for a, b in zip(got, body()):
            assert torch.equal(a, b)
        assert torch.equal(state, cache)
        torch.cuda.synchronize()


def test_binding_refuses():
    t = make([8, 8], 32, 4, F32, seed=90, slots=3)
    call = lambda **c: ssm.short_conv(**dict(dict(x=t["x"], weight=t["weight"], bias=t["bias"], offsets=t["offsets"],  # noqa: E731
                                                  state=t["state"], slots=t["slots"], resume=t["resume"]), **c))
    call()
    for c in (dict(x=t["x"].cpu()), dict(x=t["x"].half()), dict(x=t["x"].t()), dict(x=t["x"][:, ::2]), dict(x=t["x"].unsqueeze(0)),
              dict(offsets=None), dict(offsets=t["offsets"].long()), dict(weight=t["weight"][:8]), dict(weight=t["weight"].bfloat16()),
              dict(weight=torch.zeros(32, 5, device="cuda")), dict(bias=t["bias"][:3]), dict(act="gelu"), dict(state=t["state"][:, :, :2]),
              dict(state=None), dict(slots=None), dict(slots=t["slots"].long()), dict(resume=t["resume"][:1]), dict(y=t["x"]),
              dict(y=t["x"].bfloat16())):
        with pytest.raises(ValueError):
            call(**c)
    for args in ((t["state"], t["x"][:4], t["weight"]), (t["state"].bfloat16(), t["x"][:3], t["weight"]),
                 (t["state"][:, :8], t["x"][:3], t["weight"])):
        with pytest.raises(ValueError):
            ssm.short_conv_step(*args)
    with pytest.raises(ValueError):
        ssm.short_conv_bwd(t["x"], t["weight"], t["dy"][:3], offsets=t["offsets"])
    with pytest.raises(ValueError):
        ssm.short_conv_bwd(t["x"], t["weight"], t["dy"].bfloat16(), offsets=t["offsets"])
