"""Where NaN and infinities of one token go in decay attention: to the outputs
that the recurrence takes them to, and no others.  A causal model's earlier
tokens do not see a later one, whatever it holds."""
import pytest
import torch

import mixer_ref as R
import selective_state_space_83_amd as ssm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
L, H, DK, DV = 150, 2, 32, 48


def make(dtype, seed):
    gen = torch.Generator().manual_seed(4000 + seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = {"q": n(1, L, 1, DK), "k": n(1, L, 1, DK) * DK ** -0.5, "v": n(1, L, H, DV), "dout": n(1, L, H, DV),
         "g": -0.2 * torch.rand(1, L, H, generator=gen)}
    return {name: x.to(dtype).cuda() for name, x in t.items()}


def same_places(name, got, ref, low):
    """Finite exactly where the recurrence is, and right there."""
    value, mag = ref
    fine = torch.isfinite(value)
    g = got.detach().cpu().double()
    wrong = torch.isfinite(g) != fine
    assert not wrong.any(), "%s: %d entries, first %s" % (name, int(wrong.sum()),
                                                          tuple(int(i) for i in torch.nonzero(wrong)[0]))
    zero = torch.zeros((), dtype=torch.float64)
    R.check(name, torch.where(fine, g, zero), (torch.where(fine, value, zero), torch.where(fine, mag, zero)), low,
            norm=False)


def planted(name):
    # the places in v and dout leave a head untouched, those in q and k are shared
    return {"q": (0, 85, 0, 3), "k": (0, 85, 0, 3), "v": (0, 85, 1, 7), "dout": (0, 85, 1, 7)}[name]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("span", [0, 64])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_outputs_before_the_token_stay(dtype, name, span, bad):
    t = make(dtype, 1)
    t[name][planted(name)] = bad
    ref = R.attn(t["q"], t["k"], t["v"], t["g"])
    o, h = ssm.decay_attn(t["q"], t["k"], t["v"], t["g"], span=span)
    torch.cuda.synchronize()
    same_places("o", o, ref["o"], dtype == BF16)
    same_places("h_last", h, ref["h_last"], False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("span", [0, 64])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_rows_the_token_does_not_reach(dtype, name, span, bad):
    t = make(dtype, 2)
    t[name][planted(name)] = bad
    ref = R.attn(t["q"], t["k"], t["v"], t["g"], dout=t["dout"])
    g = ssm.decay_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], span=span)
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv"):
        same_places(n, g[n], ref[n], dtype == BF16)
    same_places("dh0", g["dh0"], ref["dh0"], False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_heads(dtype):
    """Several waves and columns tiles: the token in each of them."""
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    for col in (0, 70, 130, 199):
        q, k, v = n(1, 100, 1, 128), n(1, 100, 1, 128) * 0.1, n(1, 100, 1, 200)
        g = -0.1 * torch.ones(1, 100, 1, device="cuda")
        v[0, 40, 0, col] = float("nan")
        ref = R.attn(q, k, v, g)
        o, h = ssm.decay_attn(q, k, v, g)
        torch.cuda.synchronize()
        same_places("o", o, ref["o"], dtype == BF16)
        same_places("h_last", h, ref["h_last"], False)
