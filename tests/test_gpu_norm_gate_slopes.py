"""The gate's gradient where the gate is nearly open or shut: by its own size, element by element.

dgate is a product of factors near one and of the slope of the gate. Bound 1e-5 of the slope's
terms: e^-|z| by an argument rounded to 32 bits (|z| up to 30: 30 x 2^-24 = 1.8e-6 of it), the
exponential's and the reciprocal's own errors (2^-22 and 2^-23), ten more products, the norm's sum of
64 squares and its root (under 20 half steps of 2^-24 together: 1.2e-6)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_slope(act):
    import rwkv_linear_attention_wkv_b200 as W
    gen = torch.Generator().manual_seed(1)
    R, C, eps = 40, 64, 1e-6
    z = torch.linspace(-30, 30, R * C).reshape(R, C)
    h, dout = torch.randn(R, C, generator=gen), torch.randn(R, C, generator=gen)
    got = W.wkv_norm_gate_backward(h.cuda(), None, dout.cuda(), gate=z.cuda(), group=C, act=act,
                                   eps=eps)["dgate"].cpu().double()
    z, h, dout = z.double(), h.double(), dout.double()
    rest = (dout * h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)).abs()
    sig, off = torch.sigmoid(z), torch.sigmoid(-z)
    slope = sig * off if act == "sigmoid" else sig + z * sig * off
    terms = sig * off if act == "sigmoid" else sig + z.abs() * sig * off
    want = torch.sign(dout * h) * rest * slope
    worst = ((got - want).abs() / (rest * terms)).max()
    assert float(worst) <= 1e-5, float(worst)
