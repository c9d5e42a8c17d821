"""GPU parity of the norms around a block against their definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def make(R, C, dtype, seed, parts):
    """CPU inputs; parts: which optional inputs there are, by first letter (w, g, x, s, n)."""
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = {"h": (normal(R, C) * (0.2 + normal(R, 1).abs())).to(dtype), "weight": 1 + 0.3 * normal(C),
         "gate": normal(R, C).to(dtype), "x": (1.5 * normal(R, C)).to(dtype),
         "scale": 0.5 + 0.3 * normal(C), "next_weight": 1 + 0.3 * normal(C)}
    return {n: t if n == "h" or n[0] in parts else None for n, t in x.items()}


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def close(got, want, what, extra=0.0):
    """fp32: 1e-5 (1 + the row's largest); bf16 half a step on top. The sums behind a row's value
    are of up to 8192 squares (no cancellation: relative error below 14 half steps for a tree of
    14 levels), rsqrt is good to 2 steps, and a handful of products follow: under 40 half steps of
    2^-24 = 2.4e-6 of the terms, which no larger than a few times the row's largest value."""
    x = got.detach().cpu().double()
    assert x.shape == want.shape, what
    m = want.abs().amax(-1, keepdim=True)
    bound = 1e-5 * (1 + m) + (2.0 ** -8 * want.abs() if got.dtype == BF16 else 0.0) + extra
    err = (x - want).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


SHAPES = [  # R, C, group: one row, odd and tiny rows, heads, groups that are no power of two,
    (1, 64, 64), (3, 1, 1), (5, 37, 37), (7, 768, 64), (2, 256, 32), (33, 4096, 128), (4, 520, 520),
    (3, 4096, 4096), (2, 8192, 512), (5, 8192, 8192), (6, 96, 24), (9, 240, 80), (4, 1000, 8),
    (3, 33, 11), (2, 4104, 4104), (400, 1024, 1024), (2, 6000, 6000)]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,C,group", SHAPES)
def test_forward(W, R, C, group, dtype):
    x = make(R, C, dtype, R + C, "wgxsn")
    for act in ("silu", "sigmoid"):
        out, y = W.wkv_norm_gate_forward(**cuda(x), group=group, act=act, eps=EPS)
        o, r = ref.norm_gate(**x, group=group, act=act, eps=EPS)
        close(out, o, "out")
        close(y, r, "y")


PARTS = ["", "w", "g", "x", "n", "wg", "xs", "wgx", "xn", "wgxs", "wxsn", "gn"]


@pytest.mark.parametrize("parts", PARTS)
def test_parts_left_out(W, parts):
    x = make(5, 320, FP32, 3, parts)
    act = "silu" if "g" in parts else "none"
    out, y = W.wkv_norm_gate_forward(**cuda(x), group=64, act=act, eps=EPS)
    o, r = ref.norm_gate(**x, group=64, act=act, eps=EPS)
    close(out, o, "out")
    assert (y is None) == ("n" not in parts)
    if y is not None:
        close(y, r, "y")
    backward(W, x, 64, act, 4, "n" in parts)


def backward(W, x, group, act, seed, with_dy, with_dout=True):
    h = x["h"]
    gen = torch.Generator().manual_seed(seed)
    dout = torch.randn(h.shape, generator=gen).to(h.dtype) if with_dout else None
    dy = torch.randn(h.shape, generator=gen).to(h.dtype) if with_dy else None
    c = cuda(x)
    got = W.wkv_norm_gate_backward(c["h"], c["weight"], None if dout is None else dout.cuda(),
                                   gate=c["gate"], x=c["x"], scale=c["scale"],
                                   next_weight=c["next_weight"], dy=None if dy is None else dy.cuda(),
                                   group=group, act=act, eps=EPS)
    want, sums = ref.norm_gate_gradients(x, group, act, EPS, dout, dy)
    for n in ref.NORM_NAMES:
        if n not in want:
            assert got["d" + n] is None, n
        elif n in sums:
            # a sum over rows: the terms carry the row's error (at most 1e-5 of the row's largest
            # gradient), and the sum rounds at the size of the terms
            err = (got["d" + n].cpu().double() - want[n]).abs()
            bound = 1e-5 * (1 + sums[n] + sums[n].max())
            assert bool((err <= bound).all()), (n, float((err / bound).max()))
        else:
            # dh divides by RMS(h): its terms are larger than itself where h and the gradient
            # line up, by a factor that the row's largest |dh| stands for
            close(got["d" + n], want[n], "d" + n)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,C,group", [s for s in SHAPES if s[0] * s[1] < 50000])
def test_backward(W, R, C, group, dtype):
    for act in ("silu", "sigmoid"):
        backward(W, make(R, C, dtype, R + C, "wgxsn"), group, act, C, True)


def test_backward_one_side(W):
    x = make(6, 192, FP32, 5, "wgxsn")
    backward(W, x, 64, "silu", 6, with_dy=True, with_dout=False)
    backward(W, x, 64, "silu", 7, with_dy=False, with_dout=True)


@pytest.mark.parametrize("R,C", [(2000, 768), (5000, 64), (1500, 770)])
def test_backward_many_rows_is_deterministic(W, R, C):
    # more rows than the grid holds at once: sums over rows, twice the same bits
    x = make(R, C, BF16, 8, "wgxsn")
    c = cuda(x)
    gen = torch.Generator().manual_seed(9)
    dout, dy = (torch.randn(R, C, generator=gen).to(BF16) for _ in range(2))
    group = 64 if C % 64 == 0 else C
    run = lambda: W.wkv_norm_gate_backward(  # noqa: E731
        c["h"], c["weight"], dout.cuda(), gate=c["gate"], x=c["x"], scale=c["scale"],
        next_weight=c["next_weight"], dy=dy.cuda(), group=group, eps=EPS)
    a, b = run(), run()
    assert all(torch.equal(a[n], b[n]) for n in a)
    leaves = {n: t.double().requires_grad_() for n, t in x.items()}
    out, y = ref.norm_gate(**leaves, group=group, act="silu", eps=EPS)
    ((out * dout.double()).sum() + (y * dy.double()).sum()).backward()
    for n in ("weight", "scale", "next_weight"):
        want = leaves[n].grad
        # R terms of order one, rounded at their size
        assert float((a["d" + n].cpu().double() - want).abs().max()) <= 1e-5 * (1 + R ** 0.5 + want.abs().max())
    for n in ("h", "gate", "x"):
        close(a["d" + n], leaves[n].grad, "d" + n)


def test_unaligned_rows(W):
    # storage that starts one element off a vector's boundary
    R, C = 4, 128
    x = make(R, C, BF16, 10, "wgxsn")
    c = cuda(x)
    for n in ("h", "gate", "x"):
        buf = torch.empty(R * C + 1, dtype=BF16, device="cuda")
        buf[1:] = c[n].reshape(-1)
        c[n] = buf[1:].view(R, C)
    out, y = W.wkv_norm_gate_forward(**c, group=64, eps=EPS)
    o, r = ref.norm_gate(**x, group=64, act="silu", eps=EPS)
    close(out, o, "out")
    close(y, r, "y")


@pytest.mark.parametrize("over", ["h", "x"])
def test_out_over_its_input(W, over):
    x = make(50, 768, BF16, 11, "wgxsn")
    c = cuda(x)
    out, y = W.wkv_norm_gate_forward(**c, group=64, eps=EPS, out=c[over])
    o, r = ref.norm_gate(**x, group=64, act="silu", eps=EPS)
    assert out is c[over]
    close(out, o, "out")
    close(y, r, "y")


def test_no_rows(W):
    x = cuda(make(0, 64, BF16, 12, "wgxsn"))
    out, y = W.wkv_norm_gate_forward(**x, group=64)
    assert out.shape == (0, 64) and y.shape == (0, 64)
    g = W.wkv_norm_gate_backward(x["h"], x["weight"], x["h"], gate=x["gate"], x=x["x"],
                                 scale=x["scale"], next_weight=x["next_weight"], dy=x["h"], group=64)
    assert all(bool((g[n] == 0).all()) for n in ("dweight", "dscale", "dnext_weight"))


def test_large_gates(W):
    # sigmoid at +-1e4 is 1 and 0, silu there z and -0; no NaN from the exponential
    x = make(2, 64, FP32, 13, "wg")
    x["gate"][0, :4] = torch.tensor([1e4, -1e4, 88.0, -104.0])
    for act in ("silu", "sigmoid"):
        out, _ = W.wkv_norm_gate_forward(**cuda(x), group=64, act=act, eps=EPS)
        close(out, ref.norm_gate(**x, group=64, act=act, eps=EPS)[0], "out")
        backward(W, x, 64, act, 14, with_dy=False)


def test_leading_dimensions_and_refusals(W):
    x = make(6, 64, BF16, 15, "wgxsn")
    c = cuda(x)
    shaped = {n: t.view(2, 3, 64) if t.dim() == 2 else t for n, t in c.items()}
    a, b = W.wkv_norm_gate_forward(**c, eps=EPS), W.wkv_norm_gate_forward(**shaped, eps=EPS)
    assert torch.equal(a[0].view(2, 3, 64), b[0]) and torch.equal(a[1].view(2, 3, 64), b[1])
    with pytest.raises(ValueError, match="group must divide"):
        W.wkv_norm_gate_forward(c["h"], group=48, act="none")
    with pytest.raises(ValueError, match="act must be"):
        W.wkv_norm_gate_forward(c["h"], act="gelu")
    with pytest.raises(ValueError, match="act must be"):
        W.wkv_norm_gate_forward(c["h"], gate=c["gate"], act="none")
    with pytest.raises(ValueError, match="needs x"):
        W.wkv_norm_gate_forward(c["h"], scale=c["scale"], act="none")
    with pytest.raises(TypeError, match="gate must be"):
        W.wkv_norm_gate_forward(c["h"], gate=c["gate"].float())
    with pytest.raises(ValueError, match="contiguous"):
        W.wkv_norm_gate_forward(c["h"].t().contiguous().t(), act="none")
    with pytest.raises(W.WkvError, match="UNSUPPORTED"):
        W.wkv_norm_gate_forward(torch.zeros(1, 8200, device="cuda"), act="none")
    with pytest.raises(ValueError, match="workspace"):
        W.wkv_norm_gate_backward(c["h"], None, c["h"], act="none",
                                 workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))


def test_graph(W):
    x = cuda(make(20, 768, BF16, 16, "wgxsn"))
    run = lambda c: W.wkv_norm_gate_backward(c["h"], c["weight"], c["x"], gate=c["gate"],  # noqa: E731
                                             x=c["x"], scale=c["scale"],
                                             next_weight=c["next_weight"], dy=c["gate"], group=64)
    want = run(x)
    held = {n: torch.zeros_like(t) for n, t in x.items()}
    run(held)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(held)
    for n in held:
        held[n].copy_(x[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in got)
