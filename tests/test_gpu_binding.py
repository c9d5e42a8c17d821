"""The short way into the library (_binding.so) and the long way through ctypes give the same
results, bit for bit; what the short way does not take reaches the long way's explanations."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def same(a, b):
    if isinstance(a, dict):
        assert list(a) == list(b)
        a, b = list(a.values()), list(b.values())
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and torch.equal(x, y)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_the_rule_both_ways(W, dtype, packed):
    T, H, Hk, N = 1200, 2, 1, 64
    x = [t.cuda() for t in ref.inputs((1, T), Hk, H, N, dtype, 1)]
    o = torch.tensor([0, 500, 1200], dtype=torch.int32, device="cuda") if packed else None
    n = 2 if packed else 1
    S = 0.3 * torch.randn(n, H, N, N, device="cuda")
    here = torch.cuda.current_stream()
    kw = dict(state=S, scale=0.3, seq_offsets=o)
    same(W.wkv_gdr_forward(*x, **kw), W.wkv_gdr_forward(*x, **kw, stream=here))
    a = W.wkv_gdr_forward(*x, **kw, want_state=False)
    assert a[1] is None
    same(a, W.wkv_gdr_forward(*x, **kw, want_state=False, stream=here))
    y, out = torch.empty_like(x[2]), torch.empty_like(S)
    b = W.wkv_gdr_forward(*x, **kw, y=y, state_out=out)
    assert b[0].data_ptr() == y.data_ptr() and b[1].data_ptr() == out.data_ptr()
    y1, s1, ws = W.wkv_gdr_forward_checkpointed(*x, **kw)
    y2, s2, ws2 = W.wkv_gdr_forward_checkpointed(*x, **kw, stream=here)
    same((y1, s1), (y2, s2))
    assert ws.numel() == ws2.numel()
    dy = torch.randn_like(y1)
    for more in (dict(), dict(grad_state=S), dict(want_dstate=False)):
        same(W.wkv_gdr_backward(*x, dy, ws, scale=0.3, seq_offsets=o, **more),
             W.wkv_gdr_backward(*x, dy, ws2, scale=0.3, seq_offsets=o, **more, stream=here))


def test_decode_both_ways(W):
    n, H, Hk, N = 5, 4, 2, 128
    x = [t.cuda() for t in ref.inputs((n,), Hk, H, N, BF16, 2)]
    S = 0.3 * torch.randn(7, H, N, N, device="cuda")
    slots = torch.tensor([6, 0, -1, 3, 2], dtype=torch.int32, device="cuda")
    for s in (None, slots):
        S1, S2 = S.clone(), S.clone()
        y = [torch.zeros_like(x[2]) for _ in range(2)]
        a = W.wkv_gdr_decode_step(*x, S1, slots=s, scale=0.5, y=y[0])
        b = W.wkv_gdr_decode_step(*x, S2, slots=s, scale=0.5, y=y[1],
                                  stream=torch.cuda.current_stream())
        assert a.data_ptr() == y[0].data_ptr()
        assert torch.equal(a, b) and torch.equal(S1, S2)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_the_norms_both_ways(W, dtype):
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    h, z, x = (r(3, 7, 256).to(dtype) for _ in range(3))
    w, s, nw = r(256), r(256), r(256)
    here = torch.cuda.current_stream()
    for kw in (dict(weight=w, gate=z, x=x, scale=s, next_weight=nw, group=64, act="silu"),
               dict(gate=z, act="sigmoid", eps=1e-3), dict(act="none", x=x), dict(act="none", next_weight=nw)):
        same(W.wkv_norm_gate_forward(h, **kw), W.wkv_norm_gate_forward(h, **kw, stream=here))
        kw = dict(kw)
        weight = kw.pop("weight", None)
        dy = r(3, 7, 256).to(dtype) if "next_weight" in kw else None
        same(W.wkv_norm_gate_backward(h, weight, x, dy=dy, **kw),
             W.wkv_norm_gate_backward(h, weight, x, dy=dy, **kw, stream=here))


def test_refusals_reach_their_explanation(W):
    q, k, v, g, beta = x = [t.cuda() for t in ref.inputs((2, 8), 1, 2, 64, BF16, 3)]
    for args, kw, error, match in (
            ((q, k, v, g.double(), beta), {}, TypeError, "g must be torch.float32"),
            ((q, k[:, :4], v, g, beta), {}, ValueError, "k must have shape"),
            ((q, k, v, g.cpu(), beta), {}, ValueError, "g must be a CUDA tensor"),
            (x, dict(state=torch.zeros(2, 2, 64, 64)), ValueError, "state must be a CUDA tensor"),
            (x, dict(scale="a"), TypeError, None),
            (x, dict(y=torch.empty_like(v).float()), TypeError, "y must be")):
        with pytest.raises(error, match=match):
            W.wkv_gdr_forward(*args, **kw)
    with pytest.raises(ValueError, match="at least 2 slots"):
        W.wkv_gdr_decode_step(*[t[:, 0].contiguous() for t in x], torch.zeros(1, 2, 64, 64, device="cuda"))
    with pytest.raises(ValueError, match="group must divide"):
        W.wkv_norm_gate_forward(v, group=48, act="none")
    with pytest.raises(ValueError, match="act must be one of"):
        W.wkv_norm_gate_forward(v, act="gelu")
