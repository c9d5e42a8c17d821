"""Refusals of the norms around a block, without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def problem(**over):
    from rwkv_linear_attention_wkv_b200.norm_gate import NormGateProblem
    x = dict(R=4, C=128, group=64, dtype=1, act=2, eps=1e-6)
    x.update(over)
    return ctypes.byref(NormGateProblem(*[x[n] for n, _ in NormGateProblem._fields_]))


OK = 4096


def test_forward_refusals(W):
    f = W.lib.wkv_norm_gate_forward

    def call(p=None, **at):
        x = dict(h=OK, w=OK, z=OK, x=OK, s=OK, n=OK, out=OK, y=OK)
        x.update(at)
        return f(problem(**(p or {})), *x.values(), None)

    assert f(None, *[OK] * 8, None) == 1
    for p in (dict(R=-1), dict(C=-1), dict(dtype=5), dict(eps=0.0), dict(eps=float("nan")),
              dict(act=0), dict(act=3), dict(group=0), dict(group=-64), dict(group=48)):
        assert call(p) == 1, p
    assert call(dict(C=8256)) == 5 and call(dict(R=1 << 41)) == 5
    assert call(h=None) == 1 and call(out=None) == 1
    assert call(y=None) == 1 and call(n=None) == 1      # y and its weight come together
    assert call(x=None) == 1                            # a scale without a residual
    for n in ("h", "z", "x", "out", "y"):
        assert call(**{n: OK + 1}) == 2, n
    for n in ("w", "s", "n"):
        assert call(**{n: OK + 2}) == 2, n
    assert call(dict(R=0)) == 0 and call(dict(C=0)) == 0


def test_backward_refusals(W):
    f = W.lib.wkv_norm_gate_backward
    need = W.wkv_norm_gate_workspace_bytes(4, 128)
    names = "h w z x s n dout dy dh dw dz dx ds dn ws".split()

    def call(p=None, nbytes=need, **at):
        x = {n: OK for n in names}
        x.update(at)
        return f(problem(**(p or {})), *x.values(), nbytes, None)

    assert call(dict(R=-1)) == 1 and call(dict(group=48)) == 1
    assert call(h=None) == 1 and call(dh=None) == 1
    assert call(dout=None, dy=None, dn=None) == 1
    assert call(n=None) == 1                            # dy without its weight
    assert call(z=None) == 1 and call(x=None) == 1      # gradients of what is not there
    assert call(s=None) == 1 and call(dy=None) == 1
    assert call(ws=None) == 1 and call(nbytes=need - 1) == 1
    assert call(ws=OK + 4) == 2 and call(dw=OK + 2) == 2 and call(dh=OK + 1) == 2
    assert call(dict(C=0)) == 0
    assert W.wkv_norm_gate_workspace_bytes(0, 128) == 0


def test_binding_refuses_host_tensors(W):
    h = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        W.wkv_norm_gate_forward(h, act="none")
    with pytest.raises(TypeError, match="torch.Tensor"):
        W.wkv_norm_gate_forward(h.numpy(), act="none")
    with pytest.raises(ValueError, match="dout or dy"):
        W.wkv_norm_gate_backward(h, None, None, act="none")
