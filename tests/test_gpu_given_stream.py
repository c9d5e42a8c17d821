"""Calls on a given stream while the current one is busy: what a call makes for itself is no memory
that something enqueued before, on the current stream, has still to read."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def tensors(x):
    if torch.is_tensor(x):
        return [x]
    if isinstance(x, dict):
        x = x.values()
    return [] if x is None else [t for y in x for t in tensors(y)]


def check(call, scratch=()):
    """call(stream) with blocks of all its results' sizes (and `scratch` bytes) free to take, but
    waiting to be read."""
    want = [t.clone() for t in tensors(call(None))]
    sizes = [t.numel() * t.element_size() for t in want] + list(scratch)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.full((n // 4,), float(i), device="cuda") for i, n in enumerate(sizes)]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for b, c in zip(blocks, copies):
        c.copy_(b)
    del blocks, b
    got = tensors(call(side))
    side.synchronize()
    torch.cuda.synchronize()
    for i, c in enumerate(copies):
        assert bool((c == float(i)).all()), i
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_rule(W):
    x = [t.cuda() for t in ref.inputs((1, 1100), 1, 1, 64, BF16, 1)]
    dy = torch.randn(1, 1100, 1, 64, device="cuda").to(BF16)
    _, _, ws = W.wkv_gdr_forward_checkpointed(*x)
    check(lambda s: W.wkv_gdr_forward(*x, stream=s), [8 * 10 * 64 * 64])
    check(lambda s: W.wkv_gdr_forward_checkpointed(*x, stream=s)[:2], [ws.numel()])
    check(lambda s: W.wkv_gdr_backward(*x, dy, ws, stream=s), [2 * ws.numel()])
    one = [t[:, 0].contiguous() for t in x]
    pools = [torch.zeros(1, 1, 64, 64, device="cuda") for _ in range(2)]
    check(lambda s: W.wkv_gdr_decode_step(*one, pools.pop(), stream=s))


def test_the_norms(W):
    h, z, x = (torch.randn(500, 256, device="cuda").to(BF16) for _ in range(3))
    w = torch.rand(256, device="cuda")
    check(lambda s: W.wkv_norm_gate_forward(h, w, gate=z, x=x, next_weight=w, stream=s))
    check(lambda s: W.wkv_norm_gate_backward(h, w, x, gate=z, x=x, next_weight=w, dy=z, stream=s),
          [W.wkv_norm_gate_workspace_bytes(500, 256)])


def test_the_channel_operators(W):
    B, T, C = 2, 64, 64
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    w, u = 0.1 + torch.rand(C, device="cuda"), r(C)
    k, v, g, dy = (r(B, T, C) for _ in range(4))
    ws = W.wkv_backward_workspace_bytes(B, T, C)
    check(lambda s: W.wkv_forward(w, u, k, v, g, stream=s))
    half = [t.to(BF16) for t in (k, v, g)]
    check(lambda s: W.wkv_forward_bf16(w, u, *half, stream=s))
    check(lambda s: W.wkv_forward_state(w, u, k, v, g, stream=s))
    check(lambda s: W.wkv_backward(w, u, k, v, g, dy, stream=s), [ws])
    _, kept = W.wkv_forward_checkpointed(w, u, k, v, g)
    check(lambda s: W.wkv_forward_checkpointed(w, u, k, v, g, stream=s)[0], [ws])
    check(lambda s: W.wkv_backward_checkpointed(w, u, k, v, g, dy, kept, stream=s))


def test_the_matrix_states(W):
    r, k, v = (0.3 * torch.randn(1, 70, 2, 64, device="cuda") for _ in range(3))
    w = 0.5 + 0.5 * torch.rand(1, 70, 2, 64, device="cuda")
    check(lambda s: W.wkv_mstate_forward(r, w, k, v, stream=s))
    a, b = -0.1 * k, 0.1 * k
    check(lambda s: W.wkv7_forward(r, w, k, v, a, b, stream=s))
