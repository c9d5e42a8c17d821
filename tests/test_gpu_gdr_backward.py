"""GPU parity of the gated delta rule's gradients against the adjoint of its definition in 64 bits.

Comparison: the rules of gdr_reference. A gradient is a sum over later tokens of products like the
forward's, each rounded in fp32 (for bf16 problems dq, dk, dg take factors of 2^-17 on top, which
average over the 64 or 128 channels of a sum), so the same bound, 1e-5 (1 + m) with m the largest
entry of the head, holds; dq, dk and dv of bf16 problems are rounded to bf16 once more."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
TOKENS = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


def normal(shape, seed, dtype=FP32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def gradients(x, scale, dy, S0, dS, spans):
    """Reference over spans (row, start, end), one sequence each."""
    got = {n: torch.zeros(t.shape, dtype=torch.float64)
           for n, t in zip(TOKENS, (x[0], x[1], x[2], x[3], x[4]))}
    got["dstate"] = []
    for i, (b, t0, t1) in enumerate(spans):
        r = slice(t0, t1)
        g = ref.rule_gradients(*[t[b, r] for t in x], scale, dy[b, r],
                               None if S0 is None else S0[i], None if dS is None else dS[i])
        for n in TOKENS:
            got[n][b, r] = g[n]
        got["dstate"].append(g["dstate"])
    got["dstate"] = torch.stack(got["dstate"])
    return got


def run(W, x, scale, dy, S0, dS, off=None, **kw):
    c = cuda(*x)
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    y, S, ws = W.wkv_gdr_forward_checkpointed(*c, state=None if S0 is None else S0.cuda(),
                                              scale=scale, seq_offsets=o)
    y0, S_0 = W.wkv_gdr_forward(*c, state=None if S0 is None else S0.cuda(), scale=scale,
                                seq_offsets=o, y=torch.zeros_like(y))
    rows = slice(None) if off is None else slice(off[0], off[-1])
    assert torch.equal(y[:, rows], y0[:, rows]) and torch.equal(S, S_0)
    return W.wkv_gdr_backward(*c, dy.cuda(), ws, grad_state=None if dS is None else dS.cuda(),
                              scale=scale, seq_offsets=o, **kw)


def compare(got, want, dtype, only=slice(None)):
    for n in TOKENS:
        assert got[n].dtype == (FP32 if n in ("dg", "dbeta") else dtype)
        ref.assert_close(got[n][:, only], want[n][:, only], n, head_dim=2)
    if got["dstate"] is not None:
        ref.assert_close(got["dstate"], want["dstate"], "dstate", head_dim=1)


def check(W, B, T, Hk, H, N, dtype, state, seed, strong=False):
    x = ref.inputs((B, T), Hk, H, N, dtype, seed, strong)
    dy = normal((B, T, H, N), seed + 1, dtype)
    S0 = 0.3 * normal((B, H, N, N), seed + 2) if state else None
    dS = 0.3 * normal((B, H, N, N), seed + 3) if state else None
    got = run(W, x, N ** -0.5, dy, S0, dS, want_dstate=state)
    assert state or got["dstate"] is None
    compare(got, gradients(x, N ** -0.5, dy, S0, dS, [(b, 0, T) for b in range(B)]), dtype)
    assert W.wkv_stream_status() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (2, 15, 2, 2), (1, 16, 1, 3), (3, 17, 2, 4),
                                      (1, 31, 1, 2), (1, 33, 2, 2), (2, 64, 1, 1), (1, 65, 3, 3),
                                      (1, 131, 1, 4), (1, 200, 2, 2)])
def test_backward(W, B, T, Hk, H, N, dtype):
    check(W, B, T, Hk, H, N, dtype, state=T % 2 == 1, seed=T + N)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_backward_strong_decays_and_writes(W, N, dtype):
    check(W, 2, 150, 2, 2, N, dtype, state=True, seed=7, strong=True)


@pytest.mark.parametrize("N", [64, 128])
def test_backward_no_writes_and_full_decay(W, N):
    # beta = 0 (the token writes nothing; dbeta is still defined) and g = -inf (the state is gone)
    x = list(ref.inputs((1, 70), 1, 2, N, FP32, 9))
    x[4][0, 5:9] = 0.0
    x[4][0, 40:, 1] = 0.0
    x[3][0, 20] = float("-inf")
    x[3][0, 33, 1] = float("-inf")
    dy, S0 = normal((1, 70, 2, N), 10), 0.3 * normal((1, 2, N, N), 11)
    dS = 0.3 * normal((1, 2, N, N), 12)
    compare(run(W, x, 1.0, dy, S0, dS), gradients(x, 1.0, dy, S0, dS, [(0, 0, 70)]), FP32)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_backward_packed(W, N, dtype):
    # an empty sequence, one token, ends inside and at the ends of groups and chunks; the rows that
    # no sequence covers stay as they were
    off = [2, 2, 3, 20, 36, 101, 165, 166]
    T, H, Hk, n = 180, 4, 2, 7
    x = ref.inputs((1, T), Hk, H, N, dtype, 21)
    dy = normal((1, T, H, N), 22, dtype)
    S0, dS = 0.3 * normal((n, H, N, N), 23), 0.3 * normal((n, H, N, N), 24)
    out = {m: torch.full(s, 7.0, dtype=t, device="cuda") for m, t, s in
           (("dq", dtype, (1, T, Hk, N)), ("dk", dtype, (1, T, Hk, N)), ("dv", dtype, (1, T, H, N)),
            ("dg", FP32, (1, T, H)), ("dbeta", FP32, (1, T, H)), ("dstate", FP32, (n, H, N, N)))}
    got = run(W, x, 0.5, dy, S0, dS, off, grads=out)
    assert got["dq"] is out["dq"]
    want = gradients(x, 0.5, dy, S0, dS, [(0, a, b) for a, b in zip(off[:-1], off[1:])])
    compare(got, want, dtype, slice(2, 166))
    assert torch.equal(got["dstate"][0].cpu(), dS[0])
    for m in TOKENS:
        assert bool((out[m][:, :2] == 7).all()) and bool((out[m][:, 166:] == 7).all())


@pytest.mark.parametrize("N", [64, 128])
def test_backward_first_decay_of_nothing(W, N):
    # without a state the first token's decay multiplies zero: its gradient is zero, and with one
    # it is not
    off = [0, 1, 30, 130]
    x = ref.inputs((1, 130), 1, 2, N, BF16, 29)
    dy = normal((1, 130, 2, N), 30, BF16)
    for S0 in (None, 0.3 * normal((3, 2, N, N), 31)):
        got = run(W, x, 0.5, dy, S0, None, off)
        assert bool((got["dg"][0, off[:-1]] == 0).all()) == (S0 is None)
        want = gradients(x, 0.5, dy, S0, None, [(0, a, b) for a, b in zip(off[:-1], off[1:])])
        compare(got, want, BF16)


def test_backward_many_packed_sequences(W):
    # more sequences than are ordered by length, most of a token or two, empty ones among them
    gen = torch.Generator().manual_seed(26)
    lens = torch.randint(0, 4, (1300,), generator=gen)
    lens[[5, 700, 1299]] = torch.tensor([130, 64, 65])
    off = [0] + torch.cumsum(lens, 0).tolist()
    T, H, N = off[-1], 1, 64
    x = ref.inputs((1, T), 1, H, N, FP32, 27)
    dy = normal((1, T, H, N), 28)
    spans = [(0, a, b) for a, b in zip(off[:-1], off[1:])]
    got = run(W, x, 0.5, dy, None, None, off, want_dstate=False)
    compare(got, gradients(x, 0.5, dy, None, None, spans), FP32)


# long sequences of few heads: both walks in segments of at least 256 tokens, side by side
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,B,T,Hk,H", [(64, 1, 1025, 1, 2), (128, 1, 1100, 1, 1)])
def test_backward_in_segments(W, N, B, T, Hk, H, dtype):
    check(W, B, T, Hk, H, N, dtype, state=T % 2 == 1, seed=T + N)


@pytest.mark.parametrize("N", [64, 128])
def test_backward_packed_in_segments(W, N):
    off = [3, 3, 1000, 1512, 1600]
    T, H, n = 2100, 1, 4
    x = ref.inputs((1, T), 1, H, N, FP32, 27)
    dy = normal((1, T, H, N), 28)
    S0, dS = 0.3 * normal((n, H, N, N), 29), 0.3 * normal((n, H, N, N), 30)
    got = run(W, x, 0.5, dy, S0, dS, off)
    want = gradients(x, 0.5, dy, S0, dS, [(0, a, b) for a, b in zip(off[:-1], off[1:])])
    compare(got, want, FP32, slice(3, 1600))
    assert torch.equal(got["dstate"][0].cpu(), dS[0])


def test_backward_many_heads_and_repeats(W):
    # more chunks than the GPU holds at once; a second call gives the same bits (fixed orders),
    # and the workspace is only read
    x = ref.inputs((3, 100), 8, 32, 64, BF16, 31)
    dy = normal((3, 100, 32, 64), 32, BF16)
    c, d = cuda(*x), dy.cuda()
    y, S, ws = W.wkv_gdr_forward_checkpointed(*c)
    kept = ws.clone()
    one = W.wkv_gdr_backward(*c, d, ws)
    two = W.wkv_gdr_backward(*c, d, ws)
    assert torch.equal(ws, kept)
    for n in one:
        assert torch.equal(one[n], two[n]), n
    want = gradients(x, 1.0, dy, None, None, [(b, 0, 100) for b in range(3)])
    compare(one, want, BF16)


def test_backward_no_tokens(W):
    x = cuda(*ref.inputs((2, 0), 2, 2, 64, BF16, 41))
    dS = normal((2, 2, 64, 64), 42).cuda()
    y, S, ws = W.wkv_gdr_forward_checkpointed(*x)
    got = W.wkv_gdr_backward(*x, torch.zeros_like(y), ws, grad_state=dS)
    assert torch.equal(got["dstate"], dS) and got["dq"].numel() == 0
    got = W.wkv_gdr_backward(*x, torch.zeros_like(y), ws)
    assert bool((got["dstate"] == 0).all())


def test_backward_on_a_stream_and_in_a_graph(W):
    x = cuda(*ref.inputs((2, 90), 2, 2, 64, BF16, 51))
    dy = normal((2, 90, 2, 64), 52, BF16).cuda()
    y, S, ws = W.wkv_gdr_forward_checkpointed(*x)
    want = W.wkv_gdr_backward(*x, dy, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = W.wkv_gdr_backward(*x, dy, ws)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    held, hdy = [torch.zeros_like(t) for t in x], torch.zeros_like(dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, S2, ws2 = W.wkv_gdr_forward_checkpointed(*held)
        g2 = W.wkv_gdr_backward(*held, hdy, ws2)
    for h, t in zip(held + [hdy], x + [dy]):
        h.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(g2[n], want[n]) for n in want)


def test_backward_refusals(W):
    q, k, v, g, beta = x = cuda(*ref.inputs((1, 20), 2, 4, 64, BF16, 61))
    y, S, ws = W.wkv_gdr_forward_checkpointed(*x)
    with pytest.raises(TypeError, match="dy must be"):
        W.wkv_gdr_backward(*x, y.float(), ws)
    with pytest.raises(ValueError, match="dy must have shape"):
        W.wkv_gdr_backward(*x, y[:, :10].contiguous(), ws)
    with pytest.raises(ValueError, match="workspace must be"):
        W.wkv_gdr_backward(*x, y, ws[:-1])
    with pytest.raises(TypeError, match="workspace must be"):
        W.wkv_gdr_backward(*x, y, None)
    with pytest.raises(ValueError, match="grad_state must have shape"):
        W.wkv_gdr_backward(*x, y, ws, grad_state=S[:, :2].contiguous())
    with pytest.raises(ValueError, match="scratch must be"):
        W.wkv_gdr_backward(*x, y, ws, scratch=ws[:100])
    with pytest.raises(TypeError, match="dq must be"):
        W.wkv_gdr_backward(*x, y, ws, grads={})


def test_backward_on_a_given_stream_keeps_its_memory(W):
    # the call waits behind other work on `side`; what the binding allocated for it must not be
    # handed out on the current stream meanwhile
    x = cuda(*ref.inputs((1, 1100), 1, 1, 64, BF16, 71))
    dy = normal((1, 1100, 1, 64), 72, BF16).cuda()
    y, S, ws = W.wkv_gdr_forward_checkpointed(*x)
    want = W.wkv_gdr_backward(*x, dy, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
    y2, S2, ws2 = W.wkv_gdr_forward_checkpointed(*x, stream=side)
    got = W.wkv_gdr_backward(*x, dy, ws2, stream=side)
    sizes = (ws2.numel(), 2 * ws2.numel(), 40 * 64 * 64)
    del ws2
    for n in sizes:
        [torch.full((n // 4,), 1e30, device="cuda") for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(S2, S)
    assert all(torch.equal(got[n], want[n]) for n in want)
