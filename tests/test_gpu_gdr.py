"""GPU parity of the gated delta rule (forward and decode) against its definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


def states(n, H, N, seed):
    return 0.3 * torch.randn(n, H, N, N, generator=torch.Generator().manual_seed(seed))


def check(W, lead, Hk, H, N, dtype, state, seed, strong=False):
    x = ref.inputs(lead, Hk, H, N, dtype, seed, strong)
    S0 = states(lead[0], H, N, seed + 1) if state else None
    y, S = W.wkv_gdr_forward(*cuda(*x), state=None if S0 is None else S0.cuda(), scale=N ** -0.5)
    yr, Sr = ref.rows(*x, N ** -0.5, S0)
    assert y.dtype == dtype and S.dtype == FP32
    ref.assert_close(y, yr, "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)
    assert W.wkv_stream_status() == 0


# lengths around the kernels' token groups (16, 32, 64), one token, odd ones; shared key heads
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (2, 15, 2, 2), (1, 16, 1, 3), (3, 17, 2, 4),
                                      (1, 31, 1, 2), (1, 33, 2, 2), (2, 64, 1, 1), (1, 65, 3, 3),
                                      (1, 131, 1, 4), (1, 300, 2, 2)])
def test_forward(W, B, T, Hk, H, N, dtype):
    check(W, (B, T), Hk, H, N, dtype, state=T % 2 == 1, seed=T + N)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_forward_strong_decays_and_writes(W, N, dtype):
    check(W, (2, 150), 2, 2, N, dtype, state=True, seed=7, strong=True)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_forward_many_heads(W, dtype):
    # more heads than the GPU has SMs, so that heads queue behind one another
    check(W, (5, 40), 16, 64, 64, dtype, state=True, seed=8)


@pytest.mark.parametrize("N", [64, 128])
def test_forward_forgets_at_minus_infinity(W, N):
    # g = -inf: the state before the token is gone
    x = list(ref.inputs((1, 50), 1, 2, N, FP32, 9))
    x[3][0, 20] = float("-inf")
    x[3][0, 33, 1] = float("-inf")
    S0 = states(1, 2, N, 10)
    y, S = W.wkv_gdr_forward(*cuda(*x), state=S0.cuda())
    yr, Sr = ref.rows(*x, 1.0, S0)
    ref.assert_close(y, yr, "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_forward_packed(W, N, dtype):
    # an empty sequence, one token, ends inside every token group; tokens behind the last
    # sequence, and before the first, stay as they were
    off = [2, 2, 3, 20, 36, 101, 165, 166]
    T, H, Hk = 180, 4, 2
    x = ref.inputs((1, T), Hk, H, N, dtype, 11)
    S0 = states(len(off) - 1, H, N, 12)
    y = torch.full((1, T, H, N), 7.0, dtype=dtype, device="cuda")
    _, S = W.wkv_gdr_forward(*cuda(*x), state=S0.cuda(), scale=0.5, y=y,
                             seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    yr, Sr = ref.rows(*x, 0.5, S0, list(zip(off[:-1], off[1:])))
    assert bool((y[:, :2] == 7).all()) and bool((y[:, 166:] == 7).all())
    ref.assert_close(y[:, 2:166], yr[:, 2:166], "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)
    assert torch.equal(S[0].cpu(), S0[0])  # the empty sequence's state


def test_forward_packed_offsets_out_of_range(W):
    # offsets are clamped to the row, a sequence that ends before it starts is empty
    T, N = 40, 64
    x = ref.inputs((1, T), 2, 2, N, BF16, 13)
    off = torch.tensor([-5, 12, 9, 30, 1000], dtype=torch.int32, device="cuda")
    y, S = W.wkv_gdr_forward(*cuda(*x), seq_offsets=off)
    yr, Sr = ref.rows(*x, 1.0, None, [(0, 12), (12, 9), (9, 30), (30, 40)])
    ref.assert_close(y[:, 12:], yr[:, 12:], "y", head_dim=2)
    ref.assert_close(S[2:], Sr[2:], "state", head_dim=1)
    assert bool((S[1] == 0).all())


def test_forward_no_tokens(W):
    x = ref.inputs((2, 0), 2, 2, 64, BF16, 14)
    S0 = states(2, 2, 64, 15).cuda()
    y, S = W.wkv_gdr_forward(*cuda(*x), state=S0)
    assert y.shape == (2, 0, 2, 64) and torch.equal(S, S0)
    y, S = W.wkv_gdr_forward(*cuda(*x))
    assert bool((S == 0).all())


@pytest.mark.parametrize("N", [64, 128])
def test_forward_split_with_state_in_place(W, N):
    # a sequence in pieces, the state written over the one it came from
    x = ref.inputs((2, 100), 2, 4, N, FP32, 16)
    S = states(2, 4, N, 17)
    yr, Sr = ref.rows(*x, 1.0, S)
    S = S.cuda()
    ys = [W.wkv_gdr_forward(*cuda(*[t[:, a:b].contiguous() for t in x]), state=S, state_out=S)[0]
          for a, b in ((0, 1), (1, 23), (23, 87), (87, 100))]
    ref.assert_close(torch.cat(ys, 1), yr, "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)


# long sequences of few heads are walked in segments of at least 256 tokens, side by side
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,B,T,Hk,H", [(64, 1, 1025, 1, 1), (64, 2, 1217, 1, 3), (128, 1, 1100, 1, 2),
                                        (128, 3, 1024, 1, 1)])
def test_forward_in_segments(W, N, B, T, Hk, H, dtype):
    check(W, (B, T), Hk, H, N, dtype, state=T % 2 == 1, seed=T + N)


@pytest.mark.parametrize("N", [64, 128])
def test_forward_in_segments_strong_decays_and_state_in_place(W, N):
    x = ref.inputs((1, 1100), 1, 1, N, FP32, 23, strong=True)
    S = states(1, 1, N, 24)
    yr, Sr = ref.rows(*x, 1.0, S)
    S = S.cuda()
    y, S1 = W.wkv_gdr_forward(*cuda(*x), state=S, state_out=S)
    assert S1 is S
    ref.assert_close(y, yr, "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)


@pytest.mark.parametrize("N", [64, 128])
def test_forward_packed_in_segments(W, N):
    # one sequence long enough for segments, two that are walked whole, an empty one
    off = [3, 3, 1000, 1512, 1600]
    T, H = 2100, 2
    x = ref.inputs((1, T), 1, H, N, BF16, 25)
    S0 = states(4, H, N, 26)
    y = torch.full((1, T, H, N), 7.0, dtype=BF16, device="cuda")
    _, S = W.wkv_gdr_forward(*cuda(*x), state=S0.cuda(), scale=0.5, y=y,
                             seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    yr, Sr = ref.rows(*x, 0.5, S0, list(zip(off[:-1], off[1:])))
    assert bool((y[:, :3] == 7).all()) and bool((y[:, 1600:] == 7).all())
    ref.assert_close(y[:, 3:1600], yr[:, 3:1600], "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)
    assert torch.equal(S[0].cpu(), S0[0])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_decode_with_slots(W, N, dtype):
    n, H, Hk, pool = 6, 4, 2, 9
    x = ref.inputs((n,), Hk, H, N, dtype, 18)
    S0 = states(pool, H, N, 19)
    slots = [4, 0, -1, 8, 9, 2]  # -1 and 9 are outside the pool: padding
    S, y = S0.cuda(), torch.full((n, H, N), 7.0, dtype=dtype, device="cuda")
    W.wkv_gdr_decode_step(*cuda(*x), S, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          scale=0.3, y=y)
    for i, s in enumerate(slots):
        if not 0 <= s < pool:
            assert bool((y[i] == 7).all())
            continue
        yr, Sr = ref.rule(*[t[i:i + 1] for t in x], 0.3, S0[s])
        ref.assert_close(y[i:i + 1], yr, "y", head_dim=1)
        ref.assert_close(S[s], Sr, "state", head_dim=0)
    for s in set(range(pool)) - set(slots):
        assert torch.equal(S[s].cpu(), S0[s])


def test_decode_continues_the_forward(W):
    # prefill, then token by token: the states and read-outs of one long sequence
    N, H, B, T = 64, 3, 2, 60
    x = ref.inputs((B, T), H, H, N, BF16, 20)
    yr, Sr = ref.rows(*x, 0.125, None)
    g = cuda(*x)
    y, S = W.wkv_gdr_forward(*[t[:, :40].contiguous() for t in g], scale=0.125)
    ys = [y]
    for t in range(40, T):
        ys.append(W.wkv_gdr_decode_step(*[z[:, t].contiguous() for z in g], S, scale=0.125)[:, None])
    ref.assert_close(torch.cat(ys, 1), yr, "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)


def test_streams_and_graph(W):
    # on another stream than the current one; captured once and replayed on new inputs
    x = cuda(*ref.inputs((2, 70), 2, 2, 64, BF16, 21))
    y0, S0 = W.wkv_gdr_forward(*x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, S1 = torch.empty_like(y0), torch.empty_like(S0)
    W.wkv_gdr_forward(*x, y=y1, state_out=S1, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(S0, S1)
    held = [torch.zeros_like(t) for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, S2 = W.wkv_gdr_forward(*held)
        y3 = W.wkv_gdr_decode_step(*[t[:, 0].contiguous() for t in held], S2)
    for h, t in zip(held, x):
        h.copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    Sd = S0.clone()
    yd = W.wkv_gdr_decode_step(*[t[:, 0].contiguous() for t in x], Sd)
    assert torch.equal(y2, y0) and torch.equal(S2, Sd) and torch.equal(y3, yd)


def test_binding_refusals_on_the_gpu(W):
    q, k, v, g, beta = cuda(*ref.inputs((1, 4), 2, 4, 64, BF16, 22))
    with pytest.raises(TypeError, match="q must be"):
        W.wkv_gdr_forward(q.float(), k, v, g, beta)
    with pytest.raises(ValueError, match="contiguous"):
        W.wkv_gdr_forward(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g, beta)
    with pytest.raises(ValueError, match="g must have shape"):
        W.wkv_gdr_forward(q, k, v, g[:, :, :2].contiguous(), beta)
    with pytest.raises(ValueError, match="packed into one row"):
        W.wkv_gdr_forward(*[torch.cat([t, t]) for t in (q, k, v, g, beta)],
                          seq_offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="seq_offsets must be"):
        W.wkv_gdr_forward(q, k, v, g, beta, seq_offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(W.WkvError, match="UNSUPPORTED"):
        W.wkv_gdr_forward(q[..., :32].contiguous(), k[..., :32].contiguous(),
                          v[..., :32].contiguous(), g, beta)
