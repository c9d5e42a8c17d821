"""The gated delta rule without a GPU: the 64-bit reference of the GPU tests against the C oracle
and differences, and the refusals of the C entry points and of the binding."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402
import oracle  # noqa: E402


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def test_reference_is_the_generalised_delta_rule():
    # wkv7's update with w = e^g, a = -e^g k, b = beta k and beta k as its key
    T, H, N = 37, 3, 64
    q, k, v, g, beta = ref.inputs((T,), H, H, N, torch.float32, 1)
    S0 = 0.3 * torch.randn(H, N, N, generator=torch.Generator().manual_seed(2))
    y, S = ref.rule(q, k, v, g, beta, 0.125, S0)
    d = lambda x: x.double().numpy()[None]  # noqa: E731
    al = np.exp(d(g))[..., None]
    bk = d(beta)[..., None] * d(k)
    yo, So = oracle.wkv7_recurrent(0.125 * d(q), np.broadcast_to(al, d(k).shape).copy(), bk, d(v),
                                   -al * d(k), bk, S0.double().numpy()[None], want_state=True)
    assert np.abs(y.numpy() - yo[0]).max() < 1e-12
    assert np.abs(S.numpy() - So[0]).max() < 1e-12


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "state"])
def test_reference_gradients_are_differences(name):
    T, Hk, H, N = 7, 2, 4, 8
    gen = torch.Generator().manual_seed(3)
    x = dict(zip(("q", "k", "v", "g", "beta"), (t.double() for t in ref.inputs(
        (T,), Hk, H, N, torch.float64, 4))))
    x["state"] = torch.randn(H, N, N, generator=gen, dtype=torch.float64)
    dy = torch.randn(T, H, N, generator=gen, dtype=torch.float64)
    dS = torch.randn(H, N, N, generator=gen, dtype=torch.float64)
    got = ref.rule_gradients(**{n: x[n] for n in ("q", "k", "v", "g", "beta")}, scale=0.7, dy=dy,
                             state=x["state"], dstate=dS)["d" + name]

    def loss(z):
        y, S = ref.rule(z["q"], z["k"], z["v"], z["g"], z["beta"], 0.7, z["state"])
        return float((y * dy).sum() + (S * dS).sum())

    pick = torch.randperm(x[name].numel(), generator=gen)[:12]
    for i in pick.tolist():
        far = []
        for s in (1e-5, -1e-5):
            z = dict(x)
            z[name] = x[name].clone()
            z[name].view(-1)[i] += s
            far.append(loss(z))
        assert abs((far[0] - far[1]) / 2e-5 - float(got.reshape(-1)[i])) < 1e-6


def problem(W, **over):
    from rwkv_linear_attention_wkv_b200.gdr import GdrProblem
    x = dict(B=2, T=5, Hk=2, H=4, N=64, n_seqs=0, seq_offsets=None, dtype=1, scale=1.0,
             workspace=None, workspace_bytes=0)
    x.update(over)
    return ctypes.byref(GdrProblem(*[x[n] for n, _ in GdrProblem._fields_]))


def test_forward_refusals(W):
    f, ok = W.lib.wkv_gdr_forward, 4096
    args = [ok] * 6 + [None, None, None]
    call = lambda over={}, **at: f(problem(W, **over),  # noqa: E731
                                   *[at.get("p%d" % i, x) for i, x in enumerate(args)])
    assert f(None, *args) == 1
    for over in (dict(B=-1), dict(T=-1), dict(H=-1), dict(Hk=-1), dict(N=-64), dict(dtype=2),
                 dict(seq_offsets=ok, n_seqs=-1, B=1), dict(seq_offsets=ok, n_seqs=2, B=2)):
        assert call(over) == 1, over
    for over in (dict(N=32), dict(N=96), dict(H=5), dict(Hk=0), dict(T=1 << 31), dict(B=1 << 31),
                 dict(H=1 << 20, Hk=1), dict(seq_offsets=ok, B=1, n_seqs=1 << 30)):
        assert call(over) == 5, over
    assert call(dict(seq_offsets=ok + 2, B=1, n_seqs=2)) == 2
    assert call(dict(workspace=ok + 8)) == 2
    assert W.lib.wkv_gdr_forward_workspace_bytes(problem(W, T=100, H=1, Hk=1)) == 0
    for i in range(6):
        assert call(**{"p%d" % i: None}) == 1, i
    for i in (0, 1, 2, 5, 6, 7):
        assert call(**{"p%d" % i: ok + 8}) == 2, i
    for i in (3, 4):
        assert call(**{"p%d" % i: ok + 2}) == 2, i
    assert call(dict(B=0)) == 0 and call(dict(H=0)) == 0
    assert call(dict(seq_offsets=ok, B=1, n_seqs=0)) == 0
    assert call(dict(T=0)) == 0  # no tokens and no final state wanted


def test_decode_refusals(W):
    f, ok = W.lib.wkv_gdr_decode_step, 4096
    args = [ok] * 7

    def call(over={}, n_slots=2, slots=None, **at):
        return f(problem(W, **{"T": 1, **over}), *[at.get("p%d" % i, x) for i, x in enumerate(args)],
                 n_slots, slots, None)

    assert call(dict(T=2)) == 1 and call(dict(T=0)) == 1
    assert call(dict(seq_offsets=ok, B=1, n_seqs=1)) == 1
    assert call(n_slots=1) == 1 and call(n_slots=-1) == 1
    for i in range(7):
        assert call(**{"p%d" % i: None}) == 1, i
    for i in (0, 1, 2, 5, 6):
        assert call(**{"p%d" % i: ok + 8}) == 2, i
    assert call(slots=ok + 2) == 2
    assert call(dict(N=48)) == 5 and call(slots=ok, n_slots=1 << 31) == 5
    assert call(dict(B=0), n_slots=0) == 0


def test_binding_refusals(W):
    q = torch.zeros(1, 2, 3, 64)
    g = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError, match="CUDA tensor"):
        W.wkv_gdr_forward(q, q, q, g, g)
    with pytest.raises(TypeError, match="torch.Tensor"):
        W.wkv_gdr_forward(q.numpy(), q, q, g, g)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        W.wkv_gdr_forward(q, q, q.half(), g, g)
    with pytest.raises(ValueError, match="4 dimensions"):
        W.wkv_gdr_forward(q[0], q[0], q[0], g, g)
    with pytest.raises(ValueError, match="3 dimensions"):
        W.wkv_gdr_decode_step(q, q, q, g, g, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        W.wkv_gdr_decode_step(q[0], q[0], q[0], g[0], g[0], torch.zeros(2, 3, 64, 64))


def test_training_pair_refusals(W):
    ok, big = 4096, 1 << 40
    f, b = W.lib.wkv_gdr_forward_checkpointed, W.lib.wkv_gdr_backward
    size = W.lib.wkv_gdr_checkpoint_bytes(problem(W))
    # e of 10 tokens, and the states entering and leaving each sequence
    assert size == 4 * (2 * 5 * 4 * 64 + 4 * 4 * 64 * 64)
    assert W.lib.wkv_gdr_backward_workspace_bytes(problem(W)) == size
    # packed: 80 / 64 chunks, two more a sequence, and one; fp32 heads of 128 have chunks of 32
    assert W.lib.wkv_gdr_checkpoint_bytes(problem(W, B=1, T=80, seq_offsets=ok, n_seqs=3)) == \
        4 * (80 * 4 * 64 + 8 * 4 * 64 * 64)
    assert W.lib.wkv_gdr_checkpoint_bytes(problem(W, T=80, N=128, dtype=0)) == \
        4 * (2 * 80 * 4 * 128 + 2 * 4 * 4 * 128 * 128)
    for over in (dict(B=0), dict(T=0), dict(H=0), dict(N=32), dict(B=-1)):
        assert W.lib.wkv_gdr_checkpoint_bytes(problem(W, **over)) == 0
    fa = [ok] * 6 + [None, None, ok, size, None]
    put = lambda args, i, x: args[:i] + [x] + args[i + 1:]  # noqa: E731
    for i in range(6):
        assert f(problem(W), *put(fa, i, None)) == 1, i
    assert f(problem(W), *put(fa, 8, None)) == 1
    assert f(problem(W), *put(fa, 9, size - 1)) == 1
    for i in (0, 1, 2, 5, 6, 7, 8):
        assert f(problem(W), *put(fa, i, ok + 8)) == 2, i
    assert f(problem(W, N=96), *fa) == 5 and f(problem(W, dtype=3), *fa) == 1
    assert f(problem(W, B=0), *fa) == 0
    ba = [ok] * 7 + [size, None] + [ok] * 5 + [None, ok, size, None]
    assert b(None, *ba) == 1
    for i in (0, 1, 2, 3, 4, 5, 6, 9, 10, 11, 12, 13, 15):
        assert b(problem(W), *put(ba, i, None)) == 1, i
    for i in (7, 16):
        assert b(problem(W), *put(ba, i, size - 1)) == 1, i
    for i in (0, 1, 2, 5, 6, 8, 9, 10, 11, 14, 15):
        assert b(problem(W), *put(ba, i, ok + 8)) == 2, i
    for i in (3, 4, 12, 13):
        assert b(problem(W), *put(ba, i, ok + 2)) == 2, i
    assert b(problem(W, N=96), *ba) == 5 and b(problem(W, H=5), *ba) == 5
    assert b(problem(W, H=0), *ba) == 0
    # more chunks x query/key heads than a grid holds
    assert b(problem(W, B=1 << 20, T=1 << 15, H=8, Hk=8), *put(put(ba, 7, big << 20), 16, big << 20)) == 5


def test_training_pair_binding_refusals(W):
    x = ref.inputs((1, 4), 2, 4, 64, torch.float32, 5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        W.wkv_gdr_forward_checkpointed(*x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        W.wkv_gdr_backward(*x, x[2], torch.zeros(10))
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        W.wkv_gdr_backward(None, *x[1:], x[2], None)
