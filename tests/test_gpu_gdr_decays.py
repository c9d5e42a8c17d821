"""The gradient of the log-decays, measured by its own size: dg_t carries the factor e^{g_t}, and is
nothing but rounding if it comes out as a difference of larger sums.

Bound: 1e-5 of the norm of a head's dg. Each of its terms is a product of decays, e^x by an
exponential of a 32-bit argument (half a step of an argument up to 64 is 2^-19: 1.3e-6 of the
result, for up to two factors), and of dot products of fp32 sums (up to 48 adds of 2^-23: 5.7e-6)."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def both(W, x, N, dy, S0=None, dS=None):
    at = lambda t: None if t is None else t[None].cuda()  # noqa: E731
    c = [t.cuda() for t in x]
    _, _, ws = W.wkv_gdr_forward_checkpointed(*c, state=at(S0), scale=N ** -0.5)
    got = W.wkv_gdr_backward(*c, dy[None].cuda(), ws, grad_state=at(dS), scale=N ** -0.5)
    want = ref.rule_gradients(*[t[0] for t in x], N ** -0.5, dy, S0, dS)
    return got["dg"][0].cpu().double(), want["dg"]


def near(got, want, what):
    err, size = (got - want).norm(dim=0), want.norm(dim=0)
    assert bool((err <= 1e-5 * size).all()), (what, (err / size).tolist())


def problem(T, Hk, H, N, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = list(ref.inputs((1, T), Hk, H, N, dtype, seed + 1))
    return x, r(T, H, N).to(dtype), 0.3 * r(H, N, N), 0.3 * r(H, N, N), gen


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_decays_of_every_size(W, N, dtype, shared):
    # a head for each size of decay, from nearly none to e^-40 a token
    sizes = torch.tensor([1e-3, 0.1, 1.0, 5.0, 8.0, 12.0, 16.0, 40.0])
    T, H = 150, len(sizes)
    x, dy, S0, dS, gen = problem(T, H // 2 if shared else H, H, N, dtype, 91)
    x[3] = -sizes * (0.9 + 0.2 * torch.rand(1, T, H, generator=gen))
    near(*both(W, x, N, dy, S0, dS), "with states")
    near(*both(W, x, N, dy), "from nothing")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_a_state_that_is_gone(W, N, dtype):
    # after g = -inf nothing depends on the decay: its gradient is zero, and the others are not
    # touched by it
    T, H = 140, 2
    x, dy, S0, dS, _ = problem(T, 1, H, N, dtype, 93)
    gone = [0, 7, 40, 63, 64, 100, 139]
    x[3][0, gone] = float("-inf")
    got, want = both(W, x, N, dy, S0, dS)
    assert bool((want[gone] == 0).all()) and bool((got[gone] == 0).all())
    near(got, want, "the others")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_nothing_written_yet(W, N, dtype):
    # from nothing, tokens that write nothing: up to the first that writes there is nothing to decay
    T, H = 100, 2
    x, dy, _, dS, _ = problem(T, 2, H, N, dtype, 95)
    for h, first in ((0, 20), (1, 70)):
        x[4][0, :first, h] = 0.0
    got, want = both(W, x, N, dy, None, dS)
    for h, first in ((0, 20), (1, 70)):
        assert bool((want[:first + 1, h] == 0).all()) and bool((got[:first + 1, h] == 0).all())
    near(got, want, "the others")
