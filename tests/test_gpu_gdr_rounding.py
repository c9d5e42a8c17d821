"""bf16 results of the gated delta rule are fp32 results rounded once: what is computed on the way
is as good as in an fp32 problem.

A result x of a 64-bit value r has |x - r| <= h + d: h half a step of bf16 at r (2^(e - 8), e the
exponent of r) and d what fp32 sums leave. A product's 64 or 128 terms are added by at most 24 matrix
instructions (8 steps of 16 terms, 3 parts of the factor that is not a bf16 value), each of which
cuts at most 2^-23 of the largest partial sum: 24 x 2^-23 < 2^-18 of it. Where both factors are split
(dk: 6 part pairs, 48 instructions) it is 2^-17. A partial sum is no larger than the head's largest
entry m, which is the largest of thousands of full sums. Parts of 16 bits leave 2^-15 of a value."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def assert_rounded(got, want, grade, what):
    """got: bf16 (tokens, heads, N)."""
    assert got.dtype == BF16
    err = (got.detach().cpu().double() - want).abs()
    _, e = torch.frexp(want)  # |want| in [2^(e - 1), 2^e)
    half = torch.ldexp(torch.ones_like(want), e - 1 - 8)
    over = err - half - grade * want.abs().amax((0, 2), keepdim=True)
    assert bool((over <= 0).all()), (what, int((over > 0).sum()), float((err / half).max()))


# walked by two producer warps (many heads), by four, and in segments (1100 tokens)
@pytest.mark.parametrize("N,T,Hk,H", [(64, 400, 2, 4), (128, 300, 1, 2), (64, 40, 75, 150),
                                      (64, 1100, 1, 1), (128, 1100, 1, 1)])
def test_read_outs(W, N, T, Hk, H):
    x = ref.inputs((1, T), Hk, H, N, BF16, 81)
    S0 = 0.3 * torch.randn(1, H, N, N, generator=torch.Generator().manual_seed(82))
    y, _ = W.wkv_gdr_forward(*[t.cuda() for t in x], state=S0.cuda(), scale=N ** -0.5)
    want, _ = ref.rule(*[t[0] for t in x], N ** -0.5, S0[0])
    assert_rounded(y[0], want, 2.0 ** -18, "y")


@pytest.mark.parametrize("N,T,Hk,H", [(64, 400, 4, 4), (64, 300, 2, 4), (128, 300, 2, 2),
                                      (128, 200, 1, 2)])
def test_gradients(W, N, T, Hk, H):
    gen = torch.Generator().manual_seed(83)
    x = ref.inputs((1, T), Hk, H, N, BF16, 84)
    S0, dS = (0.3 * torch.randn(1, H, N, N, generator=gen) for _ in range(2))
    dy = torch.randn(1, T, H, N, generator=gen).to(BF16)
    c = [t.cuda() for t in x]
    y, _, ws = W.wkv_gdr_forward_checkpointed(*c, state=S0.cuda(), scale=N ** -0.5)
    got = W.wkv_gdr_backward(*c, dy.cuda(), ws, grad_state=dS.cuda(), scale=N ** -0.5)
    want = ref.rule_gradients(*[t[0] for t in x], N ** -0.5, dy[0], S0[0], dS[0])
    for n in ("dq", "dv", "dk"):
        assert_rounded(got[n][0], want[n], 2.0 ** -17, n)
