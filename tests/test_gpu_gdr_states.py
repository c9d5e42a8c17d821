"""The gradient of the initial states, by its own norm: no further off than sums in 32 bits."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def off_by(T, H, N, dtype, g, seed):
    import rwkv_linear_attention_wkv_b200 as W
    gen = torch.Generator().manual_seed(seed)
    q, k, v, _, beta = ref.inputs((1, T), 1, H, N, dtype, seed + 1)
    g = g * (0.9 + 0.2 * torch.rand(1, T, H, generator=gen))
    x = (q, k, v, g, beta)
    S0, dS = (0.3 * torch.randn(1, H, N, N, generator=gen) for _ in range(2))
    dy = torch.randn(1, T, H, N, generator=gen).to(dtype)
    c = [t.cuda() for t in x]
    _, _, ws = W.wkv_gdr_forward_checkpointed(*c, state=S0.cuda(), scale=N ** -0.5)
    got = W.wkv_gdr_backward(*c, dy.cuda(), ws, grad_state=dS.cuda(), scale=N ** -0.5)["dstate"]
    want = ref.rule_gradients(*[t[0] for t in x], N ** -0.5, dy[0], S0[0], dS[0])["dstate"]
    return (got[0].cpu().double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_strong_decays(N, dtype):
    # One token, e^-45 to e^-36: the decay is a factor of all of a head's gradient. By a correction
    # of the exponential of its 32-bit argument it is off by 2^-22 and 2^-24 (without: by up to
    # 2^-19 ln 2 = 1.3e-6); two sums cut once or twice at 2^-23, three roundings of 2^-24.
    bound = 1.25 * 2.0 ** -22 + 2 * 2.0 ** -23 + 3 * 2.0 ** -24  # 7.2e-7
    worst = off_by(1, 16, N, dtype, -40.0, 3).max()
    assert float(worst) <= bound, float(worst)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 128])
def test_mild_decays(N, dtype):
    # Every group adds two products to the gradient. A matrix instruction cuts the sum that it adds
    # to, by 2^-24 of it on average, always towards zero: over many groups this is what the norm
    # shows. Two such cuts at the size of each product, two roundings to add them (2^-25 on average)
    # and as much again for the errors of dy's and de's factors: 2.4e-7. Both products in one sum
    # cut it seven times.
    worst = off_by(150, 4, N, dtype, -1.0, 5).max()
    assert float(worst) <= 4 * 2.0 ** -24, float(worst)
