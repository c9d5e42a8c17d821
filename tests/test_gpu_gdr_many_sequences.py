"""Packed rows of as many sequences as one warp orders by length and cuts into segments (two a lane:
64), and one more. Comparison: the rules of gdr_reference."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

FP32 = torch.float32


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


# long: the tokens of the long sequences; 1500 are cut into segments (up to 64 sequences), 70 are not
@pytest.mark.parametrize("long", [70, 1500])
@pytest.mark.parametrize("n", [33, 64, 65])
def test_many_sequences(W, n, long):
    H, N = 1, 64
    gen = torch.Generator().manual_seed(n + long)
    lens = torch.randint(0, 10, (n,), generator=gen)
    lens[[3, n - 2]] = torch.tensor([long - 30, long])
    off = [2] + (2 + torch.cumsum(lens, 0)).tolist()
    T = off[-1] + 3
    x = ref.inputs((1, T), 1, H, N, FP32, 5)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    S0, dS, dy = 0.3 * r(n, H, N, N), 0.3 * r(n, H, N, N), r(1, T, H, N)
    c, o = [t.cuda() for t in x], torch.tensor(off, dtype=torch.int32, device="cuda")
    y, S, ws = W.wkv_gdr_forward_checkpointed(*c, state=S0.cuda(), scale=0.5, seq_offsets=o,
                                              y=torch.full((1, T, H, N), 7.0, device="cuda"))
    spans = list(zip(off[:-1], off[1:]))
    yr, Sr = ref.rows(*x, 0.5, S0, spans)
    rows = slice(off[0], off[-1])
    assert bool((y[:, :2] == 7).all()) and bool((y[:, off[-1]:] == 7).all())
    ref.assert_close(y[:, rows], yr[:, rows], "y", head_dim=2)
    ref.assert_close(S, Sr, "state", head_dim=1)
    got = W.wkv_gdr_backward(*c, dy.cuda(), ws, grad_state=dS.cuda(), scale=0.5, seq_offsets=o)
    for i, (a, b) in enumerate(spans):
        want = ref.rule_gradients(*[t[0, a:b] for t in x], 0.5, dy[0, a:b], S0[i], dS[i])
        ref.assert_close(got["dstate"][i], want["dstate"], "dstate", head_dim=0)
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            ref.assert_close(got[m][0, a:b], want[m], m, head_dim=1)
