"""Failures of a launch, and of calls before it: each is reported by the call that it happened in,
and a call that was made is not made again."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    yield W
    W.lib.wkv_testing_fail_launches(0)


@pytest.fixture
def step(W):
    """(a decode step's inputs, the state before it, the state after one)."""
    x = [t.cuda() for t in ref.inputs((2,), 1, 2, 64, BF16, 1)]
    before = 0.3 * torch.randn(2, 2, 64, 64, device="cuda")
    after = before.clone()
    W.wkv_gdr_decode_step(*x, after)
    torch.cuda.synchronize()
    return x, before, after


def test_an_earlier_error_is_not_this_calls(W, step):
    x, before, after = step
    S = before.clone()
    assert W.lib.wkv_testing_leave_error() == 0
    W.wkv_gdr_decode_step(*x, S)
    assert torch.equal(S, after)
    assert W.lib.wkv_testing_leave_error() == 0
    y, S1 = W.wkv_gdr_forward(*[t[:, None].contiguous() for t in x], state=before)
    k = torch.randn(2, 64, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    want = W.wkv_forward(w, w, k, k)
    assert W.lib.wkv_testing_leave_error() == 0
    assert torch.equal(W.wkv_forward(w, w, k, k), want)
    assert W.wkv_stream_status() == 0


def test_a_call_that_failed_is_not_made_again(W, step):
    x, before, after = step
    S = before.clone()
    W.lib.wkv_testing_fail_launches(1)
    with pytest.raises(W.WkvError, match="wkv_gdr_decode_step"):
        W.wkv_gdr_decode_step(*x, S)
    assert torch.equal(S, after)
    # the state written over the one it came from; the norms' result over their input
    x2 = [t[:, None].contiguous() for t in x]
    want = W.wkv_gdr_forward(*x2, state=before)[1]
    S = before.clone()
    W.lib.wkv_testing_fail_launches(1)
    with pytest.raises(W.WkvError, match="wkv_gdr_forward"):
        W.wkv_gdr_forward(*x2, state=S, state_out=S)
    assert torch.equal(S, want)
    h = torch.randn(3, 64, device="cuda")
    want = W.wkv_norm_gate_forward(h, act="none")[0]
    W.lib.wkv_testing_fail_launches(1)
    with pytest.raises(W.WkvError, match="wkv_norm_gate_forward"):
        W.wkv_norm_gate_forward(h, act="none", out=h)
    assert torch.equal(h, want)


def test_the_next_call_is_sound(W, step):
    x, before, after = step
    _, _, ws = W.wkv_gdr_forward_checkpointed(*[t[:, None].contiguous() for t in x])
    x2 = [t[:, None].contiguous() for t in x]
    W.lib.wkv_testing_fail_launches(1)
    with pytest.raises(W.WkvError) as e:
        W.wkv_gdr_backward(*x2, x2[2], ws)
    assert e.value.status == 3  # WKV_ERR_CUDA
    S = before.clone()
    W.wkv_gdr_decode_step(*x, S)
    assert torch.equal(S, after)
