"""What the autograd functions meet in a program: tensors and gradients that are contiguous but start
anywhere, another default type than fp32, and calls that no backward follows."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def shifted(t):
    """A contiguous copy of t that starts one element behind an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    out = buf[1:].view(t.shape)
    out.copy_(t)
    return out


def run(x, state, off, dy, dS, change=lambda t: t):
    from rwkv_linear_attention_wkv_b200.autograd import gated_delta_rule
    leaves = [change(t.detach()).requires_grad_() for t in list(x) + [state]]
    y, S = gated_delta_rule(*leaves[:5], state=leaves[5], scale=0.25, seq_offsets=off)
    return [y, S] + list(torch.autograd.grad([y, S], leaves, [change(dy), change(dS)]))


@pytest.fixture(scope="module", params=[False, True], ids=["rows", "packed"])
def case(request):
    T, H, N = 50, 2, 64
    off = torch.tensor([1, 20, 45], dtype=torch.int32, device="cuda") if request.param else None
    n = 2 if request.param else 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = [t.cuda() for t in ref.inputs((1, T), 1, H, N, BF16, 2)]
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=FP32)  # noqa: E731
    return x, 0.3 * r(n, H, N, N), off, r(1, T, H, N).to(BF16), r(n, H, N, N)


def test_tensors_that_start_anywhere(case):
    for a, b in zip(run(*case), run(*case, change=shifted)):
        assert torch.equal(a, b)


def test_nothing_is_kept_without_a_backward(case):
    from rwkv_linear_attention_wkv_b200.autograd import gated_delta_rule
    x, state, off, dy, dS = case
    want = run(*case)[:2]
    leaves = [t.detach().requires_grad_() for t in x]
    for grad, ins in ((False, leaves), (True, x)):
        with torch.set_grad_enabled(grad):
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            got = gated_delta_rule(*ins, state=state, scale=0.25, seq_offsets=off)
            used = torch.cuda.max_memory_allocated() - before
        assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(want, got))
        # the results alone, in blocks of 512 bytes
        assert used <= sum(t.numel() * t.element_size() + 512 for t in got), used


@pytest.mark.parametrize("default", [BF16, torch.float64])
def test_another_default_type(case, default):
    want = run(*case)
    torch.set_default_dtype(default)
    try:
        got = run(*case)
    finally:
        torch.set_default_dtype(FP32)
    for a, b in zip(want, got):
        assert a.dtype == b.dtype and torch.equal(a, b)
