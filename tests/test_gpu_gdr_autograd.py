"""The autograd functions of the gated delta rule and of the norms around a block: gradients bit
for bit those of the calls they marshal, and a time-mixing block made of them (rule, per-head norm
with its gate, scaled residual, next norm), forward and backward as a user would run it.

The block as a whole is ill-conditioned where a head's read-out is nearly zero and the norm divides
by it (its first token reads beta (q . k) v, and q . k may be far below the rounding of q and k over
|q . k|), so no bound on its gradients follows from the types. Each operator in it is compared with
64 bits on the very inputs and gradients that it met there, by the rules of its own tests."""
import pytest

torch = pytest.importorskip("torch")

import gdr_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def W():
    import rwkv_linear_attention_wkv_b200 as W
    return W


def leaf(t):
    return t.cuda().requires_grad_()


@pytest.mark.parametrize("packed", [False, True])
def test_rule_gradients_are_the_calls(W, packed):
    from rwkv_linear_attention_wkv_b200.autograd import gated_delta_rule
    T, N, H, Hk = 77, 64, 4, 2
    off = torch.tensor([1, 30, 70], dtype=torch.int32, device="cuda") if packed else None
    n = 2 if packed else 1
    leaves = [leaf(t) for t in ref.inputs((1, T), Hk, H, N, BF16, 1)]
    state = leaf(0.3 * torch.randn(n, H, N, N, generator=torch.Generator().manual_seed(2)))
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(1, T, H, N, device="cuda", generator=gen).to(BF16)
    dS = torch.randn(n, H, N, N, device="cuda", generator=gen)
    y, S = gated_delta_rule(*leaves, state=state, scale=0.25, seq_offsets=off)
    torch.autograd.backward([y, S], [dy, dS])
    x = [t.detach() for t in leaves]
    zeros = {"dq": x[0], "dk": x[1], "dv": x[2], "dg": x[3], "dbeta": x[4], "dstate": state.detach()}
    y2, S2, ws = W.wkv_gdr_forward_checkpointed(*x, state=state.detach(), scale=0.25,
                                                seq_offsets=off, y=torch.zeros_like(y))
    want = W.wkv_gdr_backward(*x, dy, ws, grad_state=dS, scale=0.25, seq_offsets=off,
                              grads={m: torch.zeros_like(t) for m, t in zeros.items()})
    assert torch.equal(y, y2) and torch.equal(S, S2)
    for t, m in zip(leaves + [state], ("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        assert torch.equal(t.grad, want[m]), m


def test_rule_one_result_unused_and_strided_inputs(W):
    from rwkv_linear_attention_wkv_b200.autograd import gated_delta_rule
    x = ref.inputs((2, 40), 2, 2, 64, FP32, 4)
    leaves = [leaf(t) for t in x]
    y, S = gated_delta_rule(*leaves)
    S.sum().backward()
    only_state = [t.grad.clone() for t in leaves]
    assert bool((only_state[0] == 0).all())  # q does not reach the states
    # the same values, time and heads exchanged in memory
    other = [leaf(t.transpose(1, 2).contiguous()) for t in x]
    y2, S2 = gated_delta_rule(*[t.transpose(1, 2) for t in other])
    assert torch.equal(y, y2)
    S2.sum().backward()
    for a, b in zip(only_state, other):
        assert torch.equal(a, b.grad.transpose(1, 2))
    k = leaf(x[1])
    y, S = gated_delta_rule(x[0].cuda(), k, *[t.cuda() for t in x[2:]])
    g, = torch.autograd.grad((y * y).sum(), k, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_norm_gate_gradients_are_the_calls(W):
    from rwkv_linear_attention_wkv_b200.autograd import norm_gate
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    h, z, x = (leaf(r(3, 5, 128).to(BF16)) for _ in range(3))
    w, s, nw = (leaf(1 + 0.3 * r(128)) for _ in range(3))
    out, y = norm_gate(h, w, z, x, s, nw, group=64, act="silu")
    dout, dy = (r(3, 5, 128).to(BF16).cuda() for _ in range(2))
    torch.autograd.backward([out, y], [dout, dy])
    d = [t.detach() for t in (h, w, z, x, s, nw)]
    want = W.wkv_norm_gate_backward(d[0], d[1], dout, gate=d[2], x=d[3], scale=d[4],
                                    next_weight=d[5], dy=dy, group=64, act="silu")
    for t, n in ((h, "dh"), (w, "dweight"), (z, "dgate"), (x, "dx"), (s, "dscale"),
                 (nw, "dnext_weight")):
        assert torch.equal(t.grad, want[n]), n
    # only y used, no residual
    h2 = leaf(r(7, 96))
    out, y = norm_gate(h2, act="none")
    assert y is None
    out.sum().backward()
    assert h2.grad.shape == h2.shape


def block_parameters(C, H, Hk, N, gen):
    r = lambda *s: torch.randn(*s, generator=gen) / s[0] ** 0.5  # noqa: E731
    return {"q": r(C, Hk * N), "k": r(C, Hk * N), "v": r(C, H * N), "a": r(C, H), "b": r(C, H),
            "z": r(C, H * N), "norm": 1 + 0.2 * r(1, H * N)[0], "o": r(H * N, C),
            "post": 1 + 0.2 * r(1, C)[0], "scale": 0.5 + 0.1 * r(1, C)[0].abs(),
            "next": 1 + 0.2 * r(1, C)[0]}


def block(x, P, H, Hk, N, rule, norm):
    """A time-mixing block with the gated delta rule: x (B, T, C) to the residual stream after it
    and the next block's normed input."""
    B, T, C = x.shape
    unit = torch.nn.functional.normalize
    q = unit((x @ P["q"]).view(B, T, Hk, N).to(torch.promote_types(x.dtype, FP32)), dim=-1).to(x.dtype)
    k = unit((x @ P["k"]).view(B, T, Hk, N).to(torch.promote_types(x.dtype, FP32)), dim=-1).to(x.dtype)
    v = (x @ P["v"]).view(B, T, H, N)
    wide = torch.promote_types(x.dtype, FP32)
    g = -torch.nn.functional.softplus((x @ P["a"]).to(wide))
    beta = torch.sigmoid((x @ P["b"]).to(wide))
    y = rule(q, k, v, g, beta, N ** -0.5)
    m = norm(y.reshape(B, T, H * N), P["norm"], x @ P["z"], None, None, None, N, "silu")[0]
    return norm(m @ P["o"], P["post"], None, x, P["scale"], P["next"], C, "none")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_block_of_them(W, dtype):
    from rwkv_linear_attention_wkv_b200.autograd import gated_delta_rule, norm_gate
    B, T, C, H, Hk, N = 2, 50, 96, 2, 1, 64
    gen = torch.Generator().manual_seed(6)
    vectors = ("norm", "post", "scale", "next")
    P = {n: leaf(t if n in vectors else t.to(dtype)) for n, t in
         block_parameters(C, H, Hk, N, gen).items()}
    x = leaf(torch.randn(B, T, C, generator=gen).to(dtype))
    d0, d1 = (torch.randn(B, T, C, generator=gen).to(dtype).cuda() for _ in range(2))
    met = []

    def watched(t):
        # a copy of its own, so that its gradient is this operator's alone
        if t is not None:
            t = t.clone()
            t.retain_grad()
        return t

    def rule(*args):
        ins = [watched(t) for t in args[:5]]
        y, S = gated_delta_rule(*ins, scale=args[5])
        y.retain_grad()
        met.append(("rule", ins, args[5], y))
        return y

    def norm(h, w, z, r, s, nw, group, act):
        ins = [watched(t) for t in (h, w, z, r, s, nw)]
        outs = norm_gate(*ins, group=group, act=act)
        outs = [None if t is None else watched(t) for t in outs]
        met.append(("norm", ins, (group, act), outs))
        return outs

    out, y = block(x, P, H, Hk, N, rule, norm)
    torch.autograd.backward([out, y], [d0, d1])
    assert W.wkv_stream_status() == 0 and len(met) == 3
    assert all(t.grad is not None for t in list(P.values()) + [x])
    at = lambda t: None if t is None else t.detach().cpu()  # noqa: E731
    for kind, ins, how, got in met:
        data = [at(t) for t in ins]
        if kind == "rule":
            yr, _ = ref.rows(*data, how)
            ref.assert_close(got, yr, "rule y", head_dim=2)
            for b in range(B):
                want = ref.rule_gradients(*[t[b] for t in data], how, at(got.grad)[b])
                for t, n in zip(ins, ("dq", "dk", "dv", "dg", "dbeta")):
                    ref.assert_close(t.grad[b], want[n], n, head_dim=1)
            continue
        flat = [None if t is None else t.reshape(-1, t.shape[-1]) if t.dim() > 1 else t
                for t in data]
        wide = flat[0].shape
        want, sums = ref.norm_gate_gradients(
            dict(zip(ref.NORM_NAMES, flat)), *how, 1e-6, at(got[0].grad).reshape(wide),
            None if got[1] is None else at(got[1].grad).reshape(wide))
        o, n = ref.norm_gate(*flat, *how, 1e-6)
        ref.assert_close(got[0].reshape(wide), o, "out", head_dim=0)
        if n is not None:
            ref.assert_close(got[1].reshape(wide), n, "y", head_dim=0)
        for t, name in zip(ins, ref.NORM_NAMES):
            if t is None:
                continue
            if name in sums:
                bound = 1e-5 * (1 + sums[name] + sums[name].max())
                assert bool(((at(t.grad).double() - want[name]).abs() <= bound).all()), name
            else:
                ref.assert_close(t.grad.reshape(wide), want[name], name, head_dim=0)
