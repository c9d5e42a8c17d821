"""The gated delta rule and the norms around it, from their definitions in 64 bits (torch on the
CPU), token by token, with the adjoint of every step. No code of the library is used here.

Comparison rules:
  fp32 results: |x - ref| <= 1e-5 (1 + m), m the largest |ref| of the same head and sequence (of
    the same row for a norm): the library's fp32 rule. 1e-5 is 168 half steps of 2^-24. A state
    entry, and a read-out, is a sum of 64 or 128 products of entries up to m, each rounded once,
    and what a token adds is damped by every later token (|I - beta k k^T| <= 1), so an error of
    a few times sqrt(128) half steps at the size of the terms is what 32-bit sums leave.
  bf16 results: half a step of bf16 on top, 2^-8 |ref|.
"""
import torch


def rule(q, k, v, g, beta, scale, state=None):
    """One sequence: q, k (T, Hk, N); v (T, H, N); g, beta (T, H); state (H, N, N)."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    T, H, N = v.shape
    G = H // q.shape[1]
    S = torch.zeros(H, N, N, dtype=torch.float64) if state is None else state.double().clone()
    y = torch.zeros(T, H, N, dtype=torch.float64)
    for t in range(T):
        kt, qt = k[t].repeat_interleave(G, 0), q[t].repeat_interleave(G, 0)
        A = torch.exp(g[t])[:, None, None] * S
        e = v[t] - (A * kt[:, None, :]).sum(-1)
        S = A + (beta[t][:, None] * e)[:, :, None] * kt[:, None, :]
        y[t] = scale * (S * qt[:, None, :]).sum(-1)
    return y, S


def rule_gradients(q, k, v, g, beta, scale, dy, state=None, dstate=None):
    """Gradients of sum(dy y) + sum(dstate S_T) for one sequence: the adjoint of each token's
    three lines, from the last token to the first."""
    q, k, v, g, beta, dy = (x.double() for x in (q, k, v, g, beta, dy))
    T, H, N = v.shape
    Hk = q.shape[1]
    G = H // Hk
    S = torch.zeros(H, N, N, dtype=torch.float64) if state is None else state.double().clone()
    seen = []
    for t in range(T):
        kt = k[t].repeat_interleave(G, 0)
        A = torch.exp(g[t])[:, None, None] * S
        e = v[t] - (A * kt[:, None, :]).sum(-1)
        S = A + (beta[t][:, None] * e)[:, :, None] * kt[:, None, :]
        seen.append((A, e, S))
    D = torch.zeros(H, N, N, dtype=torch.float64) if dstate is None else dstate.double().clone()
    dq, dk = torch.zeros(T, H, N, dtype=torch.float64), torch.zeros(T, H, N, dtype=torch.float64)
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        A, e, St = seen[t]
        kt, qt = k[t].repeat_interleave(G, 0), q[t].repeat_interleave(G, 0)
        dq[t] = scale * (St * dy[t][:, :, None]).sum(1)
        D = D + scale * dy[t][:, :, None] * qt[:, None, :]
        du = (D * kt[:, None, :]).sum(-1)
        dk[t] = (D * (beta[t][:, None] * e)[:, :, None]).sum(1)
        db[t] = (du * e).sum(-1)
        de = beta[t][:, None] * du
        dv[t] = de
        dk[t] -= (A * de[:, :, None]).sum(1)
        D = D - de[:, :, None] * kt[:, None, :]
        dg[t] = (D * A).sum((-1, -2))
        D = torch.exp(g[t])[:, None, None] * D
    together = lambda x: x.reshape(T, Hk, G, N).sum(2)  # noqa: E731
    return {"dq": together(dq), "dk": together(dk), "dv": dv, "dg": dg, "dbeta": db, "dstate": D}


def inputs(lead, Hk, H, N, dtype, seed, strong=False):
    """q, k unit vectors, v ~ N(0, 1) rounded to dtype; g, beta as a model's; CPU tensors.
    strong: decays down to e^-40 a token and write strengths up to 2 (beta |k|^2 = 2)."""
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda: torch.nn.functional.normalize(normal(*lead, Hk, N), dim=-1).to(dtype)  # noqa: E731
    q, k, v = unit(), unit(), normal(*lead, H, N).to(dtype)
    g = -torch.nn.functional.softplus(normal(*lead, H) - 1.0)
    beta = torch.sigmoid(normal(*lead, H))
    if strong:
        g = torch.where(torch.rand(g.shape, generator=gen) < 0.1, 40 * g, g)
        beta = 1.98 * beta
    return q, k, v, g.float(), beta.float()


def rows(q, k, v, g, beta, scale, state=None, spans=None):
    """rule() over the batch rows, or over the spans (start, end) of one packed row. Rows of y
    that no span covers are NaN."""
    if spans is None:
        got = [rule(q[b], k[b], v[b], g[b], beta[b], scale, None if state is None else state[b])
               for b in range(v.shape[0])]
        return torch.stack([x[0] for x in got]), torch.stack([x[1] for x in got])
    y = torch.full(v.shape, float("nan"), dtype=torch.float64)
    states = []
    for i, (a, b) in enumerate(spans):
        r = slice(a, max(a, b))
        y[0, r], S = rule(q[0, r], k[0, r], v[0, r], g[0, r], beta[0, r], scale,
                          None if state is None else state[i])
        states.append(S)
    return y, torch.stack(states)


def assert_close(got, ref, what, head_dim=None):
    """The rules above; head_dim: the dimension of ref that counts heads (m is then taken over
    everything else), None: m is the largest |ref| of all."""
    x = got.detach().cpu().double()
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    if ref.numel() == 0:
        return
    if head_dim is None:
        m = ref.abs().max()
    else:
        m = ref.abs().amax([d for d in range(ref.dim()) if d != head_dim % ref.dim()], keepdim=True)
    bound = 1e-5 * (1 + m) + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 0.0)
    err = (x - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound).nan_to_num(9e9).max()))


def norm_gate(h, weight, gate, x, scale, next_weight, group, act, eps):
    """out and y of the norm around a block; everything (R, C) or (C,), None where left out."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    h, weight, gate, x, scale, next_weight = map(d, (h, weight, gate, x, scale, next_weight))
    R, C = h.shape
    hg = h.reshape(R, C // group, group)
    m = (hg / torch.sqrt((hg ** 2).mean(-1, keepdim=True) + eps)).reshape(R, C)
    if weight is not None:
        m = m * weight
    if gate is not None:
        m = m * torch.sigmoid(gate) * (gate if act == "silu" else 1.0)
    out = m if x is None else x + (m if scale is None else scale * m)
    if next_weight is None:
        return out, None
    return out, out / torch.sqrt((out ** 2).mean(-1, keepdim=True) + eps) * next_weight


NORM_NAMES = ("h", "weight", "gate", "x", "scale", "next_weight")


def norm_gate_gradients(inputs, group, act, eps, dout, dy):
    """Gradients by autograd in 64 bits, and for the sums over rows the sums of |terms|."""
    leaves = {n: t.double().requires_grad_() for n, t in inputs.items() if t is not None}
    out, y = norm_gate(*[leaves.get(n) for n in NORM_NAMES], group, act, eps)
    per_row = torch.zeros(out.shape[0], dtype=torch.float64)
    if dout is not None:
        per_row = per_row + (out * dout.double()).sum(1)
    if dy is not None:
        per_row = per_row + (y * dy.double()).sum(1)
    wanted = [n for n in leaves if not (n == "next_weight" and dy is None)]
    grads = dict(zip(wanted, torch.autograd.grad(per_row.sum(), [leaves[n] for n in wanted],
                                                 retain_graph=True)))
    sums = {}
    for n in ("weight", "scale", "next_weight"):
        if n in grads:
            sums[n] = sum(torch.autograd.grad(r, leaves[n], retain_graph=True)[0].abs()
                          for r in per_row)
    return grads, sums
