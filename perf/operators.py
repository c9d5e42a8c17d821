"""What a time-mixing layer with the gated delta rule costs: the rule over whole sequences
(prefill), for one token of many sequences (decode) and with its gradients (training), and the
norms, gate and scaled residual around the layer, forward and with gradients.

Per head with a state S (value channel x key channel), log-decay g_t <= 0 and write strength
beta_t, the gated delta rule is

    e_t = v_t - exp(g_t) S_{t-1} k_t
    S_t = exp(g_t) S_{t-1} + beta_t e_t k_t^T
    y_t = scale * S_t q_t

H value heads share Hk query/key heads in groups of H / Hk. The norm around the layer is, per
token, with RMS(x) the root of the mean square plus eps over a group of channels (a head, or the
row),

    m   = act(gate) * (weight * h / RMS_group(h))
    out = x + residual_scale * m
    y   = next_weight * out / RMS_row(out)
"""
import math

import torch

own = False

CHUNK = 64


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence being decoded, a small model's heads: what a call costs
        {"name": "decode_1x12x64", "op": "decode", "n": 1, "slots": 1, "H": 12, "Hk": 12, "N": 64,
         "dtype": "bf16"},
        # a serving batch with a state pool: some rows are padding, heads of 128 share keys
        {"name": "decode_93x32x128", "op": "decode", "n": 93, "slots": 120, "H": 32, "Hk": 16,
         "N": 128, "dtype": "bf16"},
        # the large decode batch, fp32 activations
        {"name": "decode_256x64x64_fp32", "op": "decode", "n": 256, "slots": 256, "H": 64,
         "Hk": 64, "N": 64, "dtype": "fp32"},
        # a short prompt entering with a state (one request of a chat)
        {"name": "forward_1x133x12x64", "op": "forward", "B": 1, "T": 133, "H": 12, "Hk": 12,
         "N": 64, "dtype": "bf16", "packed": 0, "state": True},
        # the 8 x 4096 x 64-head prefill that the matrix-state forms of this library are timed on
        {"name": "forward_8x4096x64x64", "op": "forward", "B": 8, "T": 4096, "H": 64, "Hk": 64,
         "N": 64, "dtype": "bf16", "packed": 0, "state": False},
        # prompts of very different lengths packed into one row, heads of 128 in pairs
        {"name": "forward_packed_17x128", "op": "forward", "B": 1, "T": 9001, "H": 32, "Hk": 16,
         "N": 128, "dtype": "bf16", "packed": 17, "state": True},
        # one long fp32 sequence with few heads
        {"name": "forward_1x16384x8x64_fp32", "op": "forward", "B": 1, "T": 16384, "H": 8, "Hk": 4,
         "N": 64, "dtype": "fp32", "packed": 0, "state": True},
        # the 16 x 1024 x 768 training shape, forward and backward
        {"name": "train_16x1024x12x64", "op": "train", "B": 16, "T": 1024, "H": 12, "Hk": 12,
         "N": 64, "dtype": "bf16", "packed": 0, "state": False},
        # training on a packed row with states in and out, shared keys, fp32
        {"name": "train_packed_5x128_fp32", "op": "train", "B": 1, "T": 1811, "H": 8, "Hk": 4,
         "N": 128, "dtype": "fp32", "packed": 5, "state": True},
        # residual stream and next norm of a wide model's prefill, gated per-row norm
        {"name": "norm_32768x4096", "op": "norm", "R": 32768, "C": 4096, "group": 4096,
         "dtype": "bf16", "gate": "silu", "residual": True, "next": True},
        # the per-head norm and gate after the read-out, a decode batch
        {"name": "norm_heads_256x4096", "op": "norm", "R": 256, "C": 4096, "group": 64,
         "dtype": "bf16", "gate": "silu", "residual": False, "next": False},
        # the norms' training step at the 16 x 1024 x 768 shape
        {"name": "norm_train_16384x768", "op": "norm_train", "R": 16384, "C": 768, "group": 64,
         "dtype": "bf16", "gate": "sigmoid", "residual": True, "next": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "forward", "forward", "train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_train"):
        group = rng.choice([64, 64, 128, 0])
        if group:
            C = group * _log_int(rng, 1, 4096 // group)
        else:
            C = group = _log_int(rng, 32, 4096)
        most = (32768 * 4096 if op == "norm" else 16384 * 768) // (2 if dtype == "fp32" else 1)
        R = _log_int(rng, 1, min(32768, most // C))
        residual = rng.random() < 0.7
        return {"op": op, "R": R, "C": C, "group": group, "dtype": dtype,
                "gate": rng.choice(["silu", "sigmoid", "none"]), "residual": residual,
                "next": residual and rng.random() < 0.8}
    N = rng.choice([64, 128])
    Hk = _log_int(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 2, 3, 4])
    if op == "decode":
        n = _log_int(rng, 1, max(1, 256 * 64 * 64 * 64 // (H * N * N)) if H * N * N > 262144 else 256)
        return {"op": op, "n": n, "slots": n + rng.choice([0, 0, 1, 7, 30]), "H": H, "Hk": Hk,
                "N": N, "dtype": dtype}
    tokens = (8 * 4096 * 64 * 64 if op == "forward" else 16 * 1024 * 12 * 64) // (H * N * N // 64)
    tokens = max(1, min(16384, tokens // (2 if dtype == "fp32" else 1)))
    state = rng.random() < 0.6
    if rng.random() < 0.4:
        T = _log_int(rng, 1, tokens)
        return {"op": op, "B": 1, "T": T, "H": H, "Hk": Hk, "N": N, "dtype": dtype,
                "packed": _log_int(rng, 1, min(64, T)), "state": state}
    T = _log_int(rng, 1, tokens)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(32, tokens // T))), "T": T, "H": H, "Hk": Hk,
            "N": N, "dtype": dtype, "packed": 0, "state": state}


# --------------------------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _offsets(T, n, seed):
    """n + 1 offsets of n sequences of uneven lengths (some may be empty) over T tokens."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.rand(n, generator=g, dtype=torch.float64).square() + 1e-3
    ends = torch.round(torch.cumsum(cuts, 0) / cuts.sum() * T).to(torch.int64)
    ends[-1] = T
    return torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32)


def _live(case):
    """Rows of a decode batch that are no padding: with a pool of more slots than rows, some are."""
    n = case["n"]
    return n - (n // 16 + 1) if case["slots"] > n and n > 4 else n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_train"):
        R, C = case["R"], case["C"]
        s["h"] = (normal(R, C) * (0.2 + 2.0 * uniform(R, 1))).to(dt)
        s["weight"] = 1.0 + 0.3 * normal(C)
        s["gate"] = None if case["gate"] == "none" else normal(R, C).to(dt)
        s["x"] = (1.5 * normal(R, C)).to(dt) if case["residual"] else None
        s["scale"] = 0.1 + uniform(C) if case["residual"] else None
        s["next_weight"] = 1.0 + 0.3 * normal(C) if case["next"] else None
        if case["op"] == "norm_train":
            s["dout"] = normal(R, C).to(dt)
            s["dy"] = normal(R, C).to(dt) if case["next"] else None
        return s
    N, H, Hk = case["N"], case["H"], case["Hk"]
    lead = (case["n"],) if case["op"] == "decode" else (case["B"], case["T"])

    def unit(heads):
        x = normal(*lead, heads, N)
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    s["q"], s["k"] = unit(Hk), unit(Hk)
    s["v"] = normal(*lead, H, N).to(dt)
    rate = torch.exp(uniform(H) * math.log(16.0)) * 0.2  # per-head decay rates, 0.2 .. 3.2
    s["g"] = -rate * torch.log1p(torch.exp(normal(*lead, H) - 2.0))
    s["beta"] = torch.sigmoid(normal(*lead, H))
    s["scale"] = N ** -0.5
    if case["op"] == "decode":
        n, slots = case["n"], case["slots"]
        s["state"] = 0.3 * normal(slots, H, N, N)
        order = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
        s["live"] = _live(case)
        order[s["live"]:] = -1  # padding rows at the end of the batch
        s["slots"] = order if slots > n else None
        s["y"] = torch.zeros(n, H, N, device="cuda", dtype=dt)
        return s
    seqs = case["packed"] or case["B"]
    s["offsets"] = None
    if case["packed"]:
        offsets = _offsets(case["T"], case["packed"], int(seed))
        s["longest"] = max(1, int((offsets[1:] - offsets[:-1]).max()))
        s["offsets"] = offsets.cuda()
    s["state"] = 0.3 * normal(seqs, H, N, N) if case["state"] else None
    if case["op"] == "train":
        s["dy"] = normal(*lead, H, N).to(dt)
        s["dstate"] = 0.3 * normal(seqs, H, N, N) if case["state"] else None
    return s


# ---------------------------------------------------------------------------- plain forms

def _rows(offsets, longest, tokens):
    """Packed sequences as rows of a padded batch: the token of each place (sequences, longest),
    which places hold one, and each token's sequence and place in it."""
    off = offsets.to(torch.int64)
    t = torch.arange(longest, device=off.device)
    mask = t[None, :] < (off[1:] - off[:-1])[:, None]
    token = torch.arange(tokens, device=off.device)
    seq = torch.searchsorted(off[1:].contiguous(), token, right=True)
    return (off[:-1, None] + t[None, :]) * mask, mask, seq, token - off[seq]


def _plain_rule(q, k, v, g, beta, state, scale):
    """The rule over (B, T, heads, N) in chunks: inside a chunk the tokens' writes u solve a unit
    lower triangular system, the state passes from chunk to chunk. fp32, decays summed in fp64."""
    B, T, H, N = v.shape
    n = -(-T // CHUNK)

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - T))
        return x.reshape(B, n, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    q = q.repeat_interleave(H // q.shape[2], 2)
    k = k.repeat_interleave(H // k.shape[2], 2)
    q, k, v, g, beta = chunks(q), chunks(k), chunks(v), chunks(g.double()[..., None]), chunks(beta[..., None])
    total = torch.cumsum(g, 3)
    lower = torch.ones(CHUNK, CHUNK, device=q.device, dtype=torch.bool).tril()
    apart = (total - total.transpose(3, 4)).masked_fill(~lower, 0.0)
    decay = torch.exp(apart).float() * lower
    since = torch.exp(total).float()
    until = torch.exp(total[:, :, :, -1:] - total).float()
    eye = torch.eye(CHUNK, device=q.device)
    inner = eye + beta * decay * (k @ k.transpose(3, 4)) * (1 - eye)
    solved = torch.linalg.solve_triangular(inner, torch.cat([beta * v, beta * since * k], -1),
                                           upper=False, unitriangular=True)
    u0, w = solved[..., :N], solved[..., N:]
    reads = scale * decay * (q @ k.transpose(3, 4))
    qs, kw, end = scale * since * q, until * k, since[:, :, :, -1:]
    S = torch.zeros(B, H, N, N, device=q.device) if state is None else state
    ys = []
    for c in range(n):
        u = u0[:, :, c] - w[:, :, c] @ S.transpose(2, 3)
        ys.append(qs[:, :, c] @ S.transpose(2, 3) + reads[:, :, c] @ u)
        S = end[:, :, c] * S + u.transpose(2, 3) @ kw[:, :, c]
    y = torch.stack(ys, 2).permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, N)[:, :T]
    return y, S


def _plain_sequences(s, leaves):
    """The rule over the case's sequences, packed or not: outputs and final states, fp32."""
    q, k, v, g, beta, state = leaves
    if s["offsets"] is None:
        return _plain_rule(q, k, v, g, beta, state, s["scale"])
    at, mask, seq, place = _rows(s["offsets"], s["longest"], v.shape[1])
    parts = [x[0][at] * mask.reshape(mask.shape + (1,) * (x.dim() - 2)) for x in (q, k, v, g, beta)]
    y, last = _plain_rule(*parts, state, s["scale"])
    return y[seq, place][None], last


def _plain_forward(s):
    leaves = [x if x is None else x.float() for x in (s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"])]
    y, last = _plain_sequences(s, leaves)
    return y.to(s["v"].dtype), last


def _plain_train(s):
    leaves = [x if x is None else x.detach().float().requires_grad_()
              for x in (s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"])]
    y, last = _plain_sequences(s, leaves)
    loss = (y * s["dy"].float()).sum()
    if s["dstate"] is not None:
        loss = loss + (last * s["dstate"]).sum()
    wanted = [x for x in leaves if x is not None]
    grads = list(torch.autograd.grad(loss, wanted)) + [None] * (6 - len(wanted))
    dt = s["v"].dtype
    out = {"y": y.detach().to(dt), "state": last.detach(), "dq": grads[0].to(dt),
           "dk": grads[1].to(dt), "dv": grads[2].to(dt), "dg": grads[3], "dbeta": grads[4]}
    if s["state"] is not None:
        out["dstate"] = grads[5]
    return out


def _plain_decode(s):
    H, dt = s["case"]["H"], s["v"].dtype
    rows = slice(0, s["live"])
    at = rows if s["slots"] is None else s["slots"][rows].long()
    q, k, v = s["q"][rows].float(), s["k"][rows].float(), s["v"][rows].float()
    q = q.repeat_interleave(H // q.shape[1], 1)
    k = k.repeat_interleave(H // k.shape[1], 1)
    S = torch.exp(s["g"][rows])[..., None, None] * s["state"][at]
    e = v - (S * k[:, :, None, :]).sum(-1)
    S = S + (s["beta"][rows][..., None] * e)[..., None] * k[:, :, None, :]
    s["state"][at] = S
    s["y"][rows] = (s["scale"] * (S * q[:, :, None, :]).sum(-1)).to(dt)
    return s["y"], s["state"]


_EPS = 1e-6


def _plain_norm(case, h, weight, gate, x, scale, next_weight):
    R, C = h.shape
    hg = h.reshape(R, C // case["group"], case["group"])
    m = (hg * torch.rsqrt(hg.square().mean(-1, keepdim=True) + _EPS)).reshape(R, C) * weight
    if gate is not None:
        m = m * torch.sigmoid(gate) * (gate if case["gate"] == "silu" else 1.0)
    out = m if x is None else x + scale * m
    if next_weight is None:
        return out, None
    return out, out * torch.rsqrt(out.square().mean(-1, keepdim=True) + _EPS) * next_weight


_NORM = ("h", "weight", "gate", "x", "scale", "next_weight")


def _plain_norm_forward(s):
    dt = s["h"].dtype
    out, y = _plain_norm(s["case"], *[x if x is None else x.float() for x in (s[n] for n in _NORM)])
    return {"out": out.to(dt)} if y is None else {"out": out.to(dt), "y": y.to(dt)}


def _plain_norm_train(s):
    dt = s["h"].dtype
    leaves = {n: s[n].detach().float().requires_grad_() for n in _NORM if s[n] is not None}
    out, y = _plain_norm(s["case"], *[leaves.get(n) for n in _NORM])
    loss = (out * s["dout"].float()).sum() + (0.0 if y is None else (y * s["dy"].float()).sum())
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    got = {"out": out.detach().to(dt)}
    if y is not None:
        got["y"] = y.detach().to(dt)
    got.update({"d" + n: x.to(s[n].dtype) for n, x in grads.items()})
    return got


# -------------------------------------------------------------------------- the framework

def _own_forward(s):
    import rwkv_linear_attention_wkv_b200 as W
    return W.wkv_gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"],
                             scale=s["scale"], seq_offsets=s["offsets"])


def _own_train(s):
    import rwkv_linear_attention_wkv_b200 as W
    y, last, workspace = W.wkv_gdr_forward_checkpointed(
        s["q"], s["k"], s["v"], s["g"], s["beta"], state=s["state"], scale=s["scale"],
        seq_offsets=s["offsets"])
    grads = W.wkv_gdr_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], workspace,
                               grad_state=s["dstate"], scale=s["scale"],
                               seq_offsets=s["offsets"], want_dstate=s["state"] is not None)
    out = {"y": y, "state": last}
    out.update({n: x for n, x in grads.items() if x is not None})
    return out


def _own_decode(s):
    import rwkv_linear_attention_wkv_b200 as W
    y = W.wkv_gdr_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                              slots=s["slots"], scale=s["scale"], y=s["y"])
    return y, s["state"]


def _own_norm_forward(s):
    import rwkv_linear_attention_wkv_b200 as W
    out, y = W.wkv_norm_gate_forward(s["h"], s["weight"], gate=s["gate"], x=s["x"],
                                     scale=s["scale"], next_weight=s["next_weight"],
                                     group=s["case"]["group"], act=s["case"]["gate"], eps=_EPS)
    return {"out": out} if y is None else {"out": out, "y": y}


def _own_norm_train(s):
    import rwkv_linear_attention_wkv_b200 as W
    got = _own_norm_forward(s)
    grads = W.wkv_norm_gate_backward(s["h"], s["weight"], s["dout"], gate=s["gate"], x=s["x"],
                                     scale=s["scale"], next_weight=s["next_weight"], dy=s["dy"],
                                     group=s["case"]["group"], act=s["case"]["gate"], eps=_EPS)
    got.update({n: x for n, x in grads.items() if x is not None})
    return got


_PLAIN = {"forward": _plain_forward, "train": _plain_train, "decode": _plain_decode,
          "norm": _plain_norm_forward, "norm_train": _plain_norm_train}
_OWN = {"forward": _own_forward, "train": _own_train, "decode": _own_decode,
        "norm": _own_norm_forward, "norm_train": _own_norm_train}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# -------------------------------------------------------------------------- work and 64 bits

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        e, C = case["R"] * case["C"], case["C"]
        gate, res, nxt = case["gate"] != "none", case["residual"], case["next"]
        arrays = 2 + gate + res + nxt                        # h, gate, x in; out, y out
        params = 1 + res + nxt
        flops = e * (5 + 5 * gate + 2 * res + 4 * nxt)
        if case["op"] == "norm_train":
            arrays += 1 + nxt + 1 + gate + res               # dout, dy in; dh, dgate, dx out
            params *= 2
            flops *= 4
        return {"bytes": e * size * arrays + 4 * C * params, "flops": flops}
    N, H, Hk = case["N"], case["H"], case["Hk"]
    if case["op"] == "decode":
        n = _live(case)
        return {"bytes": n * (H * (N * N * 8 + 8) + (2 * Hk + 2 * H) * N * size), "flops": n * H * 6 * N * N}
    tokens = case["B"] * case["T"]
    states = (case["packed"] or case["B"]) * H * N * N * 4
    bytes_ = tokens * ((2 * Hk + 2 * H) * N * size + 8 * H) + states * (1 + case["state"])
    flops = tokens * H * 6 * N * N
    if case["op"] == "train":
        bytes_ += tokens * ((2 * Hk + 2 * H) * N * size + 8 * H) + states * 2 * case["state"]
        flops += tokens * H * 14 * N * N
    return {"bytes": bytes_, "flops": flops}


def _exact_sequence(q, k, v, g, beta, S, scale, dy=None, dS=None):
    """Token by token in fp64 for sequences of one length: (b, t, heads, N), S (b, heads, N, N).
    With dy, also the gradients: the adjoint of each token's update, the states between recomputed
    from those kept every 64 tokens."""
    T = v.shape[1]
    y, kept, alpha = torch.empty_like(v), [], torch.exp(g)

    def step(S, t):
        A = alpha[:, t, :, None, None] * S
        e = v[:, t] - torch.einsum("bhij,bhj->bhi", A, k[:, t])
        return A, e, A + torch.einsum("bhi,bhj->bhij", beta[:, t, :, None] * e, k[:, t])

    for t in range(T):
        if dy is not None and t % 64 == 0:
            kept.append(S.clone())
        S = step(S, t)[2]
        y[:, t] = scale * torch.einsum("bhij,bhj->bhi", S, q[:, t])
    if dy is None:
        return y, S
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    dS = torch.zeros_like(S) if dS is None else dS.clone()
    for c in range(len(kept) - 1, -1, -1):
        walk, X = [], kept[c]
        for t in range(64 * c, min(T, 64 * c + 64)):
            A, e, X = step(X, t)
            walk.append((t, A, e, X))
        for t, A, e, X in reversed(walk):
            dq[:, t] = scale * torch.einsum("bhij,bhi->bhj", X, dy[:, t])
            dS += scale * torch.einsum("bhi,bhj->bhij", dy[:, t], q[:, t])
            du = torch.einsum("bhij,bhj->bhi", dS, k[:, t])
            db[:, t] = (du * e).sum(-1)
            de = beta[:, t, :, None] * du
            dv[:, t] = de
            dk[:, t] = (torch.einsum("bhij,bhi->bhj", dS, beta[:, t, :, None] * e)
                        - torch.einsum("bhij,bhi->bhj", A, de))
            dS -= torch.einsum("bhi,bhj->bhij", de, k[:, t])
            dg[:, t] = (dS * A).sum((-1, -2))
            dS *= alpha[:, t, :, None, None]
    return y, S, dq, dk, dv, dg, db, dS


def _exact_rule(case, s):
    H, Hk, train = case["H"], case["Hk"], case["op"] == "train"
    spread = lambda x: x.double().repeat_interleave(H // Hk, 2)  # noqa: E731
    together = lambda x: x.reshape(*x.shape[:2], Hk, H // Hk, -1).sum(3)  # noqa: E731
    q, k, v, g, beta = spread(s["q"]), spread(s["k"]), s["v"].double(), s["g"].double(), s["beta"].double()
    count = case["packed"] or case["B"]
    S = torch.zeros(count, H, case["N"], case["N"], device="cuda", dtype=torch.float64) \
        if s["state"] is None else s["state"].double()
    dy = s["dy"].double() if train else None
    dS = s["dstate"].double() if train and s["dstate"] is not None else None
    if s["offsets"] is None:
        got = _exact_sequence(q, k, v, g, beta, S, s["scale"], dy, dS)
    else:
        off, parts = s["offsets"].tolist(), []
        for i in range(count):
            r = slice(off[i], off[i + 1])
            parts.append(_exact_sequence(q[:, r], k[:, r], v[:, r], g[:, r], beta[:, r], S[i:i + 1].clone(),
                                         s["scale"], None if dy is None else dy[:, r],
                                         None if dS is None else dS[i:i + 1]))
        by_token = {0, 2, 3, 4, 5, 6}
        got = [torch.cat(x, 1 if j in by_token else 0) for j, x in enumerate(zip(*parts))]
    if not train:
        return got[0], got[1]
    out = {"y": got[0], "state": got[1], "dq": together(got[2]), "dk": together(got[3]),
           "dv": got[4], "dg": got[5], "dbeta": got[6]}
    if s["state"] is not None:
        out["dstate"] = got[7]
    return out


def _exact_decode(case, s):
    y, state = torch.zeros(s["y"].shape, device="cuda", dtype=torch.float64), s["state"].double()
    rows = [i for i in range(case["n"])] if s["slots"] is None else \
        [i for i, p in enumerate(s["slots"].tolist()) if p >= 0]
    at = rows if s["slots"] is None else [s["slots"].tolist()[i] for i in rows]
    spread = lambda x: x[rows].double().repeat_interleave(case["H"] // case["Hk"], 1)[:, None]  # noqa: E731
    got, last = _exact_sequence(spread(s["q"]), spread(s["k"]), s["v"][rows].double()[:, None],
                                s["g"][rows].double()[:, None], s["beta"][rows].double()[:, None],
                                state[at], s["scale"])
    y[rows], state[at] = got[:, 0], last
    return y, state


def _exact_norm(case, s):
    d = {n: None if s[n] is None else s[n].double() for n in _NORM}
    R, C, G = case["R"], case["C"], case["group"]
    groups = lambda x: x.reshape(R, C // G, G)  # noqa: E731
    r1 = 1.0 / torch.sqrt((groups(d["h"]) ** 2).sum(-1, keepdim=True) / G + _EPS)
    hn = (groups(d["h"]) * r1).reshape(R, C)
    sig = None if d["gate"] is None else 1.0 / (1.0 + torch.exp(-d["gate"]))
    act = 1.0 if sig is None else sig * d["gate"] if case["gate"] == "silu" else sig
    m = act * hn * d["weight"]
    out = m if d["x"] is None else d["x"] + d["scale"] * m
    got, xn = {"out": out}, None
    if d["next_weight"] is not None:
        r2 = 1.0 / torch.sqrt((out ** 2).sum(-1, keepdim=True) / C + _EPS)
        xn = out * r2
        got["y"] = xn * d["next_weight"]
    if case["op"] == "norm":
        return got
    dout = s["dout"].double()
    if xn is not None:
        dy = s["dy"].double()
        got["dnext_weight"] = (dy * xn).sum(0)
        dn = dy * d["next_weight"]
        dout = dout + r2 * (dn - xn * (dn * xn).sum(-1, keepdim=True) / C)
    dm = dout
    if d["x"] is not None:
        got["dx"] = dout
        got["dscale"] = (dout * m).sum(0)
        dm = dout * d["scale"]
    if sig is not None:
        slope = sig * (1.0 - sig)
        got["dgate"] = dm * hn * d["weight"] * (sig + d["gate"] * slope if case["gate"] == "silu" else slope)
    da = dm * act
    got["dweight"] = (da * hn).sum(0)
    dn = groups(da * d["weight"])
    got["dh"] = (r1 * (dn - groups(hn) * (dn * groups(hn)).sum(-1, keepdim=True) / G)).reshape(R, C)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return _exact_rule(case, s)
