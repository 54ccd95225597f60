"""Cases for the gated linear recurrence and the q / k norm with rotation.

Two operators and the forms a user runs them in:

* the gated linear recurrence ``S_t = e^{g_t} S_{t-1} + k_t^T v_t``,
  ``o_t = q_t S_t`` per head: forward over a sequence (``fwd``), forward and
  backward (``train``) and one token with the state updated in place
  (``step``);
* the per-head norm of q and k with the rotation by position in the same pass
  (``qk``), and the same with its backward (``qk_train``).

``run`` computes them in plain torch operations where ``own`` is false, and
through the library's entry points where it is true.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128      # rows of a chunk of the plain form
WIPE = -200.0    # e^-200 is zero in 32 bits: stands for a log decay of -inf


def _rec(name, op, dtype, B, H, Hqk, L, dk, dv, s0=False, docs=0):
    c = {"op": op, "dtype": dtype, "B": B, "H": H, "Hqk": Hqk, "L": L, "dk": dk, "dv": dv,
         "s0": s0, "docs": docs}
    return {"name": name, **c} if name else c


def _step(name, dtype, B, H, Hqk, dk, dv):
    c = {"op": "step", "dtype": dtype, "B": B, "H": H, "Hqk": Hqk, "dk": dk, "dv": dv}
    return {"name": name, **c} if name else c


def _qk(name, op, dtype, B, Hq, Hk, L, d, drot, axes, interleaved):
    c = {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "L": L, "d": d, "drot": drot,
         "axes": axes, "interleaved": interleaved}
    return {"name": name, **c} if name else c


def listed():
    return [
        # A prompt of a small model: four requests of equal length.
        _rec("fwd_prompt", "fwd", "bf16", 4, 12, 12, 2048, 64, 64),
        # A later piece of a prompt: from a state, q and k shared by four value
        # heads, several documents in a row, a length that fits no tile.
        _rec("fwd_groups_ragged", "fwd", "bf16", 3, 16, 4, 1777, 128, 64, s0=True, docs=5),
        # A whole long context in one call.
        _rec("fwd_long", "fwd", "bf16", 1, 32, 32, 65536, 128, 128),
        # The smallest training step, in 32 bits: a check of a model's gradients.
        _rec("train_f32_small", "train", "f32", 1, 2, 2, 256, 64, 64, s0=True),
        # Training on packed documents with shared q and k heads.
        _rec("train_groups_ragged", "train", "bf16", 2, 12, 4, 1501, 64, 128, s0=True, docs=7),
        # Training with the state carried from the piece before (truncated in time).
        _rec("train_mid", "train", "bf16", 2, 16, 16, 8192, 128, 128, s0=True),
        # Training on a long context.
        _rec("train_long", "train", "bf16", 1, 32, 32, 65536, 128, 128),
        # One request's next token: latency counts.
        _step("step_one", "bf16", 1, 32, 32, 128, 128),
        # The next token of a full batch: the states' bytes count.
        _step("step_batch", "bf16", 256, 32, 32, 128, 128),
        # q and k of a full batch's next token.
        _qk("qk_one_token", "qk", "bf16", 256, 32, 8, 1, 128, 128, 1, False),
        # q and k of a long context, out of the fused projection.
        _qk("qk_long", "qk", "bf16", 1, 32, 32, 65536, 128, 128, 1, False),
        # Training on text, pictures and video: time, height and width.
        _qk("qk_train_axes", "qk_train", "bf16", 2, 16, 4, 4097, 128, 128, 3, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "step", "qk", "qk_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("fwd", "train"):
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        Hqk, group = _log(rng, 1, 32), rng.choice([1, 1, 2, 3, 4])
        B = _log(rng, 1, 8)
        # At most a quarter of the long context's tokens x heads, so that 32
        # bits and shared heads cost no more than it either.
        most = max(1, 524288 // (B * Hqk * group) // (2 if dtype == "f32" else 1))
        L = _log(rng, 1, min(32768, most))
        return _rec("", op, dtype, B, Hqk * group, Hqk, L, dk, dv, s0=rng.random() < 0.5,
                    docs=rng.choice([0, 0, 1, 3]))
    if op == "step":
        Hqk, group = _log(rng, 1, 32), rng.choice([1, 1, 2, 4])
        B = _log(rng, 1, max(1, 4096 // (Hqk * group)))
        return _step("", dtype, B, Hqk * group, Hqk, rng.choice([64, 128]), rng.choice([64, 128]))
    d = rng.choice([64, 128])
    Hk, group = _log(rng, 1, 16), rng.choice([1, 2, 4, 7])
    B = _log(rng, 1, 64)
    L = _log(rng, 1, min(32768, max(1, 1048576 // (B * Hk * (group + 1)))))
    drot = rng.choice([d, d, d // 2, 48])
    return _qk("", op, dtype, B, Hk * group, Hk, L, d, drot, rng.choice([1, 1, 2, 3]),
               rng.random() < 0.5)


def sections_of(case):
    """Pairs per position axis: the whole rotation, halves, or a quarter and two three-eighths."""
    n = case["drot"] // 2
    if case["axes"] == 1:
        return [n]
    if case["axes"] == 2:
        return [n // 2, n - n // 2]
    return [n // 4, (n - n // 4) // 2, n - n // 4 - (n - n // 4) // 2]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return (x * std).to(dtype)

    s = dict(case)
    if case["op"] in ("fwd", "train", "step"):
        B, H, Hqk, dk, dv = (case[n] for n in ("B", "H", "Hqk", "dk", "dv"))
        L = (case["L"],) if "L" in case else ()
        s["q"] = normal(B, Hqk, *L, dk)
        s["k"] = normal(B, Hqk, *L, dk, std=dk ** -0.5)
        s["v"] = normal(B, H, *L, dv)
        # A decay of sigmoid(N(3, 1)), as a gate's projection gives.
        g = torch.nn.functional.logsigmoid(normal(B, H, *L, dtype=torch.float32) + 3.0)
        if case.get("docs") and case["L"] > 1:
            # Documents packed in a row: the first token of each forgets the one before.
            first = torch.randint(1, case["L"], (B, case["docs"]), generator=gen, device=DEV)
            start = torch.zeros(B, case["L"], dtype=torch.bool, device=DEV).scatter_(1, first, True)
            g = g.masked_fill(start[:, None], -math.inf)
        s["g"] = g.contiguous()
        state = normal(B, H, dk, dv, std=0.1, dtype=torch.float32)
        if case["op"] == "step":
            s["S"] = state
        else:
            s["S0"] = state if case["s0"] else None
        if case["op"] == "train":
            s["dO"] = normal(B, H, *L, dv)
            s["dS"] = normal(B, H, dk, dv, dtype=torch.float32)
        return s
    B, Hq, Hk, L, d = (case[n] for n in ("B", "Hq", "Hk", "L", "d"))
    # q and k lie in the fused projection's rows, [B, L, (q heads, k heads, v heads) d].
    proj = normal(B, L, Hq + 2 * Hk, d)
    s["q_raw"] = proj[:, :, :Hq].transpose(1, 2)
    s["k_raw"] = proj[:, :, Hq:Hq + Hk].transpose(1, 2)
    s["q_weight"] = 1.0 + normal(d, std=0.2, dtype=torch.float32)
    s["k_weight"] = 1.0 + normal(d, std=0.2, dtype=torch.float32)
    n = case["drot"] // 2
    s["inv_freq"] = (10000.0 ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n)).float()
    # One axis: every request at a place of its own in a long context.  Several:
    # frames, rows and columns of a picture's patches behind it.
    far = torch.randint(0, 1 << 20, (B, 1), generator=gen, device=DEV)
    at = torch.arange(L, device=DEV)
    if case["axes"] == 1:
        p = (far + at)[None]
    else:
        p = torch.stack([far + at // 1024, far + at // 32 % 32, far + at % 32][:case["axes"]])
    s["positions"] = p.to(torch.int32).contiguous()
    s["sections"] = sections_of(case)
    if case["op"] == "qk_train":
        s["dq_hat"] = normal(B, Hq, L, d)
        s["dk_hat"] = normal(B, Hk, L, d)
    return s


# ---- the recurrence in plain operations --------------------------------------------------


def _pieces(x, fill=0.0):
    """[B, H, L, ...] -> [B, H, chunks, CHUNK, ...], the last chunk filled up."""
    L = x.shape[2]
    n = -(-L // CHUNK)
    if n * CHUNK != L:
        rest = x.new_full((*x.shape[:2], n * CHUNK - L, *x.shape[3:]), fill)
        x = torch.cat([x, rest], 2)
    return x.reshape(*x.shape[:2], n, CHUNK, *x.shape[3:])


def _decays(g):
    """Factors of the chunked form: of pairs within a chunk, from a chunk's
    start to a row, from a row to its chunk's end, and between chunks."""
    g = _pieces(g.double().clamp_min(WIPE))
    G = g.cumsum(-1)
    row = torch.arange(CHUNK, device=g.device)
    pair = (G[..., :, None] - G[..., None, :]).masked_fill(row[:, None] < row, -math.inf).exp()
    # T[c]: log decay of everything before chunk c, for c = 0 .. chunks.
    T = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))
    return pair.float(), G.exp().float(), (G[..., -1:] - G).exp().float(), T


def _entering(U, T, S0):
    """States entering each chunk, and after the last one, from what each chunk adds."""
    n = U.shape[2]
    c = torch.arange(n + 1, device=U.device)
    M = (T[..., :, None] - T[..., None, 1:]).masked_fill(c[:, None] <= c[:n], -math.inf).exp().float()
    S = (M @ U.flatten(3)).unflatten(3, U.shape[3:])
    return S if S0 is None else S + T.exp().float()[..., None, None] * S0[:, :, None]


def _leaving(U, T, dS):
    """Gradients of the states that leave each chunk, and (first) of the state before the first."""
    n = U.shape[2]
    c = torch.arange(n + 1, device=U.device)
    M = (T[..., None, :-1] - T[..., :, None]).masked_fill(c[:, None] > c[:n], -math.inf).exp().float()
    return (M @ U.flatten(3)).unflatten(3, U.shape[3:]) \
        + (T[..., -1:] - T).exp().float()[..., None, None] * dS[:, :, None]


def _heads(x, H):
    return x.float().repeat_interleave(H // x.shape[1], 1)


def _rows(x, L):
    return x.flatten(2, 3)[:, :, :L]


def _plain_forward(s):
    H, L = s["v"].shape[1], s["v"].shape[2]
    q, k, v = _pieces(_heads(s["q"], H)), _pieces(_heads(s["k"], H)), _pieces(s["v"].float())
    pair, down, up, T = _decays(s["g"])
    U = (k * up[..., None]).transpose(-1, -2).contiguous() @ v
    S = _entering(U, T, s["S0"])
    o = (q @ k.transpose(-1, -2).contiguous() * pair) @ v + (q @ S[:, :, :-1]) * down[..., None]
    return _rows(o, L).to(s["v"].dtype), S[:, :, -1].contiguous()


def _plain_backward(s):
    B, H, L, dv_ = s["v"].shape
    Hqk, t = s["q"].shape[1], s["v"].dtype
    q, k, v = _pieces(_heads(s["q"], H)), _pieces(_heads(s["k"], H)), _pieces(s["v"].float())
    dO = _pieces(s["dO"].float())
    pair, down, up, T = _decays(s["g"])
    turned = lambda x: x.transpose(-1, -2).contiguous()  # noqa: E731
    S = _entering(turned(k * up[..., None]) @ v, T, s["S0"])[:, :, :-1]
    X = _leaving(turned(q * down[..., None]) @ dO, T, s["dS"])
    dS0, X = X[:, :, 0].contiguous(), X[:, :, 1:]
    qk, dP = q @ turned(k), (dO @ turned(v)) * pair
    both = qk * dP
    q_in, k_out = (dO @ turned(S)) * down[..., None], (v @ turned(X)) * up[..., None]
    dq, dk = dP @ k + q_in, turned(dP) @ q + k_out
    dv = turned(qk * pair) @ dO + (k @ X) * up[..., None]
    # e^{g_t} <S_{t-1}, dS_t>: what the rows from t on read of what was there
    # before t, and what the state that leaves the chunk holds of it.
    read = ((q * q_in).sum(-1) + both.sum(-1) - both.sum(-2)).double()
    kept = (k * k_out).sum(-1).double()
    through = (T.diff(dim=-1).exp() * (S * X).sum((-1, -2)).double())[..., None]
    dg = read.flip(-1).cumsum(-1).flip(-1) + kept.cumsum(-1) - kept + through
    dg = _rows(dg, L).masked_fill(s["g"] <= WIPE, 0.0).float()
    shared = lambda x: _rows(x, L).unflatten(1, (Hqk, H // Hqk)).sum(2).to(t)  # noqa: E731
    return shared(dq), shared(dk), _rows(dv, L).to(t), dg, dS0


def _plain_step(s):
    H = s["v"].shape[1]
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), s["v"].float()
    s["S"].mul_(s["g"].exp()[..., None, None]).add_(k[..., :, None] * v[..., None, :])
    return (q[..., :, None] * s["S"]).sum(-2).to(s["v"].dtype), s["S"]


# ---- norm and rotation in plain operations -------------------------------------------------

EPS = 1e-6


def _angles(s):
    p = s["positions"].double().repeat_interleave(
        torch.tensor(s["sections"], device=DEV), 0)                    # [pairs, B, L]
    a = p * s["inv_freq"].double()[:, None, None]
    a = a.permute(1, 2, 0)[:, None]                                    # [B, 1, L, pairs]
    return a.cos().float(), a.sin().float()


def _turn(x, cos, sin, s):
    """Rotates the pairs of the first drot elements by the angles."""
    n = s["drot"]
    r, rest = x[..., :n], x[..., n:]
    if s["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :n // 2], r[..., n // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, rest], -1)


def _plain_qk(s):
    cos, sin = _angles(s)
    out = []
    for n in ("q", "k"):
        x = s[n + "_raw"].float()
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s[n + "_weight"]
        out.append(_turn(x, cos, sin, s).to(s[n + "_raw"].dtype))
    return out


def _plain_qk_backward(s):
    cos, sin = _angles(s)
    dx, dw = [], []
    for n in ("q", "k"):
        x, w = s[n + "_raw"].float(), s[n + "_weight"]
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        dn = _turn(s["d" + n + "_hat"].float(), cos, -sin, s)
        xh = x * r
        dw.append((dn * xh).double().sum((0, 1, 2)).float())
        dn = dn * w
        dx.append((r * (dn - xh * (xh * dn).mean(-1, keepdim=True))).to(s[n + "_raw"].dtype))
    return dx + dw


# ---- one pass ------------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "fwd":
        return _plain_forward(s)
    if s["op"] == "train":
        return (*_plain_forward(s), *_plain_backward(s))
    if s["op"] == "step":
        return _plain_step(s)
    if s["op"] == "qk":
        return _plain_qk(s)
    return (*_plain_qk(s), *_plain_qk_backward(s))


def _run_own(s):
    from deltanet_delta_rule_chunk_amd import binding

    if s["op"] == "step":
        o = binding.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"],
                                       out_dtype=s["v"].dtype)
        return o, s["S"]
    if s["op"] in ("fwd", "train"):
        out = binding.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"],
                                       out_dtype=s["v"].dtype)
        if s["op"] == "fwd":
            return out
        return (*out, *binding.linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["S0"], s["dO"],
                                                s["dS"]))
    how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], sections=s["sections"], eps=EPS,
               interleaved=s["interleaved"])
    out = binding.qk_norm_rope(s["q_raw"], s["k_raw"], s["positions"], s["inv_freq"], **how)
    if s["op"] == "qk":
        return out
    return (*out, *binding.qk_norm_rope_bwd(s["q_raw"], s["k_raw"], s["positions"], s["inv_freq"],
                                            s["dq_hat"], s["dk_hat"], **how))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("fwd", "train", "step"):
        B, H, Hqk, dk, dv, L = (case.get(n, 1) for n in ("B", "H", "Hqk", "dk", "dv", "L"))
        qk, v, state = B * Hqk * L * dk * size, B * H * L * dv * size, B * H * dk * dv * 4
        g, products = B * H * L * 4, 2 * B * H * L * dk * dv
        if case["op"] == "step":
            return {"bytes": 2 * qk + 2 * v + g + 2 * state, "flops": 2 * products}
        s0 = state if case["s0"] else 0
        w = {"bytes": 2 * qk + 2 * v + g + s0 + state, "flops": 2 * products}
        if case["op"] == "train":
            # The backward reads q, k, v, dO, the decays and both states again
            # and writes the gradients of each input.
            w = {"bytes": w["bytes"] + 4 * qk + 3 * v + 2 * g + s0 + 2 * state,
                 "flops": w["flops"] + 5 * products}
        return w
    B, Hq, Hk, L, d = (case[n] for n in ("B", "Hq", "Hk", "L", "d"))
    rows, pos = B * (Hq + Hk) * L * d * size, 4 * case["axes"] * B * L
    if case["op"] == "qk":
        return {"bytes": 2 * rows + pos, "flops": 7 * B * (Hq + Hk) * L * d}
    return {"bytes": 5 * rows + 2 * pos, "flops": 22 * B * (Hq + Hk) * L * d}


# ---- in 64 bits, from the definitions -------------------------------------------------------


def _token_by_token(s):
    """The recurrence and its reverse as loops over tokens."""
    B, H, L, dv = s["v"].shape
    Hqk, dk = s["q"].shape[1], s["q"].shape[3]
    t_first = lambda x: x.double().expand(B, H, L, -1).permute(2, 0, 1, 3).contiguous()  # noqa: E731
    every = lambda x: x[:, :, None].expand(B, Hqk, H // Hqk, L, dk).reshape(B, H, L, dk)  # noqa: E731
    q, k, v = t_first(every(s["q"])), t_first(every(s["k"])), t_first(s["v"])
    a = s["g"].double().exp().permute(2, 0, 1)[..., None, None].contiguous()
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=q.device)
    if s["S0"] is not None:
        S += s["S0"].double()
    train = "dO" in s
    dO = t_first(s["dO"]) if train else None
    o, dq = torch.empty_like(v), torch.empty_like(q) if train else None
    for t in range(L):
        S.mul_(a[t]).addcmul_(k[t, ..., None], v[t, :, :, None, :])
        torch.sum(q[t, ..., None] * S, -2, out=o[t])
        if train:
            torch.sum(dO[t, :, :, None, :] * S, -1, out=dq[t])
    b_first = lambda x: x.permute(1, 2, 0, 3)  # noqa: E731
    if not train:
        return b_first(o), S
    R = s["dS"].double().clone()
    # <S_t, dS_t> after the last token; from there back by what each token reads and adds.
    held = (S * R).sum((-1, -2))
    dk_, dv_, dg = torch.empty_like(k), torch.empty_like(v), torch.empty_like(a[..., 0, 0])
    for t in range(L - 1, -1, -1):
        R.addcmul_(q[t, ..., None], dO[t, :, :, None, :])
        torch.sum(v[t, :, :, None, :] * R, -1, out=dk_[t])
        torch.sum(k[t, ..., None] * R, -2, out=dv_[t])
        R.mul_(a[t])
    step = (q * dq).sum(-1) - (k * dk_).sum(-1)
    dg = step.flip(0).cumsum(0).flip(0) + held
    dg[a[..., 0, 0] == 0] = 0
    shared = lambda x: b_first(x).reshape(B, Hqk, H // Hqk, L, dk).sum(2)  # noqa: E731
    return b_first(o), S, shared(dq), shared(dk_), b_first(dv_), dg.permute(1, 2, 0), R


def _as_complex(x, s):
    n = s["drot"]
    if s["interleaved"]:
        return torch.view_as_complex(x[..., :n].unflatten(-1, (n // 2, 2)).contiguous())
    return torch.complex(x[..., :n // 2].contiguous(), x[..., n // 2:n].contiguous())


def _norm_and_rotation(x, w, s):
    norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    y = x / torch.sqrt(norm ** 2 / x.shape[-1] + EPS) * w
    axis = torch.cat([torch.full((c,), i) for i, c in enumerate(s["sections"])]).to(DEV)
    angle = s["positions"].double()[axis].movedim(0, -1)[:, None] * s["inv_freq"].double()
    z = _as_complex(y, s) * torch.polar(torch.ones_like(angle), angle)
    r = torch.view_as_real(z).flatten(-2) if s["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([r, y[..., s["drot"]:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "train"):
        with torch.no_grad():
            return _token_by_token(s)
    if case["op"] == "step":
        one = {n: s[n][:, :, None] for n in ("q", "k", "v", "g")}
        o, S = _token_by_token({**one, "S0": s["S"]})
        return o[:, :, 0], S
    x = [s[n + "_raw"].double().requires_grad_() for n in ("q", "k")]
    w = [s[n + "_weight"].double().requires_grad_() for n in ("q", "k")]
    y = [_norm_and_rotation(a, b, s) for a, b in zip(x, w)]
    if case["op"] == "qk":
        return [a.detach() for a in y]
    d = torch.autograd.grad(y, x + w, [s["dq_hat"].double(), s["dk_hat"].double()])
    return [a.detach() for a in y] + list(d)
