"""Cases for a state space layer's operators: the short causal convolution, the
selective state space scan, and the root-mean-square norm with the residual's
addition.

* convolution of the last K tokens of each channel, ``y_t = silu(b + sum_j w_j
  x_{t-K+1+j})``: over a sequence (``conv``), with its gradient
  (``conv_train``), one token with the kept rows updated in place (``conv_step``);
* scan ``h_t = e^{dt_t A} h_{t-1} + dt_t u_t B_t``, ``y_t = (C_t h_t + D u_t)
  silu(z_t)`` with ``dt = softplus(raw + bias)``: ``scan``, ``scan_train``,
  ``scan_step``;
* ``total = x + residual``, ``y = total / rms(total) * weight``: ``norm``, with
  y in 8 bits and a scale for each token ``norm8``, with its gradient
  ``norm_train``.

Sequences come as a batch of equal ones, or packed in a row (``seqs`` > 0), with
``cu_seqlens`` where each begins and ends; rows behind the last one (``pad``) give
zeros.

``run`` computes them in plain torch operations where ``own`` is false, and
through the library's entry points where it is true.
"""

import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
E4M3_MAX = 448.0


def _conv(name, op, dtype, B, L, D, K, seqs=0, pad=0, state=False, bias=True, silu=True):
    c = {"op": op, "dtype": dtype, "B": B, "L": L, "D": D, "K": K, "seqs": seqs, "pad": pad,
         "state": state, "bias": bias, "silu": silu}
    return {"name": name, **c} if name else c


def _scan(name, op, dtype, B, L, D, N, seqs=0, pad=0, state=False, gate=True):
    c = {"op": op, "dtype": dtype, "B": B, "L": L, "D": D, "N": N, "seqs": seqs, "pad": pad,
         "state": state, "gate": gate}
    return {"name": name, **c} if name else c


def _norm(name, op, dtype, rows, D, wide=False):
    """``wide``: the residual stream is kept in 32 bits."""
    c = {"op": op, "dtype": dtype, "rows": rows, "D": D, "wide": wide}
    return {"name": name, **c} if name else c


def listed():
    return [
        # q, k and v of 12 heads of 64 in one convolution: prompts of different
        # lengths in a row, each going on from its own last tokens.
        _conv("conv_prompts_ragged", "conv", "bf16", 1, 6001, 2304, 4, seqs=7, pad=47, state=True),
        # Training on a long context, the channels of 32 heads of 128.
        _conv("conv_train_long", "conv_train", "bf16", 1, 65536, 4096, 4),
        # The next token of a full batch.
        _conv("conv_step_batch", "conv_step", "bf16", 256, 1, 4096, 4, state=True),
        # A prompt of a small model: four requests of equal length.
        _scan("scan_prompt", "scan", "bf16", 4, 2048, 1536, 16),
        # A whole long context in one call.
        _scan("scan_long", "scan", "bf16", 1, 65536, 4096, 16),
        # Training on packed documents in 32 bits, a length that fits no tile.
        _scan("scan_train_ragged", "scan_train", "f32", 1, 1777, 768, 16, seqs=5, pad=23, state=True),
        # Training with the state carried from the piece before.
        _scan("scan_train_mid", "scan_train", "bf16", 2, 8192, 4096, 16, state=True),
        # One request's next token: latency counts.
        _scan("scan_step_one", "scan_step", "bf16", 1, 1, 4096, 16, state=True),
        # The next token of a full batch: the states' bytes count.
        _scan("scan_step_batch", "scan_step", "bf16", 256, 1, 4096, 16, state=True),
        # The norm in front of a full batch's next token.
        _norm("norm_one_token", "norm", "bf16", 256, 4096),
        # A long context's rows on the way into projections in 8 bits.
        _norm("norm8_long", "norm8", "bf16", 65536, 4096),
        # Training with the residual stream in 32 bits, rows of an odd number of pieces.
        _norm("norm_train_wide", "norm_train", "bf16", 16385, 2072, wide=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train",
                     "scan_step", "norm", "norm8", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = 8 * _log(rng, 2, 1024)
    if op.startswith("norm"):
        rows = _log(rng, 1, min(65536, (1 << 27) // D))
        return _norm("", op, dtype, rows, D, wide=rng.random() < 0.3)
    N = rng.choice([8, 16, 16, 16, 32])
    if op.endswith("step"):
        B = _log(rng, 1, min(1024, (1 << 20) // D))
        if op == "conv_step":
            return _conv("", op, dtype, B, 1, D, rng.choice([2, 3, 4, 4]), state=True,
                         bias=rng.random() < 0.7, silu=rng.random() < 0.7)
        return _scan("", op, dtype, B, 1, D, N, state=True, gate=rng.random() < 0.7)
    packed = rng.random() < 0.4
    B = 1 if packed else _log(rng, 1, 16)
    # Tokens x channels (x states) of a quarter of the longest listed case at most.
    most = (1 << 26) if op.startswith("conv") else (1 << 28 if op == "scan" else 1 << 27) // N
    L = _log(rng, 1, min(32768, max(1, most // (B * D))))
    seqs = _log(rng, 1, min(L, 40)) if packed else 0
    pad = rng.choice([0, 0, 5, 70]) if packed else 0
    state = rng.random() < 0.5
    if op.startswith("conv"):
        return _conv("", op, dtype, B, L + pad, D, rng.choice([2, 3, 4, 4]), seqs, pad, state,
                     bias=rng.random() < 0.7, silu=rng.random() < 0.7)
    return _scan("", op, dtype, B, L + pad, D, N, seqs, pad, state, gate=rng.random() < 0.7)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return x.mul_(std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV, dtype=torch.float32)

    s = dict(case)
    D = case["D"]
    if case["op"].startswith("norm"):
        wide = torch.float32 if case["wide"] else t
        s["x"] = normal(case["rows"], D)
        # The stream has grown over the layers before.
        s["residual"] = normal(case["rows"], D, std=4.0, dtype=wide)
        s["weight"] = 1.0 + normal(D, std=0.2, dtype=torch.float32)
        if case["op"] == "norm_train":
            s["dy"] = normal(case["rows"], D)
            s["dtotal"] = normal(case["rows"], D, dtype=wide)
        return s
    B, L = case["B"], case["L"]
    step = case["op"].endswith("step")
    tok = (B,) if step else (B, L)
    n = case["seqs"] or B  # sequences
    s["cu"] = None
    if case["seqs"]:
        # Cuts anywhere: a sequence may be empty.
        cuts = torch.randint(0, L - case["pad"] + 1, (n + 1,), generator=gen, device=DEV)
        cuts[0], cuts[-1] = 0, L - case["pad"]
        s["cu"] = cuts.sort().values.to(torch.int32)
    # The input and the gate lie side by side in the in-projection's rows.
    rows = normal(*tok, 2 * D)
    if case["op"].startswith("conv"):
        K = case["K"]
        s["x"] = rows[..., :D]
        s["weight"] = (uniform(D, K) * 2 - 1) * K ** -0.5
        s["bias"] = (uniform(D) * 2 - 1) * K ** -0.5 if case["bias"] else None
        s["state"] = normal(n, K - 1, D) if case["state"] else None
        if case["op"] == "conv_train":
            s["dy"] = normal(B, L, D)
            s["dstate"] = normal(n, K - 1, D)
        return s
    N = case["N"]
    u = normal(*tok, D, dtype=torch.float32)
    s["u"] = (u * torch.sigmoid(u)).to(t)
    s["z"] = rows[..., D:] if case["gate"] else None
    s["dt"] = normal(*tok, D, std=0.5)
    # Steps from a thousandth to a tenth, rates of 1 to N and what training made of them.
    start = torch.exp(uniform(D) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = start + torch.log(-torch.expm1(-start))
    rate = torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
    s["A"] = -(rate * torch.exp(normal(D, N, std=0.1, dtype=torch.float32)))
    # B and C lie behind the step's own low-rank part in a projection's rows.
    rank = 8 * max(1, D // 128)
    proj = normal(*tok, rank + 2 * N)
    s["B_"], s["C_"] = proj[..., rank:rank + N], proj[..., rank + N:]
    s["D_"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
    s["state"] = normal(n, D, N, std=0.1, dtype=torch.float32) if case["state"] else None
    if case["op"] == "scan_train":
        s["dy"] = normal(B, L, D)
        s["dstate"] = normal(n, D, N, dtype=torch.float32)
    return s


# ---- where the sequences lie ---------------------------------------------------------------


def _places(s):
    """For every token of a row [B, L]: its sequence, its sequence's first token, and
    whether it is in one; for every sequence [n]: its first token and the one
    behind its last."""
    B, L = s["B"], s["L"]
    at = torch.arange(L, device=DEV)
    if s["cu"] is None:
        seq = torch.arange(B, device=DEV)[:, None].expand(B, L)
        ends = torch.zeros(B, dtype=torch.long, device=DEV), torch.full((B,), L, device=DEV)
        return seq, torch.zeros_like(seq), torch.ones_like(seq, dtype=torch.bool), *ends
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, at, right=True)[None] - 1
    inside = seq < len(cu) - 1
    seq = seq.clamp_max(len(cu) - 2)
    return seq, cu[seq], inside, cu[:-1], cu[1:]


def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


# ---- the convolution in plain operations ----------------------------------------------------


def _tap(s, back, seq, first, inside):
    """x `back` tokens earlier: in the sequence, in the rows kept from before it, or nothing."""
    x, state, L = s["x"], s["state"], s["L"]
    if s["cu"] is None:
        K = s["K"]
        front = x.new_zeros(x.shape[0], K - 1, s["D"]) if state is None else state
        return torch.cat([front, x], 1)[:, K - 1 - back:K - 1 - back + L].float()
    at = torch.arange(x.shape[1], device=DEV)[None] - back
    batch = torch.arange(x.shape[0], device=DEV)[:, None]
    own_rows = (at >= first) & inside
    v = torch.where(own_rows[..., None], x[batch, at.clamp_min(0)].float(), 0.0)
    if state is not None:
        kept = state.shape[1] + at - first
        before = (kept >= 0) & (at < first) & inside
        v = v + torch.where(before[..., None], state[seq, kept.clamp(0, state.shape[1] - 1)].float(), 0.0)
    return v


def _kept_rows(s, begin, end):
    """The K - 1 rows behind which each sequence ends, and where they come from."""
    K = s["K"]
    n = len(begin)
    batch = torch.arange(n, device=DEV)[:, None] if s["cu"] is None else 0
    at = end[:, None] - (K - 1) + torch.arange(K - 1, device=DEV)          # [n, K - 1]
    inside = at >= begin[:, None]
    v = torch.where(inside[..., None], s["x"][batch, at.clamp(0, s["L"] - 1)], 0)
    if s["state"] is not None:
        back = (K - 1 + at - begin[:, None]).clamp(0, K - 2)
        v = torch.where(inside[..., None], v, s["state"][torch.arange(n, device=DEV)[:, None], back])
    return v


def _pre(s, seq, first, inside):
    K = s["K"]
    p = sum(s["weight"][:, K - 1 - b] * _tap(s, b, seq, first, inside) for b in range(K))
    return p if s["bias"] is None else p + s["bias"]


def _plain_conv(s):
    seq, first, inside, begin, end = _places(s)
    p = _pre(s, seq, first, inside)
    y = torch.where(inside[..., None], _silu(p) if s["silu"] else p, 0.0)
    return y.to(s["x"].dtype), _kept_rows(s, begin, end)


def _plain_conv_backward(s):
    seq, first, inside, begin, end = _places(s)
    K, L, t = s["K"], s["L"], s["x"].dtype
    g = s["dy"].float()
    if s["silu"]:
        g = g * _dsilu(_pre(s, seq, first, inside))
    g = torch.where(inside[..., None], g, 0.0)
    dx, dw = torch.zeros_like(g), []
    ds = torch.zeros(len(begin), K - 1, s["D"], device=DEV)
    batch = torch.arange(s["B"], device=DEV)[:, None]
    at = torch.arange(L, device=DEV)[None].expand(s["B"], L)
    n = torch.arange(len(begin), device=DEV)
    for b in range(K):
        w = s["weight"][:, K - 1 - b]
        dw.append((g * _tap(s, b, seq, first, inside)).double().sum((0, 1)).float())
        # The token `b` later, where it is of the same sequence.
        if s["cu"] is None:
            dx[:, :max(L - b, 0)] += g[:, b:] * w
        else:
            later = (at + b).clamp_max(L - 1)
            same = (at + b < L) & inside & (first[batch, later] == first) & inside[batch, later]
            dx += torch.where(same[..., None], g[batch, later], 0.0) * w
        for i in range(b):  # the sequence's token i reads the kept row K - 1 + i - b
            has = (end - begin > i)[:, None]
            rows = g[n if s["cu"] is None else 0, (begin + i).clamp_max(L - 1)]
            ds[:, K - 1 + i - b] += torch.where(has, rows, 0.0) * w
    # What the kept rows behind the end are of the sequence, or of the rows before it.
    for j in range(K - 1):
        place = end - (K - 1) + j
        row = s["dstate"][:, j].float()
        of_x = (place >= begin)[:, None]
        dx.index_put_((n if s["cu"] is None else torch.zeros_like(n), place.clamp(0, L - 1)),
                      torch.where(of_x, row, 0.0), accumulate=True)
        ds.index_put_((n, (K - 1 + place - begin).clamp(0, K - 2)), torch.where(of_x, 0.0, row), accumulate=True)
    db = None if s["bias"] is None else g.double().sum((0, 1)).float()
    return dx.to(t), torch.stack(dw[::-1], -1), db, ds.to(t) if s["state"] is not None else None


def _plain_conv_step(s):
    p = (torch.cat([s["state"], s["x"][:, None]], 1).float() * s["weight"].t()).sum(1)
    p = p if s["bias"] is None else p + s["bias"]
    s["state"].copy_(torch.cat([s["state"][:, 1:], s["x"][:, None]], 1))
    return (_silu(p) if s["silu"] else p).to(s["x"].dtype), s["state"]


# ---- the scan in plain operations -----------------------------------------------------------

CHUNK = 64  # tokens whose states are formed one after the other, for all chunks at once


def _softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


def _chunks(x, fill=0.0):
    """[B, L, ...] -> [CHUNK, B, chunks, ...], the last chunk filled up."""
    B, L = x.shape[:2]
    n = -(-L // CHUNK)
    if n * CHUNK != L:
        x = torch.cat([x, x.new_full((B, n * CHUNK - L, *x.shape[2:]), fill)], 1)
    return x.unflatten(1, (n, CHUNK)).movedim(2, 0)


def _unchunk(parts, L):
    return torch.stack(parts, 2).flatten(1, 2)[:, :L]


def _scan_inputs(s):
    """The recurrence's parts in 32 bits, in chunks: steps, what they write, and the
    rows that begin or lie outside a sequence."""
    seq, first, inside, begin, end = _places(s)
    raw = s["dt"].float() + s["dt_bias"]
    u = s["u"].float()
    dt = torch.where(inside[..., None], _softplus(raw), 0.0)
    starts = (torch.arange(s["L"], device=DEV)[None] == first) & inside
    p = {"dt": dt, "du": dt * u, "B": s["B_"].float(), "C": s["C_"].float(),
         "keep": torch.where(starts, 0.0, 1.0), "seq": seq, "starts": starts}
    p = {n: _chunks(v, 1.0 if n == "keep" else 0) for n, v in p.items()}
    return p, (raw, u, inside, begin, end)


def _decay(p, i, A):
    """e^{dt A} of token i of each chunk [B, chunks, D, N]; nothing of what came before at a start."""
    return torch.exp(p["dt"][i][..., None] * A) * p["keep"][i][..., None, None]


def _written(p, i, s):
    x = p["du"][i][..., None] * p["B"][i][..., None, :]
    if s["state"] is not None:
        # The sequence's first token also takes in the state it comes with.
        a = torch.exp(p["dt"][i][..., None] * s["A"]) * s["state"][p["seq"][i]]
        x = x + torch.where(p["starts"][i][..., None, None], a, 0.0)
    return x


def _before_chunks(added, passed, start=None):
    """States in front of every chunk from what the chunks add and pass on."""
    h = torch.zeros_like(added[:, 0]) if start is None else start
    out = []
    for c in range(added.shape[1]):
        out.append(h)
        h = passed[:, c] * h + added[:, c]
    return torch.stack(out, 1), h


def _states(s, p):
    """State in front of every chunk."""
    h, P = 0.0, 1.0
    for i in range(CHUNK):
        a = _decay(p, i, s["A"])
        h, P = a * h + _written(p, i, s), a * P
    return _before_chunks(h, P)[0]


def _plain_scan(s, keep=False):
    p, (raw, u, inside, begin, end) = _scan_inputs(s)
    h, y, kept, ends = _states(s, p), [], [], []
    n = len(begin)
    batch = torch.arange(n, device=DEV) if s["cu"] is None else torch.zeros(n, dtype=torch.long, device=DEV)
    last = (end - 1).clamp_min(0)
    final = torch.zeros(n, s["D"], s["N"], device=DEV) if s["state"] is None else s["state"].clone()
    for i in range(CHUNK):
        if keep:
            kept.append(h)
        h = _decay(p, i, s["A"]) * h + _written(p, i, s)
        y.append((h * p["C"][i][..., None, :]).sum(-1))
        here = ((last % CHUNK == i) & (end > begin))[:, None, None]
        final = torch.where(here, h[batch, last // CHUNK], final)
    y = _unchunk(y, s["L"]) + s["D_"] * u
    out = torch.where(inside[..., None], y * _silu(s["z"].float()) if s["gate"] else y, 0.0)
    return (out.to(s["u"].dtype), final), (p, raw, u, inside, begin, end, y, kept)


def _plain_scan_backward(s, forward):
    p, raw, u, inside, begin, end, y, kept = forward
    t, L, A = s["u"].dtype, s["L"], s["A"]
    dy = torch.where(inside[..., None], s["dy"].float(), 0.0)
    dz = None
    if s["gate"]:
        z = s["z"].float()
        dz = (dy * y * _dsilu(z)).to(t)
        dy = dy * _silu(z)
    g_out = _chunks(dy)
    # What arrives at a token's state from the last state of its sequence.
    batch = (torch.arange(len(begin), device=DEV) if s["cu"] is None else torch.zeros_like(begin))
    has, last = end > begin, (end - 1).clamp_min(0)

    def arriving(i):
        x = g_out[i][..., None] * p["C"][i][..., None, :]
        here = (has & (last % CHUNK == i))[:, None, None]
        return x.index_put((batch, last // CHUNK), torch.where(here, s["dstate"], 0.0), accumulate=True)

    G, P = 0.0, 1.0
    for i in range(CHUNK - 1, -1, -1):
        a = _decay(p, i, A)
        G, P = a * (arriving(i) + G), a * P
    G = _before_chunks(G.flip(1), P.flip(1))[0].flip(1)
    B, n = G.shape[:2]
    d0 = torch.zeros(len(begin), s["D"], s["N"], device=DEV)
    d0 = torch.where(has[:, None, None], d0, s["dstate"])
    dA = torch.zeros(s["D"], s["N"], device=DEV, dtype=torch.float64)
    ddt, ddu, dB, dC = ([None] * CHUNK for _ in range(4))
    for i in range(CHUNK - 1, -1, -1):
        G = arriving(i) + G
        a = torch.exp(p["dt"][i][..., None] * A)
        starts = p["starts"][i][..., None, None]
        came = torch.zeros_like(G) if s["state"] is None else s["state"][p["seq"][i]]
        before = torch.where(starts, came, kept[i])
        through = G * a * before
        h = a * before + p["du"][i][..., None] * p["B"][i][..., None, :]
        ddt[i] = (through * A).sum(-1)
        dA += (through * p["dt"][i][..., None]).double().sum((0, 1))
        ddu[i] = (G * p["B"][i][..., None, :]).sum(-1)
        dB[i] = (G * p["du"][i][..., None]).sum(-2)
        dC[i] = (h * g_out[i][..., None]).sum(-2)
        G = a * G
        at = (has & (begin % CHUNK == i))[:, None, None]
        d0 = torch.where(at, G[batch, begin.clamp_max(L - 1) // CHUNK], d0)
        G = torch.where(starts, 0.0, G)
    ddt, ddu, dB, dC = (_unchunk(v, L) for v in (ddt, ddu, dB, dC))
    dt = torch.where(inside[..., None], _softplus(raw), 0.0)
    du = ddu * dt + s["D_"] * dy
    draw_ = torch.where(inside[..., None], (ddt + ddu * u) * torch.sigmoid(raw), 0.0)
    rows = lambda x: x.double().sum((0, 1)).float()  # noqa: E731
    return (du.to(t), draw_.to(t), dA.float(), dB.to(t), dC.to(t), rows(dy * u), dz, rows(draw_),
            d0 if s["state"] is not None else None)


def _plain_scan_step(s):
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    u = s["u"].float()
    h = s["state"]
    h.mul_(torch.exp(dt[..., None] * s["A"])).add_((dt * u)[..., None] * s["B_"].float()[:, None])
    y = (h * s["C_"].float()[:, None]).sum(-1) + s["D_"] * u
    return (y * _silu(s["z"].float()) if s["gate"] else y).to(s["u"].dtype), h


# ---- norm and addition in plain operations ----------------------------------------------------


def _normed(total, weight):
    r = (total.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return total * r * weight, r


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    return _normed(total.float(), s["weight"])[0], total


def _plain_norm8(s):
    y, total = _plain_norm(s)
    most = y.abs().amax(-1)
    scale = torch.where(most > 0, most / E4M3_MAX, 1.0)
    y8 = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    # (Values of 8 bits are exact in 16.)
    return y8.to(torch.bfloat16), scale, total


def _plain_norm_backward(s, total):
    total, w, dy = total.float(), s["weight"], s["dy"].float()
    r = (total.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = total * r
    dw = (dy * n).double().sum(0).float()
    g = dy * w
    d = s["dtotal"].float() + r * (g - n * (g * n).mean(-1, keepdim=True))
    return d.to(s["x"].dtype), d.to(s["residual"].dtype), dw


# ---- one pass ------------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "conv":
        return _plain_conv(s)
    if op == "conv_train":
        return (*_plain_conv(s), *_plain_conv_backward(s))
    if op == "conv_step":
        return _plain_conv_step(s)
    if op == "scan":
        return _plain_scan(s)[0]
    if op == "scan_train":
        out, forward = _plain_scan(s, keep=True)
        return (*out, *_plain_scan_backward(s, forward))
    if op == "scan_step":
        return _plain_scan_step(s)
    if op == "norm8":
        return _plain_norm8(s)
    y, total = _plain_norm(s)
    out = y.to(s["x"].dtype), total
    return out if op == "norm" else (*out, *_plain_norm_backward(s, total))


def _run_own(s):
    from deltanet_delta_rule_chunk_amd import binding

    op = s["op"]
    if op == "conv_step":
        return binding.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], silu=s["silu"]), s["state"]
    if op.startswith("conv"):
        how = dict(silu=s["silu"], cu_seqlens=s["cu"])
        out = binding.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"], **how)
        if op == "conv":
            return out
        return (*out, *binding.short_conv_bwd(s["x"], s["weight"], s["bias"], s["state"], s["dy"], s["dstate"],
                                              want_dstate0=s["state"] is not None, **how))
    if op == "scan_step":
        y = binding.selective_scan_step(s["u"], s["dt"], s["A"], s["B_"], s["C_"], s["state"], D=s["D_"],
                                        z=s["z"], dt_bias=s["dt_bias"])
        return y, s["state"]
    if op.startswith("scan"):
        how = dict(D=s["D_"], z=s["z"], dt_bias=s["dt_bias"], h0=s["state"], cu_seqlens=s["cu"])
        args = (s["u"], s["dt"], s["A"], s["B_"], s["C_"])
        out = binding.selective_scan_fwd(*args, **how)
        if op == "scan":
            return out
        return (*out, *binding.selective_scan_bwd(*args, s["dy"], s["dstate"], want_dh0=s["state"] is not None,
                                                  **how))
    if op == "norm8":
        y8, scale, total = binding.add_rms_norm_fp8(s["x"], s["residual"], s["weight"], eps=EPS)
        return y8.to(torch.bfloat16), scale, total
    y, total = binding.add_rms_norm(s["x"], s["residual"], s["weight"], eps=EPS)
    if op == "norm":
        return y, total
    return (y, total, *binding.add_rms_norm_bwd(total, s["weight"], s["dy"], s["dtotal"], eps=EPS))


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    D, op = case["D"], case["op"]
    if op.startswith("norm"):
        x = case["rows"] * D
        r = x * (4 if case["wide"] else e)
        w = {"bytes": x * e + 2 * r + (x + 4 * case["rows"] if op == "norm8" else x * e), "flops": 6 * x}
        if op == "norm_train":
            w = {"bytes": w["bytes"] + 3 * r + 2 * x * e, "flops": w["flops"] + 12 * x}
            w["bytes"] -= x * e if r == x * e else 0  # the two gradients are one
        return w
    x, n = case["B"] * case["L"] * D, case["seqs"] or case["B"]
    if op.startswith("conv"):
        K = case["K"]
        rows = n * (K - 1) * D * e
        kept = rows * (2 if case["state"] else 1)
        w = {"bytes": 2 * x * e + kept + 4 * D * (K + 1), "flops": x * (2 * K + 5)}
        if op == "conv_train":
            w = {"bytes": w["bytes"] + 3 * x * e + rows + kept + 8 * D * (K + 1), "flops": w["flops"] + x * (6 * K + 12)}
        return w
    N, gate = case["N"], int(case["gate"])
    bc = 2 * case["B"] * case["L"] * N * e
    state = n * D * N * 4
    kept = state * (2 if case["state"] else 1)
    par = 4 * D * (N + 2)
    w = {"bytes": x * e * (3 + gate) + bc + kept + par, "flops": x * (7 * N + 20)}
    if op == "scan_train":
        w = {"bytes": w["bytes"] + x * e * (5 + 2 * gate) + 2 * bc + state + kept + 2 * par,
             "flops": w["flops"] + x * (19 * N + 50)}
    return w


# ---- in 64 bits, from the definitions -------------------------------------------------------


def _sequences(s):
    """(index, row, first token, one behind the last) of every sequence."""
    if s["cu"] is None:
        return [(b, b, 0, s["L"]) for b in range(s["B"])]
    cu = s["cu"].tolist()
    return [(i, 0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def _exact_conv(s):
    """Each sequence through torch's own convolution in 64 bits, gradients by autograd."""
    K, D = s["K"], s["D"]
    leaf = lambda x: None if x is None else x.double().clone().requires_grad_()  # noqa: E731
    x, w, b, st = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"]), leaf(s["state"])
    y, kept = torch.zeros(x.shape, dtype=torch.float64, device=DEV), []
    loss = 0.0
    for i, row, lo, hi in _sequences(s):
        front = x.new_zeros(K - 1, D) if st is None else st[i]
        ext = torch.cat([front, x[row, lo:hi]])
        kept.append(ext[hi - lo:])
        if hi > lo:
            p = torch.stack([ext[j:j + hi - lo] for j in range(K)], -1).mul(w).sum(-1)
            p = p if b is None else p + b
            o = p / (1 + torch.exp(-p)) if s["silu"] else p
            y[row, lo:hi] = o.detach()
            if s["op"] == "conv_train":
                loss = loss + (o * s["dy"][row, lo:hi].double()).sum()
    kept = torch.stack(kept)
    if s["op"] == "conv":
        return y, kept.detach()
    loss = loss + (kept * s["dstate"].double()).sum()
    some = [t for t in (x, w, b, st) if t is not None]
    d = dict(zip(map(id, some), torch.autograd.grad(loss, some, allow_unused=True)))
    return y, kept.detach(), *(None if t is None else d[id(t)] for t in (x, w, b, st))


def _exact_scan(s):
    """Token by token, then back over the kept states."""
    B, L, D, N = s["B"], s["L"], s["D"], s["N"]
    seqs = _sequences(s)
    train = s["op"] == "scan_train"
    turn = lambda x: None if x is None else x.double().movedim(1, 0).contiguous()  # noqa: E731
    raw = turn(s["dt"]) + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    u, Bm, Cm, z = turn(s["u"]), turn(s["B_"]), turn(s["C_"]), turn(s["z"])
    A, skip = s["A"].double(), s["D_"].double()
    first = torch.zeros(n_ := len(seqs), D, N, dtype=torch.float64, device=DEV)
    if s["state"] is not None:
        first += s["state"].double()
    final = first.clone()
    # Batches run side by side, packed sequences one after the other.
    begins, lasts, covered = {}, {}, torch.zeros(L, dtype=torch.bool)
    for i, row, lo, hi in seqs:
        if hi > lo:
            begins.setdefault(lo, []).append(i)
            lasts.setdefault(hi - 1, []).append(i)
            covered[lo:hi] = True
    which = lambda i: slice(None) if s["cu"] is None else i[0]  # noqa: E731
    h = torch.zeros(B, D, N, dtype=torch.float64, device=DEV)
    c = torch.empty(L, B, D, dtype=torch.float64, device=DEV)
    before = torch.empty(L, B, D, N, dtype=torch.float64, device=DEV) if train else None
    for t in range(L):
        if not covered[t]:
            c[t] = 0
            continue
        if t in begins:
            h = first[which(begins[t])].reshape(B, D, N).clone()
        if train:
            before[t] = h
        h = torch.exp(dt[t, ..., None] * A).mul_(h).addcmul_((dt[t] * u[t])[..., None], Bm[t, :, None])
        torch.sum(h * Cm[t, :, None], -1, out=c[t])
        if t in lasts:
            final[which(lasts[t])] = h.reshape(final[which(lasts[t])].shape)
    there = covered.to(DEV)[:, None, None]
    plain = c + skip * u
    sig = None if z is None else 1 / (1 + torch.exp(-z))
    y = torch.where(there, plain if z is None else plain * z * sig, 0.0)
    back = lambda x: None if x is None else x.movedim(0, 1)  # noqa: E731
    if not train:
        return back(y), final
    dy = torch.where(there, turn(s["dy"]), 0.0)
    dz = None
    if z is not None:
        dz = dy * plain * (sig + z * sig * (1 - sig))
        dy = dy * z * sig
    G = torch.zeros(B, D, N, dtype=torch.float64, device=DEV)
    d0 = s["dstate"].double().clone()
    dA = torch.zeros_like(A)
    ddt, ddu = torch.zeros_like(u), torch.zeros_like(u)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    for t in range(L - 1, -1, -1):
        if not covered[t]:
            continue
        if t in lasts:
            G = s["dstate"].double()[which(lasts[t])].reshape(B, D, N).clone()
        a = torch.exp(dt[t, ..., None] * A)
        dC[t] = ((a * before[t] + (dt[t] * u[t])[..., None] * Bm[t, :, None]) * dy[t, ..., None]).sum(1)
        G = G + dy[t, ..., None] * Cm[t, :, None]
        dB[t] = (G * (dt[t] * u[t])[..., None]).sum(1)
        ddu[t] = (G * Bm[t, :, None]).sum(-1)
        G = G * a
        e = G * before[t]
        ddt[t] = (e * A).sum(-1)
        dA += (e * dt[t, ..., None]).sum(0)
        if t in begins:
            d0[which(begins[t])] = G.reshape(d0[which(begins[t])].shape)
    du = torch.where(there, ddu * dt + skip * dy, 0.0)
    draw_ = torch.where(there, (ddt + ddu * u) / (1 + torch.exp(-raw)), 0.0)
    return (back(y), final, back(du), back(draw_), dA, back(dB), back(dC), (dy * u).sum((0, 1)), back(dz),
            draw_.sum((0, 1)), d0 if s["state"] is not None else None)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        # (The stream is what it is after its rounding.)
        total = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double().requires_grad_()
        w = s["weight"].double().requires_grad_()
        y = total / torch.sqrt(torch.linalg.vector_norm(total, dim=-1, keepdim=True) ** 2 / case["D"] + EPS) * w
        if op == "norm":
            return y.detach(), total.detach()
        if op == "norm8":
            top = torch.linalg.vector_norm(y.detach(), ord=math.inf, dim=-1)
            y8 = (y.detach() / (top / E4M3_MAX)[:, None]).float().to(torch.float8_e4m3fn)
            return y8.double(), top / E4M3_MAX, total.detach()
        loss = (y * s["dy"].double()).sum() + (total * s["dtotal"].double()).sum()
        d, dw = torch.autograd.grad(loss, [total, w])
        return y.detach(), total.detach(), d, d, dw
    if op == "conv_step":
        ext = torch.cat([s["state"], s["x"][:, None]], 1).double()
        p = torch.einsum("bkd,dk->bd", ext, s["weight"].double())
        p = p if s["bias"] is None else p + s["bias"].double()
        return p / (1 + torch.exp(-p)) if s["silu"] else p, ext[:, 1:]
    if op.startswith("conv"):
        return _exact_conv(s)
    if op == "scan_step":
        one = {n: None if s[n] is None else s[n][:, None] for n in ("u", "dt", "B_", "C_", "z")}
        y, h = _exact_scan({**s, **one, "L": 1, "op": "scan"})
        return y[:, 0], h
    with torch.no_grad():
        return _exact_scan(s)
