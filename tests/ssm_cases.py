"""Inputs, bounds and comparisons shared by the tests of the state space layer's operators.

A bound is `units` roundings of fp32 (2^-24) of a sum's terms in magnitude, and half a
step of the output's own type.
"""

import numpy as np
import torch

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ULP = 2.0 ** -24


def close(got, want, size, units, what):
    """|got - want| <= units 2^-24 size + half a step of got's type."""
    g = got.detach().to("cpu", torch.float64).numpy()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    assert np.isfinite(g).all(), what
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else ULP
    bound = units * ULP * size * (1 + half) + half * np.abs(want) + 1e-37
    over = np.abs(g - want) / bound
    at = np.unravel_index(over.argmax(), over.shape) if over.size else None
    assert over.size == 0 or over.max() <= 1, (what, at, float(over.max()), g[at], want[at])


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * std).to(dtype)


def conv_inputs(seed, B, L, D, K, dtype, n, state=True, bias=True):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    x = dict(x=normal(gen, (B, L, D), dtype=t), weight=normal(gen, (D, K), K ** -0.5),
             bias=normal(gen, (D,)) if bias else None,
             state0=normal(gen, (n, K - 1, D), dtype=t) if state else None,
             dy=normal(gen, (B, L, D), dtype=t), dstate=normal(gen, (n, K - 1, D), dtype=t))
    return x


def scan_inputs(seed, B, L, D, N, dtype, n, state=True, gate=True, skip=True, bias=True):
    """Steps of about 0.001 to 0.1 at rates of 1 to N."""
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    start = torch.exp(torch.rand((D,), generator=gen) * 4.6 - 6.9)
    dt_bias = start + torch.log(-torch.expm1(-start))
    raw = normal(gen, (B, L, D), 0.5)
    x = dict(u=normal(gen, (B, L, D), dtype=t), dt=(raw if bias else raw + dt_bias).to(t),
             A=-torch.arange(1, N + 1) * torch.exp(normal(gen, (D, N), 0.1)),
             B=normal(gen, (B, L, N), dtype=t), C=normal(gen, (B, L, N), dtype=t),
             D=normal(gen, (D,)) if skip else None, z=normal(gen, (B, L, D), dtype=t) if gate else None,
             dt_bias=dt_bias if bias else None, h0=normal(gen, (n, D, N)) if state else None,
             dy=normal(gen, (B, L, D), dtype=t), dhT=normal(gen, (n, D, N)))
    return x


def gpu(x):
    return {k: None if v is None else v.to(DEV) for k, v in x.items()}


def cu_of(cuts):
    return None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device=DEV)


#: Packed sequences: (rows, cuts).  Empty ones, single tokens, rows in front and behind.
PACKED = {"mixed": (150, [0, 0, 1, 5, 69, 69, 70, 131, 150]), "padded": (97, [3, 20, 20, 90]),
          "one": (33, [0, 33]), "none": (9, [0, 0, 0]), "tiles": (400, [0, 16, 32, 96, 160, 320, 400])}
