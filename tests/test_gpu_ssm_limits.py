"""The state space layer's operators at the ends of what their documentation allows: tensors
past 2^31 elements, many sequences, wide rows, calls under way at once, calls on another
stream than the current one.  Bounds: those of the operators' own tests."""

import threading

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import conv_forward, scan_forward, spans_of
from ssm_cases import DEV, close, conv_inputs, cu_of, f64, gpu, scan_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
D = 4096
L = 2 ** 31 // D + 100


def _rows(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=BF).mul_(std)


def test_conv_past_2_to_the_31_elements(gpu_lib):
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, dy = _rows(gen, 1, L, D), _rows(gen, 1, L, D)
    w, b = torch.randn((D, 4), generator=gen, device=DEV), torch.randn((D,), generator=gen, device=DEV)
    y, state = N.short_conv_fwd(x, w, b)
    dx, dw, db, _ = N.short_conv_bwd(x, w, b, None, dy, want_dstate0=False)
    # Rows depend on 3 neighbours alone, and their arithmetic is the same wherever they lie.
    t = L - 300
    y1, s1 = N.short_conv_fwd(x[:, t:], w, b, x[:, t - 3:t].contiguous())
    dx1 = N.short_conv_bwd(x[:, t:].contiguous(), w, b, x[:, t - 3:t].contiguous(), dy[:, t:].contiguous())[0]
    assert torch.equal(y[:, t:], y1) and torch.equal(state, s1) and torch.equal(dx[:, t:], dx1)
    y1, _ = N.short_conv_fwd(x[:, :300], w, b)
    assert torch.equal(y[:, :300], y1) and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_scan_past_2_to_the_31_elements(gpu_lib):
    """Steps of about 0.7 at rates of 1 and more: 300 tokens leave nothing of a state, so both
    ends follow from calls on their own."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    S, T = 8, 600
    u, dt, z, dy = _rows(gen, 1, L, D), _rows(gen, 1, L, D, std=0.1), _rows(gen, 1, L, D), _rows(gen, 1, L, D)
    B, C = _rows(gen, 1, L, S), _rows(gen, 1, L, S)
    A = -(1 + torch.rand((D, S), generator=gen, device=DEV))
    skip = torch.randn((D,), generator=gen, device=DEV)
    y, hT = N.selective_scan_fwd(u, dt, A, B, C, D=skip, z=z)
    got = N.selective_scan_bwd(u, dt, A, B, C, dy, D=skip, z=z, want_dh0=False)
    torch.cuda.synchronize()
    for end, keep in ((slice(L - T, L), slice(T - 300, T)), (slice(0, T), slice(0, 300))):
        part = [t[:, end].contiguous() for t in (u, dt, B, C, z, dy)]
        y1, h1 = N.selective_scan_fwd(*part[:2], A, *part[2:4], D=skip, z=part[4])
        g1 = N.selective_scan_bwd(*part[:2], A, *part[2:4], part[5], D=skip, z=part[4], want_dh0=False)
        pairs = [(y, y1, "y"), (got[0], g1[0], "du"), (got[1], g1[1], "ddt"), (got[3], g1[3], "dB"), (got[4], g1[4], "dC"),
                 (got[6], g1[6], "dz")]
        for a, b, what in pairs:
            a, b = a[:, end][:, keep].float(), b[:, keep].float()
            # (The same sums from another cut: bf16 roundings of values that differ in the last bits.)
            assert float((a - b).norm()) <= 2.0 ** -9 * float(b.norm()), what
        if end.stop == L:
            assert float((hT - h1).norm()) <= 1e-6 * float(h1.norm())
    x = {"u": u, "dt": dt, "B": B, "C": C, "z": z}
    e = {k: f64(v[:, L - 200:, :16] if k in "u dt z".split() else v[:, L - 200:]) for k, v in x.items()}
    h0 = np.zeros((1, 16, S))
    how = dict(D=f64(skip[:16]), z=e["z"], h0=h0)
    args = (e["u"], e["dt"], f64(A[:16]), e["B"], e["C"], spans_of(1, 200))
    want, size = scan_forward(*args, **how)[0], scan_forward(*args, **how, size=True)[0]
    close(y[:, L - 50:, :16], want[:, 150:], size[:, 150:], 4 * 200 + 64, "y")


def test_norm_past_2_to_the_31_elements(gpu_lib):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, res = _rows(gen, L, D), _rows(gen, L, D)
    w = torch.randn((D,), generator=gen, device=DEV)
    y, total = N.add_rms_norm(x, res, w)
    y8, scale, _ = N.add_rms_norm_fp8(x, res, w)
    d, _, dw = N.add_rms_norm_bwd(total, w, x, res)
    s = slice(L - 50, L)
    y1, t1 = N.add_rms_norm(x[s], res[s], w)
    q1, s1, _ = N.add_rms_norm_fp8(x[s], res[s], w)
    d1 = N.add_rms_norm_bwd(t1, w, x[s], res[s])[0]
    assert torch.equal(y[s], y1) and torch.equal(total[s], t1) and torch.equal(d[s], d1)
    assert torch.equal(y8[s].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(scale[s], s1)
    assert torch.isfinite(dw).all()


def test_many_sequences(gpu_lib):
    """More cuts than LDS holds, single tokens and none."""
    rng = np.random.default_rng(4)
    cuts = np.concatenate([[0], np.cumsum(rng.integers(0, 3, 3000))]).tolist()
    n, T = 3000, cuts[-1] + 7
    x = conv_inputs(1, 1, T, 16, 4, "f32", n)
    g = gpu(x)
    y, state = N.short_conv_fwd(g["x"], g["weight"], g["bias"], g["state0"], cu_seqlens=cu_of(cuts))
    e = {k: f64(v) for k, v in x.items()}
    want, kept = conv_forward(e["x"], e["weight"], e["bias"], e["state0"], spans_of(1, T, cuts))
    size = conv_forward(*(np.abs(e[k]) for k in ("x", "weight", "bias", "state0")), spans_of(1, T, cuts), False)[0]
    close(y, want, 1.1 * size + 1e-3, 20, "y")
    assert np.array_equal(f64(state), kept)
    x = scan_inputs(2, 1, T, 16, 8, "f32", n)
    g = gpu(x)
    how = {k: g[k] for k in ("D", "z", "dt_bias", "h0")}
    args = [g[k] for k in ("u", "dt", "A", "B", "C")]
    y, hT = N.selective_scan_fwd(*args, **how, cu_seqlens=cu_of(cuts))
    e = {k: f64(v) for k, v in x.items()}
    args = [e[k] for k in ("u", "dt", "A", "B", "C")]
    how = {k: e[k] for k in how}
    want = scan_forward(*args, spans_of(1, T, cuts), **how)
    size = scan_forward(*args, spans_of(1, T, cuts), **how, size=True)
    close(y, want[0], size[0], 4 * 3 + 64, "y")
    close(hT, want[1], size[1], 4 * 3 + 64, "hT")


def test_wide_rows_and_large_strides(gpu_lib):
    """Rows far apart, in tensors whose extent passes 4 GiB, channels by the thousand."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    big = torch.zeros((40, 1 << 24), device=DEV, dtype=BF)[None]
    x = _rows(gen, 1, 40, 64)
    w = torch.randn((64, 4), generator=gen, device=DEV)
    big[..., 8:72] = x
    far = big[..., 8:72]
    assert torch.equal(N.short_conv_fwd(far, w)[0], N.short_conv_fwd(x, w)[0])
    A, few = -torch.rand((64, 8), generator=gen, device=DEV), _rows(gen, 1, 40, 8)
    big[..., 128:136] = few
    a = N.selective_scan_fwd(far, far, A, big[..., 128:136], big[..., 128:136], z=far)
    b = N.selective_scan_fwd(x, x, A, few, few, z=x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = N.selective_scan_bwd(far, far, A, big[..., 128:136], big[..., 128:136], x, z=far)
    b = N.selective_scan_bwd(x, x, A, few, few, x, z=x)
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    del big, far
    wide = torch.zeros((1, 3, (1 << 24) + 64), device=DEV, dtype=BF)
    with pytest.raises(N.DeltaNetError, match="UNSUPPORTED"):
        N.short_conv_fwd(wide[..., :64], w)


def _calls():
    x = gpu(scan_inputs(3, 2, 700, 136, 16, "bf16", 2))
    c = gpu(conv_inputs(4, 2, 700, 136, 4, "bf16", 2))
    how = {k: x[k] for k in ("D", "z", "dt_bias", "h0")}
    seq = [x[k] for k in ("u", "dt", "A", "B", "C")]
    one = [x["u"][:, 0], x["dt"][:, 0], x["A"], x["B"][:, 0], x["C"][:, 0]]
    w = torch.rand((136,), device=DEV)
    conv = (c["x"], c["weight"], c["bias"], c["state0"])
    return {
        "short_conv_fwd": lambda s: N.short_conv_fwd(*conv, stream=s),
        "short_conv_bwd": lambda s: N.short_conv_bwd(*conv, c["dy"], c["dstate"], stream=s),
        "short_conv_step": lambda s: (N.short_conv_step(c["x"][:, 0], c["weight"], c["bias"], c["state0"].clone(), stream=s),),
        "selective_scan_fwd": lambda s: N.selective_scan_fwd(*seq, **how, stream=s),
        "selective_scan_bwd": lambda s: N.selective_scan_bwd(*seq, x["dy"], x["dhT"], **how, stream=s),
        "selective_scan_step": lambda s: (N.selective_scan_step(*one, x["h0"].clone(), stream=s),),
        "add_rms_norm": lambda s: N.add_rms_norm(x["u"], x["dy"], w, stream=s),
        "add_rms_norm_fp8": lambda s: tuple(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                                            for t in N.add_rms_norm_fp8(x["u"], x["dy"], w, stream=s)),
        "add_rms_norm_bwd": lambda s: N.add_rms_norm_bwd(x["u"], w, x["dy"], x["z"], stream=s),
    }


@pytest.mark.parametrize("name", ["short_conv_fwd", "short_conv_bwd", "short_conv_step", "selective_scan_fwd",
                                  "selective_scan_bwd", "selective_scan_step", "add_rms_norm", "add_rms_norm_fp8",
                                  "add_rms_norm_bwd"])
def test_memory_given_back_on_the_current_stream_is_not_written_early(gpu_lib, name):
    """Blocks of every size that the call asks for are freed with a fill of them still to
    run on the current stream, behind a wait; the call on the side stream does not wait for it."""
    call = _calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want if t is not None]
    sizes += [N._scan_workspace_bytes(b, 2, 700, 136, 16, 0, 2) for b in (False, True)]
    sizes += [N._conv_bwd_workspace_bytes(2, 700, 136, 4), N._norm_bwd_workspace_bytes(1400, 136)]
    blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda._sleep(50_000_000)
    for b in blocks:
        b.fill_(255)
    del blocks, b
    if name.endswith("step"):
        side.wait_stream(torch.cuda.current_stream())  # its state is cloned on the current stream
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


def test_two_threads_on_two_streams(gpu_lib):
    calls = [_calls(), _calls()]
    names = [n for n in calls[0] if not n.endswith("step")]
    want = [{n: c[n](None) for n in names} for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(15):
            for n in names:
                got = calls[i][n](s)
                s.synchronize()
                bad.extend((i, n) for a, b in zip(want[i][n], got) if a is not None and not torch.equal(a, b))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad[:5]


def test_a_callers_workspace_of_any_contents(gpu_lib):
    """Workspaces full of NaN give the same bits as new ones, uncut and cut, packed and not."""
    for B, T, cuts in ((2, 700, None), (1, 700, [0, 5, 5, 400, 690]), (1, 40, None)):
        n = B if cuts is None else len(cuts) - 1
        x = gpu(scan_inputs(6, B, T, 72, 16, "f32", n))
        how = {k: x[k] for k in ("D", "z", "dt_bias", "h0")}
        args, cu = [x[k] for k in ("u", "dt", "A", "B", "C")], cu_of(cuts)
        for back in (False, True):
            size = N._scan_workspace_bytes(back, B, T, 72, 16, int(cuts is not None), n)
            ws = torch.full((max(size, 16) // 4 + 4,), float("nan"), device=DEV)
            call = (lambda w: N.selective_scan_bwd(*args, x["dy"], x["dhT"], **how, cu_seqlens=cu, workspace=w)) if back else \
                (lambda w: N.selective_scan_fwd(*args, **how, cu_seqlens=cu, workspace=w))
            for a, b in zip(call(None), call(ws)):
                assert torch.equal(a, b) and torch.isfinite(a).all()
    c = gpu(conv_inputs(7, 2, 300, 72, 4, "f32", 2))
    ws = torch.full((N._conv_bwd_workspace_bytes(2, 300, 72, 4) // 4,), float("nan"), device=DEV)
    a = N.short_conv_bwd(c["x"], c["weight"], c["bias"], c["state0"], c["dy"], c["dstate"])
    b = N.short_conv_bwd(c["x"], c["weight"], c["bias"], c["state0"], c["dy"], c["dstate"], workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
