"""Calls on another stream than the current one take no memory that the current
one still works on."""

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from test_gpu_linear import _gpu, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _calls():
    x = _gpu(_inputs(100, 1, 4, 1, 1200, 128, 128, "bf16", True, "usual"))
    beta = torch.rand((1, 4, 1200), device=DEV)
    rows = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    pos, inv = torch.arange(1200, device=DEV, dtype=torch.int32)[None], torch.rand(64, device=DEV)
    return {
        "linear_chunk_fwd": lambda s: N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], stream=s),
        "linear_chunk_bwd": lambda s: N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"],
                                                         x["dS"], stream=s),
        "linear_decode_step": lambda s: (N.linear_decode_step(*rows, x["S0"].clone(), stream=s),),
        "qk_norm_rope": lambda s: N.qk_norm_rope(x["q"], x["k"], pos, inv, stream=s),
        "qk_norm_rope_bwd": lambda s: N.qk_norm_rope_bwd(x["q"], x["k"], pos, inv, x["q"], x["k"], stream=s),
        "chunk_fwd": lambda s: N.chunk_fwd(x["q"], x["k"], x["v"], beta, x["S0"], stream=s),
    }


NAMES = ("linear_chunk_fwd", "linear_chunk_bwd", "linear_decode_step", "qk_norm_rope",
         "qk_norm_rope_bwd", "chunk_fwd")


@pytest.mark.parametrize("name", NAMES)
def test_memory_given_back_on_the_current_stream_is_not_written_early(gpu_lib, name):
    """Blocks of every size that the call asks for are freed with a fill of them
    still to run on the current stream, behind a wait; the call on the side stream
    does not wait for it."""
    call = _calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want if t is not None]
    sizes += [N.linear_workspace_bytes(1, 4, 1200, 128, 128, torch.bfloat16, backward=b) for b in (0, 1)]
    blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda._sleep(50_000_000)
    for b in blocks:
        b.fill_(255)
    del blocks, b
    if name == "linear_decode_step":
        side.wait_stream(torch.cuda.current_stream())  # its state is cloned on the current stream
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        if a is not None:
            assert torch.equal(a, b)
