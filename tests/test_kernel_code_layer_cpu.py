"""What the compiler makes of the state space layer's kernels (compiled here for gfx950,
not run)."""

import re
import subprocess

import pytest

from deltanet_delta_rule_chunk_amd import build


@pytest.mark.parametrize("source", ["dn_short_conv", "dn_selective_scan", "dn_selective_scan_bwd", "dn_add_norm"])
def test_no_generic_addresses(tmp_path, source):
    """A generic address into LDS with an offset may not start in front of LDS, whatever it
    ends at: the kernels use typed ones only."""
    out = tmp_path / "code.s"
    subprocess.run([build.hipcc(), *build.COMMON_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "--cuda-device-only", "-S",
                    f"{build.CSRC}/{source}.hip", "-o", str(out)], check=True, capture_output=True)
    text = out.read_text()
    assert "global_load" in text and not re.search(r"\bflat_(load|store|atomic)", text)
