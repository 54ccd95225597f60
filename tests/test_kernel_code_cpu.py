"""What the compiler makes of the kernels' building blocks (compiled here for
gfx950, not run)."""

import re
import subprocess

from deltanet_delta_rule_chunk_amd import build

M0_KEPT = r"""
#include "dn_linear.h"
typedef __attribute__((address_space(3))) unsigned lds_u32;
extern "C" __global__ void probe(const float* p, uint32_t at) {
  __shared__ float buf[64];
  const auto rows = dn::lin::chunk_rsrc<float, 64>(p, 0, 64);
  const auto r = dn::make_rsrc(p, 256);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_u32*)buf, 4, threadIdx.x * 4, 0, 0, 0);
  dn::lin::load_to_lds(rows, threadIdx.x * 16, at);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_u32*)buf, 4, threadIdx.x * 4, 0, 0, 0);
}
"""


def test_a_value_kept_in_m0_survives_a_load_to_lds(tmp_path):
    """The assembly of load_to_lds sets m0.  A load of the compiler's own in front
    of it and one behind it, to the same place, need m0 set for each."""
    src, out = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(M0_KEPT)
    subprocess.run([build.hipcc(), *build.COMMON_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC,
                    "--cuda-device-only", "-S", str(src), "-o", str(out)], check=True,
                   capture_output=True)
    text = out.read_text()
    text = text[text.index("\nprobe:"):]
    text = text[:text.index("s_endpgm")]
    order = re.findall(r"s_mov_b32 m0|buffer_load_dword\w* .*lds", text)
    order = ["m0" if "m0" in x else "load" for x in order]
    assert order == ["m0", "load"] * 3, order
