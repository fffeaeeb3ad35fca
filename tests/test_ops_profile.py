"""The operators' profile was taken at the operators' present sources."""
import os
import re

import bench


def test_operator_profile_names_the_present_sources():
    """The summary names the hash of csrc/ops (comments and whitespace aside),
    which the layer's own hash leaves out: a kernel that changes after its
    profile was written shows here."""
    src = os.path.join(bench.ROOT, "bit_quantized_routed_router_amd", "csrc", "ops")
    text = open(os.path.join(bench.ROOT, "profiles", "ops_kernel_trace.md")).read()
    m = re.search(r"Operator source hash \(bit_quantized_routed_router_amd/csrc/ops\): `([0-9a-f]{16})`", text)
    assert m and m.group(1) == bench.kernel_source_hash(src)
