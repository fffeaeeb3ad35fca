"""The training operators' profile was taken at their present sources."""
import os
import re

import bench


def test_train_profile_names_the_present_sources():
    """The summary names the hash of csrc/train, comments and whitespace aside."""
    src = os.path.join(bench.ROOT, "bit_quantized_routed_router_amd", "csrc", "train")
    text = open(os.path.join(bench.ROOT, "profiles", "train_kernel_trace.md")).read()
    m = re.search(r"Training operator source hash \(bit_quantized_routed_router_amd/csrc/train\): `([0-9a-f]{16})`", text)
    assert m and m.group(1) == bench.kernel_source_hash(src)
