"""The committed counter summaries belong to the committed kernels: bench.py reports their figures only where the
hash of the kernel's sources is the one that the summary was taken at."""
import pytest

import bench


@pytest.mark.parametrize("summary,kernel", [("decode_layer_b64_bf16_traffic.md", "gdn_decode.hip"),
                                            ("prefill_t4096_traffic.md", "gdn_prefill.hip")])
def test_the_traffic_of_the_delta_rule_kernels_is_that_of_their_sources(summary, kernel):
    source = bench.kernel_source_hash([kernel, "gdn_device.h", "gdn_kernels.h"])
    assert bench.read_traffic(summary, source) is not None
