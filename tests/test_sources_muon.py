"""The Muon step updates the caller's momentum in its first launch, so everything else that can fail
on the host comes before it: the kernels' configuration and the tensor maps."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_nothing_that_can_fail_stands_between_the_launches():
    text = open(os.path.join(ROOT, "sample_gradient_clipping_b200", "csrc", "muon_host.cuh")).read()
    text = re.sub(r"//[^\n]*", "", text)
    start = text.index("dp_status muon_run(")
    body = text[start:text.index("}  // namespace" if "}  // namespace" in text else 'extern "C"', start)]
    launch = min(body.index("DP_LAUNCH("), body.index("ns_small<"))
    for call in ("ns_small_configure", "map_f16(", "DP_CUDA(", "cudaFuncSetAttribute", "ns_configure"):
        assert all(m.start() < launch for m in re.finditer(re.escape(call), body)), call
    # and the functions that only launch do nothing else that can fail
    for name in ("dp_status ns_launch(", "dp_status ns_small("):
        at = text.index(name)
        part = text[at:text.index("\n}\n", at)]
        assert "DP_CUDA(" not in part and "cudaFuncSetAttribute" not in part, name
