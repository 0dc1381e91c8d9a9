"""The benchmark's DRAM traffic: each committed figure belongs to the source that its kernel is built from."""
import json
import os
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "conv_batchnorm_relu_gb300", "csrc")
with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    ENTRIES = [(int(c[6:]), k, e) for c, t in json.load(f).items() if c.startswith("config") for k, e in t.items()]


@pytest.mark.parametrize("config,kernel,entry", ENTRIES, ids=lambda v: str(v) if not isinstance(v, dict) else "")
def test_figures_are_of_the_present_source(config, kernel, entry):
    assert bench.traffic_for(kernel, config) == entry["bytes_per_launch"]
    # the source defines the kernel or instantiates a header's
    with open(os.path.join(CSRC, entry["source"])) as f:
        text = f.read()
    assert "#include" in text and entry["source"].endswith(".cu")


def test_other_sources_do_not_matter_and_own_ones_do(tmp_path):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(CSRC, csrc)
    want = bench.traffic_for("conv_bwd_fused", 3)
    for fn in ("another.cu", "distill.cu", "cbr_api.cu", "norm_ops.cuh"):
        with open(os.path.join(csrc, fn), "a") as f:
            f.write("// other kernels\n")
    assert bench.traffic_for("conv_bwd_fused", 3, csrc) == want
    for fn in ("conv_bwd_fused.cu", "halo_conv.cuh", "ptx.cuh"):   # the source, a header, a header's header
        before = bench.source_sha256("conv_bwd_fused.cu", csrc)
        with open(os.path.join(csrc, fn), "a") as f:
            f.write("// changed\n")
        assert bench.source_sha256("conv_bwd_fused.cu", csrc) != before
        assert bench.traffic_for("conv_bwd_fused", 3, csrc) is None
