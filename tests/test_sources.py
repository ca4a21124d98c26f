"""What the kernels' sources hold, without a GPU."""
import glob
import os
import re

from block_quantized_matmul_gguf_gb300 import build


def test_no_bulk_load_is_sent_to_several_ctas():
    """The library is one for programs on any number of GPUs, and a workspace or an input
    may be memory that another of them holds: no copy of it is multicast in a cluster."""
    sources = [f for e in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(build.CSRC, e))]
    assert len(sources) > 10
    for f in sources:
        text = open(f).read()
        for copy in re.findall(r"cp\.async\.bulk[^;]*;", text):
            assert "multicast" not in copy, f
