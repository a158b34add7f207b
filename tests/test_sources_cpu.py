"""Rules that the CUDA sources keep, read as text."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(p for e in ("cu", "cuh", "h") for p in glob.glob(os.path.join(ROOT, "latent_moe_layer_gb300", "csrc", "*." + e)))


def test_no_load_is_multicast_across_a_cluster():
    # every rank of a node runs this library, and a multicast copy is for programs that have one GPU to themselves
    assert len(SOURCES) > 10
    for path in SOURCES:
        text = open(path).read()
        for asm in re.findall(r'"[^;]*?cp\.async\.bulk.*?;', text, re.S):
            assert "multicast" not in asm, path
