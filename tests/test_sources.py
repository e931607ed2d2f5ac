"""What the library's sources may not hold, since every rank of a multi-GPU run loads
it: loads and commits that reach several CTAs of a cluster at once."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "block_diffusion_speculative_attn_gb300")


def test_no_cluster_multicast():
    sources = [p for e in ("cu", "cuh", "h") for p in
               glob.glob(os.path.join(PACKAGE, "**", f"*.{e}"), recursive=True)]
    assert len(sources) > 10
    for p in sources:
        with open(p) as f:
            assert "multicast" not in f.read(), p
