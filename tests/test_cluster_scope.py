"""Arrivals at another CTA's barrier name the cluster as their scope: without one an mbarrier operation has the
CTA's, and orders nothing between two CTAs. Read from the kernels' inline PTX."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _instructions():
    for path in sorted(glob.glob(os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc", "*.cu*"))):
        with open(path) as f:
            for m in re.finditer(r"\bmbarrier\.[a-z_:.0-9]+", f.read()):
                yield os.path.basename(path), m.group(0)


def test_arrivals_at_another_ctas_barrier_have_cluster_scope():
    remote = [(f, i) for f, i in _instructions() if ".shared::cluster" in i]
    assert remote, "the pattern finds no instruction"
    for f, i in remote:
        assert re.match(r"mbarrier\.arrive(\.expect_tx)?\.(relaxed|release)\.cluster\.shared::cluster\.", i), (f, i)


def test_the_pairs_waits_for_the_other_cta_have_cluster_scope():
    path = os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc", "mxfp4_stream_pair.cu")
    with open(path) as f:
        text = f.read()
    for bar in ("ready", "acc_empty"):          # what the other CTA's copies and warps arrive at
        waits = re.findall(r"(\w+)\(&%s\[" % bar, text)
        assert {w for w in waits if "wait" in w} == {"mbar_wait_cluster"}, (bar, waits)
