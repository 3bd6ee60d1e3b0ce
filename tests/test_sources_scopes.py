"""Scopes of the arrivals in the CUDA sources, read as text (no GPU needed)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dropless_grouped_gemm_gb300", "csrc")


def test_an_arrival_on_another_ctas_barrier_releases_at_cluster_scope():
    """The thread that waits is in another CTA: a release whose scope does not
    hold it (.cta, which is also what an arrival without a scope has) does not
    synchronise with its acquire, whatever is handed over."""
    seen = []
    for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for m in re.finditer(r"mbarrier\.arrive[.\w:]*", open(p, encoding="utf-8").read()):
            if "shared::cluster" in m.group(0):
                seen.append((os.path.basename(p), m.group(0)))
    assert seen
    assert all(".release.cluster." in s for _, s in seen), seen


def test_waits_for_other_ctas_acquire_at_cluster_scope():
    src = open(os.path.join(CSRC, "fp4_gemm.cu"), encoding="utf-8").read()
    # the accumulator's release by both CTAs' epilogues, waited for by the first CTA's issuer
    assert "mbar_wait_cluster(tempty_bar" in src and "mbar_wait(tempty_bar" not in src
    assert "mbar_arrive_cluster(tempty0" in src
