"""What the CUDA sources may not hold, read as text (no GPU needed)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _sources():
    for p in sorted(glob.glob(os.path.join(ROOT, "dropless_grouped_gemm_gb300", "csrc", "*.cu*"))):
        yield os.path.basename(p), open(p, encoding="utf-8").read()


def test_arrivals_between_ctas_release():
    """An arrival on another CTA's barrier says that this CTA's accesses are
    done, and the other CTA then overwrites what was read, or leaves: every
    such arrival has to order the accesses before it."""
    found = [(n, m.group(0)) for n, s in _sources()
             for m in re.finditer(r"(mbarrier|barrier\.cluster)\.arrive[.\w]*\.relaxed[.\w]*", s)]
    assert not found, found
