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


def test_the_few_row_kernel_waits_for_its_copies():
    """A CTA that gives up leaves after its copies have landed (a bounded wait
    on their barriers), not after some time."""
    src = dict(_sources())["linear.cu"]
    assert "stage_drain(" in src
    spins = re.findall(r"while \(globaltimer_ns\(\)[^;{]*\)\s*(?:\{\s*\}|;)", src)
    assert not spins, spins
