"""The benchmark's HBM traffic figure: counters in profiles/, kept by a hash of
the headline GEMM's source and the headers it includes.  When those change the
line reports null, and the counters have to be taken again with the commands
that the profile gives."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_the_figure_belongs_to_these_sources():
    traffic = bench.gemm_traffic()
    assert traffic is not None, "the GEMM's sources changed since its traffic was measured"
    assert 4096 * 4096 * (2 * (0.5 + 1 / 32) + 2) <= traffic < 4 * 4096 * 4096 * 2


def test_the_hash_covers_every_header_of_the_kernel():
    seen, todo = set(), [bench.GEMM_SOURCES[0]]
    while todo:
        path = todo.pop()
        if path not in seen:
            seen.add(path)
            with open(path) as f:
                todo += [os.path.normpath(os.path.join(os.path.dirname(path), n))
                         for n in re.findall(r'^#include "(.*)"', f.read(), re.M)]
    assert seen == set(bench.GEMM_SOURCES)
