"""bench.py ties recorded counters to the kernels' sources: its lists name every file a kernel is built from."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "sparse_rank_linear_prune24_amd", "csrc")


def included(name, seen):
    seen.add(name)
    with open(os.path.join(CSRC, name)) as fh:
        for header in re.findall(r'^#include "([^"]+)"', fh.read(), re.M):
            if header not in seen:
                included(header, seen)
    return seen


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCE))
def test_a_kernels_sources_are_all_listed(kernel):
    names = bench.KERNEL_SOURCE[kernel]
    assert len(set(names)) == len(names)
    # kernels.hpp declares host functions; epilogue.hpp comes with it, and the pack kernels use nothing of it
    unused = {"kernels.hpp"} | ({"epilogue.hpp"} if kernel == "pack" else set())
    assert set(names) == included(names[0], set()) - unused
