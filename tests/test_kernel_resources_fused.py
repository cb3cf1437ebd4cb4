"""Compile-time guard on the private memory of the fused and expert products'
kernels, of routing and of the combine: no kernel may use scratch or spill a
vector register (a spill inside the expanded product's loop would wait for its
loads in flight).  No kernel is launched."""
import os
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import resources

SOURCES = ("usw_fused.hip", "usw_wide.hip", "usw_route.hip")


@pytest.mark.slow
def test_no_kernel_uses_scratch():
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        found = dict(zip(SOURCES, pool.map(resources, SOURCES)))
    for src, kernels in found.items():
        assert kernels, f"no kernels reported for {src}"
        for k, (scratch, spills) in kernels.items():
            assert scratch == 0 and spills == 0, f"{src}: {k} uses {scratch} bytes of scratch, {spills} spills"
