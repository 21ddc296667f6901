"""The bench reports committed counters only for the device code they were taken
on: a kernel's digest covers its source and the headers that hold device code."""

import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "bit_quantized_finetuning_nf4_amd", "csrc")
# declarations for the host; the mask's generator and the rides, which no headline launch of these kernels runs
NOT_COVERED = {"kernels.h", "rng.h", "ride.h", "urows.h"}


def headers(name):
    found = set(re.findall(r'#include "(\w+\.h)"', open(os.path.join(CSRC, name)).read()))
    return found.union(*(headers(h) for h in found)) if found else found


def test_digests_cover_the_headers_of_their_kernels():
    for kernel, sources in bench.KERNEL_SOURCES.items():
        covered = set(sources) | set(bench.DEVICE_HEADERS)
        for s in sources:
            assert headers(s) - NOT_COVERED <= covered, (kernel, headers(s) - covered)
