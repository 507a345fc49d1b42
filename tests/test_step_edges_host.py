"""Further checks of the serving-step operators that need no GPU: what the
sources must keep to, refusals, and the build of the two libraries."""
import glob
import os
import re

import pytest

from paged_attention_decode_v2_gb300 import build as pa_build


def _code(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


SOURCES = sorted(glob.glob(os.path.join(pa_build.CSRC, "*.cu*")))


@pytest.mark.parametrize("path", [p for p in SOURCES
                                  if "cudaGridDependencySynchronize();" in _code(p)],
                         ids=os.path.basename)
def test_results_of_the_grid_before_are_read_coherently(path):
    """A programmatic dependent runs while the grid before it still writes, so
    what it reads after its wait is not read-only for the kernel's lifetime:
    no __ldg there."""
    for kernel in _code(path).split("__global__")[1:]:
        body = kernel.split("template <", 1)[0]
        if "cudaGridDependencySynchronize();" not in body:
            continue
        after = body.split("cudaGridDependencySynchronize();", 1)[1]
        assert "__ldg" not in after and "load_row" not in after
        assert "__ldcg" in after
