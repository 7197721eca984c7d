"""Source check of the expert and 4-bit kernels.  Each is resident before the
kernel that writes its inputs has ended, so nothing it reads is read-only for
as long as it lives, and none may take the read-only load path."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_gemm_b200", "csrc")
FILES = sorted(os.path.basename(p) for pattern in ("few_rows*", "grouped*", "mx4_*")
               for p in glob.glob(os.path.join(CSRC, pattern)))


def code_of(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_the_kernels_are_looked_at():
    assert {"few_rows.cu", "grouped.cu", "grouped.cuh", "grouped_kernel.cuh", "grouped_bias.cu", "mx4_quant.cu"} <= set(FILES)
    assert all("wait_for_prior_grid()" in code_of(f) for f in FILES if "__global__" in code_of(f))


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads_in_dependent_kernels(name):
    found = re.findall(r"__ldg\w*\s*\(|ld\.global\.nc[\w.:]*|__restrict__", code_of(name))
    assert not found, (name, found)


def test_an_aborted_pair_waits_for_its_copies():
    """Two producers a CTA give up at stages of their own: behind the last role and before the pair's
    last barrier, an aborted run waits until a copy that no barrier counts has ended."""
    code = code_of("grouped_kernel.cuh")
    kernel = code[code.index("k_grouped(const"):code.index("tmem_dealloc_pair(tmem")]
    tail = kernel[kernel.rindex("bulk_wait_group<0>()"):]
    order = [tail.rindex("mbar_wait(drain"), tail.index("if (*abort_flag)"), tail.index("__nanosleep"), tail.rindex("cluster_sync_all()")]
    assert order == sorted(order)


def test_no_tensor_map_is_changed_on_the_device():
    """Copies go through maps of whole matrices, encoded by the driver.  Maps that a kernel moved to an
    expert's first row, with its row count, reached past the matrix where the box did."""
    for name in FILES:
        found = re.findall(r"tensormap\.(?:replace|cp_fenceproxy)|fence\.proxy\.tensormap", code_of(name))
        assert not found, (name, found)
