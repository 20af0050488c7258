"""The order of stores between the workgroups that draw a token (lik_rows_verify.hip),
read from the kernels' assembly on the CPU.

A workgroup stores its part's sum and then counts itself done; the last one reads all
sums.  The sum and the count lie in different places, so the count may be seen first
unless the wave waits for its store: an s_waitcnt vmcnt(0) between the two, in every
instance of the kernel.  No run on a GPU shows a missing one reliably."""

import os
import re
import subprocess

import pytest

from maxsim_scoring_02_amd import build

try:
    HIPCC = build.hipcc()
except RuntimeError:
    HIPCC = None

WAIT = re.compile(r"\bs_waitcnt\b.*\bvmcnt\(0\)")


@pytest.mark.skipif(HIPCC is None, reason="needs hipcc")
def test_sums_arrive_before_the_count(tmp_path):
    out = tmp_path / "verify.s"
    subprocess.run([HIPCC, *build.HIPCC_FLAGS, "--offload-device-only", "-S",
                    os.path.join(build.CSRC, "lik_rows_verify.hip"), "-o", str(out)], check=True,
                   stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    kernels, name = {}, None
    for line in out.read_text().splitlines():
        begins = re.match(r"(_Z\w*verify_draw_kernel\w*):", line)
        if begins:
            name = begins.group(1)
            kernels[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            kernels[name].append(line.split(";")[0])
    assert len(kernels) == 12            # three types, rows in the caches or not, ends found or not
    for name, lines in kernels.items():
        counts = [i for i, x in enumerate(lines) if "global_atomic_add" in x]
        assert len(counts) == 1, name
        stores = [i for i, x in enumerate(lines) if re.search(r"global_store_dwordx2\b.*\bsc1\b", x)]
        before = [i for i in stores if i < counts[0]]
        assert before, name
        between = lines[before[-1]:counts[0]]
        assert any(WAIT.search(x) for x in between), f"{name}: the count does not wait for the sum"
        # sums that one workgroup takes by itself: its other waves read them behind a barrier
        for i in (i for i in stores if i > counts[0]):
            rest = lines[i:]
            barrier = next(j for j, x in enumerate(rest) if "s_barrier" in x)
            assert any(WAIT.search(x) for x in rest[:barrier]), name
