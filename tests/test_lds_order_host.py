"""Order of the LDS accesses that a wave's lanes pass rows through in the few-row base product, read from the assembly
that the compiler makes of it: all of a block's rows are written before any is read. Compiled, not run."""
import os
import re
import shutil
import subprocess

import pytest

from segmented_gather_gemv_amd import build as b


@pytest.mark.parametrize("source", ["base_direct_i4.hip", "base_direct_i4z.hip"])
def test_staged_rows_are_written_before_they_are_read(source, tmp_path):
    if not shutil.which(b._hipcc()):
        pytest.skip("no hipcc")
    out = tmp_path / "kernels.s"
    subprocess.run([b._hipcc(), *b.HIP_FLAGS, "--cuda-device-only", "-S", os.path.join(b.CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    seen = 0
    # <E2M1, F32, ZERO, S, NT, TM, WAVES, STAGED>
    for m in re.finditer(r"^_ZN4sgmv18base_direct_kernelI\w+?Li\d+ELi\d+ELi(\d+)ELi\d+ELb1EE\w+:.*?^\.Lfunc_end", text, re.M | re.S):
        rows = int(m[1])
        run, runs = 0, []
        for line in m[0].splitlines():
            op = line.split()[0] if line.strip() else ""
            if re.match(r"ds_(write|store)_b128", op):
                run += 1
            elif run and (re.match(r"ds_(read|load)_b128", op) or op.startswith((".L", "s_cbranch", "s_branch"))):
                runs.append(run)
                run = 0
        assert runs and all(n == 4 * rows for n in runs), (m[0].split(":")[0], runs)
        seen += 1
    assert seen == 18  # six instances of each group
