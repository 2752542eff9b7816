"""Direct global-to-LDS loads written as asm: between the scalar write of M0
and the load that reads it the hardware needs one wait state, which the
compiler cannot insert inside an asm block."""
import glob
import os
import re

import mini_means_amd as mm

CSRC = os.path.join(os.path.dirname(os.path.abspath(mm.__file__)), "csrc")


def test_m0_is_written_a_wait_state_before_the_load():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.h*")):
        with open(path) as f:
            text = f.read()
        for block in re.findall(r'asm volatile\(\s*((?:"[^"]*"\s*)+)', text):
            steps = [s.strip() for s in re.sub(r'"\s*"', "", block).strip('" \n').split(r"\n\t")]
            for i, s in enumerate(steps):
                if "_load_lds_" in s:
                    found += 1
                    writes = [j for j in range(i) if re.match(r"s_\w+ m0\b", steps[j])]
                    assert writes, (path, steps)     # M0 is this block's own
                    assert i - writes[-1] >= 2, (path, steps)
    assert found >= 4
