"""Every kernel is launched so that it may start while the one before it ends, and
waits for that one before it reads.  Loads through the non-coherent path are made
for memory that nothing writes while the kernel lives, which begins before its wait:
the sources name none."""
import os
import re

import bit_paged_kv_gb300.build as saw_build


def test_no_load_through_the_non_coherent_path():
    found = []
    for name in sorted(os.listdir(saw_build.CSRC)):
        with open(os.path.join(saw_build.CSRC, name)) as f:
            for i, line in enumerate(f, 1):
                if re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b", line.split("//")[0]):
                    found.append(f"{name}:{i}")
    assert not found
