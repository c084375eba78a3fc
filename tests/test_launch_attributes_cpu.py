"""A kernel's limit of dynamic shared memory is an attribute of the function, not of a launch: two host
threads that set different values for one kernel can make each other's launch fail.  So the value that a
source file sets may not depend on the call's sizes."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_prologue_b200", "csrc")


def test_limits_of_shared_memory_do_not_depend_on_the_call():
    sizes = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            src = f.read()
        for m in re.finditer(r"cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^;]*)\);", src):
            size = m.group(1).strip()
            if size.isidentifier() and not size.startswith("k"):  # a local: how it is made
                made = re.findall(rf"\bint {size} = ([^;]*);", src[:m.start()])
                assert made, (path, size)
                size = made[-1]
            sizes.append((os.path.basename(path), size))
    assert len(sizes) >= 8
    constant = re.compile(r"\(int\)(sizeof\([\w<>, ]+\)|[A-Z]\w*(<\w+>)?(::k?[bB]ytes)?)|k[A-Z]\w*")
    for path, size in sizes:
        assert constant.fullmatch(size), (path, size)
