"""The sources' read-only loads (CPU). A kernel may run beside the one before it on the stream until it
waits for that one's end, so what any kernel of the library writes is never read by a load that takes
the data for constant while the kernel lives."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PLAN = ("p.cta_seg", "p.segments", "p.groups")  # copied from the host, before any kernel that reads them


def test_only_the_plan_is_read_as_constant():
    found = 0
    for path in glob.glob(os.path.join(ROOT, "bit_kv_cache_03_gb300", "csrc", "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for what in re.findall(r"__ldg\(\s*([^)]*)", text):
            found += 1
            assert what.startswith(PLAN), (os.path.basename(path), what)
    assert found
