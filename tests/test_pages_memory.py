"""The count of a cache's pages when host memory is short (CPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The process may have no more memory than it has after taking the pages and a little for the
# lists; the free pages need up to 16 MB of their own as they grow.
DROP_ALL = """
import resource
import numpy as np
import decode_gemm_bf16_amd as uw

n = 1 << 22
p = uw.Pages(n)
a = p.take(n)
used = int(open('/proc/self/statm').read().split()[0]) * resource.getpagesize()
limit = used + (4 << 20)
resource.setrlimit(resource.RLIMIT_AS, (limit, limit))
for i in range(0, n, 4096):
    left = p.left
    try:
        p.drop(a[i:i + 4096])
    except uw.UwError as e:  # a refused call changes nothing
        assert e.status == uw.ERR_OOM and p.left == left and p.holders(int(a[i])) == 1, (i, p.left, left)
        break
else:
    assert p.left == n and p.take(3).tolist() == [0, 1, 2]
print("ended", i)
"""


def test_a_refused_drop_changes_nothing():
    r = subprocess.run([sys.executable, "-c", DROP_ALL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ended" in r.stdout, r.stdout + r.stderr
