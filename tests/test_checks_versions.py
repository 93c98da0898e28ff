"""The native argument checks are used only with the torch and the Python that
they were built for (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from combine_ep_get_dispatch_amd.build import CHECKS, ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(CHECKS), reason="_checks.so is not built")
REFUSED = """
from combine_ep_get_dispatch_amd import binding as B
try:
    from combine_ep_get_dispatch_amd import _checks
except ImportError as e:
    assert "built for" in str(e), e
else:
    raise AssertionError("imported")
assert B._Checks is B._PyChecks and issubclass(B._Args, B._PyChecks)
x = B.torch.zeros(4)
A = B._Args("c")
assert A.arg("x", x, B._F32, 16) == x.data_ptr()
"""


def run(code):
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)


def test_as_built():
    run("from combine_ep_get_dispatch_amd import binding as B, _checks; assert B._Checks is _checks.Checks")


@pytest.mark.parametrize("other", ["torch.version.__version__ = '9.9.9'", "torch.version.git_version = '0' * 40",
                                   "del torch.version.git_version", "sys.hexversion = 0x030900F0"])
def test_another_version_falls_back(other):
    run("import sys, torch\n" + other + REFUSED)
