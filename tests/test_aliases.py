"""Pointers that the header allows to be the same: a kernel must not promise the
compiler that they are apart, since it could then store before it loads (no GPU needed)."""
import os
import re
import subprocess

import pytest

from nvfp4_w4a16_mtp_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Parameters of every kernel of moe_sort.hip, as the compiler takes them."""
    out = str(tmp_path_factory.mktemp("ir") / "out.ll")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-emit-llvm", "-S",
                        os.path.join(build.CSRC, "moe_sort.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = {}
    for name, params in re.findall(r"^define [^\n]*amdgpu_kernel void @(\w+)\(([^\n]*)\)[^()\n]* #[^\n]*\{$", open(out).read(), re.M):
        found[name] = re.split(r", (?=ptr|i\d+)", params)
    return found


def test_the_gradient_in_place(kernels):
    """dys (parameter 7) may be ys (1); nothing else is written where it is read."""
    grads = {n: p for n, p in kernels.items() if "k_moe_combine_grad" in n}
    assert len(grads) == 8
    for name, p in grads.items():
        assert len(p) == 9 and all("noalias" in p[i] for i in (0, 5, 6, 8)), (name, p)
        assert not any("noalias" in p[i] for i in (1, 7)), name
