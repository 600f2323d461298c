"""Which pointers the layer operators take, without a GPU: the current device's
memory and managed memory, not another device's, whose addresses a kernel here
must not use, and not the host's."""
import os
import subprocess

import pytest

from test_plan_host import _nvcc

HERE = os.path.dirname(os.path.abspath(__file__))
UNKNOWN, HOST, DEVICE, MANAGED = 0, 1, 2, 3


@pytest.mark.parametrize("kind,device,current,taken", [
    (DEVICE, 0, 0, 1), (DEVICE, 3, 3, 1), (DEVICE, 1, 0, 0), (DEVICE, 0, 1, 0), (MANAGED, 0, 1, 1), (HOST, 0, 0, 0),
    (UNKNOWN, 0, 0, 0)])
def test_memory_of_the_current_device(tmp_path_factory, kind, device, current, taken):
    exe = os.path.join(str(tmp_path_factory.getbasetemp()), "pointer_probe")
    if not os.path.exists(exe):
        nv = _nvcc()
        if nv is None:
            pytest.skip("nvcc not found")
        r = subprocess.run([nv, "-std=c++17", "-O1", os.path.join(HERE, "pointer_probe.cu"), "-o", exe],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], input="%d %d %d\n" % (kind, device, current), capture_output=True, text=True, check=True)
    assert out.stdout.split() == [str(taken)]
