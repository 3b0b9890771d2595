"""CPU check of the compiled kernels: a load straight to LDS takes its LDS address
from m0 and needs one instruction (or s_nop) between the write of m0 and itself."""

import os
import re
import subprocess

from bit_e8_lattice_amd import build


def _instructions(source, tmp_path):
    out = tmp_path / "device.s"
    cmd = [build.hipcc()] + build.FLAGS + ["-I", build.INCLUDE, "-I", build.CSRC, "-S", "--cuda-device-only",
                                           os.path.join(build.CSRC, source), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        if line and not line.endswith(":") and not line.startswith("."):
            yield line


def test_wait_state_after_m0(tmp_path):
    loads, since = 0, None                       # instructions since m0 was written
    for line in _instructions("e8q_orthogonal.hip", tmp_path):
        if re.match(r"global_load_lds|buffer_load_\w+ .*\blds\b", line):
            loads += 1
            assert since is not None and since >= 1, line
        if re.match(r"s_\w+ m0,", line):
            since = 0
        elif since is not None:
            since += 1
    assert loads > 100
