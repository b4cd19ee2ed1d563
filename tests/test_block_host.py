"""Host side of the gated recurrence, the block norms and the verification of drafts under the address and
undefined-behaviour sanitizers: their *_api.cpp built with g++ and stand-ins for the kernel launchers
(tests/sanitize/block_host.cpp)."""
import subprocess

from test_seq_host import CSRC
from test_sanitizers import ROOT, SAN


def test_indexes_and_workspaces_of_ragged_requests(tmp_path):
    exe = tmp_path / "host"
    subprocess.run(["g++", *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT / 'include'}",
                    str(ROOT / "tests" / "sanitize" / "block_host.cpp"),
                    *(str(CSRC / f"{n}_api.cpp") for n in ("scan", "norm", "draft")), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.stdout + r.stderr)[-2000:]
    assert r.stdout.startswith("ok")
