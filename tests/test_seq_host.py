"""Host side of prompts and beams under the address and undefined-behaviour
sanitizers: beam_api.cpp and linear_api.cpp built with g++ and stand-ins for the
kernel launchers (tests/sanitize/)."""
import subprocess
from pathlib import Path

import pytest

from test_sanitizers import ROOT, SAN

CSRC = ROOT / "quantized_recurrent_state_packed_amd" / "csrc"


def run(tmp_path: Path, source: str, api: str) -> str:
    exe = tmp_path / "host"
    subprocess.run(["g++", *SAN, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT / 'include'}",
                    str(ROOT / "tests" / "sanitize" / source), str(CSRC / api), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.stdout + r.stderr)[-2000:]
    return r.stdout


def test_selection_covers_every_vocabulary_it_accepts(tmp_path):
    assert run(tmp_path, "beam_host.cpp", "beam_api.cpp").startswith("ok")


@pytest.mark.gpu
@pytest.mark.parametrize("below", [0, 5])
def test_selection_over_the_largest_vocabulary(below):
    """2^31 - 1 - 1024 logits a row, the row's start off a 16-byte boundary: the best
    tokens stand at both ends and at the seams of its parts."""
    import torch
    from quantized_recurrent_state_packed_amd import beam as B
    vocab = 2 ** 31 - 1 - 1024 - below
    x = torch.full((vocab + 7,), -1.0, dtype=torch.bfloat16, device="cuda")[7:]
    at = [vocab - 1, 0, vocab // 2, vocab // 64, vocab - 1025]
    for rank, t in enumerate(at):
        x[t] = 40.0 - rank
    sel = B.BeamSelect(1, 1, vocab, len(at), torch.bfloat16)
    tokens, parents, scores = sel(x[None], torch.zeros(1, device="cuda"))
    torch.cuda.synchronize()
    assert tokens[0].tolist() == at and parents[0].tolist() == [0] * len(at)
    want = torch.tensor([40.0 - r for r in range(len(at))], dtype=torch.float64)
    rest = (vocab - len(at)) * torch.exp(torch.tensor(-1.0, dtype=torch.float64))
    want = want - torch.log(torch.exp(want).sum() + rest)
    assert (scores[0].double().cpu() - want).abs().max() <= 1e-5
