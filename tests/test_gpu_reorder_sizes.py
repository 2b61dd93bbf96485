"""vt_beam_reorder of 16-byte vectors for every number of beams: the shared memory that a launch takes
grows with it."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as m
    from drafter_sampling_gb300 import build
    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("W", [23, 24, 25, 31, 32])
def test_the_first_call_of_a_process(vt, W):
    code = f"""
import torch
import drafter_sampling_gb300 as vt
state = torch.arange(3 * {W} * 512, device="cuda", dtype=torch.int32).view(3, {W}, 512)
parent = torch.arange({W}, device="cuda", dtype=torch.int32).flip(0).expand(3, {W}).contiguous()
want = state.flip(1)
out, st = vt.vt_beam_reorder(state, parent, torch.zeros_like(state))
assert torch.equal(out, want) and int(st.item()) == 0
out, st = vt.vt_beam_reorder(state, parent)
assert torch.equal(out, want) and int(st.item()) == 0
print("equal")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("row", [4, 8, 12, 64])     # bytes: vectors of 4, 8, 4 and 16
def test_every_number_of_beams(vt, row):
    g = torch.Generator(device="cuda")
    g.manual_seed(row)
    for W in range(1, 33):
        state = torch.randint(0, 256, (3, W, 37, row), generator=g, device="cuda", dtype=torch.uint8)
        parent = torch.randint(0, W, (3, W), generator=g, device="cuda", dtype=torch.int32)
        want = state.gather(1, parent.long()[:, :, None, None].expand_as(state))
        out, st = vt.vt_beam_reorder(state, parent, torch.zeros_like(state))
        assert torch.equal(out, want) and int(st.item()) == 0
        out, st = vt.vt_beam_reorder(state, parent)
        assert torch.equal(out, want) and int(st.item()) == 0
