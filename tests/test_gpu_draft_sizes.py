"""The drafter's product on sizes whose hidden states fill 48 KB of shared memory, what a launch may
take without asking, as a process's first call.

Each logit is a sum of H products of bf16 values in fp32, by four lanes of H / 4 each and two
joins: |z - ref| <= 2^-24 (H / 4 + 10) sum |h w|.
"""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H", [(16, 1503), (16, 1505), (16, 1531), (8, 3055), (4, 6131), (2, 12257),
                                 (1, 24550), (1, 24577)])
def test_the_first_call_of_a_process(B, H):
    code = f"""
import torch
import drafter_sampling_gb300 as vt
g = torch.Generator(device="cuda")
g.manual_seed({H})
h = torch.randn(({B}, {H}), generator=g, device="cuda").to(torch.bfloat16)
W = torch.randn((77, {H}), generator=g, device="cuda").to(torch.bfloat16)
z = vt.vt_draft_logits(h, W)
ref = h.double() @ W.double().t()
tol = 2.0 ** -24 * ({H} / 4 + 10) * (h.double().abs() @ W.double().abs().t())
assert bool(((z.double() - ref).abs() <= tol).all())
print("equal")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]
