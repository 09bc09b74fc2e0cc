"""The stand-alone operators captured into a CUDA graph by the first calls of
their process (kernel attributes and cluster sizes are then looked up while the
stream is capturing), and replayed on changed inputs."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import sys
sys.path.insert(0, {root!r})
import numpy as np, torch
from block_speculative_decoding_dflash2_gb300 import binding as B
from tests import sampling_reference as R

torch.manual_seed(5)
M, K, V, b, rows = 6144, 1024, 6144, 2, 4
codes = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
scale = (torch.rand((M, K // 64), device="cuda") * 0.01 + 0.01).to(torch.bfloat16)
q = torch.stack((codes & 15, codes >> 4), 2).reshape(M, K).double() - 8
w = (q.reshape(M, K // 64, 64) * scale.double()[:, :, None]).reshape(M, K)
xs = [torch.zeros((n, K), dtype=torch.bfloat16, device="cuda") for n in (b * rows, 40)]
ys = [torch.empty((n, M), device="cuda") for n in (b * rows, 40)]
path = torch.zeros((b, rows - 1), dtype=torch.int32, device="cuda")
ua, u = torch.zeros((b, rows - 1), device="cuda"), torch.zeros((b,), device="cuda")
temp, top_p = torch.full((b,), 0.8, device="cuda"), torch.full((b,), 0.9, device="cuda")
i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
acc, out, n_out, nxt, tok = i32(b), i32(b, rows), i32(b), i32(b), i32(b)
prob = torch.empty((b, rows, V), device="cuda")
ws = torch.zeros(B.dflash2_verify_logits_workspace(b, rows), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for x, y in zip(xs, ys):
        B.dflash2_linear_w4(codes, scale, 64, x, y)
    z = ys[0].view(b, rows, V)
    B.dflash2_sample(z[:, 0], temp, None, top_p, None, u, tok)
    B.dflash2_target_probs(z, temp, None, top_p, None, prob)
    B.dflash2_verify_logits(path, None, z, temp, None, top_p, None, ua, u, acc, out, n_out, nxt, ws)
for turn in range(3):
    for x in xs:
        x.copy_(torch.randn(x.shape, device="cuda"))
    u.copy_(torch.rand(u.shape, device="cuda")); ua.copy_(torch.rand(ua.shape, device="cuda") * 0.2)
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        ref = x.double() @ w.T  # fp32 sums of 64 products, 16 groups and a scaling: (64 + 16 + 2) 2^-24 of the magnitudes
        assert ((y.double() - ref).abs() <= 1e-5 * (x.double().abs() @ w.T.abs())).all()
    zv, un = z.double().cpu().numpy(), u.cpu().numpy()
    spec = (float(np.float32(0.8)), 0, float(np.float32(0.9)), 0.0)
    for s in range(b):
        mass = [R.masses(zv[s, i], *spec) for i in range(rows)]
        assert int(tok[s]) == R.draw(mass[0], un[s])
        for i in range(rows):
            p = mass[i] / mass[i].sum()
            np.testing.assert_allclose(prob[s, i].cpu().numpy(), p, rtol=2.0 ** -20, atol=2.0 ** -126)
        n, v = R.verify(zv[s], path[s].cpu().numpy(), rows - 1, spec, ua[s].cpu().numpy(), un[s])
        assert (int(acc[s]), int(nxt[s])) == (n, v)
    path.copy_(z[:, :-1].argmax(2).to(torch.int32))
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=root)], capture_output=True, text=True, timeout=300,
                       cwd=root)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
