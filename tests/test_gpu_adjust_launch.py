"""dflash2_adjust_logits where a block's shared memory is just below 48 KB, by the first call of a process: what an
earlier call has set for the kernel does not help it.  Masks alone change the rows, so they are compared exactly."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import sys
sys.path.insert(0, {root!r})
import torch
from block_speculative_decoding_dflash2_gb300 import binding as B

batch, rows, vocab, most, biased = {args}
g = torch.Generator(device="cuda").manual_seed(1)
z = torch.randn((batch, rows, vocab), generator=g, device="cuda").bfloat16()
words = -(-vocab // 32)
mask = torch.randint(-2 ** 31, 2 ** 31, (batch, rows, words), generator=g, dtype=torch.int32, device="cuda")
tokens = torch.randint(0, vocab, (batch, most), generator=g, dtype=torch.int32, device="cuda") if most else None
n = torch.full((batch,), most, dtype=torch.int32, device="cuda") if most else None
bias_id = torch.full((batch, 1), 7, dtype=torch.int32, device="cuda") if biased else None
bias = torch.full((batch, 1), 2.0, device="cuda") if biased else None
out = torch.empty_like(z)
B.dflash2_adjust_logits(z, tokens, n, out, bias_id=bias_id, bias=bias, mask=mask)
torch.cuda.synchronize()
if biased:
    z[:, :, 7] += 2
keep = ((mask[..., None] >> torch.arange(32, device="cuda")) & 1).flatten(2)[..., :vocab] > 0
assert torch.equal(out, torch.where(keep, z, float("-inf")))
print("same")
"""


# (batch, rows, vocabulary, tokens, a bias): slices of 5952, 4736 and 3968 tokens
@pytest.mark.parametrize("args", [(128, 1, 151936, 0, False), (36, 1, 151936, 3000, False), (86, 2, 151000, 0, False),
                                  (72, 2, 151000, 0, True), (200, 1, 151936, 8, True)])
def test_first_call_of_a_process(args):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=root, args=args)], capture_output=True, text=True,
                       timeout=300, cwd=root)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
