"""Workspaces that the logits operators cannot write are refused: by the C
entry points before any CUDA call (dummy pointers; only calls that must be
refused are made), by the binding for tensors of another device, layout or
size."""

import os

import pytest

pytestmark = pytest.mark.skipif(
    not (os.path.exists("/usr/local/cuda/bin/nvcc") or __import__("shutil").which("nvcc")),
    reason="nvcc is needed to build the library")

P = 4096  # a dummy, aligned, non-null pointer


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import build as bld
    bld.build()
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_status_words_are_refused(B, off):
    L = B.lib()
    assert L.dflash2_sample(0, 2, 100, P, 100, None, None, None, None, P, P, None, P + off, None) == -5
    assert L.dflash2_target_probs(0, 2, 3, 100, P, 100, None, None, None, None, P, P + off, None) == -5


class Fake:
    """What the check reads of a tensor."""

    def __init__(self, device=0, contiguous=True, n=256):
        self.device, self.contiguous, self.n = device, contiguous, n

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.n

    def element_size(self):
        return 1

    def data_ptr(self):
        return P


def test_the_bindings_check(B):
    assert B._workspace("f", None, 0, 256) is None
    assert B._workspace("f", P, 0, 256) == P
    assert B._workspace("f", Fake(), 0, 256) == P and B._workspace("f", Fake(n=0), 0) == P
    for bad in (Fake(device=-1), Fake(device=1), Fake(contiguous=False), Fake(n=255), Fake(n=0)):
        with pytest.raises(B.DFlash2Error) as e:
            B._workspace("f", bad, 0, 256)
        assert e.value.status == -5


@pytest.mark.gpu
def test_calls_with_such_workspaces_are_refused(B):
    import torch
    c = dict(device="cuda")
    z, u, tok = torch.zeros((3, 10), **c), torch.zeros((3,), **c), torch.zeros((3,), dtype=torch.int32, **c)
    none = (None,) * 4
    byte = dict(dtype=torch.uint8)
    bad = [torch.zeros(256, **byte), torch.zeros(512, **byte, **c)[::2], torch.zeros(255, **byte, **c),
           torch.zeros(0, **byte, **c), torch.zeros(1, **byte, **c).expand(256), torch.zeros(300, **byte, **c)[1:257]]
    for ws in bad:
        with pytest.raises(B.DFlash2Error) as e:
            B.dflash2_sample(z, *none, u, tok, None, ws)
        assert e.value.status == -5
        with pytest.raises(B.DFlash2Error) as e:
            B.dflash2_target_probs(z[:, None], *none, torch.zeros((3, 1, 10), **c), ws)
        assert e.value.status == -5
    z3, i = torch.zeros((2, 3, 10), **c), lambda *s: torch.zeros(s, dtype=torch.int32, **c)
    f = lambda *s: torch.zeros(s, **c)
    for ws in (torch.zeros(1 << 16, **byte), torch.zeros(1 << 16, **byte, **c)[::2],
               torch.zeros(1, **byte, **c).expand(1 << 16), torch.zeros(16, **byte, **c)):
        with pytest.raises(B.DFlash2Error) as e:
            B.dflash2_verify_logits(i(2, 2), None, z3, *none, f(2, 2), f(2), i(2), i(2, 3), i(2), i(2), ws)
        assert e.value.status == -5
    ok = torch.zeros(256, **byte, **c)
    B.dflash2_sample(z, *none, u, tok, None, ok)
    assert B.dflash2_read_device_status(ok) == 0 and tok.tolist() == [0, 0, 0]
