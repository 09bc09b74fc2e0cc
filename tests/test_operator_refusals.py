"""Host-side refusals of the logits and 4-bit operators: the C entry points
return before any CUDA call (dummy pointers are never dereferenced), and the
binding refuses tensors of another type, shape or device."""

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


def test_sample_refusals(B):
    f = B.lib().dflash2_sample

    def call(dtype=0, rows=2, vocab=100, logits=P, stride=100, u=P, token=P):
        return f(dtype, rows, vocab, logits, stride, None, None, None, None, u, token, None, None, None)

    assert call(dtype=2) == -4 and call(dtype=-1) == -4
    assert call(rows=0) == -2 and call(rows=-1) == -2 and call(rows=(1 << 20) + 1) == -2
    assert call(vocab=0) == -2 and call(vocab=1048577, stride=1 << 21) == -2
    assert call(stride=99) == -2 and call(stride=-100) == -2
    assert call(logits=None) == -1 and call(u=None) == -1 and call(token=None) == -1
    assert call(logits=P + 2) == -1 and call(dtype=1, logits=P + 1) == -1


def test_target_probs_refusals(B):
    f = B.lib().dflash2_target_probs

    def call(dtype=0, batch=2, rows=3, vocab=100, logits=P, stride=100, prob=P):
        return f(dtype, batch, rows, vocab, logits, stride, None, None, None, None, prob, None, None)

    assert call(dtype=2) == -4
    assert call(batch=0) == -2 and call(rows=0) == -2 and call(batch=1 << 11, rows=1 << 10) == -2
    assert call(batch=1 << 30, rows=1 << 30) == -2
    assert call(vocab=0) == -2 and call(stride=7) == -2
    assert call(logits=None) == -1 and call(prob=None) == -1


def test_verify_logits_refusals(B):
    L = B.lib()

    def call(dtype=0, batch=2, block=4, vocab=100, path=P, logits=P, stride=100, ua=P, us=P, a=P, out=P, n=P, nxt=P,
             ws=P, ws_bytes=1 << 20):
        return L.dflash2_verify_logits(dtype, batch, block, vocab, path, None, logits, stride, None, None, None, None,
                                       ua, us, a, out, n, nxt, None, None, ws, ws_bytes, None)

    assert call(block=1) == -3 and call(block=33) == -3
    assert call(dtype=3) == -4 and call(batch=0) == -2 and call(vocab=0) == -2 and call(stride=99) == -2
    for name in ("path", "logits", "ua", "us", "a", "out", "n", "nxt"):
        assert call(**{name: None}) == -1, name
    assert call(ws=None) == -5 and call(ws=P + 8) == -5
    need = L.dflash2_verify_logits_workspace(2, 4)
    assert need >= 256 + 2 * 4 * 8 and call(ws_bytes=need - 1) == -5
    assert L.dflash2_verify_logits_workspace(0, 4) == 0
    assert L.dflash2_verify_logits_workspace(1, 1) == 0 and L.dflash2_verify_logits_workspace(1, 33) == 0


def test_linear_w4_refusals(B):
    f = B.lib().dflash2_linear_w4

    def call(codes=P, scale=P, group=64, m=8, k=128, x=P, xs=128, rows=2, out=P, os_=8, dt=0):
        return f(codes, scale, group, m, k, x, xs, rows, out, os_, dt, 0, None)

    for group in (0, 16, 48, 256, -64):
        assert call(group=group) == -2
    assert call(k=96) == -2 and call(k=0) == -2 and call(m=0) == -2 and call(rows=-1) == -2
    assert call(m=(1 << 24) + 1, os_=1 << 25) == -2 and call(k=(1 << 24) + 64, xs=1 << 25) == -2
    assert call(xs=120) == -2 and call(xs=132) == -2 and call(os_=7) == -2
    assert call(dt=2) == -4 and call(dt=-1) == -4
    for name in ("codes", "scale", "x", "out"):
        assert call(**{name: None}) == -1, name
    assert call(codes=P + 8) == -1 and call(x=P + 2) == -1 and call(scale=P + 2) == -1 and call(out=P + 2) == -1
    assert call(rows=0) == 0 and call(rows=0, x=None, out=None) == 0


def test_binding_refuses_tensors_it_cannot_pass(B):
    import torch
    z = torch.zeros((2, 10))
    i = torch.zeros((2,), dtype=torch.int32)
    u = torch.zeros((2,))
    with pytest.raises(B.DFlash2Error) as e:  # host tensors
        B.dflash2_sample(z, None, None, None, None, u, i)
    assert e.value.status == -1
    with pytest.raises(B.DFlash2Error) as e:
        B.dflash2_target_probs(z[:, None], None, None, None, None, z[:, None])
    assert e.value.status == -1
    with pytest.raises(B.DFlash2Error) as e:
        B.dflash2_verify_logits(i[:, None], None, z[:, None].expand(2, 2, 10), None, None, None, None, u[:, None], u,
                                i, i, i, i, u)
    assert e.value.status == -1
    with pytest.raises(B.DFlash2Error) as e:
        B.dflash2_linear_w4(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.bfloat16), 64,
                            torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((2, 4)))
    assert e.value.status == -1


@pytest.mark.gpu
def test_binding_refuses_types_shapes_and_layouts(B):
    import torch
    c = dict(device="cuda")
    z, u, tok = torch.zeros((3, 10), **c), torch.zeros((3,), **c), torch.zeros((3,), dtype=torch.int32, **c)

    def status(fn, *a, **k):
        with pytest.raises(B.DFlash2Error) as e:
            fn(*a, **k)
        return e.value.status

    none = (None,) * 4
    s = B.dflash2_sample
    assert status(s, z.double(), *none, u, tok) == -4
    assert status(s, z.t(), *none, torch.zeros((10,), **c), torch.zeros((10,), dtype=torch.int32, **c)) == -2
    assert status(s, z, *none, u.double(), tok) == -4
    assert status(s, z, *none, u, tok.long()) == -4
    assert status(s, z, *none, u[:2], tok) == -2
    assert status(s, z, u[:2], None, None, None, u, tok) == -2
    assert status(s, z, None, u, None, None, u, tok) == -4
    assert status(s, z, *none, u, tok, z) == -2
    assert status(s, z, *none, u, None) == -1
    assert status(s, z[0], *none, u, tok) == -2
    z3 = torch.zeros((2, 3, 10), **c)
    assert status(B.dflash2_target_probs, z3.transpose(0, 1), *none, torch.zeros((3, 2, 10), **c)) == -2
    assert status(B.dflash2_target_probs, z3, *none, z3[:, :2]) == -2
    assert status(B.dflash2_target_probs, z3, *none, z3.to(torch.bfloat16)) == -4
    codes, scale = torch.zeros((4, 64), dtype=torch.uint8, **c), torch.zeros((4, 2), dtype=torch.bfloat16, **c)
    x, out = torch.zeros((2, 128), dtype=torch.bfloat16, **c), torch.zeros((2, 4), **c)
    w = B.dflash2_linear_w4
    assert status(w, codes, scale, 64, x.float(), out) == -4
    assert status(w, codes, scale, 64, x, out.half()) == -4
    assert status(w, codes, scale, 128, x, out) == -2
    assert status(w, codes, scale, 48, x, out) == -2
    assert status(w, codes[:, :32], scale, 64, x, out) == -2
    assert status(w, codes, scale.float(), 64, x, out) == -4
    assert status(w, codes, scale, 64, x, out[:1]) == -2
    assert status(w, codes, scale, 64, x, out.t()) == -2
    assert status(w, codes, scale, 64, torch.zeros((2, 129), dtype=torch.bfloat16, **c)[:, :128], out) == -2
    assert status(w, codes, scale, 64, torch.zeros((2 * 128 + 8,), dtype=torch.bfloat16, **c)[4:260].view(2, 128),
                  out) == -1
