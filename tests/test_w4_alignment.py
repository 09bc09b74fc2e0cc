"""DFLASH2_W4 entry points refuse addresses that the 4-bit contraction's vector
loads cannot take, on the host and before any CUDA call (dummy pointers, never
dereferenced; every call made here is one that must be refused)."""

import ctypes
import os

import pytest

import dflash2_synth as S

pytestmark = pytest.mark.skipif(
    not (os.path.exists("/usr/local/cuda/bin/nvcc") or __import__("shutil").which("nvcc")),
    reason="nvcc is needed to build the library")

P = 4096  # a dummy, aligned, non-null pointer
MATRICES = ("tapgen_attn", "qkv", "o", "tapgen_mlp", "gate_up", "down")


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash2_gb300 import build as bld
    bld.build()
    from block_speculative_decoding_dflash2_gb300 import binding
    binding.lib()
    return binding


def config(B):
    return B.make_config(S.small_bf16_config(dtype="w4"))


def weights(B, n_layers, **off):
    """WeightSet of dummy addresses; off: name or scales_name -> bytes added
    (a layer's matrix: in the last layer only)."""
    at = lambda name, l=None: P + (off.get(name, 0) if l in (None, n_layers - 1) else 0)
    layers = [{f: at(f, l) for f in B._LAYER_FIELDS} for l in range(n_layers)]
    scales = {f: at("scales_" + f) for f in ("lm_head", "fc", "sel")}
    scales["layers"] = [{f: at("scales_" + f, l) for f in MATRICES} for l in range(n_layers)]
    return B.WeightSet({**{f: at(f) for f in B._TOP_FIELDS}, "layers": layers, "scales": scales})


def draft(B, w, taps=P, n_new=3, ws=P):
    c = config(B)
    return B.lib().dflash2_draft_step(ctypes.byref(c), ctypes.byref(w.struct), P, P, 8, P, 4, 2, P, n_new, taps, P, P, P,
                                      P, None, ws, 1 << 40, None)


def append(B, w, taps=P, n_new=3, ws=P):
    c = config(B)
    return B.lib().dflash2_append_context(ctypes.byref(c), ctypes.byref(w.struct), P, P, 8, P, 4, 2, P, n_new, taps, P,
                                          ws, 1 << 40, None)


@pytest.mark.parametrize("name,off", [(n, o) for n in ("lm_head", "fc", "sel") + MATRICES for o in (1, 2, 8)]
                         + [("scales_" + n, 1) for n in ("lm_head", "fc", "sel") + MATRICES])
def test_misaligned_weights_are_refused(B, name, off):
    w = weights(B, config(B).n_layers, **{name: off})
    assert draft(B, w) == -1 and append(B, w) == -1


def test_a_misaligned_embedding_is_refused(B):
    w = weights(B, config(B).n_layers, embed=8)
    assert draft(B, w) == -1 and append(B, w) == -1


@pytest.mark.parametrize("off", [2, 4, 8])
def test_misaligned_taps_and_workspaces_are_refused(B, off):
    w = weights(B, config(B).n_layers)
    assert draft(B, w, taps=P + off) == -1 and append(B, w, taps=P + off) == -1
    assert draft(B, w, ws=P + off) == -5 and append(B, w, ws=P + off) == -5
    assert draft(B, w, taps=None, n_new=0, ws=P + off) == -5


@pytest.mark.parametrize("name,off", [("sel", 8), ("scales_sel", 1), ("embed", 2)])
def test_misaligned_selector_weights_are_refused(B, name, off):
    c = config(B)
    w = weights(B, c.n_layers, **{name: off})
    assert B.lib().dflash2_build_selector_table(ctypes.byref(c), ctypes.byref(w.struct), P, None) == -1
    assert B.lib().dflash2_select_path(ctypes.byref(c), ctypes.byref(w.struct), 2, P, P, P, P, None, P, 1 << 40,
                                       None) == -1
    w = weights(B, c.n_layers)
    assert B.lib().dflash2_select_path(ctypes.byref(c), ctypes.byref(w.struct), 2, P, P, P, P, None, P + 8, 1 << 40,
                                       None) == -5
