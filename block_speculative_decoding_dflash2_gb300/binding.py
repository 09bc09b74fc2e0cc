"""ctypes binding of libdflash2.so: argument marshalling only.

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it turns torch tensors into device pointers, Python
numbers into C ints/floats, and raises ``DFlash2Error`` on a non-OK status.
There is no fallback: without the built library, loading raises.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdflash2.so")
TEST_LIB_PATH = os.path.join(_PKG, "libdflash2_testing.so")

F32 = 0
BF16 = 1
FP8W = 2
W4 = 3
W4_GROUP = 64
STATUS_BYTES = 256  # of a workspace that only its status word is used of

STATUS = {0: "ok", -1: "invalid argument", -2: "shape", -3: "block size", -4: "dtype",
          -5: "workspace", -6: "cuda", -7: "unsupported"}
DEV_BAD_PAGE, DEV_BAD_TOKEN, DEV_WAIT_TIMEOUT, DEV_BAD_LENGTH, DEV_EMPTY_ROW = 0x1, 0x2, 0x4, 0x8, 0x10


class DFlash2Error(RuntimeError):
    def __init__(self, fn, status, text):
        super().__init__(f"{fn} failed: status {status} ({text})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "hidden", "n_q_heads", "n_kv_heads", "head_dim", "intermediate", "vocab",
        "n_layers", "n_taps", "block_size", "conv_kernel_size", "conv_group_size",
        "top_k", "selector_rank", "page_size", "mask_token_id", "dtype")] + \
        [(n, ctypes.c_float) for n in (
            "rms_eps", "rope_theta", "input_embedding_scale", "output_multiplier",
            "final_logit_softcap")] + [("sliding_window", ctypes.c_int)]


_LAYER_FIELDS = ("attn_norm", "tapgen_attn", "qkv", "q_norm", "k_norm", "o", "mlp_norm",
                 "tapgen_mlp", "gate_up", "down")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LAYER_FIELDS]


_TOP_FIELDS = ("embed", "lm_head", "fc", "hidden_norm", "final_norm", "sel")


_LAYER_SCALE_FIELDS = ("tapgen_attn", "qkv", "o", "tapgen_mlp", "gate_up", "down")


class LayerScales(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LAYER_SCALE_FIELDS]


class Scales(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("lm_head", "fc", "sel")] + \
        [("layers", ctypes.POINTER(LayerScales))]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _TOP_FIELDS] + [("layers", ctypes.POINTER(LayerWeights)),
                                                              ("scales", ctypes.POINTER(Scales))]


_lib = None
_tlib = None


def testing_lib():
    """The test-hook library (include/dflash2_testing.h), loaded after the
    product library it links against."""
    global _tlib
    if _tlib is None:
        lib()
        if not os.path.exists(TEST_LIB_PATH):
            raise ImportError(f"{TEST_LIB_PATH} is missing: build it with __graft_entry__.build()")
        T = ctypes.CDLL(TEST_LIB_PATH)
        P, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER
        T.dflash2_test_last_schedule.restype = I
        T.dflash2_test_last_schedule.argtypes = []
        T.dflash2_test_gemm_workspace.restype = S
        T.dflash2_test_gemm_workspace.argtypes = [I, I]
        T.dflash2_test_gemm.restype = I
        T.dflash2_test_gemm.argtypes = [I, P, I, I, P, I, I, I, P, P, S, P]
        T.dflash2_test_gemm_fp8.restype = I
        T.dflash2_test_force_cluster_split.restype = I
        T.dflash2_test_force_cluster_split.argtypes = [I]
        T.dflash2_test_force_attention.restype = I
        T.dflash2_test_force_attention.argtypes = [I]
        T.dflash2_test_w4_withhold.restype = I
        T.dflash2_test_w4_withhold.argtypes = [I]
        T.dflash2_test_last_attention.restype = I
        T.dflash2_test_last_attention.argtypes = []
        T.dflash2_test_gemm_fp8.argtypes = [P, P, I, I, P, I, I, I, P, P, S, P]
        T.dflash2_test_layout.restype = I
        T.dflash2_test_layout.argtypes = [F(Config), I, I, I, F(ctypes.c_size_t), I]
        T.dflash2_test_topk_workspace.restype = S
        T.dflash2_test_topk_workspace.argtypes = [I, I, I]
        T.dflash2_test_gemm_topk.restype = I
        T.dflash2_test_gemm_topk.argtypes = [I, P, I, I, P, I, I, ctypes.c_float, ctypes.c_float, P, P, P,
                                             P, S, P]
        _tlib = T
    return _tlib


def lib():
    """The loaded library (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(the product path has no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER
        L.dflash2_status_string.restype = ctypes.c_char_p
        L.dflash2_status_string.argtypes = [I]
        L.dflash2_version.restype = I
        L.dflash2_validate_config.restype = I
        L.dflash2_validate_config.argtypes = [F(Config)]
        L.dflash2_workspace_size.restype = S
        L.dflash2_workspace_size.argtypes = [F(Config), I, I, I]
        L.dflash2_append_context.restype = I
        L.dflash2_append_context.argtypes = [F(Config), F(Weights), P, P, I, P, I, I, P, I, P, P, P, S, P]
        L.dflash2_draft_step.restype = I
        L.dflash2_draft_step.argtypes = [F(Config), F(Weights), P, P, I, P, I, I, P, I, P, P, P,
                                         P, P, P, P, S, P]
        L.dflash2_select_path.restype = I
        L.dflash2_select_path.argtypes = [F(Config), F(Weights), I, P, P, P, P, P, P, S, P]
        L.dflash2_verify_accept.restype = I
        L.dflash2_verify_accept.argtypes = [I, I, P, P, P, P, P, P, P, P, P]
        L.dflash2_read_device_status.restype = I
        L.dflash2_read_device_status.argtypes = [P, S, P]
        L.dflash2_select_path_static.restype = I
        L.dflash2_select_path_static.argtypes = [F(Config), F(Weights), I, P, P, P, P, P, P]
        L.dflash2_select_path_static_capacity.restype = S
        L.dflash2_select_path_static_read_status.restype = I
        L.dflash2_select_path_static_read_status.argtypes = [P]
        L.dflash2_selector_table_bytes.restype = S
        L.dflash2_selector_table_bytes.argtypes = [F(Config)]
        L.dflash2_build_selector_table.restype = I
        L.dflash2_build_selector_table.argtypes = [F(Config), F(Weights), P, P]
        L.dflash2_select_path_table.restype = I
        L.dflash2_select_path_table.argtypes = [F(Config), I, P, P, P, P, P, P, P, P]
        L.dflash2_select_path_table_ex.restype = I
        L.dflash2_select_path_table_ex.argtypes = [F(Config), I, P, P, P, P, F(DraftOpts), P, P, P, P, P]
        L.dflash2_select_path_ex.restype = I
        L.dflash2_select_path_ex.argtypes = [F(Config), F(Weights), I, P, P, P, F(DraftOpts), P, P, P, P, S, P]
        L.dflash2_select_top1.restype = I
        L.dflash2_select_top1.argtypes = [F(Config), I, P, P, F(DraftOpts), P, P, P, P, P]
        L.dflash2_verify_sampled.restype = I
        L.dflash2_verify_sampled.argtypes = [I, I, I, P, P, P, P, P, P, P, P, P, P, P, P]
        L.dflash2_verify_accept_ex.restype = I
        L.dflash2_verify_accept_ex.argtypes = [I, I, P, P, P, P, P, P, P, P, P, P]
        I64 = ctypes.c_int64
        L.dflash2_sample.restype = I
        L.dflash2_sample.argtypes = [I, I, I, P, I64] + [P] * 9
        L.dflash2_target_probs.restype = I
        L.dflash2_target_probs.argtypes = [I, I, I, I, P, I64] + [P] * 7
        L.dflash2_verify_logits_workspace.restype = S
        L.dflash2_verify_logits_workspace.argtypes = [I, I]
        L.dflash2_verify_logits.restype = I
        L.dflash2_verify_logits.argtypes = [I, I, I, I, P, P, P, I64] + [P] * 13 + [S, P]
        L.dflash2_linear_w4.restype = I
        L.dflash2_linear_w4.argtypes = [P, P, I, I, I, P, I64, I, P, I64, I, I, P]
        L.dflash2_launch_count.restype = ctypes.c_int64
        L.dflash2_set_stage_events.restype = None
        L.dflash2_set_stage_events.argtypes = [P]
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:  # the handle of torch's current stream, without building a Stream around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, rc):
    if rc != 0:
        raise DFlash2Error(fn, rc, lib().dflash2_status_string(rc).decode())
    return rc


def make_config(d):
    """Config struct from a dict with the header's field names (extra keys ignored)."""
    c = Config()
    for name, _ in Config._fields_:
        v = d.get(name, 0) if name == "sliding_window" else d[name]
        if name == "dtype" and isinstance(v, str):
            v = {"f32": F32, "bf16": BF16, "fp8w": FP8W, "w4": W4}[v]
        setattr(c, name, v)
    return c


class DraftOpts(ctypes.Structure):
    _fields_ = [("n_max", ctypes.c_int), ("p_min", ctypes.c_float)]


class WeightSet:
    """Holds a Weights struct over torch device tensors (kept alive here);
    tensors["scales"] (fp8 and 4-bit weights) fills its Scales struct."""

    def __init__(self, tensors):
        self.tensors = tensors
        n = len(tensors["layers"])
        self._layers = (LayerWeights * n)()
        for i, L in enumerate(tensors["layers"]):
            for f in _LAYER_FIELDS:
                setattr(self._layers[i], f, _ptr(L[f]))
        scales = None
        sc = tensors.get("scales")
        if sc is not None:
            self._layer_scales = (LayerScales * n)()
            for i, L in enumerate(sc["layers"]):
                for f in _LAYER_SCALE_FIELDS:
                    setattr(self._layer_scales[i], f, _ptr(L[f]))
            self._scales = Scales(*[_ptr(sc[f]) for f in ("lm_head", "fc", "sel")],
                                  ctypes.cast(self._layer_scales, ctypes.POINTER(LayerScales)))
            scales = ctypes.pointer(self._scales)
        self.struct = Weights(*[_ptr(tensors[f]) for f in _TOP_FIELDS],
                              ctypes.cast(self._layers, ctypes.POINTER(LayerWeights)), scales)


def dflash2_status_string(status):
    return lib().dflash2_status_string(status).decode()


def dflash2_version():
    return lib().dflash2_version()


def dflash2_validate_config(cfg):
    return lib().dflash2_validate_config(ctypes.byref(cfg))


def dflash2_workspace_size(cfg, max_batch, max_new_rows, max_ctx):
    return lib().dflash2_workspace_size(ctypes.byref(cfg), max_batch, max_new_rows, max_ctx)


def dflash2_append_context(cfg, w, k_cache, v_cache, n_pages, block_table, max_pages, batch, ctx_len,
                           n_new, new_taps, new_off, workspace, stream=None):
    return _check("dflash2_append_context", lib().dflash2_append_context(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(k_cache), _ptr(v_cache), n_pages,
        _ptr(block_table), max_pages, batch, _ptr(ctx_len), n_new, _ptr(new_taps), _ptr(new_off),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_draft_step(cfg, w, k_cache, v_cache, n_pages, block_table, max_pages, batch, ctx_len,
                       n_new, new_taps, new_off, anchor, cand_id, cand_logit, debug_logits,
                       workspace, stream=None):
    return _check("dflash2_draft_step", lib().dflash2_draft_step(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(k_cache), _ptr(v_cache), n_pages,
        _ptr(block_table), max_pages, batch, _ptr(ctx_len), n_new, _ptr(new_taps), _ptr(new_off),
        _ptr(anchor), _ptr(cand_id), _ptr(cand_logit), _ptr(debug_logits),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_select_path(cfg, w, batch, anchor, cand_id, cand_logit, path, path_score, workspace,
                        stream=None):
    return _check("dflash2_select_path", lib().dflash2_select_path(
        ctypes.byref(cfg), ctypes.byref(w.struct), batch, _ptr(anchor), _ptr(cand_id),
        _ptr(cand_logit), _ptr(path), _ptr(path_score), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_selector_table_bytes(cfg):
    return lib().dflash2_selector_table_bytes(ctypes.byref(cfg))


def dflash2_build_selector_table(cfg, w, table, stream=None):
    return _check("dflash2_build_selector_table", lib().dflash2_build_selector_table(
        ctypes.byref(cfg), ctypes.byref(w.struct), _ptr(table), _stream(stream)))


def dflash2_select_path_table(cfg, batch, anchor, cand_id, cand_logit, table, path, path_score,
                              workspace=None, stream=None):
    return _check("dflash2_select_path_table", lib().dflash2_select_path_table(
        ctypes.byref(cfg), batch, _ptr(anchor), _ptr(cand_id), _ptr(cand_logit), _ptr(table), _ptr(path),
        _ptr(path_score), _ptr(workspace), _stream(stream)))


def _opts(n_max, p_min):
    return ctypes.byref(DraftOpts(int(n_max), float(p_min)))


def dflash2_select_path_ex(cfg, w, batch, anchor, cand_id, cand_logit, n_max, p_min, path, path_score, n_draft,
                           workspace, stream=None):
    return _check("dflash2_select_path_ex", lib().dflash2_select_path_ex(
        ctypes.byref(cfg), ctypes.byref(w.struct), batch, _ptr(anchor), _ptr(cand_id), _ptr(cand_logit),
        _opts(n_max, p_min), _ptr(path), _ptr(path_score), _ptr(n_draft), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_select_path_table_ex(cfg, batch, anchor, cand_id, cand_logit, table, n_max, p_min, path, path_score,
                                 n_draft, workspace=None, stream=None):
    return _check("dflash2_select_path_table_ex", lib().dflash2_select_path_table_ex(
        ctypes.byref(cfg), batch, _ptr(anchor), _ptr(cand_id), _ptr(cand_logit), _ptr(table), _opts(n_max, p_min),
        _ptr(path), _ptr(path_score), _ptr(n_draft), _ptr(workspace), _stream(stream)))


def dflash2_select_top1(cfg, batch, cand_id, cand_logit, n_max, p_min, path, path_score, n_draft, workspace=None,
                        stream=None):
    return _check("dflash2_select_top1", lib().dflash2_select_top1(
        ctypes.byref(cfg), batch, _ptr(cand_id), _ptr(cand_logit), _opts(n_max, p_min), _ptr(path),
        _ptr(path_score), _ptr(n_draft), _ptr(workspace), _stream(stream)))


def dflash2_verify_sampled(batch, block_size, vocab, path, n_draft, target_prob, u_accept, u_sample, accept_len,
                           out_tok, n_out, next_anchor, seq_len=None, counters=None, stream=None):
    return _check("dflash2_verify_sampled", lib().dflash2_verify_sampled(
        batch, block_size, vocab, _ptr(path), _ptr(n_draft), _ptr(target_prob), _ptr(u_accept), _ptr(u_sample),
        _ptr(accept_len), _ptr(out_tok), _ptr(n_out), _ptr(next_anchor), _ptr(seq_len), _ptr(counters),
        _stream(stream)))


# The operators below read their sizes from the tensors, so they check them:
# a tensor of another type, shape or layout, or on another device than the
# current one, is refused before the call.

def _refuse(fn, name, t, dev, dtype, shape):
    if t is None or t.get_device() != dev or dev < 0:
        raise DFlash2Error(fn, -1, f"{name} must be on the current device")
    if t.dtype is not dtype:
        raise DFlash2Error(fn, -4, f"{name} must be {dtype}")
    raise DFlash2Error(fn, -2, f"{name} must be contiguous, of shape {tuple(shape)}")


def _at(fn, name, t, dev, dtype, shape):
    """Address of a contiguous tensor of this type and shape on device dev."""
    if (t is None or t.get_device() != dev or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _refuse(fn, name, t, dev, dtype, shape)
    return t.data_ptr()


def _workspace(fn, ws, dev, least=0):
    """Address of a workspace (or None, or a raw address): contiguous, on
    device dev, of at least `least` bytes."""
    if ws is None or isinstance(ws, int):
        return ws
    if ws.get_device() != dev or not ws.is_contiguous():
        raise DFlash2Error(fn, -5, "workspace must be contiguous and on the current device")
    if ws.numel() * ws.element_size() < least:
        raise DFlash2Error(fn, -5, f"workspace must have at least {least} bytes")
    return ws.data_ptr()


_LOGIT_TYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _rows_of(fn, name, t, dims):
    """(device, type code, distance of the rows) of a [..., n] tensor on the
    current device whose rows are evenly spaced."""
    dev = -1 if t is None else t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise DFlash2Error(fn, -1, f"{name} must be on the current device")
    code = _LOGIT_TYPES.get(t.dtype)
    if code is None:
        raise DFlash2Error(fn, -4, f"{name} must be float32 or bfloat16")
    st, sz = t.stride(), t.shape
    if len(sz) != dims or (st[-1] != 1 and sz[-1] > 1):
        raise DFlash2Error(fn, -2, f"{name} must have {dims} dimensions, the last one contiguous")
    if dims == 2:
        return dev, code, st[0] if sz[0] > 1 else sz[1]
    row = st[1] if sz[1] > 1 else (st[0] if sz[0] > 1 else sz[2])
    if sz[0] > 1 and sz[1] > 1 and st[0] != sz[1] * row:
        raise DFlash2Error(fn, -2, f"the rows of {name} must be evenly spaced")
    return dev, code, row


def _settings(fn, dev, n, temperature, top_k, top_p, min_p):
    f32, shape = torch.float32, (n,)
    return (None if temperature is None else _at(fn, "temperature", temperature, dev, f32, shape),
            None if top_k is None else _at(fn, "top_k", top_k, dev, torch.int32, shape),
            None if top_p is None else _at(fn, "top_p", top_p, dev, f32, shape),
            None if min_p is None else _at(fn, "min_p", min_p, dev, f32, shape))


def dflash2_sample(logits, temperature, top_k, top_p, min_p, u, token, prob=None, workspace=None, stream=None):
    """logits: [rows, vocab] float32 or bfloat16, rows evenly spaced; the
    settings: [rows] tensors or None; u, token, prob: [rows]."""
    fn = "dflash2_sample"
    dev, code, stride = _rows_of(fn, "logits", logits, 2)
    n, vocab = logits.shape
    return _check(fn, lib().dflash2_sample(
        code, n, vocab, logits.data_ptr(), stride, *_settings(fn, dev, n, temperature, top_k, top_p, min_p),
        _at(fn, "u", u, dev, torch.float32, (n,)), _at(fn, "token", token, dev, torch.int32, (n,)),
        None if prob is None else _at(fn, "prob", prob, dev, torch.float32, (n,)),
        _workspace(fn, workspace, dev, STATUS_BYTES), _stream(stream)))


def dflash2_target_probs(logits, temperature, top_k, top_p, min_p, prob, workspace=None, stream=None):
    """logits: [batch, rows, vocab] float32 or bfloat16, rows evenly spaced;
    the settings: [batch] tensors or None; prob: [batch, rows, vocab] float32."""
    fn = "dflash2_target_probs"
    dev, code, stride = _rows_of(fn, "logits", logits, 3)
    batch, rows, vocab = logits.shape
    return _check(fn, lib().dflash2_target_probs(
        code, batch, rows, vocab, logits.data_ptr(), stride,
        *_settings(fn, dev, batch, temperature, top_k, top_p, min_p),
        _at(fn, "prob", prob, dev, torch.float32, logits.shape), _workspace(fn, workspace, dev, STATUS_BYTES),
        _stream(stream)))


def dflash2_verify_logits_workspace(batch, block_size):
    return lib().dflash2_verify_logits_workspace(batch, block_size)


def dflash2_verify_logits(path, n_draft, logits, temperature, top_k, top_p, min_p, u_accept, u_sample, accept_len,
                          out_tok, n_out, next_anchor, workspace, seq_len=None, counters=None, stream=None):
    """logits: [batch, block_size, vocab] float32 or bfloat16, rows evenly
    spaced; path, u_accept: [batch, block_size - 1]; the settings: [batch]
    tensors or None."""
    fn = "dflash2_verify_logits"
    dev, code, stride = _rows_of(fn, "logits", logits, 3)
    batch, B, vocab = logits.shape
    i32, f32, one, drafts = torch.int32, torch.float32, (batch,), (batch, B - 1)
    if workspace is None:
        raise DFlash2Error(fn, -5, "workspace must be on the current device")
    ws = _workspace(fn, workspace, dev)
    return _check(fn, lib().dflash2_verify_logits(
        code, batch, B, vocab, _at(fn, "path", path, dev, i32, drafts),
        None if n_draft is None else _at(fn, "n_draft", n_draft, dev, i32, one), logits.data_ptr(), stride,
        *_settings(fn, dev, batch, temperature, top_k, top_p, min_p),
        _at(fn, "u_accept", u_accept, dev, f32, drafts), _at(fn, "u_sample", u_sample, dev, f32, one),
        _at(fn, "accept_len", accept_len, dev, i32, one), _at(fn, "out_tok", out_tok, dev, i32, (batch, B)),
        _at(fn, "n_out", n_out, dev, i32, one), _at(fn, "next_anchor", next_anchor, dev, i32, one),
        None if seq_len is None else _at(fn, "seq_len", seq_len, dev, i32, one),
        None if counters is None else _at(fn, "counters", counters, dev, torch.int64, (4 + 2 * B - 1,)),
        ws, workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_linear_w4(codes, scale, group, x, out, accumulate=False, stream=None):
    """codes: [out_features, in_features / 2] uint8; scale: [out_features,
    in_features / group] bfloat16; x: [rows, in_features] bfloat16, out:
    [rows, out_features] float32 or bfloat16, both with evenly spaced rows."""
    fn = "dflash2_linear_w4"
    dev, xcode, x_stride = _rows_of(fn, "x", x, 2)
    _, code, out_stride = _rows_of(fn, "out", out, 2)
    if xcode != BF16:
        raise DFlash2Error(fn, -4, "x must be bfloat16")
    n, k = x.shape
    rows, m = out.shape
    if group not in (32, 64, 128) or k % group or rows != n:
        raise DFlash2Error(fn, -2, "group must be 32, 64 or 128 and divide in_features, x and out have as many rows")
    return _check(fn, lib().dflash2_linear_w4(
        _at(fn, "codes", codes, dev, torch.uint8, (m, k // 2)),
        _at(fn, "scale", scale, dev, torch.bfloat16, (m, k // group)), group, m, k, x.data_ptr(), x_stride, n,
        out.data_ptr(), out_stride, code, int(accumulate), _stream(stream)))


def dflash2_verify_accept_ex(batch, block_size, path, n_draft, target, accept_len, out_tok, n_out, next_anchor,
                             seq_len=None, counters=None, stream=None):
    return _check("dflash2_verify_accept_ex", lib().dflash2_verify_accept_ex(
        batch, block_size, _ptr(path), _ptr(n_draft), _ptr(target), _ptr(accept_len), _ptr(out_tok), _ptr(n_out),
        _ptr(next_anchor), _ptr(seq_len), _ptr(counters), _stream(stream)))


def dflash2_verify_accept(batch, block_size, path, target, accept_len, out_tok, n_out, next_anchor,
                          seq_len=None, counters=None, stream=None):
    return _check("dflash2_verify_accept", lib().dflash2_verify_accept(
        batch, block_size, _ptr(path), _ptr(target), _ptr(accept_len), _ptr(out_tok), _ptr(n_out),
        _ptr(next_anchor), _ptr(seq_len), _ptr(counters), _stream(stream)))


def dflash2_read_device_status(workspace, stream=None):
    rc = lib().dflash2_read_device_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream))
    if rc < 0:
        _check("dflash2_read_device_status", rc)
    return rc


# --------------------------------------------------------------- test hooks
# (include/dflash2_testing.h: the internal contraction and the lm_head top-k
# path on their own, for parity tests)

def dflash2_test_gemm_workspace(M, N):
    return testing_lib().dflash2_test_gemm_workspace(M, N)


def dflash2_test_gemm(dtype, W, X, ctas, out, workspace, accumulate=False, stream=None):
    """ctas: 0 = the library's schedule, > 0 = stream-K over that many CTAs,
    -1 = whole tiles, -2..-8 = cluster split-K of -ctas slices per tile.
    Returns the CTA count launched."""
    M, K = W.shape
    N = X.shape[0]
    rc = testing_lib().dflash2_test_gemm(dtype, _ptr(W), M, K, _ptr(X), N, ctas, int(accumulate), _ptr(out),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc < 0:
        _check("dflash2_test_gemm", rc)
    return rc


def dflash2_test_force_cluster_split(cs):
    """Force cluster split-K of cs slices on the library's own contractions
    (0 = its own schedule)."""
    _check("dflash2_test_force_cluster_split", testing_lib().dflash2_test_force_cluster_split(int(cs)))


def dflash2_test_force_attention(mode):
    """Attention kernel of later draft steps: 0 the library's choice, 1 the
    mma.sync cluster kernel, 2 the tcgen05 kernel wherever it applies."""
    _check("dflash2_test_force_attention", testing_lib().dflash2_test_force_attention(int(mode)))


def dflash2_test_last_attention():
    """Attention kernel of the last draft step: 1 mma.sync cluster, 2
    tcgen05, 3 SIMT (0 before any)."""
    return int(testing_lib().dflash2_test_last_attention())


def dflash2_test_gemm_fp8(W8, scale, X, ctas, out, workspace, accumulate=False, stream=None):
    """W8: uint8 e4m3 codes [M, K]; scale: float32 [M]; X: bf16 [N, K]."""
    M, K = W8.shape
    N = X.shape[0]
    rc = testing_lib().dflash2_test_gemm_fp8(_ptr(W8), _ptr(scale), M, K, _ptr(X), N, ctas, int(accumulate), _ptr(out),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc < 0:
        _check("dflash2_test_gemm_fp8", rc)
    return rc


def dflash2_test_topk_workspace(dtype, M, N):
    return testing_lib().dflash2_test_topk_workspace(dtype, M, N)


def dflash2_test_gemm_topk(dtype, W, X, k, mult, cap, cand_id, cand_logit, debug, workspace, stream=None):
    M, K = W.shape
    N = X.shape[0]
    return _check("dflash2_test_gemm_topk", testing_lib().dflash2_test_gemm_topk(
        dtype, _ptr(W), M, K, _ptr(X), N, k, mult, cap, _ptr(cand_id), _ptr(cand_logit), _ptr(debug),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def dflash2_test_layout(cfg, batch, n_new, max_ctx):
    """Workspace byte offsets of {f, h, u, u2, q, kb, vb, O, act, hn, ua, u2a, cnt, cnta}."""
    out = (ctypes.c_size_t * 14)()
    _check("dflash2_test_layout", testing_lib().dflash2_test_layout(ctypes.byref(cfg), batch, n_new, max_ctx, out, 14))
    return dict(zip(("f", "h", "u", "u2", "q", "kb", "vb", "O", "act", "hn", "ua", "u2a", "cnt", "cnta"),
                    list(out)))


SCHED_FUSED_PROLOGUE, SCHED_SPLIT_SMS, SCHED_FUSED_QKV, SCHED_KV_BESIDE_QKV, SCHED_MERGED = 1, 2, 4, 8, 16


def dflash2_test_last_schedule():
    """Schedule bits (SCHED_*) of the last draft step in this process."""
    return testing_lib().dflash2_test_last_schedule()


def dflash2_launch_count():
    return lib().dflash2_launch_count()


def dflash2_set_stage_events(events):
    """events: None, or 5 torch.cuda.Event(enable_timing=True) already recorded once.

    Returns a holder that the caller keeps alive for as long as the library
    (or a graph captured while the events were set) may record into them."""
    if events is None:
        lib().dflash2_set_stage_events(None)
        return None
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    lib().dflash2_set_stage_events(ctypes.cast(arr, ctypes.c_void_p))
    # a graph captured with these events records into them at every replay:
    # the holder keeps the event objects (not only their handles) alive
    return (arr, tuple(events))


def dflash2_select_path_static(cfg, w, batch, anchor, cand_id, cand_logit, path, path_score, stream=None):
    """dflash2_select_path for callers that cannot allocate device memory: the
    library's own fixed scratch array replaces the workspace (see the header)."""
    return _check("dflash2_select_path_static", lib().dflash2_select_path_static(
        ctypes.byref(cfg), ctypes.byref(w.struct), batch, _ptr(anchor), _ptr(cand_id), _ptr(cand_logit),
        _ptr(path), _ptr(path_score), _stream(stream)))


def dflash2_select_path_static_capacity():
    return lib().dflash2_select_path_static_capacity()


def dflash2_select_path_static_read_status(stream=None):
    """Device status word (DFLASH2_DEV_* bits) of the last static selector
    call on the current device, read and cleared; synchronises the stream."""
    rc = lib().dflash2_select_path_static_read_status(_stream(stream))
    if rc < 0:
        _check("dflash2_select_path_static_read_status", rc)
    return rc
