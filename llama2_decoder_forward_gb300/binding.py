"""Python binding of the C ABI in include/llama_gb300.h.

Argument marshalling only: every step of the forward pass runs in the CUDA
library. PyTorch tensors supply device memory and the stream; their data
pointers go through ctypes. If the shared library is missing the binding
raises at once; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os

from .build import CHECKED_LIB
from .build import LIB as _MAIN_LIB

# LLAMA_GB300_BOUNDS_CHECK=1 selects the bounds-check build of the same sources
LIB = CHECKED_LIB if os.environ.get("LLAMA_GB300_BOUNDS_CHECK") == "1" else _MAIN_LIB

c_int32 = ctypes.c_int32
c_void_p = ctypes.c_void_p

F32, BF16 = 0, 1
EPI_STORE_F32, EPI_RESID_F32, EPI_STORE_T, EPI_SWIGLU = 0, 1, 2, 3
EPI_SPLIT_X = 16  # OR-ed flag: x (and bf16 outputs) in the hi/lo pair layout
KERNELS = ("rmsnorm", "gemm", "rope_append", "attn_decode", "attn_prefill", "embed", "argmax",
           "sample")
FLAG_TOKEN_RANGE, FLAG_POS_RANGE, FLAG_PAGE_RANGE, FLAG_WAIT_TIMEOUT, FLAG_INDEX = 1, 2, 4, 8, 16
STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "OUT_OF_RANGE", 4: "CUDA",
          5: "DEVICE_CHECK", 6: "WORKSPACE"}


class LlamaConfig(ctypes.Structure):
    _fields_ = [("n_layers", c_int32), ("hidden", c_int32), ("n_q_heads", c_int32),
                ("n_kv_heads", c_int32), ("head_dim", c_int32), ("intermediate", c_int32),
                ("vocab", c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("dtype", c_int32), ("max_batch", c_int32), ("max_tokens", c_int32),
                ("max_seq", c_int32), ("has_embed_head", c_int32), ("weight_dtype", c_int32)]


LAYER_MATS = ("attn_norm", "wqkv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")
PROJECTIONS = ("wqkv", "wo", "w_gate", "w_up", "w_down")
W_MODEL, W_E4M3 = 0, 1


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in LAYER_MATS] + [(n + "_scale", c_void_p) for n in PROJECTIONS]


class Weights(ctypes.Structure):
    _fields_ = [("embed", c_void_p), ("final_norm", c_void_p), ("lm_head", c_void_p),
                ("layers", ctypes.POINTER(LayerWeights))]


class Sampling(ctypes.Structure):
    """llama_sampling: temperature (0 = greedy), top_k (<= 0 off), top_p (1 = off),
    repetition_penalty (1 = off)."""
    _fields_ = [("temperature", ctypes.c_float), ("top_k", c_int32), ("top_p", ctypes.c_float),
                ("repetition_penalty", ctypes.c_float)]


ALL_LAYERS = -1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BANDS = 0, 1, 2
ROPE_ADJACENT, ROPE_HALF = 0, 1


class RopeScaling(ctypes.Structure):
    """llama_rope_scaling: kind ROPE_PLAIN, ROPE_LINEAR or ROPE_BANDS."""
    _fields_ = [("kind", c_int32), ("theta", ctypes.c_float), ("factor", ctypes.c_float),
                ("low_turns", ctypes.c_float), ("high_turns", ctypes.c_float),
                ("original_len", c_int32), ("magnitude", ctypes.c_float)]


class _Rope(ctypes.Structure):
    _fields_ = [("layout", c_int32), ("rotary_dim", c_int32), ("table", c_void_p),
                ("n_pos", c_int32)]


class _Scores(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("cap", ctypes.c_float), ("slopes", c_void_p)]


KV_MODEL, KV_E4M3 = 0, 1


class KV(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("page_size", c_int32), ("capacity", c_int32),
                ("batch_capacity", c_int32), ("n_pages", c_int32), ("page_table", c_void_p),
                ("max_pages_per_seq", c_int32), ("kv_dtype", c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


_SIGS = {
    "llama_workspace_bytes": (c_int32, [ctypes.POINTER(LlamaConfig), ctypes.POINTER(ctypes.c_size_t)]),
    "llama_workspace_least_bytes": (c_int32, [ctypes.POINTER(LlamaConfig),
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "llama_init": (c_int32, [ctypes.POINTER(LlamaConfig), ctypes.POINTER(Weights), c_void_p,
                             ctypes.c_size_t, c_void_p, ctypes.POINTER(c_void_p)]),
    "llama_set_stream": (c_int32, [c_void_p, c_void_p]),
    "llama_prefill": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, ctypes.POINTER(KV), c_void_p,
                                c_void_p]),
    "llama_decode_step": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, ctypes.POINTER(KV),
                                    c_void_p, c_void_p]),
    "llama_decode_step_host": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, ctypes.POINTER(KV),
                                         c_void_p, c_void_p]),
    "llama_prefill_hidden": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, ctypes.POINTER(KV)]),
    "llama_decode_hidden": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, ctypes.POINTER(KV)]),
    "llama_extend": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                               ctypes.POINTER(KV), c_void_p, c_void_p]),
    "llama_extend_hidden": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                      c_int32, ctypes.POINTER(KV)]),
    "llama_graph_capture_decode": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, ctypes.POINTER(KV),
                                             c_void_p, c_void_p, c_int32]),
    "llama_graph_launch": (c_int32, [c_void_p]),
    "llama_sync_status": (c_int32, [c_void_p]),
    "llama_last_device_flags": (ctypes.c_uint32, [c_void_p]),
    "llama_check_wait_timeout": (c_int32, [c_void_p, c_int32]),
    "llama_quantize_rows_e4m3": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                           c_void_p]),
    "llama_bounds_checked": (c_int32, []),
    "llama_strerror": (ctypes.c_char_p, [c_int32]),
    "llama_free": (c_int32, [c_void_p]),
    "llama_profile_enable": (c_int32, [c_void_p, ctypes.c_uint32]),
    "llama_profile_read": (c_int32, [c_void_p, c_int32, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int64)]),
    "llama_launch_count": (ctypes.c_int64, [c_void_p]),
    "llama_op_rmsnorm": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p]),
    "llama_op_linear": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                  c_int32, c_void_p]),
    "llama_op_rope_append": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int32,
                                       ctypes.POINTER(KV), c_void_p, c_void_p, c_void_p]),
    "llama_op_attention_decode": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                            ctypes.POINTER(KV), c_void_p]),
    "llama_attention_decode_noalloc": (c_int32, [ctypes.POINTER(LlamaConfig), c_void_p, c_void_p, c_int32,
                                                 c_int32, ctypes.POINTER(KV), c_void_p, c_void_p]),
    "llama_op_attention_prefill": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                             c_void_p]),
    "llama_op_embed": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p]),
    "llama_rope_table": (c_int32, [ctypes.POINTER(RopeScaling), c_int32, c_int32, c_void_p,
                                   c_void_p]),
    "llama_op_rope_norm_append": (c_int32, [c_void_p, c_void_p, c_int32, ctypes.c_int64, c_int32,
                                            c_void_p, c_void_p, c_int32, ctypes.POINTER(_Rope),
                                            c_void_p, c_void_p, ctypes.c_float, c_int32,
                                            ctypes.POINTER(KV), c_void_p, c_void_p, c_void_p]),
    "llama_op_attention_docs": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p,
                                          c_int32, c_void_p, ctypes.POINTER(_Scores), c_void_p]),
    "llama_op_attention_decode_shared": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                                   ctypes.POINTER(KV), c_int32, c_int32,
                                                   ctypes.POINTER(_Scores), c_void_p]),
    "llama_op_rope_norm_append_at": (c_int32, [c_void_p, c_void_p, c_int32, ctypes.c_int64, c_int32,
                                               c_void_p, c_void_p, c_int32, c_void_p,
                                               ctypes.POINTER(_Rope), c_void_p, c_void_p,
                                               ctypes.c_float, c_int32, ctypes.POINTER(KV), c_void_p,
                                               c_void_p, c_void_p]),
    "llama_op_attention_decode_weights": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                                    ctypes.POINTER(KV), ctypes.POINTER(_Scores),
                                                    c_void_p, ctypes.c_int64, c_void_p, c_void_p]),
    "llama_op_attention_tree": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                          c_void_p, c_int32, c_void_p, c_int32, ctypes.POINTER(KV),
                                          ctypes.POINTER(_Scores), c_void_p]),
    "llama_op_cache_commit": (c_int32, [c_void_p, ctypes.POINTER(KV), c_int32, c_void_p, c_int32,
                                        c_void_p, c_int32, c_void_p]),
    "llama_op_cache_evict": (c_int32, [c_void_p, ctypes.POINTER(KV), c_int32, c_void_p, c_int32, c_int32,
                                       c_int32, c_int32, c_void_p, ctypes.c_int64, c_void_p, c_void_p]),
    "llama_op_argmax": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p]),
    "llama_sample": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, ctypes.POINTER(Sampling), c_void_p,
                               c_void_p, c_int32, c_void_p, c_void_p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError("%s is not built (run llama2_decoder_forward_gb300.build."
                               "build_library() or __graft_entry__.build())" % os.path.basename(LIB))
        l = ctypes.CDLL(LIB)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def exported_symbols():
    return list(_SIGS)


class LlamaError(RuntimeError):
    def __init__(self, rc, what, flags=0):
        self.rc = rc
        self.flags = flags
        msg = "%s failed: %s (%s)" % (what, STATUS.get(rc, rc), lib().llama_strerror(rc).decode())
        if flags:
            msg += " device flags 0x%x" % flags
        super().__init__(msg)


def _p(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return c_void_p(s.cuda_stream)


def make_config(shape, max_batch, max_tokens, max_seq, has_embed_head=True,
                weight_dtype=W_MODEL) -> LlamaConfig:
    return LlamaConfig(shape.n_layers, shape.hidden, shape.n_q_heads, shape.n_kv_heads,
                       shape.head_dim, shape.intermediate, shape.vocab if has_embed_head else 0,
                       shape.rms_eps, shape.rope_theta, F32 if shape.dtype == "f32" else BF16,
                       max_batch, max_tokens, max_seq, 1 if has_embed_head else 0, weight_dtype)


def quantize_rows_e4m3(w, stream=None):
    """E4M3 codes (uint8 [rows, cols]) and per-row fp32 scales of a bf16 device
    matrix, by the library's quantiser (llama_quantize_rows_e4m3)."""
    import torch
    w = w.contiguous()
    rows, cols = w.shape
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=w.device)
    scales = torch.empty(rows, dtype=torch.float32, device=w.device)
    rc = lib().llama_quantize_rows_e4m3(_p(w), rows, cols, _p(codes), _p(scales),
                                        _stream_handle(stream))
    if rc:
        raise LlamaError(rc, "llama_quantize_rows_e4m3")
    return codes, scales


def quantize_layer_e4m3(lw, stream=None):
    """A layer's weight dict with its five projections as E4M3 codes plus
    "<name>_scale" row scales (norm gains unchanged)."""
    out = dict(lw)
    for n in PROJECTIONS:
        out[n], out[n + "_scale"] = quantize_rows_e4m3(lw[n], stream)
    return out


def workspace_bytes(cfg: LlamaConfig) -> int:
    n = ctypes.c_size_t(0)
    rc = lib().llama_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n))
    if rc:
        raise LlamaError(rc, "llama_workspace_bytes")
    return n.value


def workspace_least_bytes(cfg: LlamaConfig) -> int:
    n = ctypes.c_size_t(0)
    rc = lib().llama_workspace_least_bytes(ctypes.byref(cfg), ctypes.byref(n))
    if rc:
        raise LlamaError(rc, "llama_workspace_least_bytes")
    return n.value


def rope_table(n_pos, rotary_dim, *, theta=10000.0, kind=ROPE_PLAIN, factor=1.0, low_turns=1.0,
               high_turns=32.0, original_len=4096, magnitude=1.0, stream=None):
    """Rotation angles of scaled positions (llama_rope_table): a device tensor
    [n_pos, rotary_dim / 2, 2] of fp32 (cos, sin), for Rope."""
    import torch
    if n_pos < 1 or rotary_dim < 8 or rotary_dim % 8:
        raise ValueError("rope_table: n_pos %r, rotary_dim %r" % (n_pos, rotary_dim))
    table = torch.empty(n_pos, rotary_dim // 2, 2, dtype=torch.float32, device="cuda")
    sc = RopeScaling(kind, theta, factor, low_turns, high_turns, original_len, magnitude)
    rc = lib().llama_rope_table(ctypes.byref(sc), rotary_dim, n_pos, _p(table),
                                _stream_handle(stream))
    if rc:
        raise LlamaError(rc, "llama_rope_table")
    return table


class _Kept:
    """Keeps the C struct of its attributes until one of them is assigned; tensors'
    addresses are read at every call."""

    def __setattr__(self, name, value):
        d = self.__dict__
        d[name] = value
        d["_c"] = None

    def _keep(self, c):
        d = self.__dict__
        d["_c"], d["_ref"] = c, ctypes.byref(c)
        return c


class Rope(_Kept):
    """How heads rotate (llama_rope). table: [n_pos, rotary_dim / 2, 2] fp32 from
    rope_table, or None for the context's own (whole heads). Keeps the table alive."""

    def __init__(self, table=None, layout=ROPE_ADJACENT, rotary_dim=None):
        if table is None and rotary_dim is None:
            raise ValueError("Rope: without a table give rotary_dim (the head size)")
        self.table, self.layout = table, layout
        self.rotary_dim = 2 * table.shape[1] if rotary_dim is None and table.dim() == 3 else rotary_dim
        self._struct()

    def _struct(self):
        import torch
        t = self.table
        if t is None:
            return self._keep(_Rope(self.layout, self.rotary_dim, None, 0))
        if t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 3 or t.shape[2] != 2:
            raise ValueError("Rope: the table is a contiguous fp32 [n_pos, rotary_dim / 2, 2]")
        if self.rotary_dim not in (0, 2 * t.shape[1]):
            raise ValueError("Rope: rotary_dim %d, the table has %d pairs" % (self.rotary_dim, t.shape[1]))
        return self._keep(_Rope(self.layout, self.rotary_dim, t.data_ptr(), t.shape[0]))

    def _now(self, dev):
        """The C struct of the present attributes; ValueError unless the table is on device dev."""
        c, t = self._c or self._struct(), self.table
        if t is not None:
            if t.get_device() != dev:
                raise ValueError("rope: the table is not on cuda:%d" % dev)
            c.table = t.data_ptr()
        return self._ref


class Scores(_Kept):
    """Score options (llama_scores): scale (0: 1/sqrt(d)), cap (0: none), slopes
    fp32 [n_q] on the device or None. Keeps the slopes alive."""

    def __init__(self, scale=0.0, cap=0.0, slopes=None):
        import torch
        if slopes is not None and (slopes.dtype != torch.float32 or not slopes.is_contiguous()):
            raise ValueError("Scores: slopes are a contiguous fp32 tensor")
        self.scale, self.cap, self.slopes = scale, cap, slopes

    def _now(self, dtype, n_q, dev):
        """The C struct of the present attributes; ValueError unless the slopes are
        n_q values of dtype on device dev."""
        c, t = self._c or self._keep(_Scores(self.scale, self.cap, None)), self.slopes
        if t is not None:
            c.slopes = _need("slopes", t, dtype, n_q, dev)
        return self._ref


def _need(what, t, dtype, n, dev):
    """The tensor's address; ValueError unless it is a contiguous tensor of that
    type and element count on device number dev."""
    if t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s: want a contiguous tensor of %d %s on cuda:%d, got %s %s on %s%s" %
                     (what, n, dtype, dev, tuple(t.shape), t.dtype, t.device,
                      "" if t.is_contiguous() else " (strided)"))


class KVCache(_Kept):
    """Caller-owned KV cache in the library's layout (torch device memory).

    contiguous: k, v [n_layers, batch, n_kv, capacity, d]
    paged     : k, v [n_layers, n_pages, n_kv, page_size, d] + page_table [B, max_pages] int32
    e4m3=(k_scale, v_scale): one FP8 E4M3 byte per value (uint8 tensors), read
    back as e4m3 * scale.
    """

    def __init__(self, shape, *, batch=None, capacity=None, n_pages=None, page_size=0,
                 page_table=None, dtype=None, device="cuda", k=None, v=None, e4m3=None):
        import torch
        self.kv_dtype = KV_E4M3 if e4m3 else KV_MODEL
        self.k_scale, self.v_scale = e4m3 if e4m3 else (1.0, 1.0)
        dt = torch.uint8 if e4m3 else (dtype or shape.torch_dtype)
        L, nkv, d = shape.n_layers, shape.n_kv_heads, shape.head_dim
        self.page_size = page_size
        self.page_table = page_table
        if page_size == 0:
            full = (L, batch, nkv, capacity, d)
            self.batch, self.capacity, self.n_pages, self.max_pages = batch, capacity, 0, 0
        else:
            full = (L, n_pages, nkv, page_size, d)
            self.batch, self.capacity, self.n_pages = 0, 0, n_pages
            self.max_pages = page_table.shape[1]
        self.k = k if k is not None else torch.zeros(full, dtype=dt, device=device)
        self.v = v if v is not None else torch.zeros(full, dtype=dt, device=device)
        assert tuple(self.k.shape) == full and tuple(self.v.shape) == full

    def _struct(self, shape, dtype):
        """The struct of the present attributes; ValueError unless the tensors are of the
        layout's type and cover it, and the page table is as wide as it says."""
        import torch
        rows = self.n_pages * self.page_size if self.page_size else self.batch * self.capacity
        need, pt = shape.n_layers * shape.n_kv_heads * shape.head_dim * rows, self.page_table
        for t in (self.k, self.v):
            if t.numel() < need or not t.is_contiguous() or \
                    (t.dtype is not dtype if self.kv_dtype == KV_MODEL else t.element_size() != 1):
                raise ValueError("cache: want contiguous k and v of %d %s, got %s %s%s" %
                                 (need, dtype if self.kv_dtype == KV_MODEL else "E4M3 bytes", tuple(t.shape),
                                  t.dtype, "" if t.is_contiguous() else " (strided)"))
        if self.page_size and (pt is None or pt.dtype != torch.int32 or pt.dim() != 2 or
                               pt.shape[1] != self.max_pages or not pt.is_contiguous()):
            raise ValueError("cache: want a contiguous int32 page table of max_pages = %d columns, got %s" %
                             (self.max_pages, None if pt is None else "%s %s" % (tuple(pt.shape), pt.dtype)))
        d = self.__dict__
        d["_shape"], d["_rows"] = shape, pt.shape[0] if self.page_size else 1 << 31
        return self._keep(self.struct())

    def _now(self, shape, dtype, B, dev):
        """The C struct of the present attributes for a call on B sequences of a model of
        this shape and type; ValueError unless they fit and are on device dev."""
        c, k, v, pt = self._c, self.k, self.v, self.page_table
        if c is None or self._shape is not shape:
            c = self._struct(shape, dtype)
        if k.get_device() != dev or v.get_device() != dev or \
                (pt is not None and pt.get_device() != dev):
            raise ValueError("cache: not on cuda:%d" % dev)
        if B > self._rows:
            raise ValueError("cache: %d sequences, the page table has %d rows" % (B, self._rows))
        c.k, c.v = k.data_ptr(), v.data_ptr()
        if pt is not None:
            c.page_table = pt.data_ptr()
        return self._ref

    def struct(self) -> KV:
        return KV(self.k.data_ptr(), self.v.data_ptr(), self.page_size, self.capacity, self.batch,
                  self.n_pages, None if self.page_table is None else self.page_table.data_ptr(),
                  self.max_pages, self.kv_dtype, self.k_scale, self.v_scale)


class Model:
    """A library context over device-resident weights.

    weights: dict as produced by synth.model_weights / layer_weights, already
    on the GPU ({"embed", "final_norm", "lm_head", "layers": [...]}); a
    layer-only model passes {"layers": [...]} and has_embed_head=False.
    Layers made by quantize_layer_e4m3 (E4M3 projections with row scales)
    select weight_dtype LLAMA_W_E4M3. tree_room=False leaves out the part of the workspace
    that op_attention_tree alone needs to run on every SM (llama_workspace_least_bytes).
    """

    def __init__(self, shape, weights, *, max_batch, max_tokens, max_seq, has_embed_head=True,
                 stream=None, tree_room=True):
        import torch
        self.shape = shape
        self.weights = weights  # keep the tensors alive
        self._bind(shape)
        layers = weights["layers"]
        if len(layers) != shape.n_layers:
            raise ValueError("shape has %d layers, weights have %d" % (shape.n_layers, len(layers)))
        # E4M3 projections (quantize_layer_e4m3) carry "<name>_scale" entries
        w8 = "wqkv_scale" in layers[0]
        self.cfg = make_config(shape, max_batch, max_tokens, max_seq, has_embed_head,
                               W_E4M3 if w8 else W_MODEL)
        nbytes = workspace_bytes(self.cfg) if tree_room else workspace_least_bytes(self.cfg)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        arr = (LayerWeights * len(layers))()
        for i, lw in enumerate(layers):
            scales = [lw[n + "_scale"].data_ptr() if w8 else None for n in PROJECTIONS]
            arr[i] = LayerWeights(*([lw[n].data_ptr() for n in LAYER_MATS] + scales))
        self._layers_arr = arr
        w = Weights(_p(weights.get("embed")), _p(weights.get("final_norm")), _p(weights.get("lm_head")),
                    ctypes.cast(arr, ctypes.POINTER(LayerWeights)))
        ctx = c_void_p()
        rc = lib().llama_init(ctypes.byref(self.cfg), ctypes.byref(w), _p(self.workspace), nbytes,
                              _stream_handle(stream), ctypes.byref(ctx))
        if rc:
            raise LlamaError(rc, "llama_init")
        self.ctx = ctx

    def _bind(self, shape):
        """What the attention-form calls look up every time."""
        import torch
        l = lib()
        self._append, self._docs = l.llama_op_rope_norm_append, l.llama_op_attention_docs
        self._tree = l.llama_op_attention_tree
        self._append_at, self._weights = l.llama_op_rope_norm_append_at, l.llama_op_attention_decode_weights
        self._shared = l.llama_op_attention_decode_shared
        self._dt, self._qkv_rows = shape.torch_dtype, shape.qkv_rows
        self._i32, self._f32 = torch.int32, torch.float32
        self._dev = torch.cuda.current_device() if torch.cuda.is_available() else 0

    def __del__(self):
        ctx = getattr(self, "ctx", None)
        if ctx is not None and _lib is not None:
            _lib.llama_free(ctx)
            self.ctx = None

    def _chk(self, rc, what):
        if rc:
            raise LlamaError(rc, what)

    def set_stream(self, stream):
        self._chk(lib().llama_set_stream(self.ctx, _stream_handle(stream)), "llama_set_stream")

    # ---- forward pass
    def prefill(self, tokens, kv: KVCache, logits, next_ids=None):
        B, T = tokens.shape
        self._chk(lib().llama_prefill(self.ctx, _p(tokens), B, T, ctypes.byref(kv.struct()),
                                      _p(logits), _p(next_ids)), "llama_prefill")

    def extend(self, tokens, cu_rows, start_pos, kv: KVCache, logits, next_ids=None,
               max_rows=None):
        """Continuous-batching step (llama_extend): tokens [n_rows] packed by
        cu_rows [B+1] (device int32), sequence b's first row at start_pos[b]."""
        B = start_pos.shape[0]
        if max_rows is None:
            max_rows = int((cu_rows[1:] - cu_rows[:-1]).max())
        self._chk(lib().llama_extend(self.ctx, _p(tokens), tokens.shape[0], _p(cu_rows),
                                     _p(start_pos), B, max_rows, ctypes.byref(kv.struct()),
                                     _p(logits), _p(next_ids)), "llama_extend")

    def extend_hidden(self, hidden, cu_rows, start_pos, kv: KVCache, max_rows=None):
        B = start_pos.shape[0]
        if max_rows is None:
            max_rows = int((cu_rows[1:] - cu_rows[:-1]).max())
        self._chk(lib().llama_extend_hidden(self.ctx, _p(hidden), hidden.shape[0], _p(cu_rows),
                                            _p(start_pos), B, max_rows,
                                            ctypes.byref(kv.struct())), "llama_extend_hidden")

    def decode_step(self, tokens, positions, kv: KVCache, logits, next_ids=None):
        self._chk(lib().llama_decode_step(self.ctx, _p(tokens), _p(positions), tokens.shape[0],
                                          ctypes.byref(kv.struct()), _p(logits), _p(next_ids)),
                  "llama_decode_step")

    def decode_step_host(self, tokens, positions, kv: KVCache, logits=None, next_ids=None):
        rc = lib().llama_decode_step_host(self.ctx, _p(tokens), _p(positions), tokens.shape[0],
                                          ctypes.byref(kv.struct()), _p(logits), _p(next_ids))
        if rc:
            raise LlamaError(rc, "llama_decode_step_host", lib().llama_last_device_flags(self.ctx))

    def capture_decode(self, tokens, positions, kv: KVCache, logits, next_ids=None, advance=False):
        """Capture one decode step into a CUDA graph (the context's stream must be a
        non-default stream, see set_stream). Keep the buffers alive while replaying."""
        self._graph_args = (tokens, positions, kv, logits, next_ids)
        self._graph_kv = kv.struct()
        self._chk(lib().llama_graph_capture_decode(self.ctx, _p(tokens), _p(positions), tokens.shape[0],
                                                   ctypes.byref(self._graph_kv), _p(logits),
                                                   _p(next_ids), 1 if advance else 0),
                  "llama_graph_capture_decode")

    def graph_launch(self):
        self._chk(lib().llama_graph_launch(self.ctx), "llama_graph_launch")

    def prefill_hidden(self, hidden, B, T, kv: KVCache):
        self._chk(lib().llama_prefill_hidden(self.ctx, _p(hidden), B, T, ctypes.byref(kv.struct())),
                  "llama_prefill_hidden")

    def decode_hidden(self, hidden, positions, kv: KVCache):
        self._chk(lib().llama_decode_hidden(self.ctx, _p(hidden), _p(positions), hidden.shape[0],
                                            ctypes.byref(kv.struct())), "llama_decode_hidden")

    def sync(self):
        """Synchronise; raise LlamaError carrying the device flags on a kernel-side check."""
        rc = lib().llama_sync_status(self.ctx)
        if rc:
            raise LlamaError(rc, "llama_sync_status", lib().llama_last_device_flags(self.ctx))

    def sync_status(self):
        rc = lib().llama_sync_status(self.ctx)
        return rc, lib().llama_last_device_flags(self.ctx)

    def check_wait_timeout(self, limit_us):
        """Enqueue the bounded-wait check (a wait that runs out after limit_us)."""
        self._chk(lib().llama_check_wait_timeout(self.ctx, int(limit_us)), "llama_check_wait_timeout")

    # ---- profiling
    def profile(self, kinds):
        mask = 0
        for k in kinds:
            mask |= 1 << KERNELS.index(k)
        self._chk(lib().llama_profile_enable(self.ctx, mask), "llama_profile_enable")

    def profile_read(self, kind):
        ms = ctypes.c_double()
        n = ctypes.c_int64()
        self._chk(lib().llama_profile_read(self.ctx, KERNELS.index(kind), ctypes.byref(ms),
                                           ctypes.byref(n)), "llama_profile_read")
        return ms.value, n.value

    def launch_count(self):
        return lib().llama_launch_count(self.ctx)

    # ---- single operations
    def op_rmsnorm(self, x, gamma, out, rows=None, stride=1, offset=0):
        rows = rows if rows is not None else x.shape[0]
        self._chk(lib().llama_op_rmsnorm(self.ctx, _p(x), rows, stride, offset, _p(gamma), _p(out)),
                  "llama_op_rmsnorm")

    def op_linear(self, x, w, out, epilogue, w_up=None, n_rows=None):
        """n_rows: logical activation rows (defaults to x.shape[0]; give it for the
        hi/lo pair layout, whose tensor has 2 * round16(n_rows) rows)."""
        M, K = w.shape
        n = x.shape[0] if n_rows is None else n_rows
        self._chk(lib().llama_op_linear(self.ctx, _p(x), n, _p(w), _p(w_up), M, K, epilogue,
                                        _p(out)), "llama_op_linear")

    def op_rope_append(self, qkv, rows_per_seq, positions, layer, kv: KVCache, q_out, k_out=None,
                       v_out=None):
        self._chk(lib().llama_op_rope_append(self.ctx, _p(qkv), qkv.shape[0], rows_per_seq,
                                             _p(positions), layer, ctypes.byref(kv.struct()),
                                             _p(q_out), _p(k_out), _p(v_out)), "llama_op_rope_append")

    def op_attention_decode(self, q, positions, layer, kv: KVCache, out):
        self._chk(lib().llama_op_attention_decode(self.ctx, _p(q), _p(positions), q.shape[0], layer,
                                                  ctypes.byref(kv.struct()), _p(out)),
                  "llama_op_attention_decode")

    def op_attention_prefill(self, q, k, v, B, T, out):
        self._chk(lib().llama_op_attention_prefill(self.ctx, _p(q), _p(k), _p(v), B, T, _p(out)),
                  "llama_op_attention_prefill")

    def op_rope_norm_append(self, qkv, start_pos, layer, kv: KVCache, q_out, *, rope=None,
                            cu_rows=None, q_gain=None, k_gain=None, eps=None, k_out=None,
                            v_out=None, positions=None):
        """Head norms, rotation and KV append of packed rows (llama_op_rope_norm_append).
        qkv [n_rows, (n_q + 2 n_kv) d], fp32 or the model's dtype, rows may be
        strided; start_pos int32 [B]; cu_rows int32 [B + 1], or None for one row
        per sequence; eps defaults to the model's rms_eps; positions int32 [n_rows]
        that the rows rotate by (llama_op_rope_norm_append_at), or None: their slots."""
        s, dt = self.shape, self._dt
        i32, f32, dev = self._i32, self._f32, self._dev
        n, width = qkv.shape
        B, d, qdt, ld = start_pos.numel(), s.head_dim, qkv.dtype, qkv.stride()
        if (qdt is not f32 and qdt is not dt) or width != self._qkv_rows or ld[1] != 1 or \
                qkv.get_device() != dev:
            raise ValueError("qkv: want rows of %d %s or fp32 on cuda:%d, got %s %s on %s"
                             % (s.qkv_rows, dt, dev, tuple(qkv.shape), qdt, qkv.device))
        # what the two entry points share: up to the sequences, and behind them
        head = (self.ctx, qkv.data_ptr(), F32 if qdt is f32 else BF16, ld[0], n,
                None if cu_rows is None else _need("cu_rows", cu_rows, i32, B + 1, dev),
                _need("start_pos", start_pos, i32, B, dev), B)
        rest = (None if rope is None else rope._now(dev),
                None if q_gain is None else _need("q_gain", q_gain, dt, d, dev),
                None if k_gain is None else _need("k_gain", k_gain, dt, d, dev),
                s.rms_eps if eps is None else eps, layer, kv._now(s, dt, B, dev),
                _need("q_out", q_out, dt, n * s.n_q_heads * d, dev),
                None if k_out is None else _need("k_out", k_out, dt, n * s.n_kv_heads * d, dev),
                None if v_out is None else _need("v_out", v_out, dt, n * s.n_kv_heads * d, dev))
        if positions is None:
            rc = self._append(*head, *rest)
        else:
            rc = self._append_at(*head, _need("positions", positions, i32, n, dev), *rest)
        if rc:
            raise LlamaError(rc, "llama_op_rope_norm_append")

    def op_attention_docs(self, q, k, v, cu_rows, out, *, prefix=None, scores=None):
        """Prompt attention over packed documents (llama_op_attention_docs): q
        [n_rows, n_q, d], k and v [n_rows, n_kv, d], cu_rows int32 [B + 1]; prefix
        int32 [B] rows attended both ways; scores a Scores."""
        s, dt, i32, dev = self.shape, self._dt, self._i32, self._dev
        n, B = q.shape[0], cu_rows.numel() - 1
        qn, kn = n * s.n_q_heads * s.head_dim, n * s.n_kv_heads * s.head_dim
        rc = self._docs(
            self.ctx, _need("q", q, dt, qn, dev), _need("k", k, dt, kn, dev), _need("v", v, dt, kn, dev), n,
            _need("cu_rows", cu_rows, i32, B + 1, dev), B,
            None if prefix is None else _need("prefix", prefix, i32, B, dev),
            None if scores is None else scores._now(self._f32, s.n_q_heads, dev), _need("out", out, dt, qn, dev))
        if rc:
            raise LlamaError(rc, "llama_op_attention_docs")

    def op_attention_decode_shared(self, q, positions, layer, kv: KVCache, out, *, shared_len=0,
                                   shared_seq=0, scores=None):
        """Decode attention over a cache whose first shared_len positions are
        sequence shared_seq's for the whole batch (llama_op_attention_decode_shared)."""
        s, dt, dev = self.shape, self._dt, self._dev
        B = positions.numel()
        qn = B * s.n_q_heads * s.head_dim
        rc = self._shared(
            self.ctx, _need("q", q, dt, qn, dev), _need("positions", positions, self._i32, B, dev), B, layer,
            kv._now(s, dt, B, dev), shared_len, shared_seq, None if scores is None else scores._now(self._f32, s.n_q_heads, dev),
            _need("out", out, dt, qn, dev))
        if rc:
            raise LlamaError(rc, "llama_op_attention_decode_shared")

    def op_attention_tree(self, q, cu_rows, start_pos, layer, kv: KVCache, out, *, mask=None, positions=None,
                          scores=None):
        """Attention of drafted rows over a cache (llama_op_attention_tree): q [n_rows, n_q, d]
        packed by cu_rows int32 [B + 1], row i of sequence b in slot start_pos[b] + i; mask
        int32 [n_rows, words], bit j % 32 of word j // 32 for row j of the same
        sequence, or None for chains; positions int32 [n_rows], for a distance bias."""
        s, dt, i32, dev = self.shape, self._dt, self._i32, self._dev
        n, B = q.shape[0], start_pos.numel()
        qn, words = n * s.n_q_heads * s.head_dim, 0
        if mask is not None:
            if mask.dim() != 2 or mask.shape[1] < 1:
                raise ValueError("mask: want [n_rows, words], got %s" % (tuple(mask.shape),))
            words = mask.shape[1]
        rc = self._tree(
            self.ctx, _need("q", q, dt, qn, dev), n, _need("cu_rows", cu_rows, i32, B + 1, dev),
            _need("start_pos", start_pos, i32, B, dev), B,
            None if mask is None else _need("mask", mask, i32, n * words, dev), words,
            None if positions is None else _need("positions", positions, i32, n, dev), layer,
            kv._now(s, dt, B, dev), None if scores is None else scores._now(self._f32, s.n_q_heads, dev),
            _need("out", out, dt, qn, dev))
        if rc:
            raise LlamaError(rc, "llama_op_attention_tree")

    def op_attention_decode_weights(self, q, positions, layer, kv: KVCache, out, weights, scratch, *,
                                    scores=None):
        """Decode attention that adds every key's softmax weight, summed over the query heads
        of its K/V head, to weights fp32 [B, n_kv, ld] (llama_op_attention_decode_weights).
        scratch: fp32 [B, n_q, ld] or more, its contents free."""
        s, dt, f32, dev = self.shape, self._dt, self._f32, self._dev
        B, ld = positions.numel(), weights.shape[-1]
        qn = B * s.n_q_heads * s.head_dim
        if scratch.numel() < B * s.n_q_heads * ld:
            raise ValueError("scratch: want %d values, got %d" % (B * s.n_q_heads * ld, scratch.numel()))
        rc = self._weights(
            self.ctx, _need("q", q, dt, qn, dev), _need("positions", positions, self._i32, B, dev), B, layer,
            kv._now(s, dt, B, dev), None if scores is None else scores._now(f32, s.n_q_heads, dev),
            _need("weights", weights, f32, B * s.n_kv_heads * ld, dev), ld,
            _need("scratch", scratch, f32, scratch.numel(), dev), _need("out", out, dt, qn, dev))
        if rc:
            raise LlamaError(rc, "llama_op_attention_decode_weights")

    def op_cache_commit(self, kv: KVCache, start_pos, path, path_len, *, layer=None):
        """Moves the accepted rows of a drafted tree together (llama_op_cache_commit): path
        int32 [B, W] ascending rows of each sequence's tree, path_len int32 [B] how many,
        start_pos int32 [B] the slot of row 0; layer None: every layer."""
        i32, dev = self._i32, self._dev
        B, W = path.shape
        rc = lib().llama_op_cache_commit(
            self.ctx, kv._now(self.shape, self._dt, B, dev), ALL_LAYERS if layer is None else layer,
            _need("start_pos", start_pos, i32, B, dev), B, _need("path", path, i32, B * W, dev), W,
            _need("path_len", path_len, i32, B, dev))
        if rc:
            raise LlamaError(rc, "llama_op_cache_commit")

    def op_cache_evict(self, kv: KVCache, lens, keep, weights, kept, *, layer=None, first=0, recent=0,
                       weights_out=None):
        """Keeps `keep` slots of every sequence that has more (llama_op_cache_evict): the
        first, the recent and the heaviest between. lens int32 [B] filled slots; weights
        fp32 [layers, B, n_kv, ld] (one layer: [B, n_kv, ld] will do) and weights_out, which
        may be the same (None); kept int32 [layers, B, n_kv, keep]; layer None: every layer."""
        s, i32, dev = self.shape, self._i32, self._dev
        B, ld = lens.numel(), weights.shape[-1]
        heads = (s.n_layers if layer is None else 1) * B * s.n_kv_heads
        w = _need("weights", weights, self._f32, heads * ld, dev)
        rc = lib().llama_op_cache_evict(
            self.ctx, kv._now(s, self._dt, B, dev), ALL_LAYERS if layer is None else layer,
            _need("lens", lens, i32, B, dev), B, keep, first, recent, w, ld,
            w if weights_out is None else _need("weights_out", weights_out, self._f32, heads * ld, dev),
            _need("kept", kept, i32, heads * keep, dev))
        if rc:
            raise LlamaError(rc, "llama_op_cache_evict")

    def op_embed(self, tokens, out):
        self._chk(lib().llama_op_embed(self.ctx, _p(tokens), tokens.numel(), _p(out)), "llama_op_embed")

    def op_argmax(self, logits, ids):
        B, V = logits.shape
        self._chk(lib().llama_op_argmax(self.ctx, _p(logits), B, V, _p(ids)), "llama_op_argmax")

    def sample(self, logits, uniforms, next_ids, *, temperature=1.0, top_k=0, top_p=1.0,
               repetition_penalty=1.0, history=None, history_len=None):
        """Draw next_ids[b] from logits[b] (see llama_sample). history: [B, S] int32
        device ids and history_len: [B] int32 counts, or None."""
        sp = Sampling(temperature, top_k, top_p, repetition_penalty)
        stride = history.shape[1] if history is not None else 0
        self._chk(lib().llama_sample(self.ctx, _p(logits), logits.shape[0], logits.shape[1],
                                     ctypes.byref(sp),
                                     _p(history), _p(history_len), stride, _p(uniforms),
                                     _p(next_ids)), "llama_sample")
