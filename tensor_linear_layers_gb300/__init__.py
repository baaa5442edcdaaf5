"""Thin ctypes binding of libtplinear.so (include/tp_linear.h).

Argument marshalling only: torch tensors become device pointers and the
current CUDA stream becomes the stream argument; torch allocates the outputs,
packed weights and workspaces. Every step of the block runs in the library's
CUDA kernels. There is no fallback: if the library is missing or cannot load,
every call raises.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtplinear.so")

TP_OK = 0
TP_ERR_ARG, TP_ERR_SHAPE, TP_ERR_UNSUPPORTED, TP_ERR_CUDA, TP_ERR_CAPACITY, TP_ERR_TIMEOUT = (
    -1, -2, -3, -4, -5, -6)
TP_BLOCK_MLP, TP_BLOCK_ATTN_PROJ, TP_BLOCK_MOE = 0, 1, 2
TP_FLAG_HAS_NORM = 1
TP_FLAG_GATHERED = 2
TP_ROPE_HALF, TP_ROPE_INTERLEAVED = 0, 1
TP_TREE_MAX_DRAFT = 256
TP_KV_MAX_LAYERS = 128
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}

ABI_SYMBOLS = (
    "tp_packed_weight_bytes", "tp_linear_create", "tp_linear_destroy", "tp_workspace_size",
    "tp_mlp_forward", "tp_add_rms_norm", "tp_gate_up_forward", "tp_down_forward",
    "tp_attn_proj_forward", "tp_capture_workspace_size", "tp_capture_rows", "tp_last_error",
    "tp_describe_plan", "tp_mlp_forward_no_alloc", "tp_set_wait_timeout", "tp_attention_forward",
    "tp_layer_create", "tp_layer_destroy", "tp_layer_workspace_size", "tp_decoder_layer_forward",
    "tp_moe_forward", "tp_kv_cache_write", "tp_paged_attention_workspace_size", "tp_paged_attention",
    "tp_rope_frequencies", "tp_rope_table", "tp_qk_norm_rope", "tp_layer_set_rope", "tp_tree_mask",
    "tp_tree_attention_workspace_size", "tp_tree_attention", "tp_kv_cache_copy_blocks", "tp_kv_cache_compact",
    "tp_kv_quant_write", "tp_kv_quant_read", "tp_chunk_attention_workspace_size", "tp_chunk_attention",
)


class TPError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"tp_linear error {code}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("t", ctypes.c_int32), ("hidden", ctypes.c_int64),
                ("intermediate", ctypes.c_int64), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("flags", ctypes.c_int32), ("n_experts", ctypes.c_int32)]


class LayerIO(ctypes.Structure):
    _fields_ = [("hidden_in", ctypes.c_void_p), ("residual_in", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("max_seqlen", ctypes.c_int32),
                ("residual_attn", ctypes.c_void_p), ("attn_out", ctypes.c_void_p),
                ("residual_mlp", ctypes.c_void_p), ("mlp_out", ctypes.c_void_p),
                ("residual_stream", ctypes.c_void_p)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("low_freq_factor", ctypes.c_double),
                ("high_freq_factor", ctypes.c_double), ("beta_slow", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("attn_factor", ctypes.c_double), ("original_max_position", ctypes.c_int64)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class GemmPlan(ctypes.Structure):
    _fields_ = [("swap_ab", ctypes.c_int32), ("block_n", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("units", ctypes.c_int32), ("grid", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("engine", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the in-tree library once (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    PI64 = ctypes.POINTER(ctypes.c_int64)
    sig = {
        "tp_packed_weight_bytes": [ctypes.POINTER(Config), PI64, PI64],
        "tp_linear_create": [ctypes.POINTER(Config), ctypes.POINTER(P), I32, P, P, P, P,
                             ctypes.POINTER(P)],
        "tp_linear_destroy": [P],
        "tp_workspace_size": [P, I64, PI64],
        "tp_mlp_forward": [P, I64, P, P, P, P, P, P, I64, P],
        "tp_add_rms_norm": [I64, I64, P, P, P, F, P, P, P],
        "tp_gate_up_forward": [P, I64, P, P, P, I64, P],
        "tp_down_forward": [P, I64, P, P, P, P, P, I64, P],
        "tp_attn_proj_forward": [P, I64, P, P, P, P, P, I64, P],
        "tp_capture_workspace_size": [I64, I64, PI64],
        "tp_capture_rows": [I64, I64, P, P, P, I64, I32, ctypes.POINTER(P), ctypes.POINTER(I32),
                            I32, P, P, I64, P, P, I64, P],
        "tp_describe_plan": [P, I64, ctypes.POINTER(GemmPlan), I32],
        "tp_mlp_forward_no_alloc": [P, I64, P, P, P, P, P, P, P],
        "tp_set_wait_timeout": [I64],
        "tp_attention_forward": [P, I64, P, P, I32, I32, P, P, I64, P],
        "tp_layer_create": [P, P, I64, ctypes.POINTER(P)],
        "tp_layer_destroy": [P],
        "tp_layer_workspace_size": [P, PI64],
        "tp_decoder_layer_forward": [P, I64, ctypes.POINTER(LayerIO), P, I64, P],
        "tp_moe_forward": [P, I64, I32, P, P, P, P, P, I64, P],
        "tp_kv_cache_write": [P, I64, P, P, P, P, I64, I32, P, I64, P],
        "tp_paged_attention_workspace_size": [P, I32, I32, I32, PI64],
        "tp_paged_attention": [P, I64, P, P, P, I32, I32, I32, P, I32, P, P, P, I64, I32, P, P, I64, P],
        "tp_rope_frequencies": [ctypes.POINTER(RopeConfig), ctypes.POINTER(ctypes.c_double),
                                ctypes.POINTER(ctypes.c_double)],
        "tp_rope_table": [ctypes.POINTER(RopeConfig), I64, P, P],
        "tp_qk_norm_rope": [P, I64, P, P, P, ctypes.POINTER(RopeArgs), P, P, P, I64, I32, P, I64, P],
        "tp_layer_set_rope": [P, ctypes.POINTER(RopeArgs), P],
        "tp_tree_mask": [I64, I32, I32, P, P, P, P, I32, P, P, I64, P],
        "tp_tree_attention_workspace_size": [P, I32, I32, I32, PI64],
        "tp_tree_attention": [P, I64, P, P, P, I32, I32, I32, P, I32, P, I32, P, P, I64, I32, P, P, I64, P],
        "tp_kv_quant_write": [P, I64, P, P, P, P, P, P, I64, I32, P, I64, P],
        "tp_kv_quant_read": [P, I64, P, P, P, P, P, I64, I32, P, P, P, I64, P],
        "tp_chunk_attention_workspace_size": [P, I32, I32, I32, PI64],
        "tp_chunk_attention": [P, I64, P, P, P, I32, I32, I32, P, I32, I32, I32, P, P, P, P, I64, I32, P, P, I64, P],
        "tp_kv_cache_copy_blocks": [P, P, I32, I32, P, P, I64, I32, P, I64, P],
        "tp_kv_cache_compact": [P, I32, P, P, P, I32, P, P, I32, I32, P, P, I64, I32, P, P, I64, P],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.tp_last_error.argtypes = []
    L.tp_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(rc: int) -> int:
    if rc < 0:
        raise TPError(rc, lib().tp_last_error().decode(errors="replace"))
    return rc


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# torch's own call for the current stream's handle: a stream object made for every call costs 3 us
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _bf16(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor")
    return t


_INT32, _BF16, _E4M3 = torch.int32, torch.bfloat16, torch.float8_e4m3fn


def _i32(t: torch.Tensor, name: str, index: int, numel: int = -1) -> int:
    """Device pointer of a contiguous int32 tensor on CUDA device `index` (of `numel` elements at least)."""
    if t.dtype is not _INT32 or t.get_device() != index or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor on cuda:{index}")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, {numel} needed")
    return t.data_ptr()


def _bf16_on(t: torch.Tensor, name: str, index: int, shape=None) -> int:
    """Device pointer of a contiguous bf16 tensor on CUDA device `index` (of this shape)."""
    if t.dtype is not _BF16 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 tensor on cuda:{index}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    return t.data_ptr()


def _new(shape, dtype: torch.dtype, device, stream, zero: bool = False) -> torch.Tensor:
    """A tensor for work on `stream` (None: the current one), allocated and zeroed in that stream's order: a fill
    on another stream could come after the kernels, and its memory go to other work while they run. The caller
    has it on the current stream, so its memory is not given away before what runs there either."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        x = make(shape, dtype=dtype, device=device)
    x.record_stream(torch.cuda.current_stream(device))
    return x


def _contiguous(x: torch.Tensor, stream) -> torch.Tensor:
    """x, or a contiguous copy of it made on `stream`; to be held until the kernels that read it are launched."""
    if stream is None or x.is_contiguous():
        return x.contiguous()
    with torch.cuda.stream(stream):
        return x.contiguous()


def _workspace(ws: Optional[torch.Tensor], need: int, index: int, stream) -> torch.Tensor:
    if ws is None:
        return _new(need, torch.uint8, torch.device("cuda", index), stream, zero=True)
    if ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{index}")
    return ws


def make_config(kind: int, t: int, hidden: int, intermediate: int = 0, n_q_heads: int = 0,
                n_kv_heads: int = 0, head_dim: int = 0, rms_eps: float = 1e-5, flags: int = 0,
                n_experts: int = 0) -> Config:
    return Config(kind, t, hidden, intermediate, n_q_heads, n_kv_heads, head_dim, rms_eps, flags, n_experts)


def packed_weight_bytes(cfg: Config):
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().tp_packed_weight_bytes(ctypes.byref(cfg), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def set_wait_timeout(ns: int) -> None:
    """Wall-clock limit (ns) of every on-chip wait in kernels launched afterwards (default 2 s)."""
    _check(lib().tp_set_wait_timeout(int(ns)))


def capture_workspace_size(T: int, n_sel: int) -> int:
    b = ctypes.c_int64()
    _check(lib().tp_capture_workspace_size(T, n_sel, ctypes.byref(b)))
    return b.value


class TPLinear:
    """One tensor-parallel block (MLP or attention projections) on the current GPU.

    ``weights``: MLP (w_gate [I,H], w_up [I,H], w_down [H,I]); attention
    (w_q, w_k, w_v, w_o), all bf16 CUDA tensors in nn.Linear layout. The
    packed shard buffers are allocated here and owned by this object.
    """

    def __init__(self, cfg: Config, weights: Sequence[torch.Tensor], gamma: Optional[torch.Tensor] = None,
                 stream=None):
        L = lib()
        self.cfg = cfg
        col, row = packed_weight_bytes(cfg)
        dev = weights[0].device
        self.w_col = _new(col // 2, torch.bfloat16, dev, stream)
        self.w_row = _new(row // 2, torch.bfloat16, dev, stream)
        self.gamma = None if gamma is None else _bf16(gamma, "gamma")
        ws = [_bf16(w, "weight") for w in weights]
        arr = (ctypes.c_void_p * len(ws))(*[w.data_ptr() for w in ws])
        h = ctypes.c_void_p()
        _check(L.tp_linear_create(ctypes.byref(cfg), arr, len(ws), _ptr(self.w_col), _ptr(self.w_row),
                                  _ptr(self.gamma), _stream(stream), ctypes.byref(h)))
        self.handle = h
        self._ws = None
        self._ws_sizes = {}
        self._dev, self._index = dev, dev.index
        if cfg.kind == TP_BLOCK_ATTN_PROJ:     # per-shard head counts and row widths of qkv and of the attention output
            self._kv_per = 1 if cfg.t >= cfg.n_kv_heads else cfg.n_kv_heads // cfg.t
            q_per = cfg.n_q_heads // cfg.t
            self._qkv_width, self._attn_width = (q_per + 2 * self._kv_per) * cfg.head_dim, q_per * cfg.head_dim
            self._gathered = bool(cfg.flags & TP_FLAG_GATHERED)
            self._shape = (cfg.t, self._kv_per, cfg.head_dim)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().tp_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ workspace
    def workspace_size(self, max_tokens: int) -> int:
        got = self._ws_sizes.get(max_tokens)
        if got is None:
            b = ctypes.c_int64()
            _check(lib().tp_workspace_size(self.handle, max_tokens, ctypes.byref(b)))
            got = self._ws_sizes[max_tokens] = b.value
        return got

    def workspace(self, max_tokens: int, stream=None) -> torch.Tensor:
        """A zero-filled workspace for calls of up to max_tokens tokens on `stream` (cached, grows on demand).
        It is one for all streams: calls that overlap need workspaces of their own."""
        need = self.workspace_size(max_tokens)
        if self._ws is None or self._ws.numel() < need:
            self._ws = _new(need, torch.uint8, self.w_col.device, stream, zero=True)
        elif stream is not None:
            self._ws.record_stream(stream)     # a larger one may take its place while this call runs
        return self._ws

    def plan(self, T: int):
        arr = (GemmPlan * 2)()
        n = _check(lib().tp_describe_plan(self.handle, T, arr, 2))
        return [{k: getattr(arr[i], k) for k, _ in GemmPlan._fields_} for i in range(n)]

    # ------------------------------------------------------------------ MLP
    def mlp_forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                    residual_stream: bool = True, out: Optional[dict] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> dict:
        T, H = x.shape
        norm = bool(self.cfg.flags & TP_FLAG_HAS_NORM)
        o = out if out is not None else {}
        if "mlp_out" not in o:
            o["mlp_out"] = _new(x.shape, x.dtype, x.device, stream)
        if norm and "residual_out" not in o:
            o["residual_out"] = _new(x.shape, x.dtype, x.device, stream)
        if residual_stream and residual is not None and "residual_stream" not in o:
            o["residual_stream"] = _new(x.shape, x.dtype, x.device, stream)
        ws = self.workspace(T, stream) if ws is None else ws
        _check(lib().tp_mlp_forward(self.handle, T, _ptr(_bf16(x, "x")), _ptr(residual), _ptr(o.get("residual_out")),
                                    _ptr(o["mlp_out"]), _ptr(o.get("residual_stream")), _ptr(ws), ws.numel(),
                                    _stream(stream)))
        return o

    def mlp_forward_no_alloc(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                             residual_stream: bool = True, out: Optional[dict] = None,
                             status: Optional[torch.Tensor] = None, stream=None) -> dict:
        """tp_mlp_forward_no_alloc: the decode-shaped block with the library's fixed scratch."""
        T, H = x.shape
        norm = bool(self.cfg.flags & TP_FLAG_HAS_NORM)
        o = out if out is not None else {}
        if "mlp_out" not in o:
            o["mlp_out"] = _new(x.shape, x.dtype, x.device, stream)
        if norm and "residual_out" not in o:
            o["residual_out"] = _new(x.shape, x.dtype, x.device, stream)
        if residual_stream and residual is not None and "residual_stream" not in o:
            o["residual_stream"] = _new(x.shape, x.dtype, x.device, stream)
        if status is not None and (status.dtype != torch.int32 or not status.is_cuda or status.numel() < 1
                                   or status.device != self.w_col.device):
            raise ValueError("status must be an int32 CUDA tensor of at least one element on the block's device")
        _check(lib().tp_mlp_forward_no_alloc(self.handle, T, _ptr(_bf16(x, "x")), _ptr(residual),
                                             _ptr(o.get("residual_out")), _ptr(o["mlp_out"]),
                                             _ptr(o.get("residual_stream")), _ptr(status), _stream(stream)))
        return o

    @property
    def gathered(self) -> bool:
        return bool(self.cfg.flags & TP_FLAG_GATHERED)

    def gate_up(self, x: torch.Tensor, h_out: Optional[torch.Tensor] = None, ws=None, stream=None) -> torch.Tensor:
        """h [t][T][I/t] (shard-major), or [T][I] with TP_FLAG_GATHERED."""
        T = x.shape[0]
        t, Is = self.cfg.t, self.cfg.intermediate // self.cfg.t
        if h_out is None:
            shape = (T, t * Is) if self.gathered else (t, T, Is)
            h_out = _new(shape, torch.bfloat16, x.device, stream)
        ws = self.workspace(T, stream) if ws is None else ws
        _check(lib().tp_gate_up_forward(self.handle, T, _ptr(_bf16(x, "x")), _ptr(h_out), _ptr(ws), ws.numel(),
                                        _stream(stream)))
        return h_out

    def down(self, h_in: torch.Tensor, residual: Optional[torch.Tensor] = None, out=None, stream_out=None,
             ws=None, stream=None):
        T = h_in.shape[0] if self.gathered else h_in.shape[1]
        H = self.cfg.hidden
        out = _new((T, H), torch.bfloat16, h_in.device, stream) if out is None else out
        if residual is not None and stream_out is None:
            stream_out = _new((T, H), torch.bfloat16, h_in.device, stream)
        ws = self.workspace(T, stream) if ws is None else ws
        _check(lib().tp_down_forward(self.handle, T, _ptr(_bf16(h_in, "h_in")), _ptr(residual), _ptr(out),
                                     _ptr(stream_out), _ptr(ws), ws.numel(), _stream(stream)))
        return out, stream_out

    # ------------------------------------------------------------------ paged KV cache
    def kv_cache_shape(self, num_blocks: int, block_size: int):
        """Shape of one of the two caches: [t][num_blocks][block_size][kv heads per shard][head_dim]."""
        c = self.cfg
        kv_per = 1 if c.t >= c.n_kv_heads else c.n_kv_heads // c.t
        return (c.t, num_blocks, block_size, kv_per, c.head_dim)

    def _attention_handle(self) -> None:
        if self.cfg.kind != TP_BLOCK_ATTN_PROJ:
            raise ValueError("not an attention handle")

    def _rows(self, x: torch.Tensor, width: int):
        """Tokens of a shard-major [t][T][width] or gathered [T][t * width] tensor, and the shape it must have."""
        t = self._shape[0]
        if self._gathered:
            return x.shape[0], (x.shape[0], t * width)
        if x.dim() != 3:
            raise ValueError(f"expected [t, T, {width}], got {tuple(x.shape)}")
        return x.shape[1], (t, x.shape[1], width)

    def _cache_shape(self, cache: torch.Tensor):
        """The shape a cache with as many blocks of that size must have."""
        if cache.dim() != 5:
            raise ValueError("a cache has the shape of kv_cache_shape()")
        _, nb, bs, _, _ = cache.shape
        t, kv_per, hd = self._shape
        return nb, bs, (t, nb, bs, kv_per, hd)

    def _layer_pointers(self, caches_k: Sequence[torch.Tensor], caches_v: Sequence[torch.Tensor]):
        """Number of layers, HOST addresses of the arrays of their k and v pointers, blocks and block size of
        the caches (all of one size), and the object that holds the arrays."""
        if len(caches_k) != len(caches_v) or not caches_k:
            raise ValueError("caches_k and caches_v must list the same layers, one at least")
        self._attention_handle()
        nb, bs, shape = self._cache_shape(caches_k[0])
        dev, n = self._index, len(caches_k)
        both = [*caches_k, *caches_v]
        _bf16_on(both[0], "cache_k", dev, shape)
        # A call names every layer's caches, 64 tensors for 32 layers: the same checks of all of them, one
        # attribute at a time.
        T = torch.Tensor
        if (list(map(T.size, both)).count(shape) != len(both) or False in map(T.is_contiguous, both)
                or set(map(T.dtype.__get__, both)) != {_BF16}):
            raise ValueError(f"every cache must be a contiguous bf16 tensor of the shape {tuple(shape)}")
        if set(map(T.get_device, both)) != {dev}:
            raise ValueError(f"every cache must be on cuda:{dev}")
        ptrs = array.array("Q", map(T.data_ptr, both))
        at = ptrs.buffer_info()[0]
        return n, at, at + 8 * n, nb, bs, ptrs

    def qk_norm_rope(self, qkv: torch.Tensor, positions: torch.Tensor, rope: "Rope", out: Optional[torch.Tensor] = None,
                     slot_mapping: Optional[torch.Tensor] = None, cache_k: Optional[torch.Tensor] = None,
                     cache_v: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
        """Per-head norm (where the Rope has gammas) and rotation of q and k at positions (int32 [T],
        negative = padding); out: a new tensor of qkv's shape, or qkv itself (in place). With slot_mapping
        (int32 [T], negative = none) k and v also go to their cache slots. Returns (out, 16-byte workspace
        whose first word is the status)."""
        self._attention_handle()
        dev = self._index
        T, shape = self._rows(qkv, self._qkv_width)
        src = _bf16_on(qkv, "qkv", dev, shape)
        if out is None:
            out = _new(qkv.shape, qkv.dtype, self._dev, stream)
        ws = _workspace(ws, 16, dev, stream)
        ck = cv = slots = None
        nb = bs = 0
        if slot_mapping is not None:
            if cache_k is None or cache_v is None:
                raise ValueError("slot_mapping needs cache_k and cache_v")
            slots = _i32(slot_mapping, "slot_mapping", dev, T)
            nb, bs, cshape = self._cache_shape(cache_k)
            ck, cv = _bf16_on(cache_k, "cache_k", dev, cshape), _bf16_on(cache_v, "cache_v", dev, cshape)
        rope.check(dev, self._shape[2])
        _check(lib().tp_qk_norm_rope(self.handle, T, src, _bf16_on(out, "out", dev, shape),
                                     _i32(positions, "positions", dev, T), rope.args, slots, ck, cv, nb, bs,
                                     ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return out, ws

    def kv_cache_copy_blocks(self, block_pairs: torch.Tensor, caches_k: Sequence[torch.Tensor],
                             caches_v: Sequence[torch.Tensor], ws: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
        """Copy block src to block dst for every (src, dst) row of block_pairs (int32 [n, 2], src < 0 = skip)
        in the caches of all listed layers. Returns the workspace whose first word is the status."""
        if block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
            raise ValueError("block_pairs must be [n, 2]")
        dev = self._index
        n, ks, vs, nb, bs, _hold = self._layer_pointers(caches_k, caches_v)
        ws = _workspace(ws, 16, dev, stream)
        _check(lib().tp_kv_cache_copy_blocks(self.handle, _i32(block_pairs, "block_pairs", dev), block_pairs.shape[0],
                                             n, ks, vs, nb, bs, ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return ws

    def kv_cache_compact(self, query_start_loc: torch.Tensor, seq_lens: torch.Tensor, accepted: torch.Tensor,
                         src_tables: torch.Tensor, dst_tables: torch.Tensor, caches_k: Sequence[torch.Tensor],
                         caches_v: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, stream=None):
        """Move the accepted drafted tokens of every request (accepted int32 [n_reqs, m], rising draft
        indices, ended by -1) from src_tables' pages to the positions after the cached tokens in dst_tables'
        (the same tensor: in place), in the caches of all listed layers. Returns (new lengths, workspace)."""
        dev = self._index
        n_reqs = seq_lens.numel()
        if accepted.dim() != 2 or src_tables.dim() != 2 or src_tables.shape != dst_tables.shape:
            raise ValueError("accepted is [n_reqs, m], src_tables and dst_tables [n_reqs, max_blocks]")
        n, ks, vs, nb, bs, _hold = self._layer_pointers(caches_k, caches_v)
        if out is None:
            out = _new(n_reqs, torch.int32, self._dev, stream)
        ws = _workspace(ws, 16, dev, stream)
        mb = src_tables.shape[1]
        _check(lib().tp_kv_cache_compact(
            self.handle, n_reqs, _i32(query_start_loc, "query_start_loc", dev, n_reqs + 1),
            _i32(seq_lens, "seq_lens", dev), _i32(accepted, "accepted", dev, n_reqs * accepted.shape[1]),
            accepted.shape[1], _i32(src_tables, "src_tables", dev, n_reqs * mb), _i32(dst_tables, "dst_tables", dev),
            mb, n, ks, vs, nb, bs, _i32(out, "out", dev, n_reqs), ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return out, ws

    def tree_attention_workspace_size(self, n_reqs: int, max_query_len: int, max_seq_len: int) -> int:
        b = ctypes.c_int64()
        _check(lib().tp_tree_attention_workspace_size(self.handle, n_reqs, max_query_len, max_seq_len,
                                                      ctypes.byref(b)))
        return b.value

    def tree_attention(self, qkv: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                       block_tables: torch.Tensor, mask: torch.Tensor, cache_k: torch.Tensor, cache_v: torch.Tensor,
                       max_query_len: int, max_seq_len: int, out=None, ws=None, stream=None):
        """Attention of every request's drafted tokens (rows of qkv, already in the cache as its last
        positions) over its cached tokens and over the drafted ones that their mask rows (tree_mask) name.
        Returns (attn in the attention core's output layout, workspace)."""
        self._attention_handle()
        dev, n_reqs = self._index, seq_lens.numel()
        T, shape = self._rows(qkv, self._qkv_width)
        nb, bs, cshape = self._cache_shape(cache_k)
        t, w = self._shape[0], self._attn_width
        out_shape = (T, t * w) if self._gathered else (t, T, w)
        if out is None:
            out = _new(out_shape, torch.bfloat16, self._dev, stream)
        need = self.tree_attention_workspace_size(n_reqs, max_query_len, max_seq_len) if ws is None else 0
        ws = _workspace(ws, need, dev, stream)
        if block_tables.dim() != 2 or mask.dim() != 2:
            raise ValueError("block_tables is [n_reqs, max_blocks], mask [T, words]")
        max_blocks, words = block_tables.shape[1], mask.shape[1]
        _check(lib().tp_tree_attention(
            self.handle, T, _bf16_on(qkv, "qkv", dev, shape),
            _i32(query_start_loc, "query_start_loc", dev, n_reqs + 1), _i32(seq_lens, "seq_lens", dev), n_reqs,
            max_query_len, max_seq_len, _i32(block_tables, "block_tables", dev, n_reqs * max_blocks), max_blocks,
            _i32(mask, "mask", dev, T * words), words, _bf16_on(cache_k, "cache_k", dev, cshape),
            _bf16_on(cache_v, "cache_v", dev, cshape), nb, bs, _bf16_on(out, "out", dev, out_shape),
            ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return out, ws

    def kv_quant_cache(self, num_blocks: int, block_size: int, stream=None):
        """A new, zero-filled cache in 8 bits: (codes_k, codes_v float8_e4m3fn [t, blocks, block_size, kv heads
        of the shard, 128], scales_k, scales_v uint8 [t, blocks, block_size, kv heads of the shard])."""
        shape = self.kv_cache_shape(num_blocks, block_size)
        codes = [_new(shape, torch.uint8, self._dev, stream, zero=True).view(_E4M3) for _ in range(2)]
        return (*codes, *(_new(shape[:-1], torch.uint8, self._dev, stream, zero=True) for _ in range(2)))

    def _quant(self, codes_k: torch.Tensor, codes_v: torch.Tensor, scales_k: torch.Tensor, scales_v: torch.Tensor):
        """(blocks, block size, the four device pointers) of a cache in 8 bits on this handle's device."""
        nb, bs, shape = self._cache_shape(codes_k)
        dev, flat = self._index, shape[:-1]
        if not (codes_k.dtype is codes_v.dtype is _E4M3 and scales_k.dtype is scales_v.dtype is torch.uint8
                and codes_v.shape == shape and scales_k.shape == flat and scales_v.shape == flat and codes_k.shape == shape
                and codes_k.get_device() == codes_v.get_device() == scales_k.get_device() == scales_v.get_device() == dev
                and codes_k.is_contiguous() and codes_v.is_contiguous() and scales_k.is_contiguous()
                and scales_v.is_contiguous()):
            for name, x, dtype, want in (("codes_k", codes_k, _E4M3, shape), ("codes_v", codes_v, _E4M3, shape),
                                         ("scales_k", scales_k, torch.uint8, flat),
                                         ("scales_v", scales_v, torch.uint8, flat)):
                if x.dtype is not dtype or x.get_device() != dev or not x.is_contiguous() or x.shape != want:
                    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(want)} on cuda:{dev}")
        return nb, bs, codes_k.data_ptr(), codes_v.data_ptr(), scales_k.data_ptr(), scales_v.data_ptr()

    def kv_quant_write(self, qkv: torch.Tensor, slot_mapping: torch.Tensor, codes_k: torch.Tensor,
                       codes_v: torch.Tensor, scales_k: torch.Tensor, scales_v: torch.Tensor,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Quantise every token's k and v heads into its slot of a cache in 8 bits (slot_mapping int32 [T],
        negative = skip). Returns the 16-byte workspace whose first word is the status."""
        self._attention_handle()
        dev = self._index
        T, shape = self._rows(qkv, self._qkv_width)
        nb, bs, ck, cv, sk, sv = self._quant(codes_k, codes_v, scales_k, scales_v)
        ws = _workspace(ws, 16, dev, stream)
        _check(lib().tp_kv_quant_write(self.handle, T, _bf16_on(qkv, "qkv", dev, shape),
                                       _i32(slot_mapping, "slot_mapping", dev, T), ck, cv, sk, sv, nb, bs,
                                       ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return ws

    def kv_quant_read(self, slots: torch.Tensor, codes_k: torch.Tensor, codes_v: torch.Tensor,
                      scales_k: torch.Tensor, scales_v: torch.Tensor, out=None, ws: Optional[torch.Tensor] = None,
                      stream=None):
        """What the heads in these slots (int32 [n], negative = zeros) of a cache in 8 bits stand for: (k, v bf16
        [t, n, kv heads of the shard, 128], workspace whose first word is the status); out: (k, v) to write
        instead of new tensors."""
        self._attention_handle()
        dev, n = self._index, slots.numel()
        nb, bs, ck, cv, sk, sv = self._quant(codes_k, codes_v, scales_k, scales_v)
        t, kv_per, hd = self._shape
        shape = (t, n, kv_per, hd)
        k, v = (_new(shape, torch.bfloat16, self._dev, stream) for _ in range(2)) if out is None else out
        ws = _workspace(ws, 16, dev, stream)
        _check(lib().tp_kv_quant_read(self.handle, n, _i32(slots, "slots", dev), ck, cv, sk, sv, nb, bs,
                                      _bf16_on(k, "out[0]", dev, shape), _bf16_on(v, "out[1]", dev, shape),
                                      ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
        return k, v, ws

    def chunk_attention_workspace_size(self, n_reqs: int, max_query_len: int, max_seq_len: int) -> int:
        b = ctypes.c_int64()
        _check(lib().tp_chunk_attention_workspace_size(self.handle, n_reqs, max_query_len, max_seq_len,
                                                       ctypes.byref(b)))
        return b.value

    def chunk_attention(self, qkv: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                        block_tables: torch.Tensor, cache_k: torch.Tensor, cache_v: torch.Tensor, max_query_len: int,
                        max_seq_len: int, window: int = 0, sinks: int = 0, scales_k: Optional[torch.Tensor] = None,
                        scales_v: Optional[torch.Tensor] = None, out=None, ws=None, stream=None):
        """Attention of every request's new tokens (rows of qkv, already in the cache as its last positions)
        over its cached tokens, causal: with a window, over the last `window` of them and the first `sinks`.
        The caches are bf16, or e4m3 codes with their scales (kv_quant_write). Returns (attn in the
        attention core's output layout, workspace whose first word is the status)."""
        self._attention_handle()
        dev, n_reqs = self._index, seq_lens.numel()
        T, shape = self._rows(qkv, self._qkv_width)
        if (scales_k is None) != (scales_v is None):
            raise ValueError("scales_k and scales_v: both (a cache in 8 bits) or neither (in bf16)")
        if scales_k is not None:
            nb, bs, ck, cv, sk, sv = self._quant(cache_k, cache_v, scales_k, scales_v)
        else:
            nb, bs, cshape = self._cache_shape(cache_k)
            ck, cv = _bf16_on(cache_k, "cache_k", dev, cshape), _bf16_on(cache_v, "cache_v", dev, cshape)
            sk = sv = None
        t, w = self._shape[0], self._attn_width
        out_shape = (T, t * w) if self._gathered else (t, T, w)
        if out is None:
            out = _new(out_shape, torch.bfloat16, self._dev, stream)
        need = self.chunk_attention_workspace_size(n_reqs, max_query_len, max_seq_len) if ws is None else 0
        ws = _workspace(ws, need, dev, stream)
        if block_tables.dim() != 2:
            raise ValueError("block_tables is [n_reqs, max_blocks]")
        max_blocks = block_tables.shape[1]
        _check(lib().tp_chunk_attention(
            self.handle, T, _bf16_on(qkv, "qkv", dev, shape),
            _i32(query_start_loc, "query_start_loc", dev, n_reqs + 1), _i32(seq_lens, "seq_lens", dev), n_reqs,
            max_query_len, max_seq_len, _i32(block_tables, "block_tables", dev, n_reqs * max_blocks), max_blocks,
            window, sinks, ck, cv, sk, sv, nb, bs, _bf16_on(out, "out", dev, out_shape), ws.data_ptr(), ws.numel(),
            _stream_ptr(stream)))
        return out, ws

    def kv_cache_write(self, qkv: torch.Tensor, slot_mapping: torch.Tensor, cache_k: torch.Tensor,
                       cache_v: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Copy every token's k and v heads into its slot (slot_mapping int32 [T], -1 = skip).
        Returns the 16-byte workspace whose first word is the status."""
        T = qkv.shape[0] if self.gathered else qkv.shape[1]
        _, nb, bs, _, _ = cache_k.shape
        ws = _new(16, torch.uint8, qkv.device, stream, zero=True) if ws is None else ws
        _check(lib().tp_kv_cache_write(self.handle, T, _ptr(_bf16(qkv, "qkv")), _ptr(slot_mapping),
                                       _ptr(_bf16(cache_k, "cache_k")), _ptr(_bf16(cache_v, "cache_v")), nb, bs,
                                       _ptr(ws), ws.numel(), _stream(stream)))
        return ws

    def paged_attention_workspace_size(self, n_reqs: int, max_query_len: int, max_seq_len: int) -> int:
        b = ctypes.c_int64()
        _check(lib().tp_paged_attention_workspace_size(self.handle, n_reqs, max_query_len, max_seq_len,
                                                       ctypes.byref(b)))
        return b.value

    def paged_attention(self, qkv: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                        block_tables: torch.Tensor, cache_k: torch.Tensor, cache_v: torch.Tensor,
                        max_query_len: int, max_seq_len: int, out=None, ws=None, stream=None, slot_mapping=None):
        """Attention of the new tokens (rows of qkv) over their requests' cached keys; with
        slot_mapping (int32 [T]) the call also writes the new tokens' k and v to their slots.
        Returns (attn in the attention core's output layout, workspace)."""
        c = self.cfg
        T = qkv.shape[0] if self.gathered else qkv.shape[1]
        n_reqs = query_start_loc.numel() - 1
        _, nb, bs, _, _ = cache_k.shape
        if out is None:
            shape = (T, c.n_q_heads * c.head_dim) if self.gathered else (c.t, T, c.n_q_heads // c.t * c.head_dim)
            out = _new(shape, torch.bfloat16, qkv.device, stream)
        if ws is None:
            ws = _new(self.paged_attention_workspace_size(n_reqs, max_query_len, max_seq_len), torch.uint8, qkv.device,
                      stream, zero=True)
        for name, a in (("query_start_loc", query_start_loc), ("seq_lens", seq_lens), ("block_tables", block_tables),
                        ("slot_mapping", slot_mapping)):
            if a is None and name == "slot_mapping":
                continue
            if a.dtype != torch.int32 or not a.is_cuda or not a.is_contiguous():
                raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
        _check(lib().tp_paged_attention(self.handle, T, _ptr(_bf16(qkv, "qkv")), _ptr(query_start_loc),
                                        _ptr(seq_lens), n_reqs, int(max_query_len), int(max_seq_len),
                                        _ptr(block_tables), block_tables.shape[1],
                                        _ptr(slot_mapping), _ptr(_bf16(cache_k, "cache_k")),
                                        _ptr(_bf16(cache_v, "cache_v")), nb, bs, _ptr(out), _ptr(ws), ws.numel(),
                                        _stream(stream)))
        return out, ws

    # ------------------------------------------------------------------ mixture of experts
    def moe_forward(self, x: torch.Tensor, expert_ids: torch.Tensor, gates: torch.Tensor, out=None, ws=None,
                    stream=None) -> torch.Tensor:
        """y [T, H] = sum_j gates[:, j] * expert_{ids[:, j]}(x); ids int32 [T, k], gates fp32 [T, k]."""
        T, k = expert_ids.shape
        if expert_ids.dtype != torch.int32 or gates.dtype != torch.float32 or not expert_ids.is_cuda:
            raise TypeError("expert_ids must be int32 and gates float32 CUDA tensors")
        ids, gates = _contiguous(expert_ids, stream), _contiguous(gates, stream)
        out = _new(x.shape, x.dtype, x.device, stream) if out is None else out
        ws = self.workspace(T * k, stream) if ws is None else ws
        _check(lib().tp_moe_forward(self.handle, T, k, _ptr(_bf16(x, "x")), _ptr(ids), _ptr(gates), _ptr(out),
                                    _ptr(ws), ws.numel(), _stream(stream)))
        return out

    # ------------------------------------------------------------------ attention projections
    def attn_proj_forward(self, x: Optional[torch.Tensor], attn_in: Optional[torch.Tensor],
                          qkv_out=None, o_out=None, ws=None, stream=None):
        c = self.cfg
        T = x.shape[0] if x is not None else (attn_in.shape[0] if self.gathered else attn_in.shape[1])
        q_per = c.n_q_heads // c.t
        kv_per = 1 if c.t >= c.n_kv_heads else c.n_kv_heads // c.t
        w_s = (q_per + 2 * kv_per) * c.head_dim
        dev = self.w_col.device
        if x is not None and qkv_out is None:
            shape = (T, c.t * w_s) if self.gathered else (c.t, T, w_s)
            qkv_out = _new(shape, torch.bfloat16, dev, stream)
        if attn_in is not None and o_out is None:
            o_out = _new((T, c.hidden), torch.bfloat16, dev, stream)
        ws = self.workspace(T, stream) if ws is None else ws
        _check(lib().tp_attn_proj_forward(self.handle, T, _ptr(x), _ptr(qkv_out if x is not None else None),
                                          _ptr(attn_in), _ptr(o_out if attn_in is not None else None),
                                          _ptr(ws), ws.numel(), _stream(stream)))
        return qkv_out, o_out

    # ------------------------------------------------------------------ attention core
    def attention_forward(self, qkv: torch.Tensor, cu_seqlens: torch.Tensor, max_seqlen: int,
                          out=None, ws=None, stream=None) -> torch.Tensor:
        """Causal GQA attention of every shard's local heads: qkv [t][T][w_s] (the
        projection's output) -> attn [t][T][nq*hd/t] (o_proj's input). cu_seqlens:
        int32 device tensor [n_seqs + 1] of sequence offsets."""
        c = self.cfg
        T = qkv.shape[0] if self.gathered else qkv.shape[1]
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens must be an int32 CUDA tensor")
        if out is None:
            shape = (T, c.n_q_heads * c.head_dim) if self.gathered else (c.t, T, c.n_q_heads // c.t * c.head_dim)
            out = _new(shape, torch.bfloat16, qkv.device, stream)
        ws = self.workspace(T, stream) if ws is None else ws
        _check(lib().tp_attention_forward(self.handle, T, _ptr(_bf16(qkv, "qkv")), _ptr(cu_seqlens),
                                          cu_seqlens.numel() - 1, int(max_seqlen), _ptr(out), _ptr(ws),
                                          ws.numel(), _stream(stream)))
        return out


class TPLayer:
    """One decoder layer (tp_decoder_layer_forward) over an attention handle and an
    MLP handle, both created with TP_FLAG_HAS_NORM (the input and post-attention
    norms). The handles must outlive this object."""

    def __init__(self, attn: TPLinear, mlp: TPLinear, max_tokens: int):
        self.attn, self.mlp, self.max_tokens = attn, mlp, max_tokens
        h = ctypes.c_void_p()
        _check(lib().tp_layer_create(attn.handle, mlp.handle, max_tokens, ctypes.byref(h)))
        self.handle = h
        b = ctypes.c_int64()
        _check(lib().tp_layer_workspace_size(h, ctypes.byref(b)))
        self.workspace_bytes = b.value
        self._ws = None

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().tp_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, stream=None) -> torch.Tensor:
        if self._ws is None:
            self._ws = _new(self.workspace_bytes, torch.uint8, self.attn.w_col.device, stream, zero=True)
        elif stream is not None:
            self._ws.record_stream(stream)
        return self._ws

    def set_rope(self, rope: Optional["Rope"], positions: Optional[torch.Tensor] = None) -> None:
        """Rotate (and norm) q and k of every later forward() between the projection and the attention:
        token i at positions[i] (int32 [max_tokens] on the GPU, read at each call). None: no rotation again."""
        if rope is None:
            _check(lib().tp_layer_set_rope(self.handle, None, None))
        else:
            dev = self.attn._index
            if positions is None:
                raise ValueError("set_rope needs positions")
            rope.check(dev, self.attn.cfg.head_dim)
            _check(lib().tp_layer_set_rope(self.handle, rope.args, _i32(positions, "positions", dev, self.max_tokens)))
        self._rope = (rope, positions)     # borrowed by the handle

    def forward(self, hidden: torch.Tensor, residual: Optional[torch.Tensor], cu_seqlens: torch.Tensor,
                max_seqlen: int, out: Optional[dict] = None, residual_stream: bool = True, ws=None,
                stream=None) -> dict:
        """Returns {residual_attn, attn_out, residual_mlp, mlp_out[, residual_stream]}, each [T, H]."""
        T = hidden.shape[0]
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens must be an int32 CUDA tensor")
        o = out if out is not None else {}
        for k in ("residual_attn", "attn_out", "residual_mlp", "mlp_out") + (
                ("residual_stream",) if residual_stream else ()):
            if k not in o:
                o[k] = _new(hidden.shape, hidden.dtype, hidden.device, stream)
        io = LayerIO(_bf16(hidden, "hidden").data_ptr(),
                     None if residual is None else _bf16(residual, "residual").data_ptr(),
                     cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(max_seqlen),
                     o["residual_attn"].data_ptr(), o["attn_out"].data_ptr(), o["residual_mlp"].data_ptr(),
                     o["mlp_out"].data_ptr(), o["residual_stream"].data_ptr() if "residual_stream" in o else None)
        ws = self.workspace(stream) if ws is None else ws
        _check(lib().tp_decoder_layer_forward(self.handle, T, ctypes.byref(io), _ptr(ws), ws.numel(),
                                              _stream(stream)))
        return o


def rope_frequencies(cfg: RopeConfig):
    """(angle per position of every rotated pair, factor of cos and sin) of a configuration, on the host."""
    f, m = (ctypes.c_double * 128)(), ctypes.c_double()
    _check(lib().tp_rope_frequencies(ctypes.byref(cfg), f, ctypes.byref(m)))
    return list(f[:cfg.rotary_dim // 2]), m.value


class Rope:
    """Rotary positions of a model: the cos/sin table of n_pos positions (built here, on `device`), the
    layout of the rotated pairs and the gammas of the q and k heads' norms (bf16 [head_dim] or None).

    scaling: "none", "linear", "ntk", "bands" or "yarn" (see include/tp_linear.h for the formulas).
    stream: where the table is built; uses on other streams come after that.
    """

    def check(self, index: int, head_dim: int) -> None:
        """Refuse a use on CUDA device `index` or with heads of `head_dim` elements that it does not fit."""
        if self.index != index:
            raise ValueError(f"the rope table is on cuda:{self.index}, not cuda:{index}")
        if self.gamma_dim not in (0, head_dim):
            raise ValueError(f"the norms' weights have {self.gamma_dim} elements, heads {head_dim}")

    def __init__(self, n_pos: int, rotary_dim: int, base: float = 10000.0, layout: int = TP_ROPE_HALF,
                 scaling: str = "none", factor: float = 1.0, original_max_position: int = 0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, beta_slow: float = 1.0,
                 beta_fast: float = 32.0, attn_factor: float = 0.0, q_gamma: Optional[torch.Tensor] = None,
                 k_gamma: Optional[torch.Tensor] = None, eps: float = 1e-6, device=None, stream=None):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}")
        self.config = RopeConfig(rotary_dim, ROPE_SCALINGS[scaling], base, factor, low_freq_factor, high_freq_factor,
                                 beta_slow, beta_fast, attn_factor, original_max_position)
        rope_frequencies(self.config)      # refuses a bad configuration before anything is allocated
        if n_pos < 1:
            raise ValueError("n_pos must be >= 1")
        if device is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.table = _new((n_pos, rotary_dim), torch.float32, device, stream)
        with torch.cuda.device(self.table.device):
            _check(lib().tp_rope_table(ctypes.byref(self.config), n_pos, self.table.data_ptr(), _stream(stream)))
        self.index = self.table.get_device()
        for name, g in (("q_gamma", q_gamma), ("k_gamma", k_gamma)):
            if g is not None:
                _bf16_on(g, name, self.index)
        dims = {g.numel() for g in (q_gamma, k_gamma) if g is not None}
        if len(dims) > 1:
            raise ValueError("q_gamma and k_gamma have different lengths")
        self.gammas, self.gamma_dim = (q_gamma, k_gamma), dims.pop() if dims else 0
        self.args = RopeArgs(self.table.data_ptr(), n_pos, rotary_dim, layout,
                             None if q_gamma is None else q_gamma.data_ptr(),
                             None if k_gamma is None else k_gamma.data_ptr(), eps)


def tree_mask(parents: torch.Tensor, query_start_loc: torch.Tensor, seq_lens: torch.Tensor, max_query_len: int,
              out=None, ws: Optional[torch.Tensor] = None, stream=None):
    """Mask rows and positions of drafted token trees: parents int32 [T], each token's parent among its
    request's drafted tokens (before it) or -1. Returns (mask int32 [T, words], positions int32 [T],
    workspace whose first word is the status); out: (mask, positions) to write instead of new tensors."""
    dev, T = parents.get_device(), parents.numel()
    if dev != torch.cuda.current_device():
        raise TypeError("parents must be a tensor on the current CUDA device")
    words = (max_query_len + 31) // 32
    if out is None:
        mask = _new((T, words), torch.int32, parents.device, stream)
        positions = _new(T, torch.int32, parents.device, stream)
    else:
        mask, positions = out
        if mask.dim() != 2 or mask.shape[0] != T:
            raise ValueError("the mask is [T, words]")
        words = mask.shape[1]
    n_reqs = seq_lens.numel()
    ws = _workspace(ws, 16, dev, stream)
    _check(lib().tp_tree_mask(T, n_reqs, max_query_len, _i32(parents, "parents", dev),
                              _i32(query_start_loc, "query_start_loc", dev, n_reqs + 1),
                              _i32(seq_lens, "seq_lens", dev), _i32(mask, "mask", dev), words,
                              None if positions is None else _i32(positions, "positions", dev, T), ws.data_ptr(),
                              ws.numel(), _stream_ptr(stream)))
    return mask, positions, ws


def add_rms_norm(a: torch.Tensor, residual: Optional[torch.Tensor], gamma: torch.Tensor, eps: float,
                 residual_out=None, x_out=None, stream=None):
    T, H = a.shape
    residual_out = _new(a.shape, a.dtype, a.device, stream) if residual_out is None else residual_out
    x_out = _new(a.shape, a.dtype, a.device, stream) if x_out is None else x_out
    _check(lib().tp_add_rms_norm(T, H, _ptr(_bf16(a, "a")), None if residual is None else _ptr(_bf16(residual, "residual")),
                                 _ptr(_bf16(gamma, "gamma")), eps, _ptr(residual_out), _ptr(x_out),
                                 _stream(stream)))
    return x_out, residual_out


def capture_rows(row_req: torch.Tensor, row_pos: torch.Tensor, sel_keys: torch.Tensor,
                 tensors: Sequence[torch.Tensor], tensor_types: Sequence[int], layer: int, capacity: int,
                 ws: Optional[torch.Tensor] = None, stream=None, out=None):
    """Returns (headers int32 [capacity, 6], rows [capacity, H], n_out int64 device scalar, ws).

    out: optional (headers, rows, n_out) tensors to write instead of new ones."""
    T, H = tensors[0].shape
    dev = tensors[0].device
    if out is not None:
        hdr, rows, n_out = out
        if (hdr.dtype != torch.int32 or hdr.shape[0] < max(capacity, 1) or hdr.shape[1] != 6
                or rows.dtype != torch.bfloat16 or rows.shape[0] < max(capacity, 1) or rows.shape[1] != H
                or n_out.dtype != torch.int64 or n_out.numel() < 1):
            raise ValueError("capture out tensors: int32 [capacity, 6], bf16 [capacity, H], int64 [1]")
    else:
        hdr = _new((max(capacity, 1), 6), torch.int32, dev, stream)
        rows = _new((max(capacity, 1), H), torch.bfloat16, dev, stream)
        n_out = _new(1, torch.int64, dev, stream, zero=True)
    need = capture_workspace_size(T, sel_keys.numel())
    ws = _new(need, torch.uint8, dev, stream, zero=True) if ws is None else ws
    arr = (ctypes.c_void_p * len(tensors))(*[_bf16(t, "tensor").data_ptr() for t in tensors])
    types = (ctypes.c_int32 * len(tensors))(*tensor_types)
    _check(lib().tp_capture_rows(T, H, _ptr(row_req), _ptr(row_pos), _ptr(sel_keys), sel_keys.numel(),
                                 len(tensors), arr, types, layer, _ptr(hdr), _ptr(rows), capacity,
                                 _ptr(n_out), _ptr(ws), ws.numel(), _stream(stream)))
    return hdr, rows, n_out, ws
