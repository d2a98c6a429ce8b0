"""Python binding of libkvq (quantised KV cache + decode attention on B200).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libkvq.so``; PyTorch tensors only provide device memory and streams.  The
functions carry the C ABI's names (``include/kvq.h``) and raise ``KvqError``
on a non-zero status.  If the shared library is missing the import fails: there
is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK = 0
KVQ_MODE_KV, KVQ_MODE_H = 0, 1
KVQ_FMT_INT, KVQ_FMT_E4M3, KVQ_FMT_ASYM, KVQ_FMT_TENSOR = 0, 1, 2, 3
KVQ_F16, KVQ_F32, KVQ_BF16 = 0, 1, 2
KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED = 0, 1
KVQ_ROPE_PLAIN, KVQ_ROPE_LINEAR, KVQ_ROPE_NTK, KVQ_ROPE_YARN, KVQ_ROPE_BANDS = 0, 1, 2, 3, 4
KVQ_TREE_MAX = 64

EXPORTED = ("kvq_cache_bytes", "kvq_layer_buffer_bytes", "kvq_append", "kvq_workspace_bytes",
            "kvq_h_scratch_bytes", "kvq_decode_attn", "kvq_decode_partials", "kvq_merge_partials",
            "kvq_h_reconstruct", "kvq_workspace_status", "kvq_status_string",
            "kvq_last_error_detail", "kvq_decode_attn_noalloc", "kvq_h_operand_bytes",
            "kvq_append_decode_attn", "kvq_h_absorbed_scratch_bytes", "kvq_h_decode_absorbed",
            "kvq_h_fused_scratch_bytes", "kvq_h_decode_fused", "kvq_selftest_bounded_wait",
            "kvq_selftest_decode_timeout", "kvq_noalloc_status", "kvq_selftest_noalloc_timeout",
            "kvq_decode_plan_info", "kvq_rope_table", "kvq_rope_append", "kvq_read",
            "kvq_tree_workspace_bytes", "kvq_tree_attn", "kvq_tree_commit", "kvq_selftest_tree_timeout")


class KvqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        detail = _lib.kvq_last_error_detail().decode() if status == -6 else ""
        super().__init__(f"{fn} failed: {status} ({status_string(status)}) {detail}".rstrip())


class KvqConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "mode", "batch", "capacity", "n_layers", "n_q_heads", "n_kv_heads", "head_dim",
        "k_bits", "v_bits", "k_group", "v_group", "d_model", "h_bits", "h_groups",
        "window", "n_anchor", "page_tokens", "n_pages", "kv_format")]


class KvqDecodePlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "engine", "num_ctas", "ctas_per_sm_planned", "stages", "stage_bytes", "smem_bytes",
        "threads", "packed_columns")]


KVQ_ENGINE_WARP_MMA, KVQ_ENGINE_TCGEN05 = 0, 1


class KvqLayer(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p)]


class KvqRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class KvqRopeConfig(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("rot_dim", "layout", "scaling", "orig_len")] +
                [(n, ctypes.c_double) for n in ("base", "factor", "low", "high", "gain")])


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkvq.so not built ({LIB_PATH}); run quantized_kv_cache_22_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64
    pu64 = ctypes.POINTER(u64)
    cfgp = ctypes.POINTER(KvqConfig)
    layp = ctypes.POINTER(KvqLayer)
    sig = {
        "kvq_cache_bytes": [cfgp, pu64, pu64, pu64],
        "kvq_layer_buffer_bytes": [cfgp, pu64, pu64, pu64, pu64],
        "kvq_append": [cfgp, layp, P, P, i32, P, i32, i32, P],
        "kvq_workspace_bytes": [cfgp, i32, pu64],
        "kvq_h_scratch_bytes": [cfgp, i32, pu64],
        "kvq_decode_attn": [cfgp, layp, P, i32, P, i32, ctypes.c_float, P, i32, P, u64, i32, P, P,
                            u64, P],
        "kvq_decode_partials": [cfgp, layp, P, i32, P, i32, ctypes.c_float, P, u64, i32, P],
        "kvq_append_decode_attn": [cfgp, layp, P, P, i32, P, i32, P, i32, ctypes.c_float, P, i32,
                                   P, u64, i32, P],
        "kvq_merge_partials": [cfgp, P, P, i32, P, u64, i32, P],
        "kvq_h_operand_bytes": [cfgp, i32, pu64],
        "kvq_h_reconstruct": [cfgp, layp, P, i32, P, P, i32, P, u64, P],
        "kvq_workspace_status": [P, ctypes.POINTER(i32), P],
        "kvq_h_absorbed_scratch_bytes": [cfgp, i32, pu64],
        "kvq_h_fused_scratch_bytes": [cfgp, i32, pu64],
        "kvq_selftest_bounded_wait": [P, u64, P],
        "kvq_selftest_decode_timeout": [cfgp, layp, P, i32, P, P, i32, P, u64, u64, P],
        "kvq_h_decode_fused": [cfgp, layp, P, P, i32, P, i32, ctypes.c_float, P, i32, P, u64, P],
        "kvq_h_decode_absorbed": [cfgp, layp, P, P, i32, P, i32, ctypes.c_float, P, i32, P, u64, P],
        "kvq_decode_attn_noalloc": [cfgp, layp, P, i32, P, i32, ctypes.c_float, P, i32, i32, P],
        "kvq_noalloc_status": [ctypes.POINTER(i32), P],
        "kvq_selftest_noalloc_timeout": [cfgp, layp, P, i32, P, P, i32, u64, P],
        "kvq_decode_plan_info": [cfgp, i32, ctypes.POINTER(KvqDecodePlan)],
    }
    ropep = ctypes.POINTER(KvqRopeConfig)
    # (kvq_rows and arrays of kvq_layer are passed as their bytes)
    sig.update({
        "kvq_rope_table": [ropep, i32, i32, P, P],
        "kvq_rope_append": [cfgp, layp, ropep, P, i32, P, P, P, P, i32, P, i32, i32, P,
                            P, P],
        "kvq_read": [cfgp, layp, P, P, i32, P, i32, i32, P, P],
        "kvq_tree_workspace_bytes": [cfgp, i32, i32, pu64],
        "kvq_tree_attn": [cfgp, layp, P, i32, i32, P, i32, P, P, ctypes.c_float, P, i32, P, u64,
                          i32, P],
        "kvq_tree_commit": [cfgp, P, i32, P, i32, i32, P, i32, P, P, P],
        "kvq_selftest_tree_timeout": [cfgp, layp, P, i32, i32, P, i32, P, i32, P, u64, i32, i32, u64, P],
    })
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.kvq_status_string.argtypes = [ctypes.c_int]
    lib.kvq_status_string.restype = ctypes.c_char_p
    lib.kvq_last_error_detail.argtypes = []
    lib.kvq_last_error_detail.restype = ctypes.c_char_p
    return lib


_lib = _load()


def lib():
    return _lib


def status_string(status: int) -> str:
    return _lib.kvq_status_string(int(status)).decode()


def _check(fn, rc):
    if rc != KVQ_OK:
        raise KvqError(fn, rc)


def _ptr(t):
    # plain ints: ctypes converts them for c_void_p arguments
    return None if t is None else t.data_ptr()


_DTYPE_CODES = {torch.float16: KVQ_F16, torch.float32: KVQ_F32, torch.bfloat16: KVQ_BF16}


def _dtype_code(t: torch.Tensor) -> int:
    return _DTYPE_CODES[t.dtype]


def _stream(stream):
    if stream is None:
        # the current stream's handle without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


class _Memo:
    """A place for the C struct of a Python object, emptied when one of its attributes is set."""
    __slots__ = ("_memo", "__dict__")

    def __new__(cls, *args, **kw):
        self = object.__new__(cls)
        object.__setattr__(self, "_memo", None)
        return self

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_memo":
            object.__setattr__(self, "_memo", None)

    def __getstate__(self):
        return self.__dict__.copy()     # copies and pickles make their own struct


_CFG_MEMO = {}   # field tuple -> (KvqConfig, byref); the library only reads the struct


@dataclass
class Config(_Memo):
    """Python view of ``kvq_config`` (see include/kvq.h for the meaning of each field)."""
    batch: int
    capacity: int
    n_q_heads: int = 0
    n_kv_heads: int = 0
    head_dim: int = 128
    k_bits: int = 8
    v_bits: int = 8
    k_group: int = 0
    v_group: int = 0
    n_layers: int = 1
    mode: int = KVQ_MODE_KV
    d_model: int = 0
    h_bits: int = 4
    h_groups: int = 0
    window: int = 0       # sliding window: ring of recent tokens (capacity = n_anchor + window)
    n_anchor: int = 0     # tokens kept at the start of the sequence
    page_tokens: int = 0  # 128: paged cache (a pool of n_pages pages, block table per layer)
    n_pages: int = 0
    kv_format: int = 0    # KVQ_FMT_INT; or, with k_bits = v_bits = 8, KVQ_FMT_E4M3 (FP8),
    #                       KVQ_FMT_ASYM (zero-point) or KVQ_FMT_TENSOR (one scale per tensor)

    def _key(self):
        return (self.mode, self.batch, self.capacity, self.n_layers, self.n_q_heads,
                self.n_kv_heads, self.head_dim, self.k_bits, self.v_bits,
                self.k_group or self.head_dim, self.v_group or self.head_dim,
                self.d_model, self.h_bits, self.h_groups, self.window, self.n_anchor,
                self.page_tokens, self.n_pages, self.kv_format)

    def c(self) -> KvqConfig:
        """A new ``kvq_config`` struct with these fields."""
        return KvqConfig(*self._key())

    def _ref(self):
        """byref() of a shared struct with these fields (read-only use by the wrappers)."""
        if self._memo is not None:
            return self._memo
        key = self._key()
        r = _CFG_MEMO.get(key)
        if r is None:
            if len(_CFG_MEMO) > 256:
                _CFG_MEMO.clear()
            c = KvqConfig(*key)
            r = _CFG_MEMO[key] = (c, ctypes.byref(c))
        self._memo = r[1]
        return r[1]


# ----------------------------------------------------------------------------- host-only calls

def kvq_cache_bytes(cfg: Config):
    a, b, c = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    _check("kvq_cache_bytes", _lib.kvq_cache_bytes(ctypes.byref(cfg.c()), ctypes.byref(a),
                                                   ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def kvq_layer_buffer_bytes(cfg: Config):
    v = [ctypes.c_uint64() for _ in range(4)]
    _check("kvq_layer_buffer_bytes",
           _lib.kvq_layer_buffer_bytes(ctypes.byref(cfg.c()), *[ctypes.byref(x) for x in v]))
    return tuple(x.value for x in v)


def kvq_workspace_bytes(cfg: Config, num_ctas: int = 0) -> int:
    v = ctypes.c_uint64()
    _check("kvq_workspace_bytes", _lib.kvq_workspace_bytes(ctypes.byref(cfg.c()), num_ctas,
                                                           ctypes.byref(v)))
    return v.value


def kvq_decode_plan_info(cfg: Config, num_ctas: int = 0) -> dict:
    """The decode launch the library makes for cfg: engine, CTAs, ring depth, shared memory."""
    v = KvqDecodePlan()
    _check("kvq_decode_plan_info", _lib.kvq_decode_plan_info(ctypes.byref(cfg.c()), num_ctas,
                                                             ctypes.byref(v)))
    return {n: getattr(v, n) for n, _ in KvqDecodePlan._fields_}


def kvq_h_scratch_bytes(cfg: Config, max_len: int) -> int:
    v = ctypes.c_uint64()
    _check("kvq_h_scratch_bytes", _lib.kvq_h_scratch_bytes(ctypes.byref(cfg.c()), max_len,
                                                           ctypes.byref(v)))
    return v.value


# ----------------------------------------------------------------------------- device buffers

class LayerCache(_Memo):
    """One layer's cache buffers, allocated with torch on `device` (caller-owned memory).
    A paged config allocates the page pool; `block_table` (int32 [B][capacity/128] on
    the device) then maps each sequence's logical pages to pool pages."""

    block_table = None

    def __init__(self, cfg: Config, device="cuda", zero: bool = False, block_table=None):
        kc, ks, vc, vs = kvq_layer_buffer_bytes(cfg)
        alloc = torch.zeros if zero else torch.empty
        self.k_codes = alloc(max(kc, 16), dtype=torch.uint8, device=device)
        self.k_scales = alloc(max(ks // 2, 8), dtype=torch.float16, device=device) if ks else None
        self.v_codes = alloc(max(vc, 16), dtype=torch.uint8, device=device) if vc else None
        self.v_scales = alloc(max(vs // 2, 8), dtype=torch.float16, device=device) if vs else None
        self.cfg = cfg
        self.block_table = block_table

    @classmethod
    def from_buffers(cls, cfg: Config, k_codes, k_scales, v_codes, v_scales, block_table=None):
        """A layer over buffers the caller already holds (contiguous; sized as
        ``kvq_layer_buffer_bytes`` says; None for one the config does not use)."""
        self = cls.__new__(cls)
        parts = (k_codes, k_scales, v_codes, v_scales)
        for t, need in zip(parts, kvq_layer_buffer_bytes(cfg)):
            have = 0 if t is None else t.numel() * t.element_size()
            if have < need or (t is not None and not t.is_contiguous()):
                raise ValueError(f"a layer buffer is not contiguous or holds {have} of {need} bytes")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = parts
        self.cfg = cfg
        self.block_table = block_table
        return self

    def c(self) -> KvqLayer:
        """A new ``kvq_layer`` struct with these buffers."""
        return KvqLayer(*(None if t is None else t.data_ptr()
                          for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales,
                                    self.block_table)))

    def _kept(self):
        """A struct kept for these buffers (read-only use by the wrappers): byref() of it, its
        bytes (for arrays of layers), the buffers' device."""
        if self._memo is None:
            c = self.c()
            self._memo = (ctypes.byref(c), bytes(c), self.k_codes.get_device())
        return self._memo

    def _ref(self):
        return self._kept()[0]


class Workspace:
    """Split-KV partials and merge counters, sized by kvq_workspace_bytes and zero-filled
    (a call leaves it ready for the next; zero it again after a timeout status)."""

    def __init__(self, cfg: Config, num_ctas: int = 0, device="cuda"):
        self.nbytes = kvq_workspace_bytes(cfg, num_ctas)
        self.buf = torch.zeros(self.nbytes // 4 + 64, dtype=torch.float32, device=device)


# ----------------------------------------------------------------------------- device calls

def kvq_append(cfg: Config, layer: LayerCache, k: torch.Tensor, v, d_pos: torch.Tensor,
               max_pos: int, n_new: int, stream=None):
    _check("kvq_append", _lib.kvq_append(cfg._ref(), layer._ref(), _ptr(k),
                                         _ptr(v), _dtype_code(k), _ptr(d_pos), int(max_pos),
                                         int(n_new), _stream(stream)))


def kvq_decode_attn(cfg: Config, layer: LayerCache, q: torch.Tensor, d_len: torch.Tensor,
                    max_len: int, out: torch.Tensor, ws: Workspace, softmax_scale: float = 0.0,
                    num_ctas: int = 0, w_kv=None, kv_scratch=None, stream=None):
    scratch_bytes = 0 if kv_scratch is None else kv_scratch.numel() * kv_scratch.element_size()
    _check("kvq_decode_attn",
           _lib.kvq_decode_attn(cfg._ref(), layer._ref(), _ptr(q),
                                _dtype_code(q), _ptr(d_len), int(max_len), float(softmax_scale),
                                _ptr(out), _dtype_code(out), _ptr(ws.buf), ws.nbytes,
                                int(num_ctas), _ptr(w_kv), _ptr(kv_scratch), scratch_bytes,
                                _stream(stream)))


def kvq_append_decode_attn(cfg: Config, layer: LayerCache, k_new: torch.Tensor,
                           v_new: torch.Tensor, q: torch.Tensor, d_len: torch.Tensor, max_len: int,
                           out: torch.Tensor, ws: Workspace, softmax_scale: float = 0.0,
                           num_ctas: int = 0, stream=None):
    """One decode step: quantise k_new/v_new ([B][Hkv][Dh]) into position d_len-1, then attend."""
    if k_new.dtype != v_new.dtype:
        raise ValueError("k_new and v_new must share a dtype")
    _check("kvq_append_decode_attn",
           _lib.kvq_append_decode_attn(cfg._ref(), layer._ref(), _ptr(k_new),
                                       _ptr(v_new), _dtype_code(k_new), _ptr(q), _dtype_code(q),
                                       _ptr(d_len), int(max_len), float(softmax_scale), _ptr(out),
                                       _dtype_code(out), _ptr(ws.buf), ws.nbytes, int(num_ctas),
                                       _stream(stream)))


def kvq_decode_partials(cfg: Config, layer: LayerCache, q: torch.Tensor, d_len: torch.Tensor,
                        max_len: int, ws: Workspace, softmax_scale: float = 0.0, num_ctas: int = 0,
                        stream=None):
    _check("kvq_decode_partials",
           _lib.kvq_decode_partials(cfg._ref(), layer._ref(), _ptr(q),
                                    _dtype_code(q), _ptr(d_len), int(max_len), float(softmax_scale),
                                    _ptr(ws.buf), ws.nbytes, int(num_ctas), _stream(stream)))


def kvq_merge_partials(cfg: Config, d_len: torch.Tensor, out: torch.Tensor, ws: Workspace,
                       num_ctas: int = 0, stream=None):
    _check("kvq_merge_partials",
           _lib.kvq_merge_partials(cfg._ref(), _ptr(d_len), _ptr(out), _dtype_code(out),
                                   _ptr(ws.buf), ws.nbytes, int(num_ctas), _stream(stream)))


def kvq_h_operand_bytes(cfg: Config, max_len: int) -> int:
    v = ctypes.c_uint64()
    _check("kvq_h_operand_bytes", _lib.kvq_h_operand_bytes(cfg._ref(), max_len,
                                                           ctypes.byref(v)))
    return v.value


def kvq_h_reconstruct(cfg: Config, layer: LayerCache, w_kv: torch.Tensor, max_len: int,
                      k_out: torch.Tensor, v_out: torch.Tensor, out_capacity: int,
                      operand: torch.Tensor, stream=None):
    _check("kvq_h_reconstruct",
           _lib.kvq_h_reconstruct(cfg._ref(), layer._ref(), _ptr(w_kv),
                                  int(max_len), _ptr(k_out), _ptr(v_out), int(out_capacity),
                                  _ptr(operand), operand.numel() * operand.element_size(),
                                  _stream(stream)))


def kvq_h_absorbed_scratch_bytes(cfg: Config, max_len: int) -> int:
    v = ctypes.c_uint64()
    _check("kvq_h_absorbed_scratch_bytes",
           _lib.kvq_h_absorbed_scratch_bytes(cfg._ref(), int(max_len), ctypes.byref(v)))
    return v.value


def kvq_h_decode_absorbed(cfg: Config, layer: LayerCache, w_kv: torch.Tensor, q: torch.Tensor,
                          d_len: torch.Tensor, max_len: int, out: torch.Tensor,
                          scratch: torch.Tensor, softmax_scale: float = 0.0, stream=None):
    """h-mode decode attention by query absorption (W_k^T q against the h codes)."""
    _check("kvq_h_decode_absorbed",
           _lib.kvq_h_decode_absorbed(cfg._ref(), layer._ref(), _ptr(w_kv), _ptr(q),
                                      _dtype_code(q), _ptr(d_len), int(max_len),
                                      float(softmax_scale), _ptr(out), _dtype_code(out),
                                      _ptr(scratch), scratch.numel() * scratch.element_size(),
                                      _stream(stream)))


def kvq_h_fused_scratch_bytes(cfg: Config, max_len: int) -> int:
    v = ctypes.c_uint64()
    _check("kvq_h_fused_scratch_bytes",
           _lib.kvq_h_fused_scratch_bytes(cfg._ref(), int(max_len), ctypes.byref(v)))
    return v.value


def kvq_h_decode_fused(cfg: Config, layer: LayerCache, w_kv: torch.Tensor, q: torch.Tensor,
                       d_len: torch.Tensor, max_len: int, out: torch.Tensor, scratch: torch.Tensor,
                       softmax_scale: float = 0.0, stream=None):
    """h-mode decode attention with the K/V reconstruction fused into the GEMM epilogue.
    `scratch` starts with a status word (zero it once; read it with kvq_workspace_status)."""
    _check("kvq_h_decode_fused",
           _lib.kvq_h_decode_fused(cfg._ref(), layer._ref(), _ptr(w_kv), _ptr(q),
                                   _dtype_code(q), _ptr(d_len), int(max_len),
                                   float(softmax_scale), _ptr(out), _dtype_code(out),
                                   _ptr(scratch), scratch.numel() * scratch.element_size(),
                                   _stream(stream)))


def kvq_selftest_bounded_wait(ws, timeout_ns: int, stream=None):
    """Run the kernels' bounded wait on a barrier nothing completes (see kvq.h)."""
    buf = ws.buf if isinstance(ws, Workspace) else ws
    _check("kvq_selftest_bounded_wait",
           _lib.kvq_selftest_bounded_wait(_ptr(buf), int(timeout_ns), _stream(stream)))


def kvq_selftest_decode_timeout(cfg: Config, layer: LayerCache, q: torch.Tensor,
                                d_len: torch.Tensor, out: torch.Tensor, ws: Workspace,
                                timeout_ns: int, stream=None):
    """The decode kernel with a producer that copies nothing: its waits run out (see kvq.h)."""
    _check("kvq_selftest_decode_timeout",
           _lib.kvq_selftest_decode_timeout(cfg._ref(), layer._ref(), _ptr(q), _dtype_code(q),
                                            _ptr(d_len), _ptr(out), _dtype_code(out),
                                            _ptr(ws.buf), ws.nbytes, int(timeout_ns),
                                            _stream(stream)))


def kvq_decode_attn_noalloc(cfg: Config, layer: LayerCache, q: torch.Tensor, d_len: torch.Tensor,
                            max_len: int, out: torch.Tensor, softmax_scale: float = 0.0,
                            num_ctas: int = 0, stream=None):
    """kvq_decode_attn with the library's own fixed device array as the workspace
    (for callers that may not allocate device memory; see kvq.h)."""
    _check("kvq_decode_attn_noalloc",
           _lib.kvq_decode_attn_noalloc(cfg._ref(), layer._ref(), _ptr(q), _dtype_code(q),
                                        _ptr(d_len), int(max_len), float(softmax_scale), _ptr(out),
                                        _dtype_code(out), int(num_ctas), _stream(stream)))


def kvq_noalloc_status(stream=None) -> int:
    """Read and clear the status word of the noalloc entry point's device array."""
    st = ctypes.c_int32()
    _check("kvq_noalloc_status", _lib.kvq_noalloc_status(ctypes.byref(st), _stream(stream)))
    return st.value


def kvq_selftest_noalloc_timeout(cfg: Config, layer: LayerCache, q: torch.Tensor,
                                 d_len: torch.Tensor, out: torch.Tensor, timeout_ns: int,
                                 stream=None):
    """The stalled-producer decode kernel run on the noalloc array (see kvq.h)."""
    _check("kvq_selftest_noalloc_timeout",
           _lib.kvq_selftest_noalloc_timeout(cfg._ref(), layer._ref(), _ptr(q), _dtype_code(q),
                                             _ptr(d_len), _ptr(out), _dtype_code(out),
                                             int(timeout_ns), _stream(stream)))


def kvq_workspace_status(ws, stream=None) -> int:
    """Read and clear the status word of a Workspace (or of a scratch tensor that starts
    with one, as the fused h-mode path's)."""
    st = ctypes.c_int32()
    buf = ws.buf if isinstance(ws, Workspace) else ws
    _check("kvq_workspace_status", _lib.kvq_workspace_status(_ptr(buf), ctypes.byref(st),
                                                             _stream(stream)))
    return st.value


# ----------------------------------------------------------------------------- drafted tokens

@dataclass
class RopeConfig(_Memo):
    """Python view of ``kvq_rope_config`` (see include/kvq.h for the meaning of each field).
    ``low`` and ``high`` default to 1 and 32 turns (YARN) or 1 and 4 (BANDS)."""
    rot_dim: int
    layout: int = KVQ_ROPE_HALF
    scaling: int = KVQ_ROPE_PLAIN
    base: float = 10000.0
    factor: float = 1.0
    orig_len: int = 0
    low: float = 1.0
    high: float = 0.0
    gain: float = 0.0

    def c(self) -> KvqRopeConfig:
        high = self.high or (32.0 if self.scaling == KVQ_ROPE_YARN else 4.0)
        return KvqRopeConfig(self.rot_dim, self.layout, self.scaling, self.orig_len, self.base,
                             self.factor, self.low, high, self.gain)

    def _ref(self):
        if self._memo is None:
            self._memo = ctypes.byref(self.c())
        return self._memo


class TreeWorkspace(Workspace):
    """Workspace of ``kvq_tree_attn`` (as Workspace: zero-filled, ready after every call)."""

    def __init__(self, cfg: Config, n_tree: int, num_ctas: int = 0, device="cuda"):
        v = ctypes.c_uint64()
        _check("kvq_tree_workspace_bytes",
               _lib.kvq_tree_workspace_bytes(cfg._ref(), int(n_tree), int(num_ctas), ctypes.byref(v)))
        self.nbytes = v.value
        self.n_tree = n_tree
        self.buf = torch.zeros(self.nbytes // 4 + 64, dtype=torch.float32, device=device)


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _here(stream, layers, *tensors):
    """The kernels run on the current device: every layer and tensor has to be there.  Returns the
    stream's handle (the current one's for None)."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")
    for x in layers:
        if x._kept()[2] != dev:
            raise ValueError(f"a layer is on {x.k_codes.device}, the current device is cuda:{dev}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _ints(t, shape, what: str):
    if t is not None and (t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what} is a contiguous int32 tensor of shape {tuple(shape)}")


_pack_rows = struct.Struct("Pqq").pack


def _rows(t: torch.Tensor, n: int, heads: int, dim: int, batch: int, dtype, what: str):
    """The kvq_rows of a [B][n][heads][dim] view, as its bytes (None for None)."""
    if t is None:
        return None
    if t.shape != (batch, n, heads, dim) or t.dtype is not dtype:
        raise ValueError(f"{what} is {dtype} of shape {(batch, n, heads, dim)}")
    sb, st, sh, sd = t.stride()
    if (sd != 1 and dim > 1 or sh != dim and heads > 1) and t.numel():
        raise ValueError(f"the heads of a token of {what} are contiguous")
    # a stride that no index uses is whatever torch says: 0 selects the contiguous one
    if batch == 1:
        sb = 0
    elif sb == 0:
        raise ValueError(f"{what} is an expanded view: its rows share memory")
    if n == 1:
        st = 0
    elif st == 0 and n:
        raise ValueError(f"{what} is an expanded view: its rows share memory")
    return _pack_rows(t.data_ptr(), sb, st)


def kvq_rope_table(rope: RopeConfig, n_pos: int, first_pos: int = 0, table=None, device="cuda",
                   stream=None) -> torch.Tensor:
    """(cos, sin) of positions first_pos ..: float32 [n_pos][rot_dim/2][2], made once per model."""
    if table is None:
        table = torch.empty(n_pos, rope.rot_dim // 2, 2, dtype=torch.float32, device=device)
    _need(table.dtype == torch.float32 and table.is_contiguous() and
          table.shape == (n_pos, rope.rot_dim // 2, 2), "table is contiguous float32 [n_pos][rot_dim/2][2]")
    _check("kvq_rope_table", _lib.kvq_rope_table(rope._ref(), int(first_pos), int(n_pos),
                                                 _ptr(table), _here(stream, (), table)))
    return table


def kvq_rope_append(cfg: Config, layer: LayerCache, rope: RopeConfig, table: torch.Tensor, q, k: torch.Tensor,
                    v: torch.Tensor, q_out, d_pos: torch.Tensor, max_pos: int, d_count=None, d_rope_pos=None,
                    stream=None):
    """Rotate new queries and keys and quantise keys and values into the cache, in one launch.
    q, q_out [B][n][Hq][Dh] (both None: keys only), k, v [B][n][Hkv][Dh]: views whose token and
    batch strides are free (e.g. parts of one projection's output)."""
    B, n = k.shape[:2]
    rows = table.shape[0] if table.dim() else 0
    _need(table.dtype is torch.float32 and table.is_contiguous() and table.shape == (rows, rope.rot_dim // 2, 2),
          "table is contiguous float32 [positions][rot_dim/2][2]")
    st = _here(stream, (layer,), table, q, k, v, q_out, d_pos, d_count, d_rope_pos)
    _ints(d_pos, (cfg.batch,), "d_pos")
    _ints(d_count, (cfg.batch,), "d_count")
    _ints(d_rope_pos, (cfg.batch, n), "d_rope_pos")
    _check("kvq_rope_append", _lib.kvq_rope_append(
        cfg._ref(), layer._ref(), rope._ref(), table.data_ptr(), rows,
        _rows(q, n, cfg.n_q_heads, cfg.head_dim, cfg.batch, k.dtype, "q"),
        _rows(k, n, cfg.n_kv_heads, cfg.head_dim, cfg.batch, k.dtype, "k"),
        _rows(v, n, cfg.n_kv_heads, cfg.head_dim, cfg.batch, k.dtype, "v"),
        _rows(q_out, n, cfg.n_q_heads, cfg.head_dim, cfg.batch, k.dtype, "q_out"),
        _dtype_code(k), _ptr(d_pos), int(max_pos), n, _ptr(d_count), _ptr(d_rope_pos), st))


def kvq_read(cfg: Config, layer: LayerCache, k_out, v_out, d_pos: torch.Tensor, max_pos: int, d_count=None,
             stream=None):
    """Cached tokens d_pos .. d_pos + n - 1 as values: k_out, v_out [B][n][Hkv][Dh] (either None;
    h-mode: k_out [B][n][d_model]), views as in kvq_rope_append."""
    some = k_out if k_out is not None else v_out
    _need(some is not None, "k_out or v_out is given")
    n = some.shape[1]
    st = _here(stream, (layer,), k_out, v_out, d_pos, d_count)
    _ints(d_pos, (cfg.batch,), "d_pos")
    _ints(d_count, (cfg.batch,), "d_count")
    heads, dim = cfg.n_kv_heads, cfg.head_dim
    if cfg.mode == KVQ_MODE_H:
        heads, dim = 1, cfg.d_model
        k_out = None if k_out is None else k_out.unsqueeze(2)
    _check("kvq_read", _lib.kvq_read(
        cfg._ref(), layer._ref(), _rows(k_out, n, heads, dim, cfg.batch, some.dtype, "k_out"),
        _rows(v_out, n, heads, dim, cfg.batch, some.dtype, "v_out"), _dtype_code(some), _ptr(d_pos),
        int(max_pos), n, _ptr(d_count), st))


def kvq_tree_attn(cfg: Config, layer: LayerCache, q: torch.Tensor, d_len: torch.Tensor, max_len: int, d_mask,
                  out: torch.Tensor, ws: TreeWorkspace, d_n_tree=None, softmax_scale: float = 0.0,
                  num_ctas: int = 0, stream=None):
    """Attention of drafted tokens: q, out [B][n_tree][Hq][Dh], d_len cached tokens before them,
    d_mask int64 [B][n_tree] (bit j: the token attends drafted token j; None: causal)."""
    shape = (cfg.batch, q.shape[1], cfg.n_q_heads, cfg.head_dim)
    _need(q.shape == shape and out.shape == shape and q.is_contiguous() and out.is_contiguous(),
          "q and out are contiguous [B][n_tree][Hq][Dh]")
    if d_mask is not None:
        _need(d_mask.dtype == torch.int64 and d_mask.shape == shape[:2] and d_mask.is_contiguous(),
              "d_mask is a contiguous int64 tensor [B][n_tree]")
    st = _here(stream, (layer,), q, d_len, d_mask, d_n_tree, out, ws.buf)
    _ints(d_len, (cfg.batch,), "d_len")
    _ints(d_n_tree, (cfg.batch,), "d_n_tree")
    _check("kvq_tree_attn", _lib.kvq_tree_attn(
        cfg._ref(), layer._ref(), _ptr(q), _dtype_code(q), shape[1], _ptr(d_len), int(max_len), _ptr(d_n_tree),
        _ptr(d_mask), float(softmax_scale), _ptr(out), _dtype_code(out), _ptr(ws.buf), ws.nbytes, int(num_ctas), st))


def kvq_tree_commit(cfg: Config, layers, d_len: torch.Tensor, max_len: int, d_path: torch.Tensor,
                    d_n_path: torch.Tensor, n_tree: int, d_len_out=None, stream=None):
    """Keep the accepted path of every sequence in all `layers` (LayerCache objects) at once:
    row d_len + path[i] moves to d_len + i; d_len_out receives d_len + the path's length."""
    _need(d_path.dim() == 2, "d_path is a contiguous int32 tensor [B][n]")
    st = _here(stream, layers, d_len, d_path, d_n_path, d_len_out)
    _ints(d_len, (cfg.batch,), "d_len")
    _ints(d_path, (cfg.batch, d_path.shape[1]), "d_path")
    _ints(d_n_path, (cfg.batch,), "d_n_path")
    _ints(d_len_out, (cfg.batch,), "d_len_out")
    _check("kvq_tree_commit", _lib.kvq_tree_commit(
        cfg._ref(), b"".join([x._kept()[1] for x in layers]), len(layers), _ptr(d_len), int(max_len), int(n_tree), _ptr(d_path), d_path.shape[1],
        _ptr(d_n_path), _ptr(d_len_out), st))


def kvq_selftest_tree_timeout(cfg: Config, layer: LayerCache, q: torch.Tensor, d_len: torch.Tensor, max_len: int,
                              out: torch.Tensor, ws: TreeWorkspace, n_segments: int, timeout_ns: int,
                              num_ctas: int = 0, stream=None):
    """kvq_tree_attn with a producer that stops after n_segments segments: its waits run out (see kvq.h)."""
    _need(q.dim() == 4 and q.shape == out.shape == (cfg.batch, q.shape[1], cfg.n_q_heads, cfg.head_dim)
          and q.is_contiguous() and out.is_contiguous(), "q and out are contiguous [B][n_tree][Hq][Dh]")
    st = _here(stream, (layer,), q, d_len, out, ws.buf)
    _ints(d_len, (cfg.batch,), "d_len")
    _check("kvq_selftest_tree_timeout", _lib.kvq_selftest_tree_timeout(
        cfg._ref(), layer._ref(), _ptr(q), _dtype_code(q), q.shape[1], _ptr(d_len), int(max_len), _ptr(out),
        _dtype_code(out), _ptr(ws.buf), ws.nbytes, int(num_ctas), int(n_segments), int(timeout_ns), st))
