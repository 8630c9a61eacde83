"""Thin ctypes binding of liblyc.so (declared in include/lyc.h).

Every step of the decode path runs in the library's CUDA kernels; this module
only marshals arguments.  The functions ``lyc_*`` mirror the C entry points
one to one (raw pointers and sizes); ``Lyc`` is a convenience wrapper that
takes torch tensors and passes their device pointers.  Importing this module
on a machine where the library is not built raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblyc.so")

LYC_OK = 0
LYC_ERR_INVALID_ARG = -1
LYC_ERR_UNSUPPORTED = -2
LYC_ERR_OOM = -3
LYC_ERR_CUDA = -4
LYC_ERR_BAD_INDEX = -5
LYC_ERR_TIMEOUT = -6
LYC_ERR_SCRATCH_LIMIT = -7

LYC_NOALLOC_MAX_SETS = 256
LYC_NOALLOC_MAX_CTAS = 32

LYC_BF16 = 0
LYC_FP32 = 1
LYC_SELECT_PER_QHEAD = 0
LYC_SELECT_KVGROUP_MEAN = 1

LYC_CFG_TMA_GATHER = 0x1
LYC_CFG_TCGEN05 = 0x2

LYC_STEP_S_IN = 0x1
LYC_STEP_NO_GRAPH = 0x2
LYC_STEP_VALIDATE_S = 0x4

LYC_TIMING_OFF = 0
LYC_TIMING_ON = 1

LYC_RULE_TOPK = 0
LYC_RULE_RATIO = 1
LYC_RULE_BLOCK_TOPK = 2
LYC_RULE_TOPP = 3
LYC_RULE_THRESHOLD = 4

LYC_TOPK_FIXED = 0
LYC_TOPK_RULES = 1

LYC_CACHE_BF16 = 0
LYC_CACHE_E4M3 = 1
LYC_OP_BAD_LENGTH = 0x1
LYC_OP_BAD_PAGE = 0x2
LYC_OP_BAD_INDEX = 0x4
LYC_OP_TIMEOUT = 0x8

EXPORTED = ["lyc_create", "lyc_decode_step", "lyc_decode_step_host", "lyc_decode_step_batch",
            "lyc_sync_status",
            "lyc_set_s_trace", "lyc_step_bytes", "lyc_step_launches", "lyc_topk_f32", "lyc_topk_f32_ex",
            "lyc_set_timing",
            "lyc_kernel_times", "lyc_set_timeline", "lyc_status_string", "lyc_last_error",
            "lyc_destroy", "lyc_sparse_attention_noalloc", "lyc_set_selection", "lyc_cache_correction",
            "lyc_qk_norm_rope", "lyc_cache_append", "lyc_cache_read", "lyc_tree_workspace_bytes",
            "lyc_tree_attention", "lyc_operator_error", "lyc_operator_status"]


class lyc_config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("batch", ctypes.c_int),
                ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_ctx", ctypes.c_int64),
                ("max_k", ctypes.c_int), ("dtype", ctypes.c_int),
                ("select_mode", ctypes.c_int), ("device", ctypes.c_int),
                ("flags", ctypes.c_uint32)]


class lyc_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("s_layer", ctypes.c_int64), ("s_batch", ctypes.c_int64),
                ("s_head", ctypes.c_int64), ("s_token", ctypes.c_int64)]


class lyc_kv_batch(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n", ctypes.c_void_p),
                ("s_layer", ctypes.c_int64), ("s_batch", ctypes.c_int64),
                ("s_head", ctypes.c_int64), ("s_token", ctypes.c_int64),
                ("s_page", ctypes.c_int64), ("block_table", ctypes.c_void_p),
                ("page_rows", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("k_new", ctypes.c_void_p),
                ("v_new", ctypes.c_void_p)]


class lyc_selection(ctypes.Structure):
    _fields_ = [("rule", ctypes.c_int32), ("block", ctypes.c_int32),
                ("ratio_num", ctypes.c_int64), ("ratio_den", ctypes.c_int64),
                ("p", ctypes.c_double), ("tau", ctypes.c_double)]


class lyc_kernel_time(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("layer", ctypes.c_int), ("ms", ctypes.c_float)]


def _struct(name, doc, **fields):
    """A ctypes mirror of a struct of include/lyc.h: p = pointer, i = int32, l = int64, f = float,
    each value the fields of that type in a row, in the header's order."""
    types = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float}
    flat = [(n, types[key[0]]) for key, names in fields.items() for n in names.split()]
    return type(name, (ctypes.Structure,), {"_fields_": flat, "__doc__": doc})


lyc_layer_cache = _struct(
    "lyc_layer_cache", "One layer's cache (include/lyc.h).",
    p1="k v k_scale v_scale",
    l1="s_batch s_head s_token s_page ss_batch ss_head ss_token ss_page",
    p2="block_table", l2="rows num_pages",
    i1="page_rows max_blocks type batch num_kv_heads head_dim device")
lyc_rope_args = _struct(
    "lyc_rope_args", "Arguments of lyc_qk_norm_rope.",
    p1="q k q_out k_out",
    l1="q_row q_head k_row k_head qo_row qo_head ko_row ko_head",
    p2="pos inv_freq q_weight k_weight", l2="rows",
    i1="num_q_heads num_kv_heads head_dim rot_dim interleaved", f1="eps", i2="dtype device")
lyc_append_args = _struct(
    "lyc_append_args", "Arguments of lyc_cache_append.",
    p1="k v q q_out",
    l1="k_batch k_token k_head v_batch v_token v_head q_batch q_token q_head qo_batch qo_token qo_head",
    p2="n t_len pos inv_freq q_weight k_weight",
    i1="T num_q_heads rot_dim interleaved", f1="eps", p3="status")
lyc_read_args = _struct(
    "lyc_read_args", "Arguments of lyc_cache_read.",
    p1="k_out v_out", l1="o_batch o_head o_row", p2="n sets", l2="first",
    i1="m num_heads dtype", p3="status")
lyc_tree_args = _struct(
    "lyc_tree_args", "Arguments of lyc_tree_attention.",
    p1="q out", l1="q_batch q_token q_head o_batch o_token o_head",
    p2="n t_len mask", i1="T num_q_heads", f1="scale", p3="workspace", l2="workspace_bytes", p4="status")


class LycError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code}) {detail}".rstrip())


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblyc.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m hybrid_head_sparse_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(path)
    P = ctypes.c_void_p
    I = ctypes.c_int
    L.lyc_create.argtypes = [ctypes.POINTER(lyc_config), ctypes.POINTER(P)]
    L.lyc_decode_step.argtypes = [P, P, ctypes.POINTER(lyc_kv_cache), P, I, P, P, P, ctypes.c_uint32]
    L.lyc_decode_step_host.argtypes = [P, P, ctypes.POINTER(lyc_kv_cache), P, I, P, P, P,
                                       ctypes.c_uint32]
    L.lyc_decode_step_batch.argtypes = [P, P, ctypes.POINTER(lyc_kv_batch), P, I, P, P, P,
                                        ctypes.c_uint32]
    L.lyc_sync_status.argtypes = [P]
    L.lyc_set_selection.argtypes = [P, ctypes.POINTER(lyc_selection)]
    L.lyc_cache_correction.argtypes = [P, P, ctypes.POINTER(lyc_kv_cache), I, P, P, P, P]
    L.lyc_set_s_trace.argtypes = [P, P]
    L.lyc_step_bytes.argtypes = [ctypes.POINTER(lyc_config), P, ctypes.c_int64, I, I,
                                 ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)]
    L.lyc_step_launches.argtypes = [P, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I)]
    L.lyc_topk_f32.argtypes = [P, P, ctypes.c_int64, I, P, P]
    L.lyc_topk_f32_ex.argtypes = [P, P, ctypes.c_int64, I, P, I, I, P]
    L.lyc_set_timing.argtypes = [P, I]
    L.lyc_set_timeline.argtypes = [P, P, I]
    L.lyc_kernel_times.argtypes = [P, ctypes.POINTER(lyc_kernel_time), I, ctypes.POINTER(I)]
    L.lyc_status_string.argtypes = [I]
    L.lyc_status_string.restype = ctypes.c_char_p
    L.lyc_last_error.argtypes = [P]
    L.lyc_last_error.restype = ctypes.c_char_p
    L.lyc_destroy.argtypes = [P]
    L.lyc_destroy.restype = None
    L.lyc_sparse_attention_noalloc.argtypes = [P, ctypes.POINTER(lyc_kv_cache), I, I, I, I, P, I,
                                               P, P, P]
    L.lyc_qk_norm_rope.argtypes = [P, P]
    L.lyc_cache_append.argtypes = [ctypes.POINTER(lyc_layer_cache), P, P]
    L.lyc_cache_read.argtypes = [ctypes.POINTER(lyc_layer_cache), P, P]
    L.lyc_tree_workspace_bytes.argtypes = [ctypes.POINTER(lyc_layer_cache), I, I]
    L.lyc_tree_attention.argtypes = [ctypes.POINTER(lyc_layer_cache), P, P]
    for name in EXPORTED:
        if name not in ("lyc_status_string", "lyc_last_error", "lyc_destroy"):
            getattr(L, name).restype = I
    L.lyc_tree_workspace_bytes.restype = ctypes.c_uint64
    L.lyc_operator_error.restype = ctypes.c_char_p
    _lib = L
    return L


# ------------------------------------------------------------ C-named functions


def lyc_create(cfg: lyc_config) -> int:
    ctx = ctypes.c_void_p()
    rc = load().lyc_create(ctypes.byref(cfg), ctypes.byref(ctx))
    if rc != LYC_OK:
        raise LycError(rc, "lyc_create")
    return ctx.value


def lyc_decode_step(ctx, q, kv: lyc_kv_cache, role_mask, k, out, S, stream, flags) -> int:
    return load().lyc_decode_step(ctx, q, ctypes.byref(kv), role_mask, k, out, S, stream, flags)


def lyc_decode_step_host(ctx, q, kv: lyc_kv_cache, role_mask, k, out, S, stream, flags) -> int:
    return load().lyc_decode_step_host(ctx, q, ctypes.byref(kv), role_mask, k, out, S, stream,
                                       flags)


def lyc_decode_step_batch(ctx, q, kv: lyc_kv_batch, role_mask, k, out, S, stream, flags) -> int:
    return load().lyc_decode_step_batch(ctx, q, ctypes.byref(kv), role_mask, k, out, S, stream,
                                        flags)


def lyc_sparse_attention_noalloc(q, kv: lyc_kv_cache, batch, num_q_heads, num_kv_heads,
                                 head_dim, S, k, out, status, stream) -> int:
    """The allocation-free sparse attention of one layer (include/lyc.h).
    Pointers are ints (device addresses); status may be None."""
    return load().lyc_sparse_attention_noalloc(q, ctypes.byref(kv), batch, num_q_heads,
                                               num_kv_heads, head_dim, S, k, out, status,
                                               stream)


def lyc_sync_status(ctx) -> int:
    return load().lyc_sync_status(ctx)


def lyc_set_selection(ctx, sel: lyc_selection | None) -> int:
    return load().lyc_set_selection(ctx, None if sel is None else ctypes.byref(sel))


def lyc_cache_correction(ctx, q, kv: lyc_kv_cache, T, k_new, v_new, out, stream) -> int:
    return load().lyc_cache_correction(ctx, q, ctypes.byref(kv), T, k_new, v_new, out, stream)


def lyc_set_s_trace(ctx, trace) -> int:
    return load().lyc_set_s_trace(ctx, trace)


def lyc_step_bytes(cfg: lyc_config, role_mask: np.ndarray, n: int, k: int, s_in: bool = False):
    a = ctypes.c_uint64()
    d = ctypes.c_uint64()
    role_mask = np.ascontiguousarray(role_mask, dtype=np.uint8)
    rc = load().lyc_step_bytes(ctypes.byref(cfg), role_mask.ctypes.data, n, k, int(s_in),
                               ctypes.byref(a), ctypes.byref(d))
    if rc != LYC_OK:
        raise LycError(rc, "lyc_step_bytes")
    return a.value, d.value


def lyc_topk_f32(ctx, keys, n, k, S, stream) -> int:
    return load().lyc_topk_f32(ctx, keys, n, k, S, stream)


def lyc_topk_f32_ex(ctx, keys, n, k, S, cluster, variant, stream) -> int:
    return load().lyc_topk_f32_ex(ctx, keys, n, k, S, cluster, variant, stream)


def lyc_set_timing(ctx, mode: int) -> int:
    return load().lyc_set_timing(ctx, mode)


def lyc_kernel_times(ctx, cap: int = 1 << 16):
    arr = (lyc_kernel_time * cap)()
    cnt = ctypes.c_int()
    rc = load().lyc_kernel_times(ctx, arr, cap, ctypes.byref(cnt))
    if rc != LYC_OK:
        raise LycError(rc, "lyc_kernel_times")
    return [(arr[i].kind, arr[i].layer, arr[i].ms) for i in range(cnt.value)]


def lyc_set_timeline(ctx, buf, cap: int) -> int:
    return load().lyc_set_timeline(ctx, buf, cap)


def lyc_status_string(code: int) -> str:
    return load().lyc_status_string(code).decode()


def status_string(code: int) -> str:
    try:
        return lyc_status_string(code)
    except Exception:  # library missing: still format the error
        return "status"


def lyc_last_error(ctx) -> str:
    return load().lyc_last_error(ctx).decode()


def lyc_destroy(ctx) -> None:
    load().lyc_destroy(ctx)


def lyc_qk_norm_rope(args: lyc_rope_args, stream) -> int:
    return load().lyc_qk_norm_rope(ctypes.byref(args), stream)


def lyc_cache_append(cache: lyc_layer_cache, args: lyc_append_args, stream) -> int:
    return load().lyc_cache_append(cache, ctypes.byref(args), stream)


def lyc_cache_read(cache: lyc_layer_cache, args: lyc_read_args, stream) -> int:
    return load().lyc_cache_read(cache, ctypes.byref(args), stream)


def lyc_tree_workspace_bytes(cache: lyc_layer_cache, T: int, num_q_heads: int) -> int:
    """0 where lyc_tree_attention would refuse the arguments."""
    return load().lyc_tree_workspace_bytes(cache, T, num_q_heads)


def lyc_tree_attention(cache: lyc_layer_cache, args: lyc_tree_args, stream) -> int:
    return load().lyc_tree_attention(cache, ctypes.byref(args), stream)


def lyc_operator_error() -> str:
    return load().lyc_operator_error().decode()


def lyc_operator_status() -> int:
    """The code of this thread's last failing serving operator, LYC_OK if none did."""
    return load().lyc_operator_status()


# ------------------------------------------------------------ torch wrapper


def _dtype_code(dtype) -> int:
    import torch
    if dtype in ("bf16", torch.bfloat16, LYC_BF16):
        return LYC_BF16
    if dtype in ("fp32", torch.float32, LYC_FP32):
        return LYC_FP32
    raise ValueError(f"unsupported dtype {dtype}")


def _mode_code(mode) -> int:
    if mode in ("per_qhead", LYC_SELECT_PER_QHEAD):
        return LYC_SELECT_PER_QHEAD
    if mode in ("kvgroup_mean", LYC_SELECT_KVGROUP_MEAN):
        return LYC_SELECT_KVGROUP_MEAN
    raise ValueError(f"unknown select mode {mode}")


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class Lyc:
    """One library context.  Tensors are passed by device pointer."""

    def __init__(self, L, B, Hq, Hkv, d, max_ctx, max_k, dtype="bf16", select_mode="per_qhead",
                 device=0, flags=0):
        self.cfg = lyc_config(L, B, Hq, Hkv, d, max_ctx, max_k, _dtype_code(dtype),
                              _mode_code(select_mode), device, flags)
        self.ctx = lyc_create(self.cfg)
        self.Hs = Hkv if self.cfg.select_mode == LYC_SELECT_KVGROUP_MEAN else Hq
        self._trace = None

    def close(self):
        if self.ctx:
            lyc_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc, where):
        if rc != LYC_OK:
            raise LycError(rc, where, lyc_last_error(self.ctx))

    @staticmethod
    def kv_cache(K, V, n) -> lyc_kv_cache:
        """Describe [L][B][Hkv][rows][d]-strided torch tensors K, V."""
        assert K.stride() == V.stride() and K.shape == V.shape and K.stride(-1) == 1
        s = K.stride()
        return lyc_kv_cache(K.data_ptr(), V.data_ptr(), n, s[0], s[1], s[2], s[3])

    def decode_step(self, q, K, V, n, role_mask, k, out, S, stream=None, s_in=False,
                    no_graph=False, validate_s=False):
        role = np.ascontiguousarray(role_mask, dtype=np.uint8)
        self._role = role  # keep alive while the call runs
        flags = ((LYC_STEP_S_IN if s_in else 0) | (LYC_STEP_NO_GRAPH if no_graph else 0)
                 | (LYC_STEP_VALIDATE_S if validate_s else 0))
        kv = self.kv_cache(K, V, n)
        rc = lyc_decode_step(self.ctx, q.data_ptr(), kv, role.ctypes.data, k, out.data_ptr(),
                             S.data_ptr(), _stream_ptr(stream), flags)
        self._check(rc, "lyc_decode_step")

    def decode_step_batch(self, q, K, V, n, role_mask, k, out, S, stream=None, s_in=False,
                          validate_s=False, k_new=None, v_new=None, block_table=None,
                          page_rows=0, strides=None):
        """The serving form: n is a sequence of B row counts.  Contiguous cache:
        K, V are [L][B][Hkv][rows][d]-strided tensors.  Paged cache: K, V are
        [L][pages][page_rows][Hkv][d] tensors and block_table a device int32
        [B][max_blocks] tensor.  k_new/v_new: [L][B][Hkv][d] rows appended at
        n[b]-1 before attention, or None.  strides: optional (s_layer, s_batch,
        s_head, s_token, s_page) override in elements."""
        role = np.ascontiguousarray(role_mask, dtype=np.uint8)
        nn = np.ascontiguousarray(np.asarray(n, dtype=np.int64))
        self._role, self._n = role, nn  # keep alive while the call runs
        flags = (LYC_STEP_S_IN if s_in else 0) | (LYC_STEP_VALIDATE_S if validate_s else 0)
        assert K.stride() == V.stride() and K.shape == V.shape and K.stride(-1) == 1
        st = K.stride()
        if strides is not None:
            s_layer, s_batch, s_head, s_token, s_page = strides
        elif block_table is None:
            s_layer, s_batch, s_head, s_token, s_page = st[0], st[1], st[2], st[3], 0
        else:
            s_layer, s_batch, s_head, s_token, s_page = st[0], 0, st[3], st[2], st[1]
        kv = lyc_kv_batch(K.data_ptr(), V.data_ptr(), nn.ctypes.data, s_layer, s_batch, s_head,
                          s_token, s_page,
                          None if block_table is None else block_table.data_ptr(),
                          int(page_rows), 0 if block_table is None else int(block_table.shape[1]),
                          0 if block_table is None else int(K.shape[1]),
                          None if k_new is None else k_new.data_ptr(),
                          None if v_new is None else v_new.data_ptr())
        rc = lyc_decode_step_batch(self.ctx, q.data_ptr(), kv, role.ctypes.data, k,
                                   out.data_ptr(), S.data_ptr(), _stream_ptr(stream), flags)
        self._check(rc, "lyc_decode_step_batch")

    def decode_step_host(self, q_host, K, V, n, role_mask, k, out_host, S_host, stream=None,
                         s_in=False):
        role = np.ascontiguousarray(role_mask, dtype=np.uint8)
        self._role = role
        kv = self.kv_cache(K, V, n)
        flags = LYC_STEP_S_IN if s_in else 0
        rc = lyc_decode_step_host(self.ctx, q_host.data_ptr(), kv, role.ctypes.data, k,
                                  out_host.data_ptr(), S_host.data_ptr(), _stream_ptr(stream), flags)
        self._check(rc, "lyc_decode_step_host")

    def sync_status(self) -> int:
        return lyc_sync_status(self.ctx)

    def set_selection(self, rule=LYC_RULE_TOPK, block=64, ratio=(1, 2), p=0.9, tau=1e-3):
        """The selection rule of the steps that follow (lyc_set_selection)."""
        sel = lyc_selection(int(rule), int(block), int(ratio[0]), int(ratio[1]), float(p),
                            float(tau))
        self._check(lyc_set_selection(self.ctx, sel), "lyc_set_selection")

    def cache_correction(self, q, K, V, n, out, k_new=None, v_new=None, stream=None):
        """Cache Correction's dense causal attention: q [L][B][Hq][T][d] bf16,
        out [L][B][Hq][T][d] fp32, K/V as in decode_step (n counts the T
        positions); k_new/v_new [L][B][Hkv][T][d] written at rows n-T..n-1 first."""
        kv = self.kv_cache(K, V, n)
        rc = lyc_cache_correction(self.ctx, q.data_ptr(), kv, int(q.shape[3]),
                                  None if k_new is None else k_new.data_ptr(),
                                  None if v_new is None else v_new.data_ptr(), out.data_ptr(),
                                  _stream_ptr(stream))
        self._check(rc, "lyc_cache_correction")

    def set_trace(self, trace):
        self._trace = trace
        self._check(lyc_set_s_trace(self.ctx, None if trace is None else trace.data_ptr()),
                    "lyc_set_s_trace")

    def set_timing(self, on: bool):
        self._check(lyc_set_timing(self.ctx, LYC_TIMING_ON if on else LYC_TIMING_OFF),
                    "lyc_set_timing")

    def kernel_times(self):
        return lyc_kernel_times(self.ctx)

    def set_timeline(self, buf, cap: int):
        """buf: device int64 tensor of 1 + 3*cap words (word 0 zeroed), or None."""
        self._timeline = buf
        self._check(lyc_set_timeline(self.ctx, None if buf is None else buf.data_ptr(), cap),
                    "lyc_set_timeline")

    def topk_f32(self, keys, n, k, S, stream=None, cluster=None, variant=LYC_TOPK_FIXED):
        """The selection kernel alone; cluster (4, 8, 16) and variant choose its
        launch form (lyc_topk_f32_ex), None the context's default."""
        if cluster is None and variant == LYC_TOPK_FIXED:
            self._check(lyc_topk_f32(self.ctx, keys.data_ptr(), n, k, S.data_ptr(),
                                     _stream_ptr(stream)), "lyc_topk_f32")
        else:
            self._check(lyc_topk_f32_ex(self.ctx, keys.data_ptr(), n, k, S.data_ptr(),
                                        cluster or 0, variant, _stream_ptr(stream)),
                        "lyc_topk_f32_ex")

    def step_bytes(self, role_mask, n, k, s_in=False):
        return lyc_step_bytes(self.cfg, role_mask, n, k, s_in)

    def step_launches(self):
        """(attention, selection, other) kernel launches of the most recent step."""
        a, t, o = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        self._check(load().lyc_step_launches(self.ctx, ctypes.byref(a), ctypes.byref(t), ctypes.byref(o)),
                    "lyc_step_launches")
        return a.value, t.value, o.value


# ------------------------------------------------------------ serving operators
#
# Functions on one layer's torch tensors (include/lyc.h, "Serving operators").
# Tensors must lie on one device and stay valid until the stream has run the
# call; `stream` is a torch.cuda.Stream of that device (None: its current
# stream).  `status`: an int32 or uint32 tensor of one element that collects the
# LYC_OP_* bits of what only the device can see, or None.  Wrong arguments raise
# LycError (LYC_ERR_INVALID_ARG or LYC_ERR_UNSUPPORTED) and enqueue nothing.


def _refuse(where: str, what: str, code: int = LYC_ERR_INVALID_ARG):
    raise LycError(code, where, what)


def _operator_check(rc: int, where: str):
    if rc != LYC_OK:
        raise LycError(rc, where, lyc_operator_error())


# The argument structs are packed by `struct` in the C compiler's layout: a
# small call's host time is a good part of it, and filling a ctypes.Structure
# of some thirty fields takes about three times as long.
_ROPE_ARGS = struct.Struct("@4P8q4Pq5if2i")
_APPEND_ARGS = struct.Struct("@4P12q6P4ifP")
_READ_ARGS = struct.Struct("@2P3q2Pq3iP")
_TREE_ARGS = struct.Struct("@2P6q3P2ifPQP")
_NO_FIT = (struct.error, OverflowError)


def _operators():
    return _lib if _lib is not None else load()


def _rows_in(where, name, t, dtype, shape, index):
    """(address, strides) of a tensor whose rows (last dimension) are contiguous."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or st[-1] != 1:
        _refuse(where, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device} with strides {st}, where {dtype} "
                       f"{tuple(shape)} on cuda:{index} with contiguous rows is needed")
    return t.data_ptr(), st


def _packed(where, name, t, dtype, shape, index):
    """Address of a contiguous tensor, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(where, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, where a contiguous {dtype} "
                       f"{tuple(shape)} on cuda:{index} is needed")
    return t.data_ptr()


def _stream_on(index: int, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same pointer without a Stream object
    return raw(index) if raw else torch.cuda.current_stream(index).cuda_stream


def _status_ptr(where, status, index):
    import torch
    if status is None:
        return 0
    if status.dtype not in (torch.int32, torch.uint32) or status.numel() != 1 or status.get_device() != index:
        _refuse(where, f"status must be one int32 or uint32 on cuda:{index}")
    return status.data_ptr()


class KvCache:
    """One layer's cache, described once and handed to cache_append, cache_read
    and tree_attention (lyc_layer_cache).

      contiguous  k, v [B][Hkv][rows][d]
      paged       k, v [pages][page_rows][Hkv][d] and block_table int32 [B][max_blocks]

    k and v: bf16, or float8_e4m3fn with k_scale and v_scale of their shape
    without d (float8_e8m0fnu or uint8 bytes).  Any strides with the d elements
    of a row contiguous; K and V alike.  The object holds the tensors; it is
    valid while they are not moved."""

    def __init__(self, k, v, k_scale=None, v_scale=None, block_table=None):
        import torch
        where = "KvCache"
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            _refuse(where, "k must be a 4-D bf16 or float8_e4m3fn tensor")
        if not k.is_cuda:
            _refuse(where, f"k is on {k.device}: the cache lies on a GPU")
        index = self.device_index = k.get_device()
        kp, st = _rows_in(where, "k", k, k.dtype, k.shape, index)
        vp, sv = _rows_in(where, "v", v, k.dtype, k.shape, index)
        if st != sv:
            _refuse(where, "k and v must have the same strides")
        self.e4m3 = k.dtype == torch.float8_e4m3fn
        if (k_scale is None) == self.e4m3 or (v_scale is None) == self.e4m3:
            _refuse(where, "a float8_e4m3fn cache has scales, a bf16 cache has none")
        ss, ksp, vsp = (0, 0, 0), None, None
        if self.e4m3:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t.dtype not in (torch.uint8, torch.float8_e8m0fnu) or t.shape != k.shape[:3] or t.get_device() != index:
                    _refuse(where, f"{name} must be float8_e8m0fnu or uint8 of shape {tuple(k.shape[:3])} on cuda:{index}")
            if k_scale.stride() != v_scale.stride():
                _refuse(where, "k_scale and v_scale must have the same strides")
            ss, ksp, vsp = k_scale.stride(), k_scale.data_ptr(), v_scale.data_ptr()
        self.tensors = (k, v, k_scale, v_scale, block_table)
        kind = LYC_CACHE_E4M3 if self.e4m3 else LYC_CACHE_BF16
        if block_table is None:
            self.batch, self.heads, rows, self.d = k.shape
            self.desc = lyc_layer_cache(
                kp, vp, ksp, vsp, st[0], st[1], st[2], 0, ss[0], ss[1], ss[2], 0,
                None, rows, 0, 0, 0, kind, self.batch, self.heads, self.d, index)
        else:
            pages, page_rows, self.heads, self.d = k.shape
            if block_table.dim() != 2:
                _refuse(where, "block_table must be [B][max_blocks]")
            bt = _packed(where, "block_table", block_table, torch.int32, block_table.shape, index)
            self.batch = block_table.shape[0]
            self.desc = lyc_layer_cache(
                kp, vp, ksp, vsp, 0, st[2], st[1], st[0], 0, ss[2], ss[1], ss[0],
                bt, 0, pages, page_rows, block_table.shape[1], kind, self.batch, self.heads, self.d, index)
        self._desc_ref = ctypes.byref(self.desc)
        self._workspace = {}  # bytes by (T, query heads)

    @staticmethod
    def empty(batch, heads, d, rows=None, page_rows=None, num_pages=None, block_table=None, e4m3=True, device="cuda"):
        """A zeroed cache: contiguous of `rows` rows, or `num_pages` pages of
        page_rows rows named by block_table."""
        import torch
        shape = (batch, heads, rows, d) if block_table is None else (num_pages, page_rows, heads, d)
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        k, v = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else dtype, device=device).view(dtype) for _ in range(2))
        scales = (None, None)
        if e4m3:
            # a head's scales lie together: in a page, [Hkv][page_rows]
            inner = shape[:3] if block_table is None else (num_pages, heads, page_rows)
            scales = [torch.zeros(inner, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu) for _ in range(2)]
            if block_table is not None:
                scales = [t.transpose(1, 2) for t in scales]
        return KvCache(k, v, *scales, block_table=block_table)


def qk_norm_rope(q, k, pos, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 stream=None):
    """Per-head RMS norm (where weights are given) and rotation of q [rows][Hq][d]
    and k [rows][Hkv][d] by pos int32 [rows] and inv_freq fp32 [rot_dim/2] (None:
    no rotation), into q_out and k_out (lyc_qk_norm_rope).  bf16 or fp32; q and
    q_out, or k and k_out, may be None; an output may be its input."""
    import torch
    where = "qk_norm_rope"
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        _refuse(where, "q or k must be a [rows][heads][d] tensor")
    rows, _, d = x.shape
    dtype, index = x.dtype, x.get_device()
    if index < 0 or (dtype is not torch.bfloat16 and dtype is not torch.float32):
        _refuse(where, f"{dtype} on {x.device}: bfloat16 or float32 on a GPU is needed")
    weight = (d,)
    qp = qo = kp = ko = qw = kw = hq = hk = 0
    sq = sqo = sk = sko = (0, 0, 0)
    if q is not None:
        if q_out is None:
            _refuse(where, "q without q_out")
        hq = q.shape[1]
        shape = (rows, hq, d)
        qp, sq = _rows_in(where, "q", q, dtype, shape, index)
        qo, sqo = _rows_in(where, "q_out", q_out, dtype, shape, index)
        qw = _packed(where, "q_weight", q_weight, dtype, weight, index)
    elif q_out is not None or q_weight is not None:
        _refuse(where, "q_out or q_weight without q")
    if k is not None:
        if k_out is None or k.dim() != 3:
            _refuse(where, "k must be a [rows][heads][d] tensor and have a k_out")
        hk = k.shape[1]
        shape = (rows, hk, d)
        kp, sk = _rows_in(where, "k", k, dtype, shape, index)
        ko, sko = _rows_in(where, "k_out", k_out, dtype, shape, index)
        kw = _packed(where, "k_weight", k_weight, dtype, weight, index)
    elif k_out is not None or k_weight is not None:
        _refuse(where, "k_out or k_weight without k")
    rot = fp = pp = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        rot = 2 * half
        if pos is None:
            _refuse(where, "a rotation needs pos")
        fp = _packed(where, "inv_freq", inv_freq, torch.float32, (half,), index)
        pp = _packed(where, "pos", pos, torch.int32, (rows,), index)
    try:
        args = _ROPE_ARGS.pack(qp, kp, qo, ko, sq[0], sq[1], sk[0], sk[1], sqo[0], sqo[1], sko[0], sko[1], pp, fp, qw, kw,
                               rows, hq, hk, d, rot, 1 if interleaved else 0, eps,
                               LYC_BF16 if dtype is torch.bfloat16 else LYC_FP32, index)
    except _NO_FIT as e:
        _refuse(where, f"a number does not fit its argument: {e}")
    rc = _operators().lyc_qk_norm_rope(args, _stream_on(index, stream))
    if rc:
        _operator_check(rc, "lyc_qk_norm_rope")


def cache_append(cache, n, k, v, t_len=None, q=None, q_out=None, pos=None, inv_freq=None, q_weight=None,
                 k_weight=None, eps=1e-6, interleaved=False, status=None, stream=None):
    """The last t_len[b] (default T) tokens' k, v [B][T][Hkv][d] bf16 written at
    rows n[b] - t_len[b] + t of `cache`, quantised where it is e4m3, the keys
    normed and rotated on the way where k_weight and inv_freq are given, and the
    same tokens' queries q [B][T][Hq][d] with them into q_out (lyc_cache_append).
    n, t_len: int32 [B] on the device; pos: int32 [B][T], default the row."""
    import torch
    where = "cache_append"
    index, bf16, i32, B, d = cache.device_index, torch.bfloat16, torch.int32, cache.batch, cache.d
    if k.dim() != 4:
        _refuse(where, "k must be [B][T][Hkv][d]")
    T = k.shape[1]
    shape = (B, T, cache.heads, d)
    kp, sk = _rows_in(where, "k", k, bf16, shape, index)
    vp, sv = _rows_in(where, "v", v, bf16, shape, index)
    hq = qp = qo = qw = 0
    sq = sqo = (0, 0, 0)
    if q is not None:
        if q_out is None or q.dim() != 4:
            _refuse(where, "q must be [B][T][Hq][d] and have a q_out")
        hq = q.shape[2]
        shape = (B, T, hq, d)
        qp, sq = _rows_in(where, "q", q, bf16, shape, index)
        qo, sqo = _rows_in(where, "q_out", q_out, bf16, shape, index)
        qw = _packed(where, "q_weight", q_weight, bf16, (d,), index)
    elif q_out is not None or q_weight is not None:
        _refuse(where, "q_out or q_weight without q")
    rot = fp = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        rot = 2 * half
        fp = _packed(where, "inv_freq", inv_freq, torch.float32, (half,), index)
    try:
        args = _APPEND_ARGS.pack(
            kp, vp, qp, qo, sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], sq[0], sq[1], sq[2], sqo[0], sqo[1], sqo[2],
            _packed(where, "n", n, i32, (B,), index), _packed(where, "t_len", t_len, i32, (B,), index),
            _packed(where, "pos", pos, i32, (B, T), index), fp, qw, _packed(where, "k_weight", k_weight, bf16, (d,), index),
            T, hq, rot, 1 if interleaved else 0, eps, _status_ptr(where, status, index))
    except _NO_FIT as e:
        _refuse(where, f"a number does not fit its argument: {e}")
    rc = _operators().lyc_cache_append(cache._desc_ref, args, _stream_on(index, stream))
    if rc:
        _operator_check(rc, "lyc_cache_append")


def cache_read(cache, n, k_out, v_out, sets=None, first=0, status=None, stream=None):
    """Rows of `cache` read back, dequantised, into k_out and v_out [B][H][m][d]
    (bf16 or fp32): rows first .. first+m-1 below n[b] (H = Hkv), or the rows of
    sets int32 [B][H][m] (H a multiple of Hkv: the step's S) (lyc_cache_read)."""
    import torch
    where = "cache_read"
    index, B, dtype = cache.device_index, cache.batch, k_out.dtype
    if k_out.dim() != 4 or (dtype is not torch.bfloat16 and dtype is not torch.float32):
        _refuse(where, "k_out must be a [B][H][m][d] bf16 or fp32 tensor")
    _, H, m, _ = k_out.shape
    shape = (B, H, m, cache.d)
    kp, so = _rows_in(where, "k_out", k_out, dtype, shape, index)
    vp, sv = _rows_in(where, "v_out", v_out, dtype, shape, index)
    if so != sv:
        _refuse(where, "k_out and v_out must have the same strides")
    try:
        args = _READ_ARGS.pack(kp, vp, so[0], so[1], so[2], _packed(where, "n", n, torch.int32, (B,), index),
                               _packed(where, "sets", sets, torch.int32, (B, H, m), index), first, m, H,
                               LYC_BF16 if dtype is torch.bfloat16 else LYC_FP32, _status_ptr(where, status, index))
    except _NO_FIT as e:
        _refuse(where, f"a number does not fit its argument: {e}")
    rc = _operators().lyc_cache_read(cache._desc_ref, args, _stream_on(index, stream))
    if rc:
        _operator_check(rc, "lyc_cache_read")


def tree_attention(q, cache, n, out, mask=None, t_len=None, scale=None, workspace=None, status=None, stream=None):
    """Attention of the last t_len[b] (default T) of n[b] rows' queries q
    [B][T][Hq][d] over `cache` into out (lyc_tree_attention): every row before
    the drafted ones, and the drafted nodes of mask int64 [B][T][ceil(T/64)]
    (None: a chain; T = 1: one token's dense attention).  scale: default
    d ** -0.5.  workspace: a device tensor of tree_workspace_bytes(...) bytes
    that no other call uses meanwhile; by default one is taken from torch's
    allocator for this call."""
    import torch
    where = "tree_attention"
    index, bf16, i32, B = cache.device_index, torch.bfloat16, torch.int32, cache.batch
    if q.dim() != 4:
        _refuse(where, "q must be [B][T][Hq][d]")
    _, T, hq, _ = q.shape
    shape = (B, T, hq, cache.d)
    qp, sq = _rows_in(where, "q", q, bf16, shape, index)
    op, so = _rows_in(where, "out", out, bf16, shape, index)
    mp = 0
    if mask is not None:
        mp = _packed(where, "mask", mask, torch.uint64 if mask.dtype is torch.uint64 else torch.int64,
                     (B, T, (T + 63) // 64), index)
    if workspace is None:
        need = tree_workspace_bytes(cache, T, hq)
        if stream is None:
            workspace = q.new_empty((need + 1) // 2)
        else:
            with torch.cuda.stream(stream):  # the allocator orders its reuse on the call's stream
                workspace = q.new_empty((need + 1) // 2)
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        _refuse(where, f"workspace must be contiguous, on cuda:{index}")
    try:
        args = _TREE_ARGS.pack(qp, op, sq[0], sq[1], sq[2], so[0], so[1], so[2], _packed(where, "n", n, i32, (B,), index),
                               _packed(where, "t_len", t_len, i32, (B,), index), mp, T, hq,
                               cache.d**-0.5 if scale is None else scale, workspace.data_ptr(), workspace.nbytes,
                               _status_ptr(where, status, index))
    except _NO_FIT as e:
        _refuse(where, f"a number does not fit its argument: {e}")
    rc = _operators().lyc_tree_attention(cache._desc_ref, args, _stream_on(index, stream))
    if rc:
        _operator_check(rc, "lyc_tree_attention")


def tree_workspace_bytes(cache, T: int, num_q_heads: int) -> int:
    """Bytes of tree_attention's workspace for q [B][T][num_q_heads][d] over `cache`."""
    need = cache._workspace.get((T, num_q_heads))
    if need is None:
        need = lyc_tree_workspace_bytes(cache.desc, T, num_q_heads)
        if need == 0:
            raise LycError(lyc_operator_status(), "lyc_tree_workspace_bytes", lyc_operator_error())
        cache._workspace[(T, num_q_heads)] = need
    return need
