"""ctypes binding of the attention C ABI (``include/attn.h``).

Argument marshalling only: every step of the computation runs in the CUDA
library ``libattn_sm103.so``.  PyTorch supplies device memory and the stream.
Loading fails loudly (RuntimeError) when the library is missing; there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libattn_sm103.so")

ATTN_PARAMS_VERSION = 6

LAYOUTS = {"3HD": 0, "HD_2HD": 1, "HD_HD_HD": 2}
FORMATS = {"BSHD": 0, "THD_SEGMENTS": 1, "THD_CU_SEQLENS": 2}
MASKS = {"NONE": 0, "CAUSAL": 1, "PADDING": 2, "PADDING_CAUSAL": 3}
DQ_MODES = {"atomic": 0, "deterministic": 1}
DTYPES = {"bf16": 0, "fp16": 1, "fp8_e4m3": 2}
STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
          3: "ATTN_ERR_SHAPE_MISMATCH", 4: "ATTN_ERR_WORKSPACE_TOO_SMALL", 5: "ATTN_ERR_CUDA",
          6: "ATTN_ERR_DEVICE_TIMEOUT", 7: "ATTN_ERR_DEVICE_BOUNDS"}
BUILD_DEVICE_CHECKS = 1
EXPORTED = ("attn_abi_version", "attn_status_string", "attn_fwd_workspace_size",
            "attn_bwd_workspace_size", "attn_resolve_layout", "attn_fwd", "attn_bwd",
            "attn_read_status", "attn_set_trace_events", "attn_event_create",
            "attn_event_destroy", "attn_event_elapsed_ms", "attn_fwd_noalloc",
            "attn_build_flags", "attn_paged_workspace_size", "attn_paged_append",
            "attn_paged_fwd", "attn_rope_table", "attn_rope", "attn_latent_expand",
            "attn_latent_expand_bwd", "attn_latent_workspace_size", "attn_latent_append",
            "attn_latent_fwd")
ATTN_PAGED_PARAMS_VERSION = 1
ATTN_ROPE_TABLE_PARAMS_VERSION = 1
ATTN_ROPE_PARAMS_VERSION = 1
ATTN_LATENT_EXPAND_PARAMS_VERSION = 1
ATTN_LATENT_PARAMS_VERSION = 1
ROPE_SCALINGS = {"NONE": 0, "LINEAR": 1, "BASE": 2, "TURNS": 3}
FWD_NOALLOC_SCRATCH_BYTES = 4 << 20
TRACE_SLOTS = ("meta", "fwd", "bwd_pre", "dkdv", "dq", "dbias")

c_i32, c_i64, c_f32, c_f64, c_vp, c_sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                          ctypes.c_double, ctypes.c_void_p, ctypes.c_size_t)


class attn_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("fmt", c_i32), ("layout", c_i32), ("mask", c_i32),
        ("dq_mode", c_i32),
        ("B", c_i32), ("Sq", c_i32), ("Skv", c_i32), ("Hq", c_i32), ("Hkv", c_i32),
        ("d_qk", c_i32), ("d_v", c_i32),
        ("scale", c_f32),
        ("q", c_vp), ("k", c_vp), ("v", c_vp),
        ("q_seg_ids", c_vp), ("q_seg_pos", c_vp), ("kv_seg_ids", c_vp), ("kv_seg_pos", c_vp),
        ("q_ids_dims", c_i64 * 2), ("q_pos_dims", c_i64 * 2), ("kv_ids_dims", c_i64 * 2),
        ("kv_pos_dims", c_i64 * 2),
        ("cu_seqlens_q", c_vp), ("cu_seqlens_kv", c_vp), ("num_segments", c_i32),
        ("bias", c_vp), ("bias_b", c_i32), ("bias_h", c_i32),
        ("force_general_path", c_i32),
        ("metadata_from_forward", c_i32),
        ("max_logit", c_vp),
        ("sink", c_vp), ("dsink", c_vp),
        ("band", c_i32), ("window_left", c_i32), ("window_right", c_i32),
        ("bottom_right", c_i32),
        ("dtype", c_i32),
        ("test_wait_timeout", c_i32),
        ("descale_q", c_f32), ("descale_k", c_f32), ("descale_v", c_f32),
    ]


class attn_stats_t(ctypes.Structure):
    _fields_ = [("status", c_i32), ("path", c_i32), ("reason", c_i32), ("dq_mode", c_i32),
                ("tile_pairs", c_i64), ("wait_site", c_i32), ("reserved", c_i32)]


class attn_resolved_t(ctypes.Structure):
    _fields_ = [("q", c_vp), ("k", c_vp), ("v", c_vp), ("q_token_stride", c_i64),
                ("k_token_stride", c_i64), ("v_token_stride", c_i64), ("dq", c_vp), ("dk", c_vp),
                ("dv", c_vp)]


class attn_paged_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("dtype", c_i32), ("cache_dtype", c_i32), ("mask", c_i32),
        ("num_seqs", c_i32), ("num_tokens", c_i32), ("max_q_len", c_i32),
        ("Hq", c_i32), ("Hkv", c_i32), ("d_qk", c_i32), ("d_v", c_i32),
        ("page_size", c_i32), ("num_pages", c_i32), ("max_pages", c_i32),
        ("page_table", c_vp), ("table_stride", c_i64), ("seq_lens", c_vp),
        ("cu_seqlens_q", c_vp),
        ("k_cache", c_vp), ("v_cache", c_vp), ("k_cache_stride", c_i64 * 3),
        ("v_cache_stride", c_i64 * 3),
        ("k_scale", c_vp), ("v_scale", c_vp), ("status", c_vp),
        ("q", c_vp), ("k_new", c_vp), ("v_new", c_vp), ("q_rot", c_vp),
        ("q_stride", c_i64), ("k_new_stride", c_i64), ("v_new_stride", c_i64),
        ("q_rot_stride", c_i64),
        ("rot_dim", c_i32), ("rot_interleaved", c_i32), ("rope_len", c_i32),
        ("rope_cos", c_vp), ("rope_sin", c_vp), ("rope_pos", c_vp),
        ("scale", c_f32), ("window_left", c_i32), ("sink", c_vp),
    ]


class attn_rope_table_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("scaling", c_i32), ("rope_len", c_i32), ("rot_dim", c_i32),
        ("base", c_f64), ("factor", c_f64), ("turns_low", c_f64), ("turns_high", c_f64),
        ("trained_len", c_i32), ("magnitude", c_f32), ("rope_cos", c_vp), ("rope_sin", c_vp),
    ]


class attn_rope_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("dtype", c_i32), ("num_tokens", c_i32), ("Hq", c_i32),
        ("Hkv", c_i32), ("d", c_i32), ("rot_start", c_i32), ("rot_dim", c_i32),
        ("rot_interleaved", c_i32), ("inverse", c_i32), ("rope_len", c_i32), ("seq_len", c_i32),
        ("num_segments", c_i32), ("positions", c_vp), ("cu_seqlens", c_vp), ("rope_cos", c_vp),
        ("rope_sin", c_vp), ("q", c_vp), ("k", c_vp), ("q_out", c_vp), ("k_out", c_vp),
        ("q_stride", c_i64), ("k_stride", c_i64), ("q_out_stride", c_i64), ("k_out_stride", c_i64),
        ("status", c_vp),
    ]


class attn_latent_expand_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("dtype", c_i32), ("num_tokens", c_i32), ("H", c_i32),
        ("d_n", c_i32), ("d_v", c_i32), ("d_r", c_i32), ("rot_interleaved", c_i32),
        ("rope_len", c_i32), ("seq_len", c_i32), ("num_segments", c_i32), ("positions", c_vp),
        ("cu_seqlens", c_vp), ("rope_cos", c_vp), ("rope_sin", c_vp), ("kv", c_vp),
        ("k_rope", c_vp), ("k", c_vp), ("v", c_vp), ("kv_stride", c_i64), ("k_rope_stride", c_i64),
        ("k_stride", c_i64), ("v_stride", c_i64), ("status", c_vp),
    ]


class attn_latent_params_t(ctypes.Structure):
    _fields_ = [
        ("struct_version", c_i32), ("dtype", c_i32), ("mask", c_i32), ("num_seqs", c_i32),
        ("num_tokens", c_i32), ("max_q_len", c_i32), ("H", c_i32), ("d_c", c_i32), ("d_r", c_i32),
        ("page_size", c_i32), ("num_pages", c_i32), ("max_pages", c_i32), ("page_table", c_vp),
        ("table_stride", c_i64), ("seq_lens", c_vp), ("cu_seqlens_q", c_vp), ("cache", c_vp),
        ("cache_stride", c_i64 * 2), ("status", c_vp), ("c_new", c_vp), ("k_rope", c_vp),
        ("q_rope", c_vp), ("q_lat", c_vp), ("q_rot", c_vp), ("c_new_stride", c_i64),
        ("k_rope_stride", c_i64), ("q_rope_stride", c_i64 * 2), ("q_lat_stride", c_i64 * 2),
        ("q_rot_stride", c_i64 * 2), ("rot_interleaved", c_i32), ("rope_len", c_i32),
        ("rope_cos", c_vp), ("rope_sin", c_vp), ("rope_pos", c_vp), ("scale", c_f32),
        ("window_left", c_i32), ("sink", c_vp),
    ]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (built by ``bwd_tcgen05_tma_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA attention library not built: {path} is missing "
                           "(run bwd_tcgen05_tma_gb300.build.build())")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(attn_params_t)
    lib.attn_abi_version.restype = c_i32
    lib.attn_build_flags.restype = c_i32
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_status_string.argtypes = [c_i32]
    lib.attn_fwd_workspace_size.restype = c_sz
    lib.attn_fwd_workspace_size.argtypes = [P]
    lib.attn_bwd_workspace_size.restype = c_sz
    lib.attn_bwd_workspace_size.argtypes = [P]
    lib.attn_resolve_layout.restype = c_i32
    lib.attn_resolve_layout.argtypes = [P, c_vp, c_vp, c_vp, ctypes.POINTER(attn_resolved_t)]
    lib.attn_fwd.restype = c_i32
    lib.attn_fwd.argtypes = [P, c_vp, c_vp, c_vp, c_sz, c_vp]
    lib.attn_bwd.restype = c_i32
    lib.attn_bwd.argtypes = [P, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    lib.attn_read_status.restype = c_i32
    lib.attn_read_status.argtypes = [c_vp, c_vp, ctypes.POINTER(attn_stats_t)]
    lib.attn_set_trace_events.restype = c_i32
    lib.attn_set_trace_events.argtypes = [ctypes.POINTER(c_vp)]
    lib.attn_fwd_noalloc.restype = c_i32
    lib.attn_fwd_noalloc.argtypes = [P, c_vp, c_vp, c_vp]
    lib.attn_event_create.restype = c_i32
    lib.attn_event_create.argtypes = [ctypes.POINTER(c_vp)]
    lib.attn_event_destroy.restype = c_i32
    lib.attn_event_destroy.argtypes = [c_vp]
    lib.attn_event_elapsed_ms.restype = c_i32
    lib.attn_event_elapsed_ms.argtypes = [c_vp, c_vp, ctypes.POINTER(ctypes.c_float)]
    PP = ctypes.POINTER(attn_paged_params_t)
    lib.attn_paged_workspace_size.restype = c_sz
    lib.attn_paged_workspace_size.argtypes = [PP]
    lib.attn_paged_append.restype = c_i32
    lib.attn_paged_append.argtypes = [PP, c_vp]
    lib.attn_paged_fwd.restype = c_i32
    lib.attn_paged_fwd.argtypes = [PP, c_vp, c_vp, c_vp, c_sz, c_vp]
    for name, block in (("attn_rope_table", attn_rope_table_params_t),
                        ("attn_rope", attn_rope_params_t),
                        ("attn_latent_expand", attn_latent_expand_params_t),
                        ("attn_latent_expand_bwd", attn_latent_expand_params_t),
                        ("attn_latent_append", attn_latent_params_t)):
        getattr(lib, name).restype = c_i32
        getattr(lib, name).argtypes = [ctypes.POINTER(block), c_vp]
    PL = ctypes.POINTER(attn_latent_params_t)
    lib.attn_latent_workspace_size.restype = c_sz
    lib.attn_latent_workspace_size.argtypes = [PL]
    lib.attn_latent_fwd.restype = c_i32
    lib.attn_latent_fwd.argtypes = [PL, c_vp, c_vp, c_vp, c_sz, c_vp]
    if lib.attn_abi_version() != ATTN_PARAMS_VERSION:
        raise RuntimeError("attention library ABI version mismatch")
    _lib = lib
    return lib


@contextlib.contextmanager
def library_scope(path: str):
    """Route every call made inside the block to the library at ``path`` (for
    example the checking build, ``build.build(debug=True)``); the library
    loaded before is restored afterwards."""
    global _lib
    prev = _lib
    _lib = None
    try:
        yield load_library(path)
    finally:
        _lib = prev


class AttnError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        name = STATUS.get(code, str(code))
        msg = load_library().attn_status_string(code).decode()
        super().__init__(f"{what}: {name} ({msg})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    """The handle of `stream`, or of torch's current one on `device` (default: the
    current device, which takes 0.25 us to ask for)."""
    if stream is None:
        import torch

        # the raw handle: a Stream object costs 3 us, as much as a small kernel
        if device is None:
            device = torch.cuda.current_device()
        return c_vp(torch._C._cuda_getCurrentRawStream(device))
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def make_params(*, layout, fmt, mask, B, Sq, Skv, Hq, Hkv, d_qk, d_v, scale, q, k=None, v=None,
                q_seg_ids=None, q_seg_pos=None, kv_seg_ids=None, kv_seg_pos=None,
                cu_seqlens_q=None, cu_seqlens_kv=None, bias=None, dq_mode="deterministic",
                force_general_path=False, metadata_from_forward=False, max_logit=None,
                sink=None, dsink=None, window=None, bottom_right=False, dtype="bf16",
                descale=(1.0, 1.0, 1.0)):
    """Fill an ``attn_params_t`` from tensors (any object with data_ptr/shape).
    max_logit: optional fp32 [B, Hq] tensor the forward fills; sink: optional
    fp32 [Hq] sink logits; dsink: optional fp32 [Hq] tensor the backward fills
    with their gradient; window: optional (left, right) band, None for an
    unbounded side; bottom_right: align positions by Skv - Sq; dtype: "bf16",
    "fp16" or "fp8_e4m3" (forward only: Q / K / V as E4M3 codes, O in bf16);
    descale: the (q, k, v) factors the E4M3 codes stand scaled by (see attn.h)."""
    p = attn_params_t()
    p.struct_version = ATTN_PARAMS_VERSION
    p.fmt = FORMATS[fmt]
    p.layout = LAYOUTS[layout]
    p.mask = MASKS[mask]
    p.dq_mode = DQ_MODES[dq_mode]
    p.B, p.Sq, p.Skv, p.Hq, p.Hkv, p.d_qk, p.d_v = B, Sq, Skv, Hq, Hkv, d_qk, d_v
    p.scale = float(scale)
    p.q, p.k, p.v = _ptr(q), _ptr(k), _ptr(v)
    for name, t in (("q_seg_ids", q_seg_ids), ("q_seg_pos", q_seg_pos), ("kv_seg_ids", kv_seg_ids),
                    ("kv_seg_pos", kv_seg_pos)):
        setattr(p, name, _ptr(t))
        if t is not None:
            dims = tuple(t.shape)
            if len(dims) == 1:
                dims = (1,) + dims
            key = {"q_seg_ids": "q_ids_dims", "q_seg_pos": "q_pos_dims",
                   "kv_seg_ids": "kv_ids_dims", "kv_seg_pos": "kv_pos_dims"}[name]
            arr = getattr(p, key)
            arr[0] = int(dims[-2]) if len(dims) >= 2 else 1
            arr[1] = int(dims[-1])
            if len(dims) > 2:  # extra leading dims: a mismatch the library reports
                arr[0] = -1
    p.cu_seqlens_q, p.cu_seqlens_kv = _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv)
    p.num_segments = 0 if cu_seqlens_q is None else int(cu_seqlens_q.shape[0]) - 1
    p.bias = _ptr(bias)
    if bias is not None:
        p.bias_b, p.bias_h = int(bias.shape[0]), int(bias.shape[1])
    p.force_general_path = 1 if force_general_path else 0
    p.metadata_from_forward = 1 if metadata_from_forward else 0
    p.max_logit = _ptr(max_logit)
    p.sink = _ptr(sink)
    p.dsink = _ptr(dsink)
    if window is not None:
        left, right = window
        p.band = 1
        p.window_left = -1 if left is None else int(left)
        p.window_right = -1 if right is None else int(right)
    p.bottom_right = 1 if bottom_right else 0
    p.dtype = DTYPES[dtype]
    p.descale_q, p.descale_k, p.descale_v = (float(x) for x in descale)
    return p


def attn_fwd_workspace_size(p):
    return int(load_library().attn_fwd_workspace_size(ctypes.byref(p)))


def attn_bwd_workspace_size(p):
    return int(load_library().attn_bwd_workspace_size(ctypes.byref(p)))


def attn_resolve_layout(p, dq=None, dk=None, dv=None):
    r = attn_resolved_t()
    s = load_library().attn_resolve_layout(ctypes.byref(p), dq, dk, dv, ctypes.byref(r))
    if s != 0:
        raise AttnError(s, "attn_resolve_layout")
    return r


def attn_fwd(p, o, lse, ws, stream=None):
    """Enqueue the forward on `stream` (default: torch's current stream)."""
    s = load_library().attn_fwd(ctypes.byref(p), _ptr(o), _ptr(lse), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream))
    if s != 0:
        raise AttnError(s, "attn_fwd")


def attn_fwd_noalloc(p, o, lse, stream=None):
    """Forward without a workspace: the library's fixed device scratch array is
    used instead (no allocation).  For callers that cannot allocate device
    memory at run time.  Overlapping calls on the GPU race on that array."""
    s = load_library().attn_fwd_noalloc(ctypes.byref(p), _ptr(o), _ptr(lse), _stream(stream))
    if s != 0:
        raise AttnError(s, "attn_fwd_noalloc")


def attn_bwd(p, o, d_o, lse, dq, dk, dv, dbias, ws, stream=None):
    """Enqueue the backward on `stream` (default: torch's current stream)."""
    s = load_library().attn_bwd(ctypes.byref(p), _ptr(o), _ptr(d_o), _ptr(lse), _ptr(dq), _ptr(dk),
                                _ptr(dv), _ptr(dbias), _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(stream))
    if s != 0:
        raise AttnError(s, "attn_bwd")


def _rows(name, t, heads, dim):
    """Token stride in elements of a [tokens, heads, dim] tensor whose rows may
    lie apart (a slice of a fused projection) but are whole inside."""
    if t.dim() != 3 or tuple(t.shape[1:]) != (heads, dim):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [tokens, {heads}, {dim}]")
    if t.shape[0] and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name}: heads and dims must be contiguous inside a token's row")
    return t.stride(0) if t.shape[0] > 1 else heads * dim


def _one_device(tensors):
    """The device all of a block's tensors are on, which has to be current."""
    import torch

    devices = {t.device for t in tensors.values() if t is not None}
    if len(devices) != 1:
        raise ValueError(f"tensors on several devices: {sorted(map(str, devices))}")
    device = devices.pop()
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return device


def _check_types(tensors, dtypes):
    for name, t in tensors.items():
        if t is not None and t.dtype != dtypes[name]:
            raise ValueError(f"{name}: {t.dtype}, expected {dtypes[name]}")


def _check_contiguous(tensors, names):
    for name in names:
        if tensors[name] is not None and not tensors[name].is_contiguous():
            raise ValueError(f"{name}: must be contiguous")


def _elem16(dtype):
    import torch

    if dtype not in ("bf16", "fp16"):
        raise ValueError(f"dtype: {dtype}, expected bf16 or fp16")
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def make_paged_params(*, dtype, cache_dtype, k_cache, v_cache, page_table, seq_lens, q=None,
                      k_new=None, v_new=None, q_rot=None, k_scale=None, v_scale=None,
                      cu_seqlens_q=None, max_q_len=1, rope_cos=None, rope_sin=None,
                      rope_pos=None, rope_interleaved=False, scale=None, mask="CAUSAL",
                      window_left=None, sink=None, status=None):
    """Fill an ``attn_paged_params_t`` from tensors (see attn.h).

    k_cache / v_cache: [num_pages, Hkv, page_size, dim] views in any order of
    memory with contiguous dims (a cache kept as [num_pages, page_size, Hkv,
    dim] is passed as ``cache.transpose(1, 2)``); page_table: int32 [num_seqs,
    max_pages]; seq_lens: int32 [num_seqs], new tokens included; q, q_rot
    [tokens, Hq, d_qk], k_new, v_new [tokens, Hkv, dim]; rope_cos, rope_sin:
    fp32 [rope_len, rot_dim / 2] (None: no rotation); scale: softmax scale
    (None: d_qk ** -0.5).  The block holds the tensors' addresses and keeps them
    alive; their contents may change between calls.  All tensors are on the
    device that is current when the block is made and when it is used."""
    import torch

    if q is None and q_rot is None and k_new is None:
        raise ValueError("neither queries nor new keys are given")
    Hkv, page, d_qk = (int(x) for x in k_cache.shape[1:])
    d_v = int(v_cache.shape[3])
    if k_cache.dim() != 4 or v_cache.dim() != 4 or v_cache.shape[:3] != k_cache.shape[:3]:
        raise ValueError("k_cache and v_cache: [num_pages, Hkv, page_size, dim] with the same "
                         "pages, heads and page size")
    elem = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8_e4m3": torch.float8_e4m3fn}
    want = {}
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        ok = (elem[cache_dtype], torch.uint8) if cache_dtype == "fp8_e4m3" else (elem[cache_dtype],)
        if t.dtype not in ok:
            raise ValueError(f"{name}: {t.dtype}, expected {cache_dtype}")
        if t.stride(3) != 1:
            raise ValueError(f"{name}: dims must be contiguous")
    for name, t, dt in (("q", q, elem[dtype]), ("k_new", k_new, elem[dtype]),
                        ("v_new", v_new, elem[dtype]), ("q_rot", q_rot, elem[dtype]),
                        ("k_scale", k_scale, torch.float32), ("v_scale", v_scale, torch.float32),
                        ("rope_cos", rope_cos, torch.float32),
                        ("rope_sin", rope_sin, torch.float32), ("sink", sink, torch.float32),
                        ("rope_pos", rope_pos, torch.int32), ("status", status, torch.int32),
                        ("page_table", page_table, torch.int32),
                        ("seq_lens", seq_lens, torch.int32),
                        ("cu_seqlens_q", cu_seqlens_q, torch.int32)):
        if t is not None and t.dtype != dt:
            raise ValueError(f"{name}: {t.dtype}, expected {dt}")
        want[name] = t
    given = dict(want, k_cache=k_cache, v_cache=v_cache)
    device = _one_device(given)
    for name in ("k_scale", "v_scale", "rope_cos", "rope_sin", "rope_pos", "sink", "seq_lens",
                 "cu_seqlens_q"):
        if given[name] is not None and not given[name].is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    num_seqs = int(seq_lens.shape[0])
    if page_table.dim() != 2 or page_table.shape[0] != num_seqs or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table: [num_seqs, max_pages] with contiguous rows")
    if cu_seqlens_q is not None and tuple(cu_seqlens_q.shape) != (num_seqs + 1,):
        raise ValueError("cu_seqlens_q: [num_seqs + 1]")
    for name in ("k_scale", "v_scale"):
        if given[name] is not None and tuple(given[name].shape) != (k_cache.shape[0], Hkv):
            raise ValueError(f"{name}: [num_pages, Hkv]")

    p = attn_paged_params_t()
    p.tensors, p.device = given, device.index
    p.struct_version = ATTN_PAGED_PARAMS_VERSION
    p.dtype, p.cache_dtype, p.mask = DTYPES[dtype], DTYPES[cache_dtype], MASKS[mask]
    rows = next(t for t in (q, q_rot, k_new) if t is not None)
    heads = next((t for t in (q, q_rot) if t is not None), None)
    p.num_seqs, p.num_tokens, p.max_q_len = num_seqs, int(rows.shape[0]), int(max_q_len)
    p.Hq, p.Hkv = (Hkv if heads is None else int(heads.shape[1])), Hkv
    p.d_qk, p.d_v = d_qk, d_v
    p.page_size, p.num_pages = page, int(k_cache.shape[0])
    p.max_pages = int(page_table.shape[1])
    p.page_table, p.seq_lens, p.cu_seqlens_q = (_ptr(page_table), _ptr(seq_lens),
                                                _ptr(cu_seqlens_q))
    p.table_stride = page_table.stride(0) if num_seqs > 1 else p.max_pages
    p.k_cache, p.v_cache = _ptr(k_cache), _ptr(v_cache)
    for field, t in ((p.k_cache_stride, k_cache), (p.v_cache_stride, v_cache)):
        for i in range(3):  # the stride of an axis of one is never used
            field[i] = t.stride(i) if t.shape[i] > 1 else 16
    p.k_scale, p.v_scale, p.status = _ptr(k_scale), _ptr(v_scale), _ptr(status)
    for name, t, h, d in (("q", q, p.Hq, d_qk), ("q_rot", q_rot, p.Hq, d_qk),
                          ("k_new", k_new, Hkv, d_qk), ("v_new", v_new, Hkv, d_v)):
        if t is not None:
            if t.shape[0] != p.num_tokens:
                raise ValueError(f"{name}: {t.shape[0]} rows, expected {p.num_tokens}")
            setattr(p, name + "_stride", _rows(name, t, h, d))
            setattr(p, name, _ptr(t))
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin go together")
    if rope_cos is not None:
        if rope_cos.dim() != 2 or rope_cos.shape != rope_sin.shape:
            raise ValueError("rope_cos, rope_sin: [rope_len, rot_dim / 2]")
        p.rot_dim, p.rope_len = 2 * int(rope_cos.shape[1]), int(rope_cos.shape[0])
        p.rope_cos, p.rope_sin = _ptr(rope_cos), _ptr(rope_sin)
    if rope_pos is not None and tuple(rope_pos.shape) != (p.num_tokens,):
        raise ValueError("rope_pos: [tokens]")
    p.rope_pos = _ptr(rope_pos)
    p.rot_interleaved = 1 if rope_interleaved else 0
    p.scale = float(d_qk ** -0.5 if scale is None else scale)
    p.window_left = -1 if window_left is None else int(window_left)
    if sink is not None and tuple(sink.shape) != (p.Hq,):
        raise ValueError("sink: [Hq]")
    p.sink = _ptr(sink)
    return p


def attn_paged_workspace_size(p):
    return int(load_library().attn_paged_workspace_size(ctypes.byref(p)))


def _on_device(p):
    import torch

    current = torch.cuda.current_device()
    if current != p.device:
        raise ValueError(f"tensors on cuda:{p.device}, the current device is cuda:{current}")


def attn_paged_append(p, stream=None):
    """Enqueue the append on `stream` (default: torch's current stream)."""
    _on_device(p)
    s = load_library().attn_paged_append(ctypes.byref(p), _stream(stream))
    if s != 0:
        raise AttnError(s, "attn_paged_append")


def _check_outputs(p, o, lse, ws, want, n_o, n_lse):
    import torch

    for name, t, n, dt in (("o", o, n_o, want), ("lse", lse, n_lse, torch.float32)):
        if t is not None and (t.numel() != n or not t.is_contiguous() or t.dtype != dt or
                              t.get_device() != p.device):
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected a "
                             f"contiguous {dt} tensor of {n} elements on cuda:{p.device}")
    if ws.get_device() != p.device or not ws.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{p.device}, got one "
                         f"on {ws.device}")


def attn_paged_fwd(p, o, lse, ws, stream=None):
    """Enqueue the attention over the cache on `stream` (default: torch's
    current stream).  o: [tokens, Hq, d_v]; lse: fp32 [Hq, tokens] or None;
    both contiguous, as is ws, and all on the block's device."""
    import torch

    _on_device(p)
    want = torch.bfloat16 if p.dtype == DTYPES["bf16"] else torch.float16
    _check_outputs(p, o, lse, ws, want, p.num_tokens * p.Hq * p.d_v, p.num_tokens * p.Hq)
    s = load_library().attn_paged_fwd(ctypes.byref(p), _ptr(o), _ptr(lse), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream))
    if s != 0:
        raise AttnError(s, "attn_paged_fwd")


def _check_tables(rope_cos, rope_sin):
    if rope_cos.dim() != 2 or rope_cos.shape != rope_sin.shape:
        raise ValueError("rope_cos, rope_sin: [rope_len, rot_dim / 2]")


def make_rope_table_params(*, cos, sin, base=10000.0, scaling="NONE", factor=1.0, trained_len=1,
                           turns=(1.0, 32.0), magnitude=1.0):
    """Fill an ``attn_rope_table_params_t`` (see attn.h).  cos, sin: fp32
    [rope_len, rot_dim / 2], which ``attn_rope_table`` fills; scaling: "NONE",
    "LINEAR", "BASE" or "TURNS", with its factor (and, for "TURNS", the trained
    length and the turns between which frequencies go from stretched to kept, linearly
    in the turns and not in the pair's index)."""
    import torch

    given = dict(rope_cos=cos, rope_sin=sin)
    _check_types(given, dict.fromkeys(given, torch.float32))
    _check_tables(cos, sin)
    _check_contiguous(given, given)
    p = attn_rope_table_params_t()
    p.tensors, p.device = given, _one_device(given).index
    p.struct_version = ATTN_ROPE_TABLE_PARAMS_VERSION
    p.scaling = ROPE_SCALINGS[scaling]
    p.rope_len, p.rot_dim = int(cos.shape[0]), 2 * int(cos.shape[1])
    p.base, p.factor, p.magnitude = float(base), float(factor), float(magnitude)
    p.trained_len = int(trained_len)
    p.turns_low, p.turns_high = (float(x) for x in turns)
    p.rope_cos, p.rope_sin = _ptr(cos), _ptr(sin)
    return p


def _fill_places(p, given, tokens, seq_len):
    """Positions, tables and status of a block that turns packed tokens."""
    pos, cu = given["positions"], given["cu_seqlens"]
    if pos is not None and cu is not None:
        raise ValueError("positions and cu_seqlens: one of the two")
    if pos is not None and tuple(pos.shape) != (tokens,):
        raise ValueError("positions: [tokens]")
    if cu is not None and (cu.dim() != 1 or cu.shape[0] < 1):
        raise ValueError("cu_seqlens: [num_segments + 1]")
    _check_contiguous(given, ("positions", "cu_seqlens", "rope_cos", "rope_sin"))
    _check_tables(given["rope_cos"], given["rope_sin"])
    p.num_tokens = tokens
    p.seq_len = max(1, tokens) if seq_len is None else int(seq_len)
    p.num_segments = 0 if cu is None else int(cu.shape[0]) - 1
    p.rope_len = int(given["rope_cos"].shape[0])
    for name in ("positions", "cu_seqlens", "rope_cos", "rope_sin", "status"):
        setattr(p, name, _ptr(given[name]))


def make_rope_params(*, dtype, rope_cos, rope_sin, q=None, k=None, q_out=None, k_out=None,
                     positions=None, cu_seqlens=None, seq_len=None, rot_start=0,
                     interleaved=False, inverse=False, status=None):
    """Fill an ``attn_rope_params_t`` from tensors (see attn.h).  q [tokens, Hq,
    d] and k [tokens, Hkv, d]: rows may lie apart (slices of a packed layout); one
    of them may be None; q_out, k_out: None turns in place; rope_cos, rope_sin: fp32 [rope_len,
    rot_dim / 2]; positions int32 [tokens], or cu_seqlens int32 [segments + 1], or
    rows of seq_len tokens (None: one row).  The block keeps the tensors alive."""
    import torch

    if q is None and k is None:
        raise ValueError("neither q nor k is given")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    given = dict(q=q, k=k, q_out=q_out, k_out=k_out, rope_cos=rope_cos, rope_sin=rope_sin,
                 positions=positions, cu_seqlens=cu_seqlens, status=status)
    e16, f32, i32 = _elem16(dtype), torch.float32, torch.int32
    _check_types(given, dict(q=e16, k=e16, q_out=e16, k_out=e16, rope_cos=f32, rope_sin=f32,
                             positions=i32, cu_seqlens=i32, status=i32))
    p = attn_rope_params_t()
    p.tensors, p.device = given, _one_device(given).index
    p.struct_version, p.dtype = ATTN_ROPE_PARAMS_VERSION, DTYPES[dtype]
    rows = q if q is not None else k
    if rows.dim() != 3:
        raise ValueError("q, k: [tokens, heads, d]")
    tokens, d = int(rows.shape[0]), int(rows.shape[2])
    _fill_places(p, given, tokens, seq_len)
    p.d, p.rot_start, p.rot_dim = d, int(rot_start), 2 * int(rope_cos.shape[1])
    p.rot_interleaved, p.inverse = int(bool(interleaved)), int(bool(inverse))
    for heads, names in (("Hq", ("q", "q_out")), ("Hkv", ("k", "k_out"))):
        t = given[names[0]]
        if t is None:
            continue
        h = int(t.shape[1])
        setattr(p, heads, h)
        for name in names:
            if given[name].shape[0] != tokens:
                raise ValueError(f"{name}: {given[name].shape[0]} rows, expected {tokens}")
            setattr(p, name + "_stride", _rows(name, given[name], h, d))
            setattr(p, name, _ptr(given[name]))
    return p


def make_latent_expand_params(*, dtype, kv, k_rope, k, v, rope_cos, rope_sin, positions=None,
                              cu_seqlens=None, seq_len=None, interleaved=False, status=None):
    """Fill an ``attn_latent_expand_params_t`` from tensors (see attn.h): kv
    [tokens, H, d_n + d_v], k_rope [tokens, d_r], k [tokens, H, d_n + d_r], v
    [tokens, H, d_v]; ``attn_latent_expand`` reads the first two and writes the
    others, ``attn_latent_expand_bwd`` takes gradients the other way.  Positions
    as in ``make_rope_params``.  The block keeps the tensors alive."""
    import torch

    given = dict(kv=kv, k_rope=k_rope, k=k, v=v, rope_cos=rope_cos, rope_sin=rope_sin,
                 positions=positions, cu_seqlens=cu_seqlens, status=status)
    e16, f32, i32 = _elem16(dtype), torch.float32, torch.int32
    _check_types(given, dict(kv=e16, k_rope=e16, k=e16, v=e16, rope_cos=f32, rope_sin=f32,
                             positions=i32, cu_seqlens=i32, status=i32))
    p = attn_latent_expand_params_t()
    p.tensors, p.device = given, _one_device(given).index
    p.struct_version, p.dtype = ATTN_LATENT_EXPAND_PARAMS_VERSION, DTYPES[dtype]
    if kv.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k_rope.dim() != 2:
        raise ValueError("kv, k, v: [tokens, H, dim]; k_rope: [tokens, d_r]")
    tokens, H = int(kv.shape[0]), int(kv.shape[1])
    d_r, d_v = int(k_rope.shape[1]), int(v.shape[2])
    d_n = int(k.shape[2]) - d_r
    _fill_places(p, given, tokens, seq_len)
    if 2 * rope_cos.shape[1] != d_r:
        raise ValueError("rope_cos, rope_sin: [rope_len, d_r / 2]")
    p.H, p.d_n, p.d_r, p.d_v = H, d_n, d_r, d_v
    p.rot_interleaved = int(bool(interleaved))
    for name, t, h, d in (("kv", kv, H, d_n + d_v), ("k_rope", k_rope.unsqueeze(1), 1, d_r),
                          ("k", k, H, d_n + d_r), ("v", v, H, d_v)):
        if t.shape[0] != tokens:
            raise ValueError(f"{name}: {t.shape[0]} rows, expected {tokens}")
        setattr(p, name + "_stride", _rows(name, t, h, d))
        setattr(p, name, _ptr(t))
    return p


def _heads(name, t, tokens, heads, dim):
    """Strides of tokens and heads of a [tokens, heads, dim] tensor in any order
    of memory with contiguous dims."""
    if tuple(t.shape) != (tokens, heads, dim):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{tokens}, {heads}, {dim}]")
    if t.numel() and t.stride(2) != 1:
        raise ValueError(f"{name}: dims must be contiguous")
    # the stride of an axis of one is never used
    return (t.stride(0) if tokens > 1 else heads * dim), (t.stride(1) if heads > 1 else dim)


def make_latent_params(*, dtype, cache, d_c, page_table, seq_lens, c_new=None, k_rope=None,
                       q_rope=None, q_lat=None, q_rot=None, cu_seqlens_q=None, max_q_len=1,
                       rope_cos=None, rope_sin=None, rope_pos=None, rope_interleaved=False,
                       scale=None, mask="CAUSAL", window_left=None, sink=None, status=None):
    """Fill an ``attn_latent_params_t`` from tensors (see attn.h).

    cache: [num_pages, page_size, d_c + d_r] with contiguous dims; page_table,
    seq_lens, cu_seqlens_q, max_q_len: as in ``make_paged_params``; c_new
    [tokens, d_c], k_rope [tokens, d_r], q_rope [tokens, H, d_r] and the tables
    fp32 [rope_len, d_r / 2] are what ``attn_latent_append`` reads, q_rot [tokens,
    H, d_r] what it writes; q_lat [tokens, H, d_c] and q_rot are what
    ``attn_latent_fwd`` reads, with the softmax scale, which it needs.  The block
    keeps the tensors alive; their contents may change between calls."""
    import torch

    given = dict(cache=cache, page_table=page_table, seq_lens=seq_lens, c_new=c_new,
                 k_rope=k_rope, q_rope=q_rope, q_lat=q_lat, q_rot=q_rot,
                 cu_seqlens_q=cu_seqlens_q, rope_cos=rope_cos, rope_sin=rope_sin,
                 rope_pos=rope_pos, sink=sink, status=status)
    e16, f32, i32 = _elem16(dtype), torch.float32, torch.int32
    _check_types(given, dict(cache=e16, page_table=i32, seq_lens=i32, c_new=e16, k_rope=e16,
                             q_rope=e16, q_lat=e16, q_rot=e16, cu_seqlens_q=i32, rope_cos=f32,
                             rope_sin=f32, rope_pos=i32, sink=f32, status=i32))
    if cache.dim() != 3 or (cache.numel() and cache.stride(2) != 1):
        raise ValueError("cache: [num_pages, page_size, d_c + d_r] with contiguous dims")
    num_pages, page, width = (int(x) for x in cache.shape)
    d_c, d_r = int(d_c), width - int(d_c)
    rows = next((t for t in (q_lat, q_rope, q_rot, c_new) if t is not None), None)
    if rows is None:
        raise ValueError("neither queries nor new tokens are given")
    heads = next((t for t in (q_lat, q_rope, q_rot) if t is not None), None)
    if heads is not None and heads.dim() != 3:
        raise ValueError("q_lat, q_rope, q_rot: [tokens, H, dim]")
    tokens, H = int(rows.shape[0]), 1 if heads is None else int(heads.shape[1])
    num_seqs = int(seq_lens.shape[0])
    if page_table.dim() != 2 or page_table.shape[0] != num_seqs or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table: [num_seqs, max_pages] with contiguous rows")
    if cu_seqlens_q is not None and tuple(cu_seqlens_q.shape) != (num_seqs + 1,):
        raise ValueError("cu_seqlens_q: [num_seqs + 1]")
    _check_contiguous(given, ("seq_lens", "cu_seqlens_q", "rope_cos", "rope_sin", "rope_pos",
                              "sink"))
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin go together")
    p = attn_latent_params_t()
    p.tensors, p.device = given, _one_device(given).index
    p.struct_version, p.dtype, p.mask = ATTN_LATENT_PARAMS_VERSION, DTYPES[dtype], MASKS[mask]
    p.num_seqs, p.num_tokens, p.max_q_len = num_seqs, tokens, int(max_q_len)
    p.H, p.d_c, p.d_r = H, d_c, d_r
    p.page_size, p.num_pages, p.max_pages = page, num_pages, int(page_table.shape[1])
    p.page_table, p.seq_lens, p.cu_seqlens_q = (_ptr(page_table), _ptr(seq_lens),
                                                _ptr(cu_seqlens_q))
    p.table_stride = page_table.stride(0) if num_seqs > 1 else p.max_pages
    p.cache, p.status = _ptr(cache), _ptr(status)
    for i in range(2):  # the stride of an axis of one is never used
        p.cache_stride[i] = cache.stride(i) if cache.shape[i] > 1 else page * width
    for name, t, d in (("c_new", c_new, d_c), ("k_rope", k_rope, d_r)):
        if t is not None:
            if tuple(t.shape) != (tokens, d):
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{tokens}, {d}]")
            setattr(p, name + "_stride", _rows(name, t.unsqueeze(1), 1, d))
            setattr(p, name, _ptr(t))
    for name, t, d in (("q_rope", q_rope, d_r), ("q_lat", q_lat, d_c), ("q_rot", q_rot, d_r)):
        if t is not None:
            field = getattr(p, name + "_stride")
            field[0], field[1] = _heads(name, t, tokens, H, d)
            setattr(p, name, _ptr(t))
    if rope_cos is not None:
        _check_tables(rope_cos, rope_sin)
        if 2 * rope_cos.shape[1] != d_r:
            raise ValueError("rope_cos, rope_sin: [rope_len, d_r / 2]")
        p.rope_len = int(rope_cos.shape[0])
        p.rope_cos, p.rope_sin = _ptr(rope_cos), _ptr(rope_sin)
    if rope_pos is not None and tuple(rope_pos.shape) != (tokens,):
        raise ValueError("rope_pos: [tokens]")
    p.rope_pos = _ptr(rope_pos)
    p.rot_interleaved = int(bool(rope_interleaved))
    p.scale = 0.0 if scale is None else float(scale)
    p.window_left = -1 if window_left is None else int(window_left)
    if sink is not None and tuple(sink.shape) != (H,):
        raise ValueError("sink: [H]")
    p.sink = _ptr(sink)
    return p


def _enqueue(name, p, stream):
    _on_device(p)
    s = getattr(load_library(), name)(ctypes.byref(p), _stream(stream, p.device))
    if s != 0:
        raise AttnError(s, name)


def attn_rope_table(p, stream=None):
    """Enqueue the filling of the tables on `stream` (default: torch's current
    stream), as the other calls of this module do."""
    _enqueue("attn_rope_table", p, stream)


def attn_rope(p, stream=None):
    """Enqueue the rotation of q and k."""
    _enqueue("attn_rope", p, stream)


def attn_latent_expand(p, stream=None):
    """Enqueue the making of K and V from kv and k_rope."""
    _enqueue("attn_latent_expand", p, stream)


def attn_latent_expand_bwd(p, stream=None):
    """Enqueue the gradients of kv and k_rope from those of K and V."""
    _enqueue("attn_latent_expand_bwd", p, stream)


def attn_latent_workspace_size(p):
    return int(load_library().attn_latent_workspace_size(ctypes.byref(p)))


def attn_latent_append(p, stream=None):
    """Enqueue the append to the latent cache."""
    _enqueue("attn_latent_append", p, stream)


def attn_latent_fwd(p, o, lse, ws, stream=None):
    """Enqueue the attention over the latent cache.  o: [tokens, H, d_c]; lse:
    fp32 [H, tokens] or None; both contiguous, as is ws, and all on the block's
    device."""
    import torch

    _on_device(p)
    want = torch.bfloat16 if p.dtype == DTYPES["bf16"] else torch.float16
    _check_outputs(p, o, lse, ws, want, p.num_tokens * p.H * p.d_c, p.num_tokens * p.H)
    s = load_library().attn_latent_fwd(ctypes.byref(p), _ptr(o), _ptr(lse), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream, p.device))
    if s != 0:
        raise AttnError(s, "attn_latent_fwd")


def attn_read_status(ws, stream=None):
    """Synchronise and return (status, attn_stats_t) of the last call on `ws`."""
    st = attn_stats_t()
    s = load_library().attn_read_status(_ptr(ws), _stream(stream), ctypes.byref(st))
    return s, st


class Event:
    """A CUDA timing event owned by this object (created through the library)."""

    def __init__(self):
        h = c_vp()
        s = load_library().attn_event_create(ctypes.byref(h))
        if s != 0:
            raise AttnError(s, "attn_event_create")
        self.handle = h.value

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.attn_event_destroy(self.handle)
            self.handle = None


def attn_event_elapsed_ms(start, end):
    """Milliseconds between two recorded events, or None if either is unrecorded."""
    ms = ctypes.c_float()
    s = load_library().attn_event_elapsed_ms(start.handle, end.handle, ctypes.byref(ms))
    return float(ms.value) if s == 0 else None


def attn_set_trace_events(events):
    """events: None, or a sequence of 2 * len(TRACE_SLOTS) Event objects (or None)
    as (start, end) per slot.  The caller keeps the events alive."""
    lib = load_library()
    if events is None:
        return lib.attn_set_trace_events(None)
    arr = (c_vp * (2 * len(TRACE_SLOTS)))()
    for i, e in enumerate(events):
        arr[i] = None if e is None else c_vp(e.handle)
    s = lib.attn_set_trace_events(arr)
    if s != 0:
        raise AttnError(s, "attn_set_trace_events")
